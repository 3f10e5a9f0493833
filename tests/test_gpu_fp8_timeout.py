"""The 8-bit kernels' bounded waits, made to run out on purpose: with the wait
limit at 1 ns each call returns and reports the timeout, and with the limit back
the next one is clean and gives the bits of a call before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def _product(api, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randint(0, 0x7F, (r, k), generator=g, dtype=torch.uint8, device="cuda") for r in (m, n))
    sa, sb = torch.rand((m, k // 128), generator=g, device="cuda"), torch.rand((-(-n // 128), k // 128), generator=g, device="cuda")
    c = torch.empty((m, n), device="cuda")
    return c, lambda: api.dsa_dense_mm_fp8(a, sa, b, sb, c)


def _scores(api, lens, heads):
    g = torch.Generator(device="cuda").manual_seed(2)
    rows, total, top = len(lens), sum(lens), max(lens)
    q = torch.randint(0, 0x7F, (rows, heads, 128), generator=g, dtype=torch.uint8, device="cuda")
    k = torch.randint(0, 0x7F, (total, 128), generator=g, dtype=torch.uint8, device="cuda")
    one = torch.rand((rows, heads), generator=g, device="cuda")
    ks = torch.rand(total, generator=g, device="cuda")
    base = torch.tensor([sum(lens[:i]) for i in range(rows)], device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.zeros((rows, top), device="cuda")
    r = api.make_rows(seq)
    keep = (seq, r)
    return out, lambda: api.dsa_index_scores_fp8(keep[1], q, one, one, k, ks, None, base, 1, top, out)


@pytest.mark.parametrize("make", [
    lambda api: _product(api, 4, 2048, 4096), lambda api: _product(api, 200, 4096, 4096),
    lambda api: _product(api, 700, 8192, 2048), lambda api: _scores(api, [5000], 32),
    lambda api: _scores(api, [3000 + 40 * i for i in range(30)], 64)],
    ids=["row tiles", "tiles", "pairs", "direct", "persistent"])
def test_timeouts_are_reported_and_the_next_call_is_clean(api, make):
    out, call = make(api)
    call()
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    want = out.clone()
    try:
        api.dsa_set_wait_limit_ns(1)
        for _ in range(2):
            call()
            torch.cuda.synchronize()   # the call returns: nothing hangs
            code, _, count = api.dsa_get_error(reset=True)
            assert api.DEVERR[code] == "timeout" and count >= 1
    finally:
        api.dsa_set_wait_limit_ns(0)
    for _ in range(2):
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert api.dsa_get_error(reset=True)[0] == 0 and torch.equal(out, want)
