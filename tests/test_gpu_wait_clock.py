"""Wait limits and the kernel before.

A call may start while the kernel before it still runs, but how long that takes is
not its waits' concern: with a limit far below the other kernel's time a call must
still end without a timeout, and with its usual bits.  The kernel before is a product
that keeps 80 SMs busy for some 400 us and leaves the others free for CTAs of the
call behind it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

LIMIT_NS = 100_000


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def _codes(*shape):
    return torch.randint(0, 0x7F, shape, dtype=torch.uint8, device="cuda")


def _product(api, m, n, k):
    a, b = _codes(m, k), _codes(n, k)
    sa, sb = torch.rand((m, k // 128), device="cuda"), torch.rand((-(-n // 128), k // 128), device="cuda")
    c = torch.zeros((m, n), device="cuda")
    return c, lambda: api.dsa_dense_mm_fp8(a, sa, b, sb, c)


@pytest.fixture(scope="module")
def busy(api):
    _, call = _product(api, 1280, 2048, 131072)      # 40 tiles of 256 x 256
    call()
    times = []
    for _ in range(3):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        call()
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]) * 1e6)
    assert min(times) > 2.5 * LIMIT_NS
    return call


def _bf16_product(api, m, n, k):
    a, b = (torch.randn((r, k), device="cuda").to(torch.bfloat16) for r in (m, n))
    c = torch.zeros((m, n), device="cuda")
    ws = torch.empty(max(256, api.dsa_dense_mm_workspace_bytes(n, k)), dtype=torch.uint8, device="cuda")
    return c, lambda: api.dsa_dense_mm_bf16(a, b, c, ws)


def _scores(api, lens, per, fp8):
    """Rows of sequences of ``lens`` keys; inputs_early."""
    rows, total, top = len(lens) * per, sum(lens), max(lens)
    seq = torch.tensor([n - per + 1 + i for n in lens for i in range(per)], dtype=torch.int32, device="cuda")
    base = torch.tensor([sum(lens[:i]) for i in range(len(lens))], device="cuda").repeat_interleave(per)
    gate = torch.rand(total, device="cuda").to(torch.bfloat16)
    w = torch.rand((rows, 32), device="cuda")
    out = torch.zeros((rows, top), device="cuda")
    block = (seq, api.make_rows(seq))
    if fp8:
        q, k, ks = _codes(rows, 32, 128), _codes(total, 128), torch.rand(total, device="cuda")
        qs = torch.rand((rows, 32), device="cuda")
        return out, lambda: api.dsa_index_scores_fp8(block[1], q, qs, w, k, ks, gate, base, per, top, out, inputs_early=True)
    q, k = torch.randn((rows, 32, 128), device="cuda"), torch.randn((total, 128), device="cuda").to(torch.bfloat16)
    return out, lambda: api.dsa_index_scores(block[1], q, w, k, gate, base, per, top, out, inputs_early=True)


CALLS = {
    "row tiles": lambda api: _product(api, 4, 2048, 4096),
    "tiles": lambda api: _product(api, 200, 4096, 2048),
    "pairs": lambda api: _product(api, 1280, 2048, 512),
    "bf16 product": lambda api: _bf16_product(api, 4, 2048, 4096),
    "fp8 scores, a few tiles": lambda api: _scores(api, [5000], 1, True),
    "fp8 scores, two tiles of several": lambda api: _scores(api, [60000], 2, True),
    "fp8 scores, one sequence": lambda api: _scores(api, [200000], 2, True),
    "fp8 scores, many sequences": lambda api: _scores(api, [3000 + 97 * i for i in range(40)], 2, True),
    "fp8 scores, short sequences": lambda api: _scores(api, [2 + i % 90 for i in range(900)], 1, True),
    "bf16 scores, a few tiles": lambda api: _scores(api, [5000], 1, False),
    "bf16 scores, two tiles of several": lambda api: _scores(api, [60000], 2, False),
    "bf16 scores, one sequence": lambda api: _scores(api, [200000], 2, False),
    "bf16 scores, many sequences": lambda api: _scores(api, [3000 + 97 * i for i in range(40)], 2, False),
    "bf16 scores, short sequences": lambda api: _scores(api, [2 + i % 90 for i in range(900)], 1, False),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_long_kernel_before_is_not_a_timeout(api, busy, name):
    torch.manual_seed(len(name))
    out, call = CALLS[name](api)
    call()
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    want = out.clone()
    try:
        for _ in range(20):
            out.zero_()
            busy()
            api.dsa_set_wait_limit_ns(LIMIT_NS)       # of the calls from here on
            call()
            api.dsa_set_wait_limit_ns(0)
            torch.cuda.synchronize()
            assert api.dsa_get_error(reset=True)[0] == 0
            assert torch.equal(out, want)
    finally:
        api.dsa_set_wait_limit_ns(0)
