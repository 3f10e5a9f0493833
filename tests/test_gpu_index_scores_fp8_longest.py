"""dsa_index_scores_fp8 over the longest sequences that a length holds, 2^31 - 1 tokens and
some fewer (155 GB on the device)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1
NEED = 165 << 30


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def test_longest(api):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < NEED:
        pytest.skip("needs 165 GB of device memory")
    H, D = 16, 64
    k = torch.zeros((MOST, D), dtype=torch.uint8, device="cuda")
    ks = torch.zeros(MOST, device="cuda")
    scores = torch.empty((1, MOST), device="cuda")
    one = 0x38                                   # E4M3 1
    q = torch.full((1, H, D), one, dtype=torch.uint8, device="cuda")
    qs, w = torch.ones((1, H), device="cuda"), torch.ones((1, H), device="cuda")
    base = torch.zeros(1, dtype=torch.int64, device="cuda")
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = api.make_rows(seq)
    try:
        for n in (MOST, MOST - 126, MOST - 127, MOST - 128):
            places = [0, 1, 127, 128, 2 ** 30, n - 129, n - 128, n - 127, n - 1]
            for i, at in enumerate(places):      # D products of 1, in H heads, times the key's scale
                k[at] = one
                ks[at] = 2.0 ** i
            seq.fill_(n)
            scores.fill_(-1.0)
            api.dsa_index_scores_fp8(rows, q, qs, w, k, ks, None, base, 1, MOST, scores)
            torch.cuda.synchronize()
            assert api.dsa_get_error(reset=True)[0] == 0
            for i, at in enumerate(places):
                assert float(scores[0, at]) == H * D * 2.0 ** i, (n, at)
                scores[0, at] = 0.0
                k[at] = 0
                ks[at] = 0.0
            assert not scores[0, :n].any() and (scores[0, n:] == -1.0).all()
    finally:
        del k, ks, scores
        torch.cuda.empty_cache()
