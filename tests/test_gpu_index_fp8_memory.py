"""DeviceWorkload(index_fp8=True) keeps its index keys once, as codes and scales, and so
does a clone."""
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


def _tensors(dw):
    return {n: t for n, t in vars(dw).items() if isinstance(t, torch.Tensor)}


def test_the_keys_are_kept_once(api):
    from sparse_attention_mla_dsa_gb300 import path, workloads
    wl = workloads.scaled("long", seqs=3, len_div=32)
    T, D = wl.idx_k.shape
    wide, narrow = path.DeviceWorkload(wl), path.DeviceWorkload(wl, index_fp8=True)
    queries = wl.q_idx.size + 4 * wl.q_idx.shape[0] * wl.q_idx.shape[1]     # the step's, as codes and scales
    held = [sum(t.numel() * t.element_size() for t in _tensors(dw).values()) for dw in (wide, narrow)]
    assert held[0] - held[1] == 2 * T * D - T * (D + 4) - queries
    assert wide.input_bytes() - narrow.input_bytes() == 2 * T * D - T * (D + 4)
    twin = narrow.clone()
    assert {n: t.shape for n, t in _tensors(twin).items()} == {n: t.shape for n, t in _tensors(narrow).items()}
    narrow.step()
    twin.step()
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    for n in ("scores", "sel", "out"):
        a, b = getattr(narrow, n), getattr(twin, n)
        if n == "scores":                        # rows are written up to their lengths
            a, b = ([x[r, :int(wl.seq_lens[r])] for r in range(wl.rows)] for x in (a, b))
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        else:
            assert torch.equal(a, b)
