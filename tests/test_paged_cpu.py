"""Row plan and chunk attention without a GPU: argument errors of the C entry
points (returned before any CUDA call), the binding's checks, and the plain
forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged_ref

X = 1 << 20  # a dummy, 256-byte aligned address


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_mla_dsa_gb300 import api, build
    build.build()
    return api.load()


def _plan(**changes):
    from sparse_attention_mla_dsa_gb300 import api
    p = api.Plan()
    for name, kind in api.Plan._fields_:
        setattr(p, name, X if kind is ctypes.c_void_p else 0)
    p.seqs, p.rows, p.max_blocks_per_seq, p.bt_stride, p.row_bt_stride = 2, 4, 8, 8, 8
    p.block_size, p.free_capacity = 64, 16
    for k, v in changes.items():
        setattr(p, k, v)
    return ctypes.byref(p)


@pytest.mark.parametrize("changes, status", [
    *[({n: None}, 1) for n in ("seq_lens", "new_tokens", "held_in", "held_out", "block_table",
                               "free_blocks", "free_in", "free_out", "row_start", "positions",
                               "slots", "row_lens")],
    ({"seqs": 0}, 1), ({"rows": 0}, 1), ({"rows": -1}, 1), ({"max_blocks_per_seq": 0}, 1),
    ({"block_size": 0}, 1), ({"bt_stride": 7}, 1), ({"row_bt_stride": 7}, 1),
    ({"free_capacity": 0}, 1), ({"reserved": 1}, 1),
    ({"seqs": 8193}, 2), ({"rows": 65536}, 2),
    ({"seqs": 8192, "max_blocks_per_seq": 1 << 18, "bt_stride": 1 << 18, "row_bt_stride": 1 << 18}, 2),
    ({"block_size": 1 << 28}, 2),
    *[({n: X + 2}, 1) for n in ("seq_lens", "held_out", "block_table", "free_out", "row_start", "row_table")],
    ({"slots": X + 4}, 1),
])
def test_plan_refusals(lib, changes, status):
    assert lib.dsa_plan_rows(_plan(**changes), None) == status


def test_plan_refuses_served_lengths_off_their_alignment(lib):
    assert lib.dsa_plan_rows(_plan(served_lens=X + 2), None) == 1


@pytest.mark.parametrize("changes", [{"flags": 2}, {"flags": 1 << 31}, {"reserved2": 1}])
def test_plan_refuses_unknown_flags(lib, changes):
    assert lib.dsa_plan_rows(_plan(**changes), None) == 1


def test_plan_without_a_plan(lib):
    assert lib.dsa_plan_rows(None, None) == 1


def _chunk(lib, *, q=X, pool=X, nslots=64, rows=4, heads=64, dim=512, out=X, lse=X, ws=X, wsb=1 << 40, **seq):
    from sparse_attention_mla_dsa_gb300 import api
    s = api.Seqs()
    s.seq_lens = s.row_start = s.block_table = X
    s.max_blocks_per_seq, s.bt_stride, s.block_size, s.seqs = 4, 4, 64, 2
    for k, v in seq.items():
        setattr(s, k, v)
    return lib.dsa_mla_chunk_fp8(ctypes.byref(s), q, pool, nslots, rows, heads, dim, 0.02, 0.06, out,
                                 lse, ws, wsb, None)


@pytest.mark.parametrize("kw, status", [
    ({"q": None}, 1), ({"pool": None}, 1), ({"out": None}, 1), ({"seq_lens": None}, 1),
    ({"row_start": None}, 1), ({"block_table": None}, 1),
    ({"rows": 0}, 1), ({"nslots": 0}, 1), ({"seqs": 0}, 1), ({"block_size": 0}, 1),
    ({"max_blocks_per_seq": 0}, 1), ({"bt_stride": 3}, 1),
    ({"q": X + 8}, 1), ({"pool": X + 8}, 1), ({"out": X + 8}, 1), ({"lse": X + 2}, 1),
    ({"seq_lens": X + 2}, 1), ({"row_start": X + 1}, 1), ({"block_table": X + 3}, 1),
    ({"dim": 576}, 2), ({"heads": 8}, 2), ({"heads": 24}, 2), ({"heads": 4112}, 2),
    ({"rows": 65536}, 2), ({"seqs": 8193}, 2), ({"nslots": 1 << 31}, 2), ({"block_size": 1 << 30}, 2),
])
def test_chunk_refusals(lib, kw, status):
    assert _chunk(lib, **kw) == status


def test_chunk_workspace_of_bad_shapes(lib):
    for rows, heads in ((0, 64), (65536, 64), (4, 0), (4, 24), (4, 4112)):
        assert lib.dsa_chunk_workspace_bytes(rows, heads) == 0


def test_binding_refuses_host_tensors():
    from sparse_attention_mla_dsa_gb300 import api
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.make_seqs(i, torch.zeros(5, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32), 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.make_plan(i, i, i, i, torch.zeros((4, 2), dtype=torch.int32), 64, i, i[:1], i[:2],
                      torch.zeros(5, dtype=torch.int32), i, i.long(), i)


def test_table_strides():
    from sparse_attention_mla_dsa_gb300 import api
    t = torch.zeros((4, 10), dtype=torch.int32)
    assert api._table(t, 4, "t")[1:] == (10, 10)
    assert api._table(t[:, :7], 4, "t")[1:] == (7, 10)
    assert api._table(t[:1, 2:7], 1, "t")[1:] == (5, 5)
    for bad in (t.t(), t[:, ::2], t.long(), t[0], t[:3], t[:, :1].expand(4, 3)):
        with pytest.raises(ValueError):
            api._table(bad, 4, "t")


def test_error_codes_match_the_header():
    import os
    import re

    from sparse_attention_mla_dsa_gb300 import api
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    hdr = open(os.path.join(root, "include", "dsa.h")).read()
    codes = {int(v): n.lower() for n, v in re.findall(r"DSA_DEVERR_(\w+) = (\d+)", hdr)}
    assert codes == api.DEVERR


def test_plain_plan_by_hand():
    # Two requests, pages of 4: the first grows from 4 to 5 tokens, the second
    # ends (its two blocks go back first and are popped first).
    r = paged_ref.plan([5, 0], [1, 0], np.array([1, 2]), np.array([[7, -1], [3, 9]]),
                       np.array([1, 2, 0, 0, 0]), 2, 4, 8)
    assert r["table"].tolist() == [[7, 9], [3, 9]] and r["held"].tolist() == [2, 0]
    assert r["free"] == [1, 2, 3] and r["row_start"] == [0, 1, 1]
    assert (r["positions"], r["slots"], r["row_lens"], r["row_table"]) == ([4], [36], [5], [[7, 9]])


def test_plain_chunk_matches_the_oracle(oracle):
    # One request, every visible token selected: the gather-attend's oracle.
    rng = np.random.default_rng(3)
    L, n, H, block = 37, 3, 16, 8
    pool = rng.integers(0, 120, (64, 512)).astype(np.uint8)
    table = rng.permutation(8).astype(np.int32)[None]
    q = torch.from_numpy(rng.standard_normal((n, H, 512)) * 0.05).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    out, lse = paged_ref.chunk([L], [0, n], table, block, q, pool, 0.02, 0.0625)[:2]
    for i in range(n):
        vis = L - n + i + 1
        sel = np.arange(vis, dtype=np.int32)
        o, e = oracle.mla_decode_row(q[i], pool, table[0], block, vis, sel, 0.02, 0.0625)
        # the oracle takes the scales as fp32 (2^-24 of a logit of up to ~6)
        assert np.allclose(out[i], o, rtol=1e-5, atol=1e-9) and np.allclose(lse[i], e, rtol=0, atol=1e-5)
