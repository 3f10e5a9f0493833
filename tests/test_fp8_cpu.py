"""The 8-bit operators without a GPU: the tests' own 64-bit forms against the
format's closed forms, and the host's argument checks (which return before any
CUDA call, so the dummy pointers are never followed)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import fp8_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
X = 1 << 20                          # a dummy, aligned address


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_mla_dsa_gb300 import build
    return ctypes.CDLL(build.build())


def _fn(lib, name, args):
    types = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float,
             "u": ctypes.c_uint32}
    f = getattr(lib, name)
    f.argtypes = [types[a] for a in args]
    f.restype = ctypes.c_int
    return f


# ----------------------------------------------------------------------------- the reference itself
def test_encode_inverts_decode_and_rounds_to_even():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    assert np.array_equal(ref.encode(ref.E4M3[codes]), codes)
    mid = (ref.POSITIVE[1:] + ref.POSITIVE[:-1]) / 2              # ties: the even code
    lower = np.arange(126)
    assert np.array_equal(ref.encode(mid), np.where(lower % 2 == 0, lower, lower + 1))
    assert np.array_equal(ref.encode(np.nextafter(mid, np.inf)), lower + 1)
    assert np.array_equal(ref.encode(np.nextafter(mid, 0)), lower)
    assert list(ref.encode(np.array([np.nan, np.inf, -np.inf, 1e9, -0.0]))) == [0x7F, 0x7E, 0xFE, 0x7E, 0x80]


def test_encode_agrees_with_torch_on_floats():
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * 40
    t = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x.astype(np.float64)), t)


def test_scale_is_the_smallest_power_of_two():
    for top in (0.0, 1e-45, 2.0 ** -120, 0.3, 447.9, 448.0, np.nextafter(np.float32(448), np.float32(449)), 3.4e38):
        s = ref.pow2_scale(top)
        assert s >= 2.0 ** -126 and np.log2(s) == np.round(np.log2(s))
        assert top <= 448 * s and (s == 2.0 ** -126 or top > 448 * s / 2)


# ----------------------------------------------------------------------------- refusals
def test_quantize_refusals(lib):
    f = _fn(lib, "dsa_quantize_fp8", "piiiippp")
    assert f(None, 0, 4, 128, 1, X, X, None) == INVALID
    assert f(X, 0, 4, 128, 1, None, X, None) == INVALID
    assert f(X, 0, 4, 128, 1, X, None, None) == INVALID
    assert f(X, 2, 4, 128, 1, X, X, None) == INVALID              # type flag
    assert f(X, 0, 0, 128, 1, X, X, None) == INVALID              # no rows
    assert f(X, 0, 4, 0, 1, X, X, None) == INVALID
    assert f(X, 0, 4, 24, 1, X, X, None) == INVALID               # k not a multiple of 16
    assert f(X, 0, 4, 128, 64, X, X, None) == INVALID             # block rows
    assert f(X + 8, 0, 4, 128, 1, X, X, None) == INVALID          # alignment
    assert f(X, 0, 4, 128, 1, X + 4, X, None) == INVALID
    assert f(X, 0, 4, 128, 1, X, X + 2, None) == INVALID
    assert f(X, 0, 2 ** 31 - 1, 144, 1, X, X, None) == UNSUPPORTED
    assert f(X, 0, 65535 * 128 + 1, 128, 128, X, X, None) == UNSUPPORTED


def test_dense_mm_refusals(lib):
    f = _fn(lib, "dsa_dense_mm_fp8", "pppppiiiip")
    good = [X, X, X, X, X, 4, 256, 512, 0, None]
    for i in range(5):
        assert f(*(good[:i] + [None] + good[i + 1:])) == INVALID
    for i, v in ((5, 0), (6, 0), (7, 0), (7, 24), (8, 2)):        # rows, columns, k, k % 16, type flag
        assert f(*(good[:i] + [v] + good[i + 1:])) == INVALID
    for i, off in ((0, 8), (2, 8), (4, 8), (1, 2), (3, 2)):       # alignment
        assert f(*(good[:i] + [X + off] + good[i + 1:])) == INVALID
    assert f(*(good[:5] + [65536] + good[6:])) == UNSUPPORTED
    assert f(*(good[:6] + [65535 * 128 + 1] + good[7:])) == UNSUPPORTED


class _Rows(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32),
                ("bt_stride", ctypes.c_int32), ("block_size", ctypes.c_int32), ("rows", ctypes.c_int32)]


def _all_refused(f, good, bads):
    for at, v, want in bads:
        args = list(good)
        args[at] = v
        assert f(*args) == want, (at, v)


def test_indexer_write_refusals(lib):
    f = _fn(lib, "dsa_indexer_write_fp8", "ppppfppppplipip")
    rows = _Rows(X, None, X, None, 0, 0, 0, 6)
    good = [ctypes.byref(rows), X, X, X, 1e-6, X, X, X, X, X, 1000, 128, X, 2, None]
    _all_refused(f, good, [(i, None, INVALID) for i in (0, 1, 2, 3, 6, 7, 8, 9)]
                 + [(4, -1.0, INVALID), (4, float("nan"), INVALID), (10, 0, INVALID), (13, 4, INVALID),
                    (13, 0, INVALID), (13, 33, INVALID), (11, 96, UNSUPPORTED)]
                 + [(1, X + 4, INVALID), (2, X + 2, INVALID), (7, X + 2, INVALID), (8, X + 1, INVALID),
                    (6, X + 4, INVALID), (12, X + 2, INVALID)])
    _all_refused(f, good, [(0, ctypes.byref(_Rows(None, None, X, None, 0, 0, 0, 6)), INVALID),
                           (0, ctypes.byref(_Rows(X, None, X, None, 0, 0, 0, 0)), INVALID),
                           (0, ctypes.byref(_Rows(X, None, X, None, 0, 0, 0, 65536)), UNSUPPORTED)])


def test_index_scores_refusals(lib):
    f = _fn(lib, "dsa_index_scores_fp8", "ppppppplpiiiippup")
    rows = _Rows(None, None, X, None, 0, 0, 0, 6)
    good = [ctypes.byref(rows), X, X, X, X, X, X, 1000, X, 32, 128, 2, 500, X, X, 0, None]
    _all_refused(f, good, [(i, None, INVALID) for i in (0, 1, 2, 3, 4, 5, 8, 13)]
                 + [(7, 0, INVALID), (11, 4, INVALID), (11, 0, INVALID), (12, -1, INVALID), (15, 2, INVALID),
                    (9, 0, UNSUPPORTED), (9, 257, UNSUPPORTED), (10, 32, UNSUPPORTED), (7, 2 ** 31, UNSUPPORTED)]
                 + [(1, X + 8, INVALID), (4, X + 8, INVALID), (5, X + 2, INVALID), (6, X + 1, INVALID)])
    assert f(*(good[:12] + [0] + good[13:])) == OK                # no tokens: nothing to do


def test_binding_refuses_host_tensors():
    from sparse_attention_mla_dsa_gb300 import api
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.dsa_quantize_fp8(x, torch.zeros((2, 128), dtype=torch.uint8), torch.zeros((2, 1)))
    u = torch.zeros((2, 128), dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.dsa_dense_mm_fp8(u, torch.zeros((2, 1)), u, torch.zeros((1, 1)), torch.zeros((2, 2)))


class _Sized:
    """What the binding looks at before a size is refused."""
    dtype = torch.uint8

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0


def test_binding_refuses_sizes_that_an_argument_does_not_hold(monkeypatch):
    from sparse_attention_mla_dsa_gb300 import api
    monkeypatch.setattr(api, "_current_index", lambda: 0)
    t, much = _Sized(4, 32), 2 ** 32 + 1
    rows = api.Rows()
    rows.rows = 1
    for call in (lambda: api.dsa_quantize_fp8(_Sized(much, 16), t, t),
                 lambda: api.dsa_quantize_fp8(_Sized(1, 2 ** 32 + 16), t, t),
                 lambda: api.dsa_dense_mm_fp8(_Sized(much, 16), t, t, t, t),
                 lambda: api.dsa_dense_mm_fp8(t, t, _Sized(much, 32), t, t),
                 lambda: api.dsa_index_scores_fp8(rows, _Sized(1, 32, 128), t, t, _Sized(9, 128), t, t, t, 1, much, t)):
        with pytest.raises(api.DsaError) as e:
            call()
        assert e.value.status == UNSUPPORTED
