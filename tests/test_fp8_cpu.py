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


def test_binding_refuses_host_tensors():
    from sparse_attention_mla_dsa_gb300 import api
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.dsa_quantize_fp8(x, torch.zeros((2, 128), dtype=torch.uint8), torch.zeros((2, 1)))
    u = torch.zeros((2, 128), dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.dsa_dense_mm_fp8(u, torch.zeros((2, 1)), u, torch.zeros((1, 1)), torch.zeros((2, 2)))
