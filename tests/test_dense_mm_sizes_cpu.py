"""dsa_dense_mm_splits at the largest sizes its arguments hold (host arithmetic)."""
import ctypes

import pytest

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def splits():
    from sparse_attention_mla_dsa_gb300 import build
    f = ctypes.CDLL(build.build()).dsa_dense_mm_splits
    f.argtypes, f.restype = [ctypes.c_int32] * 3, ctypes.c_int32
    return f


@pytest.mark.parametrize("n,k,sms", [
    (128, MOST - 7, 152), (1, MOST - 7, 1), (300, MOST - 7, MOST), (MOST, 64, 152), (MOST, MOST - 7, 152),
    (MOST - 127, 8, MOST), (1, 8, MOST), (2 ** 30, 4096, 152), (4096, 1536, 152), (32768, 1536, 152)])
def test_largest(splits, n, k, sms):
    tiles, blocks = -(-n // 128), -(-k // 64)
    want = 1 if tiles >= sms else min(-(-sms // tiles), max(blocks // 4, 1))
    per = -(-blocks // want)
    assert splits(n, k, sms) == -(-blocks // per)
