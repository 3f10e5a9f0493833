"""The 8-bit quantiser and product at the longest k that their arguments hold: 2^31 - 16
values a row, 2^24 blocks, the last of them 112 long."""
import ctypes

import pytest
import torch

K = 2 ** 31 - 16
BLOCKS = 2 ** 24
UNSUPPORTED = 2


def test_too_many_blocks_are_refused():
    # 128 rows of 2^24 blocks: 2^31 scales, one more than an int32 counts
    from sparse_attention_mla_dsa_gb300 import build
    f = ctypes.CDLL(build.build()).dsa_quantize_fp8
    f.argtypes = [ctypes.c_void_p] + [ctypes.c_int32] * 4 + [ctypes.c_void_p] * 3
    at = 1 << 20                     # a dummy address, not followed
    for rows in (128, 1000, 2 ** 31 - 1):
        for block_rows in (1, 128):
            assert f(at, 0, rows, K, block_rows, at, at, None) == UNSUPPORTED


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


PLACES = [0, 127, 128, 2 ** 30 + 5, K - 113, K - 112, K - 1]    # the last two in the last block


@pytest.mark.gpu
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise(api, block_rows):
    x = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    x[0, PLACES] = torch.tensor([448.0 * 2.0 ** i for i in range(len(PLACES))], dtype=torch.bfloat16, device="cuda")
    codes = torch.full((1, K), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, BLOCKS), device="cuda")
    api.dsa_quantize_fp8(x, codes, scales, block_rows=block_rows)
    torch.cuda.synchronize()
    want = torch.full((BLOCKS,), 2.0 ** -126, device="cuda")
    for i, at in enumerate(PLACES):              # (where two share a block, the larger one comes later)
        want[at // 128] = 2.0 ** i
    assert torch.equal(scales[0], want)
    for i, at in enumerate(PLACES):
        assert int(codes[0, at]) == int((torch.tensor(448.0 * 2.0 ** i) / want[at // 128].cpu()).to(torch.float8_e4m3fn).view(torch.uint8))
    assert int(torch.count_nonzero(codes)) == len(PLACES)


@pytest.mark.gpu
def test_product(api):
    # few values that are not 0, whose sum FP32 holds
    a = torch.zeros((1, K), dtype=torch.uint8, device="cuda")
    b = torch.zeros((1, K), dtype=torch.uint8, device="cuda")
    one, two = 0x38, 0x40                        # E4M3 1 and 2
    a[0, PLACES], b[0, PLACES] = one, two
    sa, sb = torch.ones((1, BLOCKS), device="cuda"), torch.ones((1, BLOCKS), device="cuda")
    for i, at in enumerate(PLACES):
        sa[0, at // 128], sb[0, at // 128] = 2.0 ** i, 0.25
    want = sum(2.0 * float(sa[0, at // 128]) * 0.25 for at in PLACES)
    c = torch.full((1, 1), -1.0, device="cuda")
    api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0 and float(c) == want
