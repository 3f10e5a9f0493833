"""dsa_quantize_fp8 against the 64-bit form: codes and scales exactly equal
(x / scale is exact and the code is its one rounding)."""
import numpy as np
import pytest
import torch

from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    return api


def _outputs(rows, k, block_rows, guard=64):
    """Buffers with guard bytes behind them."""
    codes = torch.full((rows * k + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    n = -(-rows // block_rows) * ref.blocks(k)
    scales = torch.full((n + guard,), -7.0, device="cuda")
    return codes, codes[:rows * k].view(rows, k), scales, scales[:n].view(-1, ref.blocks(k))


def _check(api, x, block_rows):
    rows, k = x.shape
    all_codes, codes, all_scales, scales = _outputs(rows, k, block_rows)
    api.dsa_quantize_fp8(x, codes, scales, block_rows=block_rows)
    torch.cuda.synchronize()
    want_codes, want_scales = ref.quantize(x.double().cpu().numpy(), block_rows)
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    got = codes.cpu().numpy()
    assert np.array_equal(got, want_codes), np.argwhere(got != want_codes)[:5]
    assert (all_codes[rows * k:] == 0xA5).all() and (all_scales[scales.numel():] == -7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,k", [
    (1, 16), (1, 128), (1, 4096), (3, 144), (7, 112), (127, 272), (128, 128), (129, 1536), (300, 4112), (1000, 256)])
def test_matches_the_formula(api, rows, k, block_rows, dtype):
    g = torch.Generator().manual_seed(rows * 131 + k)
    x = torch.randn((rows, k), generator=g) * torch.randn((rows, 1), generator=g).mul(3).exp()
    _check(api, x.to(dtype).cuda(), block_rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_extreme_values(api, block_rows, dtype):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((12, 384), generator=g)
    x[0] = 0                                               # nothing at all: scale 2^-126
    x[1, 128:256] = 0
    x[2, :128] *= 1e-40                                    # below 2^-126 (subnormal)
    x[3] *= 1e36
    x[4, 7], x[4, 200], x[4, 300] = float("inf"), -float("inf"), float("nan")
    x[5, :128] = float("inf")                              # no finite element
    x[6, 128:256] = float("nan")
    x[7, 0], x[7, 1] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x[8, :128], x[8, 5] = 0, 448.0                         # the borders of the scale
    x[9, :128], x[9, 5] = 0, 450.0
    x[10, :128] = 0
    x[10, 3], x[10, 4], x[10, 5] = 448.0, 2.0 ** -10, 2.0 ** -10 * 1.5   # ties and a rounding at the smallest codes
    x[11, :128] = -0.0
    if block_rows == 128:
        for r in range(12):
            _check(api, x[r:r + 1].to(dtype).cuda(), block_rows)
    else:
        _check(api, x.to(dtype).cuda(), block_rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_tie_rounds_to_even(api, dtype):
    # every midpoint of neighbouring codes and its neighbours in the type, beside a 448 that fixes the scale at 1
    mid = torch.from_numpy((ref.POSITIVE[1:] + ref.POSITIVE[:-1]) / 2).to(dtype)
    bits = torch.int32 if dtype is torch.float32 else torch.int16
    near = torch.cat([mid, (mid.view(bits) + 1).view(dtype), (mid.view(bits) - 1).view(dtype)])
    near = torch.cat([near, -near])
    x = torch.zeros((-(-near.numel() // 100), 128), dtype=dtype)
    for r in range(x.shape[0]):
        part = near[r * 100:(r + 1) * 100]
        x[r, :part.numel()] = part
        x[r, 127] = 448.0
    _check(api, x.cuda(), 1)


def test_values_quantised_again_stay(api):
    x = torch.randn((64, 512), device="cuda").to(torch.bfloat16)
    codes, scales = torch.empty((64, 512), dtype=torch.uint8, device="cuda"), torch.empty((64, 4), device="cuda")
    api.dsa_quantize_fp8(x, codes, scales)
    values = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1)
    api.dsa_quantize_fp8(values, codes, scales)
    assert torch.equal(codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1), values)


def test_queries_and_unaligned_starts(api):
    # [rows, heads, 128]: one scale a head; buffers that start inside others, bf16 bits as int16
    rows, heads = 5, 24
    big = torch.randn((rows * heads * 128 + 8,), device="cuda").to(torch.bfloat16)
    x = big[8:].view(rows, heads, 128)
    codes = torch.empty(rows * heads * 128 + 16, dtype=torch.uint8, device="cuda")[16:].view(rows, heads, 128)
    scales = torch.empty(rows * heads + 1, device="cuda")[1:].view(rows, heads)
    api.dsa_quantize_fp8(x.view(torch.int16), codes, scales)
    want_codes, want_scales = ref.quantize(x.reshape(-1, 128).double().cpu().numpy())
    assert np.array_equal(codes.view(-1, 128).cpu().numpy(), want_codes)
    assert np.array_equal(scales.reshape(-1, 1).cpu().numpy(), want_scales)


def test_offsets_past_32_bits(api):
    # 2^31 elements and some: the last rows' bytes lie past 4 GB in x
    k, rows = 32768, 65536 + 3
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, k), device="cuda").to(torch.bfloat16)
    codes, scales = torch.empty((rows, k), dtype=torch.uint8, device="cuda"), torch.empty((rows, k // 128), device="cuda")
    for tile in (1, 128):
        s = scales if tile == 1 else scales[:-(-rows // 128)]
        api.dsa_quantize_fp8(x, codes, s, block_rows=tile)
        part = x[-3:] if tile == 1 else x[-(rows % 128):]
        want_codes, want_scales = ref.quantize(part.double().cpu().numpy(), tile)
        assert np.array_equal(codes[-part.shape[0]:].cpu().numpy(), want_codes)
        assert np.array_equal(s[-want_scales.shape[0]:].cpu().numpy(), want_scales)


def test_refusals(api):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.zeros((4, 256), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), device="cuda")
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(codes=codes[:3]), dict(codes=codes.short()),
                dict(scales=scales[:, :1]), dict(scales=scales.double()), dict(x=x[:, ::2], codes=codes[:, :128]),
                dict(block_rows=128), dict(x=x.view(2, 2, 256), codes=codes.view(2, 2, 256), block_rows=128)):
        with pytest.raises(ValueError):
            api.dsa_quantize_fp8(**(dict(x=x, codes=codes, scales=scales) | bad))
    with pytest.raises(api.DsaError) as e:
        api.dsa_quantize_fp8(x[:, :24].contiguous(), codes[:, :24].contiguous(), scales[:, :1].contiguous())
    assert e.value.status == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [157, 601, 1501])
def test_more_blocks_at_a_time(api, rows, dtype):
    """Numbers of blocks at which a group of lanes takes one, two and four of them."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, 4112), generator=g) * torch.randn((rows, 1), generator=g).mul(3).exp()
    x[::7, 130], x[3::11, 4100], x[5::13, 1000:1300] = float("inf"), float("nan"), -float("inf")
    _check(api, x.to(dtype).cuda(), 1)


@pytest.mark.parametrize("block_rows", [0, 64, 2])
def test_refused_block_rows(api, block_rows):
    x = torch.zeros((1, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(api.DsaError) as e:
        api.dsa_quantize_fp8(x, torch.zeros((1, 256), dtype=torch.uint8, device="cuda"),
                             torch.zeros((1, 2), device="cuda"), block_rows=block_rows)
    assert e.value.status == 1
