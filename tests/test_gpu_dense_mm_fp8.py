"""dsa_dense_mm_fp8 against the product in 64 bits.

Tolerance, with T the sum of the terms' magnitudes and J = ceil(k / 128):
  - a block's 128 exact products: four MMAs of 32 terms and the running sum,
    added with the larger one's last bits (2^-23 of it, cut off, at most): at most
    4 * 33 * 2^-23 < 2^-15 of the block's part of T;
  - the product of two scales (2^-24), its product with the block's sum and the
    addition (one rounding, 2^-24 of the running sum) for each block, and up to
    seven additions of ranges: (J + 8) * 2^-24 of T;
  - a bf16 result: half a step, 2^-8 of it.
"""
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
    api.dsa_get_error(reset=True)
    return api


def _operands(seed, m, n, k, wide=False):
    """Codes and scales: every code but NaN, scales of a checkpoint's size (``wide``:
    over 2^-40 .. 2^40, signs and zeros among them)."""
    rng = np.random.default_rng(seed)
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    a, b = (ref.encode(rng.standard_normal(s) * 60) for s in ((m, k), (n, k)))
    a.flat[:finite.size] = finite[:a.size]
    kb, nb = ref.blocks(k), ref.blocks(n)
    if wide:
        sa, sb = (rng.standard_normal(s) * np.exp2(rng.uniform(-40, 40, s)) for s in ((m, kb), (nb, kb)))
        sa.flat[::7], sb.flat[::5] = 0.0, 0.0
    else:
        sa, sb = (np.exp(rng.standard_normal(s)) * 0.01 for s in ((m, kb), (nb, kb)))
    return a, sa.astype(np.float32), b, sb.astype(np.float32)


def _dev(ops):
    return [torch.from_numpy(x).cuda() for x in ops]


def _run(api, ops, out=torch.float32, guard=256):
    a, sa, b, sb = _dev(ops)
    m, n = a.shape[0], b.shape[0]
    whole = torch.full((m * n + guard,), -77.0, dtype=out, device="cuda")
    c = whole[:m * n].view(m, n)
    c.fill_(float("nan"))
    api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    assert (whole[m * n:] == -77.0).all()
    return c


def _check(api, ops, out=torch.float32):
    c = _run(api, ops, out).double().cpu().numpy()
    want, size = ref.product(*ops)
    tol = (2.0 ** -15 + (ref.blocks(ops[0].shape[1]) + 8) * 2.0 ** -24) * size
    if out is torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    bad = ~(np.abs(c - want) <= tol + 1e-300)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], c[bad][:4], want[bad][:4])


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 128, 128), (1, 2048, 4096), (2, 7, 48), (16, 128, 4096), (17, 129, 144), (31, 300, 272),
    (32, 2048, 1536), (33, 127, 1024), (64, 520, 640), (65, 257, 256), (100, 33, 4112), (128, 128, 128),
    (129, 1000, 400), (200, 96, 8192), (257, 513, 528), (300, 2048, 1536), (777, 1003, 208), (1024, 640, 384),
    (1300, 2056, 272), (1281, 1999, 144), (300, 5200, 528), (2500, 1025, 128), (5000, 520, 48), (70, 20000, 256),
    (65, 4000, 4096), (100, 2500, 8192), (129, 1001, 12304), (400, 1000, 4112), (777, 1003, 4112), (128, 300, 32768)])
def test_matches_64_bits(api, m, n, k, out):
    _check(api, _operands(m + n + k, m, n, k), out)


@pytest.mark.parametrize("m,n,k", [(5, 300, 1040), (90, 400, 1040), (700, 520, 656)])
def test_scales_of_all_sizes(api, m, n, k):
    _check(api, _operands(3, m, n, k, wide=True))


def test_quantised_operands_together(api):
    # the framework's quantiser on both sides, the product of the values against 64 bits
    m, n, k = 150, 200, 1552
    x = torch.randn((m, k), device="cuda").to(torch.bfloat16)
    w = torch.randn((n, k), device="cuda") / k ** 0.5
    a, sa = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty((m, 13), device="cuda")
    b, sb = torch.empty((n, k), dtype=torch.uint8, device="cuda"), torch.empty((2, 13), device="cuda")
    c = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    api.dsa_quantize_fp8(w, b, sb, block_rows=128)
    api.dsa_quantize_fp8(x, a, sa)
    api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    torch.cuda.synchronize()
    want, size = ref.product(*(t.cpu().numpy() for t in (a, sa, b, sb)))
    err = np.abs(c.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * size).all()
    # and against the product of what was quantised: an E4M3 rounding is off by 2^-4 at most on each side,
    # or by half of the smallest code (2^-10) where it is one of the smallest
    x64, w64 = x.double().cpu().numpy(), w.double().cpu().numpy()
    def off(v, s):
        return np.maximum(np.abs(v) * 2.0 ** -4, s.double().cpu().numpy().repeat(128, 1)[:, :k] * 2.0 ** -10)
    ex, ew = off(x64, sa), off(w64, sb.repeat_interleave(128, 0)[:n])
    tol = ex @ np.abs(w64).T + np.abs(x64) @ ew.T + ex @ ew.T + 2.0 ** -7 * size
    assert (np.abs(c.double().cpu().numpy() - x64 @ w64.T) <= tol).all()


def test_integers_are_exact(api):
    # small integers, scales 1: every sum is a whole number below 2^24
    rng = np.random.default_rng(8)
    for m, n, k in ((3, 200, 528), (70, 140, 528), (600, 300, 528)):
        a, b = (ref.encode(rng.integers(-8, 9, s).astype(np.float64)) for s in ((m, k), (n, k)))
        ones = [np.ones((r, ref.blocks(k)), np.float32) for r in (m, ref.blocks(n))]
        c = _run(api, (a, ones[0], b, ones[1])).cpu().numpy()
        assert np.array_equal(c, ref.E4M3[a] @ ref.E4M3[b].T)


@pytest.mark.parametrize("n,k", [(2048, 4096), (128, 1536), (5000, 528), (40000, 272)])
def test_up_to_64_rows_do_not_depend_on_each_other(api, n, k):
    ops = _operands(11, 64, n, k)
    whole = _run(api, ops)
    for m in (1, 2, 15, 16, 17, 32, 33, 63):
        for first in {0, 64 - m}:
            part = (ops[0][first:first + m], ops[1][first:first + m], ops[2], ops[3])
            assert torch.equal(_run(api, part), whole[first:first + m]), (m, first)


@pytest.mark.parametrize("m", [4, 96, 600])
def test_not_a_number_stays_in_its_row_and_column(api, m):
    n, k = 300, 400
    ops = _operands(12, m, n, k)
    clean = _run(api, ops)
    a, b = ops[0].copy(), ops[2].copy()
    a[1, 390], b[77, 5], b[299, 130] = 0x7F, 0xFF, 0x7F
    c = _run(api, (a, ops[1], b, ops[3]))
    nan = torch.zeros_like(c, dtype=torch.bool)
    nan[1], nan[:, 77], nan[:, 299] = True, True, True
    assert torch.equal(torch.isnan(c), nan) and torch.equal(c[~nan], clean[~nan])


def test_what_lies_behind_the_operands_is_not_read(api):
    # rows of NaN codes and scales right behind each operand
    m, n, k = 70, 200, 208
    ops = _operands(13, m, n, k)
    want = _run(api, ops)
    padded = []
    for x in _dev(ops):
        fill = 0x7F if x.dtype is torch.uint8 else float("nan")
        big = torch.full((x.shape[0] + 300, x.shape[1]), fill, dtype=x.dtype, device="cuda")
        big[:x.shape[0]] = x
        padded.append(big[:x.shape[0]])
    c = torch.empty((m, n), device="cuda")
    api.dsa_dense_mm_fp8(*padded, c)
    assert torch.equal(c, want)


@pytest.mark.parametrize("m", [1, 50, 500])
def test_same_call_same_bits_and_replay(api, m):
    a, sa, b, sb = _dev(_operands(14, m, 2000, 2064))
    c = torch.empty((m, 2000), dtype=torch.bfloat16, device="cuda")
    api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    first = c.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    for _ in range(20):
        c.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, first) and api.dsa_get_error(reset=True)[0] == 0


def test_activations_written_by_the_kernel_just_before(api):
    # quantiser and product back to back, the codes poisoned before each pass
    for m in (4, 200):
        x = torch.randn((m, 4096), device="cuda").to(torch.bfloat16)
        _, _, b, sb = _dev(_operands(15, 1, 512, 4096))
        codes, scales = torch.empty((m, 4096), dtype=torch.uint8, device="cuda"), torch.empty((m, 32), device="cuda")
        c = torch.empty((m, 512), device="cuda")
        api.dsa_quantize_fp8(x, codes, scales)
        torch.cuda.synchronize()
        api.dsa_dense_mm_fp8(codes, scales, b, sb, c)
        want = c.clone()
        for _ in range(20):
            codes.fill_(0x7F)
            scales.fill_(float("nan"))
            api.dsa_quantize_fp8(x, codes, scales)
            api.dsa_dense_mm_fp8(codes, scales, b, sb, c)
            assert torch.equal(c, want)


@pytest.mark.parametrize("m,n,k", [(4, 4096, 4096), (200, 4096, 4096), (600, 8192, 1024)])
def test_weight_written_by_the_kernel_just_before(api, m, n, k):
    a, sa, _, _ = _dev(_operands(17, m, n, k))
    ws = [torch.randn((n, k), device="cuda") for _ in range(2)]
    b, sb = torch.empty((n, k), dtype=torch.uint8, device="cuda"), torch.empty((n // 128, k // 128), device="cuda")
    c, want = torch.empty((m, n), device="cuda"), []
    for w in ws:
        api.dsa_quantize_fp8(w, b, sb, block_rows=128)
        torch.cuda.synchronize()
        api.dsa_dense_mm_fp8(a, sa, b, sb, c)
        want.append(c.clone())
    for i in range(20):
        api.dsa_quantize_fp8(ws[i % 2], b, sb, block_rows=128)
        api.dsa_dense_mm_fp8(a, sa, b, sb, c)
        assert torch.equal(c, want[i % 2]), i


def test_two_streams_at_once(api):
    sets = [_dev(_operands(20 + i, m, 1500, 2048)) for i, m in enumerate((8, 300))]
    want = []
    for s in sets:
        c = torch.empty((s[0].shape[0], 1500), device="cuda")
        api.dsa_dense_mm_fp8(*s, c)
        want.append(c)
    streams = [torch.cuda.Stream() for _ in sets]
    got = [torch.empty_like(c) for c in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, stream, c in zip(sets, streams, got):
            api.dsa_dense_mm_fp8(*s, c, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(api):
    a, sa, b, sb = _dev(_operands(16, 4, 200, 256))
    c = torch.empty((4, 200), device="cuda")
    good = dict(a=a, a_scale=sa, b=b, b_scale=sb, c=c)
    for bad in (dict(a=a[:, :128]), dict(a=a.float()), dict(a_scale=sa[:3]), dict(a_scale=sa.double()),
                dict(b_scale=sb[:1]), dict(c=c[:, :199]), dict(c=c.half()), dict(c=c.t()), dict(b=b[:, 0])):
        with pytest.raises(ValueError):
            api.dsa_dense_mm_fp8(**(good | bad))
    with pytest.raises(api.DsaError) as e:
        api.dsa_dense_mm_fp8(a[:, :40].contiguous(), sa[:, :1].contiguous(), b[:, :40].contiguous(),
                             sb[:, :1].contiguous(), c)
    assert e.value.status == 1


@pytest.mark.parametrize("n", [60000, 60001])                # rows of 16 bytes, and not
def test_offsets_past_32_bits(api, n):
    """An output of more than 2^31 elements: its first and last rows against 64 bits."""
    m, k = 40000, 32
    ops = _operands(30, 64, n, k)
    a = np.zeros((m, k), np.uint8)
    sa = np.ones((m, 1), np.float32)
    a[:32], a[-32:], sa[:32], sa[-32:] = ops[0][:32], ops[0][32:], ops[1][:32], ops[1][32:]
    c = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    a, sa, b, sb = _dev((a, sa, *ops[2:]))
    api.dsa_dense_mm_fp8(a, sa, b, sb, c)
    got = torch.cat([c[:32], c[-32:]]).double().cpu().numpy()
    assert not torch.any(c[32:-32] != 0)                     # (NaN is not 0 either)
    del c
    torch.cuda.empty_cache()
    want, size = ref.product(*ops)
    tol = (2.0 ** -15 + 9 * 2.0 ** -24) * size
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-300).all()


@pytest.mark.parametrize("m,n,k", [
    (20, 5120, 2048), (33, 7000, 2064), (7, 12000, 1040), (60, 4608, 912),        # row tiles in 6, 4, 2 and 3 ranges
    (300, 2048, 2048), (65, 1024, 512), (400, 1500, 2320), (90, 1001, 1936)])     # 128 x 128 in 2, 2, 3 and 4
def test_numbers_of_ranges(api, m, n, k):
    _check(api, _operands(m + n, m, n, k))
