"""Plain 64-bit forms of the 8-bit operators, for their tests: E4M3 from the
format's definition, the block scales, the scaled product, the indexer key's
write and the index scores, in numpy."""
import numpy as np

from tests.paged_ref import E4M3, bf16

BLOCK = 128
# values of the codes 0 .. 126, ascending
POSITIVE = E4M3[:127]


def encode(x):
    """E4M3 codes nearest to x (float64), ties to the even code, saturating."""
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = POSITIVE[hi] - a, a - POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)).astype(np.uint8)


def pow2_scale(top):
    """Smallest power of two, 2^-126 at least, with top <= 448 times it."""
    top = np.asarray(top, np.float64)
    powers = 2.0 ** np.arange(-126, 122)
    return powers[np.searchsorted(448.0 * powers, top)]


def blocks(n):
    return -(-n // BLOCK)


def quantize(x, block_rows=1):
    """(codes, scales) of x [rows, k]."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    scales = np.empty((-(-rows // block_rows), blocks(k)))
    codes = np.empty((rows, k), np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
            part = x[at]
            finite = np.where(np.isfinite(part), np.abs(part), 0.0)
            scales[i, j] = pow2_scale(finite.max())
            codes[at] = encode(part / scales[i, j])
    return codes, scales


def values(codes, scales, block_rows=1):
    """What codes [rows, k] with their scales stand for."""
    rows, k = codes.shape
    s = np.asarray(scales, np.float64).repeat(block_rows, 0)[:rows].repeat(BLOCK, 1)[:, :k]
    return E4M3[codes] * s


def product(a, sa, b, sb):
    """c = (a sa) (b sb)^T and the sum of the terms' magnitudes."""
    x, w = values(a, sa), values(b, sb, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def layer_norm(k_raw, w, b, eps):
    """LayerNorm with bias of bf16 bit patterns [rows, d], in 64 bits."""
    x = bf16(k_raw)
    d = x - x.mean(1, keepdims=True)
    return d / np.sqrt((d * d).mean(1, keepdims=True) + np.float64(np.float32(eps))) * bf16(w) + bf16(b)


def index_scores(q, q_scale, head_w, k, k_scale, gate):
    """Scores of one row against every key: q [H, D] codes, q_scale, head_w [H],
    k [T, D] codes, k_scale [T], gate [T]; and the sum over heads of the terms'
    magnitudes (for tolerances)."""
    x = E4M3[q] * np.asarray(q_scale, np.float64)[:, None]
    y = E4M3[k] * np.asarray(k_scale, np.float64)[:, None]
    w = np.asarray(head_w, np.float64)[:, None]
    g = np.asarray(gate, np.float64)
    dots = x @ y.T
    mags = np.abs(x) @ np.abs(y).T
    return g * (w * np.maximum(dots, 0.0)).sum(0), np.abs(g) * (np.abs(w) * mags).sum(0)
