"""Plain 64-bit forms of the paged step's operators, for their tests: the row
plan as a loop over the requests, the chunk attention from its definition."""
import numpy as np


def plan(seq_lens, new_tokens, held, table, free, count, block, rows):
    """One step of the bookkeeping, request by request.  Returns a dict of what
    dsa_plan_rows writes (rows past the last are absent) and `errors`, the codes
    it may record."""
    S, width = table.shape
    table, free, held = table.copy(), list(free[:count]), held.copy()
    out = dict(positions=[], slots=[], row_lens=[], row_seq=[], row_table=[])
    start, errors = [0], set()
    need, ok = [], []
    for s in range(S):
        L, n, h = int(seq_lens[s]), int(new_tokens[s]), int(held[s])
        blocks = -(-L // block)
        ok.append(0 <= n <= min(L, rows) and blocks <= width and 0 <= h <= width)
        need.append(blocks)
        if not ok[s]:
            errors.add("seq_len")
    for s in range(S):                                   # what is given back
        if ok[s] and need[s] < held[s]:
            free += [int(b) for b in table[s, need[s]:held[s]]]
            held[s] = need[s]
    wanted, avail = 0, len(free)
    for s in range(S):                                   # what is taken
        L, n = int(seq_lens[s]), int(new_tokens[s])
        live = ok[s]
        if ok[s] and need[s] > held[s]:
            wanted += need[s] - int(held[s])
            for b in range(held[s], need[s]):
                table[s, b] = free.pop() if wanted <= avail else -1
            if wanted <= avail:
                held[s] = need[s]
            else:
                live = False
                errors.add("free")
        places = n if 0 <= n <= rows else 0
        start.append(start[-1] + places)
        for i in range(places):
            pos = L - n + i if live else 0
            out["positions"].append(pos)
            out["slots"].append(int(table[s, pos // block]) * block + pos % block if live else -1)
            out["row_lens"].append(pos + 1 if live else 0)
            out["row_seq"].append(s)
            out["row_table"].append([int(table[s, b]) if live and b < need[s] else -1 for b in range(width)])
    if start[-1] > rows:
        errors.add("rows")
        out = {k: v[:rows] for k, v in out.items()}
    return dict(out, row_start=start, held=held, table=table, free=free, errors=errors)


E4M3 = np.array([(-1.0) ** (c >> 7) * (np.nan if c & 0x7F == 0x7F else
                 (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10))
                 for c in range(256)])


def bf16(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def chunk(seq_lens, row_start, table, block, q_bits, pool, kv_scale, sm_scale):
    """The chunk attention in 64 bits, and what its tolerances are made of; NaN
    where no request has the row.  A token is absent where its block is missing.
      out  [R, H, 512], lse [R, H]
      zmag [R, H]       max_j sum_d |sm_scale q_d K_jd|: conditioning of the logits
      mag  [R, H, 512]  sum_j w_j |K_jd| of the softmax weights w
      tail [R, H]       tokens seen * the largest weight * the largest |K|
      live [R]          whether a request has the row
    """
    R, H, D = q_bits.shape
    out, mag = np.full((R, H, D), np.nan), np.full((R, H, D), np.nan)
    lse, zmag, tail = (np.full((R, H), np.nan) for _ in range(3))
    live = np.zeros(R, bool)
    for s in range(len(seq_lens)):
        L, r0, r1 = int(seq_lens[s]), int(row_start[s]), int(row_start[s + 1])
        n = r1 - r0
        if n <= 0 or r0 < 0 or r1 > R or L < n or L > table.shape[1] * block:
            continue
        j = np.arange(L)
        ids = table[s, j // block].astype(np.int64)
        slot = ids * block + j % block
        there = (ids >= 0) & (slot < pool.shape[0])
        k = np.where(there[:, None], E4M3[pool[np.where(there, slot, 0)]] * kv_scale, 0.0)
        for i in range(n):
            r, vis = r0 + i, np.flatnonzero(there[:L - n + i + 1])
            live[r] = True
            if not len(vis):
                out[r], mag[r], lse[r], zmag[r], tail[r] = 0.0, 0.0, -np.inf, 0.0, 0.0
                continue
            x, kv = bf16(q_bits[r]), k[vis]
            z = sm_scale * (x @ kv.T)
            zmag[r] = (abs(sm_scale) * (np.abs(x) @ np.abs(kv).T)).max(1)
            top = z.max(1, keepdims=True)
            w = np.exp(z - top)
            tot = w.sum(1, keepdims=True)
            w /= tot
            out[r], mag[r] = w @ kv, w @ np.abs(kv)
            lse[r] = (top + np.log(tot))[:, 0]
            tail[r] = len(vis) * w.max(1) * np.abs(kv).max()
    return out, lse, zmag, mag, tail, live


def check_chunk(gpu_out, gpu_lse, ref, tag=""):
    """Compares a result [R, H, 512] float with chunk()'s, rows of a request only.

    An output is rounded once to bf16 (half a step: 2^-8 of itself).  A softmax
    weight p enters the weighted sum as an E4M3 term and an E5M2 term of its
    remainder: the remainder is at most 2^-4 of p (4 significant bits, half a
    step) and its own rounding at most 2^-3 of that (3 bits), 2^-7 in all; below
    E4M3's normal range the remainder alone carries p, to within half of E5M2's
    smallest step, 2^-17, where the largest weight is at least 2^8: 2^-25 of the
    largest weight for each token, and 2^-3 of a weight under 2^-18 of the
    largest (its own share of `tail`).  A logit's error d moves a weight by d and
    the sum by d: 2 d of mag; the logits are FP32 sums of 512 exact products in
    two terms, 8e-6 of their magnitudes (the bound of the gather-attend's tests).
    lse: that error, and the normaliser's FP32 sum and logarithm."""
    out, lse, zmag, mag, tail, live_rows = ref
    g = gpu_out.astype(np.float64)
    for r in np.flatnonzero(live_rows):
        nan = np.isnan(out[r])
        assert np.array_equal(np.isnan(g[r]), nan), f"{tag}: NaN of row {r}"
        small = 2.0 ** -25 + 2.0 ** -3 * 2.0 ** -18
        tol = (2.0 ** -8 * np.abs(out[r]) + (2.0 ** -7 + 2 * 8e-6 * zmag[r][:, None] + 1e-5) * mag[r]
               + small * tail[r][:, None])
        err = np.abs(g[r] - out[r])
        ok = nan | (err <= tol)
        assert ok.all(), f"{tag}: row {r}: {int((~ok).sum())} outputs off, worst {np.nanmax(err / tol):.2f} of the bound"
        if gpu_lse is not None:
            e = lse[r]
            both = np.isneginf(e) & np.isneginf(gpu_lse[r])
            with np.errstate(invalid="ignore"):
                d = np.where(both, 0.0, np.abs(gpu_lse[r] - e))
            lim = 1e-5 + 2e-6 * np.abs(np.where(np.isfinite(e), e, 0)) + 8e-6 * zmag[r]
            assert ((d <= lim) | (np.isnan(e) & np.isnan(gpu_lse[r]))).all(), f"{tag}: lse of row {r}: {d.max()}"
        live = ~nan.any(1)
        if not live.any():
            continue
        rms = np.linalg.norm(g[r][live] - out[r][live]) / max(np.linalg.norm(out[r][live]), 1e-300)
        assert rms <= 4e-3 or not out[r][live].any(), f"{tag}: row {r}: rel-L2 {rms:.2e}"
