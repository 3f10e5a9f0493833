"""The paged serving step's operators as they are measured: the row plan made
on the GPU from request lengths (``dsa_plan_rows``) and the dense causal
attention of each request's new tokens over its paged FP8 latent cache
(``dsa_mla_chunk_fp8``).

``own`` picks the side: False computes the plain forms in torch, True makes
the framework's calls.  A case's request lengths follow from the case alone
(``mix`` seeds them); the contents follow from ``prepare``'s seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

LATENT = 512
KV_SCALE = 0.02
SM_SCALE = 256 ** -0.5


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # One request decoding at 32k context: the bookkeeping of one step, pure latency.
        dict(name="plan, one request", op="plan", seqs=1, ctx_lo=32767, ctx_hi=32767, new_lo=1,
             new_hi=1, block=64, max_blocks=513, turnover=0.0, mix=1),
        # A decode batch at 8k to 64k context, a few requests ending or rewound by a rejected verify.
        dict(name="plan, decode batch", op="plan", seqs=32, ctx_lo=8192, ctx_hi=65536, new_lo=1,
             new_hi=1, block=64, max_blocks=1025, turnover=0.1, mix=2),
        # The last 1,024 tokens of a 9,000-token prompt: one request, many rows.
        dict(name="plan, prompt chunk", op="plan", seqs=1, ctx_lo=7976, ctx_hi=7976, new_lo=1024,
             new_hi=1024, block=64, max_blocks=141, turnover=0.0, mix=3),
        # A large mixed batch: 1,000 requests of odd lengths and small pages, decodes and chunks together.
        dict(name="plan, large mix", op="plan", seqs=1000, ctx_lo=1, ctx_hi=16384, new_lo=1, new_hi=64,
             block=16, max_blocks=1031, turnover=0.1, mix=4),
        # The first token of a request at few heads: the smallest call.
        dict(name="attend, first token", op="attend", seqs=1, ctx_lo=0, ctx_hi=0, new_lo=1, new_hi=1,
             heads=16, block=64, mix=5),
        # One request decoding one token at 32k context.
        dict(name="attend, one decode", op="attend", seqs=1, ctx_lo=32767, ctx_hi=32767, new_lo=1,
             new_hi=1, heads=64, block=64, mix=6),
        # A decode batch at 8k to 64k context.
        dict(name="attend, decode batch", op="attend", seqs=32, ctx_lo=8191, ctx_hi=65535, new_lo=1,
             new_hi=1, heads=64, block=64, mix=7),
        # Long-context decode at 128 heads: the most cache read by one call.
        dict(name="attend, long decode", op="attend", seqs=64, ctx_lo=4095, ctx_hi=131071, new_lo=1,
             new_hi=1, heads=128, block=64, mix=8),
        # A four-token verify of eight requests at 64k to 128k context.
        dict(name="attend, verify", op="attend", seqs=8, ctx_lo=65535, ctx_hi=131067, new_lo=4,
             new_hi=4, heads=64, block=64, mix=9),
        # The last 1,024 tokens of a 9,000-token prompt.
        dict(name="attend, prompt chunk", op="attend", seqs=1, ctx_lo=7976, ctx_hi=7976, new_lo=1024,
             new_hi=1024, heads=64, block=64, mix=10),
        # A whole prompt of an odd length at 128 heads, nothing cached before it.
        dict(name="attend, whole prompt", op="attend", seqs=1, ctx_lo=0, ctx_hi=0, new_lo=2049,
             new_hi=2049, heads=128, block=64, mix=11),
        # Chunks and decodes of 24 requests together: odd lengths, 48 heads, pages of 20 tokens.
        dict(name="attend, ragged mix", op="attend", seqs=24, ctx_lo=1, ctx_hi=12000, new_lo=1,
             new_hi=200, heads=48, block=20, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        mix = rng.randrange(1 << 30)
        seqs = _log(rng, 1, 1000)
        ctx_hi = _log(rng, 1, 131071)
        new_hi = _log(rng, 1, 2048)
        block = rng.choice([1, 5, 8, 16, 20, 32, 48, 64, 64, 64, 100, 128])
        case = dict(op=rng.choice(["plan", "attend", "attend"]), seqs=seqs,
                    ctx_lo=rng.choice([0, 1, ctx_hi // 8, ctx_hi]), ctx_hi=ctx_hi,
                    new_lo=rng.choice([1, new_hi]), new_hi=new_hi, block=block, mix=mix)
        need = -(-(ctx_hi + new_hi) // block)
        if case["op"] == "plan":
            case.update(max_blocks=need + rng.randrange(1, 40),
                        turnover=rng.choice([0.0, 0.1, 0.3]) if seqs >= 8 else 0.0)
            rows = sum(n for _, n in _previous(case)[1])
            if not 0 < rows <= 16384 or rows * case["max_blocks"] > 12_000_000 or seqs * need > 2_000_000:
                continue
        else:
            case.update(heads=rng.choice([16, 32, 48, 64, 64, 80, 128]))
            lens = _lengths(case)
            rows = sum(n for _, n in lens)
            top_l, top_n = max(c + n for c, n in lens), max(n for _, n in lens)
            # no more than the largest listed case, padded (the plain form) or not
            if (not 0 < rows <= 8192 or seqs * top_l > 5_000_000
                    or seqs * top_n * case["heads"] * top_l > 1_000_000_000
                    or work(case)["flops"] > 1.0e12):
                continue
        return case


def _lengths(case):
    """[(cached tokens, new tokens)] of the case's requests: spread over the
    logarithm of the range, one in eight of a larger batch without new tokens."""
    rng = random.Random(case["mix"])
    out = []
    for s in range(case["seqs"]):
        ctx = _log(rng, case["ctx_lo"] + 1, case["ctx_hi"] + 1) - 1
        new = _log(rng, case["new_lo"], case["new_hi"])
        if case["seqs"] >= 16 and case["new_hi"] > 1 and s % 8 == 5:
            new = 0
        out.append((ctx, new))
    return out


def _previous(case):
    """Blocks that each request of a plan case holds before the step, and the
    requests' lengths after it.  ``turnover`` of them end (length 0) and as many
    hold a block or two more than they need (tokens a verify rejected)."""
    rng = random.Random(case["mix"] + 1)
    block, held, lens = case["block"], [], []
    for ctx, new in _lengths(case):
        have = -(-ctx // block)
        u = rng.random()
        if u < case["turnover"]:
            ctx, new = 0, 0
        elif u < 2 * case["turnover"]:
            have = min(case["max_blocks"], -(-(ctx + new) // block) + rng.randrange(1, 3))
        held.append(have)
        lens.append((ctx + new, new))
    return held, lens


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_plan if case["op"] == "plan" else _prepare_attend)(case, g)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _prepare_plan(case, g):
    held, lens = _previous(case)
    seqs, width = case["seqs"], case["max_blocks"]
    want = sum(max(0, -(-n // case["block"]) - h) for (n, _), h in zip(lens, held))
    total = sum(held) + want + 64
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    have = _int(held)
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(have, 0) - have)[:, None] + col
    table = torch.where(col < have[:, None], ids[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    free[:total - sum(held)] = ids[sum(held):]
    rows = sum(n for _, n in lens)
    st = dict(op="plan", block=case["block"], seq_lens=_int([n for n, _ in lens]),
              new_tokens=_int([n for _, n in lens]), held=have, table=table, free=free,
              free_count=_int([total - sum(held)]), rows=rows,
              held_out=torch.zeros(seqs, dtype=torch.int32, device="cuda"),
              free_out=torch.zeros(2, dtype=torch.int32, device="cuda"),
              row_start=torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"),
              positions=torch.zeros(rows, dtype=torch.int32, device="cuda"),
              slots=torch.zeros(rows, dtype=torch.int64, device="cuda"),
              row_lens=torch.zeros(rows, dtype=torch.int32, device="cuda"),
              row_seq=torch.zeros(rows, dtype=torch.int32, device="cuda"),
              row_table=torch.zeros((rows, width), dtype=torch.int32, device="cuda"))
    if own:  # the argument block that a server builds once over its buffers
        from sparse_attention_mla_dsa_gb300 import api
        st["plan"] = api.make_plan(st["seq_lens"], st["new_tokens"], st["held"], st["held_out"],
                                   st["table"], st["block"], st["free"], st["free_count"],
                                   st["free_out"], st["row_start"], st["positions"], st["slots"],
                                   st["row_lens"], st["row_table"], st["row_seq"])
    return st


def _prepare_attend(case, g):
    lens = _lengths(case)
    block, heads = case["block"], case["heads"]
    blocks = [-(-(c + n) // block) for c, n in lens]
    total, width = sum(blocks) + 8, max(1, max(blocks))
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    have = _int(blocks)
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(have, 0) - have)[:, None] + col
    table = torch.where(col < have[:, None], ids[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    slots = total * block
    pool = torch.empty((slots, LATENT), dtype=torch.uint8, device="cuda")
    for lo in range(0, slots, 1 << 20):      # normalised latents, stored as the latent write stores them
        n = min(1 << 20, slots - lo)
        x = torch.randn((n, LATENT), generator=g, device="cuda") * (1.0 / KV_SCALE)
        pool[lo:lo + n] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    rows = sum(n for _, n in lens)
    q = (0.05 * torch.randn((rows, heads, LATENT), generator=g, device="cuda")).to(torch.bfloat16)
    new = [n for _, n in lens]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    seq_of = [s for s, n in enumerate(new) for _ in range(n)]
    place = [i for n in new for i in range(n)]
    st = dict(op="attend", block=block, max_new=max(new), max_len=max(c + n for c, n in lens),
              seq_lens=_int([c + n for c, n in lens]), new=_int(new), row_start=_int(starts),
              seq_of=_int(seq_of, torch.int64), place=_int(place, torch.int64), table=table, pool=pool, q=q,
              out=torch.zeros_like(q), lse=torch.zeros((rows, heads), dtype=torch.float32, device="cuda"))
    if own:  # what a server keeps: the argument block over its buffers, and the workspace
        from sparse_attention_mla_dsa_gb300 import api
        st["seqs"] = api.make_seqs(st["seq_lens"], st["row_start"], st["table"], st["block"])
        st["workspace"] = torch.empty(api.dsa_chunk_workspace_bytes(rows, heads), dtype=torch.uint8,
                                      device="cuda")
    return st


# ---------------------------------------------------------------------------- one pass
def run(st):
    if st["op"] == "plan":
        return _own_plan(st) if own else _plain_plan(st)
    return _own_attend(st) if own else _plain_attend(st)


def _own_plan(st):
    from sparse_attention_mla_dsa_gb300 import api
    api.dsa_plan_rows(st["plan"])
    return {k: st[k] for k in ("row_start", "positions", "slots", "row_lens", "row_seq", "row_table",
                               "held_out", "table", "free")} | {"free_count": st["free_out"][:1]}


def _own_attend(st):
    from sparse_attention_mla_dsa_gb300 import api
    api.dsa_mla_chunk_fp8(st["seqs"], st["q"], st["pool"], KV_SCALE, SM_SCALE, st["out"], st["lse"],
                          st["workspace"])
    return {"out": st["out"], "lse": st["lse"]}


def _plain_plan(st):
    """Blocks wanted and given back per request, the popped ids, the rows."""
    block, table, free = st["block"], st["table"], st["free"]
    lens, new, held = st["seq_lens"].long(), st["new_tokens"].long(), st["held"].long()
    count = st["free_count"].long()
    seqs, width = table.shape
    need = (lens + block - 1) // block
    want, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    upto, back_upto = torch.cumsum(want, 0), torch.cumsum(back, 0)
    avail = count + back_upto[-1:]
    granted = (upto <= avail) | (want == 0)
    taken = torch.where(upto <= avail, upto, 0).amax()
    col = torch.arange(width, device="cuda")
    # the free ids with the returned ones above them, the last one popped first
    i = torch.arange(free.shape[0], device="cuda")
    src = torch.searchsorted(back_upto, (i - count).clamp(min=0), right=True).clamp(max=seqs - 1)
    ret = table[src, (need[src] + (i - count) - (back_upto - back)[src]).clamp(0, width - 1)]
    stack = torch.where((i >= count) & (i < avail), ret, free)
    pop = (avail - 1 - ((upto - want)[:, None] + col - held[:, None])).clamp(0, free.shape[0] - 1)
    fresh = (col >= held[:, None]) & (col < need[:, None])
    table = torch.where(fresh, torch.where(granted[:, None], stack[pop], -1), table)
    after = avail - taken
    free = torch.where((i >= count) & (i < after), stack, free)
    held = torch.where(granted, need, held)
    row_start = torch.zeros(seqs + 1, dtype=torch.int64, device="cuda")
    row_start[1:] = torch.cumsum(new, 0)
    row = torch.arange(st["rows"], device="cuda")
    s = torch.searchsorted(row_start[1:], row, right=True)
    pos = lens[s] - new[s] + row - row_start[s]
    ok = granted[s]
    slot = table[s, (pos // block).clamp(0, width - 1)].long() * block + pos % block
    row_table = torch.where((col < need[s][:, None]) & ok[:, None], table[s], -1)
    return {"row_start": row_start.int(), "positions": torch.where(ok, pos, 0).int(),
            "slots": torch.where(ok, slot, -1), "row_lens": torch.where(ok, pos + 1, 0).int(),
            "row_seq": s.int(), "row_table": row_table, "held_out": held.int(), "table": table,
            "free": free, "free_count": after.int()}


def _plain_attend(st):
    """softmax(sm_scale * q K^T) K per request under the causal mask, on
    sequences and chunks padded to the longest, in 32 bits."""
    block, heads = st["block"], st["q"].shape[1]
    j = torch.arange(st["max_len"], device="cuda")
    there = j < st["seq_lens"][:, None]
    slot = st["table"][:, j // block].long() * block + j % block
    k = st["pool"].view(torch.float8_e4m3fn)[torch.where(there, slot, 0)].float() * KV_SCALE
    i = torch.arange(st["max_new"], device="cuda")
    row = (st["row_start"][:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()
    z = st["q"].float()[row].flatten(1, 2) @ k.transpose(1, 2) * SM_SCALE
    seen = j <= (st["seq_lens"] - st["new"])[:, None, None] + i[:, None]
    seen = (seen & there[:, None]).repeat_interleave(heads, 1)
    z = z.masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = (z - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ k) / total
    lse = (top + total.log())[..., 0]
    out = out.unflatten(1, (st["max_new"], heads))[st["seq_of"], st["place"]]
    lse = lse.unflatten(1, (st["max_new"], heads))[st["seq_of"], st["place"]]
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ---------------------------------------------------------------------------- measures
def work(case):
    if case["op"] == "plan":
        held, lens = _previous(case)
        rows, seqs = sum(n for _, n in lens), case["seqs"]
        need = [-(-n // case["block"]) for n, _ in lens]
        moved = sum(abs(n - h) for n, h in zip(need, held))
        tables = sum(min(n, h) for n, h in zip(need, held))
        return {"bytes": 4 * (3 * seqs + tables + 2 * moved) + 4 * (2 * seqs + 2)
                + rows * (4 + 8 + 4 + 4 + 4 * case["max_blocks"]), "flops": rows * case["max_blocks"]}
    lens, heads = _lengths(case), case["heads"]
    rows = sum(n for _, n in lens)
    seen = sum(n * c + n * (n + 1) // 2 for c, n in lens)
    read = sum(c + n for c, n in lens if n)
    return {"bytes": read * LATENT + 2 * rows * heads * LATENT * 2 + rows * heads * 4
            + 4 * sum(-(-(c + n) // case["block"]) for c, n in lens if n),
            "flops": 4 * LATENT * heads * seen}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    heads = case["heads"]
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    outs, lses, first = [], [], 0
    for s, (ctx, new) in enumerate(_lengths(case)):
        n = ctx + new
        if not new:
            continue
        j = torch.arange(n, device="cuda")
        slot = st["table"][s].long().repeat_interleave(case["block"])[:n] * case["block"] + j % case["block"]
        k = codes[st["pool"][slot].long()] * KV_SCALE
        step = max(1, (1 << 28) // (n * heads))
        for lo in range(0, new, step):
            hi = min(new, lo + step)
            q = st["q"][first + lo:first + hi].double()
            z = torch.einsum("rhd,jd->rhj", q, k) * SM_SCALE
            i = torch.arange(lo, hi, device="cuda")[:, None, None]
            z[(j > ctx + i).expand_as(z)] = -math.inf
            lse = torch.logsumexp(z, -1)
            outs.append(torch.einsum("rhj,jd->rhd", (z - lse[..., None]).exp(), k))
            lses.append(lse)
        first += new
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
