"""dsa_mla_chunk_fp8 against its definition in 64 bits (tests/paged_ref.py, where
the tolerances are derived)."""
import numpy as np
import pytest
import torch

from tests import paged_ref

pytestmark = pytest.mark.gpu
MARK = 0x4242          # bf16 bits left in rows that must not be written
NAN8 = 0x7F


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16)


class Case:
    """Requests [(tokens cached, tokens new)] over shuffled blocks of a pool
    whose every unused byte is the FP8 NaN."""

    def __init__(self, reqs, heads, block, seed=0, q_scale=0.05, kv_scale=0.02, sm_scale=0.0625,
                 spare_rows=0, spare_blocks=3, stride=0):
        rng = np.random.default_rng(seed)
        self.heads, self.block, self.kv_scale, self.sm_scale = heads, block, kv_scale, sm_scale
        self.lens = np.array([c + n for c, n in reqs], np.int32)
        self.start = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
        self.rows = max(1, int(self.start[-1]) + spare_rows)
        blocks = [-(-int(n) // block) for n in self.lens]
        ids = rng.permutation(sum(blocks) + spare_blocks)
        width = max(1, max(blocks))
        self.table = np.full((len(reqs), width + stride), -1, np.int32)
        self.pool = np.full(((sum(blocks) + spare_blocks) * block, 512), NAN8, np.uint8)
        at = 0
        for s, nb in enumerate(blocks):
            self.table[s, :nb] = ids[at:at + nb]
            at += nb
            n = int(self.lens[s])
            x = torch.from_numpy(rng.standard_normal((n, 512), dtype=np.float32) / np.float32(kv_scale))
            slot = self.table[s, np.arange(n) // block].astype(np.int64) * block + np.arange(n) % block
            self.pool[slot] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.width = width
        self.q = bf16_bits(rng.standard_normal((self.rows, heads, 512)) * q_scale)

    def slot(self, s, j):
        return int(self.table[s, j // self.block]) * self.block + j % self.block

    def upload(self, api):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d_table = d(self.table)
        self.seqs = api.make_seqs(d(self.lens), d(self.start), self.d_table[:, :self.width], self.block)
        self.d_q, self.d_pool = d(self.q.view(np.int16)), d(self.pool)
        self.out = torch.full((self.rows, self.heads, 512), MARK, dtype=torch.int16, device="cuda")
        self.lse = torch.full((self.rows, self.heads), 77.0, device="cuda")
        self.ws = torch.full((api.dsa_chunk_workspace_bytes(self.rows, self.heads),), 0xFF,
                             dtype=torch.uint8, device="cuda")
        return self

    def call(self, api, stream=None, lse=True):
        api.dsa_mla_chunk_fp8(self.seqs, self.d_q, self.d_pool, self.kv_scale, self.sm_scale, self.out,
                              self.lse if lse else None, self.ws, stream)

    def reference(self):
        return paged_ref.chunk(self.lens, self.start, self.table[:, :self.width], self.block, self.q,
                               self.pool, self.kv_scale, self.sm_scale)

    def result(self):
        torch.cuda.synchronize()
        return self.out.view(torch.bfloat16).float().cpu().numpy(), self.lse.cpu().numpy()

    def check(self, api, ref=None, tag="", code=0):
        ref = self.reference() if ref is None else ref
        out, lse = self.result()
        assert api.dsa_get_error(reset=True)[0] == code
        paged_ref.check_chunk(out, lse, ref, tag)
        idle = torch.from_numpy(~ref[5])
        assert (self.out[idle.cuda()] == MARK).all() and (self.lse[idle.cuda()] == 77.0).all(), "an idle row was written"


def run(api, case, **kw):
    case.upload(api).call(api)
    case.check(api, **kw)


@pytest.mark.parametrize("ctx, new", [(0, 1), (1, 1), (62, 1), (63, 1), (127, 1), (128, 1), (255, 1), (256, 1),
                                      (257, 1), (700, 1), (5000, 1), (0, 2), (0, 3), (0, 129), (125, 5),
                                      (254, 3), (255, 130), (1000, 33), (513, 257)])
def test_lengths(api, ctx, new):
    run(api, Case([(ctx, new)], 64, 64, seed=ctx * 7 + new))


@pytest.mark.parametrize("heads", [16, 32, 48, 64, 80, 112, 128, 144, 256])
@pytest.mark.parametrize("new", [1, 7])
def test_head_counts(api, heads, new):
    run(api, Case([(300, new), (0, new), (129, new)], heads, 64, seed=heads))


@pytest.mark.parametrize("block", [1, 2, 3, 4, 5, 7, 8, 12, 16, 20, 24, 32, 48, 64, 96, 100, 128, 192, 256, 1000])
def test_block_sizes(api, block):
    run(api, Case([(333, 3), (64, 1), (0, 70), (block, 1)], 64, block, seed=block))


@pytest.mark.parametrize("seed", range(6))
def test_ragged_batches(api, seed):
    rng = np.random.default_rng(seed)
    reqs = [(int(rng.integers(0, 900)), int(rng.choice([0, 0, 1, 1, 2, 5, 40]))) for _ in range(rng.integers(1, 40))]
    reqs.insert(int(rng.integers(0, len(reqs) + 1)), (0, 0))
    run(api, Case(reqs, int(rng.choice([16, 48, 64, 128])), int(rng.choice([5, 16, 64])), seed=seed,
                  spare_rows=int(rng.integers(0, 4)), stride=int(rng.integers(0, 3))))


@pytest.mark.parametrize("kind", ["runs", "reversed", "strided"])
@pytest.mark.parametrize("block", [1, 4, 20])
def test_orders_of_pages(api, kind, block):
    # Gathered pages that follow each other in the pool, backwards, with gaps.
    c = Case([(777, 9)], 64, block, seed=3, spare_blocks=1)
    n = -(-786 // block)
    ids = {"runs": np.arange(n), "reversed": np.arange(n)[::-1], "strided": np.arange(n) * 2}[kind]
    pool = np.full(((int(ids.max()) + 1) * block, 512), NAN8, np.uint8)
    for b in range(n):
        pool[int(ids[b]) * block:][:block] = c.pool[int(c.table[0, b]) * block:][:block]
    c.table[0, :n], c.pool = ids, pool
    run(api, c)


def test_many_requests(api):
    run(api, Case([(s % 37, s % 3) for s in range(1100)], 16, 16, seed=3, spare_rows=2))


@pytest.mark.parametrize("heads, block", [(48, 16), (64, 5), (80, 64)])
def test_full_and_partly_filled_items_in_turn(api, heads, block):
    # Every range has several items, of few lines and of many, of one tile and of
    # more; the tokens after each one's last are NaN.
    rng = np.random.default_rng(heads)
    reqs = [(int(rng.integers(0, 600)) if s % 5 == 0 else int(rng.integers(0, 40)), int(rng.choice([1, 1, 1, 2, 3, 5])))
            for s in range(400)]
    run(api, Case(reqs, heads, block, seed=heads, spare_rows=1))


def test_no_new_tokens_at_all(api):
    run(api, Case([(50, 0), (0, 0)], 64, 64, spare_rows=3))


def test_without_lse(api):
    c = Case([(400, 3)], 64, 64).upload(api)
    c.call(api, lse=False)
    out, _ = c.result()
    paged_ref.check_chunk(out, None, c.reference())
    assert (c.lse == 77.0).all()


@pytest.mark.parametrize("new", [1, 9, 130])
def test_nan_in_tokens_a_row_does_not_see(api, new):
    # Every new token but the first is NaN: only the rows that see one may be.
    c = Case([(200, new), (31, new)], 64, 64, seed=new)
    for s in range(2):
        n = int(c.lens[s])
        for j in range(n - new + 1, n, 3):
            c.pool[c.slot(s, j), 5::100] = NAN8 if j % 2 else NAN8 | 0x80
    run(api, c)


def test_one_nan_latent_reaches_its_rows_only(api):
    c = Case([(700, 40)], 64, 64)
    c.pool[c.slot(0, 715), 300] = NAN8
    run(api, c)


def test_missing_blocks_are_left_out(api):
    c = Case([(300, 2), (500, 1), (10, 3), (0, 5)], 64, 16, seed=5)
    c.table[0, 3], c.table[1, 0], c.table[1, 20] = -1, 10 ** 6, -2 ** 31
    c.table[2, :] = -1                                   # nothing left to see
    run(api, c, code=4)


def test_a_block_past_the_end_of_the_pool(api):
    # The last block of the pool is cut short: its missing slots are left out.
    c = Case([(100, 3)], 64, 64, spare_blocks=0)
    c.table[0, 1], c.table[0, 0] = c.table[0, :2].tolist()
    c.pool = c.pool[:100]
    run(api, c, code=4)


def test_refused_requests_keep_their_rows(api):
    # Too short for its rows, past its table, and rows past the buffers.
    c = Case([(10, 4), (20, 3), (30, 2), (5, 6)], 64, 16, seed=2)
    c.lens[0], c.lens[1] = 3, 20 * 16 * c.width
    run(api, c, code=1)
    c = Case([(10, 4), (20, 3)], 64, 16, seed=2)
    c.start[2] += 1
    run(api, c, code=9)


def empty_requests(c, which):
    """Sets the requests' lengths to 0, and gives the reference for that."""
    c.lens[which] = 0
    ref = c.reference()
    for s in which:
        rows = slice(int(c.start[s]), int(c.start[s + 1]))
        ref[1][rows], ref[5][rows] = -np.inf, True
        for k in (0, 2, 3, 4):
            ref[k][rows] = 0.0
    return ref


@pytest.mark.parametrize("reqs, which", [
    ([(0, 1)], [0]), ([(500, 3)], [0]), ([(70, 5), (300, 2)], [0]), ([(300, 2), (70, 5)], [1]),
    ([(10, 300), (700, 40), (0, 1), (5, 2)], [0, 3]), ([(40, 3)] * 3, [0, 1, 2])])
@pytest.mark.parametrize("heads, block", [(16, 64), (64, 20), (128, 16)])
def test_empty_requests_see_nothing(api, reqs, which, heads, block):
    # A length of 0 with rows: what their tables name (latents of an earlier owner,
    # NaN behind them) is not read.
    c = Case(reqs, heads, block, seed=len(reqs), spare_rows=1)
    run(api, c, ref=empty_requests(c, which))


def test_empty_requests_among_many(api):
    rng = np.random.default_rng(3)
    c = Case([(int(rng.integers(0, 300)), int(rng.choice([0, 1, 1, 3, 9]))) for _ in range(300)], 48, 16, seed=9)
    run(api, c, ref=empty_requests(c, rng.permutation(300)[:100]))


@pytest.mark.parametrize("kind", ["sharp", "dominant", "rising", "mixed", "flat"])
@pytest.mark.parametrize("ctx, new", [(2045, 3), (300, 40)])
def test_peaked_rows(api, kind, ctx, new):
    c = Case([(ctx, new)], 64, 64, seed=11, kv_scale=0.05 if kind == "rising" else 0.02)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((new, 64, 512))
    k = np.stack([paged_ref.E4M3[c.pool[c.slot(0, j)]] for j in range(ctx + new)]) * c.kv_scale
    if kind == "sharp":
        q = 5 * x
    elif kind == "dominant":
        q = 0.5 * k[rng.integers(0, ctx, (new, 64))] + 0.02 * x
    elif kind == "mixed":
        q = x * np.logspace(-2, 0.9, 64)[rng.permutation(64)][None, :, None]
    elif kind == "flat":
        q = np.zeros_like(x)
    else:                                                # a maximum that moves in every tile
        v = rng.standard_normal(512)
        for j in range(ctx + new):
            y = (k[j] + 0.1 * (j // 64) / 8 * v) / c.kv_scale
            c.pool[c.slot(0, j)] = torch.from_numpy(y).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        q = rng.uniform(0.3, 0.6, (new, 64, 1)) * v + 0.05 * x
    c.q = bf16_bits(q)
    run(api, c, tag=kind)


def test_one_token_over_a_long_flat_tail(api):
    # A token whose weight is 2^19 of each other's: the others' small weights
    # add up to a share of the output that must not be lost.
    n = 30000
    c = Case([(n - 1, 1)], 64, 64, seed=8)
    v = np.zeros(512)
    v[0] = 1.0
    base = torch.from_numpy(np.full(512, 1.0 / c.kv_scale)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    for j in range(n):
        c.pool[c.slot(0, j)] = base
        c.pool[c.slot(0, j), 0] = 0
    hot = c.slot(0, 777)
    c.pool[hot] = 0
    c.pool[hot, 0] = 0x78                                # 256
    # logit of the hot token above the others': 19 ln 2
    q = np.zeros((1, 64, 512))
    q[..., 0] = 19 * np.log(2) / (c.sm_scale * 256 * c.kv_scale)
    c.q = bf16_bits(q)
    run(api, c)


@pytest.mark.parametrize("heads, q_scale", [(64, 0.05), (16, 1.0), (128, 0.3)])
def test_one_decode_of_more_than_64_parts(api, heads, q_scale):
    # 391 tiles are six a pair of SMs: 66 parts, which the merge takes in two rounds.
    run(api, Case([(99_999, 1)], heads, 64, seed=heads, q_scale=q_scale))


def test_long_tails_of_like_weights(api):
    # The same context 160 times, so that a range has it whole: one hot token,
    # every other's weight 2^-13 to 2^-24 of it, another in each head.  What the tail
    # gives is compared with its own size.  A weight is off by 2^-8 (two terms) and
    # 2^-11 (fp16) down to 2^-14; the mean of a tile's like ones below by 1/256 of a step
    # of a quarter or, in the last octaves, of up to the weight itself: 2^-8, and
    # half of fp16's last step, 2^-9.  Then bf16's half step and the logits' error.
    n, S = 156 * 256, 160
    c = Case([(n - 1, 1)], 64, 64, seed=8)
    base = torch.from_numpy(np.random.default_rng(0).uniform(0.5, 1.5, 512) / c.kv_scale).float()
    codes = base.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    codes[0] = 0
    c.pool[c.pool[:, 0] != NAN8] = codes
    hot = c.slot(0, 777)
    c.pool[hot] = 0
    c.pool[hot, 0] = 0x78                                # 256
    q = np.zeros((1, 64, 512))
    q[0, :, 0] = np.linspace(13, 24, 64) * np.log(2) / (c.sm_scale * 256 * c.kv_scale)
    c.q = bf16_bits(q)
    out, lse, zmag = c.reference()[:3]
    c.lens, c.start = np.repeat(c.lens, S), np.arange(S + 1, dtype=np.int32)
    c.table, c.q, c.rows = np.repeat(c.table, S, 0), np.repeat(c.q, S, 0), S
    c.upload(api).call(api)
    g, e = c.result()
    assert api.dsa_get_error(reset=True)[0] == 0
    tol = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -8 + 16e-6 * zmag[0] + 1e-5
    off = np.abs(g[:, :, 1:] - out[:, :, 1:]) / np.abs(out[:, :, 1:])
    assert (off <= tol[None, :, None]).all(), f"{off.max((0, 2))}"
    assert (np.abs(e - lse) <= 1e-5 + 8e-6 * zmag).all()


def test_hidden_tokens_have_no_weight_at_all(api):
    # Latents of zero where the rows see, as large as they can be where they do not.
    c = Case([(300, 40), (0, 3), (20, 1)], 64, 64, seed=2)
    c.pool[:] = 0
    for s, last in ((0, 339), (1, 2)):
        c.pool[c.slot(s, last)] = 0x7E
    c.upload(api).call(api)
    out, _ = c.result()
    assert api.dsa_get_error(reset=True)[0] == 0
    seen = np.isin(np.arange(c.rows), [39, 42])
    assert (out[~seen] == 0).all() and (out[seen] != 0).any()


def test_non_finite_queries_stay_in_their_head(api):
    c = Case([(200, 3)], 64, 64)
    q = c.q.copy()
    q[0, 3, 100], q[1, 20, 0], q[2, 63, 511] = 0x7F80, 0xFF80, 0x7FC0   # inf, -inf, NaN
    ref = c.reference()
    for r, h in ((0, 3), (1, 20), (2, 63)):
        for a in ref[:2]:
            a[r, h] = np.nan
    c.q = q
    run(api, c, ref=ref)


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_non_finite_queries_that_see_nothing(api, heads):
    # All blocks missing, or a length of 0: 0 and -inf whatever the query is; beside
    # a row that sees the one block there is.
    c = Case([(100, 3), (20, 2), (0, 40)], heads, 16, seed=4)
    c.table[0, :] = -1
    c.table[2, 1:] = -1
    c.lens[1] = 0
    ref = empty_requests(c, [1])
    ref[0][20, 9], ref[1][20, 9] = np.nan, np.nan
    for r in (0, 2, 3, 4):
        c.q[r, :5, 7], c.q[r, 5:9, 400], c.q[r, 9:, 0] = 0x7F80, 0xFF80, 0x7FC0
    c.q[20, 9, 3] = 0x7F80
    run(api, c, ref=ref, code=4)


def test_huge_and_tiny_queries(api):
    c = Case([(100, 2)], 64, 64, seed=6)
    rng = np.random.default_rng(1)
    c.q = bf16_bits(rng.standard_normal((2, 64, 512)) * np.logspace(-30, 1, 64)[None, :, None])
    c.q[0, 5] = 0
    run(api, c)


@pytest.mark.parametrize("sm_scale, kv_scale", [(-0.0625, 0.02), (0.0, 0.02), (0.0625, -0.02), (0.0625, 0.0),
                                                (1e-30, 0.02), (0.0625, 1e-6)])
def test_other_scales(api, sm_scale, kv_scale):
    c = Case([(300, 3), (0, 2)], 64, 64, seed=7, q_scale=0.5)
    c.sm_scale, c.kv_scale = sm_scale, kv_scale
    c.q[1, 5] = 0
    run(api, c)


def test_offsets_past_32_bits(api):
    # Blocks at both ends of a pool of more than 2^32 bytes.
    c = Case([(500, 3)], 64, 64, seed=9)
    c.upload(api)
    far = (1 << 32) // (512 * 64) + 1000
    big = torch.empty(((far + 2 * c.width) * 64, 512), dtype=torch.uint8, device="cuda")
    table = np.array([[far + 2 * b if b % 2 else b for b in range(c.width)]], np.int32)
    for b in range(c.width):
        big[int(table[0, b]) * 64:][:64] = c.d_pool[int(c.table[0, b]) * 64:][:64]
    c.d_table.copy_(torch.from_numpy(table))
    c.d_pool = big
    c.call(api)
    c.check(api)


def test_same_call_twice_is_bit_identical(api):
    c = Case([(3000, 5), (10, 70), (900, 1)], 64, 64, seed=4).upload(api)
    c.call(api)
    torch.cuda.synchronize()
    a, b = c.out.clone(), c.lse.clone()
    c.ws.fill_(0x7F)
    for _ in range(3):
        c.call(api)
    torch.cuda.synchronize()
    assert torch.equal(a, c.out) and torch.equal(b, c.lse)


def test_captured_replayed_with_other_lengths(api):
    # A graph captured once serves other lengths, tables and row counts.
    c = Case([(300, 6), (40, 6)], 64, 64, seed=1).upload(api)
    d = Case([(301, 5), (900, 2)], 64, 64, seed=2, spare_rows=5)
    width = max(c.width, d.width)
    pool = max(len(c.pool), len(d.pool))
    for x in (c, d):
        x.table = np.pad(x.table[:, :x.width], ((0, 0), (0, width - x.width)), constant_values=-1)
        x.pool = np.pad(x.pool, ((0, pool - len(x.pool)), (0, 0)))
        x.width = width
    assert c.rows == d.rows == 12
    c.upload(api)
    c.call(api)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(api)
    for x in (d, c, d):
        for dst, src in zip((*c.seqs.tensors[:2], c.d_table, c.d_pool, c.d_q),
                            (x.lens, x.start, x.table, x.pool, x.q.view(np.int16))):
            dst.copy_(torch.from_numpy(np.ascontiguousarray(src)))
        c.out.fill_(MARK)
        c.lse.fill_(77.0)
        g.replay()
        x.out, x.lse = c.out, c.lse
        x.check(api)


def test_two_streams_at_once(api):
    cases = [Case([(4000, 3)], 64, 64, seed=1), Case([(100, 200)], 64, 64, seed=2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in cases:
        c.upload(api)
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(cases, streams):
            c.call(api, stream=s)
    for c in cases:
        c.check(api)


def test_binding_checks(api):
    c = Case([(30, 2)], 64, 16).upload(api)
    bad = [dict(q=c.d_q[:, :, :256]), dict(q=c.d_q[0]), dict(out=c.out[:1]), dict(lse=c.lse[:, :5]),
           dict(q=c.d_q.float()), dict(pool=c.d_pool[:, :256]), dict(pool=c.d_pool.view(torch.int8)),
           dict(out=c.out.cpu()), dict(q=c.d_q.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(workspace=c.ws.cpu())]
    base = dict(seqs=c.seqs, q=c.d_q, pool=c.d_pool, kv_scale=0.02, sm_scale=0.1, out=c.out, lse=c.lse,
                workspace=c.ws)
    for kw in bad:
        with pytest.raises(ValueError):
            api.dsa_mla_chunk_fp8(**{**base, **kw})
    with pytest.raises(api.DsaError) as e:
        api.dsa_mla_chunk_fp8(**{**base, "workspace": c.ws[:128]})
    assert e.value.status == 5
    with pytest.raises(api.DsaError) as e:
        api.dsa_mla_chunk_fp8(**{**base, "workspace": c.ws[1:]})
    assert e.value.status == 5


def test_plan_write_attend_together(api):
    # A server's steps: prompts, chunks, decodes, a rejected verify and an end,
    # all bookkeeping on the device; then every latent written and attended.
    rng = np.random.default_rng(21)
    S, width, block, rows, heads, cap = 5, 12, 16, 96, 64, 40
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    lens_d, new_d, held, table = i32(S), i32(S), i32(S), torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(cap).astype(np.int32)).cuda()
    count = torch.tensor([cap, 0], dtype=torch.int32, device="cuda")
    start, pos, row_lens, row_seq, row_table = i32(S + 1), i32(rows), i32(rows), i32(rows), i32(rows, width)
    slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    plan = api.make_plan(lens_d, new_d, held, held, table, block, free, count, count, start, pos, slots,
                         row_lens, row_table, row_seq)
    seqs = api.make_seqs(lens_d, start, table, block)
    pool = torch.full((cap * block, 512), NAN8, dtype=torch.uint8, device="cuda")
    norm_w = torch.from_numpy(bf16_bits(rng.standard_normal(512) * 0.1 + 1).view(np.int16)).cuda()
    ws = torch.empty(api.dsa_chunk_workspace_bytes(rows, heads), dtype=torch.uint8, device="cuda")
    lens = np.zeros(S, np.int64)
    steps = [[60, 1, 0, 17, 0], [1, 1, 33, 4, 0], [1, 1, 20, 1, 0], [4, -1, 1, 1, 40], [2, 30, 1, 1, 1]]
    for k, new in enumerate(steps):
        new = np.array(new)
        if k == 4:
            lens[0] -= 3                                  # three of the four verified tokens rejected
        lens = np.where(new < 0, 0, lens + np.maximum(new, 0))
        new = np.maximum(new, 0)
        n = int(new.sum())
        lens_d.copy_(torch.from_numpy(lens))
        new_d.copy_(torch.from_numpy(new))
        kv_a = torch.from_numpy(bf16_bits(rng.standard_normal((n, 512))).view(np.int16)).cuda()
        q = torch.from_numpy(bf16_bits(rng.standard_normal((n, heads, 512)) * 0.1).view(np.int16)).cuda()
        out, lse = torch.zeros_like(q), torch.zeros((n, heads), device="cuda")
        api.dsa_plan_rows(plan)
        r = api.make_rows(row_lens[:n], row_table[:n], block, slots[:n], pos[:n])
        api.dsa_latent_write(r, kv_a, norm_w, pool, 1e-6, 0.02)
        api.dsa_mla_chunk_fp8(seqs, q, pool, 0.02, 0.0625, out, lse, ws)
        torch.cuda.synchronize()
        assert api.dsa_get_error(reset=True)[0] == 0
        ref = paged_ref.chunk(lens, start.cpu().numpy(), table.cpu().numpy(), block,
                              q.cpu().numpy().view(np.uint16), pool.cpu().numpy(), 0.02, 0.0625)
        assert not np.isnan(ref[0]).any()
        paged_ref.check_chunk(out.view(torch.bfloat16).float().cpu().numpy(), lse.cpu().numpy(), ref, f"step {k}")
        # and the gather-attend over the whole visible context says the same
        topk = int(lens.max())
        sel = torch.arange(topk, dtype=torch.int32, device="cuda").repeat(n, 1)
        sel = torch.where(sel < row_lens[:n, None], sel, -1).contiguous()
        out2 = torch.zeros_like(out)
        w2 = torch.empty(api.dsa_workspace_bytes(n, heads, topk), dtype=torch.uint8, device="cuda")
        api.dsa_mla_decode_fp8(r, q, pool, sel, topk, 0.02, 0.0625, out2, None, w2)
        torch.cuda.synchronize()
        paged_ref.check_chunk(out2.view(torch.bfloat16).float().cpu().numpy(), None, ref, f"gather step {k}")


def test_plan_write_attend_captured_once(api):
    # The three calls of a step in one graph over all rows of its buffers, replayed
    # with the state in place: prompts, chunks, decodes, a rejected verify, an end, a
    # request out of blocks, a step with no new tokens, one that fills the buffers.
    rng = np.random.default_rng(22)
    S, width, block, rows, heads, cap = 5, 12, 16, 96, 64, 15
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    lens_d, new_d, held, served = i32(S), i32(S), i32(S), i32(S)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(cap).astype(np.int32)).cuda()
    count = torch.tensor([cap, 0], dtype=torch.int32, device="cuda")
    start, pos, row_lens, row_table = i32(S + 1), i32(rows), i32(rows), i32(rows, width)
    slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    plan = api.make_plan(lens_d, new_d, held, held, table, block, free, count, count, start, pos, slots,
                         row_lens, row_table, served_lens=served, empty_tail=True)
    seqs = api.make_seqs(served, start, table, block)
    r = api.make_rows(row_lens, row_table, block, slots, pos)
    pool = torch.full((cap * block, 512), NAN8, dtype=torch.uint8, device="cuda")
    norm_w = torch.from_numpy(bf16_bits(rng.standard_normal(512) * 0.1 + 1).view(np.int16)).cuda()
    ws = torch.empty(api.dsa_chunk_workspace_bytes(rows, heads), dtype=torch.uint8, device="cuda")
    kv_a = torch.zeros((rows, 512), dtype=torch.int16, device="cuda")
    q = torch.zeros((rows, heads, 512), dtype=torch.int16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((rows, heads), device="cuda")

    def step():
        api.dsa_plan_rows(plan)
        api.dsa_latent_write(r, kv_a, norm_w, pool, 1e-6, 0.02)
        api.dsa_mla_chunk_fp8(seqs, q, pool, 0.02, 0.0625, out, lse, ws)

    step()                                               # (nothing yet: no tokens, no rows)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens = np.zeros(S, np.int64)
    steps = [([60, 1, 0, 17, 0], set()), ([1, 1, 33, 4, 0], set()), ([0] * 5, set()), ([1, 1, 0, 1, 90], {4}),
             ([4, -1, 1, 1, 40], set()), ([2, 30, 1, 1, 1], set()), ([90, 0, 2, 3, 1], set())]
    for k, (new, refused) in enumerate(steps):
        new = np.array(new)
        if k == 5:
            lens[0] -= 3                                 # three of the four verified tokens rejected
        if k == 6:
            lens[0] = lens[1] = 0                        # ends; another takes its place at once
        lens = np.where(new < 0, 0, lens + np.maximum(new, 0))
        new = np.maximum(new, 0)
        n = int(new.sum())
        assert n <= rows and (k != 6 or n == rows)
        lens_d.copy_(torch.from_numpy(lens))
        new_d.copy_(torch.from_numpy(new))
        kv_a.copy_(torch.from_numpy(bf16_bits(rng.standard_normal((rows, 512))).view(np.int16)))
        q.copy_(torch.from_numpy(bf16_bits(rng.standard_normal((rows, heads, 512)) * 0.1).view(np.int16)))
        out.fill_(MARK)
        lse.fill_(77.0)
        before = pool.clone()
        g.replay()
        torch.cuda.synchronize()
        code = api.DEVERR[api.dsa_get_error(reset=True)[0]]
        assert code == ("free" if refused else "none"), f"step {k}: {code}"
        live = np.where(np.isin(np.arange(S), list(refused)), 0, lens)
        assert served.tolist() == live.tolist()
        wrote = torch.unique((pool != before).any(1).nonzero()[:, 0])
        mine = torch.unique(slots[:n][slots[:n] >= 0])
        assert torch.isin(wrote, mine).all(), f"step {k}: a latent of no new token was written"
        assert (slots[n:] == -1).all() and len(mine) == int(new[live > 0].sum())
        case = Case([(0, 1)], heads, block)              # (only for the reference of empty requests)
        case.lens, case.start, case.table, case.width = live.copy(), start.cpu().numpy(), table.cpu().numpy(), width
        case.q, case.pool = q.cpu().numpy().view(np.uint16), pool.cpu().numpy()
        ref = empty_requests(case, sorted(refused))
        paged_ref.check_chunk(out.view(torch.bfloat16).float().cpu().numpy(), lse.cpu().numpy(), ref, f"step {k}")
        assert ref[5].sum() == n and (out[n:] == MARK).all() and (lse[n:] == 77.0).all()
        for s in refused:                                # its caller takes the step back
            lens[s] -= new[s]


def test_a_request_out_of_blocks_reads_nothing(api):
    # Request 1 has a last block with room, which holds what an earlier owner left
    # there; it wants more blocks than there are.  Request 0 is served beside it.
    rng = np.random.default_rng(5)
    S, width, block, rows, heads = 2, 8, 16, 60, 64
    d = lambda a, t=torch.int32: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    table[0, :1], table[1, :2] = d([3]), d([1, 4])
    held, free, count = d([1, 2]), d([0, 2, 7, 7]), d([2, 0])
    lens, new = np.array([20, 70]), np.array([8, 45])    # tokens 25 to 31 of request 1 would be new in what it has
    start, pos, row_lens, served = d([0] * 3), d([0] * rows), d([0] * rows), d([9, 9])
    slots, row_table = d([0] * rows, torch.int64), torch.zeros((rows, width), dtype=torch.int32, device="cuda")
    pool = torch.from_numpy(rng.integers(0, 120, (5 * block, 512)).astype(np.uint8)).cuda()
    plan = api.make_plan(d(lens), d(new), held, held, table, block, free, count, count, start, pos, slots,
                         row_lens, row_table, served_lens=served)
    n = int(new.sum())
    kv_a = torch.from_numpy(bf16_bits(rng.standard_normal((n, 512))).view(np.int16)).cuda()
    q = torch.from_numpy(bf16_bits(rng.standard_normal((n, heads, 512)) * 0.1).view(np.int16)).cuda()
    out, lse = torch.full_like(q, MARK), torch.full((n, heads), 77.0, device="cuda")
    ws = torch.empty(api.dsa_chunk_workspace_bytes(n, heads), dtype=torch.uint8, device="cuda")
    api.dsa_plan_rows(plan)
    assert api.DEVERR[api.dsa_get_error(reset=True)[0]] == "free"
    api.dsa_latent_write(api.make_rows(row_lens[:n], row_table[:n], block, slots[:n], pos[:n]), kv_a,
                         torch.full((512,), 0x3F80, dtype=torch.int16, device="cuda"), pool, 1e-6, 0.02)
    api.dsa_get_error(reset=True)                        # the refused rows' slots
    api.dsa_mla_chunk_fp8(api.make_seqs(served, start, table, block), q, pool, 0.02, 0.0625, out, lse, ws)
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    assert served.tolist() == [20, 0] and row_lens[:n].tolist() == list(range(13, 21)) + [0] * 45
    assert (out[8:] == 0).all() and torch.isneginf(lse[8:]).all()
    ref = paged_ref.chunk([20], [0, 8], table[:1].cpu().numpy(), block, q[:8].cpu().numpy().view(np.uint16),
                          pool.cpu().numpy(), 0.02, 0.0625)
    paged_ref.check_chunk(out[:8].view(torch.bfloat16).float().cpu().numpy(), lse[:8].cpu().numpy(), ref)


def test_forced_timeouts_are_reported_and_the_next_call_is_clean(api):
    # Every wait in the kernel gives up at once: the call returns, says so, and
    # leaves nothing behind.
    default = api.dsa_get_wait_limit_ns()
    c = Case([(3000, 4), (300, 60)], 64, 64, seed=13).upload(api)
    c.call(api)
    c.check(api)
    out, lse = c.out.clone(), c.lse.clone()
    try:
        api.dsa_set_wait_limit_ns(1)
        for _ in range(3):
            c.call(api)
            torch.cuda.synchronize()
            code, _, count = api.dsa_get_error(reset=True)
            assert api.DEVERR[code] == "timeout" and count >= 1
    finally:
        api.dsa_set_wait_limit_ns(0)
    assert api.dsa_get_wait_limit_ns() == default
    for _ in range(2):
        c.out.fill_(MARK)
        c.lse.fill_(77.0)
        c.call(api)
        c.check(api)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
