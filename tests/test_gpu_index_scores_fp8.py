"""dsa_index_scores_fp8 against the 64-bit form.

Tolerance, with M the sum over heads and dims of the terms' magnitudes: a head's
128 exact products in four MMAs of 32, added with the last bits of the largest
(2^-23 of it, cut off, at most), 4 * 33 * 2^-23 < 2^-15; the product of weight and
query scale, each head's addition, the product of gate and key scale and the last
product, each 2^-24 of the running sum: (H + 4) * 2^-24.  Together of M.
"""
import numpy as np
import pytest
import torch

from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu

UNWRITTEN = -123.0


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


class Case:
    """Sequences of given row lengths ([[lengths of a sequence's rows], ...]), their
    keys one behind the other with NaN codes and scales between them."""

    def __init__(self, api, lens, H, D, seed=0, gate=True, gap=130):
        rng = np.random.default_rng(seed)
        self.per = len(lens[0])
        longest = [max(row) for row in lens]
        self.start = np.cumsum([0] + [n + gap for n in longest])[:-1] + gap
        T = int(self.start[-1] + longest[-1] + gap)
        self.k = np.full((T, D), 0x7F, np.uint8)
        self.ks = np.full(T, np.nan, np.float32)
        self.g = np.full(T, np.nan)
        for s, n in zip(self.start, longest):
            self.k[s:s + n] = ref.encode(rng.standard_normal((n, D)) * 100)
            self.ks[s:s + n] = np.exp(rng.standard_normal(n)) * 0.01
            self.g[s:s + n] = torch.from_numpy(rng.uniform(0, 1, n)).to(torch.bfloat16).double().numpy()
        self.lens = np.array(lens).reshape(-1)
        self.R, self.H, self.D = self.lens.size, H, D
        self.q = ref.encode(rng.standard_normal((self.R, H, D)) * 100)
        self.qs = (np.exp(rng.standard_normal((self.R, H))) * 0.01).astype(np.float32)
        self.w = (rng.standard_normal((self.R, H)) * H ** -0.5).astype(np.float32)
        self.max_len = max(1, int(self.lens.max()))
        self.with_gate = gate
        self.upload(api)

    def upload(self, api):
        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.d = dict(q=dev(self.q), q_scale=dev(self.qs), head_w=dev(self.w), idx_k=dev(self.k), idx_scale=dev(self.ks),
                      idx_gate=dev(self.g).to(torch.bfloat16) if self.with_gate else None,
                      idx_base=dev(np.repeat(self.start, self.per).astype(np.int64)))
        self.seq_lens = dev(self.lens.astype(np.int32))
        self.rows = api.make_rows(self.seq_lens)
        self.whole = torch.full((self.R * self.max_len + 64,), UNWRITTEN, device="cuda")
        self.scores = self.whole[:self.R * self.max_len].view(self.R, self.max_len)

    def run(self, api, per=None, **kw):
        api.dsa_index_scores_fp8(self.rows, **(self.d | dict(rows_per_seq=per or self.per, max_len=self.max_len,
                                                             scores=self.scores) | kw))
        torch.cuda.synchronize()
        return self.scores.clone()

    def check(self, live=None):
        got = self.scores.double().cpu().numpy()
        for r in range(self.R):
            n = int(self.lens[r]) if live is None or r in live else 0
            s = int(self.start[r // self.per])
            want, size = ref.index_scores(self.q[r], self.qs[r], self.w[r], self.k[s:s + n], self.ks[s:s + n],
                                          self.g[s:s + n] if self.with_gate else np.ones(n))
            tol = (2.0 ** -15 + (self.H + 4) * 2.0 ** -24) * size
            assert (np.abs(got[r, :n] - want) <= tol).all(), (r, np.abs(got[r, :n] - want).max())
            assert (got[r, n:] == UNWRITTEN).all(), r
        assert (self.whole[self.R * self.max_len:] == UNWRITTEN).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 24, 32, 48, 64, 100, 128, 256])
def test_heads_and_dims(api, H, D):
    c = Case(api, [[1], [300], [0], [128]], H, D, seed=H)
    c.run(api)
    c.check()
    assert api.dsa_get_error(reset=True)[0] == 0


@pytest.mark.parametrize("lens", [
    [[1]], [[0]], [[127]], [[129]], [[5000]], [[40000]],
    [[9, 10]], [[0, 0, 1, 2]], [[255, 256, 257, 258, 259]], [[100, 3, 50, 0, 77, 128, 200]],
    [[n] for n in (1, 0, 64, 128, 129, 1000, 4097)],
    [[700 + i for i in range(33)], [i for i in range(33)]],
    [[n, n + 1, n + 2, n + 3] for n in (4000, 17, 9000, 1, 250)]], ids=lambda x: f"{len(x)}x{len(x[0])}")
def test_lengths(api, lens):
    c = Case(api, lens, 32, 128, seed=len(lens))
    c.run(api)
    c.check()
    assert api.dsa_get_error(reset=True)[0] == 0


@pytest.mark.parametrize("D,H", [(128, 32), (128, 64), (64, 16), (128, 24)])
def test_many_tiles(api, D, H):
    # more tiles than a wave of CTAs holds, whose ranges run over several sequences
    rng = np.random.default_rng(H)
    lens = [[int(n), int(n) + 1] for n in np.exp(rng.uniform(0, np.log(9000), 60)).astype(int)]
    c = Case(api, lens, H, D, seed=1)
    c.run(api)
    c.check()
    assert api.dsa_get_error(reset=True)[0] == 0


def test_without_gates(api):
    c = Case(api, [[500, 501], [40, 41]], 32, 128, gate=False)
    c.run(api)
    c.check()


def test_rows_do_not_depend_on_each_other(api):
    lens = [[3000 + i for i in range(8)], [90 + i for i in range(8)]]
    c = Case(api, lens, 32, 128)
    whole = c.run(api)
    for per in (1, 2, 4):
        c.scores.fill_(UNWRITTEN)
        assert torch.equal(c.run(api, per=per), whole)
    for r in (0, 5, 11):                         # a row by itself
        one = {n: t[r:r + 1] for n, t in c.d.items() if n in ("q", "q_scale", "head_w", "idx_base")}
        out = torch.full((1, c.max_len), UNWRITTEN, device="cuda")
        api.dsa_index_scores_fp8(api.make_rows(c.seq_lens[r:r + 1]), **(c.d | one), rows_per_seq=1,
                                 max_len=c.max_len, scores=out)
        assert torch.equal(out[0], whole[r])


def test_not_a_number_takes_its_head_out(api):
    c = Case(api, [[400]], 16, 128)
    s = c.start[0]
    c.k[s + 7, 100] = 0x7F                       # every head's product with key 7
    c.q[0, 3, 90] = 0xFF                         # head 3's with every key
    c.upload(api)
    got = c.run(api)[0]
    assert not torch.isnan(got[:400]).any() and float(got[7]) == 0.0
    c.w[0, 3] = 0
    c.q[0, 3, 90] = 0
    c.upload(api)
    other = c.run(api)[0]
    keep = torch.arange(400, device="cuda") != 7
    assert torch.equal(got[:400][keep], other[:400][keep])


def test_rows_that_are_out_of_order_are_recorded_and_skipped(api):
    c = Case(api, [[50, 51], [60, 61], [70, 71], [80, 81]], 32, 128)
    c.lens[3] = c.max_len + 1                    # longer than max_len
    base = c.d["idx_base"]
    c.seq_lens.copy_(torch.from_numpy(c.lens.astype(np.int32)))
    base[4] = base[5] = c.k.shape[0] - 10        # past the arena
    written = torch.tensor([51, 61, 71, 80], dtype=torch.int32, device="cuda")
    c.run(api, idx_written=written)              # row 7 sees 81 of 80 written keys
    c.check(live={0, 1, 2, 6})
    assert api.dsa_get_error(reset=True)[2] == 4


def test_offsets_past_32_bits(api):
    # keys that lie past 4 GB of the arena
    T, n = (1 << 25) + 5000, 3000
    c = Case(api, [[n]], 32, 128, gap=0)
    k = torch.full((T, 128), 0x7F, dtype=torch.uint8, device="cuda")
    ks, g = torch.zeros(T, device="cuda"), torch.zeros(T, dtype=torch.bfloat16, device="cuda")
    at = T - n
    k[at:], ks[at:], g[at:] = c.d["idx_k"], c.d["idx_scale"], c.d["idx_gate"]
    c.run(api, idx_k=k, idx_scale=ks, idx_gate=g, idx_base=c.d["idx_base"] + at)
    c.check()


@pytest.mark.parametrize("lens", [[[6000]], [[n] for n in range(100, 20000, 200)]])
def test_inputs_early_waits_for_readers_of_the_scores(api, lens):
    # the kernel before reads the scores; the call after it may start, not store, before it is done
    c = Case(api, lens, 32, 128)
    first = c.run(api)
    sel = [torch.empty((c.R, 64), dtype=torch.int32, device="cuda") for _ in range(2)]
    api.dsa_select_topk(c.rows, first, c.max_len, 64, sel[0])
    other = torch.randint(0, 0x7F, c.d["q"].shape, device="cuda").to(torch.uint8)
    for _ in range(10):
        c.scores.copy_(first)
        api.dsa_select_topk(c.rows, c.scores, c.max_len, 64, sel[1])
        c.run(api, inputs_early=True, q=other)
        assert torch.equal(sel[0], sel[1])
    want = c.scores.clone()
    c.scores.copy_(first)
    assert torch.equal(c.run(api, q=other), want)


def test_same_call_same_bits_replayed(api):
    c = Case(api, [[n, n + 1] for n in range(50, 9000, 300)], 32, 128)
    first = c.run(api)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.dsa_index_scores_fp8(c.rows, **c.d, rows_per_seq=c.per, max_len=c.max_len, scores=c.scores)
    for _ in range(10):
        c.scores.fill_(UNWRITTEN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.scores, first)


def test_refusals(api):
    c = Case(api, [[50, 51]], 32, 128)
    good = c.d | dict(rows=c.rows, rows_per_seq=2, max_len=c.max_len, scores=c.scores)
    for bad in (dict(q=c.d["q"][:1]), dict(q=c.d["q"].float()), dict(q_scale=c.d["q_scale"][:, :3]),
                dict(idx_scale=c.d["idx_scale"][:9]), dict(idx_k=c.d["idx_k"][:, :64]), dict(scores=c.scores[:, :9]),
                dict(head_w=c.d["head_w"].double()), dict(idx_base=c.d["idx_base"][:1]),
                dict(idx_written=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            api.dsa_index_scores_fp8(**(good | bad))
    with pytest.raises(api.DsaError) as e:
        api.dsa_index_scores_fp8(**(good | dict(rows_per_seq=3)))
    assert e.value.status == 1
    assert (c.whole == UNWRITTEN).all()
