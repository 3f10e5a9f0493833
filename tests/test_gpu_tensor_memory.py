"""Kernels that take all of an SM's tensor memory with others right behind them.

Scores of more than 128 heads take every column.  A kernel that lets the next one
start before its columns are its own would wait for them for ever behind a CTA that
took them first; every kernel here takes them before.  The calls go through a
captured graph, so that nothing of the host lies between them, and each is held to
its 64-bit form.
"""
import numpy as np
import pytest
import torch

from tests import fp8_ref as ref
from tests.test_gpu_index_scores_fp8 import Case

pytestmark = pytest.mark.gpu

H = 256


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


class Bf16Scores:
    """The bf16 form of a Case: one row a sequence.

    Tolerance, with M the sum over heads and dims of the terms' magnitudes: a query
    is two bf16 terms, 2^-17 of it at most away; D / 8 MMAs of 16 exact products and
    the running sum, the last bits cut off, (D / 8) * 17 * 2^-23 < 2^-14; each
    head's addition and the gate's product, (H + 4) * 2^-24."""

    def __init__(self, api, lens, D, seed):
        rng = np.random.default_rng(seed)
        self.lens, self.start = lens, np.cumsum([0] + lens)[:-1]
        T, R = sum(lens), len(lens)
        self.q = torch.from_numpy(rng.standard_normal((R, H, D), dtype=np.float32)).cuda()
        self.w = torch.from_numpy(rng.standard_normal((R, H), dtype=np.float32)).cuda()
        self.k = torch.from_numpy(rng.standard_normal((T, D), dtype=np.float32)).to(torch.bfloat16).cuda()
        self.g = torch.from_numpy(rng.uniform(0, 1, T)).to(torch.bfloat16).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.base = torch.from_numpy(self.start).cuda()
        self.rows = api.make_rows(self.seq_lens)
        self.scores = torch.zeros((R, max(lens)), device="cuda")

    def call(self, api):
        api.dsa_index_scores(self.rows, self.q, self.w, self.k, self.g, self.base, 1, self.scores.shape[1], self.scores)

    def check(self):
        for r, (n, s) in enumerate(zip(self.lens, self.start)):
            q, k = self.q[r].double().cpu().numpy(), self.k[s:s + n].double().cpu().numpy()
            w, g = self.w[r].double().cpu().numpy(), self.g[s:s + n].double().cpu().numpy()
            want = g * (w[:, None] * np.maximum(q @ k.T, 0.0)).sum(0)
            size = g * (np.abs(w)[:, None] * (np.abs(q) @ np.abs(k).T)).sum(0)
            got = self.scores[r, :n].double().cpu().numpy()
            assert (np.abs(got - want) <= (2.0 ** -17 + 2.0 ** -14 + (H + 4) * 2.0 ** -24) * size).all(), r


class Fp8Scores(Case):
    def __init__(self, api, lens, D, seed):
        super().__init__(api, [[n] for n in lens], H, D, seed=seed)

    def call(self, api):
        api.dsa_index_scores_fp8(self.rows, **self.d, rows_per_seq=1, max_len=self.max_len, scores=self.scores)


class Fp8Product:
    """Tolerance: as test_gpu_dense_mm_fp8."""

    def __init__(self, api, m, n, k):
        rng = np.random.default_rng(m)
        self.ops = [ref.encode(rng.standard_normal((m, k)) * 60), rng.uniform(0.5, 1, (m, k // 128)).astype(np.float32),
                    ref.encode(rng.standard_normal((n, k)) * 60), rng.uniform(0.5, 1, (n // 128, k // 128)).astype(np.float32)]
        self.dev = [torch.from_numpy(x).cuda() for x in self.ops]
        self.c = torch.zeros((m, n), device="cuda")

    def call(self, api):
        api.dsa_dense_mm_fp8(*self.dev, self.c)

    def check(self):
        want, size = ref.product(*self.ops)
        tol = (2.0 ** -15 + (self.ops[0].shape[1] // 128 + 8) * 2.0 ** -24) * size
        assert (np.abs(self.c.double().cpu().numpy() - want) <= tol).all()


class Bf16Product:
    """Tolerance, of the terms' magnitudes: k / 16 MMAs of 16 exact products and the running sum,
    17 * 2^-23 each, and the ranges' sums."""

    def __init__(self, api, m, n, k):
        g = torch.Generator(device="cuda").manual_seed(m)
        self.a, self.b = (torch.randn((r, k), generator=g, device="cuda").to(torch.bfloat16) for r in (m, n))
        self.c = torch.zeros((m, n), device="cuda")
        self.ws = torch.empty(max(256, api.dsa_dense_mm_workspace_bytes(n, k)), dtype=torch.uint8, device="cuda")

    def call(self, api):
        api.dsa_dense_mm_bf16(self.a, self.b, self.c, self.ws)

    def check(self):
        x, w = self.a.double(), self.b.double()
        tol = (self.a.shape[1] / 16 * 17 * 2.0 ** -23 + 152 * 2.0 ** -24) * (x.abs() @ w.abs().t())
        assert ((self.c.double() - x @ w.t()).abs() <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scores", [Fp8Scores, Bf16Scores])
def test_calls_right_behind_scores_that_take_all_of_it(api, scores, D):
    long = scores(api, [6000, 2500, 6500, 5000], D, seed=D)       # more tiles than SMs
    short = scores(api, [700, 90], D, seed=D + 1)                 # a few tiles a CTA, set up before the wait
    calls = [long, Fp8Product(api, 16, 1024, 2048), long, Fp8Product(api, 30, 512, 1024), short, long,
             Fp8Product(api, 60, 384, 1536), long, Bf16Product(api, 16, 1000, 1024), long, long,
             Fp8Product(api, 200, 512, 1024), long, short]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c.call(api)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for c in calls:
        c.check()
    for c in calls:                                               # and from the host
        c.call(api)
    torch.cuda.synchronize()
    for c in calls:
        c.check()
    assert api.dsa_get_error(reset=True)[0] == 0


def test_two_streams_at_once(api):
    # each stream's kernels beside the other's on the same SMs, clusters among them
    def calls(seed):
        return [Fp8Scores(api, [6000, 2500, 6500, 5000], 64, seed), Fp8Product(api, 60, 1024, 2048),
                Fp8Scores(api, [700, 90], 64, seed + 1), Fp8Product(api, 16, 2048, 1024),
                Bf16Scores(api, [3000, 9000, 4000], 64, seed + 2), Fp8Product(api, 40, 4096, 1024),
                Bf16Product(api, 16, 1000, 1024), Fp8Product(api, 200, 512, 1024)]

    streams = [torch.cuda.Stream() for _ in range(2)]
    sets, graphs = [calls(1), calls(11)[::-1]], []
    for s, mine in zip(streams, sets):
        s.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            for c in mine * 3:
                c.call(api)
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for mine in sets:
        for c in mine:
            c.check()
    assert api.dsa_get_error(reset=True)[0] == 0
