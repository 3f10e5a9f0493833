"""dsa_indexer_write_fp8 against the 64-bit form: codes and scales equal.  The
kernel's are those of the norm in 64 bits, rounded once, so a code may differ only
where the value lies within 1e-12 of a border between two codes; the count is
asserted to be 0 for these inputs."""
import numpy as np
import pytest
import torch

from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6
OLD = 0x5A                                      # what the cache holds before


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


class Case:
    """Rows at given positions of a cache of T keys, with its host copies."""

    def __init__(self, api, pos, base, T, D, seed=0, lens=None, x=None, written=None, per=1, gate=True):
        rng = np.random.default_rng(seed)
        R = len(pos)
        def bf(v):
            return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16)
        self.k_raw = bf(rng.standard_normal((R, D)) * 2 + 0.7 if x is None else x)
        self.w, self.b = bf(1 + 0.2 * rng.standard_normal(D)), bf(0.2 * rng.standard_normal(D))
        self.g = bf(rng.uniform(0, 1, R))
        self.pos, self.base, self.per, self.T, self.D = np.asarray(pos), np.asarray(base, np.int64), per, T, D
        lens = self.pos + 1 if lens is None else np.asarray(lens)
        self.lens = torch.from_numpy(lens.astype(np.int32)).cuda()
        self.position = torch.from_numpy(self.pos.astype(np.int32)).cuda()
        self.rows = api.make_rows(self.lens, positions=self.position)
        self.idx_base = torch.from_numpy(self.base).cuda()
        self.idx_k = torch.full((T, D), OLD, dtype=torch.uint8, device="cuda")
        self.idx_scale = torch.full((T,), -3.0, device="cuda")
        self.idx_gate = torch.full((T,), -5.0, dtype=torch.bfloat16, device="cuda")
        self.written = None if written is None else torch.tensor(written, dtype=torch.int32, device="cuda")
        self.with_gate = gate

    def run(self, api, stream=None):
        api.dsa_indexer_write_fp8(self.rows, self.k_raw.cuda(), self.w.cuda(), self.b.cuda(), EPS, self.idx_base,
                                  self.idx_k, self.idx_scale, self.idx_gate if self.with_gate else None,
                                  self.g.cuda() if self.with_gate else None, self.written, self.per, stream)
        torch.cuda.synchronize()

    def want(self, live):
        k = np.full((self.T, self.D), OLD, np.uint8)
        s, g = np.full(self.T, -3.0), np.full(self.T, -5.0)
        y = ref.layer_norm(self.k_raw.view(torch.int16).numpy().view(np.uint16),
                           self.w.view(torch.int16).numpy().view(np.uint16),
                           self.b.view(torch.int16).numpy().view(np.uint16), EPS)
        for r in live:
            t = self.base[r] + self.pos[r]
            finite = np.where(np.isfinite(y[r]), np.abs(y[r]), 0.0)
            s[t] = ref.pow2_scale(finite.max())
            k[t] = ref.encode(y[r] / s[t])
            if self.with_gate:
                g[t] = float(self.g[r])
        return k, s, g

    def check(self, live):
        k, s, g = self.want(live)
        assert np.array_equal(self.idx_scale.cpu().numpy(), s)
        got = self.idx_k.cpu().numpy()
        assert np.array_equal(got, k), np.argwhere(got != k)[:5]
        assert np.array_equal(self.idx_gate.float().cpu().numpy(), g)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 5, 64, 777])
def test_matches_the_formula(api, rows, D):
    rng = np.random.default_rng(rows)
    T = rows + 50
    c = Case(api, rng.permutation(T)[:rows], np.zeros(rows), T, D, seed=rows)
    c.run(api)
    c.check(range(rows))
    assert api.dsa_get_error(reset=True)[0] == 0


@pytest.mark.parametrize("D", [64, 128])
def test_inputs_of_all_kinds(api, D):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((9, D))
    x[0] = 3.0                                  # no variance: y = b
    x[1] = 1e4 + rng.standard_normal(D)         # a mean far above the deviation
    x[2] *= 1e-20
    x[3] *= 1e18
    x[4] = 0
    x[4, 5] = 1.0
    x[5, 3] = np.nan
    x[6, 3] = np.inf
    x[7] = -x[7] ** 3
    x[8, ::2] = -x[8, 1::2]
    c = Case(api, np.arange(9), np.zeros(9), 9, D, x=x, gate=False)
    c.run(api)
    c.check(range(9))


def test_large_weights(api):
    c = Case(api, np.arange(6), np.zeros(6), 6, 128)
    c.w = (c.w.float() * torch.tensor([1e30, 1e-30]).repeat(64)).to(torch.bfloat16)
    c.b[7] = 3.0e38
    c.run(api)
    c.check(range(6))


@pytest.mark.parametrize("per", [1, 2, 4, 7, 32])
def test_lockstep(api, per):
    # level, ahead (rewound), behind (refused), at the start of a sequence
    seqs, room = 5, 200
    p0 = [10, 50, 60, 0, 168]
    written = [10, 55, 59, 0, 200]
    pos = np.concatenate([p + np.arange(per) for p in p0])
    base = np.repeat(np.arange(seqs) * room, per)
    c = Case(api, pos, base, seqs * room, 128, written=written, per=per)
    c.run(api)
    c.check([r for r in range(seqs * per) if r // per != 2])
    want = [p + per for p in p0]
    want[2] = 59
    assert c.written.tolist() == want
    code, row, count = api.dsa_get_error(reset=True)
    assert (api.DEVERR[code], row, count) == ("behind", 2 * per, 1)


def test_a_sequence_is_written_whole_or_not_at_all(api):
    per, room = 4, 64
    pos = np.concatenate([np.arange(4) + 8] * 4)
    lens = pos + 1
    pos[5] += 1                                 # sequence 1: a row out of step
    lens[10] += 1                               # sequence 2: a length that is not position + 1
    base = np.repeat(np.arange(4) * room, per)
    base[14] = 4 * room                         # sequence 3: a row past the cache
    c = Case(api, pos, base, 4 * room, 128, lens=lens, written=[8] * 4, per=per)
    c.run(api)
    c.check(range(4))
    assert c.written.tolist() == [12, 8, 8, 8]
    assert api.dsa_get_error(reset=True)[2] == 3


def test_empty_rows_are_skipped(api):
    # as dsa_plan_rows leaves them: position 0, length 0
    pos, lens = np.array([5, 0, 0, 7]), np.array([6, 0, 1, 8])
    c = Case(api, pos, [0, 0, 20, 0], 40, 128, lens=lens)
    c.run(api)
    c.check([0, 2, 3])
    assert api.dsa_get_error(reset=True)[0] == 0
    c = Case(api, [3, 4, 0, 0, 0, 1], np.repeat([0, 10, 20], 2), 30, 128, lens=[4, 5, 0, 0, 0, 2],
             written=[3, 6, 0], per=2)
    c.run(api)                                  # sequence 1 empty, sequence 2 half empty
    c.check([0, 1])
    assert c.written.tolist() == [5, 6, 0]
    assert api.DEVERR[api.dsa_get_error(reset=True)[0]] == "position"


def test_rows_outside_the_cache_are_recorded(api):
    c = Case(api, [3, 3, 3], [0, -1, 7], 10, 128)
    c.run(api)
    c.check([0])
    code, row, count = api.dsa_get_error(reset=True)
    assert api.DEVERR[code] == "arena" and row in (1, 2) and count == 2


def test_offsets_past_32_bits(api):
    T = (1 << 25) + 100                         # 4 GB of keys
    c = Case(api, [70], [1 << 25], 128, 128)
    small = c.want.__func__
    c.idx_k = torch.empty((T, 128), dtype=torch.uint8, device="cuda")
    c.idx_scale, c.idx_gate = torch.zeros(T, device="cuda"), torch.zeros(T, dtype=torch.bfloat16, device="cuda")
    c.run(api)
    assert api.dsa_get_error(reset=True)[0] == 0
    c.base = np.array([0])
    k, s, g = small(c, [0])
    at = (1 << 25) + 70
    assert np.array_equal(c.idx_k[at].cpu().numpy(), k[70])
    assert float(c.idx_scale[at]) == s[70] and float(c.idx_gate[at]) == g[70]


def test_replayed_with_moving_positions(api):
    # one graph, the positions and counts kept on the device
    c = Case(api, [0, 1], [0, 0], 64, 128, written=[0], per=2)
    k_raw, w, b, g = c.k_raw.cuda(), c.w.cuda(), c.b.cuda(), c.g.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.dsa_indexer_write_fp8(c.rows, k_raw, w, b, EPS, c.idx_base, c.idx_k, c.idx_scale, c.idx_gate, g,
                                  c.written, 2)
        c.position += 2
        c.lens += 2
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0 and c.written.tolist() == [40]
    c.pos, c.base = np.array([0, 1]), np.array([0, 0])
    k, s, _ = c.want([0, 1])
    assert np.array_equal(c.idx_k[:40].cpu().numpy(), np.tile(k[:2], (20, 1)))
    assert np.array_equal(c.idx_scale[:40].cpu().numpy(), np.tile(s[:2], 20))
    assert (c.idx_k[40:] == OLD).all()


def test_refusals(api):
    c = Case(api, [0, 1], [0, 0], 8, 128, written=[0], per=2)
    good = dict(rows=c.rows, k_raw=c.k_raw.cuda(), ln_w=c.w.cuda(), ln_b=c.b.cuda(), eps=EPS, idx_base=c.idx_base,
                idx_k=c.idx_k, idx_scale=c.idx_scale, idx_gate=c.idx_gate, gate=c.g.cuda(), idx_written=c.written,
                rows_per_seq=2)
    for bad in (dict(k_raw=good["k_raw"][:1]), dict(k_raw=good["k_raw"].float()), dict(idx_k=c.idx_k.int()),
                dict(idx_scale=c.idx_scale[:4]), dict(idx_scale=c.idx_scale.double()), dict(gate=c.g.cuda()[:1]),
                dict(idx_written=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(ln_w=c.w),
                dict(idx_gate=c.idx_gate[:3]), dict(idx_base=c.idx_base.int())):
        with pytest.raises(ValueError):
            api.dsa_indexer_write_fp8(**(good | bad))
    for bad in (dict(eps=-1.0), dict(rows_per_seq=0), dict(idx_gate=None)):
        with pytest.raises(api.DsaError) as e:
            api.dsa_indexer_write_fp8(**(good | bad))
        assert e.value.status == 1
    assert (c.idx_k == OLD).all()


def test_weights_from_the_kernel_before(api):
    """The norm's weight and bias are outputs of the kernel just before each write."""
    c = Case(api, [0], [0], 1, 128, gate=False)
    g = torch.Generator().manual_seed(2)
    k_raw, one = c.k_raw.cuda(), torch.zeros((1, 16), dtype=torch.bfloat16, device="cuda")
    one[0, 0] = 1
    sides = torch.zeros((2, 256, 16), dtype=torch.bfloat16)
    sides[:, :, 0] = torch.randn((2, 256), generator=g).to(torch.bfloat16)
    dev = sides.cuda()
    wb = torch.zeros((1, 256), dtype=torch.bfloat16, device="cuda")
    workspace = torch.empty(max(api.dsa_dense_mm_workspace_bytes(256, 16), 256), dtype=torch.uint8, device="cuda")
    got_k, got_s = torch.empty((40, 128), dtype=torch.uint8, device="cuda"), torch.empty(40, device="cuda")
    for i in range(40):
        api.dsa_dense_mm_bf16(one, dev[i % 2], wb, workspace)
        api.dsa_indexer_write_fp8(c.rows, k_raw, wb[0, :128], wb[0, 128:], EPS, c.idx_base, got_k[i:i + 1],
                                  got_s[i:i + 1])
    torch.cuda.synchronize()
    for i in range(40):
        c.w, c.b = sides[i % 2, :128, 0].contiguous(), sides[i % 2, 128:, 0].contiguous()
        k, s, _ = c.want([0])
        assert np.array_equal(got_k[i].cpu().numpy(), k[0]) and got_s[i].item() == s[0], i
