"""The 8-bit operators together, as a step runs them: the layer input
quantised, projected to the indexer's key and queries, the key written into the
FP8 cache, the queries quantised, the cache scored and the top tokens selected.
Each stage is checked against the 64-bit form of the stage on what the stage
before it left."""
import numpy as np
import pytest
import torch

from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu

HIDDEN, H, D, EPS = 1024, 32, 128, 1e-6


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def _weight(api, n, k):
    w = torch.randn((n, k), device="cuda").to(torch.bfloat16) / k ** 0.5
    codes = torch.empty((n, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty((-(-n // 128), -(-k // 128)), device="cuda")
    api.dsa_quantize_fp8(w, codes, scales, block_rows=128)
    return codes, scales


class Step:
    """A step of ``per`` new tokens for each of some sequences, all buffers resident."""

    def __init__(self, api, lens, per, seed):
        torch.manual_seed(seed)
        self.api, self.per, seqs = api, per, len(lens)
        R = self.R = seqs * per
        room = max(lens) + 64
        self.T = seqs * room
        self.wk, self.wq = _weight(api, D, HIDDEN), _weight(api, H * D, HIDDEN)
        self.ln_w = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16)
        self.ln_b = (0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16)
        pos = torch.tensor([[n - per + i for i in range(per)] for n in lens], dtype=torch.int32, device="cuda")
        self.positions, self.seq_lens = pos.view(-1).clone(), (pos + 1).view(-1).clone()
        self.base = (torch.arange(seqs, device="cuda") * room).repeat_interleave(per)
        self.written = torch.tensor([n - per for n in lens], dtype=torch.int32, device="cuda")
        self.idx_k = torch.empty((self.T, D), dtype=torch.uint8, device="cuda")
        self.idx_scale = torch.empty(self.T, device="cuda")
        old = torch.randn((self.T, D), device="cuda")
        api.dsa_quantize_fp8(old, self.idx_k, self.idx_scale)      # the keys of the tokens before
        self.idx_gate = torch.rand(self.T, device="cuda").to(torch.bfloat16)
        self.hidden = torch.randn((R, HIDDEN), device="cuda").to(torch.bfloat16)
        self.gate = torch.rand(R, device="cuda").to(torch.bfloat16)
        self.head_w = torch.randn((R, H), device="cuda") * H ** -0.5
        self.x, self.xs = torch.empty((R, HIDDEN), dtype=torch.uint8, device="cuda"), torch.empty((R, HIDDEN // 128), device="cuda")
        self.k_raw = torch.empty((R, D), dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty((R, H * D), device="cuda")
        self.q8, self.qs = torch.empty((R, H, D), dtype=torch.uint8, device="cuda"), torch.empty((R, H), device="cuda")
        self.max_len = room
        self.scores = torch.zeros((R, room), device="cuda")
        self.sel = torch.empty((R, 64), dtype=torch.int32, device="cuda")
        self.rows = api.make_rows(self.seq_lens, positions=self.positions)

    def run(self):
        api = self.api
        api.dsa_quantize_fp8(self.hidden, self.x, self.xs)
        api.dsa_dense_mm_fp8(self.x, self.xs, *self.wk, self.k_raw)
        api.dsa_dense_mm_fp8(self.x, self.xs, *self.wq, self.q)
        api.dsa_indexer_write_fp8(self.rows, self.k_raw, self.ln_w, self.ln_b, EPS, self.base, self.idx_k,
                                  self.idx_scale, self.idx_gate, self.gate, self.written, self.per)
        api.dsa_quantize_fp8(self.q.view(self.R, H, D), self.q8, self.qs)
        api.dsa_index_scores_fp8(self.rows, self.q8, self.qs, self.head_w, self.idx_k, self.idx_scale, self.idx_gate,
                                 self.base, self.per, self.max_len, self.scores, self.written)
        api.dsa_select_topk(self.rows, self.scores, self.max_len, 64, self.sel)

    def check(self):
        torch.cuda.synchronize()
        assert self.api.dsa_get_error(reset=True)[0] == 0
        def host(t):
            return (t.view(torch.int16) if t.dtype is torch.bfloat16 else t).cpu().numpy()
        codes, scales = ref.quantize(self.hidden.double().cpu().numpy())
        assert np.array_equal(host(self.x), codes) and np.array_equal(host(self.xs), scales)
        for w, out, half in ((self.wk, self.k_raw, 2.0 ** -8), (self.wq, self.q, 0.0)):
            want, size = ref.product(codes, scales, host(w[0]), host(w[1]))
            assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -14 * size + half * np.abs(want)).all()
        y = ref.layer_norm(*(host(t).view(np.uint16) for t in (self.k_raw, self.ln_w, self.ln_b)), EPS)
        at = (self.base + self.positions).cpu().numpy()
        s = ref.pow2_scale(np.abs(y).max(1))
        assert np.array_equal(host(self.idx_scale)[at], s)
        assert np.array_equal(host(self.idx_k)[at], ref.encode(y / s[:, None]))
        q8, qs = ref.quantize(self.q.double().cpu().numpy().reshape(-1, D))
        assert np.array_equal(host(self.q8).reshape(-1, D), q8) and np.array_equal(host(self.qs).reshape(-1, 1), qs)
        scores, sel, gates = host(self.scores), host(self.sel), self.idx_gate.double().cpu().numpy()
        for r in range(self.R):
            n, b = int(self.seq_lens[r]), int(self.base[r])
            want, size = ref.index_scores(host(self.q8)[r], host(self.qs)[r], host(self.head_w)[r],
                                          host(self.idx_k)[b:b + n], host(self.idx_scale)[b:b + n], gates[b:b + n])
            assert (np.abs(scores[r, :n] - want) <= 2.0 ** -14 * size).all()
            order = np.lexsort((np.arange(n), -scores[r, :n]))[:64]
            assert np.array_equal(sel[r][sel[r] >= 0], np.sort(order))


@pytest.mark.parametrize("lens,per", [([1], 1), ([500], 1), ([70, 900, 33, 1500], 4), ([3000 + 7 * i for i in range(20)], 1)])
def test_decode_step(api, lens, per):
    step = Step(api, lens, per, seed=len(lens))
    step.run()
    step.check()


def test_steps_captured_once_and_replayed(api):
    step = Step(api, [100, 700, 40], 2, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.run()
    for _ in range(4):
        graph.replay()
        step.check()
        step.positions += 2
        step.seq_lens += 2
        step.hidden.copy_(torch.randn(step.hidden.shape, device="cuda"))


@pytest.mark.parametrize("name,kw", [("tiny", dict(len_div=4)), ("verify", dict(seqs=2, len_div=64)),
                                     ("long", dict(seqs=3, len_div=32))])
def test_decode_path_over_fp8_index_keys(api, oracle, name, kw):
    from sparse_attention_mla_dsa_gb300 import path, workloads
    from tests import parity
    wl = workloads.scaled(name, **kw)
    dw = path.DeviceWorkload(wl, index_fp8=True)
    dw.step()
    torch.cuda.synchronize()
    assert api.dsa_get_error(reset=True)[0] == 0
    scores, sel, out = dw.scores.cpu().numpy(), dw.sel.cpu().numpy(), dw.out_f32()
    T, dim = wl.idx_k.shape
    pool = wl.pool.copy()
    if wl.kv_a is not None:
        oracle.latent_write(pool, wl.kv_a, wl.norm_w, wl.slots, wl.eps, wl.kv_scale)
    for r in range(wl.rows):
        L, base = int(wl.seq_lens[r]), int(wl.idx_base[r])
        k8, ks = ref.quantize(ref.bf16(wl.idx_k[base:base + L]))
        q8, qs = ref.quantize(wl.q_idx[r])
        want, size = ref.index_scores(q8, qs[:, 0], wl.head_w[r], k8, ks[:, 0], ref.bf16(wl.idx_gate[base:base + L]))
        assert (np.abs(scores[r, :L] - want) <= 2.0 ** -14 * size).all()
        assert np.array_equal(oracle.select_topk_row(scores[r, :L].astype(np.float64), L, wl.topk), sel[r])
        o_ref, _ = oracle.mla_decode_row(wl.Q[r], pool, wl.block_table[r], wl.block_size, L, sel[r], wl.kv_scale, wl.sm_scale)
        parity.assert_out(out[r], o_ref, f"{name} row {r}")
    twin = dw.clone()
    twin.scores.zero_()
    twin.step()
    for n in ("sel", "out"):
        assert torch.equal(getattr(twin, n), getattr(dw, n))
