"""Entry points called from host threads: one whose first CUDA call it is, and two at
once on streams of their own with calls of different sizes, where the shared memory
that one call asks for must not be taken away by the other before its launch."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def topk(api, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    rows = api.make_rows(lens)
    scores = torch.randn((2, n), generator=g, device="cuda")
    sel = torch.full((2, 512), -7, dtype=torch.int32, device="cuda")
    return lambda stream=None: api.dsa_select_topk(rows, scores, n, 512, sel, stream=stream), sel, (lens, scores)


def pools(api, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    pos = torch.full((2,), 4 * n, dtype=torch.int32, device="cuda")
    lens = pos + 1
    rows = api.make_rows(lens, positions=pos)
    scores = torch.randn((2, n), generator=g, device="cuda")
    valid = torch.ones((2, n), dtype=torch.uint8, device="cuda")
    sel = torch.full((2, 32), -7, dtype=torch.int32, device="cuda")
    return (lambda stream=None: api.dsa_select_pools(rows, scores, valid, 4, 32, sel, stream=stream), sel,
            (pos, lens, scores, valid))


def scores(api, heads):
    g = torch.Generator(device="cuda").manual_seed(heads)
    n = 5000
    lens, base = torch.full((1,), n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    rows = api.make_rows(lens)
    q, w = torch.randn((1, heads, 128), generator=g, device="cuda"), torch.randn((1, heads), generator=g, device="cuda")
    k = torch.randn((n, 128), generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.zeros((1, n), device="cuda")
    return (lambda stream=None: api.dsa_index_scores(rows, q, w, k, gate, base, 1, n, out, stream=stream), out,
            (lens, base, q, w, k, gate))


def latents(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    return torch.randint(0, 120, (n, 512), generator=g, device="cuda", dtype=torch.uint8)


def decode(api, n):
    pool, lens = latents(n), torch.full((1,), n, dtype=torch.int32, device="cuda")
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None].contiguous()
    sel = torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()
    q = torch.full((1, 64, 512), 0x3C00, dtype=torch.int16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(api.dsa_workspace_bytes(1, 64, n), dtype=torch.uint8, device="cuda")
    rows = api.make_rows(lens, table, 64)
    return (lambda stream=None: api.dsa_mla_decode_fp8(rows, q, pool, sel, n, 0.02, 0.06, out, None, ws, stream=stream),
            out, (pool, lens, table, sel, q, ws))


def chunk(api, n):
    pool, lens = latents(n), torch.full((1,), n, dtype=torch.int32, device="cuda")
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None].contiguous()
    seqs = api.make_seqs(lens, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), table, 64)
    q = torch.full((1, 64, 512), 0x3C00, dtype=torch.int16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(api.dsa_chunk_workspace_bytes(1, 64), dtype=torch.uint8, device="cuda")
    return (lambda stream=None: api.dsa_mla_chunk_fp8(seqs, q, pool, 0.02, 0.06, out, None, ws, stream=stream),
            out, (pool, q, ws))


def dense(api, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    a = torch.randn((4, n), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn((256, n), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.zeros((4, 256), device="cuda")
    ws = torch.empty(max(1, api.dsa_dense_mm_workspace_bytes(256, n)), dtype=torch.uint8, device="cuda")
    return lambda stream=None: api.dsa_dense_mm_bf16(a, b, out, ws, stream=stream), out, (a, b, ws)


@pytest.mark.parametrize("make, n", [(scores, 64), (decode, 1024), (chunk, 1024), (dense, 1024)],
                         ids=["scores", "decode", "chunk", "dense"])
def test_first_call_of_a_host_thread(api, make, n):
    # A thread that has made no CUDA call yet.
    call, out, _ = make(api, n)
    call()
    torch.cuda.synchronize()
    want, stream, failures = out.clone(), torch.cuda.current_stream().cuda_stream, []
    assert (want != 0).any()
    out.zero_()
    torch.cuda.synchronize()

    def work():
        try:
            call(stream)
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    assert torch.equal(out, want) and api.dsa_get_error(reset=True)[0] == 0


@pytest.mark.parametrize("make, small, large", [(topk, 30000, 300000), (pools, 100, 16384), (scores, 8, 64)],
                         ids=["topk", "pools", "scores"])
def test_calls_of_two_sizes_from_two_threads(api, make, small, large):
    cases = [make(api, small), make(api, large)]
    want = []
    for call, out, _ in cases:
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
    streams, failures = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()

    def work(call, stream):
        try:
            for _ in range(2000):
                call(stream)
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(c[0], s)) for c, s in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    assert api.dsa_get_error(reset=True)[0] == 0
    for (_, out, _), ref in zip(cases, want):
        assert torch.equal(out, ref)
