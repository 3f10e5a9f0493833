"""dsa_plan_rows against a loop over the requests: every output an integer,
compared exactly, with rows and table entries that must stay as they were."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from tests import paged_ref

pytestmark = pytest.mark.gpu
MARK = -7777


@pytest.fixture(scope="module")
def api():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_mla_dsa_gb300 import api
    api.load()
    api.dsa_get_error(reset=True)
    return api


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


class State:
    """A server's buffers for `seqs` requests, and a host copy of the state."""

    def __init__(self, seqs, width, block, capacity, rows, seed, stride=None, in_place=False,
                 row_table=True, row_seq=True, free=None):
        rng = np.random.default_rng(seed)
        self.block, self.rows, self.width = block, rows, width
        self.table = np.full((seqs, width), MARK, np.int32)
        self.free = rng.permutation(capacity).astype(np.int32)
        self.count = capacity if free is None else free
        self.held = np.zeros(seqs, np.int64)
        self.d_table_all = torch.full((seqs, stride or width), MARK, dtype=torch.int32, device="cuda")
        self.d_table = self.d_table_all[:, :width]
        self.d_free, self.d_held = dev(self.free), dev(self.held)
        self.d_held_out = self.d_held if in_place else torch.full_like(self.d_held, MARK)
        self.d_in = torch.tensor([self.count, 0], dtype=torch.int32, device="cuda")
        self.d_out = self.d_in if in_place else torch.tensor([MARK, 0], dtype=torch.int32, device="cuda")
        self.d_lens, self.d_new = dev(self.held), dev(self.held)
        full = lambda n, t=torch.int32: torch.full((n,), MARK, dtype=t, device="cuda")  # noqa: E731
        self.row_start, self.positions, self.row_lens = full(seqs + 1), full(rows), full(rows)
        self.slots = full(rows, torch.int64)
        self.row_seq = full(rows) if row_seq else None
        self.row_all = torch.full((rows, (stride or width) + 3), MARK, dtype=torch.int32, device="cuda")
        self.row_table = self.row_all[:, :width] if row_table else None

    def plan(self, api):
        return api.make_plan(self.d_lens, self.d_new, self.d_held, self.d_held_out, self.d_table,
                             self.block, self.d_free, self.d_in, self.d_out, self.row_start,
                             self.positions, self.slots, self.row_lens, self.row_table, self.row_seq)

    def lengths(self, lens, new):
        self.lens, self.new = np.asarray(lens), np.asarray(new)
        self.d_lens.copy_(dev(self.lens))
        self.d_new.copy_(dev(self.new))

    def expect(self):
        return paged_ref.plan(self.lens, self.new, self.held, self.table, self.free, self.count,
                              self.block, self.rows)

    def check(self, api, ref, errors=None):
        torch.cuda.synchronize()
        code = api.dsa_get_error(reset=True)[0]
        want = ref["errors"] if errors is None else errors
        assert (code == 0) == (not want), (api.DEVERR[code], want)
        assert not want or api.DEVERR[code] in want
        n = len(ref["positions"])
        assert self.row_start.tolist() == ref["row_start"]
        for name in ("positions", "slots", "row_lens", "row_seq"):
            t = getattr(self, name)
            if t is None:
                continue
            assert t[:n].tolist() == ref[name], name
            assert (t[n:] == MARK).all(), name + " behind the last row"
        if self.row_table is not None:
            assert self.row_table[:n].tolist() == ref["row_table"]
            assert (self.row_all[n:] == MARK).all() and (self.row_all[:, self.width:] == MARK).all()
        assert np.array_equal(self.d_table.cpu().numpy(), ref["table"])
        assert (self.d_table_all[:, self.width:] == MARK).all()
        assert self.d_held_out.tolist() == ref["held"].tolist()
        assert self.d_out.tolist() == [len(ref["free"]), 0]
        left = np.array(ref["free"], np.int32)
        assert np.array_equal(self.d_free.cpu().numpy()[:len(left)], left)

    def advance(self, ref):
        self.table, self.held = ref["table"], ref["held"]
        self.free[:len(ref["free"])] = ref["free"]
        self.count = len(ref["free"])


CASES = [  # seqs, width, block, rows, steps
    (1, 1, 64, 1, 3), (1, 513, 64, 4, 4), (3, 40, 5, 64, 5), (33, 17, 16, 300, 5), (64, 129, 64, 64, 4),
    (511, 9, 7, 700, 4), (513, 33, 1, 900, 3), (1000, 257, 16, 20000, 3), (2500, 12, 8, 9000, 3),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("seqs, width, block, rows, steps", CASES)
def test_steps_of_a_server(api, seqs, width, block, rows, steps, in_place):
    # Requests start, grow by odd amounts, are rewound and end; blocks given
    # back are taken again by others in the same step.
    rng = np.random.default_rng(seqs * 31 + width)
    st = State(seqs, width, block, seqs * width, rows, 1, in_place=in_place)
    plan, lens = st.plan(api), np.zeros(seqs, np.int64)
    for step in range(steps):
        act = rng.random(seqs)
        budget, new = rows, np.zeros(seqs, np.int64)
        for s in range(seqs):
            n = 0
            if act[s] < 0.15:
                lens[s] = 0
            elif act[s] < 0.3:
                lens[s] = rng.integers(0, lens[s] + 1)
            room = min(width * block - lens[s], budget)
            if act[s] > 0.05 and room > 0:
                n = int(min(room, rng.integers(0, 1 + max(1, 2 * rows // seqs))))
            lens[s] += n
            new[s], budget = n, budget - n
        st.lengths(lens, new)
        ref = st.expect()
        assert not ref["errors"]
        for _ in range(1 if in_place else 2):    # apart: the same call again gives the same
            api.dsa_plan_rows(plan)
        st.check(api, ref)
        st.advance(ref)
        if not in_place:
            st.d_held.copy_(st.d_held_out)
            st.d_in.copy_(st.d_out)
        for t in (st.row_start, st.positions, st.slots, st.row_lens, st.row_seq, st.row_all):
            t.fill_(MARK)


def test_full_prompt_and_long_tables(api):
    st = State(2, 2051, 64, 4200, 65535, 5)
    st.lengths([2050 * 64 + 1, 300], [1023, 300])
    api.dsa_plan_rows(st.plan(api))
    st.check(api, st.expect())


def test_as_many_requests_as_allowed(api):
    rng = np.random.default_rng(2)
    st = State(8192, 3, 4, 8192 * 3, 9000, 11)
    new = rng.integers(0, 2, 8192)
    st.lengths(rng.integers(1, 13, 8192), new)
    api.dsa_plan_rows(st.plan(api))
    st.check(api, st.expect())


def sizes_around_48_kb():
    # The scan's 20 bytes a request and the kernel's fixed part pass 48 KB here.
    from sparse_attention_mla_dsa_gb300 import api
    for seqs in (2405, 2406, 2430, 2436, 2437, 2438, 2450, 2456, 2457):
        rng = np.random.default_rng(seqs)
        st = State(seqs, 2, 4, seqs * 2, 2600, 13)
        st.lengths(rng.integers(1, 9, seqs), rng.integers(0, 2, seqs))
        api.dsa_plan_rows(st.plan(api))
        st.check(api, st.expect())


def test_around_48_kb_of_shared_memory(api):
    # In a process of its own, where no larger batch has been planned before.
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = "from tests.test_gpu_plan_rows import sizes_around_48_kb as f; f()"
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_with_batches_of_other_sizes(api):
    # Each thread's calls ask for another amount of shared memory; neither may
    # take away what the other has asked for.
    rng = np.random.default_rng(7)
    states, failures = [], []
    for seqs in (8192, 2500):
        st = State(seqs, 2, 4, seqs * 2, 600, 14, row_table=False)
        new = np.zeros(seqs, np.int64)
        new[rng.permutation(seqs)[:500]] = 1
        st.lengths(rng.integers(1, 9, seqs), new)
        states.append((st, st.plan(api), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(plan, stream):
        try:
            for _ in range(3000):
                api.dsa_plan_rows(plan, stream=stream)
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(plan, stream)) for _, plan, stream in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    for st, _, _ in states:
        st.check(api, st.expect())


@pytest.mark.parametrize("row_table, row_seq", [(False, True), (True, False), (False, False)])
def test_optional_outputs_and_strided_tables(api, row_table, row_seq):
    st = State(5, 6, 16, 30, 40, 3, stride=11, row_table=row_table, row_seq=row_seq)
    st.lengths([17, 0, 96, 1, 33], [3, 0, 16, 1, 20])
    api.dsa_plan_rows(st.plan(api))
    st.check(api, st.expect())


def test_out_of_blocks_refuses_in_order(api):
    # 7 free, 2 given back; wanted 3, 4, 3, 0, 1: the third and the last are
    # refused (its blocks are wanted before the last's), the others served.
    st = State(6, 8, 4, 12, 20, 4, free=7)
    st.held[3] = 1
    st.held[5] = 4
    st.table[3, 0], st.table[5, :4] = 7, [8, 9, 10, 11]
    st.d_table.copy_(dev(st.table))
    st.d_held.copy_(dev(st.held))
    st.lengths([12, 16, 9, 4, 1, 8], [4, 3, 2, 1, 1, 0])
    ref = st.expect()
    assert ref["errors"] == {"free"} and ref["row_lens"].count(0) == 3
    api.dsa_plan_rows(st.plan(api))
    st.check(api, ref)


def test_invalid_requests_change_nothing(api):
    # n < 0, n > L, n > rows, L past the table, held outside the table
    st = State(8, 4, 8, 40, 16, 6)
    st.held[:] = [1, 1, 1, 1, 1, -5, 9, 0]
    for s in (0, 1, 2, 3, 4):
        st.table[s, 0] = 30 + s
    st.d_table.copy_(dev(st.table))
    st.d_held.copy_(dev(st.held))
    st.lengths([9, 9, 2, 30, 33, 8, 8, 20], [1, -1, 3, 17, 2, 1, 1, 4])
    ref = st.expect()
    assert ref["errors"] == {"seq_len"}
    api.dsa_plan_rows(st.plan(api))
    st.check(api, ref)


def test_extreme_lengths_are_refused(api):
    big = 2 ** 31 - 1
    st = State(5, 4, 8, 40, 16, 6)
    st.held[:] = [0, big, -big, 0, 0]
    st.d_held.copy_(dev(st.held))
    st.lengths([big, 8, 8, -big, 8], [1, 1, 1, -big, 8])
    ref = st.expect()
    api.dsa_plan_rows(st.plan(api))
    st.check(api, ref)


def test_more_rows_than_the_buffers_hold(api):
    st = State(4, 8, 8, 40, 10, 8)
    st.lengths([4, 5, 6, 7], [4, 5, 6, 7])
    ref = st.expect()
    assert ref["errors"] == {"rows"} and len(ref["positions"]) == 10
    api.dsa_plan_rows(st.plan(api))
    st.check(api, ref)


def served(api, st):
    # The lengths that the attention is given; the rest of the plan as it is without.
    out = torch.full((len(st.held) + 1,), MARK, dtype=torch.int32, device="cuda")
    ref = st.expect()
    api.dsa_plan_rows(api.make_plan(
        st.d_lens, st.d_new, st.d_held, st.d_held_out, st.d_table, st.block, st.d_free, st.d_in, st.d_out,
        st.row_start, st.positions, st.slots, st.row_lens, st.row_table, st.row_seq, served_lens=out[:-1]))
    st.check(api, ref)
    assert out[-1] == MARK
    return out[:-1].tolist()


def test_served_lengths_of_refused_requests(api):
    st = State(6, 8, 4, 12, 20, 4, free=7)               # as in the test of refusals in order
    st.held[3], st.held[5] = 1, 4
    st.table[3, 0], st.table[5, :4] = 7, [8, 9, 10, 11]
    st.d_table.copy_(dev(st.table))
    st.d_held.copy_(dev(st.held))
    st.lengths([12, 16, 9, 4, 1, 8], [4, 3, 2, 1, 1, 0])
    assert served(api, st) == [12, 16, 0, 4, 0, 8]


def test_served_lengths_of_invalid_requests(api):
    st = State(9, 4, 8, 40, 16, 6)
    st.held[:] = [1, 1, 1, 1, 1, -5, 9, 0, 0]
    for s in (0, 1, 2, 3, 4):
        st.table[s, 0] = 30 + s
    st.d_table.copy_(dev(st.table))
    st.d_held.copy_(dev(st.held))
    st.lengths([9, 9, 2, 30, 33, 8, 8, 20, -3], [1, -1, 3, 17, 2, 1, 1, 4, 0])
    assert served(api, st) == [9, 0, 0, 0, 0, 0, 0, 20, 0]


@pytest.mark.parametrize("seqs", [1, 33, 1100, 8192])
def test_served_lengths_of_served_requests(api, seqs):
    st = State(seqs, 3, 4, seqs * 3, 9000, 15)
    rng = np.random.default_rng(seqs)
    st.lengths(rng.integers(1, 13, seqs), rng.integers(0, 2, seqs))
    assert served(api, st) == st.lens.tolist()


@pytest.mark.parametrize("seqs, width, block, rows, row_table, row_seq, new", [
    (1, 1, 64, 1, True, True, 0), (1, 513, 64, 9, True, True, 1), (3, 40, 5, 64, True, True, 7),
    (3, 40, 5, 64, False, True, 7), (3, 40, 5, 64, True, False, 21), (33, 17, 16, 300, True, True, 9),
    (700, 257, 16, 20000, True, True, 20), (700, 1031, 16, 1403, True, True, 2), (4, 8, 8, 10, True, True, 5)])
def test_rows_behind_the_last_made_empty(api, seqs, width, block, rows, row_table, row_seq, new):
    # (the last case has more rows than the buffers hold)
    rng = np.random.default_rng(rows)
    st = State(seqs, width, block, seqs * width, rows, 16, stride=width + 2, row_table=row_table, row_seq=row_seq)
    n = rng.integers(new // 2, new + 1, seqs)
    st.lengths(np.minimum(n + rng.integers(0, width * block, seqs), width * block), n)
    ref = st.expect()
    tail = rows - len(ref["positions"])
    api.dsa_plan_rows(api.make_plan(
        st.d_lens, st.d_new, st.d_held, st.d_held_out, st.d_table, st.block, st.d_free, st.d_in, st.d_out,
        st.row_start, st.positions, st.slots, st.row_lens, st.row_table, st.row_seq, empty_tail=True))
    for name, empty in (("positions", 0), ("slots", -1), ("row_lens", 0), ("row_seq", -1)):
        ref[name] = ref[name] + [empty] * tail
    ref["row_table"] = ref["row_table"] + [[-1] * width] * tail
    st.check(api, ref)


def test_bad_free_counts(api):
    for count in (-1, 41):
        st = State(2, 4, 8, 40, 16, 9)
        st.d_in[0] = count
        st.count = 0
        st.lengths([8, 0], [8, 0])
        ref = st.expect()
        api.dsa_plan_rows(st.plan(api))
        st.check(api, ref)
    # Blocks given back past the capacity (a block freed twice) are dropped.
    st = State(1, 4, 8, 3, 4, 9)
    st.held[:] = 2
    st.table[0, :2] = [5, 6]
    st.d_table.copy_(dev(st.table))
    st.d_held.copy_(dev(st.held))
    st.lengths([0], [0])
    ref = dict(st.expect(), errors={"free"})
    ref["free"] = ref["free"][:3]
    api.dsa_plan_rows(st.plan(api))
    st.check(api, ref)


def test_captured_and_replayed_in_place(api):
    # One graph, replayed with other lengths: a decode loop's own bookkeeping.
    st = State(4, 16, 4, 64, 8, 10, in_place=True)
    plan, lens = st.plan(api), np.zeros(4, np.int64)
    st.lengths(lens, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        api.dsa_plan_rows(plan)
    for step in range(12):
        new = np.array([1, step % 3, 2 if step % 2 else 0, 1])
        lens = lens + new
        if step == 7:
            lens[2], new[2] = 0, 0
        st.lengths(lens, new)
        ref = st.expect()
        for t in (st.positions, st.slots, st.row_lens, st.row_seq, st.row_all):
            t.fill_(MARK)
        g.replay()
        st.check(api, ref)
        st.advance(ref)


def test_on_another_stream(api):
    st = State(40, 30, 16, 1300, 400, 12)
    rng = np.random.default_rng(0)
    new = rng.integers(0, 10, 40)
    st.lengths(rng.integers(10, 400, 40), new)
    plan, s = st.plan(api), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.dsa_plan_rows(plan, stream=s)
    st.check(api, st.expect())


def test_binding_checks(api):
    st = State(3, 4, 8, 10, 6, 1)
    plan = st.plan(api)
    make = lambda **kw: api.make_plan(**{**dict(  # noqa: E731
        seq_lens=st.d_lens, new_tokens=st.d_new, held_in=st.d_held, held_out=st.d_held_out,
        block_table=st.d_table, block_size=8, free_blocks=st.d_free, free_in=st.d_in,
        free_out=st.d_out, row_start=st.row_start, positions=st.positions, slots=st.slots,
        row_lens=st.row_lens, row_table=st.row_table, row_seq=st.row_seq), **kw})
    assert make().seqs == plan.seqs
    for kw in (dict(seq_lens=st.d_lens.long()), dict(slots=st.row_lens), dict(held_in=st.d_held[:2]),
               dict(row_start=st.positions), dict(free_out=st.d_out[:1]), dict(row_seq=st.row_seq[:5]),
               dict(row_table=st.row_table[:, :3]), dict(block_table=st.d_table.t()),
               dict(positions=st.positions.cpu()), dict(free_blocks=st.d_table)):
        with pytest.raises(ValueError):
            make(**kw)
    with pytest.raises(api.DsaError):
        api.dsa_plan_rows(make(block_size=0))


def test_binding_checks_of_the_served_lengths(api):
    st = State(3, 4, 8, 10, 6, 1)
    for bad in (st.d_lens[:2], st.d_lens.long(), st.d_lens.cpu()):
        with pytest.raises(ValueError, match="served_lens"):
            api.make_plan(st.d_lens, st.d_new, st.d_held, st.d_held_out, st.d_table, 8, st.d_free, st.d_in,
                          st.d_out, st.row_start, st.positions, st.slots, st.row_lens, served_lens=bad)
