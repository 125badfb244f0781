"""Copying, forking, freeing, reserving and compacting pages against the oracle:
tables, counts and lengths entry by entry, page contents bit by bit."""
import random

import pytest
import torch

from oracle import manage
from sparse_long_context_min_b200 import binding as B

pytestmark = pytest.mark.gpu

NAMES = ("k_pool", "v_pool", "kmin", "kmax", "mean", "m2", "count")


class Both:
    """The same state on the GPU and in the oracle; page contents are the id that a page started with."""

    def __init__(self, num, rows, max_pages, ps=16, H_kv=2, d=64, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f = dict(generator=g, device="cuda")
        kv = torch.randn(2, num, H_kv, ps, d, **f).to(dtype)
        mm = torch.randn(2, num, H_kv, d, **f).to(dtype)
        ff = torch.randn(2, num, H_kv, d, **f)
        count = torch.randint(0, ps + 1, (num,), dtype=torch.int32, **f)
        self.pool = B.Pool(kv[0], kv[1], mm[0], mm[1], ff[0], ff[1], count)
        self.first = {n: getattr(self.pool, n).clone() for n in NAMES}
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(num, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.live = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = B.workspace_size(B.OP_PAGES, rows, 0, 0, 0, num, 0, 0)
        self.ws = torch.full((ws,), 255, dtype=torch.uint8, device="cuda")
        self.o = manage.State(num, rows, max_pages, ps)
        self.o.data = list(range(num))
        self.ps = ps

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def set_lens(self, lens):
        self.o.lens = list(lens)
        self.lens.copy_(self.i32(lens))

    def check(self, errors):
        torch.cuda.synchronize()
        got = int(self.status.item())
        want = {B.DEVICE_BOUNDS if e == "bounds" else B.NO_PAGES for e in errors}
        assert got in want if want else got == 0, (got, errors)
        self.status.zero_()
        assert self.table.tolist() == self.o.table
        assert self.ref.tolist() == self.o.ref
        assert self.lens.tolist() == self.o.lens
        at = torch.tensor(self.o.data, device="cuda")
        for n in NAMES:
            x, y = getattr(self.pool, n), self.first[n][at]
            assert torch.equal(x.view(torch.uint8) if x.dim() > 1 else x, y.view(torch.uint8) if y.dim() > 1 else y), n

    def reserve(self, lens):
        B.reserve_pages(self.pool, self.ref, self.table, self.lens, self.i32(lens), self.ws, self.status)
        self.check(manage.reserve(self.o, lens))

    def fork(self, src, dst):
        B.fork_sequences(self.pool, self.ref, self.table, self.lens, self.i32(src), self.i32(dst), self.ws, self.status)
        self.check(manage.fork(self.o, src, dst))

    def free(self, rows, window=None, sinks=0):
        B.free_pages(self.pool, self.ref, self.table, self.lens, None if rows is None else self.i32(rows), self.status,
                     window=window, sinks=sinks)
        self.check(manage.free(self.o, rows, window, sinks))

    def compact(self):
        B.compact_pages(self.pool, self.ref, self.table, self.live, self.ws, self.status)
        live, errors = manage.compact(self.o)
        self.check(errors)
        assert int(self.live.item()) == live

    def copy(self, src, dst):
        B.copy_pages(self.pool, self.i32(src), self.i32(dst), self.ws, self.status)
        self.check(manage.copy(self.o, src, dst))


@pytest.mark.parametrize("num,rows,max_pages,ps,H_kv,d,dtype", [
    (50, 7, 9, 16, 1, 64, torch.float32), (64, 7, 20, 64, 3, 128, torch.bfloat16),
    (33, 4, 11, 16, 8, 128, torch.bfloat16), (700, 12, 70, 16, 1, 64, torch.bfloat16)])
def test_random_traffic(num, rows, max_pages, ps, H_kv, d, dtype):
    rng = random.Random(num)
    s = Both(num, rows, max_pages, ps, H_kv, d, dtype, seed=num)
    top = max_pages * ps
    for step in range(40):
        what = rng.choice(["reserve", "reserve", "fork", "fork", "free", "trim", "compact", "copy"])
        if what == "reserve":
            want = [rng.choice([0, L, min(top, L + rng.randrange(1, 4 * ps))]) for L in s.o.lens]
            s.reserve(want)
            # the rows that got their pages are filled
            s.set_lens([max(L, w) if all(e >= 0 for e in s.o.table[b][-(-L // ps):-(-w // ps)]) else L
                        for b, (L, w) in enumerate(zip(s.o.lens, want))])
        elif what == "fork":
            names = rng.sample(range(rows), rng.randrange(2, rows + 1))
            n = rng.randrange(1, len(names))
            s.fork([rng.choice(names[n:]) for _ in range(n)], names[:n])
        elif what == "free":
            s.free([rng.randrange(rows) for _ in range(2)])
        elif what == "trim":
            s.free(rng.choice([None, [0, rows - 1]]), window=rng.randrange(3 * ps), sinks=rng.randrange(2 * ps))
        elif what == "compact":
            s.compact()
        else:
            ids = rng.sample(range(num), 12)
            s.copy(ids[:6] + [ids[0]], ids[6:] + [ids[5]] if rng.random() < 0.3 else ids[6:] + [ids[0]])


def test_refusals_leave_rows_alone():
    s = Both(40, 6, 6)
    s.reserve([50, 33, 16, 0, 0, 0])
    s.set_lens([50, 33, 16, 0, 0, 0])
    s.fork([0, 1], [3, 3])                    # one destination twice
    s.fork([0, 1], [1, 4])                    # a destination that is a source
    s.fork([0, -1, 6, 2], [3, 4, 5, 6])       # rows out of range
    s.fork([0, 0, 0], [3, 4, 5])
    s.free([6, -1, 3])
    s.copy([0, 1, 40, -1, 2, 5], [20, 20, 3, 4, 1, 5])
    s.reserve([0, 0, 0, 0, 0, 6 * 16 + 1])    # more than a table row holds
    s.set_lens([50, 33, 97, 0, 0, 0])
    s.fork([2, 0], [3, 4])                    # a length beyond the table
    s.set_lens([50, 33, 16, 0, 50, 50])
    s.table[1, 0] = s.o.table[1][0] = 40      # an entry beyond the pool
    s.fork([1], [3])
    s.free([1, 3])


def test_runs_out_of_pages():
    s = Both(9, 6, 6)
    s.reserve([40, 20, 0, 0, 0, 0])           # 3 + 2 pages
    s.set_lens([40, 20, 0, 0, 0, 0])
    s.reserve([41, 0, 33, 17, 16, 0])         # 0 + 3 pages fit, 2 do not, and nothing after them
    s.set_lens([40, 20, 33, 0, 0, 0])
    s.fork([0, 1], [3, 4])                    # one page left for two forks
    s.free(None)
    assert s.o.ref == [0] * 9


def test_counts_that_do_not_cover_the_table_are_reported():
    s = Both(12, 3, 4)
    s.reserve([30, 0, 0])
    s.ref[1] = s.o.ref[1] = 0
    s.free([0])


def test_large_pool_and_long_rows():
    """More pages than a counting CTA has threads, rows of several chunks."""
    rng = random.Random(3)
    s = Both(70001, 5, 2500, 16, 1, 64)
    s.reserve([39000, 5, 12345, 0, 0])
    s.set_lens([39000, 5, 12345, 0, 0])
    s.fork([0, 2], [3, 4])
    s.free([0])
    s.reserve([16 * 2500, 0, 0, 0, 0])
    s.set_lens([16 * 2500] + s.o.lens[1:])
    s.free([2])
    s.compact()
    s.free(None, window=1000, sinks=40)
    # pages in use near the end of the pool
    s.o.ref[70000] = s.o.ref[69000] = 1
    s.ref[70000] = s.ref[69000] = 1
    s.o.table[1][7], s.o.table[1][9] = 70000, 69000
    s.table[1, 7], s.table[1, 9] = 70000, 69000
    s.compact()
    ids = rng.sample(range(70001), 3000)
    s.copy(ids[:1500], ids[1500:])


def test_wide_tables():
    """More entries than the counting cluster takes along: releasing and counting are launches of their own."""
    s = Both(3000, 3, 17000, 16, 1, 64)
    s.reserve([20000, 0, 33])
    s.set_lens([20000, 0, 33])
    s.fork([0, 0], [1, 2])
    s.set_lens([20000, 20000, 19999])
    s.fork([2, 2], [0, 1])
    s.fork([0, 2], [0, 1])                    # a destination that is a source
    s.reserve([17000 * 16 + 1, 24000, 24001])
    s.reserve([0, 39000, 47000])              # more than there are
    s.free([0, 2])
    s.compact()


def test_many_forks_of_short_rows():
    """More forks than warps of the counting cluster, some refused."""
    rows = 700
    s = Both(1500, rows, 4)
    s.reserve([37 if b < 300 else 0 for b in range(rows)])
    s.set_lens([37 if b < 300 else 0 for b in range(rows)])
    rng = random.Random(8)
    dst = rng.sample(range(300, rows), 290)
    s.fork([rng.randrange(300) for _ in dst] + [5], dst + [dst[0]])
    s.fork([rng.randrange(300) for _ in range(40)], rng.sample(range(300, rows), 40))


def test_nothing_to_do():
    s = Both(8, 2, 4)
    s.compact()
    s.free([])
    s.fork([], [])
    s.copy([], [])
    s.reserve([0, 0])
    s.reserve([64, 64])
    s.set_lens([64, 64])
    s.compact()


def test_graph_of_a_beam_step():
    """fork, free with a window and compact captured once and replayed: each replay
    acts on the state that the last one left."""
    s = Both(60, 6, 8)
    s.reserve([70, 45, 0, 0, 0, 0])
    s.set_lens([70, 45, 0, 0, 0, 0])
    src, dst = s.i32([0, 1, 1]), s.i32([2, 3, 5])
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        B.fork_sequences(s.pool, s.ref, s.table, s.lens, src, dst, s.ws, s.status)
        B.free_pages(s.pool, s.ref, s.table, s.lens, None, s.status, window=20, sinks=16)
        B.compact_pages(s.pool, s.ref, s.table, s.live, s.ws, s.status)
    for _ in range(3):
        g.replay()
        manage.fork(s.o, [0, 1, 1], [2, 3, 5])
        manage.free(s.o, None, 20, 16)
        manage.compact(s.o)
        s.check(set())
    del g
