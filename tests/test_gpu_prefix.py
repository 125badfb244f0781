"""Softmax decode over shared prefixes against the float64 definition.

The pages of a group's prefix are shared in its page-table rows; everything that
a call must not use holds NaN or infinity.
"""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import ranges
from sparse_long_context_min_b200 import binding as B
from test_gpu_window import Cache

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Shared(Cache):
    """groups: (prefix length, lengths of its sequences); a sequence shorter than the
    prefix holds only its first tokens.  With `wide` the table's rows are so long
    that the library shares the prefix's reading (small calls read it for each
    sequence)."""

    def __init__(self, groups, H_q, H_kv, d, ps, dtype, seed=0, spread=1.0, wide=True):
        lens = [L for _, ls in groups for L in ls]
        super().__init__(lens, H_q, H_kv, d, ps, dtype, seed=seed, spread=spread)
        table = self.table.cpu()
        b = 0
        self.starts, self.prefixes = [0], []
        for prefix, ls in groups:
            # the longest row holds the whole prefix
            first = max(range(b, b + len(ls)), key=lambda i: lens[i], default=b)
            for i in range(b, b + len(ls)):
                n = min(prefix, max(lens[i], 0))
                self.keys[i][:n], self.vals[i][:n] = self.keys[first][:n], self.vals[first][:n]
                table[i, :min(prefix, max(lens[first], 0)) // ps] = table[first, :min(prefix, max(lens[first], 0)) // ps]
                # the tokens of a page that the prefix ends in are copied
                for t in range(n // ps * ps, n):
                    src, dst = int(table[first, t // ps]), int(table[i, t // ps])
                    self.pool.k_pool[dst, :, t % ps] = self.pool.k_pool[src, :, t % ps]
                    self.pool.v_pool[dst, :, t % ps] = self.pool.v_pool[src, :, t % ps]
            b += len(ls)
            self.starts.append(b)
            self.prefixes.append(prefix)
        if wide:
            entries = (64 << 20) // (ps * H_kv * d * 2 * (2 if dtype == BF16 else 4)) + 1
            pad = max(0, -(-entries // max(len(lens), 1)) - table.shape[1])
            table = torch.cat([table, torch.full((len(lens), pad), -1, dtype=torch.int32)], dim=1)
        self.table = table.cuda()

    def run(self, workspace=None, out=None, lse=None, stream=None, starts=None, prefixes=None):
        n = len(self.lens)
        if workspace is None:
            ws = B.workspace_size(B.OP_PREFIX_SOFTMAX, n, self.H_q, self.H_kv, self.table.shape[1], 0, self.ps, self.d)
            workspace = torch.full((ws,), 255, dtype=torch.uint8, device="cuda")
        out = torch.full((n, self.H_q, self.d), float("nan"), device="cuda") if out is None else out
        lse = torch.full((n, self.H_q), float("nan"), device="cuda") if lse is None else lse
        i32 = dict(dtype=torch.int32, device="cuda")
        starts = torch.tensor(self.starts, **i32) if starts is None else starts
        prefixes = torch.tensor(self.prefixes, **i32) if prefixes is None else prefixes
        B.prefix_softmax_decode(self.pool, self.q.cuda(), self.table, self.seq_lens, starts, prefixes, self.scale, out,
                                workspace, self.status, lse_out=lse, stream=stream)
        return out, lse

    def verify(self, **kw):
        out, lse = self.run(**kw)
        return self.check(out, lse, lambda b: np.arange(max(self.lens[b], 0)))


SHAPES = [(32, 8, 128, 64, BF16), (4, 4, 64, 16, BF16), (4, 1, 64, 16, F32), (8, 1, 128, 16, BF16),
          (16, 2, 64, 64, BF16), (16, 2, 128, 64, F32), (10, 5, 128, 64, BF16), (2, 2, 128, 16, F32)]


@pytest.mark.parametrize("H_q,H_kv,d,ps,dtype", SHAPES)
@pytest.mark.parametrize("prefix", [0, 1, 16, 65, 128, 129, 700])
def test_prefix_matches_definition(H_q, H_kv, d, ps, dtype, prefix):
    tails = [1, 0, 17, 64, 300]
    for wide in (True, False):
        c = Shared([(prefix, [prefix + t for t in tails])], H_q, H_kv, d, ps, dtype, seed=prefix, wide=wide)
        c.verify()


@pytest.mark.parametrize("H_q,H_kv,d,ps,dtype", SHAPES[:4])
def test_groups_of_every_kind(H_q, H_kv, d, ps, dtype):
    """Lone sequences, empty rows, sequences shorter than their prefix, groups without a
    prefix, an empty group, and more than one row tile."""
    c = Shared([(500, [600]), (333, [333, 0, 400, 340]), (200, [90, 700, 250]), (0, [50, 60]), (100, []),
                (64, [64] * 40), (257, [0, 0]), (400, [0, 800])], H_q, H_kv, d, ps, dtype, seed=7)
    c.verify()


@pytest.mark.parametrize("d,ps,dtype", [(128, 64, BF16), (64, 16, BF16), (128, 16, F32), (64, 64, F32)])
def test_long_prefix_is_cut_between_ctas(d, ps, dtype):
    c = Shared([(9000, [9000 + 13 * i for i in range(3)]), (5000, [5001] * 37)], 16, 2, d, ps, dtype, seed=11)
    c.verify()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(dtype):
    """Scores of several hundred: the accumulators are rescaled often."""
    c = Shared([(1500, [1500, 1600, 1700, 2000])], 8, 2, 128, 64, dtype, seed=13, spread=40.0)
    c.verify()


def test_rows_outside_the_groups_share_nothing():
    c = Shared([(300, [400, 350, 420]), (10, [30, 40])], 8, 2, 64, 16, BF16, seed=5)
    i32 = dict(dtype=torch.int32, device="cuda")
    c.verify(starts=torch.tensor([1, 3], **i32), prefixes=torch.tensor([300], **i32))
    c.verify(starts=torch.zeros(1, **i32), prefixes=torch.zeros(0, **i32))


def test_first_row_of_a_group_has_left():
    """A freed row holds no pages: the shared ones are read through the next row."""
    c = Shared([(300, [0, 400, 350]), (70, [0, 0, 90, 80])], 8, 2, 64, 16, BF16, seed=5)
    c.table[0], c.table[3], c.table[4] = -1, -1, -1
    c.verify()


def test_bad_groups_and_pages_are_reported():
    i32 = dict(dtype=torch.int32, device="cuda")
    for starts, wide in itertools.product(([0, 6], [-1, 3], [4, 2], [0, 4, 0, 4, 0]), (True, False)):
        c = Shared([(300, [400, 350, 420, 310])], 8, 2, 64, 16, BF16, seed=5, wide=wide)
        prefixes = torch.tensor([300] * (len(starts) - 1), **i32)
        out, lse = c.run(starts=torch.tensor(starts, **i32), prefixes=prefixes)
        torch.cuda.synchronize()
        assert int(c.status.item()) == B.DEVICE_BOUNDS
        # clipped, and held ascending: no sequence is in two groups, and the results stand
        c.status.zero_()
        c.check(out, lse, lambda b: np.arange(c.lens[b]))
    c = Shared([(300, [400, 350, 420, 310])], 8, 2, 64, 16, BF16, seed=5)
    c.table[0, 3] = c.pool.num_phys
    c.run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == B.DEVICE_BOUNDS


def test_same_bits_again_and_in_two_graphs_sharing_a_workspace():
    a = Shared([(4000, [4100, 4077, 4000, 4900])], 32, 8, 128, 64, BF16, seed=1)
    b = Shared([(900, [1000, 901]), (70, [100, 80, 90])], 32, 8, 128, 64, BF16, seed=2)
    ws = torch.full((max(B.workspace_size(B.OP_PREFIX_SOFTMAX, len(c.lens), 32, 8, c.table.shape[1], 0, 64, 128)
                         for c in (a, b)),), 255, dtype=torch.uint8, device="cuda")
    ref = [[x.clone() for x in c.run()] for c in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = a.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0][0]) and torch.equal(got[1], ref[0][1])
    graphs, outs = [], []
    i32 = dict(dtype=torch.int32, device="cuda")
    for c in (a, b):
        c.q = c.q.cuda()
        st, pf = torch.tensor(c.starts, **i32), torch.tensor(c.prefixes, **i32)
        o = torch.empty(len(c.lens), 32, 128, device="cuda"), torch.empty(len(c.lens), 32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(workspace=ws, out=o[0], lse=o[1], starts=st, prefixes=pf)
        graphs.append(g)
        outs.append((o, st, pf))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, _, _), r in zip(outs, ref):
        assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])
    graphs.clear()
