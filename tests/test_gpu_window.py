"""Softmax decode over a sliding window with sinks, against the float64 definition.

Every page of the pool that a call must not read, and every token it must not
use, holds NaN or infinity; page-table entries outside the window and the sinks
are -1 or out of range.
"""
import math

import numpy as np
import pytest
import torch

from oracle import ranges
from sparse_long_context_min_b200 import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Cache:
    """Ragged sequences in a permuted pool, poisoned outside what `visible` names."""

    def __init__(self, lens, H_q, H_kv, d, ps, dtype, visible=None, seed=0, spread=1.0, table_pad=2):
        g = torch.Generator().manual_seed(seed)
        self.H_q, self.H_kv, self.d, self.ps, self.dtype = H_q, H_kv, d, ps, dtype
        self.lens = list(lens)
        P = [-(-max(L, 0) // ps) for L in lens]
        num = sum(P) + 2
        max_pages = max(max(P), 1) + table_pad
        perm = torch.randperm(num, generator=g)
        k = torch.full((num, H_kv, ps, d), float("nan"))
        v = torch.full((num, H_kv, ps, d), float("inf"))
        table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
        table[:, -1] = num + 7                         # never to be read
        self.keys, self.vals = [], []
        at = 0
        for b, L in enumerate(lens):
            L = max(L, 0)
            kk = (torch.randn(L, H_kv, d, generator=g) * spread).to(dtype).float()
            vv = torch.randn(L, H_kv, d, generator=g).to(dtype).float()
            self.keys.append(kk.double().numpy())
            self.vals.append(vv.double().numpy())
            see = np.arange(L) if visible is None else visible(L)
            for p in sorted(set((np.asarray(see) // ps).tolist())):
                table[b, p] = perm[at + p]
            for t in np.asarray(see).tolist():
                ph = int(perm[at + t // ps])
                k[ph, :, t % ps] = kk[t]
                v[ph, :, t % ps] = vv[t]
            at += P[b]
        self.q = torch.randn(len(lens), H_q, d, generator=g)
        f = torch.zeros(num, H_kv, d, device="cuda")
        z = f.to(dtype)
        self.pool = B.Pool(k.to(dtype).cuda(), v.to(dtype).cuda(), z, z, f, f,
                           torch.zeros(num, dtype=torch.int32, device="cuda"))
        self.table = table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(d)

    def check(self, out, lse, tokens):
        """out and lse against the definition over tokens(b) of every sequence."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, B.status_string(int(self.status.item()))
        out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
        G = self.H_q // self.H_kv
        scale = float(np.float32(self.scale))
        worst = 0.0
        for b in range(len(self.lens)):
            t = tokens(b)
            for g in range(self.H_kv):
                h = slice(g * G, (g + 1) * G)
                q, k, v = self.q[b, h].numpy(), self.keys[b][t, g], self.vals[b][t, g]
                o, l = ranges.softmax_rows(q, k, v, scale)
                eo, el = ranges.error_bound(q, k, v, scale, split=self.dtype == BF16)
                assert np.all(np.abs(out[b, h] - o) <= eo + 1e-30), (b, g, np.abs(out[b, h] - o).max(), eo.min())
                if len(t) == 0:
                    assert np.all(out[b, h] == 0) and np.all(lse[b, h] == -np.inf)
                else:
                    assert np.all(np.abs(lse[b, h] - l) <= el), (b, g, np.abs(lse[b, h] - l).max(), el.min())
                    worst = max(worst, float((np.abs(out[b, h] - o) / eo).max()))
        return worst


def run_window(c, window, sinks, workspace=None, stream=None, out=None, lse=None):
    n = len(c.lens)
    ws = B.workspace_size(B.OP_WINDOW_SOFTMAX, n, c.H_q, c.H_kv, c.table.shape[1], 0, c.ps, c.d)
    workspace = torch.full((ws,), 255, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    out = torch.full((n, c.H_q, c.d), float("nan"), device="cuda") if out is None else out
    lse = torch.full((n, c.H_q), float("nan"), device="cuda") if lse is None else lse
    B.window_softmax_decode(c.pool, c.q.cuda(), c.table, c.seq_lens, window, sinks, c.scale, out, workspace, c.status,
                            lse_out=lse, stream=stream)
    return out, lse


def check_window(c, window, sinks):
    out, lse = run_window(c, window, sinks)
    return c.check(out, lse, lambda b: ranges.window_tokens(c.lens[b], window, sinks))


SHAPES = [(4, 1, 64, 16, F32), (8, 1, 128, 64, F32), (2, 2, 128, 16, F32), (16, 2, 64, 64, F32),
          (32, 8, 128, 64, BF16), (8, 1, 128, 16, BF16), (3, 3, 64, 64, BF16), (10, 5, 64, 16, BF16),
          (16, 2, 128, 64, BF16), (16, 2, 64, 16, BF16)]


@pytest.mark.parametrize("H_q,H_kv,d,ps,dtype", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (64, 64), (333, 17), (5000, 0)])
def test_window_matches_definition(H_q, H_kv, d, ps, dtype, window, sinks):
    lens = [0, 1, ps - 1, ps, ps + 1, 63, 64, 65, window, window + sinks, window + sinks + 1, 700, 1301]
    c = Cache(lens, H_q, H_kv, d, ps, dtype, visible=lambda L: ranges.window_tokens(L, window, sinks),
              seed=window + sinks)
    check_window(c, window, sinks)


def test_window_of_int32_range():
    c = Cache([5, 300, 0, 129], 8, 2, 64, 16, BF16)
    check_window(c, 2 ** 31 - 1, 0)
    check_window(c, 1, 2 ** 31 - 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_window_large_scores(dtype):
    """Scores of several hundred: the running maximum moves often and weights underflow."""
    c = Cache([900, 64, 2049], 8, 2, 128, 64, dtype, spread=40.0, seed=3)
    check_window(c, 1500, 3)


@pytest.mark.parametrize("d,ps,spread", [(64, 64, 1.0), (64, 64, 20.0), (128, 16, 3.0)])
def test_window_long_shares(d, ps, spread):
    """Enough tiles that a CTA has more than 32 of one unit: its accumulators are emptied on the way."""
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(4200, 4600, size=24)]
    c = Cache(lens, 32, 8, d, ps, BF16, visible=lambda L: ranges.window_tokens(L, 4190, 5), seed=11, spread=spread)
    check_window(c, 4190, 5)


def test_window_many_sequences():
    """More sequences than a block has threads, half of them empty, and units cut anywhere."""
    rng = np.random.default_rng(5)
    lens = [int(x) if rng.random() < 0.5 else 0 for x in rng.integers(1, 260, size=701)]
    c = Cache(lens, 2, 1, 64, 16, BF16, seed=9)
    check_window(c, 150, 5)
    c = Cache(lens[:399], 2, 1, 64, 16, F32, seed=10)
    check_window(c, 150, 5)


def test_all_rows_empty():
    c = Cache([0, 0, -3], 4, 1, 64, 16, BF16)
    out, lse = run_window(c, 10, 2)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_same_bits_on_a_side_stream_and_in_two_graphs_sharing_a_workspace():
    a = Cache([4000, 77, 1200], 32, 8, 128, 64, BF16, seed=1)
    b = Cache([300, 9000], 32, 8, 128, 64, BF16, seed=2)
    ws = torch.full((max(B.workspace_size(B.OP_WINDOW_SOFTMAX, len(c.lens), 32, 8, c.table.shape[1], 0, 64, 128)
                         for c in (a, b)),), 255, dtype=torch.uint8, device="cuda")
    ref = [[x.clone() for x in run_window(c, 2500, 4)] for c in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_window(a, 2500, 4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0][0]) and torch.equal(got[1], ref[0][1])
    graphs, outs = [], []
    for c in (a, b):
        c.q = c.q.cuda()
        o = torch.empty(len(c.lens), 32, 128, device="cuda"), torch.empty(len(c.lens), 32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_window(c, 2500, 4, workspace=ws, out=o[0], lse=o[1])
        graphs.append(g)
        outs.append(o)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])
    graphs.clear()


def test_rows_behind_the_batch_and_pinned_outputs():
    c = Cache([500, 20], 8, 2, 128, 64, BF16, seed=4)
    big = torch.full((4, 8, 128), 7.0, device="cuda")
    ref, _ = run_window(c, 100, 4, out=big)
    torch.cuda.synchronize()
    assert bool((big[2:] == 7.0).all())
    host = torch.zeros(2, 8, 128).pin_memory()
    run_window(c, 100, 4, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, ref[:2].cpu())


def test_bad_pages_and_lengths_are_reported():
    for fault in ("page", "length"):
        c = Cache([300, 200], 8, 2, 64, 16, BF16, seed=6)
        if fault == "page":
            c.table[0, 18] = c.pool.num_phys           # the page of token 299
        else:
            c.seq_lens[1] = c.table.shape[1] * 16 + 1  # longer than its table row
        out, lse = run_window(c, 50, 4)
        torch.cuda.synchronize()
        assert int(c.status.item()) == B.DEVICE_BOUNDS
        # the other sequence is as it should be
        c.status.zero_()
        b = 1 if fault == "page" else 0
        t = ranges.window_tokens(c.lens[b], 50, 4)
        o, _ = ranges.softmax_rows(c.q[b, :4].numpy(), c.keys[b][t, 0], c.vals[b][t, 0], c.scale)
        assert np.abs(out[b, :4].cpu().double().numpy() - o).max() < 1e-4
