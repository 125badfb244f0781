"""How exact the decode operators are in the 2-norm, where one CTA sums a long
sequence by itself: against float64, with what the arithmetic allows.

Half of the inputs have values around 1, whose sums do not cancel, so that a sum
that loses a little at every step shows it in full.
"""
import math

import numpy as np
import pytest
import torch

from sparse_long_context_min_b200 import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def tolerance(d, adds, parts, cut):
    """Relative 2-norm error for scores of one nat rms.  Independent errors join as the root of their squares:
      scores: the product's parts * d / 16 steps (fp32 caches: d roundings) of the tensor cores each cut off half
        a step of 2^-23 on average, all to the same side;
      the query and the weights in two bf16 parts: of a value in [1, 2) the first leaves a rest within 2^-8, whose
        rounding lies within 2^-8 2^e, e the rest's exponent, and 4^e is 2^-16 / 7 on average: 2^-16 / sqrt(21) rms,
        1 / sqrt(2) of that relative to the value, and two such errors (three parts: 2^-26, nothing beside the rest);
      weights: exp2 to two steps of 2^-23;
      output: `cut` steps of the tensor cores, each cut off half a step of the whole sum, between two rounded
        additions, and `adds` of those, 2^-25 rms each.
    Half as much again, since one output row is one sample."""
    scores = (parts * d / 16 if parts else math.sqrt(d)) * 2.0 ** -24
    split = 2.0 ** -16 / math.sqrt(21) if parts == 2 else 0.0
    return 1.5 * math.sqrt(scores ** 2 + split ** 2 + 2.0 ** -44 + (cut * 2.0 ** -24) ** 2 + adds * 2.0 ** -50)


class Long:
    """Many sequences over the same pages, each with its own query."""

    def __init__(self, rows, L, G, H_kv, d, ps, dtype, around, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        pages = -(-L // ps)
        shape = (pages, H_kv, ps, d)
        k = torch.randn(shape, generator=g, device="cuda").to(dtype)
        v = (torch.rand(shape, generator=g, device="cuda") + 0.5 if around else
             torch.randn(shape, generator=g, device="cuda")).to(dtype)
        f = torch.zeros(pages, H_kv, d, device="cuda")
        z = f.to(dtype)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pool = B.Pool(k, v, z, z, f, f, torch.zeros(pages, **i32))
        self.rows, self.L, self.G, self.H_kv, self.d, self.ps = rows, L, G, H_kv, d, ps
        self.q = torch.randn(rows, G * H_kv, d, generator=g, device="cuda")
        self.table = torch.arange(pages, **i32).repeat(rows, 1).contiguous()
        self.lens = torch.full((rows,), L, **i32)
        self.status = torch.zeros(1, **i32)
        self.out = torch.full((rows, G * H_kv, d), float("nan"), device="cuda")
        self.lse = torch.full((rows, G * H_kv), float("nan"), device="cuda")
        self.scale = float(np.float32(1 / math.sqrt(d)))

    def workspace(self, op):
        n = B.workspace_size(op, self.rows, self.G * self.H_kv, self.H_kv, self.table.shape[1], 0, self.ps, self.d)
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def window(self, window, sinks=0):
        B.window_softmax_decode(self.pool, self.q, self.table, self.lens, window, sinks, self.scale, self.out,
                                self.workspace(B.OP_WINDOW_SOFTMAX), self.status, lse_out=self.lse)

    def prefix(self, starts, prefixes):
        # rows of the table so long that the prefix is read once a group
        entries = (64 << 20) // (self.ps * self.H_kv * self.d * 4) + 1
        pad = max(0, -(-entries // self.rows) - self.table.shape[1])
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.cat([self.table, torch.full((self.rows, pad), -1, **i32)], dim=1).contiguous()
        B.prefix_softmax_decode(self.pool, self.q, self.table, self.lens, torch.tensor(starts, **i32),
                                torch.tensor(prefixes, **i32), self.scale, self.out,
                                self.workspace(B.OP_PREFIX_SOFTMAX), self.status, lse_out=self.lse)

    def errors(self, rows, first=0):
        """Of the given rows over the tokens from `first` on: (largest 2-norm error of a head's output relative to
        it, largest error of lse)."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        worst, worst_lse = 0.0, 0.0
        for g in range(self.H_kv):
            k, v = (x[:, g].reshape(-1, self.d)[first:self.L].double().cpu().numpy()
                    for x in (self.pool.k_pool, self.pool.v_pool))
            for b in rows:
                h = slice(g * self.G, (g + 1) * self.G)
                x = self.scale * (self.q[b, h].double().cpu().numpy() @ k.T)
                m = x.max(axis=1, keepdims=True)
                e = np.exp(x - m)
                o = (e @ v) / e.sum(axis=1, keepdims=True)
                lse = m[:, 0] + np.log(e.sum(axis=1))
                diff = self.out[b, h].double().cpu().numpy() - o
                worst = max(worst, float((np.linalg.norm(diff, axis=1) / np.linalg.norm(o, axis=1)).max()))
                worst_lse = max(worst_lse, float(np.abs(self.lse[b, h].double().cpu().numpy() - lse).max()))
        return worst, worst_lse


SHAPES = [(1, 128, 64), (4, 128, 64), (8, 128, 64), (8, 64, 16), (4, 64, 16)]


@pytest.mark.parametrize("around", [False, True])
@pytest.mark.parametrize("G,d,ps", SHAPES)
def test_window_of_one_cta(G, d, ps, around):
    """600 sequences of 20001 tokens: each CTA has units of 313 tiles whole."""
    c = Long(600, 20001, G, 1, d, ps, BF16, around, seed=G + d)
    c.window(2 ** 31 - 1)
    o, lse = c.errors((0, 599))
    tol = tolerance(d, 313, 3, 2)
    print("window G=%d d=%d: %.2e (tolerance %.2e), lse %.2e" % (G, d, o, tol, lse))
    assert o <= tol and lse <= tol + 2.0 ** -20        # (lse is about 11: half a step is 2^-21)


@pytest.mark.parametrize("G,dtype", [(4, BF16), (8, BF16), (4, F32)])
def test_short_window(G, dtype):
    """The bf16 parts of the query and the weights are three: with two the error is 3.3e-6."""
    c = Long(64, 5000, G, 2, 128, 64, dtype, False, seed=3)
    c.window(1020, 8)
    c.L, tokens = 5000, np.r_[0:8, 3980:5000]
    torch.cuda.synchronize()
    k, v = (x.transpose(0, 1).reshape(2, -1, 128)[:, tokens].contiguous() for x in (c.pool.k_pool, c.pool.v_pool))
    c.pool.k_pool, c.pool.v_pool, c.L = k.reshape(1, 2, -1, 128), v.reshape(1, 2, -1, 128), 1028
    o, lse = c.errors((0, 31, 63))
    tol = tolerance(128, 17, 3, 2) if dtype == BF16 else tolerance(128, 1028, 0, 0)
    print("short window G=%d %s: %.2e (tolerance %.2e), lse %.2e" % (G, dtype, o, tol, lse))
    assert o <= tol and lse <= tol + 2.0 ** -20


@pytest.mark.parametrize("around", [False, True])
@pytest.mark.parametrize("G,d,ps", SHAPES)
def test_own_tokens_of_one_cta(G, d, ps, around):
    """The same behind a prefix of nothing, where the query and the weights enter in two parts."""
    c = Long(600, 20001, G, 1, d, ps, BF16, around, seed=G + d)
    c.prefix([0, 300, 600], [0, 0])
    o, lse = c.errors((0, 599))
    tol = tolerance(d, 313, 2, 1)
    print("own tokens G=%d d=%d: %.2e (tolerance %.2e), lse %.2e" % (G, d, o, tol, lse))
    assert o <= tol and lse <= tol + 2.0 ** -20


@pytest.mark.parametrize("around", [False, True])
@pytest.mark.parametrize("G,n,d,ps", [(4, 2, 128, 64), (8, 16, 128, 64), (8, 40, 128, 16), (2, 3, 64, 16)])
def test_long_prefixes_of_one_cta(G, n, d, ps, around):
    """160 groups behind 100000 tokens: a CTA walks more than 1500 blocks of a unit (d 64, page 16: d / 16 score steps
    a part).  Of each 128 blocks a set's accumulator takes 64, 8 steps each, into a sum that grows from nothing: 256
    cut-offs of the whole sum on average."""
    c = Long(160 * n, 100000, G, 1, d, ps, BF16, around, seed=n)
    c.prefix(list(range(0, 160 * n + 1, n)), [100000] * 160)
    o, lse = c.errors((0, n - 1, 71 * n + n // 2, 160 * n - 1))
    tol = tolerance(d, 13, 2, 256)
    print("prefix G=%d x %d d=%d: %.2e (tolerance %.2e), lse %.2e" % (G, n, d, o, tol, lse))
    assert o <= tol and lse <= tol + 2.0 ** -20
