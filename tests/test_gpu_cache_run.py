"""The cache calls together, as a serving loop makes them: room is reserved, a
prompt appended, its sequence forked, tokens appended to every fork, and the
batch decoded over the shared prefix and over a window; pages behind the window
are freed and the pool compacted, eagerly and from a captured graph."""
import math

import numpy as np
import pytest
import torch

from oracle import ranges
from sparse_long_context_min_b200 import binding as B

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, PS = 8, 2, 64, 16
WINDOW, SINKS = 40, 20


class Server:
    """Four rows in use, two that wait; rows are long enough that prefixes are read once."""

    def __init__(self, dtype):
        self.dtype = dtype
        self.rows, self.max_pages, self.num = 6, 2 * (2 if dtype == torch.bfloat16 else 1) * 700, 160
        f = dict(device="cuda")
        self.pool = B.Pool.allocate(self.num, H_KV, PS, D, dtype)
        i32 = dict(dtype=torch.int32, **f)
        self.table = torch.full((self.rows, self.max_pages), -1, **i32)
        self.ref = torch.zeros(self.num, **i32)
        self.lens = torch.zeros(self.rows, **i32)
        self.want = torch.zeros(self.rows, **i32)
        self.status = torch.zeros(1, **i32)
        self.live = torch.zeros(1, **i32)
        self.starts, self.prefixes = torch.tensor([0, 4], **i32), torch.tensor([0], **i32)
        n = max(B.workspace_size(B.OP_PREFIX_SOFTMAX, self.rows, H_Q, H_KV, self.max_pages, 0, PS, D),
                B.workspace_size(B.OP_WINDOW_SOFTMAX, self.rows, H_Q, H_KV, self.max_pages, 0, PS, D),
                B.workspace_size(B.OP_FULL_SOFTMAX, self.rows, H_Q, H_KV, self.max_pages, 0, PS, D),
                B.workspace_size(B.OP_PAGES, self.rows, 0, 0, self.max_pages, self.num, PS, D))
        self.ws = torch.full((n,), 255, dtype=torch.uint8, **f)
        self.q = torch.zeros(self.rows, H_Q, D, **f)
        self.k = torch.zeros(self.rows, H_KV, 1, D, dtype=dtype, **f)
        self.v = torch.zeros_like(self.k)
        self.out = {n: torch.zeros(self.rows, H_Q, D, **f) for n in ("prefix", "window", "full")}
        self.lse = {n: torch.zeros(self.rows, H_Q, **f) for n in ("prefix", "window")}
        self.scale = 1 / math.sqrt(D)
        self.keys = [np.zeros((0, H_KV, D)) for _ in range(self.rows)]
        self.vals = [np.zeros((0, H_KV, D)) for _ in range(self.rows)]

    def prompt(self, n, g):
        """n tokens into row 0, which the rows 1 to 3 then share."""
        self.want[0] = n
        B.reserve_pages(self.pool, self.ref, self.table, self.lens, self.want, self.ws, self.status)
        kv = torch.randn(2, 1, H_KV, n, D, generator=g).to(self.dtype)
        B.append_metadata(self.pool, kv[0].cuda(), kv[1].cuda(), self.table[:1], self.lens[:1], self.status)
        i32 = dict(dtype=torch.int32, device="cuda")
        B.fork_sequences(self.pool, self.ref, self.table, self.lens, torch.zeros(3, **i32),
                         torch.tensor([1, 2, 3], **i32), self.ws, self.status)
        self.prefixes.fill_(n)
        for b in range(4):
            self.keys[b], self.vals[b] = (x[0].transpose(0, 1).double().numpy() for x in kv)

    def step(self):
        """One token for each of the first four rows: room, append, decode, pages behind the window dropped from
        nobody's table but the last two rows'."""
        torch.add(self.lens[:4], 1, out=self.want[:4])
        B.reserve_pages(self.pool, self.ref, self.table, self.lens, self.want, self.ws, self.status)
        B.append_metadata(self.pool, self.k[:4], self.v[:4], self.table[:4], self.lens[:4], self.status)
        B.prefix_softmax_decode(self.pool, self.q, self.table, self.lens, self.starts, self.prefixes, self.scale,
                                self.out["prefix"], self.ws, self.status, lse_out=self.lse["prefix"])
        B.window_softmax_decode(self.pool, self.q, self.table, self.lens, WINDOW, SINKS, self.scale, self.out["window"],
                                self.ws, self.status, lse_out=self.lse["window"])

    def token(self, g):
        for x in (self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, generator=g).to(x.dtype))
        for b in range(4):
            self.keys[b] = np.concatenate([self.keys[b], self.k[b].transpose(0, 1).double().cpu().numpy()])
            self.vals[b] = np.concatenate([self.vals[b], self.v[b].transpose(0, 1).double().cpu().numpy()])

    def check(self, names=("prefix", "window"), rows=range(6)):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, B.status_string(int(self.status.item()))
        G = H_Q // H_KV
        for name in names:
            out, lse = self.out[name].double().cpu().numpy(), self.lse[name].double().cpu().numpy()
            for b in rows:
                L = len(self.keys[b])
                t = ranges.window_tokens(L, WINDOW, SINKS) if name == "window" else np.arange(L)
                for g in range(H_KV):
                    h = slice(g * G, (g + 1) * G)
                    q, k, v = self.q[b, h].cpu().numpy(), self.keys[b][t, g], self.vals[b][t, g]
                    scale = float(np.float32(self.scale))
                    o, l = ranges.softmax_rows(q, k, v, scale)
                    eo, el = ranges.error_bound(q, k, v, scale, split=self.dtype == torch.bfloat16)
                    assert np.all(np.abs(out[b, h] - o) <= eo + 1e-30), (name, b, g)
                    assert L == 0 or np.all(np.abs(lse[b, h] - l) <= el), (name, b, g)

    def counts_cover_the_table(self):
        torch.cuda.synchronize()
        held = self.table[self.table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=self.num).int(), self.ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("prompt", [1, 16, 100, 431])
def test_a_decode_run(dtype, prompt):
    g = torch.Generator().manual_seed(prompt)
    s = Server(dtype)
    s.prompt(prompt, g)
    s.counts_cover_the_table()
    for _ in range(20):
        s.token(g)
        s.step()
        s.check()
    s.counts_cover_the_table()
    # the existing full-cache decode sees the same sequences
    B.full_softmax_decode(s.pool, s.q, s.table, s.lens, s.scale, s.out["full"], s.ws, s.status)
    torch.cuda.synchronize()
    assert (s.out["full"] - s.out["prefix"]).abs().max() < 1e-4
    # pages behind the window go, what is left is packed, and the window's decode gives the same bits
    before = [x.clone() for x in (s.out["window"], s.lse["window"])]
    B.free_pages(s.pool, s.ref, s.table, s.lens, None, s.status, window=WINDOW, sinks=SINKS)
    s.counts_cover_the_table()
    B.compact_pages(s.pool, s.ref, s.table, s.live, s.ws, s.status)
    s.counts_cover_the_table()
    held = int((s.ref > 0).sum())
    assert int(s.live.item()) == held and bool((s.ref[:held] > 0).all())
    B.window_softmax_decode(s.pool, s.q, s.table, s.lens, WINDOW, SINKS, s.scale, s.out["window"], s.ws, s.status,
                            lse_out=s.lse["window"])
    torch.cuda.synchronize()
    assert torch.equal(before[0], s.out["window"]) and torch.equal(before[1], s.lse["window"])
    # everybody leaves: the rows are empty and every page is free
    B.free_pages(s.pool, s.ref, s.table, s.lens, None, s.status)
    torch.cuda.synchronize()
    assert int(s.ref.abs().sum()) == 0 and bool((s.table == -1).all()) and bool((s.lens == 0).all())
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_step_captured_and_replayed(dtype):
    g = torch.Generator().manual_seed(3)
    s = Server(dtype)
    s.prompt(100, g)
    s.token(g)
    s.step()
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(40):
        s.token(g)
        graph.replay()
        s.check()
    s.counts_cover_the_table()
    del graph


def test_on_a_side_stream_and_on_two_streams_at_once():
    g = torch.Generator().manual_seed(4)
    a, b = Server(torch.bfloat16), Server(torch.float32)
    for s in (a, b):
        s.prompt(200, g)
        s.token(g)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s, stream in zip((a, b), streams):
        with torch.cuda.stream(stream):
            s.step()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_pool_of_another_device_is_refused(monkeypatch):
    s = Server(torch.bfloat16)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: B.copy_pages(s.pool, s.lens[:1], s.lens[:1], s.ws, s.status),
                 lambda: B.free_pages(s.pool, s.ref, s.table, s.lens, None, s.status),
                 lambda: B.window_softmax_decode(s.pool, s.q, s.table, s.lens, 5, 0, 0.1, s.out["window"], s.ws,
                                                 s.status)):
        with pytest.raises(B.EntmaxKVError, match="the pool is on cuda:0, the current device is cuda:1"):
            call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_query_off_16_bytes(dtype):
    g = torch.Generator().manual_seed(5)
    s = Server(dtype)
    s.prompt(90, g)
    raw = torch.zeros(s.q.numel() + 1, device="cuda")
    s.q = raw[1:].view(s.q.shape)
    s.token(g)
    s.step()
    s.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_in_a_query_reaches_its_row_alone(dtype):
    g = torch.Generator().manual_seed(6)
    s = Server(dtype)
    s.prompt(90, g)
    s.token(g)
    s.q[1, 5, 7] = float("nan")
    s.step()
    torch.cuda.synchronize()
    for name in ("prefix", "window"):
        assert bool(s.out[name][1, 5].isnan().all()) and bool(s.lse[name][1, 5].isnan())
        keep = torch.ones(s.rows, H_Q, dtype=torch.bool, device="cuda")
        keep[1, 5] = False
        assert not bool(s.out[name][keep].isnan().any()) and not bool(s.lse[name][keep].isnan().any())
    s.check(rows=(0, 2, 3, 4, 5))
