"""What the paged-cache operators cost: decode attention with a sliding window and sinks, decode attention
over a shared prefix, and the calls that copy, fork, free, reserve and compact the pages of the cache.

Every case is one pass as a serving loop makes it.  With `own` false the pass is made of elementary torch
operations; with `own` true it calls the CUDA library through its Python binding.  Layouts are the library's:
pools [pages][kv heads][page size][dims], page tables [rows][max_pages] with -1 where a row holds no page,
one reference count per physical page.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    llama = dict(H_q=32, H_kv=8, d=128, ps=64, dtype="bf16")      # the 32/8-head bf16 cache of the long-context runs
    tiny = dict(H_q=4, H_kv=1, d=64, ps=16, dtype="f32")          # the small fp32 configuration
    return [
        # one user, one token: a local-attention layer of a short chat, where the latency of the call counts
        dict(name="window one", op="window", B=1, lo=3001, hi=3001, window=1024, sinks=4, mix=1, **llama),
        # a full decode batch over long ragged contexts: the ordinary load of a streaming server
        dict(name="window batch", op="window", B=64, lo=1500, hi=262144, window=8192, sinks=64, mix=2, **llama),
        # the fp32 cache, odd window, rows shorter than the window and than the sinks
        dict(name="window f32", op="window", B=24, lo=1, hi=4101, window=1999, sinks=17, mix=3, **tiny),
        # four answers sampled from one short prompt
        dict(name="prefix short", op="prefix", groups=1, n=4, prefix=1000, tail_lo=1, tail_hi=90, mix=4, **llama),
        # four system prompts with eight conversations each
        dict(name="prefix groups", op="prefix", groups=4, n=8, prefix=16384, tail_lo=100, tail_hi=3000, mix=5, **llama),
        # 32 questions about one long document
        dict(name="prefix document", op="prefix", groups=1, n=32, prefix=131072, tail_lo=200, tail_hi=800, mix=6, **llama),
        # a wide batch behind one prompt: several row tiles for each kv head
        dict(name="prefix wide", op="prefix", groups=1, n=96, prefix=32768 + 41, tail_lo=1, tail_hi=1024, mix=7, **llama),
        # pages moved by a scheduler (beam reorder, cache migration)
        dict(name="copy pages", op="copy", pages=700, n=251, mix=8, **llama),
        # a beam step: four beams take over from their parents
        dict(name="fork beams", op="fork", live=4, n=4, lo=900, hi=1700, pages=256, max_pages=64, mix=9, **llama),
        # 64 samples started from long prompts
        dict(name="fork samples", op="fork", live=3, n=61, lo=90000, hi=131071, pages=8192, max_pages=2080, mix=10, **llama),
        # requests leave a full batch and new prompts take their place
        dict(name="turnover", op="turnover", B=48, n=13, lo=500, hi=30000, pages=24000, max_pages=512, mix=11, H_q=4, H_kv=1,
             d=64, ps=64, dtype="bf16"),
        # the pool after hours of traffic, packed towards its start
        dict(name="compact", op="compact", B=40, lo=2000, hi=16000, pages=6000, max_pages=256, mix=12, **llama),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "prefix", "prefix", "copy", "fork", "turnover", "compact"])
    G = rng.choice([1, 2, 4, 4, 8])
    H_kv = rng.choice([1, 2, 5, 8])
    c = dict(op=op, H_q=G * H_kv, H_kv=H_kv, d=rng.choice([64, 128, 128]), ps=rng.choice([16, 64, 64]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), mix=rng.randrange(1 << 30))
    slow = 8 if c["dtype"] == "f32" else 1          # fp32 caches are the small configurations
    if op == "window":
        hi = _log(rng, 64, 262144)
        c.update(B=_log(rng, 1, 64 // slow), lo=max(1, hi // rng.choice([1, 7, 50])), hi=hi, window=_log(rng, 1, 8192),
                 sinks=rng.choice([0, 1, 4, 4, 64, rng.randrange(1, 300)]))
    elif op == "prefix":
        n, groups = _log(rng, 2, 64 // slow), rng.choice([1, 1, 2, 3])
        c.update(groups=groups, n=max(2, n // groups), prefix=_log(rng, 30, 65536 // (slow * groups)), tail_lo=1,
                 tail_hi=_log(rng, 2, 1500))
    elif op == "copy":
        pages = _log(rng, 16, 700)
        c.update(pages=pages, n=max(1, pages * rng.randrange(5, 50) // 100))
    elif op == "fork":
        live, hi = rng.randrange(1, 5), _log(rng, 40, 60000)
        most = -(-hi // c["ps"]) + 3
        n = _log(rng, 1, 48)
        c.update(live=live, n=n, lo=max(1, hi // 3), hi=hi, max_pages=most, pages=live * most + n + rng.randrange(1, 64))
    elif op == "turnover":
        B, hi = _log(rng, 2, 48), _log(rng, 40, 8000)
        most = -(-hi // c["ps"]) + 2
        c.update(B=B, n=max(1, B * rng.randrange(10, 60) // 100), lo=max(1, hi // 6), hi=hi, max_pages=most,
                 pages=B * most + rng.randrange(1, 100), H_kv=1, H_q=G)
    else:
        B, hi = _log(rng, 2, 40), _log(rng, 40, 4000)
        most = -(-hi // c["ps"]) + 2
        c.update(B=B, lo=max(1, hi // 5), hi=hi, max_pages=most, pages=int(B * most * rng.uniform(1.0, 1.5)) + 8)
    return c


def _lengths(c, count, lo, hi):
    """`count` lengths, log-uniform in [lo, hi], of the case alone (the work of a case does not go by the seed)."""
    rng = random.Random(c["mix"])
    return [_log(rng, lo, hi) for _ in range(count)]


def _elt(c):
    return 2 if c["dtype"] == "bf16" else 4


def _page_bytes(c):
    """K, V, kmin, kmax in the cache's type, mean and m2 in fp32, the count."""
    return c["H_kv"] * c["d"] * (2 * c["ps"] * _elt(c) + 2 * _elt(c) + 8) + 4


def _spans(c, L):
    """(sink tokens, first token of the window) of a sequence of L tokens, without overlap."""
    sinks = min(c["sinks"], L)
    return sinks, max(sinks, L - c["window"], 0)


def work(c):
    H_q, H_kv, d, ps, elt = c["H_q"], c["H_kv"], c["d"], c["ps"], _elt(c)
    if c["op"] == "window":
        seen = pages = 0
        for L in _lengths(c, c["B"], c["lo"], c["hi"]):
            s, w = _spans(c, L)
            seen += s + L - w
            pages += -(-(s + L - w) // ps)
        return {"bytes": seen * H_kv * d * 2 * elt + c["B"] * H_q * (2 * d + 1) * 4 + 4 * (pages + c["B"]),
                "flops": 4 * d * H_q * seen}
    if c["op"] == "prefix":
        B = c["groups"] * c["n"]
        tails = _lengths(c, B, c["tail_lo"], c["tail_hi"])
        once = c["groups"] * c["prefix"] + sum(tails)
        return {"bytes": once * H_kv * d * 2 * elt + B * H_q * (2 * d + 1) * 4 + 4 * (once // ps + 2 * B),
                "flops": 4 * d * H_q * (B * c["prefix"] + sum(tails))}
    page = _page_bytes(c)
    if c["op"] == "copy":
        return {"bytes": c["n"] * (2 * page + 8), "flops": 0}
    if c["op"] == "fork":
        lens = _lengths(c, c["live"], c["lo"], c["hi"])
        rng = random.Random(c["mix"] + 1)
        parents = [lens[rng.randrange(c["live"])] for _ in range(c["n"])]
        copied = sum(L % ps != 0 for L in parents)
        entries = sum(-(-L // ps) for L in parents)
        # table rows: the old entries released, the parent's read, the new written; counts read and written for both
        return {"bytes": copied * 2 * page + entries * (4 * 3 + 4 * 4) + 16 * c["n"], "flops": 0}
    lens = _lengths(c, c["B"], c["lo"], c["hi"])
    held = sum(-(-L // ps) for L in lens)
    if c["op"] == "turnover":
        gone = sum(-(-L // ps) for L in lens[:c["n"]])
        # released and reserved entries (read and written, counts too), and the counts of the pool scanned for free pages
        return {"bytes": gone * (8 + 8 + 8 + 4) + 4 * c["pages"] + 12 * c["B"], "flops": 0}
    moved = sum(1 for p in _taken(c, held) if p >= held)
    return {"bytes": moved * 2 * page + 4 * c["pages"] + 4 * held + 4 * moved, "flops": 0}


def _taken(c, held):
    """The physical pages in use after some traffic, of the case alone."""
    rng = random.Random(c["mix"] + 2)
    return rng.sample(range(c["pages"]), held)


# ---------------------------------------------------------------------------- inputs
def _pool(c, pages, gen):
    H, ps, d, dt = c["H_kv"], c["ps"], c["d"], DTYPES[c["dtype"]]
    f = dict(generator=gen, device="cuda")
    # keys scatter around a centre for each page and head, as neighbouring tokens do; values are N(0, I)
    k = torch.randn(pages, H, ps, d, dtype=dt, **f).mul_(0.3).add_(torch.randn(pages, H, 1, d, dtype=dt, **f))
    v = torch.randn(pages, H, ps, d, dtype=dt, **f)
    kmin, kmax = k.amin(dim=2), k.amax(dim=2)
    mean, m2 = torch.randn(pages, H, d, **f), torch.rand(pages, H, d, **f)
    count = torch.full((pages,), ps, dtype=torch.int32, device="cuda")
    return dict(k=k, v=v, kmin=kmin, kmax=kmax, mean=mean, m2=m2, count=count)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(c, lens, most, perm):
    """Page tables whose rows hold the pages of `lens` tokens, taken from `perm` in turn."""
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for b, L in enumerate(lens):
        P = -(-L // c["ps"])
        table[b, :P] = perm[at:at + P]
        at += P
    return table, at


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    H_q, H_kv, d, ps = c["H_q"], c["H_kv"], c["d"], c["ps"]
    s = dict(case=c, scale=1.0 / math.sqrt(d))
    if c["op"] == "window":
        # only the pages that the window and the sinks still see are resident; the others' entries are -1
        lens = _lengths(c, c["B"], c["lo"], c["hi"])
        most = -(-max(lens) // ps) + 1
        table = torch.full((c["B"], most), -1, dtype=torch.int32)
        spans = []
        for L in lens:
            n_sink, w = _spans(c, L)
            spans.append(sorted(set(range(-(-n_sink // ps))) | set(range(w // ps, -(-L // ps)))))
        perm = torch.randperm(sum(map(len, spans)) + 3, generator=host).to(torch.int32)
        at = 0
        for b, ids in enumerate(spans):
            table[b, torch.tensor(ids, dtype=torch.long)] = perm[at:at + len(ids)]
            at += len(ids)
        s.update(B=c["B"], pool=_pool(c, len(perm), gen), table=table.cuda(), lens=_i32(lens),
                 most=min(c["sinks"] + c["window"], max(lens)))
    elif c["op"] == "prefix":
        B = c["groups"] * c["n"]
        tails = _lengths(c, B, c["tail_lo"], c["tail_hi"])
        lens = [c["prefix"] + t for t in tails]
        whole = c["prefix"] // ps                     # the shared pages; a fork copies the page that the prefix ends in
        most = -(-max(lens) // ps) + 1
        own_pages = [-(-L // ps) - whole for L in lens]
        perm = torch.randperm(c["groups"] * whole + sum(own_pages) + 3, generator=host).to(torch.int32)
        table = torch.full((B, most), -1, dtype=torch.int32)
        at = 0
        for j in range(c["groups"]):
            table[j * c["n"]:(j + 1) * c["n"], :whole] = perm[at:at + whole]
            at += whole
        for b, n in enumerate(own_pages):
            table[b, whole:whole + n] = perm[at:at + n]
            at += n
        s.update(B=B, pool=_pool(c, len(perm), gen), table=table.cuda(), lens=_i32(lens), whole=whole,
                 most=max(lens) - whole * ps, starts=_i32([j * c["n"] for j in range(c["groups"] + 1)]),
                 prefixes=_i32([c["prefix"]] * c["groups"]))
    elif c["op"] == "copy":
        perm = torch.randperm(c["pages"], generator=host).to(torch.int32)
        s.update(pool=_pool(c, c["pages"], gen), src=perm[:c["n"]].cuda(), dst=perm[c["n"]:2 * c["n"]].cuda())
    elif c["op"] == "fork":
        # rows [0, live) run; rows [live, live + n) hold the forks of the step before
        lens = _lengths(c, c["live"], c["lo"], c["hi"])
        rng = random.Random(c["mix"] + 1)
        parents = [rng.randrange(c["live"]) for _ in range(c["n"])]
        perm = torch.randperm(c["pages"], generator=host).to(torch.int32)
        table, at = _rows(c, lens, c["max_pages"], perm)
        old = table[torch.tensor(parents)].clone()
        ref = torch.zeros(c["pages"], dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        for i, b in enumerate(parents):
            if lens[b] % ps:
                old[i, lens[b] // ps] = perm[at]
                at += 1
        ref.index_add_(0, old[old >= 0].long(), torch.ones(int((old >= 0).sum()), dtype=torch.int32))
        s.update(pool=_pool(c, c["pages"], gen), table=torch.cat([table, old]).cuda(), ref=ref.cuda(),
                 lens=_i32(lens + [lens[b] for b in parents]), src=_i32(parents),
                 dst=_i32([c["live"] + i for i in range(c["n"])]))
    elif c["op"] == "turnover":
        # rows [0, n) have finished; prompts of the same lengths wait for their rows
        lens = _lengths(c, c["B"], c["lo"], c["hi"])
        perm = torch.randperm(c["pages"], generator=host).to(torch.int32)
        table, at = _rows(c, lens, c["max_pages"], perm)
        ref = torch.zeros(c["pages"], dtype=torch.int32)
        ref[perm[:at].long()] = 1
        s.update(pool=_pool(c, c["pages"], gen), table=table.cuda(), ref=ref.cuda(), lens=_i32(lens),
                 lens0=_i32(lens), rows=_i32(list(range(c["n"]))), want=_i32(lens))
    else:
        lens = _lengths(c, c["B"], c["lo"], c["hi"])
        taken = torch.tensor(_taken(c, sum(-(-L // ps) for L in lens)), dtype=torch.int32)
        taken = taken[torch.randperm(len(taken), generator=host)]
        table, at = _rows(c, lens, c["max_pages"], taken)
        ref = torch.zeros(c["pages"], dtype=torch.int32)
        ref[taken.long()] = 1
        # a pass starts from the tables and counts as they are; the pool's pages outlive a move
        s.update(pool=_pool(c, c["pages"], gen), table0=table.cuda(), ref0=ref.cuda())
        s.update(table=s["table0"].clone(), ref=s["ref0"].clone(), live=_i32([0]))
    if c["op"] in ("window", "prefix"):
        s["q"] = torch.randn(s["B"], H_q, d, generator=gen, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["B"], H_q, device="cuda")
    if own:
        from sparse_long_context_min_b200 import binding as K
        p = s["pool"]
        s["handle"] = K.Pool(p["k"], p["v"], p["kmin"], p["kmax"], p["mean"], p["m2"], p["count"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] in ("window", "prefix"):
            what = K.OP_WINDOW_SOFTMAX if c["op"] == "window" else K.OP_PREFIX_SOFTMAX
            size = K.workspace_size(what, s["B"], H_q, H_kv, s["table"].shape[1], 0, ps, d)
        else:
            rows, most = s["table"].shape if "table" in s else (0, 1)
            entries = max(rows, c.get("n", 0))
            size = K.workspace_size(K.OP_PAGES, entries, 0, 0, most, p["count"].numel(), ps, d)
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass
def _bits(pool):
    """The pool's contents as whole numbers: a moved page keeps every bit."""
    return {k: x if x.dtype == torch.int32 else x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)
            for k, x in pool.items()}


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return _PLAIN[c["op"]](s, c)


def _run_own(s, c):
    from sparse_long_context_min_b200 import binding as K
    p, ws, st = s["handle"], s["workspace"], s["status"]
    if c["op"] == "window":
        K.window_softmax_decode(p, s["q"], s["table"], s["lens"], c["window"], c["sinks"], s["scale"], s["out"], ws, st,
                                lse_out=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "prefix":
        K.prefix_softmax_decode(p, s["q"], s["table"], s["lens"], s["starts"], s["prefixes"], s["scale"], s["out"], ws, st,
                                lse_out=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "copy":
        K.copy_pages(p, s["src"], s["dst"], ws, st)
        return _bits(s["pool"])
    if c["op"] == "fork":
        K.fork_sequences(p, s["ref"], s["table"], s["lens"], s["src"], s["dst"], ws, st)
    elif c["op"] == "turnover":
        K.free_pages(p, s["ref"], s["table"], s["lens"], s["rows"], st)
        K.reserve_pages(p, s["ref"], s["table"], s["lens"], s["want"], ws, st)
        left = s["lens"].clone()
        s["lens"].copy_(s["lens0"])                   # the prompts are written
        return s["table"], s["ref"], left
    else:
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
        K.compact_pages(p, s["ref"], s["table"], s["live"], ws, st)
        return s["table"], s["ref"], s["live"], _bits(s["pool"])
    return s["table"], s["ref"], s["lens"], _bits(s["pool"])


def _tokens(pool, table, pos, ps):
    """K and V [B, kv heads, tokens, dims] in fp32 of the positions pos [B, tokens], through the page table."""
    pages = table.gather(1, pos // ps).clamp_min(0).long()
    slot = pos % ps
    return (pool["k"][pages, :, slot].float().transpose(1, 2), pool["v"][pages, :, slot].float().transpose(1, 2))


def _softmax(x):
    """exp(x - max), its sum, and the log of the sum of exp(x); a row without a finite score gives zeros."""
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(dim=-1, keepdim=True)
    return e, z, (m + torch.log(z)).squeeze(-1)


def _plain_window(s, c):
    B, H_kv, d, G = c["B"], c["H_kv"], c["d"], c["H_q"] // c["H_kv"]
    L = s["lens"].long()[:, None]
    t = torch.arange(s["most"], device="cuda")[None]
    n_sink = L.clamp(max=c["sinks"])
    start = torch.maximum(n_sink, L - c["window"])
    pos = torch.where(t < n_sink, t, start + t - n_sink)
    seen = pos < L
    k, v = _tokens(s["pool"], s["table"], torch.where(seen, pos, torch.zeros_like(pos)), c["ps"])
    q = s["q"].view(B, H_kv, G, d) * s["scale"]
    x = (q @ k.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    e, z, lse = _softmax(x)
    o = (e @ v) / torch.where(z > 0, z, torch.ones_like(z))
    return o.reshape(B, c["H_q"], d), lse.reshape(B, c["H_q"])


def _plain_prefix(s, c):
    J, n, B, H_kv, d, G, ps = c["groups"], c["n"], s["B"], c["H_kv"], c["d"], c["H_q"] // c["H_kv"], c["ps"]
    q = s["q"].view(B, H_kv, G, d) * s["scale"]
    shared = s["whole"] * ps
    # the prefix once for each group: its sequences' query heads are the rows of one product
    pages = s["table"][::n, :s["whole"]].long()
    kp, vp = (s["pool"][x][pages].float().permute(0, 2, 1, 3, 4).reshape(J, H_kv, shared, d) for x in ("k", "v"))
    qg = q.view(J, n, H_kv, G, d).transpose(1, 2).reshape(J, H_kv, n * G, d)
    xp = (qg @ kp.transpose(2, 3)).view(J, H_kv, n, G, shared).transpose(1, 2).reshape(B, H_kv, G, shared)
    # the tokens behind it, of each sequence
    pos = shared + torch.arange(s["most"], device="cuda")[None].expand(B, -1)
    seen = pos < s["lens"].long()[:, None]
    kt, vt = _tokens(s["pool"], s["table"], torch.where(seen, pos, torch.full_like(pos, shared)), ps)
    xt = (q @ kt.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    e, z, lse = _softmax(torch.cat([xp, xt], dim=-1))
    ep = e[..., :shared].reshape(J, n, H_kv, G, shared).transpose(1, 2).reshape(J, H_kv, n * G, shared)
    op = (ep @ vp).view(J, H_kv, n, G, d).transpose(1, 2).reshape(B, H_kv, G, d)
    o = (op + e[..., shared:] @ vt) / z
    return o.reshape(B, c["H_q"], d), lse.reshape(B, c["H_q"])


def _move(pool, src, dst):
    pool["k"][dst], pool["v"][dst] = pool["k"][src], pool["v"][src]
    pool["kmin"][dst], pool["kmax"][dst] = pool["kmin"][src], pool["kmax"][src]
    pool["mean"][dst], pool["m2"][dst] = pool["mean"][src], pool["m2"][src]
    pool["count"][dst] = pool["count"][src]


def _plain_copy(s, c):
    _move(s["pool"], s["src"].long(), s["dst"].long())
    return _bits(s["pool"])


def _count(ref, pages, by):
    """Adds `by` to the reference counts of the page entries >= 0."""
    flat = pages.reshape(-1)
    ref.index_add_(0, flat.clamp_min(0).long(), torch.where(flat >= 0, by, 0).to(torch.int32))


def _plain_fork(s, c):
    table, ref, lens, ps = s["table"], s["ref"], s["lens"], c["ps"]
    src, dst = s["src"].long(), s["dst"].long()
    _count(ref, table[dst], -1)                       # the pages that the rows held
    L = lens[src].long()
    whole, part = L // ps, L % ps != 0
    rows = table[src]
    p = torch.arange(table.shape[1], device="cuda")[None]
    rows = torch.where(p < whole[:, None], rows, -1)
    last = table[src, whole.clamp(max=table.shape[1] - 1)].long()
    free = torch.argsort((ref != 0).to(torch.int8), stable=True)
    fresh = free[(part.cumsum(0) - 1).clamp_min(0)]
    at = (p == whole[:, None]) & part[:, None]
    rows = torch.where(at, fresh[:, None].to(torch.int32), rows)
    _count(ref, rows, 1)
    table[dst] = rows
    lens[dst] = lens[src]
    keep = torch.zeros_like(fresh)                    # nothing to copy: a page onto itself
    _move(s["pool"], torch.where(part, last, keep), torch.where(part, fresh, keep))
    return table, ref, lens, _bits(s["pool"])


def _plain_turnover(s, c):
    table, ref, lens, ps = s["table"], s["ref"], s["lens"], c["ps"]
    rows = s["rows"].long()
    _count(ref, table[rows], -1)
    table[rows] = -1
    lens[rows] = 0
    p = torch.arange(table.shape[1], device="cuda")[None]
    need = (p >= (lens[:, None] + ps - 1) // ps) & (p < (s["want"][:, None] + ps - 1) // ps) & (table < 0)
    free = torch.argsort((ref != 0).to(torch.int8), stable=True).to(torch.int32)
    rank = (need.reshape(-1).cumsum(0) - 1).clamp_min(0).view_as(need)
    fresh = torch.where(need, free[rank], -1)
    table.copy_(torch.where(need, fresh, table))
    _count(ref, fresh, 1)
    left = lens.clone()
    lens.copy_(s["lens0"])                            # the prompts are written
    return table, ref, left


def _plain_compact(s, c):
    table, ref = s["table"], s["ref"]
    table.copy_(s["table0"])
    ref.copy_(s["ref0"])
    live = ref > 0
    n_live = live.sum()
    ids = torch.arange(ref.numel(), device="cuda")
    src = (live & (ids >= n_live)).nonzero().view(-1)
    dst = (~live & (ids < n_live)).nonzero().view(-1)
    _move(s["pool"], src, dst)
    to = ids.to(torch.int32)
    to[src] = dst.to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()], table))
    ref[dst] = ref[src]
    ref[src] = 0
    s["live"].copy_(n_live)
    return table, ref, s["live"], _bits(s["pool"])


_PLAIN = {"window": _plain_window, "prefix": _plain_prefix, "copy": _plain_copy, "fork": _plain_fork,
          "turnover": _plain_turnover, "compact": _plain_compact}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(c, seed):
    """o = sum_i softmax(scale q.k_i) v_i over the tokens that a sequence sees, and the log of the normaliser, in
    float64, one sequence after the other.  The page operators return whole numbers, which are compared as they are."""
    if c["op"] not in ("window", "prefix"):
        return None
    s = prepare(c, seed)
    pool, H_kv, G, d, ps = s["pool"], c["H_kv"], c["H_q"] // c["H_kv"], c["d"], c["ps"]
    o = torch.zeros(s["B"], c["H_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["B"], c["H_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        seen = list(range(L))
        if c["op"] == "window":
            seen = [t for t in range(min(c["sinks"], L))] + [t for t in range(max(0, L - c["window"]), L) if t >= c["sinks"]]
        if not seen:
            continue
        t = torch.tensor(seen, device="cuda")
        page, slot = s["table"][b, t // ps].long(), t % ps
        for g in range(H_kv):
            k, v = pool["k"][page, g, slot].double(), pool["v"][page, g, slot].double()
            x = s["scale"] * (s["q"][b, g * G:(g + 1) * G].double() @ k.T)
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(x, dim=1)
            o[b, g * G:(g + 1) * G] = torch.exp(x - lse[b, g * G:(g + 1) * G, None]) @ v
    return o, lse
