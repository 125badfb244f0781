"""Window and prefix decode and the page-management calls refuse bad arguments:
in the binding before the library is reached, and in the library before a launch."""
import ctypes
import types

import pytest
import torch

from sparse_long_context_min_b200 import binding as B


@pytest.fixture
def no_library(monkeypatch):
    def unreachable():
        raise AssertionError("the library was called although an argument was invalid")
    monkeypatch.setattr(B, "lib", unreachable)


def _pool(num=20, H_kv=8, ps=64, d=128):
    return types.SimpleNamespace(H_kv=H_kv, d=d, num_phys=num, ps=ps, k_pool=torch.empty(0, dtype=torch.bfloat16))


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _f32(*shape):
    return torch.zeros(*shape, dtype=torch.float32)


I64 = torch.zeros(3, dtype=torch.int64)


def _args():
    return dict(pool=_pool(), q=_f32(3, 32, 128), page_table=_i32(3, 10), seq_lens=_i32(3), out=_f32(3, 32, 128),
                workspace=torch.zeros(64, dtype=torch.uint8), status=_i32(1), scale=0.1, window=5, sinks=0,
                group_start=_i32(3), prefix_lens=_i32(2), lse_out=None, ref=_i32(20), src=_i32(2), dst=_i32(2),
                rows=_i32(2), lens=_i32(3), live=_i32(1))


NAMES = {
    "window_softmax_decode": ("pool", "q", "page_table", "seq_lens", "window", "sinks", "scale", "out", "workspace",
                              "status", "lse_out"),
    "prefix_softmax_decode": ("pool", "q", "page_table", "seq_lens", "group_start", "prefix_lens", "scale", "out",
                              "workspace", "status", "lse_out"),
    "copy_pages": ("pool", "src", "dst", "workspace", "status"),
    "fork_sequences": ("pool", "ref", "page_table", "seq_lens", "src", "dst", "workspace", "status"),
    "free_pages": ("pool", "ref", "page_table", "seq_lens", "rows", "status"),
    "reserve_pages": ("pool", "ref", "page_table", "seq_lens", "lens", "workspace", "status"),
    "compact_pages": ("pool", "ref", "page_table", "live", "workspace", "status"),
}

BAD = [
    ("window_softmax_decode", dict(q=_f32(3, 32, 64)), "64 dims per head"),
    ("window_softmax_decode", dict(page_table=_i32(2, 10)), "2 rows for 3 sequences"),
    ("window_softmax_decode", dict(seq_lens=_i32(2)), "seq_lens holds 2 elements"),
    ("window_softmax_decode", dict(out=_f32(3, 32, 127)), "out holds"),
    ("window_softmax_decode", dict(lse_out=_f32(3, 31)), "lse_out holds 93 elements; the call addresses 96"),
    ("window_softmax_decode", dict(window=0), "window must be at least 1"),
    ("window_softmax_decode", dict(window=2 ** 31), "window must be at least 1"),
    ("window_softmax_decode", dict(sinks=-1), "sinks at least 0"),
    ("window_softmax_decode", dict(workspace=None), "workspace is required"),
    ("window_softmax_decode", dict(out=_f32(3, 128, 32).transpose(1, 2)), "out must be contiguous"),
    ("prefix_softmax_decode", dict(group_start=_i32(2)), "group_start holds 2 elements; the call addresses 3"),
    ("prefix_softmax_decode", dict(group_start=I64), "group_start must be torch.int32"),
    ("prefix_softmax_decode", dict(prefix_lens=_i32(1, 2)), "prefix_lens must have 1 dimensions"),
    ("prefix_softmax_decode", dict(q=torch.zeros(3, 32, 128, dtype=torch.bfloat16)), "q must be torch.float32"),
    ("copy_pages", dict(src=_i32(3)), "src lists 3 entries, dst 2"),
    ("copy_pages", dict(dst=I64[:2]), "dst must be torch.int32"),
    ("copy_pages", dict(status=None), "status is required"),
    ("fork_sequences", dict(ref=_i32(19)), "ref holds 19 elements; the call addresses 20"),
    ("fork_sequences", dict(seq_lens=_i32(2)), "seq_lens holds 2 elements; the call addresses 3"),
    ("fork_sequences", dict(dst=_i32(1)), "src lists 2 entries, dst 1"),
    ("fork_sequences", dict(page_table=_i32(30)), "page_table must have 2 dimensions"),
    ("free_pages", dict(rows=I64), "rows must be torch.int32"),
    ("free_pages", dict(page_table=_i32(10, 3).t()), "page_table must be contiguous"),
    ("reserve_pages", dict(lens=_i32(2)), "lens holds 2 elements; the call addresses 3"),
    ("reserve_pages", dict(workspace=torch.zeros(8, 8).t()), "workspace must be contiguous"),
    ("compact_pages", dict(live=_i32(0)), "live holds 0 elements"),
    ("compact_pages", dict(ref=_f32(20)), "ref must be torch.int32"),
]


@pytest.mark.parametrize("name,over,words", BAD)
def test_binding_refuses(no_library, name, over, words):
    a = dict(_args(), **over)
    with pytest.raises(B.EntmaxKVError) as e:
        getattr(B, name)(*[a[n] for n in NAMES[name]])
    assert e.value.code == B.INVALID_ARG and words in str(e.value), str(e.value)


def test_binding_refuses_window_bounds_of_free_pages(no_library):
    a = _args()
    for window, sinks in ((-1, 0), (2 ** 31, 0), (5, -1)):
        with pytest.raises(B.EntmaxKVError, match="window and sinks"):
            B.free_pages(*[a[n] for n in NAMES["free_pages"]], window=window, sinks=sinks)


def test_binding_refuses_pageable_memory(no_library):
    if torch.cuda.is_available():
        pytest.skip("asks CUDA")
    a = _args()
    for name, names in NAMES.items():
        with pytest.raises((B.EntmaxKVError, RuntimeError)):
            getattr(B, name)(*[a[n] for n in names])


# ---------------------------------------------------------------- the library itself
P = ctypes.c_void_p(256)               # never dereferenced: validation fails first
BIG = 1 << 30


def _cpool(num=20, H_kv=8, ps=64, d=128, dtype=B.BF16, base=256):
    return ctypes.byref(B.CPool(base, 256, 256, 256, 256, 256, 256, num, H_kv, ps, d, dtype))


def _window(pool=None, q=P, H_q=32, table=P, max_pages=10, lens=P, n=3, window=5, sinks=0, scale=0.1, out=P, ws=P,
            size=BIG, status=P):
    return B.lib().entmaxkv_window_softmax_decode(pool or _cpool(), q, H_q, table, max_pages, lens, n, window, sinks,
                                                  scale, out, None, ws, size, status, None)


def _prefix(pool=None, H_q=32, max_pages=10, n=3, starts=P, prefixes=P, groups=2, scale=0.1, ws=P, size=BIG, status=P):
    return B.lib().entmaxkv_prefix_softmax_decode(pool or _cpool(), P, H_q, P, max_pages, P, n, starts, prefixes,
                                                  groups, scale, P, None, ws, size, status, None)


def test_window_and_prefix_validate_on_the_host():
    inf = float("inf")
    for call in (_window, _prefix):
        assert call(pool=_cpool(d=96)) == B.UNSUPPORTED
        assert call(pool=_cpool(ps=32)) == B.UNSUPPORTED
        assert call(pool=_cpool(dtype=2)) == B.UNSUPPORTED
        assert call(pool=_cpool(base=260)) == B.INVALID_ARG
        assert call(H_q=24) == B.UNSUPPORTED              # three query heads a kv head
        assert call(H_q=30) == B.INVALID_ARG
        assert call(max_pages=0) == B.INVALID_ARG
        assert call(max_pages=2 ** 25) == B.UNSUPPORTED   # positions past 31 bits
        assert call(n=-1) == B.INVALID_ARG
        assert call(n=2 ** 27) == B.UNSUPPORTED           # query rows past 31 bits
        for scale in (0.0, -1.0, inf, float("nan")):
            assert call(scale=scale) == B.INVALID_ARG
        assert call(status=None) == B.INVALID_ARG
        assert call(ws=None) == B.WORKSPACE
        assert call(ws=ctypes.c_void_p(264)) == B.WORKSPACE
        assert call(size=1000) == B.WORKSPACE
    for over in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(window=0), dict(sinks=-1)):
        assert _window(**over) == B.INVALID_ARG
    assert _window(n=0) == B.OK and _prefix(n=0, groups=0) == B.OK
    for over in (dict(groups=-1), dict(groups=4), dict(starts=None), dict(prefixes=None)):
        assert _prefix(**over) == B.INVALID_ARG


def test_page_calls_validate_on_the_host():
    L = B.lib()

    def copy(pool=None, src=P, n=2, ws=P, size=BIG):
        return L.entmaxkv_copy_pages(pool or _cpool(), src, P, n, ws, size, P, None)

    def fork(pool=None, ref=P, max_pages=10, rows=4, n=2, ws=P, size=BIG):
        return L.entmaxkv_fork_sequences(pool or _cpool(), ref, P, max_pages, P, rows, P, P, n, ws, size, P, None)

    def free(pool=None, ref=P, max_pages=10, rows=4, listed=P, n=2, window=-1, sinks=0):
        return L.entmaxkv_free_pages(pool or _cpool(), ref, P, max_pages, P, rows, listed, n, window, sinks, P, None)

    def reserve(pool=None, ref=P, max_pages=10, rows=4, ws=P, size=BIG):
        return L.entmaxkv_reserve_pages(pool or _cpool(), ref, P, max_pages, P, rows, P, ws, size, P, None)

    def compact(pool=None, ref=P, max_pages=10, rows=4, ws=P, size=BIG):
        return L.entmaxkv_compact_pages(pool or _cpool(), ref, P, max_pages, rows, P, ws, size, P, None)

    for call in (copy, fork, free, reserve, compact):
        assert call(pool=_cpool(d=96)) == B.UNSUPPORTED
        assert call(pool=_cpool(base=8)) == B.INVALID_ARG
        if call is not copy:
            assert call(max_pages=0) == B.INVALID_ARG
            assert call(rows=-1) == B.INVALID_ARG
            assert call(max_pages=2 ** 30) == B.UNSUPPORTED   # table entries past 31 bits
            assert call(ref=None) == B.INVALID_ARG
        if call is not free:
            assert call(ws=None) == B.WORKSPACE
            assert call(size=100) == B.WORKSPACE
    assert free(rows=1, max_pages=65535 * 1024 + 1, n=1) == B.UNSUPPORTED   # a row of more chunks than a grid has
    assert copy(n=-1) == B.INVALID_ARG and copy(src=None) == B.INVALID_ARG and copy(n=0) == B.OK
    assert fork(n=5) == B.INVALID_ARG and fork(n=-1) == B.INVALID_ARG and fork(n=0) == B.OK
    assert free(n=-1) == B.INVALID_ARG and free(sinks=-1) == B.INVALID_ARG and free(n=0) == B.OK
    assert free(listed=None) == B.INVALID_ARG             # every row, but n is not their number
    assert reserve(rows=0) == B.OK


def test_workspace_sizes_of_the_cache_calls():
    w = lambda op, rows=4, k=0: B.workspace_size(op, rows, 32, 8, 100, k, 64, 128)
    assert 0 < w(B.OP_WINDOW_SOFTMAX) < w(B.OP_PREFIX_SOFTMAX)
    assert B.workspace_size(B.OP_WINDOW_SOFTMAX, 0, 32, 8, 100, 0, 64, 128) == 0
    assert B.workspace_size(B.OP_PAGES, 0, 0, 0, 0, 1000, 0, 0) >= 3 * 4 * 1000
    assert B.workspace_size(B.OP_PAGES, 64, 0, 0, 0, 1000, 0, 0) > B.workspace_size(B.OP_PAGES, 0, 0, 0, 0, 1000, 0, 0)
    assert B.workspace_size(B.OP_PAGES, 4, 0, 0, 0, 0, 0, 0) == 0
    assert B.workspace_size(B.OP_PAGES, -1, 0, 0, 0, 10, 0, 0) == 0
