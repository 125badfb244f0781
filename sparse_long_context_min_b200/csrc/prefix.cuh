// Shared-prefix decode: the plan that its kernels follow (internal to the library).
#pragma once

#include "common.cuh"
#include "range.cuh"

namespace ekv {

// One group of sequences that share a prefix.
struct PrefixGroup {
    int lo, n;                 // first sequence and number of sequences
    int first;                 // the first one that is not empty: its page-table row names the shared pages
    int pages;                 // whole pages that the group shares (0: nothing is shared)
    int rows, tiles;           // query rows of one kv head (n * G), and row tiles
    int blocks;                // token blocks of the shared pages
    int unit0;                 // first unit: (kv head, row tile) in this order
    long long row0;            // partial rows of all units before
    long long block0;          // blocks of all units before
};

struct PrefixArgs {
    RangeArgs r;               // the range kernels' arguments: every sequence's own tokens
    const int32_t* group_start;   // [n_groups + 1]
    const int32_t* prefix_lens;   // [n_groups]
    int n_groups;
    int ps;
    int row_tile, block_tok;   // rows and tokens that a unit's CTA works on at once
    int C;                     // CTAs of the prefix kernel
    int32_t* shared;           // [B] first page of each sequence's own range
    int32_t* gid;              // [B] group of each sequence, -1 without one
    PrefixGroup* groups;       // [n_groups]
    long long* total;          // blocks of all units
    int2* span;                // [units] first and last CTA of a unit
    float* part_o;             // [rows][d]: a unit's rows of CTA c start at its row0 + row_tile * c
    float* part_ml;            // [rows][2]
};

// The units of all groups laid end to end, dealt to the CTAs in equal shares.
struct PrefixWalk {
    int j, g, t, k;            // group, kv head, row tile, next block
    int C;
    long long left, total;
};

// One thread: CTA c's share.
EKV_DEV PrefixWalk prefix_start(const PrefixArgs& a, int c)
{
    PrefixWalk w{};
    w.total = *a.total;
    w.C = (int)min((long long)a.C, w.total);
    if (c >= w.C) return w;
    const long long b0 = w.total * c / w.C;
    w.left = w.total * (c + 1) / w.C - b0;
    int lo = 0, hi = a.n_groups - 1;                   // last group with block0 <= b0 and blocks in it
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.groups[mid].block0 <= b0) lo = mid;
        else hi = mid - 1;
    }
    const PrefixGroup& G = a.groups[lo];
    const long long in = b0 - G.block0;
    w.j = lo;
    w.k = (int)(in % G.blocks);
    w.g = (int)(in / G.blocks / G.tiles);
    w.t = (int)(in / G.blocks % G.tiles);
    return w;
}

// Past n blocks of the current unit (at most to its end).
EKV_DEV void prefix_advance(const PrefixArgs& a, PrefixWalk& w, int n)
{
    w.k += n;
    w.left -= n;
    if (w.left <= 0 || w.k < a.groups[w.j].blocks) return;
    w.k = 0;
    if (++w.t < a.groups[w.j].tiles) return;
    w.t = 0;
    if (++w.g < a.r.H_kv) return;
    w.g = 0;
    do ++w.j;
    while (a.groups[w.j].pages == 0);
}

EKV_DEV int prefix_unit(const PrefixGroup& G, int g, int t) { return G.unit0 + g * G.tiles + t; }

// First partial row of unit (g, t) of a group at CTA c: units' rows and CTAs
// form a staircase, so the ranges of two (CTA, unit) pairs never meet.
EKV_DEV long long prefix_part_row(const PrefixArgs& a, const PrefixGroup& G, int g, int t, int c)
{
    return G.row0 + (long long)g * G.rows + (long long)t * a.row_tile + (long long)a.row_tile * c;
}

// The CTA that holds a unit's first block leaves its CTAs for the merge.
EKV_DEV void prefix_note_span(const PrefixArgs& a, const PrefixWalk& w, const PrefixGroup& G, int c)
{
    if (w.k != 0) return;
    const int u = prefix_unit(G, w.g, w.t);
    const long long at = G.block0 + (long long)(u - G.unit0) * G.blocks;
    a.span[u] = make_int2(c, range_cta_of(at + G.blocks - 1, w.total, w.C));
}

int launch_prefix(const entmaxkv_pool& pool, const PrefixArgs& a, int range_C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream);

}  // namespace ekv
