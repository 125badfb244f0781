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
    long long row0;            // partial rows of all units before ((kv head, row tile) in this order)
    long long block0;          // blocks of all units before
};

struct PrefixHead {
    long long total;           // blocks of all units
    int C;                     // CTAs that have a share of them
};

// A CTA's place in its share: group, kv head, row tile, block, and what is left.
struct PrefixWalk {
    int j, g, t, k;
    long long left;
};

struct PrefixArgs {
    RangeArgs r;               // the range kernels' arguments: every sequence's own tokens
    const int32_t* group_start;   // [n_groups + 1]
    const int32_t* prefix_lens;   // [n_groups]
    int n_groups;
    int ps;
    int row_tile, block_tok;   // rows and tokens that a unit's CTA works on at once
    int most;                  // blocks that it sums before it adds them to the unit's partial
    int C;                     // CTAs of the prefix kernel
    int32_t* shared;           // [B] first page of each sequence's own range
    int32_t* gid;              // [B] group of each sequence, -1 without one
    PrefixGroup* groups;       // [n_groups]
    PrefixHead* head;
    PrefixWalk* walks;         // [C] each CTA's share
    float* part_o;             // partials of (CTA c, unit): [d / 4][the unit's rows] float4 from row prefix_part_row on
    float* part_ml;            // [rows][2]
};

// The units of all groups laid end to end, dealt to the CTAs in equal shares.
// To start a unit costs a CTA about as long as kPrefixTurn blocks (its query,
// the end of the pipeline before, its results): every unit is laid out with as
// many blocks in front that hold no work.
constexpr int kPrefixTurn = 6;

// Blocks that the bf16 kernel's tensor cores sum by themselves (PrefixArgs::most).
// They cut every step off, always to the same side: 2e-7 of a sum of values of one
// sign a block.  A segment's result is added to the unit's partial by rounded
// adds, so that long shares lose no more than one of 128 blocks does (1.7e-5; 4.4e-4
// at 2048 blocks otherwise).  A segment's end costs about as much as a unit's start:
// 4% at 20 x 16 sequences behind 65536 tokens (1130 -> 1178 us).  Shares of 111 blocks
// (32 sequences behind 131072 tokens, one kv head's 2048 blocks for 18 CTAs) are one
// segment: 136.6 us; with segments of 64 blocks 142, of 32 152, at errors of 9.0e-6,
// 5.8e-6 and 4.3e-6, of which the two bf16 parts make 3.6e-6.
constexpr int kPrefixMost = 128;

EKV_DEV int prefix_len(const PrefixGroup& G) { return G.blocks + kPrefixTurn; }

// One thread: CTA c's share.
EKV_DEV PrefixWalk prefix_start(const PrefixArgs& a, int c, long long total, int C)
{
    PrefixWalk w{};
    const long long b0 = mul_div(total, c, C);
    w.left = mul_div(total, c + 1, C) - b0;
    int lo = 0, hi = a.n_groups - 1;                   // last group with block0 <= b0 and blocks in it
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.groups[mid].block0 <= b0) lo = mid;
        else hi = mid - 1;
    }
    const PrefixGroup& G = a.groups[lo];
    const int len = prefix_len(G);
    const long long in = b0 - G.block0, unit = in < (1ll << 31) ? (int)in / len : in / len;
    w.j = lo;
    w.k = (int)(in - unit * len);
    w.g = (int)unit / G.tiles;                         // units of a group: 31 bits
    w.t = (int)unit % G.tiles;
    return w;
}

// What a CTA does next of its current unit: blocks [k, k + n), n at most a.most.
// False at the end of its share (blocks without work may be left of it).
EKV_DEV bool prefix_segment(const PrefixArgs& a, const PrefixWalk& w, int& k, int& n)
{
    if (w.left <= kPrefixTurn - w.k || w.left <= 0) return false;
    const long long end = min((long long)prefix_len(a.groups[w.j]), w.k + w.left) - kPrefixTurn;
    k = max(w.k - kPrefixTurn, 0);
    n = min((int)end - k, a.most);
    return true;
}

// To the unit's next segment (w.k > 0), or to the next unit (w.k = 0).
EKV_DEV void prefix_advance(const PrefixArgs& a, PrefixWalk& w)
{
    const PrefixGroup& G = a.groups[w.j];
    const int len = prefix_len(G), to = min(len, max(w.k, kPrefixTurn) + a.most);
    w.left -= to - w.k;
    w.k = to < len ? to : 0;
    if (w.left <= 0 || w.k > 0 || ++w.t < G.tiles) return;
    w.t = 0;
    if (++w.g < a.r.H_kv) return;
    w.g = 0;
    do ++w.j;
    while (a.groups[w.j].pages == 0);
}

// First partial row of unit (g, t) of a group at CTA c: units' rows and CTAs
// form a staircase, so the ranges of two (CTA, unit) pairs never meet.
EKV_DEV long long prefix_part_row(const PrefixArgs& a, const PrefixGroup& G, int g, int t, int c)
{
    return G.row0 + (long long)g * G.rows + (long long)t * a.row_tile + (long long)a.row_tile * c;
}

// First and last CTA that hold blocks of unit (g, t).
EKV_DEV int2 prefix_span(const PrefixGroup& G, int g, int t, long long total, int C)
{
    const long long at = G.block0 + ((long long)g * G.tiles + t) * prefix_len(G);
    return make_int2(range_cta_of(at + kPrefixTurn, total, C), range_cta_of(at + prefix_len(G) - 1, total, C));
}

int launch_prefix(const entmaxkv_pool& pool, const PrefixArgs& a, int range_C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream);

}  // namespace ekv
