// Softmax decode attention over token ranges: what the sliding-window kernels
// and the shared-prefix kernels have in common (internal to the library).
//
// Work is cut into units (the rows that read one key/value range through one
// kv head) of 64-token tiles.  The tiles of all units, laid end to end, are
// dealt to the CTAs in equal consecutive shares, so every CTA streams the same
// number of bytes whatever the lengths of the sequences; a share that starts or
// ends inside a unit leaves a partial result (o, running maximum, sum) that a
// merge kernel joins.  (CTA c, unit u) pairs form a monotone staircase, so
// c + u names a partial's slot uniquely.
#pragma once

#include "common.cuh"
#include "kernels.cuh"

namespace ekv {

constexpr int kRangeTile = 64;           // tokens of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct RangeArgs {
    const float* q;                // [B][H_q][d]
    int H_q, H_kv, G;
    const int32_t* page_table;     // [B][max_pages]
    int max_pages;
    const int32_t* seq_lens;       // [B]
    int B;
    int num_phys;
    int window, sinks;             // window form: tokens < sinks and >= L - window
    const int32_t* group_start;    // [n_groups + 1] bounds to check only (groups too small to share), or NULL
    int n_groups;
    const int32_t* shared;         // [B] prefix form: first page of each sequence's own range, else NULL
    float xscale;                  // scale * log2(e): scores are kept in the base-2 domain
    float* part_o;                 // [CTAs + units][G][d] partial outputs
    float* part_ml;                // [CTAs + units][G][2] running maximum (base 2) and sum
    int2* span;                    // [units] first and last CTA of a unit
    float* out;                    // [B][H_q][d]
    float* lse;                    // [B][H_q] or NULL
    int32_t* status;
    int direct;                    // write finished units straight to out
};

// The kernels over each sequence's tokens behind a shared prefix (window.cu), C CTAs.
int launch_range(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                 const CUtensorMap* vmap, cudaStream_t stream);
// The kernels over windows, and the merge of units that CTAs share.
int launch_window(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream);
// The same as one launch, a cluster of `cluster` CTAs a unit.
int launch_window_cluster(const entmaxkv_pool& pool, const RangeArgs& a, int cluster, const CUtensorMap* kmap,
                          const CUtensorMap* vmap, cudaStream_t stream);

// x / ps for x >= 0 and the page sizes there are (a division by a variable takes
// longer than a step of the fp32 kernel)
template <typename T>
EKV_DEV T div_ps(T x, int ps) { return ps == 64 ? x >> 6 : x >> 4; }

// The pages a sequence's unit walks: logical pages [0, n1) and [p2, P), tokens
// valid where pos < s or w0 <= pos < L.
struct SeqSpan {
    int L, s, w0, n1, p2, P;
    EKV_DEV int pages() const { return n1 + P - p2; }
    EKV_DEV int tiles(int ps) const { return (int)(((long long)pages() * ps + kRangeTile - 1) / kRangeTile); }
    EKV_DEV int logical(int i) const { return i < n1 ? i : p2 + i - n1; }
    EKV_DEV bool valid(int pos) const { return pos < L && (pos < s || pos >= w0); }
};

EKV_DEV SeqSpan seq_span(const RangeArgs& a, int b, int ps, bool rep)
{
    SeqSpan r;
    r.L = max(a.seq_lens[b], 0);
    r.P = (int)div_ps((long long)r.L + ps - 1, ps);
    if (r.P > a.max_pages) {
        if (rep) report(a.status, ENTMAXKV_DEVICE_BOUNDS);
        r.P = a.max_pages;
    }
    if (a.shared) {
        r.s = 0;
        r.n1 = 0;
        r.p2 = min(a.shared[b], r.P);
        r.w0 = r.p2 * ps;
    } else {
        r.s = min(a.sinks, r.L);
        r.w0 = max(r.s, r.L - a.window);
        r.n1 = min((int)div_ps((long long)r.s + ps - 1, ps), r.P);
        r.p2 = min(max(div_ps(r.w0, ps), r.n1), r.P);
    }
    return r;
}

// a * b / c for a >= 0 and b, c in [0, 2^16); 64-bit division costs several times
// the 32-bit one, and nearly every total is small.
EKV_DEV long long mul_div(long long a, int b, int c)
{
    if (a < (1ll << 31) / max(b, 1)) return (int)a * b / c;
    return a * b / c;
}

// A CTA's share of the tiles: starts at tile t of unit (b, g), `left` tiles;
// C is the number of CTAs that have a share (each at least one tile).
struct RangeWalk {
    int b, g, t, C;
    long long left, total;
};

// Bounds of groups that a call does not use otherwise; one block.
EKV_DEV void range_check_groups(const RangeArgs& a)
{
    if (!a.group_start) return;
    for (int j = threadIdx.x; j <= a.n_groups; j += blockDim.x) {
        const int s = a.group_start[j];
        if (s < 0 || s > a.B || (j > 0 && s < a.group_start[j - 1])) report(a.status, ENTMAXKV_DEVICE_BOUNDS);
    }
}

// The share of the CTA `r` of a cluster of n that has unit u to itself.
EKV_DEV RangeWalk range_cluster_start(const RangeArgs& a, int ps, int u, int r, int n)
{
    if (u == 0 && r == 0) range_check_groups(a);
    RangeWalk w{};
    w.b = u / a.H_kv;
    w.g = u % a.H_kv;
    const int nt = seq_span(a, w.b, ps, w.g == 0 && r == 0).tiles(ps);
    w.t = (int)((long long)nt * r / n);
    w.left = (int)((long long)nt * (r + 1) / n) - w.t;
    return w;
}

// All threads of the block call.
EKV_DEV RangeWalk range_start(const RangeArgs& a, int ps, int c, int grid)
{
    __shared__ long long wsum[32];
    __shared__ int at[3];
    const int tid = threadIdx.x, n = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = n >> 5;
    RangeWalk w;
    long long mine = 0;
    int first = 0;                                     // tiles of sequence tid (the first chunk)
    for (int b = tid; b < a.B; b += n) {
        const int t = seq_span(a, b, ps, c == 0).tiles(ps);
        if (b == tid) first = t;
        mine += t;
    }
    if (c == 0) range_check_groups(a);
    const long long sum = warp_sum(mine);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < nw; ++i) total += wsum[i];
    total *= a.H_kv;
    const int C = (int)min((long long)grid, total);
    w.total = total;
    w.C = C;
    w.left = 0;
    w.b = w.g = w.t = 0;
    if (c >= C) return w;
    const long long t0 = mul_div(total, c, C);
    w.left = mul_div(total, c + 1, C) - t0;
    // the sequence that holds tile t0: chunks of blockDim sequences in turn
    long long before = 0;
    for (int base = 0; base < a.B; base += n) {
        const int b = base + tid;
        const int t = base == 0 ? first : (b < a.B ? seq_span(a, b, ps, false).tiles(ps) : 0);
        long long inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = inc;
        if (tid == 0) at[0] = -1;
        __syncthreads();
        long long off = before + inc - t, chunk = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < warp) off += wsum[i];
            chunk += wsum[i];
        }
        const long long in = t0 - off * a.H_kv;        // tile t0 within this sequence's units
        if (t > 0 && in >= 0 && in < (long long)t * a.H_kv) {
            at[0] = b;
            at[1] = (int)(in / t);
            at[2] = (int)(in % t);
        }
        __syncthreads();
        if (at[0] >= 0) break;
        before += chunk;
    }
    w.b = at[0];
    w.g = at[1];
    w.t = at[2];
    return w;
}

// The CTA whose share holds tile `at` of all tiles.
EKV_DEV int range_cta_of(long long at, long long total, int C)
{
    const long long x = (at + 1) * C - 1;
    return x < (1ll << 32) && total < (1ll << 32) ? (int)((uint32_t)x / (uint32_t)total) : (int)(x / total);
}

// Partial results of rows, one after the other: of partial s the row's maximum
// and sum lie at ml[s * step] and its four output dims at o[s * step * D / 4].
struct PartList {
    const float4* o;
    const float2* ml;
    long long step;
    int n;
};

// Threads of a merge CTA.  Few rows have many partials each (up to a CTA's worth)
// and SMs to spare; many rows have few.  Measured (the merge alone, profiled): 32
// CTAs of 75 partials 15.2 us with 256 threads, 10.0 with 1024; 768 CTAs of 8
// partials 11 us with 256, 16 with 512.
inline int merge_threads(int ctas) { return ctas <= num_sms() ? 1024 : 256; }

// Joins the partials of list x, then those of list y, of G rows of D dims: the
// block's threads form teams of G * D / 4 (one float4 of one row a thread),
// team t takes the partials t, t + teams, ... and the teams' results are joined
// in their order.  The first team's threads return true with the row's output
// (not yet divided by l), maximum and sum.  All threads of the block call.
template <int D, int THREADS>
EKV_DEV bool merge_parts(const PartList& x, const PartList& y, int G, float4& o, float& m, float& l)
{
    __shared__ float4 so[THREADS];
    __shared__ float2 sml[THREADS];
    const int items = G * (D / 4), teams = THREADS / items, team = threadIdx.x / items;
    m = -INFINITY;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](float4 t, float2 ml) {
        if (ml.y == 0.f) return;                       // no tokens (a sum that is NaN goes on)
        const float mn = fmaxf(m, ml.x);
        const float f = exp2f(m - mn), e = exp2f(ml.x - mn);
        m = mn;
        l = l * f + ml.y * e;
        o.x = o.x * f + t.x * e;
        o.y = o.y * f + t.y * e;
        o.z = o.z * f + t.z * e;
        o.w = o.w * f + t.w * e;
    };
    const int n = x.n + y.n;
    for (int s0 = team; s0 < n; s0 += 4 * teams) {
        float4 t[4];
        float2 ml[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int s = s0 + k * teams;
            if (s < n) {
                const PartList& p = s < x.n ? x : y;
                const long long at = (s < x.n ? s : s - x.n) * p.step;
                t[k] = p.o[at * (D / 4)];
                ml[k] = p.ml[at];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s0 + k * teams < n) join(t[k], ml[k]);
    }
    if (teams > 1 && n > 1) {
        so[threadIdx.x] = o;
        sml[threadIdx.x] = make_float2(m, l);
        __syncthreads();
        if (team == 0)
            for (int k = 1; k < min(teams, n); ++k) join(so[threadIdx.x + k * items], sml[threadIdx.x + k * items]);
    }
    return team == 0;
}

}  // namespace ekv
