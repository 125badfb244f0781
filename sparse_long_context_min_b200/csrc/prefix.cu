// Softmax decode for groups of sequences that share a prefix: the shared pages
// are read once for a whole group.
//
// All query heads of a kv head of all sequences of a group are the rows of one
// product S = Q K^T over the shared tokens (128 rows at 32 sequences of 4
// heads), so that what a decode token alone could not feed, the tensor cores,
// carries the work: tcgen05 with the accumulators in tensor memory.  The tokens
// behind the prefix are each sequence's own and go through the range kernels of
// window.cu; a merge joins a row's prefix partials and its own:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
#include "common.cuh"
#include "kernels.cuh"
#include "prefix.cuh"

#include <algorithm>

namespace ekv {

// ---------------------------------------------------------------- plan
// A group shares the whole pages below its prefix length and below its shortest
// sequence (empty sequences, as padding has them, do not count); a group with
// one sequence shares nothing.  The groups' bounds are clipped to [0, B] and
// held ascending (a running maximum), so that no sequence is in two groups
// whatever the caller passes.  One CTA.
constexpr int kPrefixPlanThreads = 512;

__global__ void __launch_bounds__(kPrefixPlanThreads) prefix_plan_kernel(const PrefixArgs a)
{
    pdl_enter();
    __shared__ long long wsum[3][kPrefixPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = kPrefixPlanThreads / 32;
    const int B = a.r.B, G = a.r.G;
    for (int b = tid; b < B; b += kPrefixPlanThreads) {
        a.shared[b] = 0;
        a.gid[b] = -1;
    }
    __shared__ int wmax[kPrefixPlanThreads / 32], end;
    int top = 0;                                       // largest bound so far
    for (int j0 = 0; j0 <= a.n_groups && a.n_groups > 0; j0 += kPrefixPlanThreads) {
        const int j = j0 + tid;
        int v = 0;
        if (j <= a.n_groups) {
            const int s = a.group_start[j];
            v = min(max(s, 0), B);
            if (v != s) report(a.r.status, ENTMAXKV_DEVICE_BOUNDS);
        }
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc = max(inc, t);
        }
        __syncthreads();
        if (lane == 31) wmax[warp] = inc;
        __syncthreads();
        int next = top;
        for (int i = 0; i < nw; ++i) {
            if (i < warp) top = max(top, wmax[i]);
            next = max(next, wmax[i]);
        }
        inc = max(inc, top);
        if (j <= a.n_groups && inc != v) report(a.r.status, ENTMAXKV_DEVICE_BOUNDS);
        if (j < a.n_groups) a.groups[j].lo = inc;
        if (j == a.n_groups) end = inc;
        top = next;
    }
    __syncthreads();
    for (int j = warp; j < a.n_groups; j += nw) {
        const int lo = a.groups[j].lo, hi = j + 1 < a.n_groups ? a.groups[j + 1].lo : end;
        int shortest = INT32_MAX, some = 0, first = INT32_MAX;
        for (int b = lo + lane; b < hi; b += 32) {
            const int L = a.r.seq_lens[b];
            if (L > 0) {
                shortest = min(shortest, L);
                first = min(first, b);
                ++some;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            shortest = min(shortest, __shfl_xor_sync(0xffffffffu, shortest, o));
            some += __shfl_xor_sync(0xffffffffu, some, o);
            first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        }
        int pages = some > 1 ? min(max(a.prefix_lens[j], 0), shortest) / a.ps : 0;
        pages = min(pages, a.r.max_pages);
        for (int b = lo + lane; b < hi; b += 32) {
            a.shared[b] = pages;
            a.gid[b] = j;
        }
        if (lane == 0) {
            PrefixGroup& g = a.groups[j];
            g.n = hi - lo;
            g.first = first;
            g.pages = pages;
            g.rows = pages ? g.n * G : 0;
            g.tiles = (g.rows + a.row_tile - 1) / a.row_tile;
            g.blocks = (int)(((long long)pages * a.ps + a.block_tok - 1) / a.block_tok);
        }
    }
    __syncthreads();
    // offsets of the groups' units, rows and blocks
    long long units = 0, rows = 0, blocks = 0;
    for (int j0 = 0; j0 < a.n_groups; j0 += kPrefixPlanThreads) {
        const int j = j0 + tid;
        long long v[3] = {0, 0, 0}, inc[3];
        if (j < a.n_groups) {
            const PrefixGroup& g = a.groups[j];
            v[0] = (long long)a.r.H_kv * g.tiles;
            v[1] = (long long)a.r.H_kv * g.rows;
            v[2] = v[0] * g.blocks;
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            inc[x] = v[x];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc[x], o);
                if (lane >= o) inc[x] += t;
            }
        }
        __syncthreads();
        if (lane == 31)
            for (int x = 0; x < 3; ++x) wsum[x][warp] = inc[x];
        __syncthreads();
        long long off[3] = {units, rows, blocks};
        for (int i = 0; i < nw; ++i) {
            units += wsum[0][i];
            rows += wsum[1][i];
            blocks += wsum[2][i];
            if (i < warp)
                for (int x = 0; x < 3; ++x) off[x] += wsum[x][i];
        }
        if (j < a.n_groups) {
            PrefixGroup& g = a.groups[j];
            g.unit0 = (int)(off[0] + inc[0] - v[0]);
            g.row0 = off[1] + inc[1] - v[1];
            g.block0 = off[2] + inc[2] - v[2];
        }
    }
    if (tid == 0) *a.total = blocks;
}

// ---------------------------------------------------------------- tensor memory
EKV_DEV void tc_alloc(uint32_t* smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
EKV_DEV void tc_dealloc(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
EKV_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
EKV_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
EKV_DEV void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
EKV_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
EKV_DEV void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// D[tmem] (+)= A[smem] B[smem], or A[tmem] B[smem]; bf16 in, fp32 accumulators
EKV_DEV void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
EKV_DEV void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
#define EKV_R8(r, o) "=r"((r)[o]), "=r"((r)[o + 1]), "=r"((r)[o + 2]), "=r"((r)[o + 3]), "=r"((r)[o + 4]), \
                     "=r"((r)[o + 5]), "=r"((r)[o + 6]), "=r"((r)[o + 7])
#define EKV_W8(r, o) "r"((r)[o]), "r"((r)[o + 1]), "r"((r)[o + 2]), "r"((r)[o + 3]), "r"((r)[o + 4]), \
                     "r"((r)[o + 5]), "r"((r)[o + 6]), "r"((r)[o + 7])
// 32 consecutive columns of this warp's 32 lanes, one lane a thread
EKV_DEV void tc_ld32(uint32_t addr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : EKV_R8(r, 0), EKV_R8(r, 8), EKV_R8(r, 16), EKV_R8(r, 24)
                 : "r"(addr));
}
EKV_DEV void tc_st32(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
                 ::EKV_W8(r, 0), EKV_W8(r, 8), EKV_W8(r, 16), EKV_W8(r, 24), "r"(addr) : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle: rows of 64 bf16, groups
// of 8 rows 1024 bytes apart.  `lead` is the distance of the next 64 columns
// of an operand whose rows run along K (V), unused where they run along K only.
EKV_DEV uint64_t tc_desc(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)((lead >> 4) & 0x3FFF) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// ---------------------------------------------------------------- bf16 cache
// One persistent CTA an SM.  Blocks of 128 tokens; S has two buffers and O two
// accumulators in tensor memory (4 x 128 columns): the two softmax warpgroups
// take the blocks in turn, each with its own running maximum, sum and O, so
// that neither waits for the other, and the products of one block run while
// the other block's weights are made.
//   warp 8  fills a ring of token blocks (K and V alternating) by TMA;
//   warp 9  issues the products: S = (Q_hi + Q_lo) K^T from shared memory,
//           O += (P_hi + P_lo) V with P read from tensor memory (it replaces S
//           there);
//   warps 0-3 / 4-7  one row a thread: maximum, weights, sum, P.
// Query and weights enter as a bf16 high and low part (2^-17 of relative error
// together), which doubles the products: at 128 rows 4 x 512 tensor cycles a
// block stand against ~2700 cycles in which HBM delivers its 64 KB, so the
// bytes still bound the time; more rows than a tile's 128 make the products
// bound it.  O is rescaled only when the maximum grew by more than 2^8, which
// keeps every weight in range and rescaling rare.
constexpr int kPfxRows = 128, kPfxTok = 128;
constexpr int kPfxThreads = 384;         // registers are dealt by warpgroup: two idle warps complete the third
constexpr float kPfxLazy = 8.f;

template <int D>
constexpr int pfx_slots() { return D == 128 ? 5 : 8; }

// 384 x 168 registers at launch: 128 x 40 for the producer and product warps
// leave 256 x 232 for the softmax, which holds a row's 128 scores.
EKV_DEV void regs_few() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
EKV_DEV void regs_many() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }

EKV_DEV void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Bounded wait of a warp, the same answer in all its lanes; a wait that ran out
// marks the CTA dead, after which every role runs to its end without waiting or
// issuing.
EKV_DEV bool pfx_wait(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status)
{
    bool ok = !*dead;
    if (ok && !mbar_wait(bar, parity, kWaitLimitNs)) {
        ok = false;
        *dead = 1;
        report(status, ENTMAXKV_TIMEOUT);
    }
    return __all_sync(0xffffffffu, ok);
}

template <int D, int PS>
__global__ void __launch_bounds__(kPfxThreads, 1) prefix_bf16_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                     const __grid_constant__ CUtensorMap vmap,
                                                                     const PrefixArgs a)
{
    pdl_enter();
    constexpr int SLOTS = pfx_slots<D>();
    constexpr int HALF = kPfxTok * 128;                // bytes of 64 columns of a block or of Q
    constexpr int TILE = HALF * (D / 64);
    constexpr int PPB = kPfxTok / PS;                  // pages a block
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    uint8_t* qs = smem;                                // Q high part, then low part
    uint8_t* ring = smem + 2 * TILE;
    __shared__ uint64_t full[SLOTS], empty[SLOTS], s_full[2], p_full[2], q_full, o_full;
    __shared__ uint32_t tmem_slot;
    __shared__ PrefixWalk start;
    __shared__ volatile int dead;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* status = a.r.status;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(&q_full, 8);
        mbar_init(&o_full, 1);
        fence_mbar_init();
        dead = 0;
        start = prefix_start(a, blockIdx.x);
    }
    __syncthreads();
    PrefixWalk w = start;
    if (w.left <= 0) return;
    if (warp == 9) tc_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t O[2] = {tmem, tmem + 128}, S[2] = {tmem + 256, tmem + 384};

    // setmaxnreg stands inside its role: code that both roles reach would get the smaller share
    if (warp < 8) {
        // ---------------------------------------------------- softmax
        regs_many();
        const int wg = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        int seg = 0, s_n = 0;
        while (w.left > 0) {
            const PrefixGroup G = a.groups[w.j];
            const int n = (int)min((long long)(G.blocks - w.k), w.left);
            const int rows = min(kPfxRows, G.rows - w.t * kPfxRows);
            if (tid == 0) prefix_note_span(a, w, G, blockIdx.x);
            // Q, scaled and split, a warp a row
            for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += 4) {
                float v[4][D / 32];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int rr = w.t * kPfxRows + r0 + r;
                    const bool in = r0 + r < rows;
                    const size_t at = ((size_t)(G.lo + rr / a.r.G) * a.r.H_q + (size_t)w.g * a.r.G + rr % a.r.G) * D;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e)
                        v[r][e] = in ? a.r.q[at + (e / 2) * 64 + 2 * lane + (e & 1)] * a.r.xscale : 0.f;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const int rr = r0 + r;
                        uint32_t h0, l0, h1, l1;
                        split_bf16(v[r][2 * h], h0, l0);
                        split_bf16(v[r][2 * h + 1], h1, l1);
                        const uint32_t o = h * HALF + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4;
                        *reinterpret_cast<uint32_t*>(qs + o) = pack2(h0, h1);
                        *reinterpret_cast<uint32_t*>(qs + TILE + o) = pack2(l0, l1);
                    }
            }
            fence_proxy_async();
            tc_fence_before();                         // the last unit's reads of O
            bar_softmax();
            if (lane == 0) mbar_arrive(&q_full);

            float m = -INFINITY, l = 0.f;
            for (int i = wg; i < n; i += 2) {
                const bool ok = pfx_wait(&s_full[wg], s_n++ & 1, &dead, status);
                tc_fence_after();
                if (ok && quad * 32 < rows) {
                    uint32_t s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_ld32(S[wg] + lanes + c * 32, s + c * 32);
                    tc_wait_ld();
                    const int valid = min(kPfxTok, (int)min((long long)G.pages * PS - (long long)(w.k + i) * kPfxTok,
                                                            (long long)kPfxTok));
                    if (valid < kPfxTok)
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c >= valid) s[c] = 0xff800000u;
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(s[c]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool grow = top > m + kPfxLazy || m == -INFINITY;
                    const float mnew = grow ? fmaxf(top, m) : m;
                    if (i >= 2 && __any_sync(0xffffffffu, grow)) {
                        // the products into this O before this block's scores have finished with them
                        const float f = m == -INFINITY ? 0.f : exp2f(m - mnew);
                        l *= f;
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tc_ld32(O[wg] + lanes + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st32(O[wg] + lanes + c, o);
                        }
                    }
                    m = mnew;
                    const float mu = m == -INFINITY ? 0.f : m;
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 128; c += 64) {
                        uint32_t hi[32], lo[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float p0 = exp2f(__uint_as_float(s[c + 2 * e]) - mu);
                            const float p1 = exp2f(__uint_as_float(s[c + 2 * e + 1]) - mu);
                            sum[0] += p0;
                            sum[1] += p1;
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi[e]) : "f"(p1), "f"(p0));
                            const float r0 = p0 - __uint_as_float(hi[e] << 16);
                            const float r1 = p1 - __uint_as_float(hi[e] & 0xffff0000u);
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo[e]) : "f"(r1), "f"(r0));
                        }
                        tc_st32(S[wg] + lanes + c / 2, hi);
                        tc_st32(S[wg] + lanes + 64 + c / 2, lo);
                    }
                    l += sum[0] + sum[1];
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[wg]);
            }
            // join the two accumulators: warpgroup x takes columns [x D/2, (x + 1) D/2) of every row
            const bool ok = pfx_wait(&o_full, seg & 1, &dead, status);
            tc_fence_after();
            float* ml = reinterpret_cast<float*>(qs);  // Q is not read any more
            ml[(wg * kPfxRows + row) * 2] = m;
            ml[(wg * kPfxRows + row) * 2 + 1] = l;
            bar_softmax();
            if (ok && quad * 32 < rows) {
                const float m0 = ml[row * 2], m1 = ml[(kPfxRows + row) * 2];
                const float M = fmaxf(m0, m1);
                const float f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - M), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M);
                const float L = ml[row * 2 + 1] * f0 + ml[(kPfxRows + row) * 2 + 1] * f1;
                const long long pr = prefix_part_row(a, G, w.g, w.t, blockIdx.x) + row;
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t x[32], y[32];
                    tc_ld32(O[0] + lanes + wg * (D / 2) + c, x);
                    if (n > 1) tc_ld32(O[1] + lanes + wg * (D / 2) + c, y);
                    tc_wait_ld();
                    if (row < rows) {
                        float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + wg * (D / 2) + c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float o[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[q] = __uint_as_float(x[4 * e + q]) * f0;
                                if (n > 1) o[q] = fmaf(__uint_as_float(y[4 * e + q]), f1, o[q]);
                            }
                            dst[e] = make_float4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                if (row < rows && wg == 0) {
                    a.part_ml[pr * 2] = M;
                    a.part_ml[pr * 2 + 1] = L;
                }
            }
            bar_softmax();                             // the maxima have been read: Q may come again
            ++seg;
            prefix_advance(a, w, n);
        }
    } else {
        regs_few();
        if (warp == 8) {
            // ---------------------------------------------------- producer
            if (lane == 0) {
                prefetch_tmap(&kmap);
                prefetch_tmap(&vmap);
            }
            int it = 0;                                    // ring slots filled so far
            auto load = [&](const CUtensorMap* map, const PrefixGroup& G, int g, int blk, int ph) {
                // lanes < PPB hold the block's physical pages (-1: none)
                const int slot = it % SLOTS;
                const bool go = it < SLOTS || pfx_wait(&empty[slot], (uint32_t)((it / SLOTS - 1) & 1), &dead, status);
                const uint32_t good = __ballot_sync(0xffffffffu, lane < PPB && ph >= 0);
                if (go) {
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], __popc(good) * PS * D * 2);
                    __syncwarp();
                    if (lane < PPB && ph >= 0)
    #pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_2d(ring + slot * TILE + h * HALF + lane * PS * 128, map, &full[slot], h * 64,
                                        (ph * a.r.H_kv + g) * PS);
                    ++it;
                }
                return go;
            };
            bool go = true;
            while (w.left > 0 && go) {
                const PrefixGroup G = a.groups[w.j];
                const int n = (int)min((long long)(G.blocks - w.k), w.left);
                // pages past the shared ones repeat the block's first page: their scores are masked, and
                // the weight of zero they get must meet a value that some row uses anyway
                auto page = [&](int blk) {
                    if (lane >= PPB) return -1;
                    int p = blk * PPB + lane;
                    if (p >= G.pages) p = blk * PPB;
                    const int ph = a.r.page_table[(size_t)G.first * a.r.max_pages + p];
                    if (ph < 0 || ph >= a.r.num_phys) {
                        report(status, ENTMAXKV_DEVICE_BOUNDS);
                        return -1;
                    }
                    return ph;
                };
                int ph = page(w.k), prev = -1;
                for (int i = 0; i <= n && go; ++i) {
                    const int next = i + 1 < n ? page(w.k + i + 1) : -1;
                    if (i < n) go = load(&kmap, G, w.g, w.k + i, ph);
                    if (i > 0 && go) go = load(&vmap, G, w.g, w.k + i - 1, prev);
                    prev = ph;
                    ph = next;
                }
                prefix_advance(a, w, n);
            }
            if (!go && lane == 0)
                for (int i = max(0, it - SLOTS); i < it; ++i)
                    mbar_wait(&full[i % SLOTS], (uint32_t)((i / SLOTS) & 1), kWaitLimitNs);
        } else if (warp == 9) {
            // ---------------------------------------------------- products
            constexpr uint32_t ID = (1u << 4) | (1u << 7) | (1u << 10) | ((kPfxRows / 16) << 24);
            constexpr uint32_t ID_QK = ID | ((kPfxTok / 8) << 17), ID_PV = ID | (1u << 16) | ((D / 8) << 17);
            const uint32_t q_addr = smem_addr(qs), r_addr = smem_addr(ring);
            int it = 0, seg = 0;
            int s_it[2] = {0, 0};                          // blocks given to each warpgroup
            while (w.left > 0) {
                const PrefixGroup G = a.groups[w.j];
                const int n = (int)min((long long)(G.blocks - w.k), w.left);
                bool ok = pfx_wait(&q_full, seg & 1, &dead, status);
                tc_fence_after();
                auto scores = [&](int i) {
                    const int slot = it % SLOTS;
                    ok = pfx_wait(&full[slot], (uint32_t)((it / SLOTS) & 1), &dead, status) && ok;
                    ++it;
                    if (!ok || lane != 0) return;
                    const uint32_t kb = r_addr + slot * TILE;
    #pragma unroll
                    for (int part = 0; part < 2; ++part)
    #pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t o = (k / 4) * HALF + (k % 4) * 32;
                            tc_mma_ss(S[i & 1], tc_desc(q_addr + part * TILE + o, 16), tc_desc(kb + o, 16), ID_QK,
                                      part + k > 0);
                        }
                    tc_commit(&empty[slot]);
                    tc_commit(&s_full[i & 1]);
                };
                auto values = [&](int i) {
                    const int slot = it % SLOTS, x = i & 1;
                    ok = pfx_wait(&full[slot], (uint32_t)((it / SLOTS) & 1), &dead, status) && ok;
                    ++it;
                    ok = pfx_wait(&p_full[x], s_it[x]++ & 1, &dead, status) && ok;
                    tc_fence_after();
                    if (!ok || lane != 0) return;
                    const uint32_t vb = r_addr + slot * TILE;
    #pragma unroll
                    for (int part = 0; part < 2; ++part)
    #pragma unroll
                        for (int k = 0; k < kPfxTok / 16; ++k)
                            tc_mma_ts(O[x], S[x] + part * 64 + k * 8, tc_desc(vb + k * 2048, HALF), ID_PV,
                                      i > 1 || part + k > 0);
                    tc_commit(&empty[slot]);
                };
                for (int i = 0; i <= n; ++i) {
                    if (i < n) scores(i);
                    if (i > 0) values(i - 1);
                }
                if (lane == 0 && ok) tc_commit(&o_full);
                __syncwarp();
                ++seg;
                prefix_advance(a, w, n);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tc_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- merge
// One CTA a (sequence, kv head): the prefix partials in CTA order, then its own.
template <int D>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixArgs a)
{
    pdl_enter();
    const RangeArgs& r = a.r;
    const int u = blockIdx.x, b = u / r.H_kv, g = u % r.H_kv;
    const SeqSpan sp = seq_span(r, b, a.ps, false);
    const int j = a.gid[b];
    int n_own = 0, n_pfx = 0;
    long long own0 = 0, pfx0 = 0;
    if (sp.pages() > 0) {
        const int2 s = r.span[u];
        n_own = s.y - s.x + 1;
        own0 = ((long long)s.x + u) * r.G;
    }
    if (sp.L > 0 && j >= 0 && a.groups[j].pages > 0) {
        const PrefixGroup G = a.groups[j];
        const int row = (b - G.lo) * r.G, t = row / a.row_tile;
        const int2 s = a.span[prefix_unit(G, g, t)];
        n_pfx = s.y - s.x + 1;
        pfx0 = prefix_part_row(a, G, g, t, s.x) + row % a.row_tile;
    }
    for (int i = threadIdx.x; i < r.G * D / 4; i += blockDim.x) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float M = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float* po, const float* pml, long long row, long long step, int n) {
            for (int s0 = 0; s0 < n; s0 += 8) {
                float4 t[8];
                float2 ml[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (s0 + k < n) {
                        const long long at = row + (s0 + k) * step;
                        t[k] = *reinterpret_cast<const float4*>(po + at * D + d);
                        ml[k] = *reinterpret_cast<const float2*>(pml + at * 2);
                    }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (s0 + k < n && ml[k].x != -INFINITY) {
                        const float mn = fmaxf(M, ml[k].x);
                        const float f = exp2f(M - mn), e = exp2f(ml[k].x - mn);
                        M = mn;
                        l = l * f + ml[k].y * e;
                        o.x = o.x * f + t[k].x * e;
                        o.y = o.y * f + t[k].y * e;
                        o.z = o.z * f + t[k].z * e;
                        o.w = o.w * f + t[k].w * e;
                    }
            }
        };
        add(a.part_o, a.part_ml, pfx0 + h, a.row_tile, n_pfx);
        add(r.part_o, r.part_ml, own0 + h, r.G, n_own);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t row = (size_t)b * r.H_q + (size_t)g * r.G + h;
        float* dst = r.out + row * D + d;
        dst[0] = o.x * inv;
        dst[1] = o.y * inv;
        dst[2] = o.z * inv;
        dst[3] = o.w * inv;
        if (d == 0 && r.lse) r.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    }
}

// ---------------------------------------------------------------- launch
template <int D, int PS>
static int launch_prefix_bf16(const PrefixArgs& a, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              cudaStream_t stream)
{
    const int smem = (2 + pfx_slots<D>()) * kPfxTok * D * 2 + 1024;
    if (ensure_smem((const void*)prefix_bf16_kernel<D, PS>, smem)) return ENTMAXKV_CUDA_ERROR;
    return launch_pdl(prefix_bf16_kernel<D, PS>, dim3(a.C), dim3(kPfxThreads), smem, stream, *kmap, *vmap, a) ==
                   cudaSuccess
               ? ENTMAXKV_OK
               : ENTMAXKV_CUDA_ERROR;
}

int launch_prefix(const entmaxkv_pool& pool, const PrefixArgs& a, int range_C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream)
{
    if (launch_pdl(prefix_plan_kernel, dim3(1), dim3(kPrefixPlanThreads), 0, stream, a) != cudaSuccess)
        return ENTMAXKV_CUDA_ERROR;
    int rc = ENTMAXKV_OK;
    if (pool.dtype == ENTMAXKV_BF16) {
        if (pool.d == 128)
            rc = pool.ps == 64 ? launch_prefix_bf16<128, 64>(a, kmap, vmap, stream)
                               : launch_prefix_bf16<128, 16>(a, kmap, vmap, stream);
        else
            rc = pool.ps == 64 ? launch_prefix_bf16<64, 64>(a, kmap, vmap, stream)
                               : launch_prefix_bf16<64, 16>(a, kmap, vmap, stream);
    }
    if (rc) return rc;
    if ((rc = launch_range(pool, a.r, range_C, kmap, vmap, stream))) return rc;
    const dim3 grid(a.r.B * a.r.H_kv);
    const cudaError_t e = pool.d == 128 ? launch_pdl(prefix_merge_kernel<128>, grid, dim3(128), 0, stream, a)
                                        : launch_pdl(prefix_merge_kernel<64>, grid, dim3(128), 0, stream, a);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

}  // namespace ekv
