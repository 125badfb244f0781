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
    constexpr int N = kPrefixPlanThreads, CHUNK = N - 1;   // groups at a time: their bounds are one more
    __shared__ int bound[N], pages_of[N], first_of[N], wmax[N / 32];
    __shared__ long long wsum[2][N / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = N / 32;
    const int B = a.r.B, G = a.r.G;
    for (int b = tid; b < B; b += N) {
        a.shared[b] = 0;
        a.gid[b] = -1;
    }
    int top = 0;                                       // largest bound so far
    long long rows0 = 0, blocks0 = 0;
    for (int j0 = 0; j0 < a.n_groups; j0 += CHUNK) {
        const int cnt = min(CHUNK, a.n_groups - j0), j = j0 + tid;
        int v = 0;
        if (tid <= cnt) {
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
        if (lane == 31) wmax[warp] = inc;
        __syncthreads();
        for (int i = 0; i < warp; ++i) top = max(top, wmax[i]);
        inc = max(inc, top);
        if (tid <= cnt && inc != v) report(a.r.status, ENTMAXKV_DEVICE_BOUNDS);
        bound[tid] = inc;
        __syncthreads();
        for (int i = warp; i < cnt; i += nw) {
            const int lo = bound[i], hi = bound[i + 1];
            int shortest = INT32_MAX, some = 0, first = INT32_MAX;
            for (int b = lo + lane; b < hi; b += 32) {
                const int L = a.r.seq_lens[b];
                if (L > 0) {
                    shortest = min(shortest, L);
                    first = min(first, b);
                    ++some;
                }
            }
            shortest = __reduce_min_sync(0xffffffffu, shortest);
            some = __reduce_add_sync(0xffffffffu, some);
            first = __reduce_min_sync(0xffffffffu, first);
            const int pages = some > 1 ? min(min(max(a.prefix_lens[j0 + i], 0), shortest) / a.ps, a.r.max_pages) : 0;
            for (int b = lo + lane; b < hi; b += 32) {
                a.shared[b] = pages;
                a.gid[b] = j0 + i;
            }
            if (lane == 0) {
                pages_of[i] = pages;
                first_of[i] = first;
            }
        }
        __syncthreads();
        // offsets of the groups' rows and blocks
        PrefixGroup g{};
        long long x[2] = {0, 0}, sum[2];
        if (tid < cnt) {
            g.lo = bound[tid];
            g.n = bound[tid + 1] - g.lo;
            g.first = first_of[tid];
            g.pages = pages_of[tid];
            g.rows = g.pages ? g.n * G : 0;
            g.tiles = (g.rows + a.row_tile - 1) / a.row_tile;
            g.blocks = (int)(((long long)g.pages * a.ps + a.block_tok - 1) / a.block_tok);
            x[0] = (long long)a.r.H_kv * g.rows;
            x[1] = (long long)a.r.H_kv * g.tiles * prefix_len(g);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] = x[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, sum[i], o);
                if (lane >= o) sum[i] += t;
            }
            if (lane == 31) wsum[i][warp] = sum[i];
        }
        __syncthreads();
        g.row0 = rows0 + sum[0] - x[0];
        g.block0 = blocks0 + sum[1] - x[1];
        for (int i = 0; i < nw; ++i) {
            if (i < warp) {
                g.row0 += wsum[0][i];
                g.block0 += wsum[1][i];
            }
            rows0 += wsum[0][i];
            blocks0 += wsum[1][i];
        }
        if (tid < cnt) a.groups[j] = g;
        top = bound[cnt];
        __syncthreads();
    }
    const int C = (int)min((long long)a.C, blocks0);
    if (tid == 0) *a.head = PrefixHead{blocks0, C};
    for (int c = tid; c < a.C; c += N) a.walks[c] = c < C ? prefix_start(a, c, blocks0, C) : PrefixWalk{};
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
// (the loaded values pass through, so that their uses stay behind the wait)
template <int N>
EKV_DEV void tc_wait_ld(uint32_t* r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
EKV_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
EKV_DEV void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// Operand descriptors in shared memory, 128-byte swizzle: rows of 64 bf16,
// groups of 8 rows 1024 bytes apart.  The low word holds the address and, for
// an operand whose rows run along K (V), the distance of the next 64 columns;
// the high word is the same for all.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
EKV_DEV uint32_t tc_desc(uint32_t addr, uint32_t lead)
{
    return ((addr & 0x3FFFF) >> 4) | (((lead >> 4) & 0x3FFF) << 16);
}
// D[tmem] (+)= A[tmem] B[smem], bf16 in, fp32 accumulators; b is a descriptor's low word.
EKV_DEV void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %4, 0;\n"
                 " mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHigh) : "memory");
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
EKV_DEV void tc_ld16(uint32_t addr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : EKV_R8(r, 0), EKV_R8(r, 8)
                 : "r"(addr));
}
EKV_DEV void tc_st16(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
                 ::EKV_W8(r, 0), EKV_W8(r, 8), "r"(addr) : "memory");
}
// 16 lanes x 8 columns: a thread's words are columns 2 (lane % 4) and the next, of rows lane / 4 and lane / 4 + 8
EKV_DEV void tc_st_16x256(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%4], {%0, %1, %2, %3};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(addr) : "memory");
}
EKV_DEV void tc_st8(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 ::EKV_W8(r, 0), "r"(addr) : "memory");
}

// ---------------------------------------------------------------- pairs of floats
EKV_DEV uint64_t pair(uint32_t x, uint32_t y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
EKV_DEV uint64_t pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
EKV_DEV float2 unpair(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
EKV_DEV uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
EKV_DEV uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
// 2^x for scores below their row's maximum (plus 8): results under 2^-126 become zero
EKV_DEV float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// integers in the order of the floats
EKV_DEV int ordered_int(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
EKV_DEV float ordered_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
EKV_DEV uint32_t bf16x2(float2 v)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}

// ---------------------------------------------------------------- bf16 cache
// One persistent CTA an SM walks its share of blocks of 64 tokens.  Tensor
// memory (512 columns at 128 dims): two accumulators O, two score buffers S,
// and Q.  Two sets of eight softmax warps take the blocks in turn, each set
// with its own running maximum, sum and O, so that neither waits for the other
// and the products of one block run while the other block's weights are made.
//   warps 0-15   four a row quarter: set, and half of the block's tokens; one
//                row a lane: maximum, weights, sum, P in place of S;
//   warp 16      fills a ring of token blocks (K and V alternating) by TMA;
//   warp 17      issues the products S = (Q_hi + Q_lo) K^T and
//                O += (P_hi + P_lo) V, with Q and P read from tensor memory, so
//                that shared memory feeds one operand only.
// Query and weights enter as a bf16 high and low part (2^-17 of relative error
// each at most, 3.4e-6 rms together), which doubles the products: at 128 rows
// 1024 tensor cycles a block, where HBM takes ~1300 cycles of a full clock to
// deliver its 32 KB.  At full clock the bytes bound the time then; when the power
// cap lowers the clock, and with more rows than a tile's 128, the products do.
// A third part would need more tensor memory than there is beside two
// accumulators.  O is rescaled only when the maximum grew by more than 2^8, which
// keeps every weight in range and rescaling rare.
//
// Measured (the kernel alone, profiled; 8 kv heads of 128 dims): 128 rows behind
// 131072 tokens 93 to 107 us, 5.8 to 5.0 TB/s, by the clock that the power cap
// leaves; 384 rows behind 32809 72 to 84 us (84 at 1.6 GHz, the tensor pipe busy 64%
// of the time: 1275 cycles a block, of which the product warp waits a fifth).
// With blocks of 128 tokens and Q in shared memory the latter took 118 us.
constexpr int kPfxRows = 128, kPfxTok = 64;
constexpr int kPfxSoft = 16;             // softmax warps
constexpr int kPfxThreads = (kPfxSoft + 2) * 32;
constexpr float kPfxLazy = 8.f;

template <int D>
constexpr int pfx_slots() { return D == 128 ? 13 : 24; }

// A value that all lanes of the warp hold, told to the compiler: the tensor
// instructions take their operands from the warp's uniform registers, and one
// that has to be moved there first costs the issuing warp more than the product.
template <typename T>
EKV_DEV T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }
EKV_DEV bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

EKV_DEV void bar_softmax() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
// the two warps that share rows' scores
EKV_DEV void bar_halves(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id + 2) : "memory"); }

// Bounded wait of a warp, the same answer in all its lanes; a wait that ran out
// marks the CTA dead, after which every role runs to its end without waiting or
// issuing.
__device__ __noinline__ bool pfx_wait_long(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status)
{
    bool ok = !*dead;
    if (ok && !mbar_wait_chain(bar, parity, kWaitLimitNs)) {
        ok = false;
        *dead = 1;
        report(status, ENTMAXKV_TIMEOUT);
    }
    return __all_sync(0xffffffffu, ok);
}
EKV_DEV bool pfx_wait(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return pfx_wait_long(bar, parity, dead, status);
}

template <int D, int PS>
__global__ void __launch_bounds__(kPfxThreads, 1) prefix_bf16_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                     const __grid_constant__ CUtensorMap vmap,
                                                                     const PrefixArgs a)
{
    constexpr int SLOTS = pfx_slots<D>();
    constexpr int HALF = kPfxTok * 128;                // bytes of 64 columns of a block
    constexpr int TILE = HALF * (D / 64);
    constexpr int PPB = kPfxTok / PS;                  // pages a block
    constexpr int QD = D / 4;                          // dims of a row that one thread stages
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align<1024>(smem_raw);
    __shared__ uint64_t full[SLOTS], empty[SLOTS], s_full[2], p_full[2], q_full, o_full, drained;
    __shared__ uint32_t tmem_slot;
    __shared__ PrefixWalk start;
    __shared__ int top_of[2][kPfxRows];                // [set][row] largest score so far, as an ordered integer
    __shared__ float2 ml[4][kPfxRows];
    __shared__ volatile int dead;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    int32_t* status = a.r.status;

    // nothing here touches global memory: it runs under the end of the kernel before
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
        }
        mbar_init(&q_full, kPfxSoft);
        mbar_init(&o_full, 1);
        mbar_init(&drained, 1);
        fence_mbar_init();
        dead = 0;
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (warp == kPfxSoft + 1) tc_alloc(&tmem_slot, 512);
    pdl_enter();
    if (tid == 0) start = a.walks[blockIdx.x];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    PrefixWalk w = start;
    const uint32_t tmem = uniform(tmem_slot);
    const uint32_t O[2] = {tmem, tmem + 128}, S[2] = {tmem + 256, tmem + 320}, Q = tmem + 384;

    if (warp < kPfxSoft) {
        // ---------------------------------------------------- softmax
        const int set = warp >> 3, half = (warp >> 2) & 1, quarter = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t at = S[set] + lanes + half * 32, acc = O[set] + lanes + half * (D / 2);
        const int lg = __ffs(a.r.G) - 1;
        // Q goes to tensor memory in blocks of 16 rows x 16 dims: a lane holds four dims of rows lane / 4 and
        // lane / 4 + 8 of each, so that four lanes read 64 consecutive bytes (a row a lane took 3 us longer to
        // fetch 128 rows)
        constexpr int QB = QD / 16;                    // such blocks along this warp's dims
        float4 qv[2][QB][2];
        auto load_q = [&] {
            const PrefixGroup& G = a.groups[w.j];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = w.t * kPfxRows + quad * 32 + i * 8 + (lane >> 2);
                const size_t at_q = (size_t)(G.lo + (r >> lg)) * a.r.H_q + ((size_t)w.g << lg) + (r & (a.r.G - 1));
                const float* q = a.r.q + at_q * D + quarter * QD + (lane & 3) * 4;
#pragma unroll
                for (int e = 0; e < QB; ++e)
                    qv[i / 2][e][i % 2] = r < G.rows ? *reinterpret_cast<const float4*>(q + e * 16)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        auto stage_q = [&] {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < QB; ++e) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 v = qv[i][e][k / 2];
                        const float2 x = k % 2 ? make_float2(v.z * a.r.xscale, v.w * a.r.xscale)
                                               : make_float2(v.x * a.r.xscale, v.y * a.r.xscale);
                        hi[k] = bf16x2(x);
                        lo[k] = bf16x2(make_float2(x.x - __uint_as_float(hi[k] << 16),
                                                   x.y - __uint_as_float(hi[k] & 0xffff0000u)));
                    }
                    const uint32_t dst = Q + lanes + (i << 20) + quarter * (QD / 2) + e * 8;
                    tc_st_16x256(dst, hi);
                    tc_st_16x256(dst + D / 2, lo);
                }
            if (half == 0) top_of[set][row] = ordered_int(-INFINITY);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
        };
        int seg = 0, s_n = 0, k, n;
        bool more = prefix_segment(a, w, k, n), again = false;   // again: the unit's partial holds segments before
        float m_unit = -INFINITY, l_unit = 0.f;        // their maximum and sum
        if (more) {
            load_q();
            stage_q();
            bar_softmax();
        }
        while (more) {
            const PrefixGroup& G = a.groups[w.j];
            const int rows = min(kPfxRows, G.rows - w.t * kPfxRows);
            // tokens from this warp's first column of the first block to the end of the shared pages
            const int ahead = (int)min((long long)G.pages * PS - (long long)k * kPfxTok - half * 32, 0x7fffffffll);
            const long long part_row = prefix_part_row(a, G, w.g, w.t, blockIdx.x);

            float m = -INFINITY, l = 0.f;
            for (int i = set; i < n; i += 2, ++s_n) {
                // whatever comes of the wait: the other half's warp counts on this one at the barrier below,
                // and scores that never came do no harm (the status says so)
                pfx_wait(&s_full[set], s_n & 1, &dead, status);
                tc_fence_after();
                if (quad * 32 < rows) {
                    uint32_t s[32];
                    tc_ld32(at, s);
                    tc_wait_ld<32>(s);
                    const int valid = ahead - i * kPfxTok;
                    if (valid < 32)                    // columns past the shared pages
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e >= valid) s[e] = 0xff800000u;
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
                    // both halves raise the row's maximum (the next block's scores only come when both have
                    // given up this block's weights, so nobody raises it before it has been read)
                    atomicMax(&top_of[set][row], ordered_int(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]))));
                    bar_halves(set * 4 + quad);
                    const float top = ordered_float(*(volatile int*)&top_of[set][row]);
                    const bool grow = top > m + kPfxLazy || m == -INFINITY;
                    const float mnew = grow ? top : m;
                    if (i >= 2 && __any_sync(0xffffffffu, grow)) {
                        // the products into this O before this block's scores have finished with them
                        const float f = m == -INFINITY ? 0.f : ex2(m - mnew);
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tc_ld16(acc + c, o);
                            tc_wait_ld<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st16(acc + c, o);
                        }
                    }
                    m = mnew;
                    const float mu = m == -INFINITY ? 0.f : m;
                    const uint64_t down = pair(-mu, -mu), minus = pair(-1.f, -1.f);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 32; c += 16) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 y = unpair(add2(pair(s[c + 2 * e], s[c + 2 * e + 1]), down));
                            const float2 p = make_float2(ex2(y.x), ex2(y.y));
                            const uint64_t pp = pair(p.x, p.y);
                            sum[e & 1] = add2(sum[e & 1], pp);
                            hi[e] = bf16x2(p);
                            lo[e] = bf16x2(unpair(fma2(pair(hi[e] << 16, hi[e] & 0xffff0000u), minus, pp)));
                        }
                        // weights in place of their scores: of 16 tokens 8 words of high, 8 of low parts
                        tc_st8(at + c, hi);
                        tc_st8(at + c + 8, lo);
                    }
                    const float2 t = unpair(add2(sum[0], sum[1]));
                    l += t.x + t.y;
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[set]);
            }
            // the next unit's query goes out before this unit's results: its first products run meanwhile
            const bool two = n > 1;
            prefix_advance(a, w);
            const bool same = w.k > 0;
            more = prefix_segment(a, w, k, n);
            if (more) load_q();
            const bool ok = pfx_wait(&o_full, seg & 1, &dead, status);
            tc_fence_after();
            ml[quarter][row] = make_float2(m, l);
            bar_softmax();                             // also: nobody reads this unit's maxima any more
            if (more) stage_q();
            // join the two accumulators: a warp takes D/4 columns of its rows
            if (ok && quad * 32 < rows) {
                const float m0 = ml[0][row].x, m1 = ml[2][row].x;
                const float M = fmaxf(again ? m_unit : -INFINITY, fmaxf(m0, m1));
                const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                const float fu = !again || m_unit == -INFINITY ? 0.f : ex2(m_unit - M);
                // partials lie [D / 4][rows] float4: the lanes of a warp store 512 consecutive bytes
                float4* dst = reinterpret_cast<float4*>(a.part_o + part_row * D) + row;
#pragma unroll
                for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); c += 16) {
                    uint32_t x[16], y[16] = {};
                    tc_ld16(O[0] + lanes + c, x);
                    if (two) tc_ld16(O[1] + lanes + c, y);
                    tc_wait_ld<16>(x);
                    tc_wait_ld<16>(y);
                    if (row < rows)
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float o[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[q] = __uint_as_float(x[e + q]) * f0;
                                if (two) o[q] = fmaf(__uint_as_float(y[e + q]), f1, o[q]);
                            }
                            float4& to = dst[(c + e) / 4 * rows];
                            if (again) {               // this thread's own words
                                const float4 u = to;
                                o[0] = fmaf(u.x, fu, o[0]);
                                o[1] = fmaf(u.y, fu, o[1]);
                                o[2] = fmaf(u.z, fu, o[2]);
                                o[3] = fmaf(u.w, fu, o[3]);
                            }
                            to = make_float4(o[0], o[1], o[2], o[3]);
                        }
                }
                l_unit = (ml[0][row].y + ml[1][row].y) * f0 + (ml[2][row].y + ml[3][row].y) * f1 +
                         (again ? l_unit * fu : 0.f);
                m_unit = M;
                if (row < rows && quarter == 0)
                    reinterpret_cast<float2*>(a.part_ml)[part_row + row] = make_float2(m_unit, l_unit);
            }
            again = same;
            tc_fence_before();
            bar_softmax();                             // O and ml may come again
            ++seg;
        }
    } else if (warp == kPfxSoft) {
        // ---------------------------------------------------- producer
        int it = 0;                                    // ring slots filled so far
        auto load = [&](const CUtensorMap* map, int g, int ph) {
            // lanes < PPB hold the block's physical pages (negative: none)
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
        for (int k, n; go && prefix_segment(a, w, k, n); prefix_advance(a, w)) {
            const PrefixGroup& G = a.groups[w.j];
            const int g = w.g;
            const int32_t* pages = a.r.page_table + (size_t)G.first * a.r.max_pages;
            // 32 pages at a time, one a lane, so that their loads are waited for once
            const int end = (k + n) * PPB;
            auto page = [&](int p) {
                if (p >= end) return -1;
                // pages past the shared ones repeat the block's first page: their scores are masked, and
                // the weight of zero they get must meet a value that some row uses anyway
                if (p >= G.pages) p &= ~(PPB - 1);
                const int ph = pages[p];
                if (ph < 0 || ph >= a.r.num_phys) {
                    report(status, ENTMAXKV_DEVICE_BOUNDS);
                    return -1;
                }
                return ph;
            };
            int batch = -1, prev = -1;
            for (int i = 0; i <= n && go; ++i) {
                const int at = i * PPB & 31;
                if (at == 0) batch = page((k + i) * PPB + lane);
                const int ph = __shfl_sync(0xffffffffu, batch, (at + lane) & 31);
                if (i < n) go = load(&kmap, g, ph);
                if (i > 0 && go) go = load(&vmap, g, prev);
                prev = ph;
            }
        }
        // nothing may be on its way when the CTA ends (roles that gave up do not wait for it)
        if (lane == 0)
            for (int i = max(0, it - SLOTS); i < it; ++i)
                mbar_wait(&full[i % SLOTS], (uint32_t)((i / SLOTS) & 1), kWaitLimitNs);
    } else {
        // ---------------------------------------------------- products
        constexpr uint32_t ID = (1u << 4) | (1u << 7) | (1u << 10) | ((kPfxRows / 16) << 24);
        constexpr uint32_t ID_QK = ID | ((kPfxTok / 8) << 17), ID_PV = ID | (1u << 16) | ((D / 8) << 17);
        const uint32_t ring0 = uniform(smem_addr(ring));
        int slot = 0, seg = 0;
        uint32_t filled = 0, given[2] = {0, 0};        // parities: ring slots, blocks given to each set
        auto next_slot = [&] {
            if (++slot == SLOTS) {
                slot = 0;
                filled ^= 1;
            }
        };
        auto scores = [&](int x) {
            if (!pfx_wait(&full[slot], filled, &dead, status)) return;
            const uint32_t kd = tc_desc(ring0 + slot * TILE, 16);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma_ts(S[x], Q + part * (D / 2) + k * 8, kd + (((k / 4) * HALF + (k % 4) * 32) >> 4), ID_QK,
                                  part + k > 0);
                tc_commit(&empty[slot]);
                tc_commit(&s_full[x]);
            }
            __syncwarp();
            next_slot();
        };
        auto values = [&](int x, bool first) {
            if (!pfx_wait(&full[slot], filled, &dead, status)) return;
            const bool ok = pfx_wait(&p_full[x], given[x], &dead, status);
            given[x] ^= 1;
            if (!ok) return;
            tc_fence_after();
            const uint32_t vd = tc_desc(ring0 + slot * TILE, HALF);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < kPfxTok / 16; ++k)
                        tc_mma_ts(O[x], S[x] + k * 16 + part * 8, vd + ((k * 2048) >> 4), ID_PV,
                                  part + k > 0 || !first);
                tc_commit(&empty[slot]);
            }
            __syncwarp();
            next_slot();
        };
        for (int k, n; uniform(prefix_segment(a, w, k, n)); prefix_advance(a, w)) {
            n = uniform(n);
            pfx_wait(&q_full, seg & 1, &dead, status);
            tc_fence_after();
            // S0, then S1 V0, S0 V1, ...: each set's scores are made while the other's weights are
            scores(0);
            int i = 1;
            for (; i + 1 < n; i += 2) {
                scores(1);
                values(0, i == 1);
                scores(0);
                values(1, i == 1);
            }
            if (i < n) {
                scores(1);
                values(0, i == 1);
                values(1, i == 1);
            } else {
                values(0, i == 1);
            }
            if (__all_sync(0xffffffffu, !dead) && elect_one()) tc_commit(&o_full);
            __syncwarp();
            ++seg;
        }
        // nor may products (where the softmax warps gave up, nobody has waited for them)
        if (elect_one()) tc_commit(&drained);
        __syncwarp();
        if (!mbar_wait(&drained, 0, kWaitLimitNs)) report(status, ENTMAXKV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kPfxSoft + 1) tc_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- fp32 cache
// The same walk with all arithmetic in fp32: 32 rows and 64 tokens at a time on
// the ordinary pipes, two multiply-adds an instruction (f32x2).  A producer warp
// keeps two blocks of keys and of values in shared memory; each of eight warps
// has 8 rows and 32 tokens of every block to itself, scores (a lane a token) and
// output (a lane D / 32 dims), with its own softmax state, so that no barrier
// stands between the blocks; the token halves are joined at a unit's end.
// Reading shared memory bounds it (its pipe is 77% busy at 64 rows): 20 cycles a
// warp for 32 multiply-adds a lane of the scores, 8 of the output, 7200 cycles a
// block of 32 rows and 128 dims against ~2600 in which HBM delivers its 64 KB;
// warps without rows stay out of the way.
constexpr int kPfxRowsF32 = 32;
constexpr int kPfxThreadsF32 = 288;

template <int D>
struct PfxF32 {
    static constexpr int KROW = D + 4, PROW = 12;      // padded rows (floats): no two lanes of a read meet in a bank
    static constexpr int K = 64 * KROW, V = 64 * D, Q = 32 * KROW, P = 8 * 32 * PROW;
    static constexpr int FLOATS = 2 * K + 2 * V + Q + P;
};

EKV_DEV void bar_f32() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int D, int PS>
__global__ void __launch_bounds__(kPfxThreadsF32, 1) prefix_f32_kernel(const float* __restrict__ k_pool,
                                                                       const float* __restrict__ v_pool,
                                                                       const PrefixArgs a)
{
    pdl_enter();
    using L = PfxF32<D>;
    constexpr int KROW = L::KROW, PROW = L::PROW, PPB = 64 / PS, W = D / 32;   // W: output dims of a lane
    extern __shared__ __align__(128) float sm[];
    float* ks = sm;                                    // [2][64][KROW]
    float* vs = ks + 2 * L::K;                         // [2][64][D]
    float* qs = vs + 2 * L::V;                         // [32][KROW]; then the second token half's output
    float* ps = qs + L::Q;                             // [8 warps][32 tokens][PROW]
    __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    __shared__ float2 ml[32];                          // the second token half's maxima and sums
    __shared__ volatile int dead;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* status = a.r.status;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&k_empty[i], 8);
            mbar_init(&v_empty[i], 8);
        }
        fence_mbar_init();
        dead = 0;
    }
    __syncthreads();
    PrefixWalk w = a.walks[blockIdx.x];
    int k0, n;
    if (warp == 8) {
        // ---------------------------------------------------- producer
        int it = 0;
        bool go = true;
        for (; go && prefix_segment(a, w, k0, n); prefix_advance(a, w)) {
            const PrefixGroup& G = a.groups[w.j];
            const int32_t* pages = a.r.page_table + (size_t)G.first * a.r.max_pages;
            for (int i = 0; i < n && go; ++i, ++it) {
                // a token's page; pages past the shared ones repeat the block's first (their scores are masked,
                // and the weight of zero must meet a value that some row uses anyway)
                int ph = -1;
                if (lane < PPB) {
                    int p = (k0 + i) * PPB + lane;
                    if (p >= G.pages) p = (k0 + i) * PPB;
                    ph = pages[p];
                    if (ph < 0 || ph >= a.r.num_phys) {
                        report(status, ENTMAXKV_DEVICE_BOUNDS);
                        ph = -1;
                    }
                }
                const int slot = it & 1;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ph >= 0)) * PS * D * 4;
                if (it >= 2) go = pfx_wait(&k_empty[slot], ((it >> 1) - 1) & 1, &dead, status);
                if (!go) break;
                if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], bytes);
                __syncwarp();
                for (int t = lane; t < 64; t += 32) {
                    const int phys = __shfl_sync(0xffffffffu, ph, t / PS);
                    if (phys >= 0)
                        bulk_load(ks + slot * L::K + t * KROW,
                                  k_pool + (((size_t)phys * a.r.H_kv + w.g) * PS + t % PS) * D, D * 4, &k_full[slot]);
                }
                if (it >= 2) go = pfx_wait(&v_empty[slot], ((it >> 1) - 1) & 1, &dead, status);
                if (!go) {                             // the keys on their way must land
                    if (lane == 0) mbar_wait(&k_full[slot], (it >> 1) & 1, kWaitLimitNs);
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&v_full[slot], bytes);
                __syncwarp();
                if (ph >= 0)
                    bulk_load(vs + slot * L::V + lane * PS * D, v_pool + ((size_t)ph * a.r.H_kv + w.g) * PS * D,
                              PS * D * 4, &v_full[slot]);
            }
        }
        if (lane == 0)                                 // and so must the blocks before, whoever gave up
            for (int i = max(0, it - 2); i < it; ++i) {
                mbar_wait(&k_full[i & 1], (i >> 1) & 1, kWaitLimitNs);
                mbar_wait(&v_full[i & 1], (i >> 1) & 1, kWaitLimitNs);
            }
        return;
    }
    // -------------------------------------------------------- consumers
    const int half = warp >> 2, r8 = (warp & 3) * 8;
    float* pw = ps + warp * 32 * PROW;
    const int lg = __ffs(a.r.G) - 1;
    int it = 0;
    for (; prefix_segment(a, w, k0, n); prefix_advance(a, w)) {
        const PrefixGroup& G = a.groups[w.j];
        const int rows = min(kPfxRowsF32, G.rows - w.t * kPfxRowsF32);
        for (int i = tid; i < 32 * D / 4; i += 256) {
            const int row = i / (D / 4), d = i % (D / 4) * 4, r = w.t * kPfxRowsF32 + row;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows) {
                x = *reinterpret_cast<const float4*>(
                    a.r.q + ((size_t)(G.lo + (r >> lg)) * a.r.H_q + ((size_t)w.g << lg) + (r & (a.r.G - 1))) * D + d);
                x.x *= a.r.xscale; x.y *= a.r.xscale; x.z *= a.r.xscale; x.w *= a.r.xscale;
            }
            *reinterpret_cast<float4*>(qs + row * KROW + d) = x;
        }
        float m[8], l[8], acc[8][W];                   // m: the same in all lanes; l: of this lane's tokens
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.f;
#pragma unroll
            for (int e = 0; e < W; ++e) acc[j][e] = 0.f;
        }
        bar_f32();
        for (int i = 0; i < n; ++i, ++it) {
            const int slot = it & 1;
            if (!pfx_wait(&k_full[slot], (it >> 1) & 1, &dead, status)) continue;
            if (r8 >= rows) {
                if (lane == 0) mbar_arrive(&k_empty[slot]);
                if (pfx_wait(&v_full[slot], (it >> 1) & 1, &dead, status) && lane == 0) mbar_arrive(&v_empty[slot]);
                continue;
            }
            uint64_t s[8] = {};
            const float* kr = ks + slot * L::K + (half * 32 + lane) * KROW;
            const float* qr = qs + r8 * KROW;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(kr + d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qr + j * KROW + d);
                    s[j] = fma2(q.x, k.x, s[j]);
                    s[j] = fma2(q.y, k.y, s[j]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_empty[slot]);
            const bool valid = half * 32 + lane < (long long)G.pages * PS - (long long)(k0 + i) * 64;
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 t = unpair(s[j]);
                p[j] = valid ? t.x + t.y : -INFINITY;
                const float mn = fmaxf(m[j], ordered_float(__reduce_max_sync(0xffffffffu, ordered_int(p[j]))));
                if (mn != m[j]) {                      // all lanes alike
                    const float f = m[j] == -INFINITY ? 0.f : exp2f(m[j] - mn);
                    m[j] = mn;
                    l[j] *= f;
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[j][e] *= f;
                }
                p[j] = exp2f(p[j] - (mn == -INFINITY ? 0.f : mn));
                l[j] += p[j];
            }
            reinterpret_cast<float4*>(pw + lane * PROW)[0] = make_float4(p[0], p[1], p[2], p[3]);
            reinterpret_cast<float4*>(pw + lane * PROW)[1] = make_float4(p[4], p[5], p[6], p[7]);
            __syncwarp();
            if (!pfx_wait(&v_full[slot], (it >> 1) & 1, &dead, status)) continue;
            const float* vr = vs + slot * L::V + half * 32 * D + lane * W;
#pragma unroll 4
            for (int t = 0; t < 32; ++t) {
                const float4 p0 = *reinterpret_cast<const float4*>(pw + t * PROW);
                const float4 p1 = *reinterpret_cast<const float4*>(pw + t * PROW + 4);
                const float pt[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
                float v[W];
                if constexpr (W == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(vr + t * D);
                else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(vr + t * D);
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float2 o = unpair(
                            fma2(pair(pt[j], pt[j]), pair(v[e], v[e + 1]), pair(acc[j][e], acc[j][e + 1])));
                        acc[j][e] = o.x;
                        acc[j][e + 1] = o.y;
                    }
            }
            __syncwarp();                              // also: the weights have been read
            if (lane == 0) mbar_arrive(&v_empty[slot]);
        }
        // join the token halves
#pragma unroll
        for (int j = 0; j < 8; ++j) l[j] = warp_sum(l[j]);
        bar_f32();                                     // Q is not read any more
        if (half == 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (lane == 0) ml[r8 + j] = make_float2(m[j], l[j]);
#pragma unroll
                for (int e = 0; e < W; ++e) qs[(r8 + j) * KROW + lane * W + e] = acc[j][e];
            }
        bar_f32();
        const long long part_row = prefix_part_row(a, G, w.g, w.t, blockIdx.x);
        if (half == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r8 + j < rows) {
                    const float2 x = ml[r8 + j];
                    const float M = fmaxf(m[j], x.x);
                    const float f0 = m[j] == -INFINITY ? 0.f : exp2f(m[j] - M);
                    const float f1 = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int d = lane * W + e;
                        a.part_o[part_row * D + ((long long)(d / 4) * rows + r8 + j) * 4 + d % 4] =
                            acc[j][e] * f0 + qs[(r8 + j) * KROW + d] * f1;
                    }
                    if (lane == 0)
                        reinterpret_cast<float2*>(a.part_ml)[part_row + r8 + j] = make_float2(M, l[j] * f0 + x.y * f1);
                }
        bar_f32();                                     // Q may come again
    }
}

// ---------------------------------------------------------------- merge
// One CTA a (sequence, kv head): the prefix partials in CTA order, then its own.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) prefix_merge_kernel(const PrefixArgs a)
{
    pdl_enter();
    const RangeArgs& r = a.r;
    const int u = blockIdx.x, b = u / r.H_kv, g = u % r.H_kv;
    const int h = threadIdx.x % r.G, d4 = threadIdx.x / r.G % (D / 4);   // a tile's partials lie [D / 4][rows] float4
    const int2 own = r.span[u];
    const PrefixHead head = *a.head;
    const SeqSpan sp = seq_span(r, b, a.ps, false);
    const int j = a.gid[b];
    PartList list[2] = {};
    if (sp.L > 0 && j >= 0 && a.groups[j].pages > 0) {
        const PrefixGroup G = a.groups[j];
        const int row = (b - G.lo) * r.G, t = row / a.row_tile;
        const int2 s = prefix_span(G, g, t, head.total, head.C);
        const long long base = prefix_part_row(a, G, g, t, s.x);
        const int rows = min(a.row_tile, G.rows - t * a.row_tile), at = row % a.row_tile + h;
        list[0] = PartList{reinterpret_cast<const float4*>(a.part_o + base * D) + d4 * rows + at,
                           reinterpret_cast<const float2*>(a.part_ml) + base + at, a.row_tile, s.y - s.x + 1};
    }
    if (sp.pages() > 0) {
        const long long row = ((long long)own.x + u) * r.G + h;
        list[1] = PartList{reinterpret_cast<const float4*>(r.part_o + row * D) + d4,
                           reinterpret_cast<const float2*>(r.part_ml) + row, r.G, own.y - own.x + 1};
    }
    float4 o;
    float m, l;
    if (!merge_parts<D, THREADS>(list[0], list[1], r.G, o, m, l)) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t row = (size_t)b * r.H_q + (size_t)g * r.G + h;
    float* dst = r.out + row * D + d4 * 4;
    dst[0] = o.x * inv;
    dst[1] = o.y * inv;
    dst[2] = o.z * inv;
    dst[3] = o.w * inv;
    if (d4 == 0 && r.lse) r.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- launch
template <int D, int PS>
static int launch_prefix_bf16(const PrefixArgs& a, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              cudaStream_t stream)
{
    const int smem = pfx_slots<D>() * kPfxTok * D * 2 + 1024;
    if (ensure_smem((const void*)prefix_bf16_kernel<D, PS>, smem)) return ENTMAXKV_CUDA_ERROR;
    return launch_pdl(prefix_bf16_kernel<D, PS>, dim3(a.C), dim3(kPfxThreads), smem, stream, *kmap, *vmap, a) ==
                   cudaSuccess
               ? ENTMAXKV_OK
               : ENTMAXKV_CUDA_ERROR;
}

template <int D, int PS>
static int launch_prefix_f32(const entmaxkv_pool& pool, const PrefixArgs& a, cudaStream_t stream)
{
    const int smem = PfxF32<D>::FLOATS * 4;
    if (ensure_smem((const void*)prefix_f32_kernel<D, PS>, smem)) return ENTMAXKV_CUDA_ERROR;
    return launch_pdl(prefix_f32_kernel<D, PS>, dim3(a.C), dim3(kPfxThreadsF32), smem, stream,
                      (const float*)pool.k_pool, (const float*)pool.v_pool, a) == cudaSuccess
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
    } else if (pool.d == 128) {
        rc = pool.ps == 64 ? launch_prefix_f32<128, 64>(pool, a, stream) : launch_prefix_f32<128, 16>(pool, a, stream);
    } else {
        rc = pool.ps == 64 ? launch_prefix_f32<64, 64>(pool, a, stream) : launch_prefix_f32<64, 16>(pool, a, stream);
    }
    if (rc) return rc;
    if ((rc = launch_range(pool, a.r, range_C, kmap, vmap, stream))) return rc;
    const int n = a.r.B * a.r.H_kv;
    const auto merge = merge_threads(n) == 1024
                           ? (pool.d == 128 ? prefix_merge_kernel<128, 1024> : prefix_merge_kernel<64, 1024>)
                           : (pool.d == 128 ? prefix_merge_kernel<128, 256> : prefix_merge_kernel<64, 256>);
    const cudaError_t e = launch_pdl(merge, dim3(n), dim3(merge_threads(n)), 0, stream, a);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

}  // namespace ekv
