// Softmax decode over a sliding window with sinks, and over the tokens that a
// sequence holds behind a shared prefix.
//
//   o = sum_i softmax(x)_i v_i,  x_i = scale q.k_i,  lse = log sum_i exp(x_i)
//
// over the tokens i < sinks and i >= L - window of a sequence of L tokens (the
// newest included).  One pass over the keys and values with a running maximum
// m and sum l: with m' = max(m, max x), l' = l 2^(m-m') + sum 2^(x-m') and the
// same factor on o (base 2: log2(e) rides in the query's scale).
//
// A decode token uses each key and value once for a group of G <= 8 query
// heads, so the bytes of the range bound the time; the tensor cores only have
// to keep up (mma.sync on 16-token slices, one warp each), and the work is to
// keep the loads in flight on every SM: see range.cuh for the equal shares.
#include "common.cuh"
#include "kernels.cuh"
#include "range.cuh"

namespace ekv {

constexpr int kRangeStages = 3;
constexpr int kRangeThreads = 160;       // four consumer warps and a producer warp
constexpr int kRedPad = 8;               // padding (floats) of a row of the joining buffer

// D = A.trans on 8x8 16-bit matrices held one row per four lanes
EKV_DEV uint32_t movmatrix_trans(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// (hi, lo) bf16 halves of f, hi in the low 16 bits; hi + lo is f to 2^-17 of f
EKV_DEV uint32_t split_pack(float f)
{
    uint32_t h, r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(0.f), "f"(f));
    const float rest = f - bf16_bits_to_f32(h & 0xFFFFu);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(rest), "f"(f));
    return r;
}

// what hi + lo of split_pack leave of f, as bf16; f is the sum of the three to 2^-26
EKV_DEV uint32_t split_rest(float f, uint32_t hilo)
{
    uint32_t r;
    const float rest = f - bf16_bits_to_f32(hilo & 0xFFFFu) - __uint_as_float(hilo & 0xFFFF0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(rest));
    return r;
}

EKV_DEV void bar_consumers() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Writes one row's joined result: a finished row, or a partial.
EKV_DEV void range_store(const RangeArgs& a, bool whole, long long slot, int b, int g, int h, int D, int d, float4 o,
                         float m, float l)
{
    float* dst;
    if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        const size_t row = (size_t)b * a.H_q + (size_t)g * a.G + h;
        dst = a.out + row * D + d;
        if (d == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
        const size_t row = (size_t)slot * a.G + h;
        dst = a.part_o + row * D + d;
        if (d == 0) {
            a.part_ml[row * 2] = m;
            a.part_ml[row * 2 + 1] = l;
        }
    }
    dst[0] = o.x; dst[1] = o.y; dst[2] = o.z; dst[3] = o.w;
}

// A CTA's part of its cluster's unit.
template <int D>
struct ClusterPart {
    float o[8][D], m[8], l[8];           // heads of the group
};

// Joins the cluster's parts in rank order and writes the unit's rows; a CTA
// takes every n-th group of four dims.  All threads of all CTAs call.
template <int D>
EKV_DEV void range_cluster_join(const RangeArgs& a, ClusterPart<D>& part, int b, int g, int r, int n)
{
    cluster_sync();
    for (int i = r + n * (int)threadIdx.x; i < a.G * D / 4; i += n * (int)blockDim.x) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float M = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < n; c0 += 8) {
            uint4 t[8];
            float m[8], s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c0 + k < n) {
                    t[k] = ld_dsmem_v4(dsmem(&part.o[h][d], c0 + k));
                    m[k] = ld_dsmem_f32(dsmem(&part.m[h], c0 + k));
                    s[k] = ld_dsmem_f32(dsmem(&part.l[h], c0 + k));
                }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c0 + k < n && s[k] != 0.f) {
                    const float mn = fmaxf(M, m[k]);
                    const float f = exp2f(M - mn), e = exp2f(m[k] - mn);
                    M = mn;
                    l = l * f + s[k] * e;
                    o.x = o.x * f + __uint_as_float(t[k].x) * e;
                    o.y = o.y * f + __uint_as_float(t[k].y) * e;
                    o.z = o.z * f + __uint_as_float(t[k].z) * e;
                    o.w = o.w * f + __uint_as_float(t[k].w) * e;
                }
        }
        range_store(a, true, 0, b, g, h, D, d, o, M, l);
    }
    cluster_sync();                      // nobody leaves while its part may still be read
}

// The CTA that holds a unit's first tile leaves the unit's first and last CTA
// for the merge.
EKV_DEV void range_note_span(const RangeArgs& a, const RangeWalk& w, int u, int nt, int done, int c)
{
    if (w.t != 0) return;
    const long long at = mul_div(w.total, c, w.C) + done;     // this unit's first tile among all tiles
    a.span[u] = make_int2(c, range_cta_of(at + nt - 1, w.total, w.C));
}

// ---------------------------------------------------------------- bf16 cache
// Per CTA: a producer warp walks the share's pages and keeps a ring of
// kRangeStages tiles (K and V, 64 tokens, 128-byte swizzle) full by TMA; four
// consumer warps each own 16 tokens of every tile from scores to P.V, so no
// block barrier stands between a tile's arrival and its release.  The query is
// the B operand of the score product, its result's layout is turned in registers
// (movmatrix) into the B operand of V^T P.  Both enter in bf16 parts: one would
// leave 2^-8 of relative error, two 2^-17, three 2^-26.  The first two are columns
// 2h and 2h + 1 of one product, the third is column 2h of a second into the same
// accumulators.  A window takes three (REST): that doubles the products, which
// the bytes hide but for 1.5% (64 sequences of 8192 + 64 tokens: 293.7 -> 298.1
// us), and brings the error of 1028 tokens from 3.2e-6 to 3.6e-7 (2-norms).  The
// tokens behind a shared prefix take two parts, as the prefix itself does (3.5e-6):
// three would cost 4 x 8 sequences behind 16384 tokens 4% (102.3 -> 106.5 us), at 8
// heads a group 11%, for sums of which the prefix makes most.
// The tensor cores cut their sums off and do not round them, always to the same
// side: left in their accumulators, a sum loses 8e-8 of itself a tile (8e-5 at
// 65536 tokens of values around 1).  So the products of a warp's 16 tokens start
// from zero and are added to the output by rounded adds (2.5e-7 there, as plain
// fp32 sums have).  Two slices of 16 dims at a time, so that no product waits for
// the one before: 64 windows of 8256 tokens 302 us at 4 heads a group; at 8 331 us
// under the power cap (one slice at a time 367), 309 at full clock.
template <int D, int PS, int NT, bool CLUSTER, bool REST>
__global__ void __launch_bounds__(kRangeThreads, 2) range_bf16_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                      const __grid_constant__ CUtensorMap vmap,
                                                                      const RangeArgs a, int cluster)
{
    pdl_enter();
    constexpr int STAGE = kRangeTile * D * 2;          // bytes of one tensor's tile
    constexpr int PPS = kRangeTile / PS;
    constexpr int KS = D / 16, MT = D / 16;
    constexpr int RED = D + kRedPad;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    float* red = reinterpret_cast<float*>(smem + 2 * kRangeStages * STAGE);   // [4 warps][4 heads][RED]
    // the query's third parts, the same for all warps, until the unit's results take their place
    uint2* q_rest = reinterpret_cast<uint2*>(red);
    static_assert(NT * KS * 32 * sizeof(uint2) <= 16 * RED * sizeof(float));
    __shared__ uint64_t full[kRangeStages], empty[kRangeStages];
    __shared__ int page_ok[kRangeStages];
    __shared__ float wm[2][4][4], wl[2][4][4];
    __shared__ volatile int dead;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c_id = blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kRangeStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        fence_mbar_init();
        dead = 0;
    }
    const int rank = CLUSTER ? c_id % cluster : 0;
    __shared__ __align__(16) uint8_t part_raw[CLUSTER ? sizeof(ClusterPart<D>) : 16];
    ClusterPart<D>& part = *reinterpret_cast<ClusterPart<D>*>(part_raw);
    RangeWalk w;
    if (CLUSTER) {
        w = range_cluster_start(a, PS, c_id / cluster, rank, cluster);
        if (w.left <= 0 && tid < 8) {
            part.m[tid] = -INFINITY;
            part.l[tid] = 0.f;
        }
    } else {
        w = range_start(a, PS, c_id, gridDim.x);       // holds block barriers
        if (w.left <= 0) return;
    }
    const int b0 = w.b, g0 = w.g;                      // a cluster's unit
    __syncthreads();

    int b = w.b;
    SeqSpan sp = seq_span(a, b, PS, false);
    int nt = sp.tiles(PS);
    // next unit with tiles (the share ends before the sequences do)
    auto advance = [&](int n) {
        w.t += n;
        w.left -= n;
        if (w.left <= 0 || w.t < nt) return;
        w.t = 0;
        if (++w.g < a.H_kv) return;
        w.g = 0;
        do {
            ++b;
            sp = seq_span(a, b, PS, false);
            nt = sp.tiles(PS);
        } while (nt == 0);
    };

    if (warp == 4) {
        // ---------------------------------------------------- producer
        if (lane == 0) {
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
        }
        long long issued = 0;
        bool stop = false;
        while (w.left > 0 && !stop) {
            const int n = (int)min((long long)(nt - w.t), w.left);
            const int i1 = min((w.t + n) * PPS, sp.pages());
            for (int base = w.t * PPS; base < (w.t + n) * PPS && !stop; base += 32) {
                // 32 listed pages at a time, one a lane
                int ph = -1;
                if (base + lane < i1) {
                    ph = a.page_table[(size_t)b * a.max_pages + sp.logical(base + lane)];
                    if (ph < 0 || ph >= a.num_phys) {
                        report(a.status, ENTMAXKV_DEVICE_BOUNDS);
                        ph = -1;
                    }
                }
                const uint32_t good = __ballot_sync(0xffffffffu, ph >= 0);
                const int tiles = min(32 / PPS, w.t + n - base / PPS);
                for (int k = 0; k < tiles; ++k, ++issued) {
                    const int slot = (int)(issued % kRangeStages);
                    const int mask = (good >> (k * PPS)) & ((1 << PPS) - 1);
                    bool ok = true;
                    if (issued >= kRangeStages && !dead)
                        ok = mbar_wait(&empty[slot], (uint32_t)((issued / kRangeStages - 1) & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok) || dead) {
                        dead = 1;
                        report(a.status, ENTMAXKV_TIMEOUT);
                        stop = true;
                        break;
                    }
                    if (lane == 0) {
                        page_ok[slot] = mask;
                        mbar_arrive_expect_tx(&full[slot], __popc(mask) * 2 * PS * D * 2);
                    }
                    __syncwarp();
                    // one lane a box: page, column half, tensor
                    constexpr int BOXES = PPS * (D / 64) * 2;
                    const int pg = lane / ((D / 64) * 2), half = (lane >> 1) % (D / 64), isv = lane & 1;
                    const int phys = __shfl_sync(0xffffffffu, ph, (k * PPS + pg) & 31);
                    if (lane < BOXES && phys >= 0)
                        tma_load_2d(smem + (2 * slot + isv) * STAGE + half * (kRangeTile * 128) + pg * PS * 128,
                                    isv ? &vmap : &kmap, &full[slot], half * 64, (phys * a.H_kv + w.g) * PS);
                }
            }
            advance(n);
        }
        // nothing of this CTA's is in flight once the last tiles have landed (consumers that gave up do not
        // wait for them)
        if (lane == 0)
            for (long long i = max(0ll, issued - kRangeStages); i < issued; ++i)
                mbar_wait(&full[i % kRangeStages], (uint32_t)((i / kRangeStages) & 1), kWaitLimitNs);
        w.left = 0;
        if (!CLUSTER) return;
    }

    // -------------------------------------------------------- consumers
    const int gi = lane >> 2, c = lane & 3;
    const uint32_t sbase = smem_addr(smem);
    const int row0 = warp * 16;
    long long tile = 0;
    int done = 0;                                      // tiles before the current unit in this share
    int flip = 0;
    while (w.left > 0) {
        const int n = (int)min((long long)(nt - w.t), w.left);
        const int u = b * a.H_kv + w.g;
        const bool whole = a.direct && n == nt;
        if (!CLUSTER && tid == 0) range_note_span(a, w, u, nt, done, c_id);

        uint32_t bq[NT][KS][2];
        if (REST) bar_consumers();                     // the last unit's reads of red are done
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int head = 4 * x + (gi >> 1);
            const float* qh = a.q + ((size_t)b * a.H_q + (size_t)w.g * a.G + head) * D;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t third[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 16 * j + 2 * c + 8 * e;
                    const float v0 = head < a.G ? qh[k] * a.xscale : 0.f;
                    const float v1 = head < a.G ? qh[k + 1] * a.xscale : 0.f;
                    const uint32_t p0 = split_pack(v0), p1 = split_pack(v1);
                    bq[x][j][e] = (gi & 1) ? __byte_perm(p0, p1, 0x7632) : __byte_perm(p0, p1, 0x5410);
                    if (REST) third[e] = (gi & 1) ? 0u : __byte_perm(split_rest(v0, p0), split_rest(v1, p1), 0x5410);
                }
                if (REST && j % 4 == warp) q_rest[(x * KS + j) * 32 + lane] = make_uint2(third[0], third[1]);
            }
        }
        if (REST) bar_consumers();
        float acc[NT][MT][2], mrun[NT], lrun[NT];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            mrun[x] = -INFINITY;
            lrun[x] = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[x][m][0] = acc[x][m][1] = 0.f;
        }
        for (int k = 0; k < n; ++k, ++tile) {
            const int slot = (int)(tile % kRangeStages);
            const bool ok = !dead && mbar_wait(&full[slot], (uint32_t)((tile / kRangeStages) & 1), kWaitLimitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (!dead) report(a.status, ENTMAXKV_TIMEOUT);
                dead = 1;
                continue;
            }
            // this warp's tokens row0 .. row0 + 15 lie in one page
            const int idx = (w.t + k) * PPS + row0 / PS;
            const bool page = (page_ok[slot] >> (row0 / PS)) & 1;
            const int pos0 = sp.logical(idx) * PS + row0 % PS;
            const bool v_lo = page && sp.valid(pos0 + gi), v_hi = page && sp.valid(pos0 + gi + 8);
            const uint32_t some = __ballot_sync(0xffffffffu, v_lo || v_hi);
            if (some) {
                const uint32_t kbase = sbase + (2 * slot) * STAGE, vbase = kbase + STAGE;
                const bool masked = !__all_sync(0xffffffffu, v_lo && v_hi);
                float sc[NT][4];
#pragma unroll
                for (int x = 0; x < NT; ++x) sc[x][0] = sc[x][1] = sc[x][2] = sc[x][3] = 0.f;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    uint32_t af[4];
                    ldsm_x4(swz_addr(kbase, row0 + (lane & 15), 2 * j + (lane >> 4)), af);
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        mma_bf16(sc[x], af, bq[x][j][0], bq[x][j][1]);
                        if (REST) {
                            const uint2 t = q_rest[(x * KS + j) * 32 + lane];
                            mma_bf16(sc[x], af, t.x, t.y);
                        }
                    }
                }
                if (masked) {
                    // a weight of zero must not meet a masked row's value: clear those rows of V
                    const int r = lane & 15;
                    const bool v = page && sp.valid(pos0 + r);
                    if (!v) {
                        for (int h = 0; h < D / 64; ++h)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t ad = vbase + h * (kRangeTile * 128) + (row0 + r) * 128 +
                                                    ((lane >> 4) * 4 + q) * 16;
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ad), "r"(0) : "memory");
                            }
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
                uint32_t pb[NT][2], pr[NT][2];
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    const float s0 = v_lo ? sc[x][0] + sc[x][1] : -INFINITY;
                    const float s1 = v_hi ? sc[x][2] + sc[x][3] : -INFINITY;
                    float mx = fmaxf(s0, s1);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mnew = fmaxf(mrun[x], mx);
                    const float mu = mnew == -INFINITY ? 0.f : mnew;
                    if (__any_sync(0xffffffffu, mnew > mrun[x])) {
                        const float corr = exp2f(mrun[x] - mu);
                        lrun[x] *= corr;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            acc[x][m][0] *= corr;
                            acc[x][m][1] *= corr;
                        }
                        mrun[x] = mnew;
                    }
                    const float p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
                    lrun[x] += p0 + p1;
                    const uint32_t h0 = split_pack(p0), h1 = split_pack(p1);
                    pb[x][0] = movmatrix_trans(h0);
                    pb[x][1] = movmatrix_trans(h1);
                    if (REST) {
                        pr[x][0] = movmatrix_trans(split_rest(p0, h0));
                        pr[x][1] = movmatrix_trans(split_rest(p1, h1));
                    }
                }
                const int trow = row0 + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                for (int m0 = 0; m0 < MT; m0 += 2) {
                    uint32_t af[2][4];
                    float t[2][NT][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        ldsm_x4_t(swz_addr(vbase, trow, 2 * (m0 + y) + ((lane >> 3) & 1)), af[y]);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int x = 0; x < NT; ++x) mma_bf16_new(t[y][x], af[y], pb[x][0], pb[x][1]);
                    if (REST)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int x = 0; x < NT; ++x) mma_bf16(t[y][x], af[y], pr[x][0], pr[x][1]);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            acc[x][m0 + y][0] += t[y][x][0] + t[y][x][1];
                            acc[x][m0 + y][1] += t[y][x][2] + t[y][x][3];
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }
        // join the four warps' states, four heads at a time
#pragma unroll
        for (int x = 0; x < NT; ++x, flip ^= 1) {
            float l = lrun[x];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (gi == 0) {
                wm[flip][warp][c] = mrun[x];
                wl[flip][warp][c] = l;
            }
            bar_consumers();                           // also: the last round's reads of red are done
            float M = fmaxf(fmaxf(wm[flip][0][c], wm[flip][1][c]), fmaxf(wm[flip][2][c], wm[flip][3][c]));
            const float f = mrun[x] == -INFINITY ? 0.f : exp2f(mrun[x] - M);
            float* rw = red + (warp * 4 + c) * RED;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                rw[16 * m + gi] = acc[x][m][0] * f;
                rw[16 * m + gi + 8] = acc[x][m][1] * f;
            }
            bar_consumers();
            const int h = tid / (D / 4), d = tid % (D / 4) * 4;
            if (h < 4 && 4 * x + h < a.G) {
                float Mh = -INFINITY, L = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) Mh = fmaxf(Mh, wm[flip][i][h]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float mi = wm[flip][i][h];
                    L += wl[flip][i][h] * (mi == -INFINITY ? 0.f : exp2f(mi - Mh));   // (a sum that is NaN stays)
                    const float4 t = *reinterpret_cast<const float4*>(red + (i * 4 + h) * RED + d);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                if (!CLUSTER) {
                    range_store(a, whole, (long long)c_id + u, b, w.g, 4 * x + h, D, d, o, Mh, L);
                } else {
                    *reinterpret_cast<float4*>(&part.o[4 * x + h][d]) = o;
                    if (d == 0) {
                        part.m[4 * x + h] = Mh;
                        part.l[4 * x + h] = L;
                    }
                }
            }
        }
        done += n;
        advance(n);
    }
    if (CLUSTER) range_cluster_join<D>(a, part, b0, g0, rank, cluster);
}

// ---------------------------------------------------------------- fp32 cache
// Each warp owns 16 tokens of a tile, which lie in one page: LPT lanes share a
// token (each holds D / LPT coordinates of the query heads and of the output),
// 32 / LPT tokens advance together, and each lane group runs its own softmax
// state, joined once at the end of a unit.  All arithmetic is fp32.  A lane
// copies what it will read of the keys and values a number of steps ahead to
// shared memory (asynchronously; nobody else reads it, so no barrier is needed),
// and looks a page up a tile before that: with one step ahead in registers every
// step waited for DRAM (about 1 us).  Masked tokens are not read.  Measured: 24
// sequences of up to 2016 tokens of 64 dims 13.8 us a call; 8 of 8256 tokens, 8 kv
// heads of 128 dims 108 us, 5.0 TB/s.
template <int D, int GT>
struct RangeF32 {
    static constexpr int LPT = GT == 8 ? 16 : 8, TPW = 32 / LPT, E = D / LPT, E4 = E / 4, STEPS = 16 / TPW;
    static constexpr int AHEAD = E4 == 4 ? 6 : 8;      // steps under way: 32 to 96 KB a CTA
    static constexpr int SMEM = AHEAD * 2 * E4 * 128 * 16;
};

template <int D, int GT, bool CLUSTER>
__global__ void __launch_bounds__(128, 2) range_f32_kernel(const float* __restrict__ k_pool,
                                                           const float* __restrict__ v_pool, int ps, const RangeArgs a,
                                                           int cluster)
{
    pdl_enter();
    using P = RangeF32<D, GT>;
    constexpr int LPT = P::LPT, TPW = P::TPW, E = P::E, E4 = P::E4, STEPS = P::STEPS, AHEAD = P::AHEAD;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t mine = smem_addr(smem_raw) + threadIdx.x * 16;   // this lane's words, 2 KB apart
    __shared__ float red[4][4][D + kRedPad];
    __shared__ float wm[2][4][4], wl[2][4][4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = lane / LPT, sub = lane % LPT;
    const int c_id = blockIdx.x;
    const int rank = CLUSTER ? c_id % cluster : 0;
    __shared__ __align__(16) uint8_t part_raw[CLUSTER ? sizeof(ClusterPart<D>) : 16];
    ClusterPart<D>& part = *reinterpret_cast<ClusterPart<D>*>(part_raw);
    RangeWalk w;
    if (CLUSTER) {
        w = range_cluster_start(a, ps, c_id / cluster, rank, cluster);
        if (w.left <= 0 && tid < 8) {
            part.m[tid] = -INFINITY;
            part.l[tid] = 0.f;
        }
    } else {
        w = range_start(a, ps, c_id, gridDim.x);
        if (w.left <= 0) return;
    }
    const int b0 = w.b, g0 = w.g;                      // a cluster's unit
    int b = w.b, done = 0, flip = 0;
    while (w.left > 0) {
        const SeqSpan sp = seq_span(a, b, ps, false);
        const int nt = sp.tiles(ps);
        if (nt == 0) {
            ++b;
            continue;
        }
        const int n = (int)min((long long)(nt - w.t), w.left);
        const int u = b * a.H_kv + w.g;
        const bool whole = a.direct && n == nt;
        if (!CLUSTER && tid == 0) range_note_span(a, w, u, nt, done, c_id);
        float q[GT][E], acc[GT][E], mrun[GT], lrun[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
            mrun[h] = -INFINITY;
            lrun[h] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = (e / 4 * LPT + sub) * 4 + e % 4;
                q[h][e] = h < a.G ? a.q[((size_t)b * a.H_q + (size_t)w.g * a.G + h) * D + d] * a.xscale : 0.f;
                acc[h][e] = 0.f;
            }
        }
        const int last = n * STEPS;
        // the page of this warp's tokens in the share's tile i (-1 behind the last), and their first position
        const auto lookup = [&](int i, int& pos) {
            const long long li = div_ps((long long)(w.t + i) * kRangeTile + warp * 16, ps);
            if (i >= n || li >= sp.pages()) return -1;
            const int lp = sp.logical((int)li);
            pos = lp * ps + ((warp * 16) & (ps - 1));
            return a.page_table[(size_t)b * a.max_pages + lp];
        };
        int pos = 0, pos_next = 0, phys, phys_next = lookup(0, pos_next);
        uint32_t live = 0;                             // one bit a slot: this lane's token is there
        int put = 0;
        const auto fetch = [&](int it) {
            if (it % STEPS == 0) {
                phys = phys_next;
                pos = pos_next;
                phys_next = lookup(it / STEPS + 1, pos_next);
                const bool walked =
                    it < last && div_ps((long long)(w.t + it / STEPS) * kRangeTile + warp * 16, ps) < sp.pages();
                if (walked && (phys < 0 || phys >= a.num_phys)) {
                    report(a.status, ENTMAXKV_DEVICE_BOUNDS);
                    phys = -1;
                }
            }
            const int tok = it % STEPS * TPW + grp;
            const bool valid = it < last && phys >= 0 && sp.valid(pos + tok);
            live = valid ? live | (1u << put) : live & ~(1u << put);
            if (valid) {
                const size_t row = (((size_t)phys * a.H_kv + w.g) * ps + ((warp * 16) & (ps - 1)) + tok) * D;
#pragma unroll
                for (int i = 0; i < E4; ++i) {
                    const size_t o = row + (i * LPT + sub) * 4;
                    cp_async16(mine + (put * 2 * E4 + i) * 2048, k_pool + o);
                    cp_async16(mine + (put * 2 * E4 + E4 + i) * 2048, v_pool + o);
                }
            }
            cp_async_commit();
            put = put + 1 == AHEAD ? 0 : put + 1;
        };
        for (int it = 0; it < AHEAD - 1; ++it) fetch(it);
        for (int it = 0, get = 0; it < last; ++it, get = get + 1 == AHEAD ? 0 : get + 1) {
            fetch(it + AHEAD - 1);
            cp_async_wait<AHEAD - 1>();
            const bool valid = (live >> get) & 1;
            float4 k4[E4], v4[E4];
#pragma unroll
            for (int i = 0; i < E4; ++i) {
                k4[i] = valid ? lds128f(mine + (get * 2 * E4 + i) * 2048) : make_float4(0.f, 0.f, 0.f, 0.f);
                v4[i] = valid ? lds128f(mine + (get * 2 * E4 + E4 + i) * 2048) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const float* k = reinterpret_cast<const float*>(k4);
            const float* v = reinterpret_cast<const float*>(v4);
            // the heads side by side: one branch for all, so that their chains overlap
            float x[GT];
            bool grow = false;
#pragma unroll
            for (int h = 0; h < GT; ++h) {
                x[h] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) x[h] = fmaf(q[h][e], k[e], x[h]);
            }
#pragma unroll
            for (int o = LPT / 2; o > 0; o >>= 1)
#pragma unroll
                for (int h = 0; h < GT; ++h) x[h] += __shfl_xor_sync(0xffffffffu, x[h], o);
#pragma unroll
            for (int h = 0; h < GT; ++h) {
                if (!valid) x[h] = -INFINITY;
                grow |= x[h] > mrun[h];
            }
            if (grow) {
#pragma unroll
                for (int h = 0; h < GT; ++h) {
                    const float mnew = fmaxf(mrun[h], x[h]);
                    const float corr = mrun[h] == mnew ? 1.f : exp2f(mrun[h] - mnew);
                    mrun[h] = mnew;
                    lrun[h] *= corr;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[h][e] *= corr;
                }
            }
#pragma unroll
            for (int h = 0; h < GT; ++h) {
                const float p = exp2f(x[h] - (mrun[h] == -INFINITY ? 0.f : mrun[h]));
                lrun[h] += p;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[h][e] = fmaf(p, v[e], acc[h][e]);
            }
        }
        // join the lane groups of each warp, then the warps, four heads at a time
        for (int x = 0; x < GT / 4; ++x, flip ^= 1) {
#pragma unroll
            for (int hh = 0; hh < GT; ++hh) {
                if (hh / 4 != x) continue;
                float M = mrun[hh];
#pragma unroll
                for (int o = LPT; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                const float f = mrun[hh] == -INFINITY ? 0.f : exp2f(mrun[hh] - M);
                float l = lrun[hh] * f;
#pragma unroll
                for (int o = LPT; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float y = acc[hh][e] * f;
#pragma unroll
                    for (int o = LPT; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                    acc[hh][e] = y;
                }
                mrun[hh] = M;
                if (lane == 0) {
                    wm[flip][warp][hh % 4] = M;
                    wl[flip][warp][hh % 4] = l;
                }
            }
            __syncthreads();
#pragma unroll
            for (int hh = 0; hh < GT; ++hh) {
                if (hh / 4 != x || grp != 0) continue;
                const int i4 = hh % 4;
                const float M = fmaxf(fmaxf(wm[flip][0][i4], wm[flip][1][i4]), fmaxf(wm[flip][2][i4], wm[flip][3][i4]));
                const float f = mrun[hh] == -INFINITY ? 0.f : exp2f(mrun[hh] - M);
#pragma unroll
                for (int e = 0; e < E; ++e) red[warp][i4][(e / 4 * LPT + sub) * 4 + e % 4] = acc[hh][e] * f;
            }
            __syncthreads();
            const int h = tid / (D / 4), d = tid % (D / 4) * 4;
            if (h < 4 && 4 * x + h < a.G) {
                float Mh = -INFINITY, L = 0.f;
                for (int i = 0; i < 4; ++i) Mh = fmaxf(Mh, wm[flip][i][h]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = 0; i < 4; ++i) {
                    const float mi = wm[flip][i][h];
                    L += wl[flip][i][h] * (mi == -INFINITY ? 0.f : exp2f(mi - Mh));   // (a sum that is NaN stays)
                    const float4 t = *reinterpret_cast<const float4*>(&red[i][h][d]);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                if (!CLUSTER) {
                    range_store(a, whole, (long long)c_id + u, b, w.g, 4 * x + h, D, d, o, Mh, L);
                } else {
                    *reinterpret_cast<float4*>(&part.o[4 * x + h][d]) = o;
                    if (d == 0) {
                        part.m[4 * x + h] = Mh;
                        part.l[4 * x + h] = L;
                    }
                }
            }
        }
        done += n;
        w.t += n;
        w.left -= n;
        if (w.t == nt) {
            w.t = 0;
            if (++w.g == a.H_kv) {
                w.g = 0;
                ++b;
            }
        }
    }
    if (CLUSTER) range_cluster_join<D>(a, part, b0, g0, rank, cluster);
}

// ---------------------------------------------------------------- merge
// One CTA a unit: rows of a unit that several CTAs share are joined; rows of a
// unit without tokens get o = 0 and lse = -infinity.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) range_merge_kernel(int ps, const RangeArgs a)
{
    pdl_enter();
    const int u = blockIdx.x, b = u / a.H_kv, g = u % a.H_kv;
    const int2 sp = a.span[u];
    const bool empty = seq_span(a, b, ps, false).pages() == 0;
    if (!empty && sp.x == sp.y) return;
    const int h = threadIdx.x / (D / 4) % a.G, d = threadIdx.x % (D / 4) * 4;
    const size_t row = ((size_t)sp.x + u) * a.G + h;
    const PartList list{reinterpret_cast<const float4*>(a.part_o + (empty ? 0 : row * D + d)),
                        reinterpret_cast<const float2*>(a.part_ml) + (empty ? 0 : row), a.G,
                        empty ? 0 : sp.y - sp.x + 1};
    float4 o;
    float m, l;
    if (merge_parts<D, THREADS>(list, PartList{}, a.G, o, m, l)) range_store(a, true, 0, b, g, h, D, d, o, m, l);
}

// ---------------------------------------------------------------- launch
// `cluster` 0: C CTAs with equal shares; else C CTAs in clusters, one a unit.
template <typename... KArgs, typename... Args>
static int launch_range_kernel(void (*kern)(KArgs...), int C, int threads, int cluster, int smem, cudaStream_t stream,
                               Args&&... args)
{
    if (smem && ensure_smem((const void*)kern, smem)) return ENTMAXKV_CUDA_ERROR;
    if (cluster > 8) {
        if (ensure_cluster_kernel((const void*)kern, smem)) return ENTMAXKV_CUDA_ERROR;
        if (max_active_clusters((const void*)kern, cluster, threads, smem) == 0) {   // no GPC holds so many
            C = C / cluster * 8;
            cluster = 8;
        }
    }
    const dim3 grid(C), block(threads);
    const cudaError_t e = cluster ? launch_pdl_cluster(kern, grid, block, cluster, smem, stream, args..., cluster)
                                  : launch_pdl(kern, grid, block, smem, stream, args..., cluster);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

template <int D, int PS, bool CLUSTER, bool REST>
static int launch_range_bf16(const RangeArgs& a, int C, int cluster, const CUtensorMap* kmap, const CUtensorMap* vmap,
                             cudaStream_t stream)
{
    const int smem = 2 * kRangeStages * kRangeTile * D * 2 + 16 * (D + kRedPad) * 4 + 1024;
    const auto kern =
        a.G == 8 ? range_bf16_kernel<D, PS, 2, CLUSTER, REST> : range_bf16_kernel<D, PS, 1, CLUSTER, REST>;
    return launch_range_kernel(kern, C, kRangeThreads, cluster, smem, stream, *kmap, *vmap, a);
}

template <int D, bool CLUSTER, bool REST>
static int launch_range_d(const entmaxkv_pool& pool, const RangeArgs& a, int C, int cluster, const CUtensorMap* kmap,
                          const CUtensorMap* vmap, cudaStream_t stream)
{
    if (pool.dtype == ENTMAXKV_F32) {
        const auto kern = a.G == 8 ? range_f32_kernel<D, 8, CLUSTER> : range_f32_kernel<D, 4, CLUSTER>;
        const int smem = a.G == 8 ? RangeF32<D, 8>::SMEM : RangeF32<D, 4>::SMEM;
        return launch_range_kernel(kern, C, 128, cluster, smem, stream, (const float*)pool.k_pool,
                                   (const float*)pool.v_pool, pool.ps, a);
    }
    return pool.ps == 64 ? launch_range_bf16<D, 64, CLUSTER, REST>(a, C, cluster, kmap, vmap, stream)
                         : launch_range_bf16<D, 16, CLUSTER, REST>(a, C, cluster, kmap, vmap, stream);
}

int launch_range(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                 const CUtensorMap* vmap, cudaStream_t stream)
{
    return pool.d == 128 ? launch_range_d<128, false, false>(pool, a, C, 0, kmap, vmap, stream)
                         : launch_range_d<64, false, false>(pool, a, C, 0, kmap, vmap, stream);
}

int launch_window_cluster(const entmaxkv_pool& pool, const RangeArgs& a, int cluster, const CUtensorMap* kmap,
                          const CUtensorMap* vmap, cudaStream_t stream)
{
    const int C = a.B * a.H_kv * cluster;
    return pool.d == 128 ? launch_range_d<128, true, true>(pool, a, C, cluster, kmap, vmap, stream)
                         : launch_range_d<64, true, true>(pool, a, C, cluster, kmap, vmap, stream);
}

int launch_window(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream)
{
    const int rc = pool.d == 128 ? launch_range_d<128, false, true>(pool, a, C, 0, kmap, vmap, stream)
                                 : launch_range_d<64, false, true>(pool, a, C, 0, kmap, vmap, stream);
    if (rc) return rc;
    const int n = a.B * a.H_kv;
    const auto merge = merge_threads(n) == 1024
                           ? (pool.d == 128 ? range_merge_kernel<128, 1024> : range_merge_kernel<64, 1024>)
                           : (pool.d == 128 ? range_merge_kernel<128, 256> : range_merge_kernel<64, 256>);
    const cudaError_t e = launch_pdl(merge, dim3(n), dim3(merge_threads(n)), 0, stream, pool.ps, a);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

}  // namespace ekv
