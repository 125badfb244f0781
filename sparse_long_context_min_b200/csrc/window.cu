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
// block barrier stands between a tile's arrival and its release.  The query
// (bf16 high + low part, columns 2h and 2h + 1) is the B operand of the score
// product, its result's layout is turned in registers (movmatrix) into the B
// operand of V^T P, and P again keeps a high and a low part: both splits leave
// about 2^-17 of relative error where one bf16 would leave 2^-9.
template <int D, int PS, int NT>
__global__ void __launch_bounds__(kRangeThreads, 2) range_bf16_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                      const __grid_constant__ CUtensorMap vmap,
                                                                      const RangeArgs a)
{
    pdl_enter();
    constexpr int STAGE = kRangeTile * D * 2;          // bytes of one tensor's tile
    constexpr int PPS = kRangeTile / PS;
    constexpr int KS = D / 16, MT = D / 16;
    constexpr int RED = D + kRedPad;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    float* red = reinterpret_cast<float*>(smem + 2 * kRangeStages * STAGE);   // [4 warps][4 heads][RED]
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
    RangeWalk w = range_start(a, PS, c_id, gridDim.x);         // holds block barriers
    if (w.left <= 0) return;
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
        // nothing of this CTA's is in flight once the last tiles have landed
        if (stop && lane == 0)
            for (long long i = max(0ll, issued - kRangeStages); i < issued; ++i)
                mbar_wait(&full[i % kRangeStages], (uint32_t)((i / kRangeStages) & 1), kWaitLimitNs);
        return;
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
        if (tid == 0) range_note_span(a, w, u, nt, done, c_id);

        uint32_t bq[NT][KS][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int head = 4 * x + (gi >> 1);
            const float* qh = a.q + ((size_t)b * a.H_q + (size_t)w.g * a.G + head) * D;
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 16 * j + 2 * c + 8 * e;
                    const float v0 = head < a.G ? qh[k] * a.xscale : 0.f;
                    const float v1 = head < a.G ? qh[k + 1] * a.xscale : 0.f;
                    const uint32_t p0 = split_pack(v0), p1 = split_pack(v1);
                    bq[x][j][e] = (gi & 1) ? __byte_perm(p0, p1, 0x7632) : __byte_perm(p0, p1, 0x5410);
                }
        }
        float acc[NT][MT][4], mrun[NT], lrun[NT];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            mrun[x] = -INFINITY;
            lrun[x] = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[x][m][0] = acc[x][m][1] = acc[x][m][2] = acc[x][m][3] = 0.f;
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
                    for (int x = 0; x < NT; ++x) mma_bf16(sc[x], af, bq[x][j][0], bq[x][j][1]);
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
                uint32_t pb[NT][2];
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
                            acc[x][m][0] *= corr; acc[x][m][1] *= corr;
                            acc[x][m][2] *= corr; acc[x][m][3] *= corr;
                        }
                        mrun[x] = mnew;
                    }
                    const float p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
                    lrun[x] += p0 + p1;
                    pb[x][0] = movmatrix_trans(split_pack(p0));
                    pb[x][1] = movmatrix_trans(split_pack(p1));
                }
                const int trow = row0 + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t af[4];
                    ldsm_x4_t(swz_addr(vbase, trow, 2 * m + ((lane >> 3) & 1)), af);
#pragma unroll
                    for (int x = 0; x < NT; ++x) mma_bf16(acc[x][m], af, pb[x][0], pb[x][1]);
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
                rw[16 * m + gi] = (acc[x][m][0] + acc[x][m][1]) * f;
                rw[16 * m + gi + 8] = (acc[x][m][2] + acc[x][m][3]) * f;
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
                    if (mi != -INFINITY) L += wl[flip][i][h] * exp2f(mi - Mh);
                    const float4 t = *reinterpret_cast<const float4*>(red + (i * 4 + h) * RED + d);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                range_store(a, whole, (long long)c_id + u, b, w.g, 4 * x + h, D, d, o, Mh, L);
            }
        }
        done += n;
        advance(n);
    }
}

// ---------------------------------------------------------------- fp32 cache
// Each warp owns 16 tokens of a tile and keeps everything in registers: LPT
// lanes share a token (each holds D / LPT coordinates of the query heads and of
// the output), 32 / LPT tokens advance together, and each lane group runs its
// own softmax state, joined once at the end of a unit.  All arithmetic is
// fp32.  Masked tokens are not read.
template <int D, int GT>
__global__ void __launch_bounds__(128, 2) range_f32_kernel(const float* __restrict__ k_pool,
                                                           const float* __restrict__ v_pool, int ps, const RangeArgs a)
{
    pdl_enter();
    constexpr int LPT = GT == 8 ? 16 : 8, TPW = 32 / LPT, E = D / LPT, E4 = E / 4;
    __shared__ float red[4][4][D + kRedPad];
    __shared__ float wm[2][4][4], wl[2][4][4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = lane / LPT, sub = lane % LPT;
    const int c_id = blockIdx.x;
    RangeWalk w = range_start(a, ps, c_id, gridDim.x);
    if (w.left <= 0) return;
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
        if (tid == 0) range_note_span(a, w, u, nt, done, c_id);
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
        const int steps = 16 / TPW;
        for (int it = 0; it < n * steps; ++it) {
            const int tok = warp * 16 + it % steps * TPW + grp;
            const long long li = ((long long)(w.t + it / steps) * kRangeTile + tok) / ps;
            const int lp = li < sp.pages() ? sp.logical((int)li) : sp.P;
            const int pos = lp * ps + tok % ps;
            bool valid = lp < sp.P && sp.valid(pos);
            int phys = 0;
            if (valid) {
                phys = a.page_table[(size_t)b * a.max_pages + lp];
                if (phys < 0 || phys >= a.num_phys) {
                    report(a.status, ENTMAXKV_DEVICE_BOUNDS);
                    valid = false;
                }
            }
            float4 k4[E4], v4[E4];
            const size_t row = valid ? (((size_t)phys * a.H_kv + w.g) * ps + tok % ps) * D : 0;
#pragma unroll
            for (int i = 0; i < E4; ++i) {
                const size_t o = row + (i * LPT + sub) * 4;
                k4[i] = valid ? __ldg(reinterpret_cast<const float4*>(k_pool + o)) : make_float4(0.f, 0.f, 0.f, 0.f);
                v4[i] = valid ? __ldg(reinterpret_cast<const float4*>(v_pool + o)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const float* k = reinterpret_cast<const float*>(k4);
            const float* v = reinterpret_cast<const float*>(v4);
#pragma unroll
            for (int h = 0; h < GT; ++h) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) x = fmaf(q[h][e], k[e], x);
#pragma unroll
                for (int o = LPT / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (!valid) x = -INFINITY;
                const float mnew = fmaxf(mrun[h], x);
                const float mu = mnew == -INFINITY ? 0.f : mnew;
                if (mnew > mrun[h]) {
                    const float corr = exp2f(mrun[h] - mu);
                    lrun[h] *= corr;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[h][e] *= corr;
                    mrun[h] = mnew;
                }
                const float p = exp2f(x - mu);
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
                    if (mi != -INFINITY) L += wl[flip][i][h] * exp2f(mi - Mh);
                    const float4 t = *reinterpret_cast<const float4*>(&red[i][h][d]);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                range_store(a, whole, (long long)c_id + u, b, w.g, 4 * x + h, D, d, o, Mh, L);
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
}

// ---------------------------------------------------------------- merge
// One CTA a unit: rows of a unit that several CTAs share are joined; rows of a
// unit without tokens get o = 0 and lse = -infinity.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) range_merge_kernel(int ps, const RangeArgs a)
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
    if (merge_parts<D, kMergeThreads>(list, PartList{}, a.G, o, m, l)) range_store(a, true, 0, b, g, h, D, d, o, m, l);
}

// ---------------------------------------------------------------- launch
template <int D, int PS, int NT>
static int launch_range_bf16(const RangeArgs& a, int C, const CUtensorMap* kmap, const CUtensorMap* vmap,
                             cudaStream_t stream)
{
    const int smem = 2 * kRangeStages * kRangeTile * D * 2 + 16 * (D + kRedPad) * 4 + 1024;
    if (ensure_smem((const void*)range_bf16_kernel<D, PS, NT>, smem)) return ENTMAXKV_CUDA_ERROR;
    const cudaError_t e = launch_pdl(range_bf16_kernel<D, PS, NT>, dim3(C), dim3(kRangeThreads), smem, stream, *kmap,
                                     *vmap, a);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

template <int D>
static int launch_range_d(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                          const CUtensorMap* vmap, cudaStream_t stream)
{
    if (pool.dtype == ENTMAXKV_F32) {
        const float* k = (const float*)pool.k_pool;
        const float* v = (const float*)pool.v_pool;
        const cudaError_t e = a.G == 8
                                  ? launch_pdl(range_f32_kernel<D, 8>, dim3(C), dim3(128), 0, stream, k, v, pool.ps, a)
                                  : launch_pdl(range_f32_kernel<D, 4>, dim3(C), dim3(128), 0, stream, k, v, pool.ps, a);
        return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
    }
    if (pool.ps == 64) return a.G == 8 ? launch_range_bf16<D, 64, 2>(a, C, kmap, vmap, stream)
                                       : launch_range_bf16<D, 64, 1>(a, C, kmap, vmap, stream);
    return a.G == 8 ? launch_range_bf16<D, 16, 2>(a, C, kmap, vmap, stream)
                    : launch_range_bf16<D, 16, 1>(a, C, kmap, vmap, stream);
}

int launch_range(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                 const CUtensorMap* vmap, cudaStream_t stream)
{
    return pool.d == 128 ? launch_range_d<128>(pool, a, C, kmap, vmap, stream)
                         : launch_range_d<64>(pool, a, C, kmap, vmap, stream);
}

int launch_window(const entmaxkv_pool& pool, const RangeArgs& a, int C, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream)
{
    const int rc = launch_range(pool, a, C, kmap, vmap, stream);
    if (rc) return rc;
    const dim3 grid(a.B * a.H_kv);
    const cudaError_t e = pool.d == 128
                              ? launch_pdl(range_merge_kernel<128>, grid, dim3(kMergeThreads), 0, stream, pool.ps, a)
                              : launch_pdl(range_merge_kernel<64>, grid, dim3(kMergeThreads), 0, stream, pool.ps, a);
    return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR;
}

}  // namespace ekv
