// Page management of the cache: copying, forking, freeing, reserving and
// compacting pages over one reference count per physical page.
//
// ref[phys] counts the page-table entries that name the page; 0 is a free page.
// There is no free list to keep in step: whoever needs pages scans the counts
// and takes the lowest-numbered free pages in ascending order, so the ids a
// call hands out depend on the counts alone, never on the order in which
// threads run.  Counts change by integer atomics (exact in any order); an entry
// is released by exchanging it for -1, so that it is released once however
// often its row is listed.
//
// Moving a page costs reading and writing its bytes (2 x 268 KB at 8 kv heads,
// 64 tokens, 128 dims, bf16), which bounds compaction and copies; everything
// else is table rows and counts, a few microseconds bound by launches.
#include "common.cuh"
#include "kernels.cuh"

#include <algorithm>

namespace ekv {

constexpr int kPlanCluster = 8;          // CTAs of the counting cluster
constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = 16384;        // bytes of a page that one CTA moves at a time
constexpr int kRowChunk = 1024;          // page-table entries that one CTA walks
constexpr int kRowThreads = 256;

// ---------------------------------------------------------------- moving pages
// A page as one run of bytes: K, V, kmin, kmax, mean, m2 (each a multiple of
// 16 bytes), and its token count.
struct PageBytes {
    uint8_t* base[6];
    uint32_t vecs[6];                    // 16-byte words of the page in each array
    uint32_t total;
    int32_t* count;
    int chunks;                          // of the whole run
    int pieces;                          // chunks that stay inside one array
};

static PageBytes page_bytes(const entmaxkv_pool& p)
{
    PageBytes b{};
    void* base[6] = {p.k_pool, p.v_pool, p.kmin, p.kmax, p.mean, p.m2};
    const uint32_t elt = p.dtype == ENTMAXKV_BF16 ? 2 : 4;
    const uint32_t row = (uint32_t)p.H_kv * p.d;
    const uint32_t bytes[6] = {row * p.ps * elt, row * p.ps * elt, row * elt, row * elt, row * 4, row * 4};
    for (int i = 0; i < 6; ++i) {
        b.base[i] = static_cast<uint8_t*>(base[i]);
        b.vecs[i] = bytes[i] / 16;
        b.total += b.vecs[i];
    }
    for (int i = 0; i < 6; ++i) b.pieces += (int)((bytes[i] + kCopyChunk - 1) / kCopyChunk);
    b.count = p.count;
    b.chunks = (int)((b.total + kCopyChunk / 16 - 1) / (kCopyChunk / 16));
    return b;
}

EKV_DEV uint4* page_word(const PageBytes& pb, int page, uint32_t v)
{
    int i = 0;
#pragma unroll
    for (int k = 0; k < 5; ++k)
        if (i == k && v >= pb.vecs[k]) {
            v -= pb.vecs[k];
            i = k + 1;
        }
    uint8_t* base = pb.base[0];
    uint32_t n = pb.vecs[0];
#pragma unroll
    for (int k = 1; k < 6; ++k)
        if (i == k) {
            base = pb.base[k];
            n = pb.vecs[k];
        }
    return reinterpret_cast<uint4*>(base) + (size_t)page * n + v;
}

// Piece `piece` of page src and where it goes; returns its bytes.
EKV_DEV uint32_t page_piece(const PageBytes& pb, int piece, int src, int dst, uint8_t*& from, uint8_t*& to)
{
    uint32_t bytes = 0;
    bool found = false;
#pragma unroll
    for (int k = 0; k < 6; ++k) {
        const uint32_t size = pb.vecs[k] * 16;
        const int n = (int)((size + kCopyChunk - 1) / kCopyChunk);
        if (!found && piece < n) {
            found = true;
            from = pb.base[k] + (size_t)src * size + (size_t)piece * kCopyChunk;
            to = pb.base[k] + (size_t)dst * size + (size_t)piece * kCopyChunk;
            bytes = min(size - (uint32_t)piece * kCopyChunk, (uint32_t)kCopyChunk);
        }
        if (!found) piece -= n;
    }
    return bytes;
}

// Copy chunk `chunk` of page src to page dst; all threads of the CTA.
EKV_DEV void copy_chunk(const PageBytes& pb, int src, int dst, int chunk)
{
    constexpr int PER = kCopyChunk / 16 / kCopyThreads;
    const uint32_t v0 = (uint32_t)chunk * (kCopyChunk / 16) + threadIdx.x;
    uint4 t[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t v = v0 + i * kCopyThreads;
        if (v < pb.total) t[i] = *page_word(pb, src, v);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t v = v0 + i * kCopyThreads;
        if (v < pb.total) *page_word(pb, dst, v) = t[i];
    }
    if (chunk == 0 && threadIdx.x == 0) pb.count[dst] = pb.count[src];
}

// Many pages: one warp a CTA moves chunks through a ring in shared memory with
// bulk copies in both directions, so that what is in flight does not go by
// threads and registers.  Measured (the kernel alone, profiled) at 251 pages of
// 268 KB: 21.7 us, 6.2 TB/s read and written, against 34.7 us by way of
// registers as above.  `pick` gives the pages of copy i, or false to skip it.
constexpr int kRingSlots = 3, kRingCtas = 4;           // 48 KB a CTA, four CTAs an SM
constexpr int kRingBytes = kRingSlots * kCopyChunk;

EKV_DEV void bulk_store(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <typename Pick>
EKV_DEV void copy_ring(const PageBytes& pb, long long copies, int first, int step, uint8_t* ring, int32_t* status,
                       const Pick& pick)
{
    __shared__ uint64_t full[kRingSlots];
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int i = 0; i < kRingSlots; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const long long units = copies * pb.pieces;
    long long loaded = 0, stored = 0;                  // chunks; the same in all lanes
    uint8_t* out[kRingSlots] = {};                     // lane 0: where a slot's chunk goes
    uint32_t size[kRingSlots] = {};
    bool ok = true;
    auto store = [&] {
        const int slot = (int)(stored % kRingSlots);
        ok = mbar_wait(&full[slot], (uint32_t)((stored / kRingSlots) & 1), kWaitLimitNs) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0)
#pragma unroll
            for (int i = 0; i < kRingSlots; ++i)
                if (i == slot) bulk_store(out[i], ring + i * kCopyChunk, size[i]);
        ++stored;
    };
    for (long long u0 = first; ok && u0 < units; u0 += 32ll * step) {
        // 32 chunks at a time, one a lane, so that the lists' latencies overlap
        const long long u = u0 + (long long)lane * step;
        uint8_t *from = nullptr, *to = nullptr;
        uint32_t bytes = 0;
        if (u < units) {
            const int i = (int)(u / pb.pieces), piece = (int)(u % pb.pieces);
            int s, d;
            if (pick(i, piece == 0, s, d)) {
                bytes = page_piece(pb, piece, s, d, from, to);
                if (piece == 0) pb.count[d] = pb.count[s];
            }
        }
        const uint32_t some = __ballot_sync(0xffffffffu, bytes != 0);
        for (uint32_t m = some; ok && m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            uint8_t* f = (uint8_t*)__shfl_sync(0xffffffffu, (unsigned long long)from, l);
            uint8_t* t = (uint8_t*)__shfl_sync(0xffffffffu, (unsigned long long)to, l);
            const uint32_t n = __shfl_sync(0xffffffffu, bytes, l);
            const int slot = (int)(loaded % kRingSlots);
            if (loaded >= kRingSlots && lane == 0)     // the chunk before in this slot has been read
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kRingSlots - 2) : "memory");
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[slot], n);
                bulk_load(ring + slot * kCopyChunk, f, n, &full[slot]);
            }
#pragma unroll
            for (int i = 0; i < kRingSlots; ++i)
                if (i == slot) {
                    out[i] = t;
                    size[i] = n;
                }
            ++loaded;
            if (loaded - stored == kRingSlots - 1) store();
        }
    }
    while (ok && stored < loaded) store();
    if (!ok) {
        if (lane == 0) report(status, ENTMAXKV_TIMEOUT);
        for (long long i = stored; i < loaded; ++i)
            mbar_wait(&full[i % kRingSlots], (uint32_t)((i / kRingSlots) & 1), kWaitLimitNs);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Which pairs may be copied at once: mark[dst] counts the pairs that write a
// page, with bit 30 set where a pair reads it.  One CTA; only listed pages are
// touched, so the marks need no clearing beforehand.
constexpr int kMarkRead = 1 << 30;

__global__ void __launch_bounds__(1024) copy_mark_kernel(const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, int n, int num_phys,
                                                         int32_t* mark, int32_t* status)
{
    pdl_enter();
    auto fine = [&](int s, int d) { return s >= 0 && s < num_phys && d >= 0 && d < num_phys; };
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = src[i], d = dst[i];
        if (fine(s, d)) mark[s] = mark[d] = 0;
        else report(status, ENTMAXKV_DEVICE_BOUNDS);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = src[i], d = dst[i];
        if (!fine(s, d) || s == d) continue;
        atomicOr(&mark[s], kMarkRead);
        atomicAdd(&mark[d], 1);
    }
}

__global__ void __launch_bounds__(32) copy_pages_kernel(const PageBytes pb, const int32_t* __restrict__ src,
                                                        const int32_t* __restrict__ dst, int n, int num_phys,
                                                        const int32_t* __restrict__ mark, int32_t* status)
{
    pdl_enter();
    extern __shared__ __align__(128) uint8_t ring[];
    copy_ring(pb, n, blockIdx.x, gridDim.x, ring, status, [&](int i, bool once, int& s, int& d) {
        s = src[i];
        d = dst[i];
        if (s < 0 || s >= num_phys || d < 0 || d >= num_phys || s == d) return false;
        if (mark[d] == 1) return true;
        if (once) report(status, ENTMAXKV_DEVICE_BOUNDS);   // written by two pairs, or read by one
        return false;
    });
}

// ---------------------------------------------------------------- counting
struct PlanHead {
    int32_t live, free, moves, pad;
};

struct PlanArgs {
    int32_t* ref;
    int num_phys;
    int slice;                           // pages a CTA of the cluster scans, a multiple of 32
    int limit;                           // free ids to list at most
    PlanHead* head;
    int32_t* free_ids;                   // ascending (compaction: the holes below the live count)
    int32_t* movers;                     // compaction: live pages at or above the live count, ascending
    int32_t* rank;                       // compaction: a mover's position, -1 for a free page, 0 for one that stays
    // rows that want pages, in order (fork: 0 or 1 each; reserve: any number)
    int rows;
    int32_t* want;                       // [rows] pages wanted
    int32_t* at;                         // [rows] pages wanted by the rows before
};

// Exclusive scan over the block; returns this thread's offset, `total` the sum.
EKV_DEV int block_scan(int v, int* sh, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int s = lane < nw ? sh[lane] : 0;
        int x = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += t;
        }
        sh[lane] = x - s;
        if (lane == 31) sh[32] = x;
    }
    __syncthreads();
    total = sh[32];
    return sh[warp] + inc - v;
}

// One cluster scans the counts: each CTA keeps a bitmap of its slice's live
// pages, the slices' totals go round the cluster, and each CTA lists the ids
// of its own slice at their place in the whole order, a warp a word of the bitmap.
// Latency bounds it (24000 pages: about 8 us as a launch of its own; one CTA
// without the cluster's barriers took 4 us longer).
template <bool COMPACT>
EKV_DEV void pages_plan(const PlanArgs& a, uint32_t* bits)
{
    __shared__ int sh[33];
    __shared__ int slice_live;
    const int tid = threadIdx.x, lane = tid & 31, r = (int)cluster_rank();
    const int base = min(r * a.slice, a.num_phys), end = min(base + a.slice, a.num_phys);
    const int words = (end - base + 31) / 32;
    int live = 0;
    for (int p = base + tid; p < base + words * 32; p += 8 * kPlanThreads) {
        bool on[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) on[k] = p + k * kPlanThreads < end && __ldcg(&a.ref[p + k * kPlanThreads]) != 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int w = (p + k * kPlanThreads - base) / 32;
            const uint32_t m = __ballot_sync(0xffffffffu, on[k]);
            if (w < words) {
                if (lane == 0) bits[w] = m;
                live += on[k];
            }
        }
    }
    int total;
    block_scan(live, sh, total);
    if (tid == 0) slice_live = total;
    cluster_sync();
    int before = 0, all = 0;
    for (int i = 0; i < kPlanCluster; ++i) {
        const int v = ld_dsmem_s32(dsmem(&slice_live, i));
        before += i < r ? v : 0;
        all += v;
    }
    cluster_arrive();                    // nobody reads another CTA's total after this
    if (r == 0 && tid == 0) {
        a.head->live = all;
        a.head->free = a.num_phys - all;
    }
    // words in runs of consecutive ones, a run a warp, a bit a lane
    const int warp = tid >> 5, run = (words + 31) / 32;
    const int w0 = min(warp * run, words), w1 = min(w0 + run, words);
    // compaction moves the live pages at or above the live count, `all`: their rank
    // counts from the number of live pages below it, free pages below are holes
    const int hole_end = COMPACT ? all : a.num_phys;
    int mine = 0, low = 0;
    for (int w = w0 + lane; w < w1; w += 32) {
        mine += __popc(bits[w]);
        if (COMPACT) {
            const int n = max(0, min(32, all - (base + w * 32)));
            low += __popc(bits[w] & (n == 32 ? 0xffffffffu : ((1u << n) - 1)));
        }
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    __syncthreads();                     // the scan's scratch is free
    if (lane == 0) sh[warp] = mine;
    __syncthreads();
    int live_at = before + __reduce_add_sync(0xffffffffu, lane < warp ? sh[lane] : 0);
    int free_at = base + w0 * 32 - live_at;            // pages below that are not live
    int below = 0;
    if (COMPACT) {
        __shared__ int slice_low;
        block_scan(low, sh, total);
        if (tid == 0) slice_low = total;
        cluster_wait();
        cluster_sync();
        for (int i = 0; i < kPlanCluster; ++i) below += ld_dsmem_s32(dsmem(&slice_low, i));
        cluster_arrive();
        if (r == 0 && tid == 0) a.head->moves = all - below;
    }
    for (int w = w0; w < w1; ++w) {
        const uint32_t m = bits[w];
        const int p = base + w * 32 + lane, lt = __popc(m & ((1u << lane) - 1)), n = min(32, end - (base + w * 32));
        if ((m >> lane) & 1) {
            if (COMPACT) {
                const int k = live_at + lt - below;
                if (p >= all) a.movers[k] = p;
                a.rank[p] = max(k, 0);
            }
        } else if (lane < n) {
            const int f = free_at + lane - lt;
            if (p < hole_end && f < a.limit) a.free_ids[f] = p;
            if (COMPACT) a.rank[p] = -1;
        }
        live_at += __popc(m);
        free_at += n - __popc(m);
    }
    if (!COMPACT && r == 0) {
        int done = 0;
        for (int i0 = 0; i0 < a.rows; i0 += kPlanThreads) {
            const int i = i0 + tid;
            const int v = i < a.rows ? __ldcg(&a.want[i]) : 0;
            const int off = block_scan(v, sh, total);
            if (i < a.rows) a.at[i] = done + off;
            done += total;
        }
    }
    cluster_wait();
}

template <bool COMPACT>
__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const PlanArgs a)
{
    pdl_enter();
    extern __shared__ uint32_t bits[];
    pages_plan<COMPACT>(a, bits);
}

// Where few table entries are concerned, the counting cluster also does what
// would be a launch before it, a warp a unit: kClusterEntries entries in all, and
// a row in pieces of kWarpChunk.  Measured: reserving for 48 rows in 24000 pages
// (with freeing 13 rows and two copies) 34.7 -> 30.7 us a pass; a fork of 4 rows
// 20.1 -> 17.6 us a call, though 14.8 -> 16.7 on the device alone.
constexpr long long kClusterEntries = 32768;
constexpr int kWarpChunk = 128;
constexpr int kPlanWarps = kPlanCluster * kPlanThreads / 32;
EKV_DEV int plan_warp() { return (int)cluster_rank() * (kPlanThreads / 32) + (int)(threadIdx.x >> 5); }

// ---------------------------------------------------------------- releasing
EKV_DEV void release_entry(int32_t* entry, int32_t* ref, int num_phys, int32_t* status)
{
    const int e = *entry < 0 ? -1 : atomicExch(entry, -1);
    if (e < 0) return;
    if (e >= num_phys) {
        report(status, ENTMAXKV_DEVICE_BOUNDS);
    } else if (atomicSub(&ref[e], 1) <= 0) {           // a page that nobody held
        atomicAdd(&ref[e], 1);
        report(status, ENTMAXKV_DEVICE_BOUNDS);
    }
}

__global__ void __launch_bounds__(kRowThreads) free_pages_kernel(int32_t* ref, int num_phys, int ps,
                                                                 int32_t* page_table, int max_pages,
                                                                 int32_t* seq_lens, int B, const int32_t* rows,
                                                                 int window, int sinks, int32_t* status)
{
    pdl_enter();
    const int b = rows ? rows[blockIdx.x] : (int)blockIdx.x;
    if (b < 0 || b >= B) {
        if (threadIdx.x == 0 && blockIdx.y == 0) report(status, ENTMAXKV_DEVICE_BOUNDS);
        return;
    }
    const int p0 = blockIdx.y * kRowChunk, p1 = min(p0 + kRowChunk, max_pages);
    // pages [0, keep_low) hold sinks, pages from keep_high on hold the window and what follows it
    int keep_low = 0, keep_high = INT32_MAX;
    if (window >= 0) {
        const int L = max(seq_lens[b], 0);
        keep_low = (int)(((long long)sinks + ps - 1) / ps);
        keep_high = max(L - window, 0) / ps;
    }
    for (int p = p0 + threadIdx.x; p < p1; p += blockDim.x)
        if (p >= keep_low && p < keep_high)
            release_entry(&page_table[(size_t)b * max_pages + p], ref, num_phys, status);
    if (window < 0 && blockIdx.y == 0 && threadIdx.x == 0) seq_lens[b] = 0;
}

// ---------------------------------------------------------------- forking
struct ForkArgs {
    int32_t* ref;
    int num_phys, ps;
    int32_t* page_table;
    int max_pages;
    int32_t* seq_lens;
    int B;
    const int32_t *src, *dst;
    int n;
    const PlanHead* head;
    const int32_t* free_ids;
    int32_t* want;                       // [n] 1 where a fork needs a page of its own (0 where it is refused)
    const int32_t* at;
    int32_t* status;
};

// Whether fork i may run: rows in range, its destination listed once and no
// fork's source.  All threads of the block call.
EKV_DEV bool fork_fine(const ForkArgs& a, int i)
{
    const int s = a.src[i], d = a.dst[i];
    bool bad = s < 0 || s >= a.B || d < 0 || d >= a.B;
    for (int j = threadIdx.x; j < a.n; j += blockDim.x) bad |= (j != i && a.dst[j] == d) || a.src[j] == d;
    return !__syncthreads_or(bad);
}

EKV_DEV bool fork_length_fine(const ForkArgs& a, int L) { return L >= 0 && L <= (long long)a.max_pages * a.ps; }

// Whether fork i needs a page of its own: its source ends inside a page that it
// holds.  One thread.
EKV_DEV int fork_need(const ForkArgs& a, int i, bool fine)
{
    if (fine) {
        const int s = a.src[i], L = a.seq_lens[s];
        if (fork_length_fine(a, L)) {
            if (L % a.ps == 0) return 0;
            const int e = a.page_table[(size_t)s * a.max_pages + L / a.ps];
            if (e < a.num_phys) return e >= 0;
        }
    }
    report(a.status, ENTMAXKV_DEVICE_BOUNDS);
    return 0;
}

// Releases what the destinations held, and says which forks need a page.
__global__ void __launch_bounds__(kRowThreads) fork_release_kernel(const ForkArgs a)
{
    pdl_enter();
    const int i = blockIdx.x;
    const bool fine = fork_fine(a, i);
    if (blockIdx.y == 0 && threadIdx.x == 0) a.want[i] = fork_need(a, i, fine);
    if (!fine) return;
    const int p0 = blockIdx.y * kRowChunk, p1 = min(p0 + kRowChunk, a.max_pages);
    for (int p = p0 + threadIdx.x; p < p1; p += blockDim.x)
        release_entry(&a.page_table[(size_t)a.dst[i] * a.max_pages + p], a.ref, a.num_phys, a.status);
}

// The same and the counting in one launch.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a, const PlanArgs plan)
{
    pdl_enter();
    extern __shared__ uint32_t bits[];
    const int lane = threadIdx.x & 31, chunks = (a.max_pages + kWarpChunk - 1) / kWarpChunk;
    for (int u = plan_warp(); u < a.n * chunks; u += kPlanWarps) {
        const int i = u / chunks, part = u % chunks;
        const int s = a.src[i], d = a.dst[i];
        bool bad = s < 0 || s >= a.B || d < 0 || d >= a.B;
        for (int j = lane; j < a.n; j += 32) bad |= (j != i && a.dst[j] == d) || a.src[j] == d;
        const bool fine = !__any_sync(0xffffffffu, bad);
        if (part == 0 && lane == 0) a.want[i] = fork_need(a, i, fine);
        if (!fine) continue;
        const int p1 = min((part + 1) * kWarpChunk, a.max_pages);
        for (int p = part * kWarpChunk + lane; p < p1; p += 32)
            release_entry(&a.page_table[(size_t)d * a.max_pages + p], a.ref, a.num_phys, a.status);
    }
    cluster_sync();
    pages_plan<false>(plan, bits);
}

// Writes the destinations' rows (blocks below n * row_chunks) and copies the
// pages that sources end inside of (the blocks after them).
__global__ void __launch_bounds__(kRowThreads) fork_apply_kernel(const ForkArgs a, const PageBytes pb, int row_chunks)
{
    pdl_enter();
    const bool row = (int)blockIdx.x < a.n * row_chunks;
    const int unit = row ? blockIdx.x : blockIdx.x - a.n * row_chunks;
    const int per = row ? row_chunks : pb.chunks;
    const int i = unit / per, part = unit % per;
    const int need = a.want[i];
    if (!row && need == 0) return;                     // also: refused forks need none
    if (row && !fork_fine(a, i)) return;
    const int s = a.src[i], d = a.dst[i];
    const int L = a.seq_lens[s];
    const int at = a.at[i];
    const bool short_of = need && at >= a.head->free;
    const int fresh = need && !short_of ? a.free_ids[at] : -1;
    const int32_t* from = a.page_table + (size_t)s * a.max_pages;
    if (!row) {
        if (fresh >= 0) copy_chunk(pb, from[L / a.ps], fresh, part);
        return;
    }
    const bool empty = short_of || !fork_length_fine(a, L);
    const int whole = empty ? 0 : L / a.ps;
    if (part == 0 && threadIdx.x == 0) {
        if (short_of) report(a.status, ENTMAXKV_NO_PAGES);
        a.seq_lens[d] = empty ? 0 : L;
        if (fresh >= 0) a.ref[fresh] = 1;
    }
    const int p1 = min((part + 1) * kRowChunk, a.max_pages);
    for (int p = part * kRowChunk + threadIdx.x; p < p1; p += blockDim.x) {
        int e = p < whole ? from[p] : -1;
        if (e >= a.num_phys) {
            report(a.status, ENTMAXKV_DEVICE_BOUNDS);
            e = -1;
        }
        if (e >= 0 && atomicAdd(&a.ref[e], 1) <= 0) report(a.status, ENTMAXKV_DEVICE_BOUNDS);
        if (fresh >= 0 && p == whole) e = fresh;
        a.page_table[(size_t)d * a.max_pages + p] = max(e, -1);
    }
}

// ---------------------------------------------------------------- reserving
struct ReserveArgs {
    int32_t* ref;
    int ps;
    int32_t* page_table;
    int max_pages;
    const int32_t* seq_lens;
    const int32_t* lens;                 // [B] tokens each row is to have room for
    const PlanHead* head;
    const int32_t* free_ids;
    int32_t* want;
    const int32_t* at;
    int32_t* status;
};

// Entries [first, last) of row b may need pages.
EKV_DEV void reserve_range(const ReserveArgs& a, int b, int& first, int& last)
{
    const int L = max(a.seq_lens[b], 0);
    first = (int)(((long long)L + a.ps - 1) / a.ps);
    last = (int)(((long long)max(a.lens[b], 0) + a.ps - 1) / a.ps);
}

__global__ void __launch_bounds__(kRowThreads) reserve_count_kernel(const ReserveArgs a)
{
    pdl_enter();
    __shared__ int red[kRowThreads / 32];
    const int b = blockIdx.x;
    int first, last, n = 0;
    reserve_range(a, b, first, last);
    if (last > a.max_pages) {
        if (threadIdx.x == 0) report(a.status, ENTMAXKV_DEVICE_BOUNDS);
        last = 0;                                      // a row that cannot hold them gets none
    }
    for (int p = first + threadIdx.x; p < last; p += blockDim.x)
        n += a.page_table[(size_t)b * a.max_pages + p] < 0;
    n = block_sum(n, red);
    if (threadIdx.x == 0) a.want[b] = n;
}

// The same and the counting in one launch, a warp a row.
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const ReserveArgs a, const PlanArgs plan)
{
    pdl_enter();
    extern __shared__ uint32_t bits[];
    const int lane = threadIdx.x & 31;
    for (int b = plan_warp(); b < plan.rows; b += kPlanWarps) {
        int first, last, n = 0;
        reserve_range(a, b, first, last);
        if (last > a.max_pages) {
            if (lane == 0) report(a.status, ENTMAXKV_DEVICE_BOUNDS);
            last = 0;                                  // a row that cannot hold them gets none
        }
#pragma unroll 4
        for (int p = first + lane; p < last; p += 32) n += a.page_table[(size_t)b * a.max_pages + p] < 0;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) a.want[b] = n;
    }
    pages_plan<false>(plan, bits);                     // its first cluster barrier stands before the rows' scan
}

__global__ void __launch_bounds__(kRowThreads) reserve_apply_kernel(const ReserveArgs a)
{
    pdl_enter();
    __shared__ int sh[33];
    const int b = blockIdx.x;
    const int want = a.want[b];
    if (want == 0) return;
    int at = a.at[b];
    if ((long long)at + want > a.head->free) {
        if (threadIdx.x == 0) report(a.status, ENTMAXKV_NO_PAGES);
        return;
    }
    int first, last, total;
    reserve_range(a, b, first, last);
    for (int p0 = first; p0 < last; p0 += kRowThreads) {
        const int p = p0 + threadIdx.x;
        int32_t* entry = &a.page_table[(size_t)b * a.max_pages + p];
        const bool need = p < last && *entry < 0;
        const int off = block_scan(need, sh, total);
        if (need) {
            const int id = a.free_ids[at + off];
            *entry = id;
            a.ref[id] = 1;
        }
        at += total;
    }
}

// ---------------------------------------------------------------- compacting
// Moves pages (CTAs below move_ctas) and renames the table's entries (the rest).
__global__ void __launch_bounds__(32) compact_apply_kernel(const PageBytes pb, int32_t* ref, int num_phys,
                                                           int32_t* page_table, long long entries, const PlanHead* head,
                                                           const int32_t* holes, const int32_t* movers,
                                                           const int32_t* rank, int32_t* live, int move_ctas,
                                                           int32_t* status)
{
    pdl_enter();
    if ((int)blockIdx.x < move_ctas) {
        extern __shared__ __align__(128) uint8_t ring[];
        copy_ring(pb, head->moves, blockIdx.x, move_ctas, ring, status, [&](int i, bool once, int& s, int& d) {
            s = movers[i];
            d = holes[i];
            if (once) {
                ref[d] = ref[s];
                ref[s] = 0;
            }
            return true;
        });
        return;
    }
    const int n_live = head->live;
    const int c = blockIdx.x - move_ctas, ctas = gridDim.x - move_ctas;
    if (c == 0 && threadIdx.x == 0) *live = n_live;
    for (long long i = (long long)c * 32 + threadIdx.x; i < entries; i += (long long)ctas * 32) {
        const int e = page_table[i];
        if (e < 0) continue;
        const int k = e < num_phys ? rank[e] : -1;
        if (k < 0) report(status, ENTMAXKV_DEVICE_BOUNDS);   // names no live page: left as it is
        else if (e >= n_live) page_table[i] = holes[k];
    }
}

// ---------------------------------------------------------------- host side
struct PagesLayout {
    size_t head, free_ids, movers, rank, want, at, total;
};

static PagesLayout pages_layout(long long entries, long long num_phys)
{
    auto r = [](size_t x) { return (x + 255) & ~size_t(255); };
    PagesLayout L{};
    size_t off = 0;
    L.head = off;     off += 256;
    L.free_ids = off; off += r(num_phys * 4);
    L.movers = off;   off += r(num_phys * 4);
    L.rank = off;     off += r(num_phys * 4);
    L.want = off;     off += r(entries * 4);
    L.at = off;       off += r(entries * 4);
    L.total = off;
    return L;
}

size_t pages_workspace(long long entries, long long num_phys)
{
    return entries < 0 || num_phys <= 0 ? 0 : pages_layout(entries, num_phys).total;
}

static int done(cudaError_t e) { return e == cudaSuccess ? ENTMAXKV_OK : ENTMAXKV_CUDA_ERROR; }

template <typename... KArgs, typename... Args>
static int launch_cluster(void (*kern)(KArgs...), const PlanArgs& a, cudaStream_t stream, const Args&... args)
{
    const int smem = a.slice / 8;                      // a bit a page: grows with the pool
    if (ensure_smem((const void*)kern, smem)) return ENTMAXKV_CUDA_ERROR;
    return done(launch_pdl_cluster(kern, dim3(kPlanCluster), dim3(kPlanThreads), kPlanCluster, smem, stream, args...));
}

static PlanArgs plan_args(char* ws, const PagesLayout& L, int32_t* ref, int num_phys)
{
    PlanArgs a{};
    a.ref = ref;
    a.num_phys = num_phys;
    a.slice = ((num_phys + kPlanCluster - 1) / kPlanCluster + 31) / 32 * 32;
    a.limit = num_phys;
    a.head = reinterpret_cast<PlanHead*>(ws + L.head);
    a.free_ids = reinterpret_cast<int32_t*>(ws + L.free_ids);
    a.movers = reinterpret_cast<int32_t*>(ws + L.movers);
    a.rank = reinterpret_cast<int32_t*>(ws + L.rank);
    a.want = reinterpret_cast<int32_t*>(ws + L.want);
    a.at = reinterpret_cast<int32_t*>(ws + L.at);
    return a;
}

static int copy_ctas(long long units) { return (int)std::min(units, (long long)num_sms() * kRingCtas); }

int launch_copy_pages(const entmaxkv_pool& pool, const int32_t* src, const int32_t* dst, int n, char* ws,
                      int32_t* status, cudaStream_t stream)
{
    const PagesLayout L = pages_layout(0, pool.num_phys_pages);
    int32_t* mark = reinterpret_cast<int32_t*>(ws + L.rank);
    const PageBytes pb = page_bytes(pool);
    int rc = done(launch_pdl(copy_mark_kernel, dim3(1), dim3(1024), 0, stream, src, dst, n, pool.num_phys_pages, mark,
                             status));
    if (rc) return rc;
    if (ensure_smem((const void*)copy_pages_kernel, kRingBytes)) return ENTMAXKV_CUDA_ERROR;
    return done(launch_pdl(copy_pages_kernel, dim3(copy_ctas((long long)n * pb.pieces)), dim3(32), kRingBytes, stream,
                           pb, src, dst, n, pool.num_phys_pages, mark, status));
}

int launch_free_pages(const entmaxkv_pool& pool, int32_t* ref, int32_t* page_table, int max_pages, int32_t* seq_lens,
                      int B, const int32_t* rows, int n, int window, int sinks, int32_t* status, cudaStream_t stream)
{
    const dim3 grid(n, (max_pages + kRowChunk - 1) / kRowChunk);
    return done(launch_pdl(free_pages_kernel, grid, dim3(kRowThreads), 0, stream, ref, pool.num_phys_pages, pool.ps,
                           page_table, max_pages, seq_lens, B, rows, window, sinks, status));
}

int launch_fork(const entmaxkv_pool& pool, int32_t* ref, int32_t* page_table, int max_pages, int32_t* seq_lens, int B,
                const int32_t* src, const int32_t* dst, int n, char* ws, int32_t* status, cudaStream_t stream)
{
    const PagesLayout L = pages_layout(n, pool.num_phys_pages);
    PlanArgs p = plan_args(ws, L, ref, pool.num_phys_pages);
    p.rows = n;
    p.limit = std::min(n, pool.num_phys_pages);        // a fork needs one page at most
    ForkArgs f{ref, pool.num_phys_pages, pool.ps, page_table, max_pages, seq_lens, B, src, dst, n,
               p.head, p.free_ids, p.want, p.at, status};
    const PageBytes pb = page_bytes(pool);
    const int row_chunks = (max_pages + kRowChunk - 1) / kRowChunk;
    if ((long long)n * (row_chunks + pb.chunks) > INT32_MAX) return ENTMAXKV_UNSUPPORTED;
    int rc;
    if ((long long)n * max_pages <= kClusterEntries && n <= kPlanWarps) {
        rc = launch_cluster(fork_plan_kernel, p, stream, f, p);
    } else {
        rc = done(launch_pdl(fork_release_kernel, dim3(n, row_chunks), dim3(kRowThreads), 0, stream, f));
        if (!rc) rc = launch_cluster(pages_plan_kernel<false>, p, stream, p);
    }
    if (rc) return rc;
    return done(launch_pdl(fork_apply_kernel, dim3(n * (row_chunks + pb.chunks)), dim3(kRowThreads), 0, stream, f, pb,
                           row_chunks));
}

int launch_reserve(const entmaxkv_pool& pool, int32_t* ref, int32_t* page_table, int max_pages,
                   const int32_t* seq_lens, int B, const int32_t* lens, char* ws, int32_t* status, cudaStream_t stream)
{
    const PagesLayout L = pages_layout(B, pool.num_phys_pages);
    PlanArgs p = plan_args(ws, L, ref, pool.num_phys_pages);
    p.rows = B;
    ReserveArgs r{ref, pool.ps, page_table, max_pages, seq_lens, lens, p.head, p.free_ids, p.want, p.at, status};
    int rc;
    if ((long long)B * max_pages <= kClusterEntries && max_pages <= 16 * kWarpChunk) {
        rc = launch_cluster(reserve_plan_kernel, p, stream, r, p);
    } else {
        rc = done(launch_pdl(reserve_count_kernel, dim3(B), dim3(kRowThreads), 0, stream, r));
        if (!rc) rc = launch_cluster(pages_plan_kernel<false>, p, stream, p);
    }
    if (rc) return rc;
    return done(launch_pdl(reserve_apply_kernel, dim3(B), dim3(kRowThreads), 0, stream, r));
}

int launch_compact(const entmaxkv_pool& pool, int32_t* ref, int32_t* page_table, int max_pages, int B, int32_t* live,
                   char* ws, int32_t* status, cudaStream_t stream)
{
    const PagesLayout L = pages_layout(0, pool.num_phys_pages);
    const PlanArgs p = plan_args(ws, L, ref, pool.num_phys_pages);
    const PageBytes pb = page_bytes(pool);
    const int rc = launch_cluster(pages_plan_kernel<true>, p, stream, p);
    if (rc) return rc;
    const long long entries = (long long)B * max_pages;
    const int move_ctas = copy_ctas((long long)pool.num_phys_pages / 2 * pb.pieces + 1);
    const int table_ctas = (int)std::min((entries + 127) / 128, 8ll * num_sms()) + 1;
    if (ensure_smem((const void*)compact_apply_kernel, kRingBytes)) return ENTMAXKV_CUDA_ERROR;
    return done(launch_pdl(compact_apply_kernel, dim3(move_ctas + table_ctas), dim3(32), kRingBytes, stream, pb, ref,
                           pool.num_phys_pages, page_table, entries, p.head, p.free_ids, p.movers, p.rank, live,
                           move_ctas, status));
}

}  // namespace ekv
