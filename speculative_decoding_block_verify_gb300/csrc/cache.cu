// The paged key-value cache around a verify step: spec_cache_append, spec_cache_resize,
// spec_cache_fork.
//
// The page table, the counts and the lengths live on the device and are only changed there, so a
// decode loop never waits for the host to learn how many tokens were kept.  All of it is integers
// whose result does not depend on the order in which threads run: reference counts change by
// atomic additions, and pages are given out by rank (the lowest free pages, in stream order),
// found by prefix sums.  A page is free when nobody holds it; there is no list to keep in step.

#include <cooperative_groups.h>

#include <atomic>

#include "blocks.cuh"
#include "host_util.h"

namespace sv {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------------------
// One CTA column per stream: the stream's rows are known from two words of cu_drafts, so no row
// searches for its stream.  A thread moves 16 bytes of K and of V (or one element of each, where a
// base or a row stride is not a multiple of 16 bytes).  Bound by latency at decode sizes (one stream's block: 2.8 us);
// 256 streams with up to 33 tokens of 8 heads of 128 (52.8 MB): 9.2 to 10.8 us from card to card, 4.9 to 5.7 TB/s.
// With resize's statuses, a stream that it had no room for is passed over: where a copy was not to be had, the table still
// has the shared page.  Of that page's holders one at most was told OK; it is passed over too where one that was not has
// tokens behind its own there (it was rolled back further).
// Every CTA checks the offsets up to its own stream, so the work of all grows with the square of the streams: one token each of one
// head of 64, from Python, takes 15.5 us for 1,024 streams (13.5 without offsets), 26 (18) for 4,096, 139 (38) for 16,384.
constexpr int kAppendThreads = 256;

template <typename U>   // the unit moved by a thread: uint4, or one element
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const spec_append_args a, const int32_t* reserved, int units_per_head) {
    __shared__ int s_first;
    __shared__ int s_page[SPEC_MAX_KMAX + 1];
    __shared__ int s_bad, s_others;
    const int b = blockIdx.x, tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = __ldcg(a.length + b);
    if (tid == 0) s_bad = s_others = 0;
    const int refused = reserved != nullptr ? __ldcg(reserved + b) : SPEC_ST_OK;
    const bool offsets_ok = valid_prefix(a.cu_drafts, a.B, a.kmax, a.rows, b + 1, &s_first) > b;
    int status = SPEC_ST_OK, n = 0;
    int64_t row0 = 0;
    if (!offsets_ok) {
        status = SPEC_ST_BAD_OFFSETS;
    } else if (refused != SPEC_ST_OK) {
        status = refused;
    } else {
        n = block_rows(a.cu_drafts, b, a.kmax);
        row0 = first_row(a.cu_drafts, b, a.kmax);
        if (len < 0 || (int64_t)len + n > (int64_t)a.max_pages * a.page_size) status = SPEC_ST_BAD_LENGTH;
    }
    const int shift = __ffs(a.page_size) - 1;
    __syncthreads();
    if (status == SPEC_ST_OK) {
        for (int i = tid; i < n; i += kAppendThreads) {
            int page = *(a.page_table + (int64_t)b * a.max_pages + ((len + i) >> shift));
            if ((unsigned)page >= (unsigned)a.num_pages) {
                page = -1;
                s_bad = 1;
            }
            s_page[i] = page;
        }
        if (reserved != nullptr && (len & (a.page_size - 1)) != 0) {
            const int32_t* table = a.page_table + (len >> shift);
            const int mine = *(table + (int64_t)b * a.max_pages);
            for (int o = tid; o < a.B; o += kAppendThreads)
                if (__ldcg(reserved + o) == SPEC_ST_NO_PAGES && __ldcg(a.length + o) > len && *(table + (int64_t)o * a.max_pages) == mine)
                    s_others = 1;
        }
    }
    __syncthreads();
    if (s_others) status = SPEC_ST_NO_PAGES;
    const bool bad_page = status == SPEC_ST_OK && s_bad;
    if (blockIdx.y == 0 && tid == 0) a.status[b] = bad_page ? SPEC_ST_BAD_PAGE : status;
    if (status != SPEC_ST_OK) return;
    const U* k = reinterpret_cast<const U*>(a.k);
    const U* v = reinterpret_cast<const U*>(a.v);
    U* kp = reinterpret_cast<U*>(a.k_pages);
    U* vp = reinterpret_cast<U*>(a.v_pages);
    const int64_t per = a.D / units_per_head;   // elements of a unit
    const int64_t kstride = a.k_row_stride / per, vstride = a.v_row_stride / per;
    const int per_row = a.Hkv * units_per_head;
    const int total = n * per_row;
    for (int u = blockIdx.y * kAppendThreads + tid; u < total; u += gridDim.y * kAppendThreads) {
        const int i = u / per_row, rest = u - i * per_row;
        const int h = rest / units_per_head, c = rest - h * units_per_head;
        const int page = s_page[i];
        if (page < 0) continue;
        const U x = *(k + (row0 + i) * kstride + rest);
        const U y = *(v + (row0 + i) * vstride + rest);
        const int64_t to = (((int64_t)page * a.Hkv + h) * a.page_size + ((len + i) & (a.page_size - 1))) * units_per_head + c;
        kp[to] = x;
        vp[to] = y;
    }
}

// ---------------------------------------------------------------------------------------
// resize
// ---------------------------------------------------------------------------------------
// Workspace: a header {pairs}, the copies, the shared pages that streams ask a copy of, and the free pages in rank order.
struct ResizeSpace {
    int32_t* header;   // [0] copies asked for
    int2* pair;        // copies {from, to}; from = -1: none was made
    int32_t* ask;      // [B] the shared page that stream b wants a copy of, or -1
    int32_t* copy;     // [B] ... and gets one
    int32_t* list;     // [num_pages] the free pages, lowest first
};

__host__ __device__ inline size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

__host__ __device__ inline ResizeSpace resize_space(void* ws, int B) {
    char* p = reinterpret_cast<char*>(ws);
    const size_t per = round16((size_t)B * 4);
    return {reinterpret_cast<int32_t*>(p), reinterpret_cast<int2*>(p + 256), reinterpret_cast<int32_t*>(p + 256 + 2 * per),
            reinterpret_cast<int32_t*>(p + 256 + 3 * per), reinterpret_cast<int32_t*>(p + 256 + 4 * per)};
}

static size_t resize_workspace(int B, int num_pages) {
    return 256 + 4 * round16((size_t)B * 4) + round16((size_t)num_pages * 4);
}

__device__ __forceinline__ bool in_pool(int page, int num_pages) { return (unsigned)page < (unsigned)num_pages; }

// What a stream keeps and needs (step 1's decisions).
struct StreamPlan {
    int status, next, keep, want, held;
    int tail;   // the page that holds kept tokens and will be written into, where it is shared, or -1
};

// A thread's stream; stream b may be past the last one (then nothing is planned).  A few pages to look at are the
// thread's own, many are looked at by the whole warp, one stream after the other.
constexpr int kOwnPages = 8;
__device__ __forceinline__ StreamPlan plan_stream(const spec_resize_args& a, int b) {
    StreamPlan s = {SPEC_ST_OK, 0, 0, 0, 0, -1};
    const int lane = threadIdx.x & 31, shift = __ffs(a.page_size) - 1;
    int full = 0, lim = 0;
    bool bad = false, mixed = false;
    if (b < a.B) {
        const int len = __ldcg(a.length + b);
        s.held = __ldcg(a.held + b);
        const int adv = a.advance != nullptr ? __ldcg(a.advance + b) : 0;
        const int room = a.room != nullptr ? __ldcg(a.room + b) : 0;
        const int64_t n = (int64_t)len + adv;
        s.next = len;
        s.keep = s.want = full = lim = s.held;
        if (len < 0 || n < 0 || room < 0 || s.held < 0 || s.held > a.max_pages || n > (int64_t)s.held << shift ||
            n + room > (int64_t)a.max_pages << shift) {
            s.status = SPEC_ST_BAD_LENGTH;
        } else {
            s.next = (int)n;
            s.want = (int)((n + room + a.page_size - 1) >> shift);
            full = (int)((n + a.page_size - 1) >> shift);
            s.keep = lim = min(s.want, s.held);
            mixed = room > 0 && (n & (a.page_size - 1)) != 0;
        }
    }
    const int32_t* row = a.page_table + (int64_t)b * a.max_pages;
    if (mixed) {
        s.tail = __ldcg(row + (s.next >> shift));
        if (!in_pool(s.tail, a.num_pages)) {
            bad = true;
            s.tail = -1;
        } else if (__ldcg(a.ref_count + s.tail) <= 1) {
            s.tail = -1;
        }
    }
    const int look = s.status == SPEC_ST_OK ? s.held - full : 0;
    if (look <= kOwnPages) {
        for (int j = full; j < full + look; ++j) {
            const int p = __ldcg(row + j);
            if (!in_pool(p, a.num_pages))
                bad = true;
            else if (j < lim && __ldcg(a.ref_count + p) > 1)
                s.keep = min(s.keep, j);
        }
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, look > kOwnPages); todo != 0; todo &= todo - 1) {
        const int who = __ffs(todo) - 1;
        const int f = __shfl_sync(0xffffffffu, full, who), h = __shfl_sync(0xffffffffu, s.held, who);
        const int l = __shfl_sync(0xffffffffu, lim, who), ob = __shfl_sync(0xffffffffu, b, who);
        const int32_t* other = a.page_table + (int64_t)ob * a.max_pages;
        int first = l;
        bool wrong = false;
#pragma unroll 4
        for (int j = f + lane; j < h; j += 32) {
            const int p = __ldcg(other + j);
            if (!in_pool(p, a.num_pages))
                wrong = true;
            else if (j < l && __ldcg(a.ref_count + p) > 1)
                first = min(first, j);
        }
        first = warp_min_i(first);
        wrong = __any_sync(0xffffffffu, wrong);
        if (lane == who) {
            s.keep = first;
            bad |= wrong;
        }
    }
    if (bad) {
        s.status = SPEC_ST_BAD_PAGE;
        s.next = __ldcg(a.length + b);
        s.keep = s.want = s.held;
        s.tail = -1;
    }
    return s;
}

// Pages [keep, held) of every thread's stream lose a reference.
__device__ __forceinline__ void drop_pages(const spec_resize_args& a, int b, int keep, int held) {
    const int lane = threadIdx.x & 31;
    int32_t* row = a.page_table + (int64_t)b * a.max_pages;
    if (held - keep <= kOwnPages) {
        for (int j = keep; j < held; ++j) {
            atomicSub(a.ref_count + __ldcg(row + j), 1);
            row[j] = -1;
        }
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, held - keep > kOwnPages); todo != 0; todo &= todo - 1) {
        const int who = __ffs(todo) - 1;
        const int k = __shfl_sync(0xffffffffu, keep, who), h = __shfl_sync(0xffffffffu, held, who);
        int32_t* other = a.page_table + (int64_t)__shfl_sync(0xffffffffu, b, who) * a.max_pages;
#pragma unroll 4
        for (int j = k + lane; j < h; j += 32) {
            atomicSub(a.ref_count + __ldcg(other + j), 1);
            other[j] = -1;
        }
    }
}

// Without room no page is asked for, no page is replaced, and no decision reads a count: every
// stream is independent, a thread each.
constexpr int kTrimThreads = 64;
__global__ void __launch_bounds__(kTrimThreads) trim_kernel(const spec_resize_args a) {
    const int b = blockIdx.x * kTrimThreads + threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const StreamPlan s = plan_stream(a, b);
    drop_pages(a, b, s.keep, s.held);
    if (b < a.B) {
        a.status[b] = s.status;
        if (s.status == SPEC_ST_OK) {
            a.length[b] = s.next;
            a.held[b] = s.keep;
        }
    }
}

// A sum that stops at 2^31 - 1.  Streams may ask for 2^28 pages each and a batch for more than an int counts; a pool has fewer than
// that, so no sum that stopped is taken for one that fits.  (Two calls of resize 10.9 -> 11.1 us; with sums in 64 bits 11.3.)
__device__ __forceinline__ int capped(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)INT32_MAX); }

// Exclusive prefix sums over the block of one int per thread (returns the block's total).
template <int kThreads, bool kCapped = false>
__device__ __forceinline__ int block_scan(int v, int* before, int* scratch /* [kThreads / 32] */) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = kCapped ? capped(x, y) : x + y;
    }
    const int left = kCapped ? __shfl_up_sync(0xffffffffu, x, 1) : 0;
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) base = kCapped ? capped(base, scratch[w]) : base + scratch[w];
        total = kCapped ? capped(total, scratch[w]) : total + scratch[w];
    }
    *before = !kCapped ? base + x - v : lane > 0 ? capped(base, left) : base;
    return total;
}

// With room: one cluster, whose barriers separate the steps (a count is read only when every
// change of the step before it is done).  A thread has neighbouring streams, as many as there are thousands of
// streams (one up to 4,096), and keeps what it planned in shared memory.  Latency: 7 us for 64 streams and for 1,024 in
// a pool of 260,000 pages (a warp per stream and six barriers took 33 us there).
constexpr int kResizeThreads = 512;
constexpr int kResizeCtas = 8;
constexpr int kScanPer = 16;   // counts that a thread looks at in one pass over the pool

struct Planned {
    int32_t status, next, keep, want, need, copy;
};

__global__ void __cluster_dims__(kResizeCtas, 1, 1) __launch_bounds__(kResizeThreads)
    resize_kernel(const spec_resize_args a, int per) {
    extern __shared__ Planned planned[];   // [per][kResizeThreads]
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int scratch[kResizeThreads / 32];
    __shared__ int s_need[kResizeCtas], s_copies[kResizeCtas], s_asks[kResizeCtas];
    __shared__ int s_count[2][kResizeCtas];
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = (int)cluster.block_rank();
    const int b0 = (rank * kResizeThreads + tid) * per;
    const ResizeSpace w = resize_space(a.workspace, a.B);
    auto tell = [&](int* slots, int value) {   // every CTA of the cluster learns this CTA's value
        if (tid < kResizeCtas) *cluster.map_shared_rank(slots + rank, tid) = value;
    };
    cluster.sync();   // every CTA's shared memory is there
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copies, which wait for the whole grid

    bool asks = false;
    for (int i = 0; i < per; ++i) {
        const int b = b0 + i;
        const StreamPlan s = plan_stream(a, b);
        planned[i * kResizeThreads + tid] = {s.status, s.next, s.keep, s.want, s.want - s.keep, s.held};
        if (b < a.B) w.ask[b] = s.tail;
        asks |= s.tail >= 0;
    }
    tell(s_asks, __syncthreads_or(asks));
    cluster.sync();   // every count that a plan looks at has been read
    bool any_asks = false;
    for (int c = 0; c < kResizeCtas; ++c) any_asks |= s_asks[c] != 0;
    for (int i = 0; i < per; ++i) {
        Planned& q = planned[i * kResizeThreads + tid];
        drop_pages(a, b0 + i, q.keep, q.copy /* held */);
        q.copy = 0;
    }
    if (any_asks) {
        cluster.sync();
        // shared pages that will be written into, now that step 1 is done
        for (int i = 0; i < per; ++i) {
            const int p = b0 + i < a.B ? __ldcg(w.ask + b0 + i) : -1;
            if (p >= 0 && __ldcg(a.ref_count + p) <= 1) w.ask[b0 + i] = -1;
        }
        cluster.sync();
        // A copy for every holder that asks, but the lowest one where all of them ask.  The askers (a fork's
        // continuations, next to one another) are spread over the cluster's warps; each looks through all streams:
        // from Python 18 us for 129 askers of 256 streams, 29 for 513 of 1,024, 133 for 2,049 of 4,096, 1,630 for 8,193 of 16,384.
        for (int b = rank * (kResizeThreads / 32) + (tid >> 5); b < a.B; b += kResizeCtas * kResizeThreads / 32) {
            const int p = __ldcg(w.ask + b);
            if (p < 0) continue;
            int same = 0;
            bool lower = false;
#pragma unroll 4
            for (int o = lane; o < a.B; o += 32) {
                const bool eq = __ldcg(w.ask + o) == p;
                same += eq;
                lower |= eq && o < b;
            }
            same = __reduce_add_sync(0xffffffffu, same);
            lower = __any_sync(0xffffffffu, lower);
            if (lane == 0) w.copy[b] = lower || same != __ldcg(a.ref_count + p);
        }
        cluster.sync();
        for (int i = 0; i < per; ++i) {
            if (b0 + i < a.B && __ldcg(w.ask + b0 + i) >= 0 && __ldcg(w.copy + b0 + i) != 0) {
                planned[i * kResizeThreads + tid].copy = 1;
                ++planned[i * kResizeThreads + tid].need;
            }
        }
    }
    // ranks of the streams' new pages and copies, in stream order
    int need = 0, copies = 0, begin, nth;
    for (int i = 0; i < per; ++i) {
        need = capped(need, planned[i * kResizeThreads + tid].need);
        copies += planned[i * kResizeThreads + tid].copy;
    }
    tell(s_need, block_scan<kResizeThreads, true>(need, &begin, scratch));
    tell(s_copies, any_asks ? block_scan<kResizeThreads>(copies, &nth, scratch) : (nth = 0));
    cluster.sync();   // (and every reference given up is given up)
    int total = 0, pairs = 0;
    for (int c = 0; c < kResizeCtas; ++c) {
        if (c < rank) {
            begin = capped(begin, s_need[c]);
            nth += s_copies[c];
        }
        total = capped(total, s_need[c]);
        pairs += s_copies[c];
    }
    if (rank == 0 && tid == 0) w.header[0] = pairs;
    // the first `total` free pages, by rank
    int found = 0;
    const bool vec = (reinterpret_cast<uintptr_t>(a.ref_count) & 15) == 0;
    constexpr int kChunk = kResizeCtas * kResizeThreads * kScanPer;
    int turn = 0;
    for (int64_t base = 0; base < a.num_pages && found < total; base += kChunk, turn ^= 1) {
        const int64_t p0 = base + ((int64_t)rank * kResizeThreads + tid) * kScanPer;
        unsigned mask = 0;
        if (vec && p0 + kScanPer <= a.num_pages) {
            int4 r[kScanPer / 4];
#pragma unroll
            for (int i = 0; i < kScanPer / 4; ++i) r[i] = __ldcg(reinterpret_cast<const int4*>(a.ref_count + p0) + i);
#pragma unroll
            for (int i = 0; i < kScanPer / 4; ++i)
                mask |= ((r[i].x == 0) | (r[i].y == 0) << 1 | (r[i].z == 0) << 2 | (r[i].w == 0) << 3) << (4 * i);
        } else {
#pragma unroll 4
            for (int i = 0; i < kScanPer; ++i)
                if (p0 + i < a.num_pages && __ldcg(a.ref_count + p0 + i) == 0) mask |= 1u << i;
        }
        int before;
        tell(s_count[turn], block_scan<kResizeThreads>(__popc(mask), &before, scratch));
        cluster.sync();
        int at = found + before;
        for (int c = 0; c < kResizeCtas; ++c) {
            const int n = s_count[turn][c];
            if (c < rank) at += n;
            found += n;
        }
        while (mask != 0 && at < total) {
            const int i = __ffs(mask) - 1;
            mask &= mask - 1;
            w.list[at++] = (int)(p0 + i);
        }
    }
    cluster.sync();   // the list is written, and nobody's shared memory is written any more
    for (int i = 0; i < per; ++i) {
        const int b = b0 + i;
        const Planned q = planned[i * kResizeThreads + tid];
        const bool fits = q.need == 0 || (int64_t)begin + q.need <= found;
        int32_t* row = a.page_table + (int64_t)b * a.max_pages;
        const int grow = fits ? q.want - q.keep : 0, from = fits ? begin + q.copy : 0;
        if (grow <= kOwnPages) {
            for (int j = 0; j < grow; ++j) {
                const int p = __ldcg(w.list + from + j);
                row[q.keep + j] = p;
                a.ref_count[p] = 1;
            }
        }
        for (unsigned todo = __ballot_sync(0xffffffffu, grow > kOwnPages); todo != 0; todo &= todo - 1) {
            const int who = __ffs(todo) - 1;
            const int g = __shfl_sync(0xffffffffu, grow, who), f = __shfl_sync(0xffffffffu, from, who);
            int32_t* other = a.page_table + (int64_t)__shfl_sync(0xffffffffu, b, who) * a.max_pages + __shfl_sync(0xffffffffu, q.keep, who);
#pragma unroll 4
            for (int j = lane; j < g; j += 32) {
                const int p = __ldcg(w.list + f + j);
                other[j] = p;
                a.ref_count[p] = 1;
            }
        }
        if (b < a.B) {
            if (q.copy) {
                int2 move = make_int2(-1, -1);
                if (fits) {
                    move = make_int2(__ldcg(w.ask + b), __ldcg(w.list + begin));
                    row[q.next / a.page_size] = move.y;
                    a.ref_count[move.y] = 1;
                    atomicSub(a.ref_count + move.x, 1);
                }
                w.pair[nth] = move;
            }
            a.status[b] = q.status == SPEC_ST_OK && !fits ? SPEC_ST_NO_PAGES : q.status;
            if (q.status == SPEC_ST_OK) {
                a.length[b] = q.next;
                a.held[b] = q.keep + grow;
            }
        }
        begin = capped(begin, q.need);
        nth += q.copy;
    }
}

// The copies that resize_kernel asked for: a warp moves up to 4 KB of one page of one layer of K
// or V, eight 16-byte loads of a lane in flight.  240 copies of 1 MB over 16 layers: 6.4 TB/s read and written.
constexpr int kCopyThreads = 256;
constexpr int kCopyPart = 4096;
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const spec_resize_args a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ResizeSpace w = resize_space(a.workspace, a.B);
    const int pairs = __ldcg(w.header);
    if (pairs == 0) return;
    const int lane = threadIdx.x & 31;
    const int64_t parts = (a.page_bytes + kCopyPart - 1) / kCopyPart;
    const int64_t per_pair = parts * a.layers * 2;
    const int64_t total = per_pair * pairs;
    for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < total;
         u += (int64_t)gridDim.x * (kCopyThreads / 32)) {
        const int64_t pr = u / per_pair, rest = u - pr * per_pair;
        const int2 move = __ldcg(w.pair + pr);
        if (move.x < 0) continue;
        const int64_t part = rest % parts, lk = rest / parts;
        char* pool = reinterpret_cast<char*>((lk & 1) ? a.v_pool : a.k_pool) + (lk >> 1) * (int64_t)a.num_pages * a.page_bytes;
        const int64_t off = part * kCopyPart;
        const int chunks = (int)((min((int64_t)kCopyPart, a.page_bytes - off)) >> 4);
        const uint4* from = reinterpret_cast<const uint4*>(pool + move.x * a.page_bytes + off);
        uint4* to = reinterpret_cast<uint4*>(pool + move.y * a.page_bytes + off);
        uint4 r[kCopyPart / 512];
#pragma unroll
        for (int i = 0; i < kCopyPart / 512; ++i)
            if (lane + 32 * i < chunks) r[i] = __ldcs(from + lane + 32 * i);
#pragma unroll
        for (int i = 0; i < kCopyPart / 512; ++i)
            if (lane + 32 * i < chunks) to[lane + 32 * i] = r[i];
    }
}

// ---------------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------------
// One CTA per pair.  A destination is nobody's source, so the rows that are read are not written.  Each CTA looks through all
// pairs for that: 14 us from Python for 512 pairs, 22 for 2,048, 50 for 8,192.
constexpr int kForkThreads = 256;
__global__ void __launch_bounds__(kForkThreads)
    fork_kernel(const int32_t* src, const int32_t* dst, int n, int B, int page_size, int num_pages, int max_pages,
                int32_t* page_table, int32_t* held, int32_t* length, int32_t* ref_count, int32_t* status) {
    const int e = blockIdx.x, tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = *(src + e), d = *(dst + e);
    bool bad = (unsigned)s >= (unsigned)B || (unsigned)d >= (unsigned)B;
    for (int o = tid; o < n; o += kForkThreads) bad |= *(src + o) == d || (o < e && *(dst + o) == d);
    if (__syncthreads_or(bad)) {
        if (tid == 0) status[e] = SPEC_ST_BAD_STREAM;
        return;
    }
    const int shift = __ffs(page_size) - 1;
    const int len = __ldcg(length + s), hs = __ldcg(held + s), hd = __ldcg(held + d);
    if (len < 0 || hs < 0 || hs > max_pages || hd < 0 || hd > max_pages || len > (int64_t)hs << shift) {
        if (tid == 0) status[e] = SPEC_ST_BAD_LENGTH;
        return;
    }
    const int pages = (int)(((int64_t)len + page_size - 1) >> shift);
    const int32_t* from = page_table + (int64_t)s * max_pages;
    int32_t* to = page_table + (int64_t)d * max_pages;
    bad = false;
    for (int j = tid; j < max(pages, hd); j += kForkThreads) {
        if (j < pages) bad |= !in_pool(__ldcg(from + j), num_pages);
        if (j < hd) bad |= !in_pool(__ldcg(to + j), num_pages);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) status[e] = SPEC_ST_BAD_PAGE;
        return;
    }
    for (int j = tid; j < max(pages, hd); j += kForkThreads) {
        const int give = j < hd ? __ldcg(to + j) : -1, take = j < pages ? __ldcg(from + j) : -1;
        if (give == take) continue;
        if (take >= 0) atomicAdd(ref_count + take, 1);
        if (give >= 0) atomicSub(ref_count + give, 1);
        to[j] = take;
    }
    if (tid == 0) {
        length[d] = len;
        held[d] = pages;
        status[e] = SPEC_ST_OK;
    }
}

static bool page_ok(int page_size) { return page_size >= 8 && page_size <= SPEC_MAX_PAGE && (page_size & (page_size - 1)) == 0; }
static bool table_ok(int max_pages, int page_size) { return (int64_t)max_pages * page_size <= INT32_MAX; }

}  // namespace sv

using namespace sv;

static int append(const spec_append_args* a, const int32_t* reserved, void* stream) {
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "spec_cache_append: args is NULL");
    if (!valid_dtype(a->dtype)) return set_error(SPEC_ERR_DTYPE, "spec_cache_append: dtype %d", a->dtype);
    if (a->B < 0 || a->B > SPEC_MAX_STREAMS || a->kmax < 0 || a->kmax > SPEC_MAX_KMAX)
        return set_error(SPEC_ERR_SHAPE, "spec_cache_append: B = %d, kmax = %d", a->B, a->kmax);
    if (a->Hkv < 1 || a->Hkv > 1024 || a->D < 8 || a->D > SPEC_MAX_HEAD || a->D % 8 != 0)
        return set_error(SPEC_ERR_SHAPE, "spec_cache_append: Hkv = %d, D = %d", a->Hkv, a->D);
    if (!page_ok(a->page_size) || a->num_pages < 1 || a->max_pages < 1 || !table_ok(a->max_pages, a->page_size))
        return set_error(SPEC_ERR_SHAPE, "spec_cache_append: page_size = %d, num_pages = %d, max_pages = %d", a->page_size,
                         a->num_pages, a->max_pages);
    if (a->k_row_stride < (int64_t)a->Hkv * a->D || a->v_row_stride < (int64_t)a->Hkv * a->D)
        return set_error(SPEC_ERR_SHAPE, "spec_cache_append: a row stride is below Hkv * D");
    if (a->rows < 0 || (a->cu_drafts == nullptr && a->rows < (int64_t)a->B * (a->kmax + 1)))
        return set_error(SPEC_ERR_SHAPE, "spec_cache_append: rows = %lld", (long long)a->rows);
    if (a->B == 0) return SPEC_OK;
    if (a->length == nullptr || a->page_table == nullptr || a->k == nullptr || a->v == nullptr || a->k_pages == nullptr ||
        a->v_pages == nullptr || a->status == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_cache_append: a required pointer is NULL");
    if (((uintptr_t)a->k_pages | (uintptr_t)a->v_pages) & 15)
        return set_error(SPEC_ERR_ARG, "spec_cache_append: the pool is not 16-byte aligned");
    const int es = a->dtype == SPEC_DTYPE_F32 ? 4 : 2;
    const bool vec = (((uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)(a->k_row_stride * es) | (uintptr_t)(a->v_row_stride * es)) & 15) == 0;
    const int upb = vec ? a->D * es / 16 : a->D;
    const int64_t units = (int64_t)(a->kmax + 1) * a->Hkv * upb;
    const int64_t want = (units + 2 * kAppendThreads - 1) / (2 * kAppendThreads);   // two units a thread
    const dim3 grid((unsigned)a->B, (unsigned)(want < 1 ? 1 : want > 64 ? 64 : want));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = vec       ? launch_after(append_kernel<uint4>, grid, dim3(kAppendThreads), 0, s, *a, reserved, upb)
                          : es == 2 ? launch_after(append_kernel<unsigned short>, grid, dim3(kAppendThreads), 0, s, *a, reserved, upb)
                                    : launch_after(append_kernel<float>, grid, dim3(kAppendThreads), 0, s, *a, reserved, upb);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_cache_append");
}

extern "C" int spec_cache_append(const spec_append_args* a, void* stream) {
    clear_error();
    return append(a, nullptr, stream);
}

extern "C" int spec_cache_append_reserved(const spec_append_args* a, const int32_t* reserved, void* stream) {
    clear_error();
    if (a != nullptr && a->B > 0 && reserved == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_cache_append_reserved: reserved is NULL");
    return append(a, reserved, stream);
}

extern "C" size_t spec_cache_resize_workspace_bytes(int32_t B, int32_t num_pages) {
    if (B <= 0 || B > SPEC_MAX_STREAMS || num_pages < 1) return 0;
    return resize_workspace(B, num_pages);
}

// The kernel's limit of dynamic shared memory, once a device and to the largest batch's: it is the function's and not
// the call's, so another host thread's smaller batch must not lower it before this one's launch.
static cudaError_t resize_limit() {
    static std::atomic<int> ready[64];
    constexpr int per = (SPEC_MAX_STREAMS + kResizeCtas * kResizeThreads - 1) / (kResizeCtas * kResizeThreads);
    constexpr int bytes = per * kResizeThreads * (int)sizeof(Planned);
    static_assert(bytes <= 200 * 1024, "shared memory of an SM");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev >= 0 && dev < 64 && ready[dev].load(std::memory_order_acquire) != 0)) return e;
    e = cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_release);
    return e;
}

extern "C" int spec_cache_resize(const spec_resize_args* a, void* stream) {
    clear_error();
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "spec_cache_resize: args is NULL");
    if (a->B < 0 || a->B > SPEC_MAX_STREAMS) return set_error(SPEC_ERR_SHAPE, "spec_cache_resize: B = %d", a->B);
    if (!page_ok(a->page_size) || a->num_pages < 1 || a->max_pages < 1 || !table_ok(a->max_pages, a->page_size))
        return set_error(SPEC_ERR_SHAPE, "spec_cache_resize: page_size = %d, num_pages = %d, max_pages = %d", a->page_size,
                         a->num_pages, a->max_pages);
    if (a->layers < 1 || a->page_bytes < 16 || a->page_bytes % 16 != 0)
        return set_error(SPEC_ERR_SHAPE, "spec_cache_resize: layers = %d, page_bytes = %lld", a->layers, (long long)a->page_bytes);
    if (a->B == 0) return SPEC_OK;
    if (a->page_table == nullptr || a->held == nullptr || a->length == nullptr || a->ref_count == nullptr ||
        a->k_pool == nullptr || a->v_pool == nullptr || a->status == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_cache_resize: a required pointer is NULL");
    if (((uintptr_t)a->k_pool | (uintptr_t)a->v_pool) & 15)
        return set_error(SPEC_ERR_ARG, "spec_cache_resize: the pool is not 16-byte aligned");
    if (a->workspace == nullptr || ((uintptr_t)a->workspace & 15) || a->workspace_bytes < resize_workspace(a->B, a->num_pages))
        return set_error(SPEC_ERR_WORKSPACE, "spec_cache_resize: workspace needs %zu bytes, 16-byte aligned",
                         resize_workspace(a->B, a->num_pages));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->room == nullptr) {
        const cudaError_t e = launch_after(trim_kernel, dim3((unsigned)((a->B + kTrimThreads - 1) / kTrimThreads)), dim3(kTrimThreads), 0, s, *a);
        return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_cache_resize");
    }
    const int per = (a->B + kResizeCtas * kResizeThreads - 1) / (kResizeCtas * kResizeThreads);
    const size_t smem = (size_t)per * kResizeThreads * sizeof(Planned);
    cudaError_t e = cudaSuccess;
    if (smem > 40000 && (e = resize_limit()) != cudaSuccess) return set_cuda_error(e, "spec_cache_resize");
    e = launch_after(resize_kernel, dim3(kResizeCtas), dim3(kResizeThreads), smem, s, *a, per);
    if (e != cudaSuccess) return set_cuda_error(e, "spec_cache_resize");
    // as many CTAs as the largest number of copies (one per stream) can keep busy, two per SM at most
    const int64_t units = (int64_t)a->B * a->layers * 2 * ((a->page_bytes + kCopyPart - 1) / kCopyPart);
    const int64_t ctas = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    e = launch_after(copy_pages_kernel, dim3((unsigned)(ctas < 608 ? ctas : 608)), dim3(kCopyThreads), 0, s, *a);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_cache_resize");
}

extern "C" int spec_cache_fork(const int32_t* src, const int32_t* dst, int32_t n, int32_t B, int32_t page_size,
                               int32_t num_pages, int32_t max_pages, int32_t* page_table, int32_t* held, int32_t* length,
                               int32_t* ref_count, int32_t* status, void* stream) {
    clear_error();
    if (n < 0 || n > SPEC_MAX_STREAMS || B < 0 || B > SPEC_MAX_STREAMS)
        return set_error(SPEC_ERR_SHAPE, "spec_cache_fork: n = %d, B = %d", n, B);
    if (!page_ok(page_size) || num_pages < 1 || max_pages < 1 || !table_ok(max_pages, page_size))
        return set_error(SPEC_ERR_SHAPE, "spec_cache_fork: page_size = %d, num_pages = %d, max_pages = %d", page_size,
                         num_pages, max_pages);
    if (n == 0) return SPEC_OK;
    if (src == nullptr || dst == nullptr || page_table == nullptr || held == nullptr || length == nullptr ||
        ref_count == nullptr || status == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_cache_fork: a required pointer is NULL");
    const cudaError_t e = launch_after(fork_kernel, dim3((unsigned)n), dim3(kForkThreads), 0, static_cast<cudaStream_t>(stream), src, dst, n, B,
                                       page_size, num_pages, max_pages, page_table, held, length, ref_count, status);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_cache_fork");
}
