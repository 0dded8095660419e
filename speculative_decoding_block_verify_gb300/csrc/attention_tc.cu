// spec_paged_attention on the tensor cores: bf16 caches.
//
// One key tile of an item (attention.cuh) is two matrix products around a softmax step,
//   S [rows x 64] = Q [rows x D] K^T,   P = 2^(scale S - m),   O [rows x D] += P V,
// with up to 128 rows (the tokens of a block times the query heads of a key head), which is the M of one
// tcgen05.mma: the block's few rows leave most of it empty, but at 64 positions a tile takes 32 KB from
// memory (about 1,400 cycles of an SM's share of the measured copy bandwidth) and the two products at M
// = 128 about 640 (8 of 48 cycles, which is what their operands take from shared memory, and 4 of 64 with P in
// tensor memory), so the tensor cores wait for memory whatever the number of rows is.
//
// A CTA has seven warps in four roles.  Warp 7 copies: the pages of K and V by TMA, 128-byte swizzled, into
// a ring of 64-position slots, and the rows of Q once per item.  Warps 5 and 6 issue the products.  Warps 0 to 3
// hold one row per thread (TMEM lane = row): they read S, keep the row's maximum and sum, write P as bf16
// over S, and scale O when the maximum has risen by more than 8 (2^8 of headroom is nothing to float32, and
// most tiles then leave O alone).  S is double-buffered, so the product of the next tile runs during the
// softmax of this one.  Two such CTAs share an SM (256 TMEM columns and half the shared memory each): the
// start and the end of an item in one overlap with the tiles of the other.
// Warps go to the quarters of an SM by their number, and a quarter's warps share what fetches their instructions.  With few rows
// the softmax's warps 2 and 3 have none: copies beside warp 3 instead of beside warp 0 (as warp 4, which is idle now)
// bring heads of 64 from 59.2 to 56.1 us for 64 streams, of 80 from 75.2 to 70.5, and no shape loses.

#include <cudaTypedefs.h>

#include <atomic>

#include "host_util.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace sv {

constexpr int kTcThreads = 256;
constexpr int kQPlace = kTcRows / 2 * 128;   // bytes to Q's second place: up to 64 rows, the next item's rows fit behind

// DP: the head padded to 64, 128 or 256 columns (TMA fills the rest with zeros).
template <int DP>
struct TcLayout {
    static constexpr int kHalves = DP / 64;                    // 64-column panels (128 bytes a row)
    static constexpr int kQBytes = kHalves * kTcRows * 128;
    static constexpr int kSlotBytes = kHalves * kTile * 128;   // K or V of one tile
    static constexpr int kSlots = DP == 64 ? 10 : DP == 128 ? 5 : 4;
    static constexpr int kCtasPerSm = DP == 256 ? 1 : 2;
    static constexpr int kTmemCols = DP == 256 ? 512 : 256;
    static constexpr int kOCol = 2 * kTile;                    // O after the two S buffers
    static constexpr int kBytes = kQBytes + kSlots * kSlotBytes;
};

struct TcShared {
    uint64_t q_full[2], q_empty[2], o_done[2], drain[2];
    uint64_t full[10], empty[10];
    uint64_t s_full[2], p_full[2];
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    Start start;
    int64_t scan[kTcThreads / 32];
    int scratch;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int rg, int z, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %2, %2, %3, %4}], "
        "[%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(rg), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// How a slot of the ring is laid out: 8-row groups and 64-column panels, in bytes.  A head of whole panels comes with
// one copy per page, [group][panel][8 rows][128 bytes]; any other width panel by panel (columns past the
// head read as zeros), [panel][64 rows][128 bytes].
template <int DP>
struct SlotLayout {
    uint32_t group, panel;
    __device__ __forceinline__ explicit SlotLayout(const AttnParams& p) {
        const bool pages = p.a.D == DP;
        group = pages ? DP / 64 * 1024 : 1024;
        panel = pages ? 1024 : kTile * 128;
    }
};

// ---- warp 7: the walk over the CTA's items, and the copies --------------------------------
template <int DP>
__device__ __forceinline__ void copy_role(const AttnParams& p, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const int lane = threadIdx.x & 31;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kQBytes;
    const int box = min(p.a.page_size, kTile);   // positions of a page's copy
    const int pages = kTile / box;
    const int q_places = p.rows <= kTcRows / 2 ? 2 : 1;
    const bool by_page = p.a.D == DP;
    // Keys and values that are read once leave L2 first: otherwise they push out the kernel's own code, the tables
    // and the parts, and every one of those is then a miss to memory (the 64-stream verify step: 124 us instead of
    // 98).  A block of several groups reads them again.
    const uint64_t stay = l2_evict_normal_policy();
    const uint64_t once = (p.a.kmax + 1) * p.G <= p.rows ? l2_evict_first_policy() : stay;
    Walk w = {};
    int told = 0, items = 0, slot = 0;
    unsigned phase = 1;   // a fresh barrier: the phase before its first is done
    bool ok = true;
    auto tell = [&](bool any) {   // the next segment, or that there is none
        Segment& seg = sh.seg[told % kSegments];
        ok = ok && warp_wait_for(&sh.seg_empty[told % kSegments], ((told / kSegments) & 1) ^ 1, &sh.abort);
        if (ok && lane == 0) {
            if (any) {
                seg = segment_of(p, w, blockIdx.x);
                if (w.begins_part()) p.desc[blockIdx.x] = w.unjoined(p, blockIdx.x, sh.start.span);
            } else {
                seg.t0 = seg.t1 = 0;
            }
            mbar_arrive(&sh.seg_full[told % kSegments]);
        }
        ++told;
    };
    // One load of the warp looks up the pages of several tiles: lane i has page i % pages of tile t + i / pages, as the map's last
    // coordinate (past the last page: zeros).  The next tiles' load is on its way while these are copied.
    const int per = 32 / pages;
    int z_now = 0, z_next = 0, z_base = 0;
    auto look_up = [&](int t) {
        const int tile = t + lane / pages;
        const int j = tile_start_past(w.it, tile) + (lane % pages) * box;
        int page = -1;
        if (tile < w.t1 && j < w.it.high && (j > w.it.low - box || j < w.it.sink))
            page = p.a.page_table[(int64_t)w.b * p.a.max_pages + (j >> p.page_shift)];
        return (unsigned)page < (unsigned)p.a.num_pages ? page * p.a.Hkv + w.h : p.a.num_pages * p.a.Hkv;
    };
    auto begin_look_up = [&](int t) {
        z_base = t;
        z_now = look_up(t);
        z_next = t + per < w.t1 ? look_up(t + per) : 0;
    };
    auto pages_of = [&](int t) {
        if (t - z_base == per) {
            z_base = t;
            z_now = z_next;
            if (t + per < w.t1) z_next = look_up(t + per);
        }
        return __shfl_sync(0xffffffffu, z_now, (t - z_base) * pages + lane % pages);
    };
    auto copy = [&](const CUtensorMap* map, int z, int y) {   // one tile of K or V into the next slot
        ok = ok && warp_wait_for(&sh.empty[slot], phase, &sh.abort);
        if (!ok) return;
        const uint32_t to = ring + slot * Lay::kSlotBytes;
        if (lane == 0) mbar_expect_tx(&sh.full[slot], Lay::kSlotBytes);
        __syncwarp();
        if (by_page) {   // a lane per page
            if (lane < pages) tma_load_5d(to + lane * box * Lay::kHalves * 128, map, y >> 3, z, &sh.full[slot], once);
        } else if (lane < pages) {
            for (int half = 0; half < Lay::kHalves; ++half)
                tma_load_3d(to + half * (kTile * 128) + lane * box * 128, map, half * 64, y, z, &sh.full[slot], once);
        }
        if (++slot == Lay::kSlots) {
            slot = 0;
            phase ^= 1;
        }
    };
    bool more = w.start(p, sh.start);
    tell(more);
    int t = more ? w.t0 : 0;
    if (more) begin_look_up(t);
    while (more && ok) {
        const int z = pages_of(t);
        const int y = pages > 1 ? 0 : tile_start(w.it, t) & (p.a.page_size - 1);
        copy(kmap, z, y);
        if (t == w.t0 && ok) {
            // the item's rows of Q, behind its first keys: they wait for the last user of their place
            const int at = items % q_places;
            ok = warp_wait_for(&sh.q_empty[at], ((items / q_places) & 1) ^ 1, &sh.abort);
            if (ok && lane == 0) {
                const int row = (int)first_row(p.a.cu_drafts, w.b, p.a.kmax) + p.by_G.of(w.it.r0);
                mbar_expect_tx(&sh.q_full[at], Lay::kHalves * p.rows * 128);
                for (int half = 0; half < Lay::kHalves; ++half)
                    tma_load_3d(q_at + half * (kTcRows * 128) + at * kQPlace, qmap, half * 64, w.h * p.G, row, &sh.q_full[at], stay);
            }
            ++items;
        }
        // the next item and its first pages, before the last values' slot is waited for
        if (++t == w.t1) {
            more = w.next(p);
            tell(more);
            t = w.t0;
            if (more) begin_look_up(t);
        }
        copy(vmap, z, y);
    }
    if (!ok) {   // gave up: whatever was copied must have arrived before the CTA's memory is given back
        for (int s = 0; s < Lay::kSlots; ++s)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
        for (int i = max(0, items - q_places); i < items; ++i)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.q_full[i % q_places], (i / q_places) & 1); ++n) {}
    }
}

// ---- warps 5 and 6: products -----------------------------------------------------------------
// Warp 5: S of tile n (its keys, the item's Q, and P of tile n - 2, whose place S takes, used up); warp 6: O += P V (P, and the
// tile's values).  A whole warp runs each loop, so that descriptors and addresses are uniform; one lane issues.  One warp that
// looked for either product's operands in turn noticed them later where the softmax is what takes the time (16 streams of 33
// tokens 51.6 us against 49.4, heads of 256 183 against 179, short streams 20.6 against 20.0).
// P beside S instead of over it, so that S need not wait for the product two tiles back, cost 7% (heads of 64).
template <int DP>
__device__ __forceinline__ bool keys_role(const AttnParams& p, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const SlotLayout<DP> lay(p);
    const uint32_t group = lay.group >> 4, panel = lay.panel >> 4;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kQBytes;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    const int ksteps = (p.a.D + 15) / 16;
    const int q_places = p.rows <= kTcRows / 2 ? 2 : 1;
    // a negative scale is a negated Q (bit 13) and its magnitude
    const uint32_t qk = mma_desc(kTile, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    int slot = 0;
    unsigned phase = 0, n = 0;
    for (int item = 0;; ++item) {
        const int at = item % kSegments;
        if (!warp_wait_for(&sh.seg_full[at], (item / kSegments) & 1, &sh.abort)) return false;
        int left = __reduce_max_sync(0xffffffffu, sh.seg[at].t1 - sh.seg[at].t0);
        if (elected()) mbar_arrive(&sh.seg_empty[at]);
        __syncwarp();
        if (left == 0) return true;
        const int q = item % q_places;
        if (!warp_wait_for(&sh.q_full[q], (item / q_places) & 1, &sh.abort)) return false;
        const uint32_t a = desc_lo(q_at + q * kQPlace, 1);
        for (; left > 0; --left, ++n) {
            const unsigned buf = n & 1;
            if (!warp_wait_for(&sh.full[slot], phase, &sh.abort)) return false;
            if (n >= 2 && !warp_wait_for(&sh.o_done[buf], ((n >> 1) - 1) & 1, &sh.abort)) return false;
            tc_fence_after();
            const uint32_t b = desc_lo(ring + slot * Lay::kSlotBytes, 1);
            if (elected()) {
#pragma unroll
                for (int k = 0; k < Lay::kHalves * 4; ++k)
                    if (k < ksteps)
                        mma_ss(tmem + buf * kTile, desc(a + (k >> 2) * (kTcRows * 128 >> 4) + (k & 3) * 2, 1024 >> 4),
                               desc(b + (k >> 2) * panel + (k & 3) * 2, group), qk, k > 0);
                mma_commit(&sh.s_full[buf]);
                mma_commit(&sh.empty[slot]);
                if (left == 1) mma_commit(&sh.q_empty[q]);
            }
            __syncwarp();
            slot += 2;
            if (slot >= Lay::kSlots) {
                slot -= Lay::kSlots;
                phase ^= 1;
            }
        }
    }
}
template <int DP>
__device__ __forceinline__ bool values_role(const AttnParams& p, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const SlotLayout<DP> lay(p);
    const uint32_t group = lay.group >> 4, panel = lay.panel >> 4;
    const uint32_t ring = smem_u32(smem) + Lay::kQBytes;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    constexpr uint32_t pv = mma_desc(DP, true);
    int slot = 1;
    unsigned phase = 0, n = 0;
    for (int item = 0;; ++item) {
        const int at = item % kSegments;
        if (!warp_wait_for(&sh.seg_full[at], (item / kSegments) & 1, &sh.abort)) return false;
        const Segment w = sh.seg[at];
        const int tiles = __reduce_max_sync(0xffffffffu, w.t1 - w.t0);
        if (elected()) mbar_arrive(&sh.seg_empty[at]);
        __syncwarp();
        if (tiles == 0) return true;
        for (int t = 0; t < tiles; ++t, ++n) {
            const unsigned buf = n & 1;
            if (!warp_wait_for(&sh.full[slot], phase, &sh.abort)) return false;
            const int j0 = w.start(w.t0 + t);
            const int from = min(kTile, w.high - j0), low = min(kTile, max(0, w.low - j0)), sink = max(0, w.sink - j0);
            if (from < kTile || sink < low) {
                // values of positions that no row of the item sees: zeros, whatever the cache holds there
                char* const to = smem + Lay::kQBytes + slot * Lay::kSlotBytes;
                constexpr int kChunks = Lay::kHalves * 8;   // 16 bytes each, of a row
                for (int u = threadIdx.x & 31; u < kTile * kChunks; u += 32) {
                    const int row = u / kChunks, c = u % kChunks;
                    if (row >= from || (row >= sink && row < low))
                        *reinterpret_cast<uint4*>(to + (row >> 3) * lay.group + (c >> 3) * lay.panel + (row & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (!warp_wait_for(&sh.p_full[buf], (n >> 1) & 1, &sh.abort)) return false;
            tc_fence_after();
            const uint32_t v = desc_lo(ring + slot * Lay::kSlotBytes, panel);
            if (elected()) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_ts(tmem + Lay::kOCol, tmem + buf * kTile + k * 8, desc(v + 2 * k * group, group), pv, t > 0 || k > 0);
                mma_commit(&sh.o_done[buf]);
                mma_commit(&sh.empty[slot]);
            }
            __syncwarp();
            slot += 2;
            if (slot >= Lay::kSlots) {
                slot -= Lay::kSlots;
                phase ^= 1;
            }
        }
    }
}

// ---- warps 0 to 3: softmax, scaling, output ---------------------------------------------
template <int DP>
__device__ __forceinline__ void softmax_role(const AttnParams& p, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    const bool wide = (((uint32_t)reinterpret_cast<uintptr_t>(p.a.out) | p.a.D * 2) & 31) == 0;   // 32-byte stores
    unsigned t_all = 0;   // tiles of the CTA so far
    bool ok = true;
    for (int n_seg = 0;; ++n_seg) {
        const int seg_at = n_seg % kSegments;
        ok = warp_wait_for(&sh.seg_full[seg_at], (n_seg / kSegments) & 1, &sh.abort);
        if (!ok) break;
        const Segment w = sh.seg[seg_at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[seg_at]);
        if (w.t0 == w.t1) break;
        const int rows = w.rows;
        const int rr = w.r0 + min(tid, rows - 1), token = p.by_G.of(rr);
        const int at = w.len + token;                                        // the row's position
        const int low = p.a.window > 0 ? at + 1 - p.a.window : 0;            // ... sees [low, at] and [0, sinks)
        const int at_first = w.len + p.by_G.of(w.r0), at_last = w.len + p.by_G.of(w.r0 + rows - 1);
        const bool work = warp * 32 < rows;                                  // any row in this warp
        const bool mine = tid < rows;
        unsigned short* const to = reinterpret_cast<unsigned short*>(p.a.out) +
                                   ((w.row0 + token) * p.a.Hq + w.head * p.G + rr - token * p.G) * (int64_t)p.a.D;
        float4* const part = p.part + (int64_t)w.slot * (p.a.D / 4) * p.rows + tid;
        float m = -kInf, l = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++t_all) {
            const unsigned buf = t_all & 1;
            const int j0 = w.start(t);
            ok = warp_wait_for(&sh.s_full[buf], (t_all >> 1) & 1, &sh.abort);
            if (!ok) break;
            float scale_o = 1.f;
            if (work) {
                tc_fence_after();
                uint32_t s[kTile];
                tmem_ld32(lanes + buf * kTile, s);
                tmem_ld32(lanes + buf * kTile + 32, s + 32);
                tc_wait_ld();
                // a tile that every row sees whole needs no mask
                const bool clean = j0 + kTile - 1 <= at_first &&
                                   (p.a.window <= 0 || j0 > at_last - p.a.window || j0 + kTile <= p.a.sinks);
                if (!clean) {
                    const int hi = at - j0, lo = low - j0, sk = p.a.sinks - j0;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!(c <= hi && (c >= lo || c < sk))) s[c] = 0xff800000u;
                }
                float x[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
                for (int c = 0; c < kTile; c += 2)   // three-way maxima
                    x[(c >> 1) & 3] = fmaxf(fmaxf(x[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;   // the scale is positive here
                if (mine && top > m + 8.f) {   // lanes without a row never ask for the scaling of O
                    scale_o = m == -kInf ? 0.f : ex2(m - top);
                    m = top;
                    l *= scale_o;
                }
                const float base = m == -kInf ? 0.f : m;
                const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[kTile / 2];
#pragma unroll
                for (int c = 0; c < kTile; c += 2) {
                    const float2 y = ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, nb);
                    // P V takes both operands in one type, so the weights are rounded to bf16, and the sum takes them as rounded.  On
                    // random values that moves an output by 1.2e-3 of it (2-norm), below the 1.7e-3 of its own rounding (64 streams of
                    // 200 to 8,000 tokens: 2.0e-3 off together); a second bf16 for what is left would double the product.
                    pk[c / 2] = pack_bf16(ex2(y.x), ex2(y.y));
                    sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], make_float2(bf16_lo(pk[c / 2]), bf16_hi(pk[c / 2])));
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                __syncwarp();
                tmem_st32(lanes + buf * kTile, pk);
            }
            if (work) {
                if (t > w.t0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
                    // the product before has to be done before O is scaled.  (Looked for only here and at the item's end: S of
                    // this tile was issued behind the product two tiles back, so the barrier is at most one phase ahead.)
                    ok = warp_wait_for(&sh.o_done[buf ^ 1], ((t_all - 1) >> 1) & 1, &sh.abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(lanes + Lay::kOCol + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale_o);
                        tmem_st32(lanes + Lay::kOCol + c, o);
                    }
                }
                tc_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[buf]);
        }
        ok = ok && warp_wait_for(&sh.o_done[(t_all - 1) & 1], ((t_all - 1) >> 1) & 1, &sh.abort);
        if (!ok) break;
        if (work) {
            tc_fence_after();
            const float inv = 1.f / l;
            if (mine && !w.whole) __stcg(p.ml + (int64_t)w.slot * p.rows + tid, make_float2(m, l));
#pragma unroll 1
            for (int c0 = 0; c0 < p.a.D; c0 += 64) {
                uint32_t o[64];
                __syncwarp();
                tmem_ld32(lanes + Lay::kOCol + c0, o);
                tmem_ld32(lanes + Lay::kOCol + c0 + 32, o + 32);
                tc_wait_ld();
                if (mine && w.whole) {
                    uint32_t x[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        x[c / 2] = pack_bf16(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv);
#pragma unroll
                    for (int c = 0; c < 64; c += 16) {
                        if (wide && c0 + c < p.a.D) {
                            store32(to + c0 + c, x + c / 2);
                        } else {
                            if (c0 + c < p.a.D)
                                *reinterpret_cast<uint4*>(to + c0 + c) = make_uint4(x[c / 2], x[c / 2 + 1], x[c / 2 + 2], x[c / 2 + 3]);
                            if (c0 + c + 8 < p.a.D)
                                *reinterpret_cast<uint4*>(to + c0 + c + 8) = make_uint4(x[c / 2 + 4], x[c / 2 + 5], x[c / 2 + 6], x[c / 2 + 7]);
                        }
                    }
                } else if (mine) {   // neighbouring rows are neighbours in memory
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        if (c0 + c >= p.a.D) break;
                        __stcg(part + (c0 + c) / 4 * p.rows,
                               make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]),
                                           __uint_as_float(o[c + 3])));
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(kTcThreads, TcLayout<DP>::kCtasPerSm)
    attention_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    using Lay = TcLayout<DP>;
    extern __shared__ __align__(1024) char smem[];
    TcShared& sh = *reinterpret_cast<TcShared*>(smem + Lay::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int cta = blockIdx.x;
    if (warp == 4 && (tid & 31) < 3) {
        const CUtensorMap* map = (tid & 31) == 0 ? &kmap : (tid & 31) == 1 ? &vmap : &qmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"((uint32_t)Lay::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        for (int i = 0; i < Lay::kSlots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], 6);   // softmax 4, products 2
        }
        mbar_init_fence();
        sh.abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join, which waits for the whole grid
    if (tid == 0) p.desc[cta].rows = 0;
    find_start<kTcThreads>(p, cta, &sh.start, sh.scan, &sh.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 7) {
        copy_role<DP>(p, &qmap, &kmap, &vmap, smem, sh);
        write_status<unsigned short>(p, cta, sh.start.valid);   // while the last tiles are computed
    } else if (warp == 5) {
        if (!keys_role<DP>(p, smem, sh)) drain(&sh.drain[0]);
    } else if (warp == 6) {
        if (!values_role<DP>(p, smem, sh)) drain(&sh.drain[1]);
    } else if (warp < 4) {
        softmax_role<DP>(p, sh);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"((uint32_t)Lay::kTmemCols));
    }
    if (tid == 0 && sh.abort) write_timeout(p);
}

// ---------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------
static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
    const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
    return f != nullptr && f(map, type, rank, const_cast<void*>(base), dims, strides, box, elem,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, rank, dims, strides, box);
}

// Rows of Q: [rows][Hq][D] as boxes of 64 columns, a key head's query heads, a group's tokens.
static bool encode_q(CUtensorMap* map, const void* base, const AttnParams& p, uint64_t stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)p.a.D, (cuuint64_t)p.a.Hq, (cuuint64_t)(p.a.q_rows > 0 ? p.a.q_rows : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)p.a.D * 2, stride};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(p.rows / p.G)};
    return encode(map, base, 3, dims, strides, box);
}

// A layer's pages: [page and head][position][D].  A head of whole 64-column panels as [page and head][position / 8][panel]
// [position % 8][64], a page (or 64 positions of one) a box; any other width in boxes of 64 columns.
static bool encode_pages(CUtensorMap* map, const void* base, const AttnParams& p) {
    const cuuint64_t D = p.a.D, P = p.a.page_size, heads = (cuuint64_t)p.a.num_pages * p.a.Hkv;
    const cuuint32_t positions = p.a.page_size < kTile ? p.a.page_size : kTile;
    if (D % 64 == 0 && D != 192) {
        const cuuint64_t dims[5] = {64, 8, D / 64, P / 8, heads}, strides[4] = {D * 2, 128, 8 * D * 2, P * D * 2};
        const cuuint32_t box[5] = {64, 8, (cuuint32_t)(D / 64), positions / 8, 1};
        return encode(map, base, 5, dims, strides, box);
    }
    const cuuint64_t dims[3] = {D, P, heads}, strides[2] = {D * 2, P * D * 2};
    const cuuint32_t box[3] = {64, positions, 1};
    return encode(map, base, 3, dims, strides, box);
}

template <int DP>
struct TcReady {
    static std::atomic<int> on[64];
};
template <int DP>
std::atomic<int> TcReady<DP>::on[64];

template <int DP>
static cudaError_t launch_tc(const AttnParams& p, const CUtensorMap (&map)[3], cudaStream_t s) {
    using Lay = TcLayout<DP>;
    constexpr int bytes = Lay::kBytes + (int)sizeof(TcShared);
    static_assert(bytes <= (Lay::kCtasPerSm == 2 ? 115712 : 232448), "shared memory of an SM");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !TcReady<DP>::on[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(attention_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) TcReady<DP>::on[dev].store(1, std::memory_order_release);
    }
    return launch_after(attention_tc_kernel<DP>, dim3(p.ctas), dim3(kTcThreads), bytes, s, p, map[0], map[1], map[2]);
}

bool tensor_q(const spec_attention_args* a) { return (((uintptr_t)a->q | (uintptr_t)(a->q_row_stride * 2)) & 15) == 0; }

// Rows of Q that do not lie on 16-byte boundaries, packed so that they do.
__global__ void __launch_bounds__(256) pack_rows_kernel(const unsigned short* q, int64_t stride, int width, uint4* to) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned short* from = q + blockIdx.x * stride;
    for (int c = threadIdx.x; c < width / 8; c += 256) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = from[8 * c + 2 * i] | (uint32_t)from[8 * c + 2 * i + 1] << 16;
        to[(int64_t)blockIdx.x * (width / 8) + c] = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

int tensor_rows(const spec_attention_args* a) {
    const int G = a->Hq / a->Hkv, most = kTcRows / G, tokens = a->kmax + 1;
    const int groups = (tokens + most - 1) / most;
    return (tokens + groups - 1) / groups * G;
}

int tensor_ctas_per_sm(const spec_attention_args* a) { return a->D > 128 ? 1 : 2; }

cudaError_t launch_attention_tc(const AttnParams& p, void* q_packed, cudaStream_t s) {
    const spec_attention_args& a = p.a;
    const void* q = a.q;
    uint64_t q_stride = (uint64_t)a.q_row_stride * 2;
    if (q_packed != nullptr && a.q_rows > 0) {
        const cudaError_t e = launch_after(pack_rows_kernel, dim3((unsigned)a.q_rows), dim3(256), 0, s,
                                           static_cast<const unsigned short*>(q), a.q_row_stride, a.Hq * a.D, static_cast<uint4*>(q_packed));
        if (e != cudaSuccess) return e;
        q = q_packed;
        q_stride = (uint64_t)a.Hq * a.D * 2;
    }
    CUtensorMap map[3];
    if (!encode_q(&map[0], q, p, q_stride) || !encode_pages(&map[1], a.k_pages, p) || !encode_pages(&map[2], a.v_pages, p))
        return cudaErrorInvalidValue;
    if (a.D <= 64) return launch_tc<64>(p, map, s);
    if (a.D <= 128) return launch_tc<128>(p, map, s);
    return launch_tc<256>(p, map, s);
}

}  // namespace sv
