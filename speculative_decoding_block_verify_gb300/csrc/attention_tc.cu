// spec_paged_attention on the tensor cores: bf16 caches.
//
// One key tile of an item (attention.cuh) is two matrix products around a softmax step,
//   S [rows x 64] = Q [rows x D] K^T,   P = 2^(scale S - m),   O [rows x D] += P V,
// with up to 128 rows (the tokens of a block times the query heads of a key head), which is the M of one
// tcgen05.mma: the block's few rows leave most of it empty, but at 64 positions a tile takes 32 KB from
// memory (about 1,400 cycles of an SM's share of the measured copy bandwidth) and the two products at M
// = 128 about 512, so the tensor cores wait for memory whatever the number of rows is.
//
// A CTA has six warps in three roles.  Warp 4 copies: the pages of K and V by TMA, 128-byte swizzled, into
// a ring of 64-position slots, and the rows of Q once per item.  Warp 5 issues the products.  Warps 0 to 3
// hold one row per thread (TMEM lane = row): they read S, keep the row's maximum and sum, write P as bf16
// over S, and scale O when the maximum has risen by more than 8 (2^8 of headroom is nothing to float32, and
// most tiles then leave O alone).  S is double-buffered, so the product of the next tile runs during the
// softmax of this one.  Two such CTAs share an SM (256 TMEM columns and half the shared memory each): the
// start and the end of an item in one overlap with the tiles of the other.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "attention.cuh"
#include "host_util.h"

namespace sv {

constexpr int kTcThreads = 192;
constexpr int kTcRows = 128;           // M of the products
constexpr int kTcSpinLimit = 1 << 20;  // polls before a wait gives up

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
    uint64_t q_full, q_empty, o_done, drain;
    uint64_t full[10], empty[10];
    uint64_t s_full[2], p_full[2];
    Start start;
    int64_t scan[kTcThreads / 32];
    int scratch;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for the phase; false when the wait (or another one of the CTA) gave up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity, int* abort) {
    for (int n = 0; !mbar_try_wait(bar, parity); ++n) {
        if (n > kTcSpinLimit) *reinterpret_cast<volatile int*>(abort) = 1;
        if (*reinterpret_cast<volatile int*>(abort)) return false;
    }
    return true;
}
__device__ __forceinline__ bool warp_wait_for(uint64_t* bar, unsigned parity, int* abort) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

// Shared-memory matrix descriptors, 128-byte swizzle: start and strides in units of 16 bytes.
// K-major (Q, K): 8 rows of 128 bytes are 1,024 bytes, rows 8 further on begin there.  MN-major (V, whose
// rows are the product's K): `lead` bytes from one 64-column panel to the next.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// kind::f16: float32 accumulator, bf16 operands, M = 128; `mn` = the B operand is MN-major
constexpr uint32_t mma_desc(int n, bool mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kTcRows >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define SV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define SV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SV_W8(r, 0),
        SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24), "r"(addr)
        : "memory");
}
#undef SV_R8
#undef SV_W8

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---- warp 4: copies -------------------------------------------------------------------
template <int DP>
__device__ __forceinline__ void copy_role(const AttnParams& p, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const int lane = threadIdx.x & 31;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kQBytes;
    Walk w;
    if (!w.start(p, sh.start)) return;
    // a lane's share of a tile: one page (or the tile's part of it) and one 64-column panel at a time
    const int box = min(p.a.page_size, kTile);          // positions of a copy
    const int pages = kTile / box;                       // copies of a panel
    int slot = 0;
    unsigned phase = 1;                                  // a fresh barrier: the phase before its first is done
    int items = 0;
    bool ok = true;
    do {
        const int32_t* table = p.a.page_table + (int64_t)w.b * p.a.max_pages;
        const int64_t row0 = first_row(p.a.cu_drafts, w.b, p.a.kmax);
        int next_z = 0;
        auto look_up = [&](int t) {   // the lane's page of tile t, as the map's third coordinate
            const int j = tile_start(w.it, t) + (lane % pages) * box;
            const int end = j + box;
            int page = -1;
            if (j < w.it.high && (end > w.it.low || j < w.it.sink)) page = __ldg(table + (j >> p.page_shift));
            // past the last page: zeros
            next_z = (unsigned)page < (unsigned)p.a.num_pages ? page * p.a.Hkv + w.h : p.a.num_pages * p.a.Hkv;
        };
        look_up(w.t0);
        for (int t = w.t0; t < w.t1 && ok; ++t) {
            const int z = next_z;
            const int y = tile_start(w.it, t) & (p.a.page_size - 1) & ~(box - 1);
            if (t + 1 < w.t1) look_up(t + 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                ok = warp_wait_for(&sh.empty[slot], phase, &sh.abort);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(&sh.full[slot], Lay::kSlotBytes);
                __syncwarp();
                const uint32_t to = ring + slot * Lay::kSlotBytes;
                for (int u = lane; u < pages * Lay::kHalves; u += 32) {
                    const int half = u / pages;   // u % pages = lane % pages: 32 is a multiple of pages
                    tma_load_3d(to + half * (kTile * 128) + (lane % pages) * box * 128, kv ? vmap : kmap, half * 64,
                                pages > 1 ? 0 : y, z, &sh.full[slot]);
                }
                if (++slot == Lay::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (t == w.t0 && ok) {
                // the item's rows of Q, behind its first keys: they wait for the item before to be through with its own
                ok = warp_wait_for(&sh.q_empty, (items & 1) ^ 1, &sh.abort);
                if (ok && lane == 0) {
                    const int tokens = p.rows / p.G;
                    mbar_expect_tx(&sh.q_full, Lay::kHalves * tokens * p.G * 128);
                    for (int half = 0; half < Lay::kHalves; ++half)
                        tma_load_3d(q_at + half * (kTcRows * 128), qmap, half * 64, w.h * p.G, (int)row0 + w.it.r0 / p.G,
                                    &sh.q_full);
                }
                ++items;
            }
        }
    } while (ok && w.next(p));
    if (!ok) {   // gave up: whatever was copied must have arrived before the CTA's memory is given back
        for (int s = 0; s < Lay::kSlots; ++s)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
        for (int n = 0; n < kTcSpinLimit / 64 && items > 0 && !mbar_try_wait(&sh.q_full, (items - 1) & 1); ++n) {}
    }
}

// ---- warp 5, one thread: products ------------------------------------------------------
template <int DP>
__device__ __forceinline__ void mma_role(const AttnParams& p, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kQBytes;
    const uint32_t tmem = sh.tmem;
    const int ksteps = (p.a.D + 15) / 16;
    // a negative scale is a negated Q (bit 13) and its magnitude
    const uint32_t qk = mma_desc(kTile, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t pv = mma_desc(DP, true);
    Walk w;   // of the tiles whose S product is issued: one tile ahead of the other product
    if (!w.start(p, sh.start)) return;
    int64_t total = min(sh.start.span, sh.start.total - sh.start.tile);
    int t_qk = w.t0;
    int items = 0;
    bool more = true, ok = true;
    int kslot = 0, vslot = 1;
    unsigned kphase = 0, vphase = 0;
    auto step = [](int& slot, unsigned& phase) {
        slot += 2;
        if (slot >= Lay::kSlots) {
            slot -= Lay::kSlots;
            phase ^= 1;
        }
    };
    unsigned firsts = 0;   // bit (tile & 1): the tile is the first of its item
    int64_t n_qk = 0;
    auto issue_qk = [&]() {
        const int buf = (int)(n_qk & 1);
        if (t_qk == w.t0) {
            ok = wait_for(&sh.q_full, items & 1, &sh.abort);
            firsts |= 1u << buf;
        } else {
            firsts &= ~(1u << buf);
        }
        ok = ok && wait_for(&sh.full[kslot], kphase, &sh.abort);
        if (!ok) return;
        tc_fence_after();
        const uint32_t k_at = ring + kslot * Lay::kSlotBytes;
        for (int k = 0; k < ksteps; ++k) {
            const int half = k >> 2, in = (k & 3) * 32;
            mma_ss(tmem + buf * kTile, smem_desc(q_at + half * (kTcRows * 128) + in, 16),
                   smem_desc(k_at + half * (kTile * 128) + in, 16), qk, k > 0);
        }
        mma_commit(&sh.s_full[buf]);
        mma_commit(&sh.empty[kslot]);
        step(kslot, kphase);
        ++n_qk;
        if (++t_qk == w.t1) {
            mma_commit(&sh.q_empty);
            ++items;
            more = w.next(p);
            t_qk = w.t0;
        }
    };
    issue_qk();
    for (int64_t t = 0; t < total && ok; ++t) {
        if (more) {
            // S of tile t + 1 goes where P of tile t - 1 was: that product has to be done
            if (t > 0) ok = wait_for(&sh.o_done, (unsigned)(t - 1) & 1, &sh.abort);
            if (ok) issue_qk();
        }
        const int buf = (int)(t & 1);
        ok = ok && wait_for(&sh.p_full[buf], (unsigned)(t >> 1) & 1, &sh.abort);
        ok = ok && wait_for(&sh.full[vslot], vphase, &sh.abort);
        if (!ok) break;
        tc_fence_after();
        const bool first = (firsts >> buf) & 1;
        const uint32_t v_at = ring + vslot * Lay::kSlotBytes;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + Lay::kOCol, tmem + buf * kTile + k * 8, smem_desc(v_at + k * 2048, kTile * 128), pv, !(first && k == 0));
        mma_commit(&sh.o_done);
        mma_commit(&sh.empty[vslot]);
        step(vslot, vphase);
    }
    if (!ok) {
        mma_commit(&sh.drain);
        for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.drain, 0); ++n) {}
    }
}

// ---- warps 0 to 3: softmax, scaling, output ---------------------------------------------
template <int DP>
__device__ __forceinline__ void softmax_role(const AttnParams& p, char* smem, TcShared& sh, int cta) {
    using Lay = TcLayout<DP>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    char* ring = smem + Lay::kQBytes;
    Walk w;
    if (!w.start(p, sh.start)) return;
    int64_t t_all = 0;   // tiles of the CTA so far
    int vslot = 1;
    unsigned vphase = 0;
    bool ok = true;
    do {
        const int rows = w.it.r1 - w.it.r0;
        const int token = (w.it.r0 + min(tid, rows - 1)) / p.G;
        const int at = w.len + token;                                        // the row's position
        const int low = p.a.window > 0 ? at + 1 - p.a.window : 0;            // ... sees [low, at] and [0, sinks)
        const int at_first = w.len + w.it.r0 / p.G;
        const bool work = warp * 32 < rows;                                  // any row in this warp
        float m = -kInf, l = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++t_all) {
            const int buf = (int)(t_all & 1);
            const int j0 = tile_start(w.it, t);
            ok = warp_wait_for(&sh.s_full[buf], (unsigned)(t_all >> 1) & 1, &sh.abort);
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
                                   (p.a.window <= 0 || j0 >= w.len + (w.it.r1 - 1) / p.G + 1 - p.a.window || j0 + kTile <= p.a.sinks);
                if (!clean) {
                    const int hi = at - j0, lo = low - j0, sk = p.a.sinks - j0;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!(c <= hi && (c >= lo || c < sk))) s[c] = 0xff800000u;
                }
                float x[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
                for (int c = 0; c < kTile; ++c) x[c & 3] = fmaxf(x[c & 3], __uint_as_float(s[c]));
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;   // the scale is positive here
                if (tid < rows && top > m + 8.f) {   // lanes without a row never ask for the scaling of O
                    scale_o = m == -kInf ? 0.f : ex2(m - top);
                    m = top;
                    l *= scale_o;
                }
                const float base = m == -kInf ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t pk[kTile / 2];
#pragma unroll
                for (int c = 0; c < kTile; c += 2) {
                    const float e0 = ex2(fmaf(__uint_as_float(s[c]), p.scale_log2, -base));
                    const float e1 = ex2(fmaf(__uint_as_float(s[c + 1]), p.scale_log2, -base));
                    pk[c / 2] = pack_bf16(e0, e1);
                    sum[c & 2] += bf16_lo(pk[c / 2]);
                    sum[(c & 2) + 1] += bf16_hi(pk[c / 2]);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                __syncwarp();
                tmem_st32(lanes + buf * kTile, pk);
            }
            // V of positions that no row of the item sees: zeros, whatever the cache holds there
            if (j0 + kTile > w.it.high || (j0 < w.it.low && j0 + kTile > w.it.sink)) {
                ok = warp_wait_for(&sh.full[vslot], vphase, &sh.abort);
                if (!ok) break;
                char* v = ring + vslot * Lay::kSlotBytes;
                for (int u = tid; u < Lay::kHalves * kTile * 8; u += 128) {
                    const int j = j0 + ((u >> 3) & (kTile - 1));
                    if (j >= w.it.high || (j < w.it.low && j >= w.it.sink))
                        *reinterpret_cast<uint4*>(v + u * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            vslot += 2;
            if (vslot >= Lay::kSlots) {
                vslot -= Lay::kSlots;
                vphase ^= 1;
            }
            if (t_all > 0) {   // the product before has to be done before O is scaled, or begun anew
                ok = warp_wait_for(&sh.o_done, (unsigned)(t_all - 1) & 1, &sh.abort);
                if (!ok) break;
            }
            if (work) {
                if (t > w.t0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
                    tc_fence_after();
#pragma unroll
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
        ok = ok && warp_wait_for(&sh.o_done, (unsigned)(t_all - 1) & 1, &sh.abort);
        if (!ok) break;
        const bool whole = w.whole();
        if (w.begins_part() && tid == 0) p.desc[cta] = make_int4(w.b, w.h, w.g, w.parts(cta, sh.start.span));
        if (work) {
            tc_fence_after();
            const bool mine = tid < rows;
            const int64_t part_row = (int64_t)w.slot(cta) * p.rows + tid;
            const int rr = w.it.r0 + tid;
            unsigned short* to = reinterpret_cast<unsigned short*>(p.a.out) +
                                 ((first_row(p.a.cu_drafts, w.b, p.a.kmax) + token) * p.a.Hq + w.h * p.G + rr - token * p.G) * (int64_t)p.a.D;
            const bool vec = (reinterpret_cast<uintptr_t>(p.a.out) & 15) == 0;
            const float inv = 1.f / l;
            if (mine && !whole) p.ml[part_row] = make_float2(m, l);
#pragma unroll
            for (int c0 = 0; c0 < DP; c0 += 32) {
                if (c0 >= p.a.D) break;
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lanes + Lay::kOCol + c0, o);
                tc_wait_ld();
                if (mine && whole) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        if (c0 + c >= p.a.D) break;
                        uint4 x;
                        x.x = pack_bf16(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv);
                        x.y = pack_bf16(__uint_as_float(o[c + 2]) * inv, __uint_as_float(o[c + 3]) * inv);
                        x.z = pack_bf16(__uint_as_float(o[c + 4]) * inv, __uint_as_float(o[c + 5]) * inv);
                        x.w = pack_bf16(__uint_as_float(o[c + 6]) * inv, __uint_as_float(o[c + 7]) * inv);
                        if (vec) {
                            *reinterpret_cast<uint4*>(to + c0 + c) = x;
                        } else {
                            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                            for (int i = 0; i < 8; ++i) to[c0 + c + i] = (unsigned short)(y[i / 2] >> (16 * (i & 1)));
                        }
                    }
                } else if (mine) {
                    float* q = p.part + part_row * p.a.D + c0;
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        if (c0 + c >= p.a.D) break;
                        *reinterpret_cast<uint4*>(q + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
        }
    } while (w.next(p));
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
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"((uint32_t)Lay::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < Lay::kSlots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
        }
        mbar_init_fence();
        sh.abort = 0;
        p.desc[cta] = make_int4(0, 0, 0, 0);
    }
    find_start<kTcThreads>(p, cta, &sh.start, sh.scan, &sh.scratch);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) {
        copy_role<DP>(p, &qmap, &kmap, &vmap, smem, sh);
    } else if (warp == 5) {
        if ((tid & 31) == 0) mma_role<DP>(p, smem, sh);
        __syncwarp();
    } else {
        softmax_role<DP>(p, smem, sh, cta);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"((uint32_t)Lay::kTmemCols));
    }
    if (tid == 0 && sh.abort) atomicOr(p.header, 1);
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

// [outer][middle][inner] of bf16 as boxes of 64 inner elements, 128-byte swizzled
static bool encode3(CUtensorMap* map, const void* base, uint64_t inner, uint64_t middle, uint64_t outer, uint64_t middle_stride,
                    uint64_t outer_stride, uint32_t box_middle, uint32_t box_outer) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {inner, middle, outer}, strides[2] = {middle_stride, outer_stride};
    const cuuint32_t box[3] = {64, box_middle, box_outer}, elem[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    attention_tc_kernel<DP><<<p.ctas, kTcThreads, bytes, s>>>(p, map[0], map[1], map[2]);
    return cudaGetLastError();
}

bool tensor_path(const spec_attention_args* a) {
    return a->dtype == SPEC_DTYPE_BF16 && a->scale != 0.f && a->Hq / a->Hkv <= kTcRows && (int64_t)a->num_pages * a->Hkv < INT32_MAX &&
           a->q_rows < INT32_MAX && (((uintptr_t)a->q | (uintptr_t)(a->q_row_stride * 2)) & 15) == 0 && encoder() != nullptr;
}

int tensor_rows(const spec_attention_args* a) {
    const int G = a->Hq / a->Hkv, most = kTcRows / G, tokens = a->kmax + 1;
    const int groups = (tokens + most - 1) / most;
    return (tokens + groups - 1) / groups * G;
}

int tensor_ctas_per_sm(const spec_attention_args* a) { return a->D > 128 ? 1 : 2; }

cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s) {
    const spec_attention_args& a = p.a;
    CUtensorMap map[3];
    const uint64_t D = a.D, P = a.page_size;
    const uint32_t box = a.page_size < kTile ? a.page_size : kTile;
    if (!encode3(&map[0], a.q, D, a.Hq, (uint64_t)a.q_rows, D * 2, (uint64_t)a.q_row_stride * 2, p.G, p.rows / p.G) ||
        !encode3(&map[1], a.k_pages, D, P, (uint64_t)a.num_pages * a.Hkv, D * 2, P * D * 2, box, 1) ||
        !encode3(&map[2], a.v_pages, D, P, (uint64_t)a.num_pages * a.Hkv, D * 2, P * D * 2, box, 1))
        return cudaErrorInvalidValue;
    if (a.D <= 64) return launch_tc<64>(p, map, s);
    if (a.D <= 128) return launch_tc<128>(p, map, s);
    return launch_tc<256>(p, map, s);
}

}  // namespace sv
