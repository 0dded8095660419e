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
constexpr int kQPlace = kTcRows / 2 * 128;   // bytes to Q's second place: up to 64 rows, the next item's rows fit behind
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
    uint64_t q_full[2], q_empty[2], o_done[2], drain;
    uint64_t full[10], empty[10];
    uint64_t s_full[2], p_full[2];
    Start start;
    int64_t scan[kTcThreads / 32];
    int scratch;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], "
        "%6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One look at the phase, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
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

// 32 bytes in one store
__device__ __forceinline__ void store32(void* to, const uint32_t* x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
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
    const int q_places = p.rows <= kTcRows / 2 ? 2 : 1;
    // Keys and values that are read once leave L2 first: otherwise they push out the kernel's own code, the tables
    // and the parts, and every one of those is then a miss to memory.  A block of several groups reads them again.
    const uint64_t stay = l2_evict_normal_policy();
    const uint64_t once = (p.a.kmax + 1) * p.G <= p.rows ? l2_evict_first_policy() : stay;
    bool ok = true;
    do {
        const int32_t* table = p.a.page_table + (int64_t)w.b * p.a.max_pages;
        const int64_t row0 = first_row(p.a.cu_drafts, w.b, p.a.kmax);
        int next_z = 0;
        auto look_up = [&](int t) {   // the lane's page of tile t, as the map's third coordinate
            const int j = tile_start(w.it, t) + (lane % pages) * box;
            const int end = j + box;
            int page = -1;
            if (j < w.it.high && (end > w.it.low || j < w.it.sink)) page = *(table + (j >> p.page_shift));
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
                                pages > 1 ? 0 : y, z, &sh.full[slot], once);
                }
                if (++slot == Lay::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (t == w.t0 && ok) {
                // the item's rows of Q, behind its first keys: they wait for the last user of their place
                const int at = items % q_places;
                ok = warp_wait_for(&sh.q_empty[at], ((items / q_places) & 1) ^ 1, &sh.abort);
                if (ok && lane == 0) {
                    mbar_expect_tx(&sh.q_full[at], Lay::kHalves * p.rows * 128);
                    for (int half = 0; half < Lay::kHalves; ++half)
                        tma_load_3d(q_at + half * (kTcRows * 128) + at * kQPlace, qmap, half * 64, w.h * p.G,
                                    (int)row0 + w.it.r0 / p.G, &sh.q_full[at], stay);
                }
                ++items;
            }
        }
    } while (ok && w.next(p));
    if (!ok) {   // gave up: whatever was copied must have arrived before the CTA's memory is given back
        for (int s = 0; s < Lay::kSlots; ++s)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
        for (int i = max(0, items - q_places); i < items; ++i)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.q_full[i % q_places], (i / q_places) & 1); ++n) {}
    }
}

// ---- warp 5, one thread: products ------------------------------------------------------
// Whichever product has its operands first: S of tile n (its keys, the item's Q, and P of tile n - 2, whose
// place S takes, used up) or O += P V of tile n (P, and the tile's values).
template <int DP>
__device__ __forceinline__ void mma_role(const AttnParams& p, char* smem, TcShared& sh) {
    using Lay = TcLayout<DP>;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kQBytes;
    const uint32_t tmem = sh.tmem;
    const int ksteps = (p.a.D + 15) / 16;
    const int q_places = p.rows <= kTcRows / 2 ? 2 : 1;
    // a negative scale is a negated Q (bit 13) and its magnitude
    const uint32_t qk = mma_desc(kTile, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t pv = mma_desc(DP, true);
    Walk w;   // of the S products
    if (!w.start(p, sh.start)) return;
    int t = w.t0, items = 0;
    bool more = true;
    unsigned n_qk = 0, n_pv = 0;   // products issued
    unsigned firsts = 0;           // bit (tile & 1): the tile is its item's first
    int kslot = 0, vslot = 1;
    unsigned kphase = 0, vphase = 0;
    auto step = [](int& slot, unsigned& phase) {
        slot += 2;
        if (slot >= Lay::kSlots) {
            slot -= Lay::kSlots;
            phase ^= 1;
        }
    };
    int spins = 0;
    while (more || n_pv != n_qk) {
        bool did = false;
        if (n_pv != n_qk) {
            const unsigned buf = n_pv & 1;
            if (mbar_test(&sh.p_full[buf], (n_pv >> 1) & 1) && mbar_test(&sh.full[vslot], vphase)) {
                tc_fence_after();
                const bool first = (firsts >> buf) & 1;
                const uint32_t v_at = ring + vslot * Lay::kSlotBytes;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_ts(tmem + Lay::kOCol, tmem + buf * kTile + k * 8, smem_desc(v_at + k * 2048, kTile * 128), pv,
                           !(first && k == 0));
                mma_commit(&sh.o_done[buf]);
                mma_commit(&sh.empty[vslot]);
                step(vslot, vphase);
                ++n_pv;
                did = true;
            }
        }
        if (more && n_qk - n_pv < 2) {
            const unsigned buf = n_qk & 1;
            const int q = items % q_places;
            if ((n_qk < 2 || mbar_test(&sh.o_done[buf], ((n_qk >> 1) - 1) & 1)) && mbar_test(&sh.full[kslot], kphase) &&
                (t != w.t0 || mbar_test(&sh.q_full[q], (items / q_places) & 1))) {
                tc_fence_after();
                firsts = (firsts & ~(1u << buf)) | (unsigned)(t == w.t0) << buf;
                const uint32_t k_at = ring + kslot * Lay::kSlotBytes;
                for (int k = 0; k < ksteps; ++k) {
                    const int half = k >> 2, in = (k & 3) * 32;
                    mma_ss(tmem + buf * kTile, smem_desc(q_at + half * (kTcRows * 128) + q * kQPlace + in, 16),
                           smem_desc(k_at + half * (kTile * 128) + in, 16), qk, k > 0);
                }
                mma_commit(&sh.s_full[buf]);
                mma_commit(&sh.empty[kslot]);
                step(kslot, kphase);
                ++n_qk;
                if (++t == w.t1) {
                    mma_commit(&sh.q_empty[q]);
                    ++items;
                    more = w.next(p);
                    t = w.t0;
                }
                did = true;
            }
        }
        spins = did ? 0 : spins + 1;
        if (spins > kTcSpinLimit) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
        if (spins > 0 && *reinterpret_cast<volatile int*>(&sh.abort)) {
            mma_commit(&sh.drain);
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.drain, 0); ++n) {}
            return;
        }
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
    unsigned t_all = 0;   // tiles of the CTA so far
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
            const unsigned buf = t_all & 1;
            const int j0 = tile_start(w.it, t);
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
                                   (p.a.window <= 0 || j0 >= w.len + (w.it.r1 - 1) / p.G + 1 - p.a.window || j0 + kTile <= p.a.sinks);
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
                if (tid < rows && top > m + 8.f) {   // lanes without a row never ask for the scaling of O
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
                    pk[c / 2] = pack_bf16(ex2(y.x), ex2(y.y));
                    sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], make_float2(bf16_lo(pk[c / 2]), bf16_hi(pk[c / 2])));
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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
                ok = warp_wait_for(&sh.o_done[buf ^ 1], ((t_all - 1) >> 1) & 1, &sh.abort);
                if (!ok) break;
            }
            if (work) {
                if (t > w.t0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
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
        const bool whole = w.whole();
        if (tid == 0 && w.begins_part()) p.desc[cta] = w.unjoined(p, cta, sh.start.span);
        if (work) {
            tc_fence_after();
            const bool mine = tid < rows;
            const int rr = w.it.r0 + tid;
            unsigned short* to = reinterpret_cast<unsigned short*>(p.a.out) +
                                 ((first_row(p.a.cu_drafts, w.b, p.a.kmax) + token) * p.a.Hq + w.h * p.G + rr - token * p.G) * (int64_t)p.a.D;
            const bool wide = (((uint32_t)reinterpret_cast<uintptr_t>(p.a.out) | p.a.D * 2) & 31) == 0;
            const int64_t slot = w.slot(cta);
            const float inv = 1.f / l;
            if (mine && !whole) __stcg(p.ml + slot * p.rows + tid, make_float2(m, l));
#pragma unroll 1
            for (int c0 = 0; c0 < p.a.D; c0 += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lanes + Lay::kOCol + c0, o);
                tc_wait_ld();
                if (mine && whole) {
                    uint32_t x[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        x[c / 2] = pack_bf16(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv);
#pragma unroll
                    for (int c = 0; c < 32; c += 16) {
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
                    for (int c = 0; c < 32; c += 4) {
                        if (c0 + c >= p.a.D) break;
                        __stcg(p.part + (slot * (p.a.D / 4) + (c0 + c) / 4) * p.rows + tid,
                               make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]),
                                           __uint_as_float(o[c + 3])));
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
        mbar_init(&sh.drain, 1);
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
    if (warp == 4) {
        copy_role<DP>(p, &qmap, &kmap, &vmap, smem, sh);
        write_status<unsigned short>(p, cta, sh.start.valid);   // while the last tiles are computed
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
    return launch_after(attention_tc_kernel<DP>, dim3(p.ctas), dim3(kTcThreads), bytes, s, p, map[0], map[1], map[2]);
}

bool tensor_q(const spec_attention_args* a) { return (((uintptr_t)a->q | (uintptr_t)(a->q_row_stride * 2)) & 15) == 0; }

// Rows of Q that do not lie on 16-byte boundaries, packed so that they do.
__global__ void __launch_bounds__(256) pack_rows_kernel(const unsigned short* q, int64_t stride, int width, uint4* to) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const uint64_t D = a.D, P = a.page_size;
    const uint32_t box = a.page_size < kTile ? a.page_size : kTile;
    if (!encode3(&map[0], q, D, a.Hq, (uint64_t)(a.q_rows > 0 ? a.q_rows : 1), D * 2, q_stride, p.G, p.rows / p.G) ||
        !encode3(&map[1], a.k_pages, D, P, (uint64_t)a.num_pages * a.Hkv, D * 2, P * D * 2, box, 1) ||
        !encode3(&map[2], a.v_pages, D, P, (uint64_t)a.num_pages * a.Hkv, D * 2, P * D * 2, box, 1))
        return cudaErrorInvalidValue;
    if (a.D <= 64) return launch_tc<64>(p, map, s);
    if (a.D <= 128) return launch_tc<128>(p, map, s);
    return launch_tc<256>(p, map, s);
}

}  // namespace sv
