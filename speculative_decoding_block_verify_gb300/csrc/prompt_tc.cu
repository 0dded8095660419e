// spec_prompt_attention on the tensor cores: bf16.
//
// One tile of an item (prompt.cuh) is two matrix products around a softmax step,
//   S [rows x keys] = Q [rows x D] K^T,   P = 2^(scale S - m),   O [rows x D] += P V.
// An item has two groups of 128 rows (heads above 128: one), which share every tile of keys and values in shared memory.  While the
// softmax of one group runs, the tensor cores have the other group's products: O0 += P0 V, S0' = Q0 K'^T, O1 += P1 V, S1' = Q1
// K'^T, and so on round.  At 128 rows, 128 keys and heads of 128 a product takes 512 tensor cycles, so a group's softmax has 1,024 to itself.
// Each group's S and P share 128 columns of tensor memory (P, bf16, over S; what is issued to the tensor cores runs in its order, so
// S' may be issued behind the product that reads P), and its O has D more.
//
// Warps 0 to 3 and 4 to 7 are a group's softmax, a row per thread (TMEM lane = row): the row's running maximum and sum in registers, O scaled in
// tensor memory when the maximum has risen by more than 8 (2^8 of headroom is nothing to float32, and most tiles then leave O alone).
// Warp 11 finds the items, warp 8 copies keys and values by TMA, warp 10 the rows of Q, warp 9 issues the products.
//
// What it measured (one GB300; a graph of 20 calls on two inputs by turns): one prompt of 16,001 tokens, 64/8 heads of 128, 2.55 to 2.64 ms, 1,589 to
// 1,642 TFLOP/s, 0.84 to 0.87 of what the library's largest bf16 product reaches (2.69 ms as calls from Python, 2.86 on a slower card); 24 prompts of 17
// to 2,000 tokens 169 us (0.59: an item's beginning and end take two tiles' time, and it has five; 12 % of the tiles' scores are unseen); six prompts of
// 2,000 to 9,000 with a window of 1,024 and 4 first tokens 575 us (0.63); 333 tokens 9.0 us, 17 tokens 7.3 (latency).
// What bounds it: a tile of both groups takes about 3,000 cycles, 2,048 of them products.  The softmax of a group takes about 1,500 (a warp alone on
// its quarter of the SM, 600 instructions one behind the other), then its products have to run before it has scores again: neither the tensor cores
// (about two thirds of the cycles) nor the function units (a third) are full, the chain is.  What did not shorten it:
//  - two threads a row, in four warpgroups that exchange maxima: 3.26 ms against 2.63 (with 96 registers a thread, and more waits);
//  - a warp of products for either group: 3.09 ms (both groups' products then run interleaved, end together, and the softmax waits together);
//  - weights against the old maximum while the new one is looked for: 2.88 ms; scores read 32 or 64 at a time in loops: 2.81, 2.95;
//  - a warpgroup of its own for the output: 2.78 to 2.94 ms, and worse for short prompts: what runs beside takes instructions' place;
//  - output through shared memory and one copy: 1.2 us more for 17 tokens; weights announced in quarters: 2.95 ms, in one piece 2.78.
// What did: one place after the other where code was long or loops were unrolled without need.  Roles share what keeps instructions, and the walk
// alone (prompt.cuh), at 54 KB, cost a call of 333 tokens 1.2 of 10.3 us.

#include <atomic>

#include "host_util.h"
#include "prompt.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace sv {

static __device__ int32_t g_mark;   // a wait gave up since it was last cleared
static __global__ void mark_kernel(int32_t marked) { g_mark = marked; }
cudaError_t mark_prompt_tc(int32_t marked, cudaStream_t s) {
    mark_kernel<<<1, 1, 0, s>>>(marked);
    return cudaGetLastError();
}

constexpr int kPromptThreads = 384;
// registers of a thread of the softmax's two warpgroups and of the last one, where the CTA was launched with kRegsStart each
constexpr int kRegsRows = 208, kRegsOthers = 88, kRegsStart = 168;
static_assert(2 * kRegsRows + kRegsOthers <= 3 * kRegsStart, "setmaxnreg would wait for ever");

// DP: the head padded to 64, 128 or 256 columns (TMA fills the rest with zeros).
template <int DP>
struct PromptLayout {
    static constexpr int kGroups = DP == 256 ? 1 : 2;
    static constexpr int kKeys = DP == 256 ? 64 : 128;         // positions of a tile
    static constexpr int kHalves = DP / 64;                    // 64-column panels (128 bytes a row)
    static constexpr int kQPanel = kTcRows * 128;              // bytes
    static constexpr int kQBytes = kHalves * kQPanel;          // of a group
    static constexpr int kPanel = kKeys * 128;
    static constexpr int kSlotBytes = kHalves * kPanel;        // K or V of one tile
    static constexpr int kSlots = DP == 64 ? 10 : 5;
    static constexpr int kHalf = kKeys / 2;                    // P comes in two halves
    static constexpr int kBuffers = 2;                         // of S: a group's, or (one group) every other tile's
    static constexpr int kOCol = kBuffers * kKeys;
    static constexpr int kCols = 512;
    static constexpr int kRing = kGroups * kQBytes, kBytes = kRing + kSlots * kSlotBytes;
    static_assert(kOCol + kGroups * DP <= kCols, "columns of tensor memory");
};

// The keys that an item's rows see are cut into tiles of kKeys positions: those of the window, or all up to the last row's, from the
// first one on (`begin`; a copy may start at any row), and in front of them the first tokens that stay visible.  Few of those (up to half a tile) get
// the first places of the first tile, rounded up to 16 (`lead`); many get tiles of their own.
struct PromptSegment {
    int tiles;           // of the item, and of each of its groups; 0: the CTA is done
    int group_tiles[2];
    int sink_tiles, begin, lead;
    int high, sink;      // visible positions end at `high`, the first tokens' at `sink`
    int at, tokens, head;
    int64_t row0;
    template <int kKeys, bool kWindow>
    __device__ __forceinline__ int start(int t) const {
        return !kWindow || t < sink_tiles ? t * kKeys : begin + (t - sink_tiles) * kKeys;
    }
};

struct PromptShared {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_done[2], drain;
    uint64_t full[10], empty[10];
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    PromptSegment seg[kSegments];
    uint32_t tmem;
    int abort;
    int moved;   // tiles copied so far
};

// ---- warp 11: the walk over the CTA's items ------------------------------------------------------
template <int DP, bool kWindow>
__device__ __forceinline__ void prompt_walk_role(const PromptParams& p, PromptShared& sh, PromptWalk& w) {
    using Lay = PromptLayout<DP>;
    const int lane = threadIdx.x & 31;
    Piece it = {};
    w.start();
    for (int told = 0;; ++told) {
        const bool any = w.next(p, &it);
        PromptSegment& seg = sh.seg[told % kSegments];
        if (!warp_wait_moving(&sh.seg_empty[told % kSegments], ((told / kSegments) & 1) ^ 1, &sh.abort, &sh.moved)) return;
        if (lane == 0) {
            seg.tiles = 0;
            if (any) {
                const int low = kWindow ? max(0, it.at + 1 - p.a.window) : 0, sink = kWindow ? min(p.a.sinks, low) : 0;
                const bool few = sink <= Lay::kKeys / 2;
                seg.sink = sink;
                seg.high = it.at + it.tokens;
                seg.lead = few ? (sink + 15) & ~15 : 0;
                seg.begin = low - seg.lead;
                seg.sink_tiles = few ? 0 : (sink + Lay::kKeys - 1) / Lay::kKeys;
                seg.tiles = seg.sink_tiles + (int)(((unsigned)(seg.high - seg.begin) + Lay::kKeys - 1) / Lay::kKeys);
#pragma unroll
                for (int g = 0; g < Lay::kGroups; ++g) {
                    const int mine = min(p.group, it.tokens - g * p.group), last = it.at + g * p.group + mine - 1;
                    seg.group_tiles[g] = mine > 0 ? seg.sink_tiles + (last - seg.begin) / Lay::kKeys + 1 : 0;
                }
                seg.at = it.at, seg.tokens = it.tokens, seg.head = it.head, seg.row0 = it.row0;
            }
            mbar_arrive(&sh.seg_full[told % kSegments]);
        }
        __syncwarp();
        if (!any) return;
    }
}

// ---- warp 8: keys and values ------------------------------------------------------------------
template <int DP, bool kWindow>
__device__ __forceinline__ void prompt_copy_role(const CUtensorMap* kmap, const CUtensorMap* vmap, const CUtensorMap* kmap16, const CUtensorMap* vmap16,
                                                 char* smem, PromptShared& sh) {
    using Lay = PromptLayout<DP>;
    const int lane = threadIdx.x & 31;
    static_assert(Lay::kKeys / 16 * Lay::kHalves <= 32, "a lane a copy");
    const uint32_t ring = smem_u32(smem) + Lay::kRing;
    const uint64_t stay = l2_evict_normal_policy();
    int slot = 0;
    unsigned phase = 1;   // a fresh barrier: the phase before its first is done
    bool ok = true;
    // a tile's rows, or (lead > 0) the first `lead` and the window's behind them, 16 rows a copy
    auto copy = [&](const CUtensorMap* map, const CUtensorMap* map16, int head, int first, int row, int lead) {
        ok = ok && warp_wait_for(&sh.empty[slot], phase, &sh.abort);
        if (!ok) return;
        if (kWindow && lead > 0) {
            if (lane == 0) mbar_expect_tx(&sh.full[slot], Lay::kSlotBytes);
            __syncwarp();
            const int i = lane / Lay::kHalves * 16, half = lane % Lay::kHalves;
            if (i < Lay::kKeys)
                tma_load_3d(ring + slot * Lay::kSlotBytes + half * Lay::kPanel + i * 128, map16, half * 64, head, (i < lead ? first : row) + i,
                            &sh.full[slot], stay);
        } else if (lane == 0) {
            mbar_expect_tx(&sh.full[slot], Lay::kSlotBytes);
#pragma unroll
            for (int half = 0; half < Lay::kHalves; ++half)
                tma_load_3d(ring + slot * Lay::kSlotBytes + half * Lay::kPanel, map, half * 64, head, row, &sh.full[slot], stay);
        }
        __syncwarp();
        if (++slot == Lay::kSlots) {
            slot = 0;
            phase ^= 1;
        }
    };
    for (int n_seg = 0; ok; ++n_seg) {
        const int place = n_seg % kSegments;
        ok = warp_wait_for(&sh.seg_full[place], (n_seg / kSegments) & 1, &sh.abort);
        if (!ok) break;
        const PromptSegment w = sh.seg[place];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[place]);
        if (w.tiles == 0) return;
        for (int t = 0; t < w.tiles && ok; ++t) {
            const int row0 = (int)w.row0, row = row0 + w.start<Lay::kKeys, kWindow>(t), lead = t == 0 ? w.lead : 0;
            copy(kmap, kmap16, w.head, row0, row, lead);
            copy(vmap, vmap16, w.head, row0, row, lead);
            if (lane == 0) *reinterpret_cast<volatile int*>(&sh.moved) += 1;
        }
    }
    // gave up: whatever was copied must have arrived before the CTA's memory is given back
    for (int s = 0; s < Lay::kSlots; ++s)
        for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
}

// ---- warp 10: the rows of Q ----------------------------------------------------------------------
// An item's rows are on their way to L2 as soon as it is known, and to shared memory when the item before has no more use of its own.
template <int DP>
__device__ __forceinline__ void prompt_queries_role(const PromptParams& p, const CUtensorMap* qmap, char* smem, PromptShared& sh) {
    using Lay = PromptLayout<DP>;
    const int lane = threadIdx.x & 31;
    const uint32_t q_at = smem_u32(smem);
    const uint64_t stay = l2_evict_normal_policy();
    unsigned copies[2] = {0, 0};
    bool ok = true;
    for (int n_seg = 0; ok; ++n_seg) {
        const int place = n_seg % kSegments;
        ok = warp_wait_moving(&sh.seg_full[place], (n_seg / kSegments) & 1, &sh.abort, &sh.moved);
        if (!ok) break;
        const int tiles = sh.seg[place].tiles, tokens = sh.seg[place].tokens, head = sh.seg[place].head * p.G;
        const int row = (int)sh.seg[place].row0 + sh.seg[place].at;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[place]);
        if (tiles == 0) break;
        if (lane < Lay::kHalves * Lay::kGroups && lane / Lay::kHalves * p.group < tokens)
            tma_prefetch_3d(qmap, lane % Lay::kHalves * 64, head, row + lane / Lay::kHalves * p.group);
#pragma unroll
        for (int g = 0; g < Lay::kGroups; ++g) {
            if (g * p.group >= tokens) break;
            ok = ok && warp_wait_moving(&sh.q_empty[g], (copies[g] & 1) ^ 1, &sh.abort, &sh.moved);
            if (!ok) break;
            if (lane == 0) {
                mbar_expect_tx(&sh.q_full[g], Lay::kHalves * p.group * p.G * 128);
#pragma unroll
                for (int half = 0; half < Lay::kHalves; ++half)
                    tma_load_3d(q_at + g * Lay::kQBytes + half * Lay::kQPanel, qmap, half * 64, head, row + g * p.group, &sh.q_full[g], stay);
            }
            __syncwarp();
            ++copies[g];
        }
    }
    if (!ok)
#pragma unroll
        for (int g = 0; g < Lay::kGroups; ++g)
            for (int n = 0; copies[g] > 0 && n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.q_full[g], (copies[g] - 1) & 1); ++n) {}
}

// ---- warp 9: products -------------------------------------------------------------------------
// The whole warp runs the loop, so that descriptors and addresses are uniform; one lane issues.
template <int DP>
__device__ __forceinline__ bool prompt_products_role(const PromptParams& p, char* smem, PromptShared& sh) {
    using Lay = PromptLayout<DP>;
    constexpr int kGroups = Lay::kGroups;
    const uint32_t q_at = smem_u32(smem), ring = q_at + Lay::kRing;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    const int ksteps = (p.a.D + 15) / 16;
    // a negative scale is a negated Q (bit 13) and its magnitude
    const uint32_t qk = mma_desc(Lay::kKeys, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    const uint32_t pv = mma_desc(ksteps * 16, true);   // as many columns of O as the head has
    int items[2] = {0, 0};                             // of each group so far
    unsigned k_at = 0, v_at = 1;                       // places in the ring, counted from the start: keys and values take turns
    unsigned s_count = 0;                              // (one group) products S so far
    unsigned p_count[2] = {0, 0};                      // products of each buffer's P so far
    auto full = [&](unsigned at) { return warp_wait_for(&sh.full[at % Lay::kSlots], (at / Lay::kSlots) & 1, &sh.abort); };
    auto keys = [&](int g, int buf, bool last) {       // S of the tile at k_at
        const uint32_t a = desc_lo(q_at + g * Lay::kQBytes, 1), b = desc_lo(ring + k_at % Lay::kSlots * Lay::kSlotBytes, 1);
        tc_fence_after();
        if (elected()) {
#pragma unroll
            for (int k = 0; k < Lay::kHalves * 4; ++k)
                if (k < ksteps)
                    mma_ss(tmem + buf * Lay::kKeys, desc(a + (k >> 2) * (Lay::kQPanel >> 4) + (k & 3) * 2, 1024 >> 4),
                           desc(b + (k >> 2) * (Lay::kPanel >> 4) + (k & 3) * 2, 1024 >> 4), qk, k > 0);
            mma_commit(&sh.s_full[buf]);
            if (last) mma_commit(&sh.q_empty[g]);
        }
        __syncwarp();
    };
    auto values = [&](int g, int buf, bool add) {      // O += P V of the tile at v_at
        const uint32_t v = desc_lo(ring + v_at % Lay::kSlots * Lay::kSlotBytes, Lay::kPanel >> 4);
        const unsigned phase = p_count[buf]++ & 1;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            if (!warp_wait_for(&sh.p_full[buf][part], phase, &sh.abort)) return false;
            tc_fence_after();
            if (elected()) {
#pragma unroll
                for (int k = part * Lay::kHalf / 16; k < (part + 1) * Lay::kHalf / 16; ++k)
                    mma_ts(tmem + Lay::kOCol + g * DP, tmem + buf * Lay::kKeys + k * 8, desc(v + 2 * k * (1024 >> 4), 1024 >> 4), pv, add || k > 0);
            }
            __syncwarp();
        }
        return true;
    };
    auto release = [&](unsigned at) {
        if (elected()) mma_commit(&sh.empty[at % Lay::kSlots]);
        __syncwarp();
    };
    int at = 0, tiles = 0, n[2] = {0, 0};
    auto next = [&](int* tiles_out, int* n_out) {      // the next item's tiles
        const int place = at % kSegments;
        if (!warp_wait_for(&sh.seg_full[place], (at / kSegments) & 1, &sh.abort)) return false;
        *tiles_out = (int)__reduce_max_sync(0xffffffffu, (unsigned)sh.seg[place].tiles);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) n_out[g] = (int)__reduce_max_sync(0xffffffffu, (unsigned)sh.seg[place].group_tiles[g]);
        if (elected()) mbar_arrive(&sh.seg_empty[place]);
        __syncwarp();
        ++at;
        return true;
    };
    if (!next(&tiles, n)) return false;
    if (tiles == 0) return true;
    if (kGroups == 2) {
        if (!full(k_at)) return false;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (n[g] == 0) continue;
            if (!warp_wait_for(&sh.q_full[g], items[g] & 1, &sh.abort)) return false;
            ++items[g];
            keys(g, g, n[g] == 1);
        }
        release(k_at);
        k_at += 2;
        for (;;) {
            int after = 0, m[2] = {0, 0};   // the next item
            for (int t = 0; t < tiles; ++t) {
                const bool last = t == tiles - 1;
                if (last && !next(&after, m)) return false;
                const bool more = !last || after > 0;   // tiles behind this one
                bool ready = false;
                if (!full(v_at)) return false;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (t < n[g]) {
                        if (!values(g, g, t > 0)) return false;
                        if (t == n[g] - 1) {
                            if (elected()) mma_commit(&sh.o_done[g]);
                            __syncwarp();
                        }
                    }
                    if (g == 1) release(v_at);
                    if (more && (last ? m[g] > 0 : t + 1 < n[g])) {
                        if (!ready && !full(k_at)) return false;
                        ready = true;
                        if (last) {
                            if (!warp_wait_for(&sh.q_full[g], items[g] & 1, &sh.abort)) return false;
                            ++items[g];
                        }
                        keys(g, g, last ? m[g] == 1 : t + 2 == n[g]);
                    }
                }
                if (more) {
                    release(k_at);
                    k_at += 2;
                }
                v_at += 2;
            }
            if (after == 0) return true;
            tiles = after;
            n[0] = m[0], n[1] = m[1];
        }
    } else {
        // S of tile t + 1 goes to the other buffer before O += P V of tile t
        unsigned o_count = 0;
        auto ahead = [&](bool begin, bool end) {
            if (!full(k_at)) return false;
            if (begin && !warp_wait_for(&sh.q_full[0], items[0]++ & 1, &sh.abort)) return false;
            keys(0, s_count++ & 1, end);
            release(k_at);
            k_at += 2;
            return true;
        };
        if (!ahead(true, tiles == 1)) return false;
        for (;;) {
            int after = 0, m[2] = {0, 0};
            for (int t = 0; t < tiles; ++t) {
                const bool last = t == tiles - 1;
                if (last && !next(&after, m)) return false;
                if ((!last || after > 0) && !ahead(last, last ? after == 1 : t + 2 == tiles)) return false;
                const int buf = o_count++ & 1;
                if (!full(v_at)) return false;
                if (!values(0, buf, t > 0)) return false;
                if (elected()) mma_commit(&sh.o_done[buf]);
                __syncwarp();
                release(v_at);
                v_at += 2;
            }
            if (after == 0) return true;
            tiles = after;
        }
    }
}

// Two sums and the bf16 pair w, each in one instruction.
__device__ __forceinline__ void add_bf16(float2& sum, uint32_t w) {
    asm("{\n\t.reg .b16 l, h, one;\n\tmov.b16 one, 0x3F80;\n\tmov.b32 {l, h}, %2;\n\t"
        "fma.rn.f32.bf16 %0, l, one, %0;\n\tfma.rn.f32.bf16 %1, h, one, %1;\n\t}"
        : "+f"(sum.x), "+f"(sum.y)
        : "r"(w));
}

// The lowest n bits of a word (none, or all, where n is outside 0 to 32).
__device__ __forceinline__ unsigned below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// Maxima of n scores, in four chains of three-way maxima.
template <int n>
__device__ __forceinline__ void tops(const uint32_t* s, float (&x)[4]) {
#pragma unroll
    for (int c = 0; c < n; c += 2) x[(c >> 1) & 3] = fmaxf(fmaxf(x[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
}
// Weights 2^(s scale - base) as bf16 pairs, and their sums.  P V takes both operands in one type, so the weights are rounded to bf16, and the
// sum takes them as rounded.
template <int n>
__device__ __forceinline__ void weights(const uint32_t* s, float2 scale, float2 minus_base, uint32_t* pk, float2 (&sum)[2]) {
#pragma unroll
    for (int c = 0; c < n; c += 2) {
        const float2 y = ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale, minus_base);
        pk[c / 2] = pack_bf16(ex2(y.x), ex2(y.y));
        add_bf16(sum[(c >> 1) & 1], pk[c / 2]);
    }
}
// Lanes l and l ^ mask exchange: of pieces i and i | mask (8 words each) the lane whose bit is 0 keeps i and gives the other, and
// so on.  With masks 1 and 2 lane l ends up with piece l & 3 of the four lanes' rows, in their order.
__device__ __forceinline__ void swap_pieces(uint32_t (&y)[32], int mask) {
    const bool up = (threadIdx.x & mask) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i & mask) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t& a = y[8 * i + c];
            uint32_t& b = y[8 * (i | mask) + c];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, mask);
            a = up ? got : a;
            b = up ? b : got;
        }
    }
}
// Half of a tile's P to tensor memory, and the products' warp told.
template <int n>
__device__ __forceinline__ void announce(uint32_t at, const uint32_t* pk, uint64_t* bar) {
    __syncwarp();
    if constexpr (n == 64)
        tmem_st32(at, pk);
    else
        tmem_st16(at, pk);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---- warps 0 to 3, 4 to 7: softmax, scaling, output ----------------------------------------------
template <int DP, bool kWindow>
__device__ __forceinline__ void prompt_softmax_role(const PromptParams& p, char* smem, PromptShared& sh, int g) {
    using Lay = PromptLayout<DP>;
    constexpr int kKeys = Lay::kKeys, kGroups = Lay::kGroups, kHalf = Lay::kHalf;
    const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t o_at = lanes + Lay::kOCol + g * DP;
    const int token_in = p.by_G.of(tid), query = tid - token_in * p.G;
    const bool wide = (((uint32_t)reinterpret_cast<uintptr_t>(p.a.out) | p.a.D * 2) & 31) == 0;   // 32-byte stores
    unsigned n_all = 0, tiles_all = 0, items = 0;   // tiles of the group, of the CTA, and the group's items so far
    for (int n_seg = 0;; ++n_seg) {
        const int place = n_seg % kSegments;
        if (!warp_wait_moving(&sh.seg_full[place], (n_seg / kSegments) & 1, &sh.abort, &sh.moved)) return;
        const PromptSegment w = sh.seg[place];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[place]);
        if (w.tiles == 0) return;
        const int n = kGroups == 1 ? w.tiles : g == 0 ? w.group_tiles[0] : w.group_tiles[1];
        const int fixes_from = g == 0 ? 0 : w.group_tiles[0];   // the tiles whose values this group looks after
        const int tokens = min(p.group, w.tokens - g * p.group);
        const int at_first = w.at + g * p.group, at_last = at_first + tokens - 1;
        const bool mine = token_in < tokens;
        const int at = min(at_first + token_in, at_last);
        const int low = kWindow ? max(0, at + 1 - p.a.window) : 0;   // the row sees [low, at] and [0, sinks)
        float m = -kInf, l = 0.f;
        for (int t = 0; t < n; ++t, ++n_all) {
            const int buf = kGroups == 2 ? g : (int)(n_all & 1);
            const unsigned uses = kGroups == 2 ? n_all : n_all >> 1;
            const int j0 = w.start<kKeys, kWindow>(t), lead = kWindow && t == 0 ? w.lead : 0;
            if (!warp_wait_moving(&sh.s_full[buf], uses & 1, &sh.abort, &sh.moved)) return;   // (the other group's items may have no rows of this one)
            tc_fence_after();
            // a tile that every row sees whole needs no mask
            const bool first = kWindow && t < w.sink_tiles;   // of the first tokens alone
            const bool clean = first ? j0 + kKeys <= w.sink : lead == 0 && at_first - j0 >= kKeys - 1 && (!kWindow || j0 > at_last - p.a.window);
            if (kWindow && !clean) {
                // A bit a column (a comparison each, as it comes from the compiler, takes 8,000 cycles), 32 columns at a time and in
                // place: unrolled, the longer masks take 2,000, of which most is waiting for instructions.
                // A first tile that begins in front of the prompt (at -15 or behind) holds no position of kKeys or more: what is near 2^31, less
                // a negative position, does not fit 32 bits.
                const int far = j0 < 0 ? kKeys : INT32_MAX;
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 32) {
                    const int j = j0 + c;
                    unsigned sees = below(min(at + 1, far) - j);
                    if (kWindow) {
                        const unsigned leads = below(lead - c);
                        sees = first ? below(w.sink - j) : (sees & (~below(low - j) | below(min(p.a.sinks, far) - j)) & ~leads) | (below(w.sink - c) & leads);
                    }
                    if (!__any_sync(0xffffffffu, sees != ~0u)) continue;
                    uint32_t s[32];
                    tmem_ld32(lanes + buf * kKeys + c, s);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = sees >> i & 1 ? s[i] : 0xff800000u;
                    __syncwarp();
                    tmem_st32(lanes + buf * kKeys + c, s);
                }
                tc_wait_st();
            }
            uint32_t s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(lanes + buf * kKeys + c, s + c);
            tc_wait_ld();
            if (!kWindow && !clean) {
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    const unsigned sees = below(at + 1 - j0 - c);
                    if (__any_sync(0xffffffffu, sees != ~0u)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[c + i] = sees >> i & 1 ? s[c + i] : 0xff800000u;
                    }
                }
            }
            float x[4] = {-kInf, -kInf, -kInf, -kInf};
            tops<kKeys>(s, x);
            const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;   // the scale is positive here
            float scale_o = 1.f;
            if (mine && top > m + 8.f) {   // lanes without a row never ask for the scaling of O
                scale_o = m == -kInf ? 0.f : ex2(m - top);
                m = top;
                l *= scale_o;
            }
            if (t > 0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
                // (two groups: S of this tile was issued behind the product before, so that is done)
                if (kGroups == 1 && !warp_wait_for(&sh.o_done[buf ^ 1], ((n_all - 1) >> 1) & 1, &sh.abort)) return;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_at + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale_o);
                    tmem_st32(o_at + c, o);
                }
            }
            // values of positions that no row of the item sees (another prompt's, or what lies behind the last): zeros, whatever is
            // there.  The first group that uses the tile sees to it, a position a thread, before its P is announced.
            const int from = min(kKeys, (first ? w.sink : w.high) - j0);
            if (!clean && t >= fixes_from && (from < kKeys || (kWindow && w.sink < lead))) {
                const unsigned in = 2 * (tiles_all + t) + 1;
                if (!warp_wait_for(&sh.full[in % Lay::kSlots], (in / Lay::kSlots) & 1, &sh.abort)) return;
                if (tid < kKeys && (tid >= from || (kWindow && tid >= w.sink && tid < lead))) {
                    char* const to = smem + Lay::kRing + in % Lay::kSlots * Lay::kSlotBytes + tid * 128;
#pragma unroll 4
                    for (int c = 0; c < Lay::kHalves * 8; ++c)
                        *reinterpret_cast<uint4*>(to + (c >> 3) * Lay::kPanel + (((c & 7) ^ (tid & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            const float base = m == -kInf ? 0.f : m;
            const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[kHalf / 2];
                weights<kHalf>(s + half * kHalf, sc, nb, pk, sum);
                announce<kHalf>(lanes + buf * kKeys + half * (kHalf / 2), pk, &sh.p_full[buf][half]);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        tiles_all += w.tiles;
        if (n == 0) continue;
        if (kGroups == 2 ? !warp_wait_for(&sh.o_done[g], items & 1, &sh.abort)
                         : !warp_wait_for(&sh.o_done[(n_all - 1) & 1], ((n_all - 1) >> 1) & 1, &sh.abort))
            return;
        ++items;
        tc_fence_after();
        const float inv = 1.f / l;
        unsigned short* const first = reinterpret_cast<unsigned short*>(p.a.out) + ((w.row0 + at_first) * p.a.Hq + w.head * p.G) * (int64_t)p.a.D;
#pragma unroll 1
        for (int c0 = 0; c0 < p.a.D; c0 += 64) {
            uint32_t o[64], y[32];
            __syncwarp();
            tmem_ld32(o_at + c0, o);
            tmem_ld32(o_at + c0 + 32, o + 32);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 64; c += 2) y[c / 2] = pack_bf16(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv);
            if (wide && p.a.D - c0 >= 64) {
                // four lanes swap pieces of 32 bytes, so that a store writes whole lines of eight rows instead of pieces of 32
                swap_pieces(y, 1);
                swap_pieces(y, 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = (tid & ~3) + i, token = p.by_G.of(row);
                    if (token < tokens) store32(first + (int64_t)token * p.a.Hq * p.a.D + (row - token * p.G) * p.a.D + c0 + (tid & 3) * 16, y + 8 * i);
                }
            } else if (mine) {
                unsigned short* const to = first + (int64_t)token_in * p.a.Hq * p.a.D + query * p.a.D + c0;
#pragma unroll
                for (int c = 0; c < 64; c += 8)
                    if (c0 + c < p.a.D) *reinterpret_cast<uint4*>(to + c) = make_uint4(y[c / 2], y[c / 2 + 1], y[c / 2 + 2], y[c / 2 + 3]);
            }
        }
        __syncwarp();
        tc_fence_before();
    }
}

template <int DP, bool kWindow>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_tc_kernel(const PromptParams p, const __grid_constant__ CUtensorMap qmap,
                                                                    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                                                    const __grid_constant__ CUtensorMap kmap16, const __grid_constant__ CUtensorMap vmap16) {
    using Lay = PromptLayout<DP>;
    extern __shared__ __align__(1024) char smem[];
    PromptShared& sh = *reinterpret_cast<PromptShared*>(smem + Lay::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 8 && (tid & 31) < 3) {
        const CUtensorMap* map = (tid & 31) == 0 ? &kmap : (tid & 31) == 1 ? &vmap : &qmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"((uint32_t)Lay::kCols)
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
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.o_done[i], 1);
            for (int half = 0; half < 2; ++half) mbar_init(&sh.p_full[i][half], 4);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], 4 * Lay::kGroups + 3);   // softmax, copies of keys and values, of queries, products
        }
        mbar_init_fence();
        sh.abort = sh.moved = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= 8) {
        if (Lay::kGroups == 2) registers_down<kRegsOthers>();
        if (warp == 8) {
            prompt_copy_role<DP, kWindow>(&kmap, &vmap, &kmap16, &vmap16, smem, sh);
        } else if (warp == 9) {
            if (!prompt_products_role<DP>(p, smem, sh)) drain(&sh.drain);
        } else if (warp == 10) {
            prompt_queries_role<DP>(p, &qmap, smem, sh);
        } else {
            PromptWalk w;
            prompt_walk_role<DP, kWindow>(p, sh, w);
            prompt_statuses(p, w, &g_mark);   // while the last tiles are computed
        }
    } else {
        if (Lay::kGroups == 2) registers_up<kRegsRows>();
        if (warp < 4 * Lay::kGroups) prompt_softmax_role<DP, kWindow>(p, smem, sh, warp >> 2);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"((uint32_t)Lay::kCols));
    }
    if (warp == 8 && sh.abort) prompt_gave_up<unsigned short>(p, 0x7fff, &g_mark);
}

// ---------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------
// [rows][heads][D] in boxes of 64 columns, some heads, some rows.
static bool encode_rows(CUtensorMap* map, const void* base, const spec_prompt_args& a, int heads, int64_t stride, int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)heads, (cuuint64_t)a.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, 3, dims, strides, box);
}

template <int DP, bool kWindow>
static cudaError_t launch(PromptParams p, int sms, cudaStream_t s) {
    using Lay = PromptLayout<DP>;
    static std::atomic<int> ready[64];   // whether the device's kernel has its shared memory
    constexpr int bytes = Lay::kBytes + (int)sizeof(PromptShared);
    static_assert(bytes <= 232448, "shared memory of an SM");
    p.piece = p.group * Lay::kGroups;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes of;
        e = cudaFuncGetAttributes(&of, prompt_tc_kernel<DP, kWindow>);
        if (e != cudaSuccess) return e;
        if (Lay::kGroups == 2 && of.numRegs != kRegsStart) return cudaErrorInvalidConfiguration;   // the shares would not add up
        e = cudaFuncSetAttribute(prompt_tc_kernel<DP, kWindow>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_release);
    }
    CUtensorMap q, k, v, k16, v16;
    if (!encode_rows(&q, p.a.q, p.a, p.a.Hq, p.a.q_row_stride, p.G, p.group) ||
        !encode_rows(&k, p.a.k, p.a, p.a.Hkv, p.a.k_row_stride, 1, Lay::kKeys) ||
        !encode_rows(&v, p.a.v, p.a, p.a.Hkv, p.a.v_row_stride, 1, Lay::kKeys))
        return cudaErrorInvalidValue;
    k16 = k, v16 = v;
    if (kWindow && p.a.sinks > 0 &&
        (!encode_rows(&k16, p.a.k, p.a, p.a.Hkv, p.a.k_row_stride, 1, 16) || !encode_rows(&v16, p.a.v, p.a, p.a.Hkv, p.a.v_row_stride, 1, 16)))
        return cudaErrorInvalidValue;
    return launch_after(prompt_tc_kernel<DP, kWindow>, dim3((unsigned)prompt_ctas(p, sms)), dim3(kPromptThreads), bytes, s, p, q, k, v, k16, v16);
}

cudaError_t launch_prompt_tc(const PromptParams& p, int sms, cudaStream_t s) {
    // Kernels of their own for the window: its masks and first tokens in the code of all tiles cost short prompts a tenth (17 tokens 7.6
    // against 8.2 us, 1,000 tokens 23.7 against 25.2).
    const bool window = p.a.window > 0;
    if (p.a.D <= 64) return window ? launch<64, true>(p, sms, s) : launch<64, false>(p, sms, s);
    if (p.a.D <= 128) return window ? launch<128, true>(p, sms, s) : launch<128, false>(p, sms, s);
    return window ? launch<256, true>(p, sms, s) : launch<256, false>(p, sms, s);
}

}  // namespace sv
