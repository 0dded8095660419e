// spec_paged_attention on the tensor cores: float32 caches, heads up to 128.
//
// A float32 is the sum of three bf16: x = x0 + x1 + x2 + O(2^-27 |x|), each the rounding of what the ones before
// leave.  A product of two such sums needs the six terms x0 y0, x0 y1, x1 y0, x1 y1, x0 y2, x2 y0 (the other three are
// below 2^-24 of x0 y0), each exact in float32, so six bf16 products with a float32 accumulator stand for a float32
// product.  At M = 128 a tile of 64 positions costs 6 x 512 = 3,072 tensor cycles against about 2,800 that its
// 64 KB take from memory; on the float pipes 32 rows alone take 8,192.
//
// One CTA per SM, fourteen warps: copies (warp 12) bring pages as they lie into a ring; warps 4 to 7 split the keys and
// warps 8 to 11 the values into swizzled bf16 planes (zeros where no row of the item sees a position, whatever the
// cache holds there), the latter also the item's rows of Q into tensor memory; warp 13 issues the products; warps 0
// to 3 hold a row per thread: softmax, P split into three planes in tensor memory, scaling of O, output.  There is
// one set of planes each for keys and values: a tile's keys are split during the product of the values before,
// and its values during its keys' product, so the tensor cores do not wait for either.
// The tensor cores cut their running sums off instead of rounding them: over 5,000 positions in one accumulator the output
// came out 1.7e-5 too small.  So every tile's P V is a product of its own, and the sums over tiles are rounded float32
// additions in shared memory: 6e-7 off there, a third of what a float32 matrix product is, at the same speed.
// An infinite key or value counts as NaN here (the difference to its rounding is).

#include <atomic>

#include "host_util.h"
#include "tcgen05.cuh"

namespace sv {

constexpr int kF32Threads = 448;
constexpr int kPlanes = 3;
constexpr int kTerms = 6;   // (plane of A, plane of B), the largest last
__host__ __device__ constexpr int term_a(int i) { return i == 0 ? 2 : i == 2 || i == 3 ? 1 : 0; }
__host__ __device__ constexpr int term_b(int i) { return i == 1 ? 2 : i == 2 || i == 4 ? 1 : 0; }

// DP: the head padded to 64 or 128 columns
template <int DP>
struct F32Layout {
    static constexpr int kPlane = DP / 64 * kTile * 128;          // one plane of 64 positions, [panel][64 rows][128 bytes]
    static constexpr int kRaw = kTile * DP * 4;                    // a tile as it lies
    static constexpr int kRaws = DP == 128 ? 2 : 8;
    static constexpr int kSums = kTcRows * DP * 4;                 // O of the tiles so far, [D / 4][row]
    static constexpr int kBytes = 2 * kPlanes * kPlane + kRaws * kRaw + kSums;
    // columns of tensor memory
    static constexpr int kQ = 0, kS = 192, kP = 256, kO = 384, kCols = 512;
};

struct F32Shared {
    uint64_t raw_full[8], raw_empty[8];
    uint64_t k_full, k_empty, v_full, v_empty;   // the planes
    uint64_t q_full, q_empty, s_full, s_empty, p_full, o_done, drain;
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    int there[8];   // bit i: page i of the slot's tile is in the pool
    Start start;
    int64_t scan[kF32Threads / 32];
    int scratch;
    uint32_t tmem;
    int abort;
};

// Two floats as three bf16 pairs.
__device__ __forceinline__ void split(float x, float y, uint32_t (&w)[kPlanes]) {
    w[0] = pack_bf16(x, y);
    x -= bf16_lo(w[0]);
    y -= bf16_hi(w[0]);
    w[1] = pack_bf16(x, y);
    x -= bf16_lo(w[1]);
    y -= bf16_hi(w[1]);
    w[2] = pack_bf16(x, y);
}

// ---- warp 12: the walk over the CTA's items, and the copies --------------------------------
template <int DP>
__device__ __forceinline__ void f32_copy_role(const AttnParams& p, char* raw, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const int lane = threadIdx.x & 31;
    const int box = min(p.a.page_size, kTile), pages = kTile / box;
    const unsigned box_bytes = box * p.a.D * 4;
    const uint64_t policy = (p.a.kmax + 1) * p.G <= p.rows ? l2_evict_first_policy() : l2_evict_normal_policy();
    const char* pool[2] = {reinterpret_cast<const char*>(p.a.k_pages), reinterpret_cast<const char*>(p.a.v_pages)};
    Walk w = {};
    int told = 0, slot = 0;
    unsigned phase = 1;
    bool ok = true;
    auto tell = [&](bool any) {
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
    auto look_up = [&](int t) -> int64_t {   // lane i: where page i of tile t lies in the pool (bytes), or -1
        const int j = tile_start(w.it, t) + lane * box;
        if (lane >= pages || j >= w.it.high || (j + box <= w.it.low && j >= w.it.sink)) return -1;
        const int page = p.a.page_table[(int64_t)w.b * p.a.max_pages + (j >> p.page_shift)];
        if ((unsigned)page >= (unsigned)p.a.num_pages) return -1;
        return ((((int64_t)page * p.a.Hkv + w.h) * p.a.page_size + (j & (p.a.page_size - 1) & ~(box - 1))) * p.a.D) * 4;
    };
    auto copy = [&](int kv, int64_t at) {
        ok = ok && warp_wait_for(&sh.raw_empty[slot], phase, &sh.abort);
        if (!ok) return;
        const unsigned there = __ballot_sync(0xffffffffu, at >= 0);
        if (lane == 0) {
            sh.there[slot] = (int)there;
            mbar_expect_tx(&sh.raw_full[slot], __popc(there) * box_bytes);
        }
        __syncwarp();
        if (at >= 0) bulk_g2s_hint(raw + slot * Lay::kRaw + lane * box_bytes, pool[kv] + at, box_bytes, &sh.raw_full[slot], policy);
        if (++slot == Lay::kRaws) {
            slot = 0;
            phase ^= 1;
        }
    };
    bool more = w.start(p, sh.start);
    tell(more);
    int t = more ? w.t0 : 0;
    int64_t at = more ? look_up(t) : -1;
    while (more && ok) {
        copy(0, at);
        const int64_t now = at;
        if (++t == w.t1) {
            more = w.next(p);
            tell(more);
            t = w.t0;
        }
        if (more) at = look_up(t);
        copy(1, now);
    }
    if (!ok)   // gave up: whatever was copied must have arrived before the CTA's memory is given back
        for (int s = 0; s < Lay::kRaws; ++s)
            for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.raw_full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
}

// ---- warps 4 to 7 (keys) and 8 to 11 (values, and Q): float32 into planes ------------------
template <int DP, int KV>
__device__ __forceinline__ void f32_split_role(const AttnParams& p, char* planes, char* raw, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
    constexpr int kChunks = DP / 8;   // of a row, eight columns each
    const int chunk = tid % kChunks, row0 = tid / kChunks;
    const int box_shift = min(p.page_shift, 6);
    const bool q_vec = ((reinterpret_cast<uintptr_t>(p.a.q) | (uintptr_t)(p.a.q_row_stride * 4)) & 15) == 0;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    uint64_t* const full = KV ? &sh.v_full : &sh.k_full;
    uint64_t* const empty = KV ? &sh.v_empty : &sh.k_empty;
    char* const to = planes + KV * kPlanes * Lay::kPlane + (chunk >> 3) * (kTile * 128);
    int slot = KV;   // keys and values alternate in the ring
    unsigned phase = 0, n_tile = 0;
    for (int n_seg = 0;; ++n_seg) {
        const int seg_at = n_seg % kSegments;
        if (!warp_wait_for(&sh.seg_full[seg_at], (n_seg / kSegments) & 1, &sh.abort)) return;
        const Segment w = sh.seg[seg_at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[seg_at]);
        if (w.t0 == w.t1) return;
        if (KV == 1) {
            // the item's rows of Q: a thread its row, once the item before is through with its own
            if (!warp_wait_for(&sh.q_empty, (n_seg & 1) ^ 1, &sh.abort)) return;
            tc_fence_after();
            const int rr = w.r0 + min(tid, w.rows - 1), token = p.by_G.of(rr);
            const float* q = reinterpret_cast<const float*>(p.a.q) + (w.row0 + token) * p.a.q_row_stride +
                             (int64_t)(w.head * p.G + rr - token * p.G) * p.a.D;
#pragma unroll 1
            for (int c0 = 0; c0 < DP; c0 += 32) {
                uint32_t x[kPlanes][16];
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c0 + c < p.a.D) {
                        const float* from = q + c0 + c;
                        y = q_vec ? *reinterpret_cast<const float4*>(from) : make_float4(from[0], from[1], from[2], from[3]);
                    }
                    uint32_t u[kPlanes], v[kPlanes];
                    split(y.x, y.y, u);
                    split(y.z, y.w, v);
#pragma unroll
                    for (int i = 0; i < kPlanes; ++i) {
                        x[i][c / 2] = u[i];
                        x[i][c / 2 + 1] = v[i];
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kPlanes; ++i) tmem_st16(lanes + Lay::kQ + i * (DP / 2) + c0 / 2, x[i]);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        }
        for (int t = w.t0; t < w.t1; ++t, ++n_tile) {
            const int j0 = w.start(t);
            if (!warp_wait_for(&sh.raw_full[slot], phase, &sh.abort)) return;
            const int there = sh.there[slot];
            if (!warp_wait_for(empty, (n_tile & 1) ^ 1, &sh.abort)) return;
            const char* from = raw + slot * Lay::kRaw;
#pragma unroll 4
            for (int r = row0; r < kTile; r += 128 / kChunks) {
                const int j = j0 + r;
                uint32_t x[kPlanes][4];
                const bool seen = chunk * 8 < p.a.D && j < w.high && (j >= w.low || j < w.sink) && (there >> (r >> box_shift)) & 1;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                if (seen) {
                    const float4* y = reinterpret_cast<const float4*>(from + (r * p.a.D + chunk * 8) * 4);
                    a = y[0];
                    b = y[1];
                }
                const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t u[kPlanes];
                    split(f[2 * c], f[2 * c + 1], u);
#pragma unroll
                    for (int i = 0; i < kPlanes; ++i) x[i][c] = u[i];
                }
                char* at = to + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);   // the 128-byte swizzle
#pragma unroll
                for (int i = 0; i < kPlanes; ++i)
                    *reinterpret_cast<uint4*>(at + i * Lay::kPlane) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&sh.raw_empty[slot]);
            }
            slot += 2;
            if (slot >= Lay::kRaws) {
                slot -= Lay::kRaws;
                phase ^= 1;
            }
        }
    }
}

// ---- warp 13: products ------------------------------------------------------------------
template <int DP>
__device__ __forceinline__ void f32_mma_role(const AttnParams& p, char* planes, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    const uint32_t k_at = desc_lo(smem_u32(planes), 1), v_at = desc_lo(smem_u32(planes) + kPlanes * Lay::kPlane, kTile * 128 >> 4);
    const int ksteps = (p.a.D + 15) / 16;
    const uint32_t qk = mma_desc(kTile, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t pv = mma_desc(DP, true);
    int items = 0, left = 0;
    bool first = false, done = false;
    unsigned n_qk = 0, n_pv = 0;
    int spins = 0;
    while (!done || n_pv != n_qk) {
        bool did = false;
        if (left == 0 && !done) {
            const int at = items % kSegments;
            if (all_test(&sh.seg_full[at], (items / kSegments) & 1)) {
                left = __reduce_max_sync(0xffffffffu, sh.seg[at].t1 - sh.seg[at].t0);
                if (elected()) mbar_arrive(&sh.seg_empty[at]);
                __syncwarp();
                done = left == 0;
                first = true;
                ++items;
                did = true;
            }
        }
        // S of tile n goes where S of tile n - 1 was, once that has been read
        if (left > 0 && n_qk - n_pv < 2 && all_test(&sh.k_full, n_qk & 1) && (n_qk == 0 || all_test(&sh.s_empty, (n_qk - 1) & 1)) &&
            (!first || all_test(&sh.q_full, (items - 1) & 1))) {
            tc_fence_after();
            first = false;
            --left;
            if (elected()) {
#pragma unroll
                for (int term = 0; term < kTerms; ++term) {
                    const uint32_t a = tmem + Lay::kQ + term_a(term) * (DP / 2), b = k_at + term_b(term) * (Lay::kPlane >> 4);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        if (k < ksteps)
                            mma_ts(tmem + Lay::kS, a + k * 8, desc(b + (k >> 2) * (kTile * 128 >> 4) + (k & 3) * 2, 1024 >> 4), qk,
                                   term > 0 || k > 0);
                }
                mma_commit(&sh.s_full);
                mma_commit(&sh.k_empty);
                if (left == 0) mma_commit(&sh.q_empty);
            }
            __syncwarp();
            ++n_qk;
            did = true;
        }
        if (n_pv != n_qk && all_test(&sh.p_full, n_pv & 1) && all_test(&sh.v_full, n_pv & 1)) {
            tc_fence_after();
            if (elected()) {
#pragma unroll
                for (int term = 0; term < kTerms; ++term) {
                    const uint32_t a = tmem + Lay::kP + term_a(term) * 32, b = v_at + term_b(term) * (Lay::kPlane >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ts(tmem + Lay::kO, a + k * 8, desc(b + k * (2048 >> 4), 1024 >> 4), pv, term > 0 || k > 0);
                }
                mma_commit(&sh.o_done);
                mma_commit(&sh.v_empty);
            }
            __syncwarp();
            ++n_pv;
            did = true;
        }
        spins = did ? 0 : spins + 1;
        if (spins == kTcSpinLimit) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
        if ((spins & 63) == 63 && __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&sh.abort) != 0)) {
            if (elected()) mma_commit(&sh.drain);
            __syncwarp();
            for (int n = 0; n < kTcSpinLimit / 64 && !all_test(&sh.drain, 0); ++n) {}
            return;
        }
    }
}

// ---- warps 0 to 3: softmax, scaling, output ---------------------------------------------
template <int DP>
__device__ __forceinline__ void f32_softmax_role(const AttnParams& p, float4* sums, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    unsigned n = 0;   // tiles of the CTA so far
    for (int n_seg = 0;; ++n_seg) {
        const int seg_at = n_seg % kSegments;
        if (!warp_wait_for(&sh.seg_full[seg_at], (n_seg / kSegments) & 1, &sh.abort)) return;
        const Segment w = sh.seg[seg_at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[seg_at]);
        if (w.t0 == w.t1) return;
        const int rows = w.rows;
        const int rr = w.r0 + min(tid, rows - 1), token = p.by_G.of(rr);
        const int at = w.len + token;
        const int low = p.a.window > 0 ? at + 1 - p.a.window : 0;
        const int at_first = w.len + p.by_G.of(w.r0), at_last = w.len + p.by_G.of(w.r0 + rows - 1);
        const bool work = warp * 32 < rows, mine = tid < rows;
        float m = -kInf, l = 0.f;
        float before = 1.f;   // scale of the sums so far, from the tile before to this one
        for (int t = w.t0; t < w.t1; ++t, ++n) {
            const int j0 = w.start(t);
            if (!warp_wait_for(&sh.s_full, n & 1, &sh.abort)) return;
            float s[kTile];
            if (work) {
                tc_fence_after();
                tmem_ld32(lanes + Lay::kS, reinterpret_cast<uint32_t*>(s));
                tmem_ld32(lanes + Lay::kS + 32, reinterpret_cast<uint32_t*>(s) + 32);
                tc_wait_ld();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_empty);   // the next tile's S may be written
            float scale_o = 1.f, base = 0.f;
            if (work) {
                const bool clean = j0 + kTile - 1 <= at_first &&
                                   (p.a.window <= 0 || j0 > at_last - p.a.window || j0 + kTile <= p.a.sinks);
                if (!clean) {
                    const int hi = at - j0, lo = low - j0, sk = p.a.sinks - j0;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!(c <= hi && (c >= lo || c < sk))) s[c] = -kInf;
                }
                float x[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
                for (int c = 0; c < kTile; c += 2) x[(c >> 1) & 3] = fmaxf(fmaxf(x[(c >> 1) & 3], s[c]), s[c + 1]);
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
                if (mine && top > m + 8.f) {
                    scale_o = m == -kInf ? 0.f : ex2(m - top);
                    m = top;
                    l *= scale_o;
                }
                base = m == -kInf ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < kTile; ++c) {
                    s[c] = ex2(fmaf(s[c], p.scale_log2, -base));
                    sum[c & 3] += s[c];
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            // the product before: P's planes are used up, and O may be scaled
            if (n > 0 && !warp_wait_for(&sh.o_done, (n - 1) & 1, &sh.abort)) return;
            if (work) {
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < kTile; c0 += 32) {
                    uint32_t pk[kPlanes][16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        uint32_t u[kPlanes];
                        split(s[c0 + c], s[c0 + c + 1], u);
#pragma unroll
                        for (int i = 0; i < kPlanes; ++i) pk[i][c / 2] = u[i];
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kPlanes; ++i) tmem_st16(lanes + Lay::kP + i * 32 + c0 / 2, pk[i]);
                }
                if (t > w.t0) {   // O of the tile before joins the sums (scaled to its maximum), or begins them
                    const bool more = t - w.t0 > 1;
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(lanes + Lay::kO + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float4* at = sums + (c + i) / 4 * kTcRows + tid;
                            float4 x = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                            if (more) {
                                const float4 y = *at;
                                x = make_float4(fmaf(y.x, before, x.x), fmaf(y.y, before, x.y), fmaf(y.z, before, x.z), fmaf(y.w, before, x.w));
                            }
                            *at = x;
                        }
                    }
                }
                before = scale_o;
                tc_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full);
        }
        if (!warp_wait_for(&sh.o_done, (n - 1) & 1, &sh.abort)) return;
        if (work) {
            tc_fence_after();
            float* const to = reinterpret_cast<float*>(p.a.out) + ((w.row0 + token) * p.a.Hq + w.head * p.G + rr - token * p.G) * (int64_t)p.a.D;
            float4* const part = p.part + (int64_t)w.slot * (p.a.D / 4) * p.rows + tid;
            const float inv = 1.f / l;
            if (mine && !w.whole) __stcg(p.ml + (int64_t)w.slot * p.rows + tid, make_float2(m, l));
            const bool summed = w.t1 - w.t0 > 1;
#pragma unroll 1
            for (int c0 = 0; c0 < p.a.D; c0 += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lanes + Lay::kO + c0, o);
                tc_wait_ld();
                if (mine) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        if (c0 + c >= p.a.D) break;
                        float4 x = make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]), __uint_as_float(o[c + 3]));
                        if (summed) {
                            const float4 y = sums[(c0 + c) / 4 * kTcRows + tid];
                            x = make_float4(fmaf(y.x, before, x.x), fmaf(y.y, before, x.y), fmaf(y.z, before, x.z), fmaf(y.w, before, x.w));
                        }
                        if (w.whole)
                            put4(to + c0 + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                        else
                            __stcg(part + (c0 + c) / 4 * p.rows, x);
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(kF32Threads, 1) attention_f32_kernel(const AttnParams p) {
    using Lay = F32Layout<DP>;
    extern __shared__ __align__(1024) char smem[];
    char* const planes = smem;
    char* const raw = smem + 2 * kPlanes * Lay::kPlane;
    float4* const sums = reinterpret_cast<float4*>(raw + Lay::kRaws * Lay::kRaw);
    F32Shared& sh = *reinterpret_cast<F32Shared*>(smem + Lay::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, cta = blockIdx.x;
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"((uint32_t)Lay::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < Lay::kRaws; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        uint64_t* four[] = {&sh.k_full, &sh.v_full, &sh.q_full, &sh.s_empty, &sh.p_full};   // four warps arrive
        for (int i = 0; i < 5; ++i) mbar_init(four[i], 4);
        uint64_t* one[] = {&sh.k_empty, &sh.v_empty, &sh.q_empty, &sh.s_full, &sh.o_done, &sh.drain};
        for (int i = 0; i < 6; ++i) mbar_init(one[i], 1);
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], 13);   // twelve warps and the products'
        }
        mbar_init_fence();
        sh.abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join, which waits for the whole grid
    if (tid == 0) p.desc[cta].rows = 0;
    find_start<kF32Threads>(p, cta, &sh.start, sh.scan, &sh.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) {
        f32_copy_role<DP>(p, raw, sh);
        write_status<float>(p, cta, sh.start.valid);
    } else if (warp == 13) {
        f32_mma_role<DP>(p, planes, sh);
    } else if (warp >= 8) {
        f32_split_role<DP, 1>(p, planes, raw, sh);
    } else if (warp >= 4) {
        f32_split_role<DP, 0>(p, planes, raw, sh);
    } else {
        f32_softmax_role<DP>(p, sums, sh);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"((uint32_t)Lay::kCols));
    }
    if (tid == 0 && sh.abort) write_timeout(p);
}

template <int DP>
static cudaError_t launch(const AttnParams& p, cudaStream_t s) {
    static std::atomic<int> ready[64];
    constexpr int bytes = F32Layout<DP>::kBytes + (int)sizeof(F32Shared);
    static_assert(bytes <= 232448, "shared memory of an SM");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(attention_f32_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_release);
    }
    return launch_after(attention_f32_kernel<DP>, dim3(p.ctas), dim3(kF32Threads), bytes, s, p);
}

cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s) { return p.a.D <= 64 ? launch<64>(p, s) : launch<128>(p, s); }

}  // namespace sv
