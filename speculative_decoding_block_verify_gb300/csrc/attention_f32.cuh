// Float32 attention on the tensor cores, heads up to 128: the roles that spec_paged_attention (attention_f32.cu) and
// spec_prompt_attention (prompt_f32.cu) share.
//
// A float32 is the sum of three bf16: x = x0 + x1 + x2 + O(2^-27 |x|), each the rounding of what the ones before
// leave.  A product of two such sums needs the six terms x0 y0, x0 y1, x1 y0, x1 y1, x0 y2, x2 y0 (the other three are
// below 2^-24 of x0 y0), each exact in float32, so six bf16 products with a float32 accumulator stand for a float32
// product.  At M = 128 a tile of 64 positions costs 48 of 32 cycles and 24 of 64, 3,072 tensor cycles, against about 2,800
// that its 64 KB take from memory; on the float pipes (128 products a cycle) 32 rows take 4,096 and 128 rows 16,384.  The price here is the same for
// any number of rows: up to about 20 the float pipes alone would need less (8 rows 1,024 cycles), which is not built for these heads.
//
// One CTA per SM, sixteen warps: copies (warp 15, beside those of the softmax's warps that have rows last) bring pages as they lie into a ring; warps 4 to 11 split the item's rows of
// Q into tensor memory and keys and values into swizzled bf16 planes (zeros where no row of the item sees a position,
// whatever the cache holds there); warps 13 and 14 issue the products; warps 0 to 3 hold a row per thread: softmax, and P split
// into three planes in tensor memory.
// There is one set of planes each for keys and values: a tile's keys are split during the product of the values before,
// and its values during its keys' product, so the tensor cores do not wait for either.
// The tensor cores cut their running sums off instead of rounding them: over 5,000 positions in one accumulator the output
// came out 1.7e-5 too small.  So every tile's P V is a product of its own, and the sums over tiles are rounded float32
// additions: 6e-7 off there, a third of what a float32 matrix product is.  Warps 4 to 11 hold them, half of a row per
// thread in DP / 2 registers, and the softmax hands them its scales through tensor memory.  (Sums in shared memory,
// added by the softmax's warps, took a third of a tile's time.)
//
// What bounds it: a tile takes about 4,600 cycles.  No pipe is full (issue slots a third, tensor cores two thirds); what it
// waits for is instructions.  Four different pieces of code run on each quarter of an SM, together more than is kept where
// instructions are fetched from, and every line of it that is not there costs a trip.  What made the code shorter made it
// faster: one piece of code for keys and values (122 -> 109 us for 16 streams of 2,100 and 5 tokens of 4 rows a key head), a
// subtraction of bf16 from float32 in one instruction (107 -> 103), waits that look for a given-up one every 16th time
// (103 -> 101), one wait less (98 -> 96), and products partly unrolled.  The same kernel with keys and values in warps of their own took 123 us.
// An infinite query, key or value counts as NaN here (the difference to its rounding is).

#pragma once

#include <atomic>

#include "host_util.h"
#include "tcgen05.cuh"

namespace sv {

constexpr int kF32Threads = 512;
// registers of a thread: softmax, splitting and sums (two warpgroups), copies and products
constexpr int kRegsSoftmax = 136, kRegsSplit = 152, kRegsRest = 72, kRegsLaunch = 128;
static_assert(kRegsSoftmax + 2 * kRegsSplit + kRegsRest <= 4 * kRegsLaunch, "setmaxnreg would wait for ever");
constexpr int kPlanes = 3;
constexpr int kTerms = 6;   // (plane of A, plane of B), the largest last
__host__ __device__ constexpr int term_a(int i) { return i == 0 ? 2 : i == 2 || i == 3 ? 1 : 0; }
__host__ __device__ constexpr int term_b(int i) { return i == 1 ? 2 : i == 2 || i == 4 ? 1 : 0; }

// DP: the head padded to 64 or 128 columns
template <int DP>
struct F32Layout {
    static constexpr int kPlane = DP / 64 * kTile * 128;          // one plane of 64 positions, [panel][64 rows][128 bytes]
    static constexpr int kRaw = kTile * DP * 4;                    // a tile as it lies
    static constexpr int kRaws = DP == 128 ? 4 : 8;
    static constexpr int kBytes = 2 * kPlanes * kPlane + kRaws * kRaw;
    // columns of tensor memory; kScale: two tiles' scale, maximum and sum of a row
    static constexpr int kQ = 0, kS = 192, kP = 256, kScale = 352, kO = 384, kCols = 512;
};

struct F32Shared {
    uint64_t raw_full[8], raw_empty[8];
    uint64_t k_full, k_empty, v_full;   // the planes; those of V are used up when O is there
    uint64_t q_full, q_empty, s_full, s_empty, p_full[2], o_done, drain[2];
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    int there[8];   // bit i: page i of the slot's tile is in the pool
    Start start;
    int64_t scan[kF32Threads / 32];
    int scratch;
    uint32_t tmem;
    int abort;
    int moved;   // tiles copied so far (prompts)
};

// x less the bf16 pair w, exact for the roundings below
__device__ __forceinline__ float2 less(float2 x, uint32_t w) {
    float2 y;
    asm("{\n\t.reg .b16 l, h, m;\n\tmov.b16 m, 0xBF80;\n\tmov.b32 {l, h}, %2;\n\t"   // m: -1
        "fma.rn.f32.bf16 %0, l, m, %3;\n\tfma.rn.f32.bf16 %1, h, m, %4;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "r"(w), "f"(x.x), "f"(x.y));
    return y;
}
// Two floats as three bf16 pairs.  The first rounding stops at bf16's largest number: a finite float above it, rounded to
// infinity, would leave NaN.
__device__ __forceinline__ void split(float2 x, uint32_t (&w)[kPlanes]) {
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(x.y), "f"(x.x));
    x = less(x, w[0]);
    w[1] = pack_bf16(x.x, x.y);
    x = less(x, w[1]);
    w[2] = pack_bf16(x.x, x.y);
}

// ---- warps 4 to 11: Q, keys and values into planes, the sums over tiles, output -----------------
// Each half of them takes half of a tile's positions, of Q's columns and of O's.  Keys go two tiles ahead of values: a tile's
// planes are free once the product before has used them, and then the other kind's product runs.  When a tile's O is there its
// planes of V are used up too; what an item's last tile has completed is written while the next item is computed.
// Keys and values share one piece of code: unrolled twice over it no longer fits where instructions are fetched from.
template <int DP>
__device__ __forceinline__ void f32_split_role(const AttnParams& p, char* planes, char* raw, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    constexpr int kHalf = DP / 2, kChunks = DP / 8;
    const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5, half = (threadIdx.x >> 7) - 1;
    const uint32_t lanes = sh.tmem + ((uint32_t)(warp * 32) << 16);
    const int part = tid % kChunks, box_shift = min(p.page_shift, 6);
    const bool q_vec = ((reinterpret_cast<uintptr_t>(p.a.q) | (uintptr_t)(p.a.q_row_stride * 4)) & 15) == 0;
    Segment wk = {}, wv = {}, was = {};   // the items of the next key and value tiles, and the one that the last value tile ended
    int tk = 0, tv = 0, segs_k = 0, segs_v = 0;
    unsigned nk = 0, nv = 0;              // tiles of the CTA so far
    bool k_end = false;
    float2 sum[kHalf / 2];
#pragma unroll
    for (int c = 0; c < kHalf / 2; ++c) sum[c] = make_float2(0.f, 0.f);
    auto next = [&](Segment& w, int& t, int& segs) {
        const int at = segs % kSegments;
        if (!warp_wait_for(&sh.seg_full[at], (segs / kSegments) & 1, &sh.abort)) return false;
        w = sh.seg[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[at]);
        ++segs;
        t = w.t0;
        return true;
    };
    for (int kv = 0;; kv ^= 1) {
        bool write = false, end = false;
        float m = 0.f, l = 1.f;
        int j0, high, low, sink;   // of the tile to split
        unsigned in;
        if (kv == 0) {
            if (k_end) continue;
            if (tk == wk.t1) {
                if (!next(wk, tk, segs_k)) return;
                k_end = wk.t0 == wk.t1;
                if (k_end) continue;
                // the item's rows of Q: a thread its row, the first columns on their way while the item before still uses its own
                const int rr = wk.r0 + min(tid, wk.rows - 1), token = p.by_G.of(rr);
                const float* q = reinterpret_cast<const float*>(p.a.q) + (wk.row0 + token) * p.a.q_row_stride +
                                 (int64_t)(wk.head * p.G + rr - token * p.G) * p.a.D;
#pragma unroll 1
                for (int c0 = half * kHalf; c0 < (half + 1) * kHalf; c0 += 32) {
                    float4 y[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (c0 + 4 * c < p.a.D) {
                            const float* from = q + c0 + 4 * c;
                            y[c] = q_vec ? *reinterpret_cast<const float4*>(from) : make_float4(from[0], from[1], from[2], from[3]);
                        }
                    }
                    if (c0 == half * kHalf) {
                        if (!warp_wait_for(&sh.q_empty, segs_k & 1, &sh.abort)) return;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        uint32_t x[kPlanes][8];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float4 f = y[side * 4 + c];
                            uint32_t u[kPlanes], v[kPlanes];
                            split(make_float2(f.x, f.y), u);
                            split(make_float2(f.z, f.w), v);
#pragma unroll
                            for (int i = 0; i < kPlanes; ++i) {
                                x[i][2 * c] = u[i];
                                x[i][2 * c + 1] = v[i];
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < kPlanes; ++i) tmem_st8(lanes + Lay::kQ + i * (DP / 2) + c0 / 2 + side * 8, x[i]);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }
            j0 = wk.start(tk++);
            high = wk.high;
            low = wk.low;
            sink = wk.sink;
            in = 2 * nk;   // keys and values alternate in the ring
        } else {
            if (nk < 2 && !k_end) continue;
            const bool first = tv == wv.t1;
            if (first) {
                was = wv;
                if (!next(wv, tv, segs_v)) return;
            }
            end = wv.t0 == wv.t1;
            if (nv > 0) {
                const unsigned before = nv - 1;
                // O, and the row's scale: its writers arrived before the product was issued
                if (!warp_wait_for(&sh.o_done, before & 1, &sh.abort)) return;
                write = first;
                if (warp * 32 < (first ? was.rows : wv.rows)) {
                    tc_fence_after();
                    uint32_t r[4];
                    tmem_ld4(lanes + Lay::kScale + (before & 1) * 4, r);
#pragma unroll
                    for (int c0 = 0; c0 < kHalf; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(lanes + Lay::kO + half * kHalf + c0, o);
                        tc_wait_ld();
                        const float2 scale = make_float2(__uint_as_float(r[0]), __uint_as_float(r[0]));
#pragma unroll
                        for (int c = 0; c < 32; c += 2)
                            sum[(c0 + c) / 2] = ffma2(sum[(c0 + c) / 2], scale, make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1])));
                    }
                    m = __uint_as_float(r[1]);
                    l = __uint_as_float(r[2]);
                    tc_fence_before();
                }
            }
            j0 = wv.start(tv++);
            high = wv.high;
            low = wv.low;
            sink = wv.sink;
            in = 2 * nv++ + 1;
        }
        if (!end) {
            const unsigned slot = in % Lay::kRaws;
            if (!warp_wait_for(&sh.raw_full[slot], (in / Lay::kRaws) & 1, &sh.abort)) return;
            if (kv == 0 && !warp_wait_for(&sh.k_empty, (nk++ & 1) ^ 1, &sh.abort)) return;
            const int there = sh.there[slot];
            const char* const from = raw + slot * Lay::kRaw;
            char* const to = planes + kv * kPlanes * Lay::kPlane + (part & 1) * 8;
            // a thread takes columns 4 part and DP / 2 + 4 part on of every kStep-th position of its half: neighbours read neighbours
            constexpr int kStep = 128 / kChunks;
#pragma unroll
            for (int i = 0; i < kTile / 2 / kStep; ++i) {
                const int r = half * (kTile / 2) + i * kStep + tid / kChunks, j = j0 + r;
                const bool seen = j < high && (j >= low || j < sink) && (there >> (r >> box_shift)) & 1;
                const float* const row = reinterpret_cast<const float*>(from) + r * p.a.D + 4 * part;
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (seen && side * kHalf + 4 * part < p.a.D) f = *reinterpret_cast<const float4*>(row + side * kHalf);
                    uint32_t u[kPlanes], v[kPlanes];
                    split(make_float2(f.x, f.y), u);
                    split(make_float2(f.z, f.w), v);
                    // panels of 64 columns, 128 bytes a row, their 16-byte pieces swizzled
                    const int piece = side * kHalf / 8 + part / 2;
                    char* const at = to + (piece >> 3) * (kTile * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
#pragma unroll
                    for (int k = 0; k < kPlanes; ++k) *reinterpret_cast<uint2*>(at + k * Lay::kPlane) = make_uint2(u[k], v[k]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(kv ? &sh.v_full : &sh.k_full);   // v_full: and O of the tile before is read
                mbar_arrive(&sh.raw_empty[slot]);
            }
        }
        if (write) {
            if (tid < was.rows) {
                const int rr = was.r0 + tid, token = p.by_G.of(rr);
                float* const to = reinterpret_cast<float*>(p.a.out) +
                                  ((was.row0 + token) * p.a.Hq + was.head * p.G + rr - token * p.G) * (int64_t)p.a.D;
                float4* const unjoined = p.part + (int64_t)was.slot * (p.a.D / 4) * p.rows + tid;
                const float inv = 1.f / l;
                if (half == 0 && !was.whole) __stcg(p.ml + (int64_t)was.slot * p.rows + tid, make_float2(m, l));
#pragma unroll
                for (int c = 0; c < kHalf; c += 4) {
                    const int col = half * kHalf + c;
                    if (col >= p.a.D) break;
                    const float2 x = sum[c / 2], y = sum[c / 2 + 1];
                    if (was.whole)
                        put4(to + col, make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv));
                    else
                        __stcg(unjoined + col / 4 * p.rows, make_float4(x.x, x.y, y.x, y.y));
                }
            }
#pragma unroll
            for (int c = 0; c < kHalf / 2; ++c) sum[c] = make_float2(0.f, 0.f);
            __syncwarp();
        }
        if (end) return;   // values, and with them the keys, are through
    }
}

// ---- warps 14 (S) and 13 (P V): products ----------------------------------------------------
// terms unrolled; measured at DP = 128 1 / 2 / 3 / 6: 101 / 99 / 101 / 106 us, at DP = 64 1 / 3 / 6: 82 / 69 / 69
constexpr int terms_unrolled(int dp) { return dp == 64 ? kTerms : 2; }
template <int DP>
__device__ __forceinline__ bool f32_keys_role(const AttnParams& p, char* planes, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    const uint32_t k_at = desc_lo(smem_u32(planes), 1);
    const int ksteps = (p.a.D + 15) / 16;
    const uint32_t qk = mma_desc(kTile, false) | (p.a.scale < 0.f ? 1u << 13 : 0u);
    unsigned n = 0;
    for (int item = 0;; ++item) {
        const int at = item % kSegments;
        if (!warp_wait_for(&sh.seg_full[at], (item / kSegments) & 1, &sh.abort)) return false;
        int left = __reduce_max_sync(0xffffffffu, sh.seg[at].t1 - sh.seg[at].t0);
        if (elected()) mbar_arrive(&sh.seg_empty[at]);
        __syncwarp();
        if (left == 0) return true;
        if (!warp_wait_for(&sh.q_full, item & 1, &sh.abort)) return false;
        for (; left > 0; --left, ++n) {
            // S of tile n goes where S of tile n - 1 was, once that has been read
            if (n > 0 && !warp_wait_for(&sh.s_empty, (n - 1) & 1, &sh.abort)) return false;
            if (!warp_wait_for(&sh.k_full, n & 1, &sh.abort)) return false;
            tc_fence_after();
            if (elected()) {
#pragma unroll(terms_unrolled(DP))
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
                if (left == 1) mma_commit(&sh.q_empty);
            }
            __syncwarp();
        }
    }
}
template <int DP>
__device__ __forceinline__ bool f32_values_role(char* planes, F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const uint32_t tmem = __reduce_or_sync(0xffffffffu, sh.tmem);
    const uint32_t v_at = desc_lo(smem_u32(planes) + kPlanes * Lay::kPlane, kTile * 128 >> 4);
    constexpr uint32_t pv = mma_desc(DP, true);
    unsigned n = 0;
    for (int item = 0;; ++item) {
        const int at = item % kSegments;
        if (!warp_wait_for(&sh.seg_full[at], (item / kSegments) & 1, &sh.abort)) return false;
        int left = __reduce_max_sync(0xffffffffu, sh.seg[at].t1 - sh.seg[at].t0);
        if (elected()) mbar_arrive(&sh.seg_empty[at]);
        __syncwarp();
        if (left == 0) return true;
        for (; left > 0; --left, ++n) {
            if (!warp_wait_for(&sh.p_full[n & 1], (n >> 1) & 1, &sh.abort)) return false;
            if (!warp_wait_for(&sh.v_full, n & 1, &sh.abort)) return false;
            tc_fence_after();
            if (elected()) {
#pragma unroll(terms_unrolled(DP))
                for (int term = 0; term < kTerms; ++term) {
                    const uint32_t a = tmem + Lay::kP + term_a(term) * 32, b = v_at + term_b(term) * (Lay::kPlane >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ts(tmem + Lay::kO, a + k * 8, desc(b + k * (2048 >> 4), 1024 >> 4), pv, term > 0 || k > 0);
                }
                mma_commit(&sh.o_done);
            }
            __syncwarp();
        }
    }
}

// ---- warps 0 to 3: softmax, P ------------------------------------------------------------
template <int DP>
__device__ __forceinline__ void f32_softmax_role(const AttnParams& p, F32Shared& sh) {
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
        for (int t = w.t0; t < w.t1; ++t, ++n) {
            const int j0 = w.start(t);
            if (!warp_wait_for(&sh.s_full, n & 1, &sh.abort)) return;
            if (!work) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty);
                if (n > 0 && !warp_wait_for(&sh.o_done, (n - 1) & 1, &sh.abort)) return;
            } else {
                float s[kTile];
                tc_fence_after();
                tmem_ld32(lanes + Lay::kS, reinterpret_cast<uint32_t*>(s));
                tmem_ld32(lanes + Lay::kS + 32, reinterpret_cast<uint32_t*>(s) + 32);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty);   // the next tile's S may be written
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
                float scale_o = 1.f;
                if (mine && top > m + 8.f) {
                    scale_o = m == -kInf ? 0.f : ex2(m - top);
                    m = top;
                    l *= scale_o;
                }
                const float base = m == -kInf ? 0.f : m;
                const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[kPlanes][kTile / 2];
#pragma unroll
                for (int c = 0; c < kTile; c += 2) {
                    float2 y = ffma2(make_float2(s[c], s[c + 1]), sc, nb);
                    y = make_float2(ex2(y.x), ex2(y.y));
                    sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], y);
                    uint32_t u[kPlanes];
                    split(y, u);
#pragma unroll
                    for (int i = 0; i < kPlanes; ++i) pk[i][c / 2] = u[i];
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                // the product before: P's planes are used up
                if (n > 0 && !warp_wait_for(&sh.o_done, (n - 1) & 1, &sh.abort)) return;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kPlanes; ++i) tmem_st32(lanes + Lay::kP + i * 32, pk[i]);
                tmem_st4(lanes + Lay::kScale + (n & 1) * 4, __float_as_uint(scale_o), __float_as_uint(m), __float_as_uint(l), 0);
                tc_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[n & 1]);
        }
    }
}

// Tensor memory and barriers, before the CTA's first __syncthreads.  `listeners`: warps that a segment is told.
template <int DP>
__device__ __forceinline__ void f32_begin(F32Shared& sh, int listeners) {
    using Lay = F32Layout<DP>;
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"((uint32_t)Lay::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < Lay::kRaws; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 8);
        }
        uint64_t* eight[] = {&sh.k_full, &sh.v_full, &sh.q_full};   // warps that arrive
        for (int i = 0; i < 3; ++i) mbar_init(eight[i], 8);
        uint64_t* four[] = {&sh.s_empty, &sh.p_full[0], &sh.p_full[1]};
        for (int i = 0; i < 3; ++i) mbar_init(four[i], 4);
        uint64_t* one[] = {&sh.k_empty, &sh.q_empty, &sh.s_full, &sh.o_done, &sh.drain[0], &sh.drain[1]};
        for (int i = 0; i < 6; ++i) mbar_init(one[i], 1);
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], listeners);
        }
        mbar_init_fence();
        sh.abort = sh.moved = 0;
    }
}
template <int DP>
__device__ __forceinline__ void f32_end(F32Shared& sh) {
    using Lay = F32Layout<DP>;
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x >> 5 == 13) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"((uint32_t)Lay::kCols));
    }
}

// Shared memory of the device's kernel, once; an error where its registers are not what the warpgroups share out.
template <typename K>
static cudaError_t f32_ready(K kernel, int bytes, std::atomic<int> (&ready)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes of;
        e = cudaFuncGetAttributes(&of, kernel);
        if (e != cudaSuccess) return e;
        if (of.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;   // the warpgroups' shares would not add up
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace sv
