// spec_prompt_attention on the tensor cores: float32 heads up to 128.
//
// The kernel of the paged attention (attention_f32.cuh) with another source: tiles of 64 keys and values come from packed rows
// by one tiled copy each, and the items are pieces of prompts (prompt.cuh), whole ones, so nothing is joined.  Five prompts of 100 to 1,500
// tokens, 32/8 heads of 128: 279 to 289 us, 188 to 195 TFLOP/s, with six bf16 products for each float32 one 0.60 to 0.62 of the measured bf16 rate (the walk and
// the copies in one warp: 282 us where this took 276); the tensor cores are busy for 53 % of the cycles, and the softmax with its split into three parts is what they wait for.
#include "attention_f32.cuh"
#include "prompt.cuh"
#include "tensor_map.h"

namespace sv {

static __device__ int32_t g_mark;   // a wait gave up since it was last cleared
static __global__ void mark_kernel(int32_t marked) { g_mark = marked; }
cudaError_t mark_prompt_f32(int32_t marked, cudaStream_t s) {
    mark_kernel<<<1, 1, 0, s>>>(marked);
    return cudaGetLastError();
}

// ---- warp 12: the walk over the CTA's items ------------------------------------------------
__device__ __forceinline__ void prompt_f32_walk_role(const PromptParams& p, F32Shared& sh, PromptWalk& w) {
    Piece it = {};
    w.start();
    for (int told = 0;; ++told) {
        const bool any = w.next(p, &it);
        Segment& seg = sh.seg[told % kSegments];
        if (!warp_wait_moving(&sh.seg_empty[told % kSegments], ((told / kSegments) & 1) ^ 1, &sh.abort, &sh.moved)) return;
        if ((threadIdx.x & 31) == 0) {
            // the piece's first token is the block's
            if (any) {
                const Keys keys = keys_of<kTile>(p, it.at, it.tokens);
                seg = {0, keys.tiles, keys.sink_tiles, keys.first_tile, keys.low, keys.high, keys.sink, it.at, 0, it.tokens * p.G, it.head, 1, 0,
                       it.row0 + it.at};
            } else {
                seg.t0 = seg.t1 = 0;
            }
            mbar_arrive(&sh.seg_full[told % kSegments]);
        }
        __syncwarp();
        if (!any) return;
    }
}

// ---- warp 15: keys and values --------------------------------------------------------------
template <int DP>
__device__ __forceinline__ void prompt_f32_copy_role(const PromptParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap, char* raw,
                                                     F32Shared& sh) {
    using Lay = F32Layout<DP>;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(raw);
    const unsigned bytes = kTile * p.a.D * 4;
    const uint64_t stay = l2_evict_normal_policy();
    int slot = 0;
    unsigned phase = 1;
    bool ok = true;
    auto copy = [&](const CUtensorMap* map, int head, int row) {
        ok = ok && warp_wait_for(&sh.raw_empty[slot], phase, &sh.abort);
        if (!ok) return;
        if (lane == 0) {
            sh.there[slot] = 1;
            mbar_expect_tx(&sh.raw_full[slot], bytes);
            tma_load_3d(ring + slot * Lay::kRaw, map, 0, head, row, &sh.raw_full[slot], stay);
        }
        __syncwarp();
        if (++slot == Lay::kRaws) {
            slot = 0;
            phase ^= 1;
        }
    };
    for (int n_seg = 0; ok; ++n_seg) {
        const int place = n_seg % kSegments;
        ok = warp_wait_for(&sh.seg_full[place], (n_seg / kSegments) & 1, &sh.abort);
        if (!ok) break;
        const Segment w = sh.seg[place];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[place]);
        if (w.t0 == w.t1) return;
        const int row0 = (int)w.row0 - w.len;   // the prompt's first row
        for (int t = 0; t < w.t1 && ok; ++t) {
            copy(kmap, w.head, row0 + w.start(t));
            copy(vmap, w.head, row0 + w.start(t));
            if (lane == 0) *reinterpret_cast<volatile int*>(&sh.moved) += 1;
        }
    }
    // gave up: whatever was copied must have arrived before the CTA's memory is given back
    for (int s = 0; s < Lay::kRaws; ++s)
        for (int n = 0; n < kTcSpinLimit / 64 && !mbar_try_wait(&sh.raw_full[s], (s < slot ? phase : phase ^ 1) ^ 1); ++n) {}
}

template <int DP>
__global__ void __launch_bounds__(kF32Threads, 1) prompt_f32_kernel(const PromptParams pp, const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap) {
    using Lay = F32Layout<DP>;
    extern __shared__ __align__(1024) char smem[];
    char* const planes = smem;
    char* const raw = smem + 2 * kPlanes * Lay::kPlane;
    F32Shared& sh = *reinterpret_cast<F32Shared*>(smem + Lay::kBytes);
    const int warp = threadIdx.x >> 5;
    f32_begin<DP>(sh, 23);   // softmax 4, keys 8, values 8, products 2, copies
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= 12) {
        registers_down<kRegsRest>();
        if (warp == 15) {
            prompt_f32_copy_role<DP>(pp, &kmap, &vmap, raw, sh);
        } else if (warp == 14) {
            if (!f32_keys_role<DP>(p, planes, sh)) drain(&sh.drain[0]);
        } else if (warp == 13) {
            if (!f32_values_role<DP>(planes, sh)) drain(&sh.drain[1]);
        } else {
            PromptWalk w;
            prompt_f32_walk_role(pp, sh, w);
            prompt_statuses(pp, w, &g_mark);
        }
    } else if (warp >= 4) {
        registers_up<kRegsSplit>();
        f32_split_role<DP>(p, planes, raw, sh);
    } else {
        registers_up<kRegsSoftmax>();
        f32_softmax_role<DP>(p, sh);
    }
    f32_end<DP>(sh);
    if (warp == 15 && sh.abort) prompt_gave_up<float>(pp, __int_as_float(0x7fffffff), &g_mark);
}

// [rows][Hkv][D] in boxes of a head and 64 rows.
static bool encode_rows(CUtensorMap* map, const void* base, const spec_prompt_args& a, int64_t stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.D * 4, (cuuint64_t)stride * 4};
    const cuuint32_t box[3] = {(cuuint32_t)a.D, 1, kTile};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_SWIZZLE_NONE, base, 3, dims, strides, box);
}

template <int DP>
static cudaError_t launch(const PromptParams& pp, int sms, cudaStream_t s) {
    static std::atomic<int> ready[64];
    constexpr int bytes = F32Layout<DP>::kBytes + (int)sizeof(F32Shared);
    static_assert(bytes <= 232448, "shared memory of an SM");
    const cudaError_t e = f32_ready(prompt_f32_kernel<DP>, bytes, ready);
    if (e != cudaSuccess) return e;
    CUtensorMap k, v;
    if (!encode_rows(&k, pp.a.k, pp.a, pp.a.k_row_stride) || !encode_rows(&v, pp.a.v, pp.a, pp.a.v_row_stride)) return cudaErrorInvalidValue;
    AttnParams p = {};   // what the shared roles read
    p.a.Hq = pp.a.Hq;
    p.a.Hkv = pp.a.Hkv;
    p.a.D = pp.a.D;
    p.a.window = pp.a.window;
    p.a.sinks = pp.a.sinks;
    p.a.scale = pp.a.scale;
    p.a.q = pp.a.q;
    p.a.q_row_stride = pp.a.q_row_stride;
    p.a.out = pp.a.out;
    p.G = pp.G;
    p.by_G = pp.by_G;
    p.rows = pp.group * pp.G;
    p.page_shift = 6;   // a tile is one page
    p.scale_log2 = pp.scale_log2;
    return launch_after(prompt_f32_kernel<DP>, dim3((unsigned)prompt_ctas(pp, sms)), dim3(kF32Threads), bytes, s, pp, p, k, v);
}

cudaError_t launch_prompt_f32(const PromptParams& p, int sms, cudaStream_t s) { return p.a.D <= 64 ? launch<64>(p, sms, s) : launch<128>(p, sms, s); }

}  // namespace sv
