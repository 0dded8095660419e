// spec_paged_attention on the tensor cores: float32 caches, heads up to 128 (attention_f32.cuh says how).
#include "attention_f32.cuh"

namespace sv {

// ---- warp 15: the walk over the CTA's items, and the copies --------------------------------
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
        if (lane >= pages || j >= w.it.high || (j <= w.it.low - box && j >= w.it.sink)) return -1;
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

template <int DP>
__global__ void __launch_bounds__(kF32Threads, 1) attention_f32_kernel(const AttnParams p) {
    using Lay = F32Layout<DP>;
    extern __shared__ __align__(1024) char smem[];
    char* const planes = smem;
    char* const raw = smem + 2 * kPlanes * Lay::kPlane;
    F32Shared& sh = *reinterpret_cast<F32Shared*>(smem + Lay::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, cta = blockIdx.x;
    f32_begin<DP>(sh, 22);   // softmax 4, keys 8, values 8, products 2
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join, which waits for the whole grid
    if (tid == 0) p.desc[cta].rows = 0;
    find_start<kF32Threads>(p, cta, &sh.start, sh.scan, &sh.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= 12) {
        registers_down<kRegsRest>();
        if (warp == 15) {
            f32_copy_role<DP>(p, raw, sh);
            write_status<float>(p, cta, sh.start.valid);
        } else if (warp == 14) {
            if (!f32_keys_role<DP>(p, planes, sh)) drain(&sh.drain[0]);
        } else if (warp == 13) {
            if (!f32_values_role<DP>(planes, sh)) drain(&sh.drain[1]);
        }
    } else if (warp >= 4) {
        registers_up<kRegsSplit>();
        f32_split_role<DP>(p, planes, raw, sh);
    } else {
        registers_up<kRegsSoftmax>();
        f32_softmax_role<DP>(p, sh);
    }
    f32_end<DP>(sh);
    if (tid == 0 && sh.abort) write_timeout(p);
}

template <int DP>
static cudaError_t launch(const AttnParams& p, cudaStream_t s) {
    static std::atomic<int> ready[64];
    constexpr int bytes = F32Layout<DP>::kBytes + (int)sizeof(F32Shared);
    static_assert(bytes <= 232448, "shared memory of an SM");
    const cudaError_t e = f32_ready(attention_f32_kernel<DP>, bytes, ready);
    if (e != cudaSuccess) return e;
    return launch_after(attention_f32_kernel<DP>, dim3(p.ctas), dim3(kF32Threads), bytes, s, p);
}

cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s) { return p.a.D <= 64 ? launch<64>(p, s) : launch<128>(p, s); }

}  // namespace sv
