// spec_paged_attention: the entry point, and the kernel on the float pipes.
//
//   out[row] = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = scale log2(e) q . k_j,  m = max_j s_j
//
// in one pass over the visible keys: a row keeps its running maximum m, its sum l and its weighted
// values o; when a tile raises m to m', l and o are scaled by 2^(m - m').  Parts of an item over
// disjoint keys join by the same rule: with M = max m_k, out = sum 2^(m_k - M) o_k / sum 2^(m_k - M) l_k.

#include "attention.cuh"
#include "host_util.h"

#include <atomic>
#include <cmath>

namespace sv {

// ---------------------------------------------------------------------------------------
// The kernel on the float pipes: float32 caches, and rows that are not 16-byte aligned.
// ---------------------------------------------------------------------------------------
// 256 threads: TK along the keys (then along the columns of the values), 256 / TK along the rows;
// a thread owns RM rows and 64 / TK keys of a tile.  Q, K, V tiles and the weights are in shared memory as
// float32.  K rows are padded by 4 floats, so that the 16-byte loads of eight neighbouring threads fall into
// different banks.
constexpr int kFloatThreads = 256;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<unsigned short>(unsigned short x) { return __uint_as_float((uint32_t)x << 16); }

static size_t float_smem(int rows, int D) {
    return sizeof(float) * ((size_t)rows * (D + 4) + 2 * (size_t)kTile * (D + 4) + (size_t)rows * (kTile + 4));
}

// Four elements as float32.
template <typename T>
__device__ __forceinline__ float4 load4(const T* x, bool vec);
template <>
__device__ __forceinline__ float4 load4<float>(const float* x, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const float4*>(x));
    return make_float4(__ldg(x), __ldg(x + 1), __ldg(x + 2), __ldg(x + 3));
}
template <>
__device__ __forceinline__ float4 load4<unsigned short>(const unsigned short* x, bool vec) {
    if (vec) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(x));
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
    return make_float4(to_float(__ldg(x)), to_float(__ldg(x + 1)), to_float(__ldg(x + 2)), to_float(__ldg(x + 3)));
}

template <typename T, int R, int TK, int ND>
__global__ void __launch_bounds__(kFloatThreads) attention_float_kernel(const AttnParams p, int q_vec) {
    constexpr int TR = kFloatThreads / TK, RM = R / TR, KN = kTile / TK;
    extern __shared__ __align__(16) float fsm[];
    __shared__ Start s_start;
    __shared__ int64_t s_scan[kFloatThreads / 32];
    __shared__ int s_int;
    const int tid = threadIdx.x, tk = tid % TK, tr = tid / TK;
    const int D = p.a.D, pitch = D + 4;
    float* qs = fsm;
    float* ks = qs + R * pitch;
    float* vs = ks + kTile * pitch;
    float* ps = vs + kTile * pitch;
    constexpr int ppitch = kTile + 4;
    const int cta = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    find_start<kFloatThreads>(p, cta, &s_start, s_scan, &s_int);
    if (tid < 32) write_status<T>(p, cta, s_start.valid);
    Walk w;
    if (!w.start(p, s_start)) return;
    const T* q = reinterpret_cast<const T*>(p.a.q);
    const T* kp = reinterpret_cast<const T*>(p.a.k_pages);
    const T* vp = reinterpret_cast<const T*>(p.a.v_pages);
    const int nd4 = D / 4;
    do {
        const int rows = w.it.r1 - w.it.r0;
        const int64_t row0 = first_row(p.a.cu_drafts, w.b, p.a.kmax);
        __syncthreads();
        for (int u = tid; u < R * nd4; u += kFloatThreads) {
            const int r = u / nd4, c = (u - r * nd4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int rr = w.it.r0 + r, i = rr / p.G;
                x = load4<T>(q + (row0 + i) * p.a.q_row_stride + (int64_t)(w.h * p.G + rr - i * p.G) * D + c, q_vec);
            }
            *reinterpret_cast<float4*>(qs + r * pitch + c) = x;
        }
        float m[RM], l[RM];
        float4 o[RM][ND];
        int at[RM];
#pragma unroll
        for (int a = 0; a < RM; ++a) {
            m[a] = -kInf;
            l[a] = 0.f;
            at[a] = w.len + (w.it.r0 + min(tr + a * TR, rows - 1)) / p.G;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[a][d] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int t = w.t0; t < w.t1; ++t) {
            const int j0 = tile_start(w.it, t);
            __syncthreads();   // the tile before has been read
            for (int u = tid; u < kTile * nd4; u += kFloatThreads) {
                const int k = u / nd4, c = (u - k * nd4) * 4;
                const int j = j0 + k;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                // positions that no row of the item sees are zeros, whatever the cache holds there
                if (j < w.it.high && (j >= w.it.low || j < w.it.sink)) {
                    const int page = __ldg(p.a.page_table + (int64_t)w.b * p.a.max_pages + (j >> p.page_shift));
                    if ((unsigned)page < (unsigned)p.a.num_pages) {
                        const int64_t off =
                            (((int64_t)page * p.a.Hkv + w.h) * p.a.page_size + (j & (p.a.page_size - 1))) * D + c;
                        x = load4<T>(kp + off, true);
                        y = load4<T>(vp + off, true);
                    }
                }
                *reinterpret_cast<float4*>(ks + k * pitch + c) = x;
                *reinterpret_cast<float4*>(vs + k * pitch + c) = y;
            }
            __syncthreads();
            float s[RM][KN];
#pragma unroll
            for (int a = 0; a < RM; ++a)
#pragma unroll
                for (int b = 0; b < KN; ++b) s[a][b] = 0.f;
#pragma unroll 2
            for (int c = 0; c < D; c += 4) {
                float4 x[RM], y[KN];
#pragma unroll
                for (int a = 0; a < RM; ++a) x[a] = *reinterpret_cast<const float4*>(qs + (tr + a * TR) * pitch + c);
#pragma unroll
                for (int b = 0; b < KN; ++b) y[b] = *reinterpret_cast<const float4*>(ks + (tk + b * TK) * pitch + c);
#pragma unroll
                for (int a = 0; a < RM; ++a)
#pragma unroll
                    for (int b = 0; b < KN; ++b)
                        s[a][b] = fmaf(x[a].x, y[b].x, fmaf(x[a].y, y[b].y, fmaf(x[a].z, y[b].z, fmaf(x[a].w, y[b].w, s[a][b]))));
            }
#pragma unroll
            for (int a = 0; a < RM; ++a) {
                float hi = -kInf;
#pragma unroll
                for (int b = 0; b < KN; ++b) {
                    s[a][b] = visible(p, at[a], j0 + tk + b * TK) ? s[a][b] * p.scale_log2 : -kInf;
                    hi = fmaxf(hi, s[a][b]);
                }
#pragma unroll
                for (int x = TK / 2; x > 0; x >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, x));
                const float mm = fmaxf(m[a], hi);
                const float base = mm == -kInf ? 0.f : mm;   // nothing visible yet: every weight is 2^-inf = 0
                const float keep = exp2f(m[a] - base);
                m[a] = mm;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < KN; ++b) {
                    const float e = exp2f(s[a][b] - base);
                    sum += e;
                    ps[(tr + a * TR) * ppitch + tk + b * TK] = e;
                }
#pragma unroll
                for (int x = TK / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[a] = l[a] * keep + sum;
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    o[a][d].x *= keep;
                    o[a][d].y *= keep;
                    o[a][d].z *= keep;
                    o[a][d].w *= keep;
                }
            }
            __syncwarp();   // the TK threads of a row lie in one warp
#pragma unroll 2
            for (int k = 0; k < kTile; k += 4) {
                float4 e[RM];
#pragma unroll
                for (int a = 0; a < RM; ++a) e[a] = *reinterpret_cast<const float4*>(ps + (tr + a * TR) * ppitch + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const int c = (tk + d * TK) * 4;
                        if (c < D) {
                            const float4 y = *reinterpret_cast<const float4*>(vs + (k + kk) * pitch + c);
#pragma unroll
                            for (int a = 0; a < RM; ++a) {
                                const float f = kk == 0 ? e[a].x : kk == 1 ? e[a].y : kk == 2 ? e[a].z : e[a].w;
                                o[a][d].x = fmaf(f, y.x, o[a][d].x);
                                o[a][d].y = fmaf(f, y.y, o[a][d].y);
                                o[a][d].z = fmaf(f, y.z, o[a][d].z);
                                o[a][d].w = fmaf(f, y.w, o[a][d].w);
                            }
                        }
                    }
                }
            }
        }
        const bool whole = w.whole();
        const int64_t slot = w.slot(cta);
#pragma unroll
        for (int a = 0; a < RM; ++a) {
            const int r = tr + a * TR;
            if (r >= rows) continue;
            if (whole) {
                const int rr = w.it.r0 + r, i = rr / p.G;
                T* to = reinterpret_cast<T*>(p.a.out) + ((row0 + i) * p.a.Hq + w.h * p.G + rr - i * p.G) * (int64_t)D;
                const float inv = 1.f / l[a];
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int c = (tk + d * TK) * 4;
                    if (c < D) put4(to + c, make_float4(o[a][d].x * inv, o[a][d].y * inv, o[a][d].z * inv, o[a][d].w * inv));
                }
            } else {
                if (tk == 0) __stcg(p.ml + slot * p.rows + r, make_float2(m[a], l[a]));
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int c = (tk + d * TK) * 4;
                    if (c < D) __stcg(p.part + (slot * nd4 + c / 4) * p.rows + r, o[a][d]);
                }
            }
        }
        if (!whole) join_parts<T, kFloatThreads, 1>(p, w, cta, s_start.span, tid, &s_int);
    } while (w.next(p));
}

// ---------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------
struct DeviceInfo {
    std::atomic<int> sms{0};
};
static DeviceInfo g_device[64];

static int sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return set_cuda_error(e, "spec_paged_attention");
    int n = dev >= 0 && dev < 64 ? g_device[dev].sms.load(std::memory_order_acquire) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return set_cuda_error(e, "spec_paged_attention");
        if (dev >= 0 && dev < 64) g_device[dev].sms.store(n, std::memory_order_release);
    }
    *sms = n;
    return SPEC_OK;
}

// Rows of a group and CTAs of the grid.
static void cut(const spec_attention_args* a, int sms, int* rows, int* ctas) {
    const int64_t need = (int64_t)(a->kmax + 1) * (a->Hq / a->Hkv);
    const bool tensor = tensor_path(a);
    *rows = tensor ? tensor_rows(a) : need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : 64;
    int64_t n = (tensor ? tensor_ctas_per_sm(a) : 2) * (int64_t)sms;
    // no more CTAs than the longest possible contexts have tiles
    const int64_t groups = (need + *rows - 1) / *rows;
    const int64_t tiles = groups * a->B * a->Hkv * (((int64_t)a->max_pages * a->page_size + kTile - 1) / kTile);
    if (n > tiles) n = tiles;
    if (n > kMaxCtas) n = kMaxCtas;
    *ctas = (int)n;
}

static int check(const spec_attention_args* a) {
    if (!valid_dtype(a->dtype)) return set_error(SPEC_ERR_DTYPE, "spec_paged_attention: dtype %d", a->dtype);
    if (a->B < 0 || a->B > SPEC_MAX_STREAMS || a->kmax < 0 || a->kmax > SPEC_MAX_KMAX)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: B = %d, kmax = %d", a->B, a->kmax);
    if (a->Hkv < 1 || a->Hq < 1 || a->Hq > 1024 || a->Hq % a->Hkv != 0)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: Hq = %d, Hkv = %d", a->Hq, a->Hkv);
    if (a->D < 8 || a->D > SPEC_MAX_HEAD || a->D % 8 != 0)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: D = %d", a->D);
    if (a->page_size < 8 || a->page_size > SPEC_MAX_PAGE || (a->page_size & (a->page_size - 1)) != 0 || a->num_pages < 1 ||
        a->max_pages < 1 || (int64_t)a->max_pages * a->page_size > INT32_MAX)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: page_size = %d, num_pages = %d, max_pages = %d",
                         a->page_size, a->num_pages, a->max_pages);
    if (a->window < 0 || a->sinks < 0)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: window = %d, sinks = %d", a->window, a->sinks);
    return SPEC_OK;
}

static size_t layout(const spec_attention_args* a, int rows, int ctas, AttnParams* p) {
    char* base = reinterpret_cast<char*>(a->workspace);
    auto take = [](size_t* at, size_t bytes) {
        const size_t from = *at;
        *at += (bytes + 255) & ~(size_t)255;
        return from;
    };
    // the arrival counts of the largest grid come first, so that every call finds them where it left them
    size_t at = 256;
    const size_t arrived = take(&at, (size_t)kJoinLevels * 2 * kMaxCtas * sizeof(int32_t));
    const size_t ml = take(&at, (size_t)kJoinLevels * 2 * ctas * rows * sizeof(float2));
    const size_t part = take(&at, (size_t)2 * ctas * rows * a->D * sizeof(float));
    if (p != nullptr) {
        p->timeout = reinterpret_cast<int32_t*>(base);
        p->arrived = reinterpret_cast<int32_t*>(base + arrived);
        p->ml = reinterpret_cast<float2*>(base + ml);
        p->part = reinterpret_cast<float4*>(base + part);
    }
    return at;
}

template <typename T, int R, int TK, int ND>
static cudaError_t launch_float(const AttnParams& p, cudaStream_t s, bool q_vec) {
    const size_t smem = float_smem(R, p.a.D);
    const cudaError_t e = cudaFuncSetAttribute(attention_float_kernel<T, R, TK, ND>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(attention_float_kernel<T, R, TK, ND>, dim3(p.ctas), dim3(kFloatThreads), smem, s, p, (int)q_vec);
}

template <typename T, int R, int TK>
static cudaError_t launch_float_d(const AttnParams& p, cudaStream_t s, bool q_vec) {
    const int nd = (p.a.D / 4 + TK - 1) / TK;
    if (nd == 1) return launch_float<T, R, TK, 1>(p, s, q_vec);
    if (nd == 2) return launch_float<T, R, TK, 2>(p, s, q_vec);
    return launch_float<T, R, TK, 64 / TK>(p, s, q_vec);
}

template <typename T>
static cudaError_t launch_float_r(const AttnParams& p, cudaStream_t s, bool q_vec) {
    if (p.rows == 8) return launch_float_d<T, 8, 32>(p, s, q_vec);
    if (p.rows == 16) return launch_float_d<T, 16, 16>(p, s, q_vec);
    if (p.rows == 32) return launch_float_d<T, 32, 16>(p, s, q_vec);
    return launch_float_d<T, 64, 16>(p, s, q_vec);
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_paged_attention_workspace_bytes(const spec_attention_args* a) {
    clear_error();
    if (a == nullptr || check(a) != SPEC_OK || a->B == 0) return 0;
    int sms = 0, rows = 0, ctas = 0;
    if (sm_count(&sms) != SPEC_OK) return 0;
    cut(a, sms, &rows, &ctas);
    return layout(a, rows, ctas, nullptr);
}

extern "C" int spec_paged_attention(const spec_attention_args* a, void* stream) {
    clear_error();
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "spec_paged_attention: args is NULL");
    int rc = check(a);
    if (rc != SPEC_OK) return rc;
    if (a->q_row_stride < (int64_t)a->Hq * a->D)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: q_row_stride is below Hq * D");
    if (a->q_rows < 0 || (a->cu_drafts == nullptr && a->q_rows < (int64_t)a->B * (a->kmax + 1)))
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: q_rows = %lld", (long long)a->q_rows);
    if (a->B == 0) return SPEC_OK;
    if (a->length == nullptr || a->page_table == nullptr || a->q == nullptr || a->k_pages == nullptr ||
        a->v_pages == nullptr || a->out == nullptr || a->status == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_paged_attention: a required pointer is NULL");
    if (((uintptr_t)a->k_pages | (uintptr_t)a->v_pages) & 15)
        return set_error(SPEC_ERR_ARG, "spec_paged_attention: the pool is not 16-byte aligned");
    if ((uintptr_t)a->out & 15) return set_error(SPEC_ERR_ARG, "spec_paged_attention: out is not 16-byte aligned");
    if (!std::isfinite(a->scale)) return set_error(SPEC_ERR_ARG, "spec_paged_attention: scale is not finite");
    int sms = 0;
    AttnParams p;
    if ((rc = sm_count(&sms)) != SPEC_OK) return rc;
    cut(a, sms, &p.rows, &p.ctas);
    const size_t need = layout(a, p.rows, p.ctas, nullptr);
    if (a->workspace == nullptr || ((uintptr_t)a->workspace & 15) || a->workspace_bytes < need)
        return set_error(SPEC_ERR_WORKSPACE, "spec_paged_attention: workspace needs %zu bytes, 16-byte aligned", need);
    layout(a, p.rows, p.ctas, &p);
    p.a = *a;
    p.G = a->Hq / a->Hkv;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
    p.scale_log2 = (float)((double)a->scale * kLog2e);
    const bool tensor = tensor_path(a);
    if (tensor) p.scale_log2 = std::fabs(p.scale_log2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int es = a->dtype == SPEC_DTYPE_F32 ? 4 : 2;
    const bool q_vec = (((uintptr_t)a->q | (uintptr_t)(a->q_row_stride * es)) & (4 * es - 1)) == 0;
    cudaError_t e = tensor                         ? launch_attention_tc(p, s)
                    : a->dtype == SPEC_DTYPE_F32 ? launch_float_r<float>(p, s, q_vec)
                                                 : launch_float_r<unsigned short>(p, s, q_vec);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_paged_attention");
}
