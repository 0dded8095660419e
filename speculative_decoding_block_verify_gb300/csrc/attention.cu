// spec_paged_attention: the entry point, the kernel on the float pipes, and the join.
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
// The kernel on the float pipes: float32 heads of more than 128.
// ---------------------------------------------------------------------------------------
// 256 threads: TK along the keys (then along the columns of the values), 256 / TK along the rows;
// a thread owns RM rows and 64 / TK keys of a tile.  Q, K, V tiles and the weights are in shared memory, rows padded by
// 4 floats, so that the 16-byte loads of eight neighbouring threads fall into different banks.  The copies are
// asynchronous: the next tile's keys arrive during this tile's second product, its values during the next one's first.
// It is bound by shared memory and the float pipes: a tile of 64 positions and 256 columns takes 12,300 cycles of the latter for 48 rows.
// Products two at a time (even and odd columns) 427 -> 369 us for 16 streams of 2,100 and 5 tokens of 8 rows a key head; groups of 48 rows
// for what 32 do not hold, instead of 64, 369 -> 248; one CTA an SM where two do not fit, one token each 118 -> 107.
constexpr int kFloatThreads = 256;

static size_t float_smem(int rows, int D) {
    return sizeof(float) * ((size_t)rows * (D + 4) + 2 * (size_t)kTile * (D + 4) + (size_t)rows * (kTile + 4));
}

// 16 bytes to shared memory, or zeros where `there` is false (nothing is read then)
__device__ __forceinline__ void cp_async16_or_zero(void* to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}

template <int R, int TK, int ND>
__global__ void __launch_bounds__(kFloatThreads, R < 48 ? 2 : 1) attention_float_kernel(const AttnParams p, int q_vec) {
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join, which waits for the whole grid
    if (tid == 0) p.desc[cta].rows = 0;
    find_start<kFloatThreads>(p, cta, &s_start, s_scan, &s_int);
    Walk w;
    const bool any = w.start(p, s_start);
    if (tid < 32) write_status<float>(p, cta, s_start.valid);
    if (!any) return;
    const float* q = reinterpret_cast<const float*>(p.a.q);
    const float* pool[2] = {reinterpret_cast<const float*>(p.a.k_pages), reinterpret_cast<const float*>(p.a.v_pages)};
    const int nd4 = D / 4;
    // copies: a thread keeps to one position of the tile, four neighbouring threads share it
    const int my_row = tid >> 2, my_col = tid & 3;
    do {
        const int rows = w.it.r1 - w.it.r0;
        const int64_t row0 = first_row(p.a.cu_drafts, w.b, p.a.kmax);
        const int32_t* table = p.a.page_table + (int64_t)w.b * p.a.max_pages;
        // where the thread's position of tile t lies in the pool, or -1
        auto look_up = [&](int t) -> int64_t {
            if (t >= w.t1) return -1;
            const int j = tile_start(w.it, t) + my_row;
            // positions that no row of the item sees are zeros, whatever the cache holds there
            if (j >= w.it.high || (j < w.it.low && j >= w.it.sink)) return -1;
            const int page = *(table + (j >> p.page_shift));
            if ((unsigned)page >= (unsigned)p.a.num_pages) return -1;
            return (((int64_t)page * p.a.Hkv + w.h) * p.a.page_size + (j & (p.a.page_size - 1))) * D;
        };
        auto copy = [&](int kv, int64_t at, bool any) {   // a group of copies, empty past the item's last tile
            float* to = (kv ? vs : ks) + my_row * pitch;
            const float* from = pool[kv] + max((int64_t)0, at);
            for (int c = any ? my_col : nd4; c < nd4; c += 4) cp_async16_or_zero(to + 4 * c, from + 4 * c, at >= 0);
            cp_async_commit();
        };
        int64_t at_now = look_up(w.t0), at_next = look_up(w.t0 + 1);
        __syncthreads();   // the item before has been read
        copy(0, at_now, true);
        copy(1, at_now, true);
        for (int u = tid; u < R * nd4; u += kFloatThreads) {
            const int r = u / nd4, c = (u - r * nd4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int rr = w.it.r0 + r, i = p.by_G.of(rr);
                const float* from = q + (row0 + i) * p.a.q_row_stride + (int64_t)(w.h * p.G + rr - i * p.G) * D + c;
                x = q_vec ? *reinterpret_cast<const float4*>(from)
                          : make_float4(*(from), *(from + 1), *(from + 2), *(from + 3));
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
            at[a] = w.len + p.by_G.of(w.it.r0 + min(tr + a * TR, rows - 1));
#pragma unroll
            for (int d = 0; d < ND; ++d) o[a][d] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int t = w.t0; t < w.t1; ++t) {
            const int j0 = tile_start(w.it, t);
            const int64_t at_after = look_up(t + 2);
            cp_async_wait<1>();   // the keys
            __syncthreads();
            float2 pair[RM][KN];   // of even and odd columns
#pragma unroll
            for (int a = 0; a < RM; ++a)
#pragma unroll
                for (int b = 0; b < KN; ++b) pair[a][b] = make_float2(0.f, 0.f);
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
                        pair[a][b] = ffma2(make_float2(x[a].x, x[a].y), make_float2(y[b].x, y[b].y),
                                           ffma2(make_float2(x[a].z, x[a].w), make_float2(y[b].z, y[b].w), pair[a][b]));
            }
            float s[RM][KN];
#pragma unroll
            for (int a = 0; a < RM; ++a) {
                float hi = -kInf;
#pragma unroll
                for (int b = 0; b < KN; ++b) {
                    s[a][b] = visible(p, at[a], j0 + tk + b * TK) ? (pair[a][b].x + pair[a][b].y) * p.scale_log2 : -kInf;
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
            __syncthreads();   // every row's weights are written, and the keys are read
            copy(0, at_next, t + 1 < w.t1);
            cp_async_wait<1>();   // the values
            __syncthreads();
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
                                const float2 u = ffma2(make_float2(f, f), make_float2(y.x, y.y), make_float2(o[a][d].x, o[a][d].y));
                                const float2 v = ffma2(make_float2(f, f), make_float2(y.z, y.w), make_float2(o[a][d].z, o[a][d].w));
                                o[a][d] = make_float4(u.x, u.y, v.x, v.y);
                            }
                        }
                    }
                }
            }
            __syncthreads();
            copy(1, at_next, t + 1 < w.t1);
            at_next = at_after;
        }
        const bool whole = w.whole();
        if (tid == 0 && w.begins_part()) p.desc[cta] = w.unjoined(p, cta, s_start.span);
        const int64_t slot = w.slot(cta);
#pragma unroll
        for (int a = 0; a < RM; ++a) {
            const int r = tr + a * TR;
            if (r >= rows) continue;
            if (whole) {
                const int rr = w.it.r0 + r, i = p.by_G.of(rr);
                float* to = reinterpret_cast<float*>(p.a.out) + ((row0 + i) * p.a.Hq + w.h * p.G + rr - i * p.G) * (int64_t)D;
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
    } while (w.next(p));
    cp_async_wait<0>();
}

// ---------------------------------------------------------------------------------------
// The join
// ---------------------------------------------------------------------------------------
// Every unjoined item has rows * D / 4 columns (four values of a row), a thread each:
//   M = max m_k,  out = sum 2^(m_k - M) o_k / sum 2^(m_k - M) l_k
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;   // parts whose loads are on their way at a time

// Four values of one row of an item that is being joined: its running maximum, sum and weighted values.
struct JoinSum {
    float m = -kInf, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void rise(float big) {   // to a maximum of `big`
        const float keep = ex2(m - (big == -kInf ? 0.f : big));   // -inf: no part has seen a key
        m = big;
        sum *= keep;
        y = make_float4(y.x * keep, y.y * keep, y.z * keep, y.w * keep);
    }
    __device__ __forceinline__ void add(float2 x, float4 o) {
        const float f = ex2(x.x - (m == -kInf ? 0.f : m));
        sum = fmaf(f, x.y, sum);
        y = make_float4(fmaf(f, o.x, y.x), fmaf(f, o.y, y.y), fmaf(f, o.z, y.z), fmaf(f, o.w, y.w));
    }
    // parts [k0, k1) of the item that CTA c begins, N loads on their way at a time
    template <int N>
    __device__ __forceinline__ void parts(const AttnParams& p, int c, int k0, int k1, int r, int col) {
#pragma unroll 1
        for (; k0 < k1; k0 += N) {
            float2 x[N];
            float4 o[N];
            float big = m;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = make_float2(-kInf, 0.f);
                o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + i < k1) {
                    const int64_t slot = 2 * (c + k0 + i) + (k0 + i == 0 ? 1 : 0);
                    x[i] = __ldcg(p.ml + slot * p.rows + r);
                    o[i] = __ldcg(p.part + (slot * (p.a.D / 4) + col) * p.rows + r);
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) big = fmaxf(big, x[i].x);
            rise(big);
#pragma unroll
            for (int i = 0; i < N; ++i) add(x[i], o[i]);
        }
    }
    template <typename T>
    __device__ __forceinline__ void write(const AttnParams& p, const Unjoined& d, int r, int col) const {
        const int rr = d.r0 + r, token = p.by_G.of(rr);
        T* out = reinterpret_cast<T*>(p.a.out) + ((d.row0 + token) * p.a.Hq + d.head * p.G + rr - token * p.G) * (int64_t)p.a.D + 4 * col;
        const float inv = 1.f / sum;
        put4(out, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    }
};

// Many items, so few parts each: CTA (c, y) takes columns of the item that CTA c began.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Unjoined d = p.desc[blockIdx.x];
    const int u = blockIdx.y * kJoinThreads + threadIdx.x;
    if (u >= d.rows * (p.a.D / 4)) return;
    const int col = u / d.rows, r = u - col * d.rows;
    JoinSum j;
    j.parts<4>(p, blockIdx.x, 0, d.parts, r, col);
    j.write<T>(p, d, r, col);
}

// Few items, so many parts each: the columns of all items are spread evenly over the grid, and `slices` threads
// share a column, each with its share of the parts in order.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attention_join_spread_kernel(const AttnParams p) {
    __shared__ int s_scan[kMaxCtas];   // columns before item c
    __shared__ int s_warp[kJoinThreads / 32];
    __shared__ float4 s_o[kJoinThreads];
    __shared__ float2 s_ml[kJoinThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nc = p.a.D / 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int total = 0;
    {   // prefix sums over the items: two neighbouring ones per thread
        static_assert(2 * kJoinThreads == kMaxCtas, "an item per entry");
        int n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) n[i] = 2 * tid + i < p.ctas ? __ldcg(&p.desc[2 * tid + i].rows) * nc : 0;
        int x = n[0] + n[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int before = x - n[0] - n[1];
        for (int w = 0; w < kJoinThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
        s_scan[2 * tid] = before;
        s_scan[2 * tid + 1] = before + n[0];
        __syncthreads();
    }
    if (total == 0) return;
    int slices = 1;
    while (slices < 16 && (int64_t)total * slices * 2 <= (int64_t)gridDim.x * kJoinThreads) slices *= 2;
    const int columns = kJoinThreads / slices;   // of the CTA at a time: neighbouring threads have neighbouring columns
    const int slice = tid / columns, mine = tid - slice * columns;
    for (int u0 = blockIdx.x * columns; u0 < total; u0 += gridDim.x * columns) {
        const int u = u0 + mine;
        JoinSum j;
        int r = 0, col = 0;
        Unjoined d;
        if (u < total) {
            int c = 0, hi = kMaxCtas;   // the item of column u: the last one that begins at or before it
            while (hi - c > 1) {
                const int mid = (c + hi) / 2;
                if (s_scan[mid] <= u)
                    c = mid;
                else
                    hi = mid;
            }
            d = p.desc[c];
            col = (u - s_scan[c]) / d.rows;
            r = u - s_scan[c] - col * d.rows;
            const int each = (d.parts + slices - 1) / slices;
            j.parts<kJoinAhead>(p, c, slice * each, min((slice + 1) * each, d.parts), r, col);
        }
        if (slices > 1) {   // the slices of a column, in order
            s_o[tid] = j.y;
            s_ml[tid] = make_float2(j.m, j.sum);
            __syncthreads();
            if (slice == 0) {
                float big = j.m;
                for (int i = 1; i < slices; ++i) big = fmaxf(big, s_ml[i * columns + mine].x);
                j.rise(big);
                for (int i = 1; i < slices; ++i) j.add(s_ml[i * columns + mine], s_o[i * columns + mine]);
            }
            __syncthreads();
        }
        if (u < total && slice == 0) j.write<T>(p, d, r, col);
    }
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

constexpr int kTensorF32 = 128;   // float32 heads up to here go to the tensor cores

// Rows of a group and CTAs of the grid.
static void cut(const spec_attention_args* a, int sms, int* rows, int* ctas) {
    const int64_t need = (int64_t)(a->kmax + 1) * (a->Hq / a->Hkv);
    const bool bf16 = a->dtype == SPEC_DTYPE_BF16, tensor = bf16 || a->D <= kTensorF32;
    if (tensor) {
        *rows = tensor_rows(a);
    } else {   // as few groups as hold the rows, and those alike
        const int64_t each = (need + (need + 63) / 64 - 1) / ((need + 63) / 64);
        *rows = each <= 8 ? 8 : each <= 16 ? 16 : each <= 32 ? 32 : each <= 48 ? 48 : 64;
    }
    const bool two = !tensor && *rows < 48 && 2 * (float_smem(*rows, a->D) + 1024) <= 228 * 1024;
    int64_t n = (bf16 ? tensor_ctas_per_sm(a) : two ? 2 : 1) * (int64_t)sms;   // as many as are resident
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
    if (a->Hq / a->Hkv > 128)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: %d query heads per key head", a->Hq / a->Hkv);
    if (a->D < 8 || a->D > SPEC_MAX_HEAD || a->D % 8 != 0)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: D = %d", a->D);
    if (a->page_size < 8 || a->page_size > SPEC_MAX_PAGE || (a->page_size & (a->page_size - 1)) != 0 || a->num_pages < 1 ||
        a->max_pages < 1 || (int64_t)a->max_pages * a->page_size > INT32_MAX)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: page_size = %d, num_pages = %d, max_pages = %d",
                         a->page_size, a->num_pages, a->max_pages);
    if (a->dtype == SPEC_DTYPE_BF16 && (int64_t)a->num_pages * a->Hkv > INT32_MAX - 1)   // the copies' last coordinate
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: num_pages * Hkv = %lld", (long long)a->num_pages * a->Hkv);
    if (a->window < 0 || a->sinks < 0)
        return set_error(SPEC_ERR_SHAPE, "spec_paged_attention: window = %d, sinks = %d", a->window, a->sinks);
    return SPEC_OK;
}

static size_t layout(const spec_attention_args* a, int rows, int ctas, AttnParams* p, void** q_packed) {
    char* base = reinterpret_cast<char*>(a->workspace);
    auto take = [](size_t* at, size_t bytes) {
        const size_t from = *at;
        *at += (bytes + 255) & ~(size_t)255;
        return from;
    };
    size_t at = 256;
    const size_t desc = take(&at, (size_t)ctas * sizeof(Unjoined));
    const size_t ml = take(&at, (size_t)2 * ctas * rows * sizeof(float2));
    const size_t part = take(&at, (size_t)2 * ctas * rows * a->D * sizeof(float));
    const bool pack = a->dtype == SPEC_DTYPE_BF16 && !tensor_q(a);
    const size_t packed = take(&at, pack ? (size_t)(a->q_rows > 0 ? a->q_rows : 0) * a->Hq * a->D * 2 : 0);
    if (p != nullptr) {
        *q_packed = pack ? base + packed : nullptr;
        p->timeout = reinterpret_cast<int32_t*>(base);
        p->desc = reinterpret_cast<Unjoined*>(base + desc);
        p->ml = reinterpret_cast<float2*>(base + ml);
        p->part = reinterpret_cast<float4*>(base + part);
    }
    return at;
}

template <int R, int TK, int ND>
static cudaError_t launch_float(const AttnParams& p, cudaStream_t s, bool q_vec) {
    static std::atomic<int> ready[64];   // whether the device's kernel has its shared memory
    const int smem = (int)float_smem(R, p.a.D);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev].load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(attention_float_kernel<R, TK, ND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)float_smem(R, 4 * TK * ND));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(1, std::memory_order_release);
    }
    return launch_after(attention_float_kernel<R, TK, ND>, dim3(p.ctas), dim3(kFloatThreads), smem, s, p, (int)q_vec);
}

static cudaError_t launch_float_r(const AttnParams& p, cudaStream_t s, bool q_vec) {
    if (p.rows == 8) return launch_float<8, 32, 2>(p, s, q_vec);
    if (p.rows == 16) return launch_float<16, 16, 4>(p, s, q_vec);
    if (p.rows == 32) return launch_float<32, 16, 4>(p, s, q_vec);
    if (p.rows == 48) return launch_float<48, 16, 4>(p, s, q_vec);
    return launch_float<64, 16, 4>(p, s, q_vec);
}

template <typename T>
static cudaError_t launch_join(const AttnParams& p, int sms, cudaStream_t s) {
    const int64_t columns = (int64_t)p.rows * (p.a.D / 4);
    const int64_t need = (int64_t)(p.a.kmax + 1) * p.G;
    const int64_t items = (int64_t)p.a.B * p.a.Hkv * ((need + p.rows - 1) / p.rows);
    const int64_t tiles = ((int64_t)p.a.max_pages * p.a.page_size + kTile - 1) / kTile;
    // Parts of an item at most, lengths alike.  One stream of 131,072 tokens, 6 rows x 8 heads: with 1, 4 and 8 key heads
    // (304, 76, 38 parts) the whole call takes 27.1, 52.8, 89.5 us with the spread join and 55.5, 60.7, 92.4 us with the
    // other; 16 parts of a 1,003-token call take 12.3 and 11.1 us, and the 64-stream verify step 102.8 and 97.4 us.
    const int64_t parts = p.ctas / items < tiles ? p.ctas / items : tiles;
    if (parts < 32)
        return launch_after(attention_join_kernel<T>, dim3((unsigned)p.ctas, (unsigned)((columns + kJoinThreads - 1) / kJoinThreads)),
                            dim3(kJoinThreads), 0, s, p);
    const int64_t ctas = (columns * p.ctas + kJoinThreads - 1) / kJoinThreads;
    return launch_after(attention_join_spread_kernel<T>, dim3((unsigned)(ctas < 4 * sms ? ctas : 4 * sms)), dim3(kJoinThreads), 0, s, p);
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_paged_attention_workspace_bytes(const spec_attention_args* a) {
    clear_error();
    if (a == nullptr || check(a) != SPEC_OK || a->B == 0) return 0;
    int sms = 0, rows = 0, ctas = 0;
    if (sm_count(&sms) != SPEC_OK) return 0;
    cut(a, sms, &rows, &ctas);
    return layout(a, rows, ctas, nullptr, nullptr);
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
    if (!std::isfinite(a->scale) || !std::isfinite((float)((double)a->scale * kLog2e)))   // scores are taken to base 2
        return set_error(SPEC_ERR_ARG, "spec_paged_attention: scale is not finite");
    int sms = 0;
    AttnParams p;
    if ((rc = sm_count(&sms)) != SPEC_OK) return rc;
    cut(a, sms, &p.rows, &p.ctas);
    const size_t need = layout(a, p.rows, p.ctas, nullptr, nullptr);
    if (a->workspace == nullptr || ((uintptr_t)a->workspace & 15) || a->workspace_bytes < need)
        return set_error(SPEC_ERR_WORKSPACE, "spec_paged_attention: workspace needs %zu bytes, 16-byte aligned", need);
    void* q_packed = nullptr;
    layout(a, p.rows, p.ctas, &p, &q_packed);
    p.a = *a;
    p.G = a->Hq / a->Hkv;
    p.by_G = divisor(p.G);
    p.by_rows = divisor(p.rows);
    p.page_shift = 0;
    while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
    p.scale_log2 = (float)((double)a->scale * kLog2e);
    // the tensor-core kernels negate Q for a negative scale, and multiply masked scores of -inf by it
    if (a->dtype == SPEC_DTYPE_BF16 || a->D <= kTensorF32) p.scale_log2 = a->scale == 0.f ? 1e-30f : std::fabs(p.scale_log2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (a->dtype == SPEC_DTYPE_BF16) {
        p.item_cost = 2;
        e = launch_attention_tc(p, q_packed, s);
        if (e == cudaSuccess) e = launch_join<unsigned short>(p, sms, s);
    } else {
        p.item_cost = 1;
        e = a->D <= kTensorF32 ? launch_attention_f32(p, s) : launch_float_r(p, s, (((uintptr_t)a->q | (uintptr_t)(a->q_row_stride * 4)) & 15) == 0);
        if (e == cudaSuccess) e = launch_join<float>(p, sms, s);
    }
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_paged_attention");
}
