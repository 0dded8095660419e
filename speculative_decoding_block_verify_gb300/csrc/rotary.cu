// Rotary positions: spec_rotate, spec_cache_append_rotated, and the host's frequencies.
//
// A head's pair (a, b) j at position p turns by the angle p f_j:
//   a' = m (a cos - b sin),   b' = m (b cos + a sin).
// The angle is kept in turns, as a 64-bit fraction: with T_j = 2^64 f_j / 2 pi the product p T_j modulo 2^64 is the
// fraction of the turn, so whole turns fall away exactly, in two integer multiplications, at any position.  (In float32 an angle of
// 131,072 radians is known to 0.008; the product here is off by p 2^-56 turns, the rounding of T_j.)  The nearest quarter
// turn is taken off in integers as well, and what is left, at most an eighth, goes to sincospif.
//
// Bound by memory: a row's sines and cosines are computed once, by a warp, into shared memory and serve all its heads; every element
// is read and written once, 16 bytes a thread.

#include <cmath>

#include "blocks.cuh"
#include "divisor.cuh"
#include "host_util.h"

namespace sv {

constexpr int kTurnThreads = 256;
constexpr int kTurnRows = kTurnThreads / 32;       // rows of a CTA: a warp prepares one
constexpr int kTurnPairs = SPEC_MAX_HEAD / 2;

// How a head is cut: units of 16 bytes (halves: 16 bytes of either half), or of one pair or element.
struct Turn {
    const uint64_t* turns;
    int D, pairs;
    int turning;        // units of a head that turn; the others are copied
    int units, copies;  // units of a head that turns, and of one that is copied as it is (values)
    Divisor by_units, by_copies;
    float magnitude;
};

__device__ __forceinline__ float2 cos_sin(int p, uint64_t turns, float m) {
    const uint64_t at = (uint64_t)(int64_t)p * turns;
    const uint32_t quarter = (uint32_t)((at + (1ull << 61)) >> 62) & 3u;
    const int64_t rest = (int64_t)(at - ((uint64_t)quarter << 62));   // within an eighth of a turn
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (quarter & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * m, s * m);
}

// Sines and cosines of one row, by a warp.
__device__ __forceinline__ void prepare_row(const Turn& t, int p, float2* cs) {
    for (int j = threadIdx.x & 31; j < t.pairs; j += 32) cs[j] = cos_sin(p, t.turns[j], t.magnitude);
}

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) { return make_float2(a * cs.x - b * cs.y, b * cs.x + a * cs.y); }

// What a thread moves in one step.
template <typename T>
struct Wide;
template <>
struct Wide<unsigned short> {
    static constexpr int kPer = 8;
    float x[8];
    __device__ __forceinline__ void load(const unsigned short* p) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(u[i]);
            x[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    __device__ __forceinline__ uint4 pack() const {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Wide<float> {
    static constexpr int kPer = 4;
    float x[4];
    __device__ __forceinline__ void load(const float* p) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    }
    __device__ __forceinline__ uint4 pack() const {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
__device__ __forceinline__ float value(unsigned short x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ void store(unsigned short* p, float x) { *p = __bfloat16_as_ushort(__float2bfloat16(x)); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }

// Unit u of a head, to one place or two (also == nullptr: one).  `from` may be a destination: what a thread writes is what it read.
template <typename T, bool kWide, bool kPairs>
__device__ __forceinline__ void turn_unit(const Turn& t, const float2* cs, int u, const T* from, T* to, T* also) {
    if constexpr (kWide) {
        constexpr int per = Wide<T>::kPer;
        if (u < t.turning) {
            if constexpr (kPairs) {
                Wide<T> w;
                w.load(from + u * per);
#pragma unroll
                for (int i = 0; i < per; i += 2) {
                    const float2 y = turned(w.x[i], w.x[i + 1], cs[(u * per + i) / 2]);
                    w.x[i] = y.x;
                    w.x[i + 1] = y.y;
                }
                const uint4 y = w.pack();
                *reinterpret_cast<uint4*>(to + u * per) = y;
                if (also != nullptr) *reinterpret_cast<uint4*>(also + u * per) = y;
            } else {
                Wide<T> a, b;
                a.load(from + u * per);
                b.load(from + t.pairs + u * per);
#pragma unroll
                for (int i = 0; i < per; ++i) {
                    const float2 y = turned(a.x[i], b.x[i], cs[u * per + i]);
                    a.x[i] = y.x;
                    b.x[i] = y.y;
                }
                const uint4 y = a.pack(), z = b.pack();
                *reinterpret_cast<uint4*>(to + u * per) = y;
                *reinterpret_cast<uint4*>(to + t.pairs + u * per) = z;
                if (also != nullptr) {
                    *reinterpret_cast<uint4*>(also + u * per) = y;
                    *reinterpret_cast<uint4*>(also + t.pairs + u * per) = z;
                }
            }
        } else {
            const int at = 2 * t.pairs + (u - t.turning) * per;
            const uint4 y = *reinterpret_cast<const uint4*>(from + at);
            *reinterpret_cast<uint4*>(to + at) = y;
            if (also != nullptr) *reinterpret_cast<uint4*>(also + at) = y;
        }
    } else if (u < t.turning) {
        const int i = kPairs ? 2 * u : u, j = kPairs ? 2 * u + 1 : u + t.pairs;
        const float2 y = turned(value(from[i]), value(from[j]), cs[u]);
        store(to + i, y.x);
        store(to + j, y.y);
        if (also != nullptr) {
            store(also + i, y.x);
            store(also + j, y.y);
        }
    } else {
        const int at = t.pairs + u;
        const T y = from[at];
        to[at] = y;
        if (also != nullptr) also[at] = y;
    }
}

// ---------------------------------------------------------------------------------------
// rows at given positions
// ---------------------------------------------------------------------------------------
template <typename T, bool kWide, bool kPairs>
__global__ void __launch_bounds__(kTurnThreads) rotate_kernel(const spec_rotate_args a, const Turn t, int rows_each, int units_each) {
    __shared__ float2 s_cs[kTurnRows][kTurnPairs];
    const int tid = threadIdx.x, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int rows = (int)min((int64_t)rows_each, a.rows - row0);
    if (warp < rows) prepare_row(t, *(a.positions + row0 + warp), s_cs[warp]);
    __syncthreads();
    const int first = blockIdx.y * units_each, n = min(units_each, a.heads * t.units - first);
    for (int r = 0, u = tid;; u += kTurnThreads) {
        while (u >= n && r < rows) {
            u -= n;
            ++r;
        }
        if (r >= rows) return;
        const int head = t.by_units.of(first + u), c = first + u - head * t.units;
        const T* from = reinterpret_cast<const T*>(a.x) + (row0 + r) * a.x_row_stride + head * t.D;
        T* to = reinterpret_cast<T*>(a.out) + (row0 + r) * a.out_row_stride + head * t.D;
        turn_unit<T, kWide, kPairs>(t, s_cs[r], c, from, to, (T*)nullptr);
    }
}

// ---------------------------------------------------------------------------------------
// append with rotation
// ---------------------------------------------------------------------------------------
// The grid is cut by packed rows, not by streams: a prompt's thousands of rows and a decode step's few spread alike.  Each of a
// CTA's up to eight rows is prepared by a warp (its stream, position, page, sines), then all threads move the rows' queries, keys
// and values.  A stream's status is the business of one warp somewhere in the grid.
__device__ __forceinline__ int64_t stream_row(const spec_append_rotated_args& a, int b) {
    return a.cu == nullptr ? (int64_t)b * a.max_rows : (int64_t)*(a.cu + b) + (int64_t)b * a.extra_rows;
}
__device__ __forceinline__ int64_t stream_rows(const spec_append_rotated_args& a, int b) {
    return a.cu == nullptr ? a.max_rows : (int64_t)*(a.cu + b + 1) - *(a.cu + b) + a.extra_rows;
}
// Offsets that break the packing at stream b: it and the streams behind it are not defined.
__device__ __forceinline__ bool broken(const spec_append_rotated_args& a, int b, int64_t row0, int64_t n) {
    return n < 0 || n < a.extra_rows || n > a.max_rows || (b == 0 && row0 != 0) || row0 + n > a.rows;
}

// Whether (and why not) stream b, whose offsets are good, is written; the warp decides together.
__device__ __forceinline__ int append_refusal(const spec_append_rotated_args& a, int b, int64_t n, int shift, int* len_out) {
    const int lane = threadIdx.x & 31;
    const int len = __ldcg(a.length + b);
    *len_out = len;
    if (a.reserved != nullptr) {
        const int st = __ldcg(a.reserved + b);
        if (st != SPEC_ST_OK) return st;
    }
    if (len < 0 || len + n > (int64_t)a.max_pages << shift) return SPEC_ST_BAD_LENGTH;
    if (a.reserved != nullptr && n > 0 && (len & (a.page_size - 1)) != 0) {
        // a page that a stream which got no copy of it holds too, with more tokens in it (see append_kernel)
        const int32_t* table = a.page_table + (len >> shift);
        const int mine = *(table + (int64_t)b * a.max_pages);
        bool other = false;
        for (int o = lane; o < a.B; o += 32)
            other |= __ldcg(a.reserved + o) == SPEC_ST_NO_PAGES && __ldcg(a.length + o) > len && *(table + (int64_t)o * a.max_pages) == mine;
        if (__any_sync(0xffffffffu, other)) return SPEC_ST_NO_PAGES;
    }
    return SPEC_ST_OK;
}

template <typename T, bool kWide, bool kPairs>
__global__ void __launch_bounds__(kTurnThreads) append_rotated_kernel(const spec_append_rotated_args a, const Turn t, int rows_each, int units_each) {
    __shared__ float2 s_cs[kTurnRows][kTurnPairs];
    __shared__ int s_stream[kTurnRows], s_page[kTurnRows], s_offset[kTurnRows];   // page -2: the row is left alone
    __shared__ int s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = __ffs(a.page_size) - 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < kTurnRows) s_stream[tid] = INT32_MAX;
    if (tid == 0) s_first = a.B;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int rows = (int)max((int64_t)0, min((int64_t)rows_each, a.rows - row0));
    const bool reports = blockIdx.y == 0 && (int64_t)blockIdx.x * kTurnRows < a.B;   // this CTA writes statuses: it looks at all offsets
    // a stream's rows lie behind those of the streams before it, so a thread whose stream begins past the CTA's rows is done
    for (int b = tid; b < a.B; b += kTurnThreads) {
        const int64_t at = stream_row(a, b), n = stream_rows(a, b);
        if (broken(a, b, at, n)) {
            atomicMin(&s_first, b);
            break;
        }
        for (int64_t r = max(at, row0); r < min(at + n, row0 + rows); ++r) atomicMin(&s_stream[r - row0], b);
        if (at >= row0 + rows && !reports) break;
    }
    __syncthreads();
    const int first_broken = s_first;
    if (warp < rows) {
        const int b = s_stream[warp];
        int page = -2, at = 0;
        if (b < first_broken) {
            int len;
            const int64_t i = row0 + warp - stream_row(a, b);
            if (append_refusal(a, b, stream_rows(a, b), shift, &len) == SPEC_ST_OK) {
                at = (int)(len + i);
                page = *(a.page_table + (int64_t)b * a.max_pages + (at >> shift));
                if ((unsigned)page >= (unsigned)a.num_pages) page = -1;
                prepare_row(t, at, s_cs[warp]);
            }
        }
        if (lane == 0) {
            s_page[warp] = page;
            s_offset[warp] = at & (a.page_size - 1);
        }
    }
    __syncthreads();
    const int first = blockIdx.y * units_each, turn_q = a.Hq * t.units, turn = turn_q + a.Hkv * t.units;
    const int n = min(units_each, turn + a.Hkv * t.copies - first);
    for (int r = 0, u = tid;; u += kTurnThreads) {
        while (u >= n && r < rows) {
            u -= n;
            ++r;
        }
        if (r >= rows) break;
        const int page = s_page[r];
        if (page == -2) continue;
        const int64_t row = row0 + r;
        int x = first + u;
        if (x < turn_q) {
            const int head = t.by_units.of(x);
            turn_unit<T, kWide, kPairs>(t, s_cs[r], x - head * t.units, reinterpret_cast<const T*>(a.q) + row * a.q_row_stride + head * t.D,
                                        reinterpret_cast<T*>(a.q_out) + row * a.q_out_row_stride + head * t.D, (T*)nullptr);
        } else if (x < turn) {
            x -= turn_q;
            const int head = t.by_units.of(x);
            T* kept = a.k_out == nullptr ? (T*)nullptr : reinterpret_cast<T*>(a.k_out) + row * a.k_out_row_stride + head * t.D;
            T* to = page < 0 ? kept : reinterpret_cast<T*>(a.k_pages) + (((int64_t)page * a.Hkv + head) * a.page_size + s_offset[r]) * t.D;
            if (to != nullptr)
                turn_unit<T, kWide, kPairs>(t, s_cs[r], x - head * t.units, reinterpret_cast<const T*>(a.k) + row * a.k_row_stride + head * t.D, to,
                                            page < 0 ? (T*)nullptr : kept);
        } else if (page >= 0) {
            x -= turn;
            const int head = t.by_copies.of(x), c = x - head * t.copies;
            const T* from = reinterpret_cast<const T*>(a.v) + row * a.v_row_stride + head * t.D;
            T* to = reinterpret_cast<T*>(a.v_pages) + (((int64_t)page * a.Hkv + head) * a.page_size + s_offset[r]) * t.D;
            if constexpr (kWide)
                *(reinterpret_cast<uint4*>(to) + c) = *(reinterpret_cast<const uint4*>(from) + c);
            else
                to[c] = from[c];
        }
    }
    if (!reports) return;
    for (int64_t b = (int64_t)blockIdx.x * kTurnRows + warp; b < a.B; b += (int64_t)gridDim.x * kTurnRows) {
        int st = SPEC_ST_BAD_OFFSETS, len;
        if (b < first_broken) {
            const int64_t rows_of = stream_rows(a, (int)b);
            st = append_refusal(a, (int)b, rows_of, shift, &len);
            if (st == SPEC_ST_OK && rows_of > 0) {
                const int32_t* table = a.page_table + b * a.max_pages;
                bool bad = false;
                for (int j = (len >> shift) + lane; j <= (int)((len + rows_of - 1) >> shift); j += 32)
                    bad |= (unsigned)*(table + j) >= (unsigned)a.num_pages;
                if (__any_sync(0xffffffffu, bad)) st = SPEC_ST_BAD_PAGE;
            }
        }
        if (lane == 0) a.status[b] = st;
    }
}

// ---------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------
static int element(int dtype) { return dtype == SPEC_DTYPE_F32 ? 4 : 2; }

// `wide`: every pointer and stride lets 16 bytes be moved at a time.
static Turn plan(int D, int dim, int interleaved, int dtype, float magnitude, const uint64_t* turns, bool* wide) {
    const int per = 16 / element(dtype);
    Turn t = {};
    *wide = *wide && (interleaved ? dim : dim / 2) % per == 0;
    t.turns = turns;
    t.D = D;
    t.pairs = dim / 2;
    t.magnitude = magnitude;
    t.turning = *wide ? (interleaved ? dim / per : dim / 2 / per) : dim / 2;
    t.units = t.turning + (*wide ? (D - dim) / per : D - dim);
    t.copies = *wide ? D / per : D;
    t.by_units = divisor(t.units);
    t.by_copies = divisor(t.copies);
    return t;
}

// Rows and units of a CTA.
static void share(int64_t rows, int64_t per_row, int* rows_each, int* units_each, dim3* grid) {
    const int64_t want = rows * per_row >= 152 * 16 * kTurnThreads ? 8 * kTurnThreads : kTurnThreads;
    const int64_t each = want / per_row < 1 ? 1 : want / per_row > kTurnRows ? kTurnRows : want / per_row;
    const int64_t splits = each > 1 ? 1 : (per_row + want - 1) / want;
    *rows_each = (int)each;
    *units_each = (int)((per_row + splits - 1) / splits);
    const int64_t x = (rows + each - 1) / each;
    *grid = dim3((unsigned)(x < 1 ? 1 : x), (unsigned)splits);
}

static int check_turn(const char* who, int dtype, int D, int dim, float magnitude, const uint64_t* turns) {
    if (!valid_dtype(dtype)) return set_error(SPEC_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (D < 8 || D > SPEC_MAX_HEAD || D % 8 != 0) return set_error(SPEC_ERR_SHAPE, "%s: D = %d", who, D);
    if (dim < 2 || dim > D || dim % 2 != 0) return set_error(SPEC_ERR_SHAPE, "%s: dim = %d of heads of %d", who, dim, D);
    if (!std::isfinite(magnitude)) return set_error(SPEC_ERR_ARG, "%s: magnitude is not finite", who);
    if ((uintptr_t)turns & 7) return set_error(SPEC_ERR_ARG, "%s: turns is not 8-byte aligned", who);
    return SPEC_OK;
}

template <typename T, typename A, template <typename, bool, bool> class K>
static cudaError_t pick(const A& a, const Turn& t, bool wide, bool pairs, int rows_each, int units_each, dim3 grid, cudaStream_t s) {
    auto* f = wide ? (pairs ? K<T, true, true>::kernel : K<T, true, false>::kernel) : pairs ? K<T, false, true>::kernel : K<T, false, false>::kernel;
    return launch_after(f, grid, dim3(kTurnThreads), 0, s, a, t, rows_each, units_each);
}
template <typename T, bool kWide, bool kPairs>
struct Rotates {
    static constexpr auto kernel = rotate_kernel<T, kWide, kPairs>;
};
template <typename T, bool kWide, bool kPairs>
struct Appends {
    static constexpr auto kernel = append_rotated_kernel<T, kWide, kPairs>;
};

}  // namespace sv

using namespace sv;

extern "C" int spec_rotary_frequencies(int32_t dim, double base, int32_t scaling, double factor, double original, double slow, double fast,
                                       double* frequency, float* magnitude) {
    clear_error();
    if (frequency == nullptr || magnitude == nullptr) return set_error(SPEC_ERR_ARG, "spec_rotary_frequencies: an output is NULL");
    if (dim < 2 || dim > SPEC_MAX_HEAD || dim % 2 != 0) return set_error(SPEC_ERR_SHAPE, "spec_rotary_frequencies: dim = %d", dim);
    if (scaling < SPEC_ROTARY_PLAIN || scaling > SPEC_ROTARY_YARN) return set_error(SPEC_ERR_ARG, "spec_rotary_frequencies: scaling = %d", scaling);
    if (!std::isfinite(base) || !(base > 1) || (scaling != SPEC_ROTARY_PLAIN && (!std::isfinite(factor) || !(factor >= 1))))
        return set_error(SPEC_ERR_ARG, "spec_rotary_frequencies: base = %g, factor = %g", base, factor);
    if (scaling == SPEC_ROTARY_YARN && (!std::isfinite(original) || !(original >= 1) || !std::isfinite(slow) || !std::isfinite(fast) || !(fast > slow)))
        return set_error(SPEC_ERR_ARG, "spec_rotary_frequencies: original = %g, slow = %g, fast = %g", original, slow, fast);
    const double pi = 3.14159265358979323846;
    double b = base;
    if (scaling == SPEC_ROTARY_NTK && dim > 2) b *= std::pow(factor, (double)dim / (dim - 2));
    for (int j = 0; j < dim / 2; ++j) {
        double f = std::pow(b, -2.0 * j / dim);
        if (scaling == SPEC_ROTARY_LINEAR) f /= factor;
        if (scaling == SPEC_ROTARY_YARN) {
            double keep = (original * f / (2 * pi) - slow) / (fast - slow);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = f * keep + f / factor * (1 - keep);
        }
        frequency[j] = f;
    }
    *magnitude = scaling == SPEC_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return SPEC_OK;
}

extern "C" int spec_rotary_turns(const double* frequency, int32_t n, uint64_t* turns) {
    clear_error();
    if (frequency == nullptr || turns == nullptr) return set_error(SPEC_ERR_ARG, "spec_rotary_turns: a pointer is NULL");
    if (n < 1 || n > SPEC_MAX_HEAD / 2) return set_error(SPEC_ERR_SHAPE, "spec_rotary_turns: n = %d", n);
    for (int j = 0; j < n; ++j)
        if (!std::isfinite(frequency[j])) return set_error(SPEC_ERR_ARG, "spec_rotary_turns: frequency[%d] is not finite", j);
    for (int j = 0; j < n; ++j) {
        double t = frequency[j] / 6.28318530717958647692;
        t -= std::floor(t);
        // two halves: a double has 53 of the 64 bits, and a fraction that rounds to a whole turn is none
        const double hi = std::floor(std::ldexp(t, 32));
        const double lo = std::floor(std::ldexp(std::ldexp(t, 32) - hi, 32) + 0.5);
        turns[j] = ((uint64_t)hi << 32) + (uint64_t)lo;
    }
    return SPEC_OK;
}

extern "C" int spec_rotate(const spec_rotate_args* a, void* stream) {
    clear_error();
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "spec_rotate: args is NULL");
    const int rc = check_turn("spec_rotate", a->dtype, a->D, a->dim, a->magnitude, a->turns);
    if (rc != SPEC_OK) return rc;
    if (a->heads < 1 || a->heads > 4096) return set_error(SPEC_ERR_SHAPE, "spec_rotate: heads = %d", a->heads);
    if (a->rows < 0 || a->rows > INT32_MAX) return set_error(SPEC_ERR_SHAPE, "spec_rotate: rows = %lld", (long long)a->rows);
    const int64_t dense = (int64_t)a->heads * a->D;
    if (a->x_row_stride < dense || a->out_row_stride < dense) return set_error(SPEC_ERR_SHAPE, "spec_rotate: a row stride is below heads * D");
    if (a->rows > 0 && a->x == a->out && a->x_row_stride != a->out_row_stride)
        return set_error(SPEC_ERR_SHAPE, "spec_rotate: in place with different row strides");
    if (a->rows == 0) return SPEC_OK;
    if (a->turns == nullptr || a->positions == nullptr || a->x == nullptr || a->out == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_rotate: a required pointer is NULL");
    const int es = element(a->dtype);
    bool wide = (((uintptr_t)a->x | (uintptr_t)a->out | (uintptr_t)(a->x_row_stride * es) | (uintptr_t)(a->out_row_stride * es)) & 15) == 0;
    const Turn t = plan(a->D, a->dim, a->interleaved, a->dtype, a->magnitude, a->turns, &wide);
    int rows_each, units_each;
    dim3 grid;
    share(a->rows, (int64_t)a->heads * t.units, &rows_each, &units_each, &grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 4 ? pick<float, spec_rotate_args, Rotates>(*a, t, wide, a->interleaved != 0, rows_each, units_each, grid, s)
                                  : pick<unsigned short, spec_rotate_args, Rotates>(*a, t, wide, a->interleaved != 0, rows_each, units_each, grid, s);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_rotate");
}

extern "C" int spec_cache_append_rotated(const spec_append_rotated_args* a, void* stream) {
    clear_error();
    const char* const who = "spec_cache_append_rotated";
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "%s: args is NULL", who);
    const int rc = check_turn(who, a->dtype, a->D, a->dim, a->magnitude, a->turns);
    if (rc != SPEC_OK) return rc;
    if (a->B < 0 || a->B > SPEC_MAX_STREAMS || a->max_rows < 0 || (a->extra_rows & ~1) != 0)
        return set_error(SPEC_ERR_SHAPE, "%s: B = %d, max_rows = %d, extra_rows = %d", who, a->B, a->max_rows, a->extra_rows);
    if (a->Hq < 0 || a->Hq > 1024 || a->Hkv < 1 || a->Hkv > 1024) return set_error(SPEC_ERR_SHAPE, "%s: Hq = %d, Hkv = %d", who, a->Hq, a->Hkv);
    if (a->page_size < 8 || a->page_size > SPEC_MAX_PAGE || (a->page_size & (a->page_size - 1)) != 0 || a->num_pages < 1 || a->max_pages < 1 ||
        (int64_t)a->max_pages * a->page_size > INT32_MAX)
        return set_error(SPEC_ERR_SHAPE, "%s: page_size = %d, num_pages = %d, max_pages = %d", who, a->page_size, a->num_pages, a->max_pages);
    const int64_t dq = (int64_t)a->Hq * a->D, dk = (int64_t)a->Hkv * a->D;
    if (a->k_row_stride < dk || a->v_row_stride < dk || (a->Hq > 0 && (a->q_row_stride < dq || a->q_out_row_stride < dq)) ||
        (a->k_out != nullptr && a->k_out_row_stride < dk))
        return set_error(SPEC_ERR_SHAPE, "%s: a row stride is below its heads * D", who);
    if (a->rows > 0 && ((a->Hq > 0 && a->q_out == a->q && a->q_out_row_stride != a->q_row_stride) ||
        (a->k_out != nullptr && a->k_out == a->k && a->k_out_row_stride != a->k_row_stride)))
        return set_error(SPEC_ERR_SHAPE, "%s: in place with different row strides", who);
    if (a->rows < 0 || a->rows > INT32_MAX || (a->cu == nullptr && a->rows < (int64_t)a->B * a->max_rows))
        return set_error(SPEC_ERR_SHAPE, "%s: rows = %lld", who, (long long)a->rows);
    if (a->B == 0) return SPEC_OK;
    if (a->turns == nullptr || a->length == nullptr || a->page_table == nullptr || a->k_pages == nullptr || a->v_pages == nullptr ||
        a->status == nullptr || (a->rows > 0 && (a->k == nullptr || a->v == nullptr || (a->Hq > 0 && (a->q == nullptr || a->q_out == nullptr)))))
        return set_error(SPEC_ERR_ARG, "%s: a required pointer is NULL", who);
    if (((uintptr_t)a->k_pages | (uintptr_t)a->v_pages) & 15) return set_error(SPEC_ERR_ARG, "%s: the pool is not 16-byte aligned", who);
    const int es = element(a->dtype);
    uintptr_t low = (uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)(a->k_row_stride * es) | (uintptr_t)(a->v_row_stride * es);
    if (a->Hq > 0) low |= (uintptr_t)a->q | (uintptr_t)a->q_out | (uintptr_t)(a->q_row_stride * es) | (uintptr_t)(a->q_out_row_stride * es);
    if (a->k_out != nullptr) low |= (uintptr_t)a->k_out | (uintptr_t)(a->k_out_row_stride * es);
    bool wide = (low & 15) == 0;
    const Turn t = plan(a->D, a->dim, a->interleaved, a->dtype, a->magnitude, a->turns, &wide);
    int rows_each, units_each;
    dim3 grid;
    share(a->rows, (int64_t)(a->Hq + a->Hkv) * t.units + (int64_t)a->Hkv * t.copies, &rows_each, &units_each, &grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 4
                              ? pick<float, spec_append_rotated_args, Appends>(*a, t, wide, a->interleaved != 0, rows_each, units_each, grid, s)
                              : pick<unsigned short, spec_append_rotated_args, Appends>(*a, t, wide, a->interleaved != 0, rows_each, units_each, grid, s);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, who);
}
