// Rotary positions: spec_rotate, spec_cache_append_rotated, and the host's frequencies.
//
// A head's pair (a, b) j at position p turns by the angle p f_j:
//   a' = m (a cos - b sin),   b' = m (b cos + a sin).
// The angle is kept in turns, as a 64-bit fraction: with T_j = 2^64 f_j / 2 pi the product p T_j modulo 2^64 is the
// fraction of the turn, so whole turns fall away exactly, in two integer multiplications, at any position.  (In float32 an angle of
// 131,072 radians is known to 0.008; the product here is off by p times what T_j is: it comes from double arithmetic, within |f_j / 2 pi| 2^-52 + 2^-54
// turns, for frequencies up to 1 within 2^-55.  At position 131,072 that is 2^-38 turns, at 2^31 2^-24.)  The nearest quarter
// turn is taken off in integers as well, and what is left, at most an eighth, goes to sincospif.
//
// Bound by memory: a row's sines and cosines are computed once, by a warp, into shared memory and serve all its heads; every element
// is read and written once, 16 bytes a thread.  8,191 rows of 72 heads of 128 (302 MB) 47.5 us, 6.35 TB/s; 24 prompts, 64/8 heads of 128,
// appended with their packed keys (617 MB) 93.5 us, 6.6 TB/s; six rows of 20 heads 1.7 us, a block of six tokens appended 3.1 (launch).

#include <cmath>

#include "blocks.cuh"
#include "divisor.cuh"
#include "host_util.h"

namespace sv {

constexpr int kTurnThreads = 256;
constexpr int kTurnRows = kTurnThreads / 32;       // rows of a CTA: a warp prepares one
// A row's sines and cosines in shared memory, one place free behind every eight: threads of neighbouring units read eight (or four) of them each, which
// without that are in the same banks (24 prompts appended 93.5 us against 97.2, 64 blocks 4.5 against 5.2; rows alone as before).
constexpr int kTurnPairs = (SPEC_MAX_HEAD / 2 + 8) / 8 * 9;   // (a ragged unit reads up to seven past the last)
__device__ __forceinline__ int place(int j) { return j + (j >> 3); }

// How a head is cut.  kWide: units of 16 bytes (halves: 16 bytes of either half).  kRagged: the same where what turns does not end on, or a half
// does not begin on, a 16-byte boundary; the second half and the rest of the head then move in pieces of what alignment they have.  kScalar: units
// of one pair or element, for rows that are not on 16-byte boundaries.
enum { kScalar, kWide, kRagged };
struct Turn {
    const uint64_t* turns;
    int D, pairs;
    int turning;        // units of a head that turn; the others are copied
    int half_align, rest_align;   // kRagged: bytes to whose multiples the second half and the rest of a head lie
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
    for (int j = threadIdx.x & 31; j < t.pairs; j += 32) cs[place(j)] = cos_sin(p, t.turns[j], t.magnitude);
}

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) { return make_float2(a * cs.x - b * cs.y, b * cs.x + a * cs.y); }

// 16 bytes as floats and back.
template <typename T>
struct Wide;
template <>
struct Wide<unsigned short> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(u[i]);
            x[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Wide<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ void unpack(uint4 w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
__device__ __forceinline__ float value(unsigned short x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ void store(unsigned short* p, float x) { *p = __bfloat16_as_ushort(__float2bfloat16(x)); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }

// A unit of a head, as it was read.  The next one is read before this one is turned and written (what is written may be the place that
// was read, but a unit is one thread's alone), and the first one before the row's sines are there.
template <typename T, int kMode, bool kPairs>
struct Held;
template <typename T, bool kPairs>
struct Held<T, kWide, kPairs> {
    static constexpr int per = Wide<T>::kPer;
    uint4 a, b;
    __device__ __forceinline__ void load(const Turn& t, int u, const T* from) {
        if (u < t.turning) {
            a = *reinterpret_cast<const uint4*>(from + u * per);
            if constexpr (!kPairs) b = *reinterpret_cast<const uint4*>(from + t.pairs + u * per);
        } else {
            a = *reinterpret_cast<const uint4*>(from + 2 * t.pairs + (u - t.turning) * per);
        }
    }
    __device__ __forceinline__ void load_copy(int u, const T* from) { a = *(reinterpret_cast<const uint4*>(from) + u); }
    __device__ __forceinline__ void store_copy(int u, T* to) const { *(reinterpret_cast<uint4*>(to) + u) = a; }
    // ... to one place or two (also == nullptr: one)
    __device__ __forceinline__ void finish(const Turn& t, const float2* cs, int u, T* to, T* also) const {
        int at = u * per;
        uint4 y = a, z = b;
        if (u >= t.turning) {
            at = 2 * t.pairs + (u - t.turning) * per;
        } else if constexpr (kPairs) {
            float x[per];
            cs += place(at / 2);
            Wide<T>::unpack(a, x);
#pragma unroll
            for (int i = 0; i < per; i += 2) {
                const float2 w = turned(x[i], x[i + 1], cs[i / 2]);
                x[i] = w.x;
                x[i + 1] = w.y;
            }
            y = Wide<T>::pack(x);
        } else {
            float x[per], v[per];
            cs += place(at);
            Wide<T>::unpack(a, x);
            Wide<T>::unpack(b, v);
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const float2 w = turned(x[i], v[i], cs[i]);
                x[i] = w.x;
                v[i] = w.y;
            }
            y = Wide<T>::pack(x);
            z = Wide<T>::pack(v);
            *reinterpret_cast<uint4*>(to + t.pairs + at) = z;
            if (also != nullptr) *reinterpret_cast<uint4*>(also + t.pairs + at) = z;
        }
        *reinterpret_cast<uint4*>(to + at) = y;
        if (also != nullptr) *reinterpret_cast<uint4*>(also + at) = y;
    }
};
template <typename T, bool kPairs>
struct Held<T, kScalar, kPairs> {   // a pair, or an element that does not turn
    T a, b;
    __device__ __forceinline__ void load(const Turn& t, int u, const T* from) {
        if (u < t.turning) {
            a = from[kPairs ? 2 * u : u];
            b = from[kPairs ? 2 * u + 1 : u + t.pairs];
        } else {
            a = from[t.pairs + u];
        }
    }
    __device__ __forceinline__ void load_copy(int u, const T* from) { a = from[u]; }
    __device__ __forceinline__ void store_copy(int u, T* to) const { to[u] = a; }
    __device__ __forceinline__ void finish(const Turn& t, const float2* cs, int u, T* to, T* also) const {
        if (u >= t.turning) {
            to[t.pairs + u] = a;
            if (also != nullptr) also[t.pairs + u] = a;
            return;
        }
        const int i = kPairs ? 2 * u : u, j = kPairs ? 2 * u + 1 : u + t.pairs;
        const float2 y = turned(value(a), value(b), cs[place(u)]);
        store(to + i, y.x);
        store(to + j, y.y);
        if (also != nullptr) {
            store(also + i, y.x);
            store(also + j, y.y);
        }
    }
};

// n elements (16 bytes, or fewer at the end of a part) of a place that lies on a multiple of `align` bytes.
__device__ __forceinline__ uint4 fetch(const unsigned short* p, int n, int align) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (n == 8 && align == 16) return *reinterpret_cast<const uint4*>(p);
    if (n == 8 && align >= 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else if (n == 8) {   // the words from the element before on (it is the head's too), and the last element
        uint32_t x[5];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = reinterpret_cast<const uint32_t*>(p - 1)[i];
        x[4] = p[7];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 fetch(const float* p, int n, int align) {
    if (n == 4 && align == 16) return *reinterpret_cast<const uint4*>(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put(unsigned short* p, uint4 x, int n, int align) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (n == 8 && align == 16) {
        *reinterpret_cast<uint4*>(p) = x;
    } else if (n == 8 && align >= 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else if (n == 8) {
        p[0] = (unsigned short)w[0];
#pragma unroll
        for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(p + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
        p[7] = (unsigned short)(w[3] >> 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (unsigned short)(w[i / 2] >> (i % 2 * 16));
    }
}
__device__ __forceinline__ void put(float* p, uint4 x, int n, int align) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (n == 4 && align == 16) {
        *reinterpret_cast<uint4*>(p) = x;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    }
}
template <typename T, bool kPairs>
struct Held<T, kRagged, kPairs> {
    static constexpr int per = Wide<T>::kPer;
    uint4 a, b;
    // where unit u lies (halves: its first element of the first half), its elements there, and whether it turns
    __device__ __forceinline__ static bool span(const Turn& t, int u, int* at, int* n) {
        if (kPairs) {
            *at = u * per;
            *n = per;
            return u < t.turning;
        }
        const bool turns = u < t.turning;
        const int first = turns ? 0 : 2 * t.pairs, end = turns ? t.pairs : t.D;
        *at = first + (turns ? u : u - t.turning) * per;
        *n = min(per, end - *at);
        return turns;
    }
    __device__ __forceinline__ void load(const Turn& t, int u, const T* from) {
        int at, n;
        const bool turns = span(t, u, &at, &n);
        a = fetch(from + at, n, kPairs || turns ? 16 : t.rest_align);
        if (!kPairs && turns) b = fetch(from + t.pairs + at, n, t.half_align);
    }
    __device__ __forceinline__ void load_copy(int u, const T* from) { a = *(reinterpret_cast<const uint4*>(from) + u); }
    __device__ __forceinline__ void store_copy(int u, T* to) const { *(reinterpret_cast<uint4*>(to) + u) = a; }
    __device__ __forceinline__ void finish(const Turn& t, const float2* cs, int u, T* to, T* also) const {
        int at, n;
        const bool turns = span(t, u, &at, &n);
        uint4 y = a;
        if (turns) {
            float x[per], v[per];
            Wide<T>::unpack(a, x);
            if constexpr (kPairs) {
#pragma unroll
                for (int i = 0; i < per; i += 2) {
                    const float2 w = turned(x[i], x[i + 1], cs[place(at / 2) + i / 2]);
                    x[i] = w.x;
                    x[i + 1] = w.y;
                }
            } else {
                Wide<T>::unpack(b, v);
#pragma unroll
                for (int i = 0; i < per; ++i) {
                    const float2 w = turned(x[i], v[i], cs[place(at) + i]);
                    x[i] = w.x;
                    v[i] = w.y;
                }
                const uint4 z = Wide<T>::pack(v);
                put(to + t.pairs + at, z, n, t.half_align);
                if (also != nullptr) put(also + t.pairs + at, z, n, t.half_align);
            }
            y = Wide<T>::pack(x);
            if constexpr (kPairs) {   // the unit's pairs behind the last that turns stay as they are
                const int left = (t.pairs - at / 2) * 2 * (int)sizeof(T) / 4;
                y.y = left > 1 ? y.y : a.y;
                y.z = left > 2 ? y.z : a.z;
                y.w = left > 3 ? y.w : a.w;
            }
        }
        const int align = kPairs || turns ? 16 : t.rest_align;
        put(to + at, y, n, align);
        if (also != nullptr) put(also + at, y, n, align);
    }
};

// The units of a CTA's rows, row by row, kTurnThreads apart.
struct Place {
    int r, u;   // row, unit of the CTA's share of it
    __device__ __forceinline__ Place(int tid, int n, int rows) : r(0), u(tid) { wrap(n, rows); }
    __device__ __forceinline__ void wrap(int n, int rows) {
        while (u >= n && r < rows) {
            u -= n;
            ++r;
        }
    }
    __device__ __forceinline__ void next(int n, int rows) {
        u += kTurnThreads;
        wrap(n, rows);
    }
};

// ---------------------------------------------------------------------------------------
// rows at given positions
// ---------------------------------------------------------------------------------------
template <typename T, int kMode, bool kPairs>
__global__ void __launch_bounds__(kTurnThreads, 6) rotate_kernel(const spec_rotate_args a, const Turn t, int rows_each, int units_each) {
    __shared__ float2 s_cs[kTurnRows][kTurnPairs];
    const int tid = threadIdx.x, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row0 = (int64_t)blockIdx.x * rows_each;
    const int rows = (int)min((int64_t)rows_each, a.rows - row0);
    const int first = blockIdx.y * units_each, n = min(units_each, a.heads * t.units - first);
    Held<T, kMode, kPairs> held = {};
    auto load = [&](const Place& at) {
        const int head = t.by_units.of(first + at.u);
        held.load(t, first + at.u - head * t.units, reinterpret_cast<const T*>(a.x) + (row0 + at.r) * a.x_row_stride + head * t.D);
    };
    Place at(tid, n, rows);
    if (at.r < rows) load(at);
    if (warp < rows) prepare_row(t, *(a.positions + row0 + warp), s_cs[warp]);
    __syncthreads();
    while (at.r < rows) {
        const Place now = at;
        const Held<T, kMode, kPairs> mine = held;
        at.next(n, rows);
        if (at.r < rows) load(at);
        const int head = t.by_units.of(first + now.u);
        mine.finish(t, s_cs[now.r], first + now.u - head * t.units,
                    reinterpret_cast<T*>(a.out) + (row0 + now.r) * a.out_row_stride + head * t.D, (T*)nullptr);
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

template <typename T, int kMode, bool kPairs>
__global__ void __launch_bounds__(kTurnThreads, 6) append_rotated_kernel(const spec_append_rotated_args a, const Turn t, int rows_each, int units_each) {
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
    const int first = blockIdx.y * units_each, turn_q = a.Hq * t.units, turn = turn_q + a.Hkv * t.units;
    const int n = min(units_each, turn + a.Hkv * t.copies - first);
    Held<T, kMode, kPairs> held = {};
    auto load = [&](const Place& at) {
        const int64_t row = row0 + at.r;
        int x = first + at.u;
        if (x < turn_q) {
            const int head = t.by_units.of(x);
            held.load(t, x - head * t.units, reinterpret_cast<const T*>(a.q) + row * a.q_row_stride + head * t.D);
        } else if (x < turn) {
            x -= turn_q;
            const int head = t.by_units.of(x);
            held.load(t, x - head * t.units, reinterpret_cast<const T*>(a.k) + row * a.k_row_stride + head * t.D);
        } else {
            x -= turn;
            const int head = t.by_copies.of(x);
            held.load_copy(x - head * t.copies, reinterpret_cast<const T*>(a.v) + row * a.v_row_stride + head * t.D);
        }
    };
    Place at(tid, n, rows);
    if (at.r < rows) load(at);   // on its way while the rows' streams are found
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
    while (at.r < rows) {
        const Place now = at;
        const Held<T, kMode, kPairs> mine = held;
        at.next(n, rows);
        if (at.r < rows) load(at);
        const int page = s_page[now.r];
        if (page == -2) continue;
        const int64_t row = row0 + now.r;
        int x = first + now.u;
        if (x < turn_q) {
            const int head = t.by_units.of(x);
            mine.finish(t, s_cs[now.r], x - head * t.units, reinterpret_cast<T*>(a.q_out) + row * a.q_out_row_stride + head * t.D, (T*)nullptr);
        } else if (x < turn) {
            x -= turn_q;
            const int head = t.by_units.of(x);
            T* kept = a.k_out == nullptr ? (T*)nullptr : reinterpret_cast<T*>(a.k_out) + row * a.k_out_row_stride + head * t.D;
            T* to = page < 0 ? kept : reinterpret_cast<T*>(a.k_pages) + (((int64_t)page * a.Hkv + head) * a.page_size + s_offset[now.r]) * t.D;
            if (to != nullptr) mine.finish(t, s_cs[now.r], x - head * t.units, to, page < 0 ? (T*)nullptr : kept);
        } else if (page >= 0) {
            x -= turn;
            const int head = t.by_copies.of(x);
            mine.store_copy(x - head * t.copies,
                            reinterpret_cast<T*>(a.v_pages) + (((int64_t)page * a.Hkv + head) * a.page_size + s_offset[now.r]) * t.D);
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

// `even`: every pointer and row stride is a multiple of 16 bytes.  Whole 16-byte units are what most heads are.  Of 4,000 rows of 40 heads of 128 in bf16
// the ragged form takes 18.7 us with 122 elements turned in pairs and 38.3 with halves of 33; one pair a thread takes 40.6 and 52.3.
static Turn plan(int D, int dim, int interleaved, int dtype, float magnitude, const uint64_t* turns, bool even, int* mode) {
    const int es = element(dtype), per = 16 / es, pairs = dim / 2, turning = interleaved ? dim : pairs;
    Turn t = {};
    *mode = !even ? kScalar : turning % per == 0 ? kWide : kRagged;
    t.turns = turns;
    t.D = D;
    t.pairs = pairs;
    t.magnitude = magnitude;
    auto align = [&](int elements) { return (elements * es) % 16 == 0 ? 16 : (elements * es) & -(elements * es); };
    t.half_align = align(pairs);
    t.rest_align = align(dim);
    t.turning = *mode == kScalar ? pairs : (turning + per - 1) / per;
    t.units = *mode == kScalar ? pairs + D - dim : interleaved ? D / per : t.turning + (D - dim + per - 1) / per;
    t.copies = *mode == kScalar ? D : D / per;
    t.by_units = divisor(t.units);
    t.by_copies = divisor(t.copies);
    return t;
}

// Rows and units of a CTA: what fills the resident CTAs (six an SM) once, from one to eight units a thread, and in whole rows where a thread has
// more than one: a row's sines, and an append's search for its stream, are every CTA's that has a part of it.  8,191 rows of 72 heads of 128 take 47.7 us with eight units, 52.0
// with six and 55.2 with sixteen; 900 float32 rows of 48 heads appended 6.9 us a row a CTA and 10.2 in three parts.
static void share(int64_t rows, int64_t per_row, int sms, int* rows_each, int* units_each, dim3* grid) {
    const int64_t fill = rows * per_row / (sms * 6);
    const int64_t want = fill < kTurnThreads ? kTurnThreads : fill > 8 * kTurnThreads ? 8 * kTurnThreads : fill;
    const int64_t each = want / per_row < 1 ? 1 : want / per_row > kTurnRows ? kTurnRows : want / per_row;
    const int64_t splits = each > 1 ? 1 : want == kTurnThreads ? (per_row + want - 1) / want : per_row < 2 * want ? 1 : per_row / want;
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

template <typename T, typename A, template <typename, int, bool> class K>
static cudaError_t pick(const A& a, const Turn& t, int mode, bool pairs, int rows_each, int units_each, dim3 grid, cudaStream_t s) {
    auto* f = mode == kWide     ? (pairs ? K<T, kWide, true>::kernel : K<T, kWide, false>::kernel)
              : mode == kRagged ? (pairs ? K<T, kRagged, true>::kernel : K<T, kRagged, false>::kernel)
                                : (pairs ? K<T, kScalar, true>::kernel : K<T, kScalar, false>::kernel);
    return launch_after(f, grid, dim3(kTurnThreads), 0, s, a, t, rows_each, units_each);
}
template <typename T, int kMode, bool kPairs>
struct Rotates {
    static constexpr auto kernel = rotate_kernel<T, kMode, kPairs>;
};
template <typename T, int kMode, bool kPairs>
struct Appends {
    static constexpr auto kernel = append_rotated_kernel<T, kMode, kPairs>;
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
    if (a->rows > 1 && a->x == a->out && a->x_row_stride != a->out_row_stride)
        return set_error(SPEC_ERR_SHAPE, "spec_rotate: in place with different row strides");
    if (a->rows == 0) return SPEC_OK;
    if (a->turns == nullptr || a->positions == nullptr || a->x == nullptr || a->out == nullptr)
        return set_error(SPEC_ERR_ARG, "spec_rotate: a required pointer is NULL");
    const int es = element(a->dtype);
    const bool even = (((uintptr_t)a->x | (uintptr_t)a->out | (uintptr_t)(a->x_row_stride * es) | (uintptr_t)(a->out_row_stride * es)) & 15) == 0;
    int mode, sms = 0;
    const int count = sm_count(&sms, "spec_rotate");
    if (count != SPEC_OK) return count;
    const Turn t = plan(a->D, a->dim, a->interleaved, a->dtype, a->magnitude, a->turns, even, &mode);
    int rows_each, units_each;
    dim3 grid;
    share(a->rows, (int64_t)a->heads * t.units, sms, &rows_each, &units_each, &grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 4 ? pick<float, spec_rotate_args, Rotates>(*a, t, mode, a->interleaved != 0, rows_each, units_each, grid, s)
                                  : pick<unsigned short, spec_rotate_args, Rotates>(*a, t, mode, a->interleaved != 0, rows_each, units_each, grid, s);
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
    if (a->rows > 1 && ((a->Hq > 0 && a->q_out == a->q && a->q_out_row_stride != a->q_row_stride) ||
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
    int mode, sms = 0;
    const int count = sm_count(&sms, who);
    if (count != SPEC_OK) return count;
    const Turn t = plan(a->D, a->dim, a->interleaved, a->dtype, a->magnitude, a->turns, (low & 15) == 0, &mode);
    int rows_each, units_each;
    dim3 grid;
    share(a->rows, (int64_t)(a->Hq + a->Hkv) * t.units + (int64_t)a->Hkv * t.copies, sms, &rows_each, &units_each, &grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 4
                              ? pick<float, spec_append_rotated_args, Appends>(*a, t, mode, a->interleaved != 0, rows_each, units_each, grid, s)
                              : pick<unsigned short, spec_append_rotated_args, Appends>(*a, t, mode, a->interleaved != 0, rows_each, units_each, grid, s);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, who);
}
