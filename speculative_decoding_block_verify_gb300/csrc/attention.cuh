// How the attention of a batch of blocks is cut into pieces, shared by its kernels.
//
// An item is (stream, key head, group of rows): the rows of one stream's block that read one key
// head are its tokens times the G query heads of that key head, row r = token * G + query head, at
// most `rows` of them in a group.  An item's keys are cut into tiles of kTile positions (the visible
// ones only: the sinks' tiles, then the window's).  The tiles of all items in order (stream, head,
// group) form one line, and CTA c takes tiles [c * span, (c + 1) * span) of it: every CTA gets the same
// number of tiles whatever the lengths are, and an item that lies across CTAs is joined afterwards
// from one part per CTA, in the order of its keys.
#pragma once

#include "blocks.cuh"

namespace sv {

constexpr int kTile = 64;          // positions of a tile
constexpr int kItemCost = 2;       // what beginning and ending an item takes, in tiles
constexpr int kMaxCtas = 512;      // CTAs of an attention grid
constexpr int kJoinFan = 8;        // parts joined at a time
constexpr int kJoinLevels = 3;     // 8^3 = kMaxCtas

struct AttnParams {
    spec_attention_args a;
    int G;            // query heads per key head
    int rows;         // rows of a full group
    int ctas;         // CTAs of the grid
    int page_shift;
    float scale_log2; // scale * log2(e)
    // workspace
    int32_t* timeout;  // a wait gave up (stays set)
    int32_t* arrived;  // [kJoinLevels][2 ctas] parts of a group of parts that are there (left at zero)
    float2* ml;        // [kJoinLevels][2 ctas][rows] maximum (of the scaled scores, base 2) and sum of a part's rows
    float4* part;      // [2 ctas][D / 4][rows] their weighted values, not yet divided
};

// The tiles of one item.
struct Item {
    int r0, r1;       // rows [r0, r1) of the block's rows * G
    int low, high;    // visible positions: [0, sink) and [low, high)
    int sink;
    int sink_tiles, first_tile, tiles;
};
__device__ __forceinline__ Item make_item(const AttnParams& p, int len, int block_rows, int group) {
    Item it;
    it.r0 = group * p.rows;
    it.r1 = min(it.r0 + p.rows, block_rows * p.G);
    const int i0 = it.r0 / p.G, i1 = (it.r1 - 1) / p.G;
    it.high = len + i1 + 1;
    it.low = p.a.window > 0 ? max(0, len + i0 + 1 - p.a.window) : 0;
    it.sink = min(p.a.sinks, it.low);
    it.sink_tiles = (it.sink + kTile - 1) / kTile;
    it.first_tile = max(it.low / kTile, it.sink_tiles);
    it.tiles = it.sink_tiles + (it.high + kTile - 1) / kTile - it.first_tile;
    return it;
}
// First position of tile t of the item.
__device__ __forceinline__ int tile_start(const Item& it, int t) {
    return (t < it.sink_tiles ? t : it.first_tile + t - it.sink_tiles) * kTile;
}

__device__ __forceinline__ bool length_ok(const AttnParams& p, int len, int n) {
    return len >= 0 && (int64_t)len + n <= (int64_t)p.a.max_pages << p.page_shift;
}

__device__ __forceinline__ int block_groups(const AttnParams& p, int n) { return (n * p.G + p.rows - 1) / p.rows; }

// Length on the line of one key head of a stream (0 where its length is not in its table row).
__device__ __forceinline__ int64_t head_cost(const AttnParams& p, int len, int n) {
    if (!length_ok(p, len, n)) return 0;
    int64_t t = 0;
    const int groups = block_groups(p, n);
    for (int g = 0; g < groups; ++g) t += make_item(p, len, n, g).tiles + kItemCost;
    return t;
}

// a / b of numbers that are nearly always below 2^32
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Where a CTA starts on the line.  Computed by the whole block; valid after the call for every thread.
struct Start {
    int64_t at;       // the CTA's first position
    int64_t span;     // positions of every CTA (the last ones may get fewer, or none)
    int64_t total;
    int64_t stream0;  // the line's position where stream `stream` begins
    int stream;       // stream that `at` lies in
    int valid;        // streams with defined rows
};

template <int kThreads>
__device__ __forceinline__ void find_start(const AttnParams& p, int cta, Start* s /* shared */,
                                           int64_t* scratch /* shared [kThreads / 32] */, int* iscratch /* shared */) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.a.B), b1 = min(b0 + per, p.a.B);
    const int32_t* cu = p.a.cu_drafts;
    if (tid == 0) *iscratch = p.a.B;
    __syncthreads();
    int valid = p.a.B;
    int64_t mine = 0, before = 0, total = 0;
    // streams are taken as they come; where offsets turn out to be broken, once more up to there
    for (int pass = 0; pass < 2; ++pass) {
        mine = 0;
        for (int b = b0; b < b1 && b < valid; ++b) {
            const int len = __ldg(p.a.length + b);
            int n = p.a.kmax + 1;
            if (cu != nullptr) {
                const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
                n = c1 - c0 + 1;
                if (n < 1 || n > p.a.kmax + 1 || (b == 0 && c0 != 0) || (int64_t)c1 + b + 1 > p.a.q_rows) {
                    atomicMin(iscratch, b);
                    break;
                }
            }
            mine += head_cost(p, len, n) * p.a.Hkv;
        }
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scratch[warp] = x;
        __syncthreads();
        before = x - mine;
        total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += scratch[w];
            total += scratch[w];
        }
        valid = *iscratch;
        if (valid == p.a.B || pass == 1) break;
        __syncthreads();
    }
    const int64_t span = quotient(total + p.ctas - 1, p.ctas);
    const int64_t at = (int64_t)cta * span;
    if (tid == 0) {
        s->at = at;
        s->span = span;
        s->total = total;
        s->valid = valid;
    }
    if (at >= before && at < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const int64_t t = head_cost(p, __ldg(p.a.length + b), block_rows(cu, b, p.a.kmax)) * p.a.Hkv;
            if (at < before + t) {
                s->stream = b;
                s->stream0 = before;
                break;
            }
            before += t;
        }
    }
    __syncthreads();
}

// The CTA's walk over its tiles, item by item.  Every role of a CTA walks by itself.  An item takes kItemCost +
// tiles positions of the line: a CTA that ends in the first kItemCost of them leaves the item to the next one.
struct Walk {
    int b, h, g;          // item
    int len, n, groups;   // its stream
    Item it;
    int t0, t1;           // tiles [t0, t1) of the item are this CTA's
    int64_t end;          // where the item ends on the line
    int64_t stop;         // where the CTA ends

    __device__ __forceinline__ bool load_stream(const AttnParams& p) {
        len = __ldg(p.a.length + b);
        n = block_rows(p.a.cu_drafts, b, p.a.kmax);
        groups = block_groups(p, n);
        return length_ok(p, len, n);
    }
    __device__ __forceinline__ bool take() {
        t1 = it.tiles - (int)max((int64_t)0, end - stop);
        return t1 > t0;
    }
    // to the item after this one
    __device__ __forceinline__ void step(const AttnParams& p) {
        if (++g == groups) {
            g = 0;
            if (++h == p.a.Hkv) {
                h = 0;
                do ++b;
                while (!load_stream(p));   // the line goes on, so some later stream has an item
            }
        }
        it = make_item(p, len, n, g);
        t0 = 0;
        end += it.tiles + kItemCost;
    }
    // false: the CTA has no tiles
    __device__ __forceinline__ bool start(const AttnParams& p, const Start& s) {
        stop = min(s.at + s.span, s.total);
        if (s.at >= stop) return false;
        b = s.stream;
        load_stream(p);
        int64_t off = s.at - s.stream0;
        const int64_t per_head = head_cost(p, len, n);
        h = (int)quotient(off, per_head);
        off -= h * per_head;
        for (g = 0;; ++g) {
            it = make_item(p, len, n, g);
            if (off < it.tiles + kItemCost) break;
            off -= it.tiles + kItemCost;
        }
        end = s.at - off + it.tiles + kItemCost;
        t0 = max(0, (int)off - kItemCost);
        return take();
    }
    // to the CTA's next item; false: the CTA is done
    __device__ __forceinline__ bool next(const AttnParams& p) {
        if (end >= stop) return false;
        step(p);
        return take();
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.tiles; }
    // slot of this CTA's part (part_slot below)
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 == 0 ? 1 : 0); }
    // CTA that holds the item's first tile, and how many CTAs hold tiles of it
    __device__ __forceinline__ int first_cta(int64_t span) const { return (int)quotient(end - it.tiles, span); }
    __device__ __forceinline__ int parts(int first, int64_t span) const { return (int)quotient(end - 1, span) - first + 1; }
};

// Is position j visible to the row of token i (its own position is len + i)?
__device__ __forceinline__ bool visible(const AttnParams& p, int at, int j) {
    return j <= at && (p.a.window <= 0 || j > at - p.a.window || j < p.a.sinks);
}

// Two floats as bf16, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Bits of a stored element, and NaN, in the output's type.
__device__ __forceinline__ void put(float* o, float x) { *o = x; }
__device__ __forceinline__ void put(unsigned short* o, float x) { *o = __bfloat16_as_ushort(__float2bfloat16(x)); }

// ... four of them; the output is 16-byte aligned and a row a multiple of 8 elements
__device__ __forceinline__ void put4(float* o, float4 x) { *reinterpret_cast<float4*>(o) = x; }
__device__ __forceinline__ void put4(unsigned short* o, float4 x) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

// The status of the streams cta, cta + ctas, ..., by one warp: the block's rows, the length, and the table
// entries of the pages with a visible position.
template <typename T>
__device__ __forceinline__ void write_status(const AttnParams& p, int cta, int valid) {
    const int lane = threadIdx.x & 31;
    for (int b = cta; b < p.a.B; b += p.ctas) {
        int st = SPEC_ST_BAD_OFFSETS;
        if (b < valid) {
            const int len = __ldg(p.a.length + b), n = block_rows(p.a.cu_drafts, b, p.a.kmax);
            if (!length_ok(p, len, n)) {
                st = SPEC_ST_BAD_LENGTH;
                T* to = reinterpret_cast<T*>(p.a.out) + first_row(p.a.cu_drafts, b, p.a.kmax) * p.a.Hq * (int64_t)p.a.D;
                for (int64_t i = lane; i < (int64_t)n * p.a.Hq * p.a.D; i += 32) put(to + i, __int_as_float(0x7fffffff));
            } else {
                const int low = p.a.window > 0 ? max(0, len + 1 - p.a.window) : 0;
                const int sp = (min(p.a.sinks, low) + p.a.page_size - 1) >> p.page_shift, lp = low >> p.page_shift;
                const int hp = (len + n + p.a.page_size - 1) >> p.page_shift;
                const int32_t* table = p.a.page_table + (int64_t)b * p.a.max_pages;
                bool bad = false;
                for (int j = lane; j < sp && j < lp; j += 32) bad |= (unsigned)__ldg(table + j) >= (unsigned)p.a.num_pages;
#pragma unroll 8
                for (int j = lp + lane; j < hp; j += 32) bad |= (unsigned)__ldg(table + j) >= (unsigned)p.a.num_pages;
                st = __any_sync(0xffffffffu, bad) ? SPEC_ST_BAD_PAGE : SPEC_ST_OK;
            }
        }
        if (lane == 0) {
            p.a.status[b] = st;
            __threadfence();
            if (*reinterpret_cast<volatile int32_t*>(p.timeout)) p.a.status[b] = SPEC_ST_TIMEOUT;
        }
    }
}
// A wait of this CTA gave up.  Whoever writes a status later sees the flag.
__device__ __forceinline__ void write_timeout(const AttnParams& p) {
    atomicExch(p.timeout, 1);
    __threadfence();
    for (int b = 0; b < p.a.B; ++b) p.a.status[b] = SPEC_ST_TIMEOUT;
}

// Slot of part k of an item whose first tile is CTA `first`'s: an item is begun in a CTA's second slot and
// carried on in the first one of the CTAs behind.
__device__ __forceinline__ int part_slot(int first, int k) { return 2 * (first + k) + (k == 0 ? 1 : 0); }

// Joins the parts of an item that lies across CTAs.  Called by `threads` threads of a CTA (`barrier` is theirs)
// that have written part k.  Parts are joined in groups of kJoinFan by the CTA that comes last to the group,
// into the group's first slot; with more than kJoinFan groups these are joined in the same way, up to the
// rows themselves.  Nobody waits, and the tree and the order of its sums do not depend on who comes last.
//   M = max m_k,  out = sum 2^(m_k - M) o_k / sum 2^(m_k - M) l_k
template <typename T, int threads, int barrier>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Walk& w, int cta, int64_t span, int tid, int* scratch /* shared */) {
    const int first = w.first_cta(span);
    int nodes = w.parts(first, span), k = cta - first, stride = 1;
    const int rows = w.it.r1 - w.it.r0;
    const int64_t slots = 2 * (int64_t)p.ctas;
    const int nc = p.a.D / 4;
    for (int level = 0;; ++level) {
        const int g0 = k / kJoinFan * kJoinFan, n = min(kJoinFan, nodes - g0);
        const bool last_level = nodes <= kJoinFan;
        const int to = part_slot(first, g0 * stride);
        asm volatile("bar.sync %0, %1;" ::"n"(barrier), "n"(threads) : "memory");
        if (tid == 0) {
            __threadfence();
            int32_t* count = p.arrived + level * slots + to;
            const bool last = atomicAdd(count, 1) == n - 1;
            if (last) *count = 0;   // for the next call
            __threadfence();
            *scratch = last;
        }
        asm volatile("bar.sync %0, %1;" ::"n"(barrier), "n"(threads) : "memory");
        if (!*scratch) return;
        // a thread keeps to one row, `step` threads share the row's columns; eight columns of two parts are on their
        // way at a time.  (Loops stay rolled: this code runs once or twice a call, and every line of it is a miss.)
        int wide = 1;
        while (wide < rows) wide *= 2;
        const int r = tid & (wide - 1), step = threads / wide;
        if (r < rows && (n > 1 || last_level)) {
            const float2* ml = p.ml + level * slots * p.rows + r;
            float big = -kInf, sum = 0.f;
#pragma unroll 1
            for (int i = 0; i < n; ++i) big = fmaxf(big, __ldcg(ml + (int64_t)part_slot(first, (g0 + i) * stride) * p.rows).x);
            const float base = big == -kInf ? 0.f : big;
            const int rr = w.it.r0 + r, token = rr / p.G;
            T* out = reinterpret_cast<T*>(p.a.out) +
                     ((first_row(p.a.cu_drafts, w.b, p.a.kmax) + token) * p.a.Hq + w.h * p.G + rr - token * p.G) * (int64_t)p.a.D;
#pragma unroll 1
            for (int c0 = tid / wide; c0 < nc; c0 += 8 * step) {
                float4 y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                sum = 0.f;
#pragma unroll 2
                for (int i = 0; i < n; ++i) {
                    const int slot = part_slot(first, (g0 + i) * stride);
                    const float2 x = __ldcg(ml + (int64_t)slot * p.rows);
                    const float4* from = p.part + ((int64_t)slot * nc + c0) * p.rows + r;
                    float4 o[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) o[c] = c0 + c * step < nc ? __ldcg(from + c * step * p.rows) : y[c];
                    const float f = ex2(x.x - base);
                    sum = fmaf(f, x.y, sum);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        y[c] = make_float4(fmaf(f, o[c].x, y[c].x), fmaf(f, o[c].y, y[c].y), fmaf(f, o[c].z, y[c].z), fmaf(f, o[c].w, y[c].w));
                }
                const float inv = last_level ? 1.f / sum : 1.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c0 + c * step >= nc) break;
                    const float4 x = make_float4(y[c].x * inv, y[c].y * inv, y[c].z * inv, y[c].w * inv);
                    if (last_level)
                        put4(out + 4 * (c0 + c * step), x);
                    else
                        __stcg(p.part + ((int64_t)to * nc + c0 + c * step) * p.rows + r, x);
                }
            }
            if (!last_level && tid == r) __stcg(p.ml + ((level + 1) * slots + to) * p.rows + r, make_float2(big, sum));
        } else if (r < rows && tid == r) {   // a group of one: only its row sums move up
            const int64_t at = (int64_t)to * p.rows + r;
            __stcg(p.ml + (level + 1) * slots * p.rows + at, __ldcg(p.ml + level * slots * p.rows + at));
        }
        if (last_level) return;
        k /= kJoinFan;
        nodes = (nodes + kJoinFan - 1) / kJoinFan;
        stride *= kJoinFan;
    }
}

// The tensor-core kernel (attention_tc.cu): whether it takes the call, the rows of its groups, the CTAs of an
// SM, the launch.
bool tensor_path(const spec_attention_args* a);
int tensor_rows(const spec_attention_args* a);
int tensor_ctas_per_sm(const spec_attention_args* a);
cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s);

}  // namespace sv
