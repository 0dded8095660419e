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
#include "divisor.cuh"

namespace sv {

constexpr int kTile = 64;          // positions of a tile
constexpr int kMaxCtas = 512;      // CTAs of an attention grid

// An item that lies across CTAs.  Part 0 is in the second slot of the CTA that begins it (an item is begun in a
// CTA's second slot and carried on in the first), part k in the first slot of the k-th CTA behind.
struct __align__(16) Unjoined {
    int32_t parts, rows;   // 0 rows: none
    int32_t r0, head;
    int64_t row0;          // the block's first packed row
    int64_t pad;
};

struct AttnParams {
    spec_attention_args a;
    int G;            // query heads per key head
    int rows;         // rows of a full group
    int ctas;         // CTAs of the grid
    int page_shift;
    Divisor by_G, by_rows;
    int item_cost;    // what beginning and ending an item takes, in tiles
    float scale_log2; // scale * log2(e)
    // workspace
    int32_t* timeout;  // a wait gave up (stays set)
    Unjoined* desc;    // [ctas] the item that CTA c begins and leaves to others
    float2* ml;        // [2 ctas][rows] maximum (of the scaled scores, base 2) and sum of a part's rows
    float4* part;      // [2 ctas][D / 4][rows] their weighted values, not yet divided
};

// The tiles of one item.
struct Item {
    int r0, r1;       // rows [r0, r1) of the block's rows * G
    int low, high;    // visible positions: [0, sink) and [low, high)
    int sink;
    int sink_tiles, first_tile, tiles;
};
// Tiles of n positions.  A table row may reach to 2^31 - 8 positions: rounded up to whole tiles they do not fit an int.
__device__ __forceinline__ int tiles_of(int n) { return (int)(((unsigned)n + kTile - 1) / kTile); }
__device__ __forceinline__ Item make_item(const AttnParams& p, int len, int block_rows, int group) {
    Item it;
    it.r0 = group * p.rows;
    it.r1 = min(it.r0 + p.rows, block_rows * p.G);
    const int i0 = p.by_G.of(it.r0), i1 = p.by_G.of(it.r1 - 1);
    it.high = len + i1 + 1;
    it.low = p.a.window > 0 ? max(0, len + i0 + 1 - p.a.window) : 0;
    it.sink = min(p.a.sinks, it.low);
    it.sink_tiles = tiles_of(it.sink);
    it.first_tile = max(it.low / kTile, it.sink_tiles);
    it.tiles = it.sink_tiles + tiles_of(it.high) - it.first_tile;
    return it;
}
// First position of tile t of the item.  Past the last tile it may not fit an int: the second form is for tiles that may be.
__device__ __forceinline__ int tile_start(const Item& it, int t) {
    return (t < it.sink_tiles ? t : it.first_tile + t - it.sink_tiles) * kTile;
}
__device__ __forceinline__ int tile_start_past(const Item& it, int t) {
    return (int)((unsigned)(t < it.sink_tiles ? t : it.first_tile + t - it.sink_tiles) * kTile);
}

__device__ __forceinline__ bool length_ok(const AttnParams& p, int len, int n) {
    return len >= 0 && (int64_t)len + n <= (int64_t)p.a.max_pages << p.page_shift;
}

__device__ __forceinline__ int block_groups(const AttnParams& p, int n) { return p.by_rows.of(n * p.G + p.rows - 1); }

// Length on the line of one key head of a stream (0 where its length is not in its table row).
__device__ __forceinline__ int64_t head_cost(const AttnParams& p, int len, int n) {
    if (!length_ok(p, len, n)) return 0;
    int64_t t = 0;
    const int groups = block_groups(p, n);
    for (int g = 0; g < groups; ++g) t += make_item(p, len, n, g).tiles + p.item_cost;
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
            const int len = *(p.a.length + b);
            int n = p.a.kmax + 1;
            if (cu != nullptr) {
                const int c0 = *(cu + b), c1 = *(cu + b + 1);
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
            const int64_t t = head_cost(p, *(p.a.length + b), block_rows(cu, b, p.a.kmax)) * p.a.Hkv;
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

// The CTA's walk over its tiles, item by item.  Every role of a CTA walks by itself.  An item takes item_cost +
// tiles positions of the line: a CTA that ends in the first item_cost of them leaves the item to the next one.
struct Walk {
    int b, h, g;          // item
    int len, n, groups;   // its stream
    Item it;
    int t0, t1;           // tiles [t0, t1) of the item are this CTA's
    int64_t end;          // where the item ends on the line
    int64_t stop;         // where the CTA ends

    __device__ __forceinline__ bool load_stream(const AttnParams& p) {
        len = *(p.a.length + b);
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
        end += it.tiles + p.item_cost;
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
            if (off < it.tiles + p.item_cost) break;
            off -= it.tiles + p.item_cost;
        }
        end = s.at - off + it.tiles + p.item_cost;
        t0 = max(0, (int)off - p.item_cost);
        return take();
    }
    // to the CTA's next item; false: the CTA is done
    __device__ __forceinline__ bool next(const AttnParams& p) {
        if (end >= stop) return false;
        step(p);
        return take();
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.tiles; }
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 == 0 ? 1 : 0); }
    __device__ __forceinline__ bool begins_part() const { return t0 == 0 && t1 < it.tiles; }
    __device__ __forceinline__ Unjoined unjoined(const AttnParams& p, int cta, int64_t span) const {
        return {(int)quotient(end - 1, span) - cta + 1, it.r1 - it.r0, it.r0, h, first_row(p.a.cu_drafts, b, p.a.kmax), 0};
    }
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
            const int len = *(p.a.length + b), n = block_rows(p.a.cu_drafts, b, p.a.kmax);
            if (!length_ok(p, len, n)) {
                st = SPEC_ST_BAD_LENGTH;
                T* to = reinterpret_cast<T*>(p.a.out) + first_row(p.a.cu_drafts, b, p.a.kmax) * p.a.Hq * (int64_t)p.a.D;
                for (int64_t i = lane; i < (int64_t)n * p.a.Hq * p.a.D; i += 32) put(to + i, __int_as_float(0x7fffffff));
            } else {
                const int low = p.a.window > 0 ? max(0, len + 1 - p.a.window) : 0;
                const int sp = (int)(((unsigned)min(p.a.sinks, low) + p.a.page_size - 1) >> p.page_shift), lp = low >> p.page_shift;
                const int hp = (int)(((unsigned)(len + n) + p.a.page_size - 1) >> p.page_shift);
                const int32_t* table = p.a.page_table + (int64_t)b * p.a.max_pages;
                bool bad = false;
                for (int j = lane; j < sp && j < lp; j += 32) bad |= (unsigned)*(table + j) >= (unsigned)p.a.num_pages;
#pragma unroll 8
                for (int j = lp + lane; j < hp; j += 32) bad |= (unsigned)*(table + j) >= (unsigned)p.a.num_pages;
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

// The tensor-core kernel (attention_tc.cu): bf16.
int tensor_rows(const spec_attention_args* a);          // rows of a group
int tensor_ctas_per_sm(const spec_attention_args* a);
bool tensor_q(const spec_attention_args* a);            // q's rows can be copied as they lie
cudaError_t launch_attention_tc(const AttnParams& p, void* q_packed, cudaStream_t s);
// ... for float32 heads up to 128 (attention_f32.cu); same groups, one CTA an SM.
cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s);

}  // namespace sv
