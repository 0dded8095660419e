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

struct AttnParams {
    spec_attention_args a;
    int G;            // query heads per key head
    int rows;         // rows of a full group
    int ctas;         // CTAs of the grid
    int page_shift;
    float scale_log2; // scale * log2(e)
    // workspace
    int32_t* header;  // [0] a wait gave up, [1] CTAs of the join that are done (both left at zero)
    int4* desc;       // [ctas] the item that CTA c begins and leaves to others: {stream, head, group, parts}
    float2* ml;       // [2 ctas][rows] maximum (of the scaled scores, base 2) and sum of a part's rows
    float* part;      // [2 ctas][rows][D] their weighted values, not yet divided
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

// Status of one stream, from its length and block (the pages are looked at by the join).
__device__ __forceinline__ bool length_ok(const AttnParams& p, int len, int n) {
    return len >= 0 && (int64_t)len + n <= (int64_t)p.a.max_pages << p.page_shift;
}

__device__ __forceinline__ int block_groups(const AttnParams& p, int n) { return (n * p.G + p.rows - 1) / p.rows; }

// Tiles of one key head of stream b (0 where the stream has no defined rows).
__device__ __forceinline__ int64_t stream_tiles(const AttnParams& p, int b) {
    const int len = __ldg(p.a.length + b), n = block_rows(p.a.cu_drafts, b, p.a.kmax);
    if (!length_ok(p, len, n)) return 0;
    int64_t t = 0;
    const int groups = block_groups(p, n);
    for (int g = 0; g < groups; ++g) t += make_item(p, len, n, g).tiles;
    return t;
}

// Where a CTA starts.  Computed by the whole block; valid after the call for every thread.
struct Start {
    int64_t tile;     // first tile of the CTA on the line
    int64_t span;     // tiles of every CTA (the last ones may get fewer, or none)
    int64_t total;
    int64_t head0;    // the line's position where stream `stream` begins
    int stream;       // stream that `tile` lies in
};

template <int kThreads>
__device__ __forceinline__ void find_start(const AttnParams& p, int cta, Start* s /* shared */,
                                           int64_t* scratch /* shared [kThreads / 32] */, int* iscratch /* shared */) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int valid = valid_prefix(p.a.cu_drafts, p.a.B, p.a.kmax, p.a.q_rows, p.a.B, iscratch);
    const int per = (valid + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, valid), b1 = min(b0 + per, valid);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += stream_tiles(p, b) * p.a.Hkv;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    before += x - mine;
    const int64_t span = (total + p.ctas - 1) / p.ctas;
    const int64_t at = (int64_t)cta * span;
    if (tid == 0) {
        s->tile = at;
        s->span = span;
        s->total = total;
        s->stream = 0;
        s->head0 = 0;
    }
    __syncthreads();
    if (at >= before && at < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const int64_t t = stream_tiles(p, b) * p.a.Hkv;
            if (at < before + t) {
                s->stream = b;
                s->head0 = before;
                break;
            }
            before += t;
        }
    }
    __syncthreads();
}

// The CTA's walk over its tiles, item by item.  Every role of a CTA walks by itself.
struct Walk {
    int b, h, g;          // item
    int len, n, groups;   // its stream
    Item it;
    int t0, t1;           // tiles [t0, t1) of the item are this CTA's
    int64_t left;         // tiles of the CTA from t0 on
    int64_t next_head;    // (t0's position - t0 + tiles): where the next item begins on the line

    __device__ __forceinline__ bool load_stream(const AttnParams& p) {
        len = __ldg(p.a.length + b);
        n = block_rows(p.a.cu_drafts, b, p.a.kmax);
        groups = block_groups(p, n);
        return length_ok(p, len, n);
    }
    __device__ __forceinline__ void take() {
        t1 = (int)min((int64_t)it.tiles, t0 + left);
    }
    // false: the CTA has no tiles
    __device__ __forceinline__ bool start(const AttnParams& p, const Start& s) {
        left = min(s.span, s.total - s.tile);
        if (left <= 0) return false;
        b = s.stream;
        load_stream(p);
        int64_t off = s.tile - s.head0;
        int64_t per_head = 0;
        for (int i = 0; i < groups; ++i) per_head += make_item(p, len, n, i).tiles;
        h = (int)(off / per_head);
        off -= h * per_head;
        for (g = 0;; ++g) {
            it = make_item(p, len, n, g);
            if (off < it.tiles) break;
            off -= it.tiles;
        }
        t0 = (int)off;
        next_head = s.tile - off + it.tiles;
        take();
        return true;
    }
    // to the next item; false: the CTA is done
    __device__ __forceinline__ bool next(const AttnParams& p) {
        left -= t1 - t0;
        if (left <= 0) return false;
        if (++g == groups) {
            g = 0;
            if (++h == p.a.Hkv) {
                h = 0;
                do ++b;
                while (!load_stream(p));   // some later stream has the tiles that are left
            }
        }
        it = make_item(p, len, n, g);
        t0 = 0;
        next_head += it.tiles;
        take();
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.tiles; }
    __device__ __forceinline__ bool begins_part() const { return t0 == 0 && t1 < it.tiles; }
    // parts of the item that CTA `cta` begins
    __device__ __forceinline__ int parts(int cta, int64_t span) const { return (int)((next_head - 1) / span) - cta + 1; }
    // slot of this CTA's part: an item is begun in the CTA's second slot and carried on in the first
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 == 0 ? 1 : 0); }
};

// Is position j visible to the row of token i (its own position is len + i)?
__device__ __forceinline__ bool visible(const AttnParams& p, int at, int j) {
    return j <= at && (p.a.window <= 0 || j > at - p.a.window || j < p.a.sinks);
}

// The tensor-core kernel (attention_tc.cu): whether it takes the call, the rows of its groups, the CTAs of an
// SM, the launch.
bool tensor_path(const spec_attention_args* a);
int tensor_rows(const spec_attention_args* a);
int tensor_ctas_per_sm(const spec_attention_args* a);
cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s);

}  // namespace sv
