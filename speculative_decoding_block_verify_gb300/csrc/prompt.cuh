// How a batch of prompts is cut into pieces, shared by the kernels of spec_prompt_attention.
//
// An item is (prompt, key head, piece of consecutive tokens): the rows of a piece are its tokens times the G query heads of the key
// head, row = token * G + query head, so that a product's 128 rows are full whatever G is and few of their scores lie above the
// diagonal.  Piece number l of a prompt sees about l pieces of keys: the later, the more work.  The items of all prompts are ranked by
// that number, the last pieces first, and the CTAs, as many as are resident, take them by turns, forwards and backwards (0 1 2 .. 2 1
// 0 0 1 ..): long and short prompts in one batch give every CTA nearly the same work, without a counter in memory and without the host
// knowing a length.  The rank of an item is not stored anywhere: a warp finds the item of a rank from how many pieces lie above a level.
#pragma once

#include "common.cuh"
#include "divisor.cuh"

namespace sv {

struct PromptParams {
    spec_prompt_args a;
    int G;             // query heads per key head
    int group;         // tokens of a group of up to 128 rows
    int piece;         // tokens of a piece
    int rows_each;     // without cu_rows: rows of a prompt
    Divisor by_G;
    float scale_log2;  // |scale| * log2(e)
};

// One item, as the walking warp tells it to the others.
struct Piece {
    int b, head;       // prompt, key head
    int n;             // tokens of the prompt
    int at, tokens;    // the piece's first token, and how many
    int64_t row0;      // the prompt's first packed row
};

// The keys that a piece's rows see, in tiles of kTile positions: those of the first tokens that stay visible, then the window's.
struct Keys {
    int low, high, sink;   // visible positions: [0, sink) and [low, high)
    int sink_tiles, first_tile, tiles;
};
template <int kTile>
__device__ __forceinline__ Keys keys_of(const PromptParams& p, int at, int tokens) {
    Keys k;
    k.high = at + tokens;
    k.low = p.a.window > 0 ? max(0, at + 1 - p.a.window) : 0;
    k.sink = min(p.a.sinks, k.low);
    k.sink_tiles = (k.sink + kTile - 1) / kTile;
    k.first_tile = max(k.low / kTile, k.sink_tiles);
    k.tiles = k.sink_tiles + (int)(((unsigned)k.high + kTile - 1) / kTile) - k.first_tile;
    return k;
}

// (there are fewer than 2^31 rows)
__device__ __forceinline__ int prompt_row(const PromptParams& p, int b) { return p.a.cu_rows == nullptr ? b * p.rows_each : *(p.a.cu_rows + b); }
// Offsets that break the packing at prompt b: it and the prompts behind it are not defined.
__device__ __forceinline__ bool prompt_broken(const PromptParams& p, int b, int row0, int end) {
    return end < row0 || (b == 0 && row0 != 0) || end > (int)p.a.rows;
}

// The CTA's items, found by one warp together (all 32 lanes call, all know the result).  A batch of kBatch prompts at a time: ranks go
// through the first batch's items, then the second's.  Ranks fit 32 bits: an item that is not a prompt's last has 64 rows of Q or more, 1 KB,
// and there are at most 2^26 last ones.  The code is short on purpose: it runs once an item beside all the other roles, and what it
// takes of the place where instructions are kept is theirs (54 KB of it, divided and unrolled without need, cost a prompt of 333 tokens 1.2 of 10.3 us
// and one of 1,000 tokens 2.6 of 24.8).
struct PromptWalk {
    static constexpr int kEach = 8, kBatch = 32 * kEach;
    int pieces[kEach];   // of prompt first + 32 i + lane
    int first;           // the batch's first prompt
    unsigned total;      // pieces of the batch
    unsigned base;       // items of the batches before
    unsigned round;
    int broken;          // the first prompt whose offsets are broken, as far as is known
    bool ended;          // no batch behind this one

    __device__ __forceinline__ unsigned above(int level) const {   // pieces of the batch with a number of `level` or more
        int s = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) s += max(0, pieces[i] - level);
        return __reduce_add_sync(0xffffffffu, (unsigned)s);
    }
    __device__ __forceinline__ void load(const PromptParams& p) {   // the batch at `first`
        const int lane = threadIdx.x & 31;
        int bad = INT32_MAX;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int b = first + 32 * i + lane;
            pieces[i] = 0;
            if (b < p.a.B) {
                const int row0 = prompt_row(p, b), end = prompt_row(p, b + 1);
                if (prompt_broken(p, b, row0, end))
                    bad = min(bad, b);
                else
                    pieces[i] = (int)(((unsigned)(end - row0) + p.piece - 1) / (unsigned)p.piece);
            }
        }
        bad = __reduce_min_sync(0xffffffffu, bad);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (first + 32 * i + lane >= bad) pieces[i] = 0;
        total = above(0);
        broken = bad;
        ended = bad != INT32_MAX || first + kBatch >= p.a.B;
    }
    __device__ __forceinline__ void start() {
        base = total = round = 0;
        first = -kBatch;
        broken = INT32_MAX;
        ended = false;
    }
    // The next item; false: there are no more.
    __device__ __forceinline__ bool next(const PromptParams& p, Piece* out) {
        const int lane = threadIdx.x & 31;
        const unsigned rank = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        ++round;
        while (rank >= base + total * (unsigned)p.a.Hkv) {
            if (ended) return false;
            base += total * (unsigned)p.a.Hkv;
            first += kBatch;
            load(p);
        }
        const unsigned at = rank - base, r = at / (unsigned)p.a.Hkv;
        out->head = (int)(at - r * (unsigned)p.a.Hkv);
        // the lowest level above which lie no more than r pieces
        int top = pieces[0];
#pragma unroll
        for (int i = 1; i < kEach; ++i) top = max(top, pieces[i]);
        int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)top) - 1;
        unsigned over = 0;   // pieces above level hi
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            const unsigned n = above(mid + 1);
            if (n <= r) {
                hi = mid;
                over = n;
            } else {
                lo = mid + 1;
            }
        }
        // the prompts with a piece of that level, in order: number r - over of them
        int nth = (int)(r - over), b = -1;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const unsigned has = __ballot_sync(0xffffffffu, pieces[i] > lo), me = 1u << lane;
            // the lane whose bit is there and has nth bits below its own
            if ((has & me) != 0 && __popc(has & (me - 1)) == nth) b = first + 32 * i + lane;
            nth -= __popc(has);
        }
        b = __reduce_max_sync(0xffffffffu, b);
        out->b = b;
        const int row0 = prompt_row(p, b);
        out->row0 = row0;
        out->n = prompt_row(p, b + 1) - row0;
        out->at = lo * p.piece;
        out->tokens = min(p.piece, out->n - out->at);
        return true;
    }
};

// The statuses, by the warp of every CTA that walked: CTA c has those of batches c, c + gridDim.x, .. of 32 prompts.  `mark` (or nullptr) is set
// where a wait has given up, which may be in another CTA and later: whoever sets it writes statuses behind that (prompt_gave_up), and whoever
// writes one looks at it behind that.
__device__ __forceinline__ void prompt_statuses(const PromptParams& p, PromptWalk& w, const int32_t* mark) {
    const int lane = threadIdx.x & 31;
    if ((int64_t)blockIdx.x * 32 >= p.a.B) return;
    while (!w.ended) {   // (a walk that was broken off, or had no item)
        w.first += PromptWalk::kBatch;
        w.load(p);
    }
    for (int64_t b = (int64_t)blockIdx.x * 32 + lane; b < p.a.B; b += (int64_t)gridDim.x * 32) {
        p.a.status[b] = b < w.broken ? SPEC_ST_OK : SPEC_ST_BAD_OFFSETS;
        if (mark == nullptr || b >= w.broken) continue;
        __threadfence();
        if (*reinterpret_cast<const volatile int32_t*>(mark) != 0) p.a.status[b] = SPEC_ST_TIMEOUT;
    }
}

// A wait of this CTA gave up: one warp sets the mark, leaves NaN in the rows of all its items, and has every prompt report it.
template <typename T>
__device__ __noinline__ void prompt_gave_up(const PromptParams& p, T nan, int32_t* mark) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) atomicExch(mark, 1);
    __syncwarp();
    __threadfence();
    PromptWalk w;
    Piece it;
    w.start();
    while (w.next(p, &it)) {
        const int per = p.G * p.a.D;
        for (int t = 0; t < it.tokens; ++t) {
            T* to = reinterpret_cast<T*>(p.a.out) + ((it.row0 + it.at + t) * p.a.Hq + (int64_t)it.head * p.G) * p.a.D;
            for (int i = lane; i < per; i += 32) to[i] = nan;
        }
    }
    for (int b = lane; b < p.a.B && b < w.broken; b += 32) p.a.status[b] = SPEC_ST_TIMEOUT;
}

cudaError_t launch_prompt_tc(const PromptParams& p, int sms, cudaStream_t s);    // bf16 (prompt_tc.cu)
cudaError_t launch_prompt_f32(const PromptParams& p, int sms, cudaStream_t s);   // float32 heads up to 128 (prompt_f32.cu)
cudaError_t mark_prompt_tc(int32_t marked, cudaStream_t s);    // each kernel's mark of a wait that gave up, on the current device
cudaError_t mark_prompt_f32(int32_t marked, cudaStream_t s);
// CTAs of a grid: what is resident, or fewer where there cannot be as many items.
inline int prompt_ctas(const PromptParams& p, int resident) {
    const int64_t items = (p.a.rows / p.piece + p.a.B) * p.a.Hkv;
    return (int)(items < resident ? items : resident);
}

}  // namespace sv
