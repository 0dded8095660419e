// The packed blocks of a verify step and their pages, as the cache calls read them.  (Plain loads throughout: these
// kernels start while the one before them still writes, and the read-only path is not ordered by
// griddepcontrol.wait.)
#pragma once

#include "common.cuh"

namespace sv {

// Streams [0, valid_prefix) have defined rows: cu[0] = 0, every count up to theirs lies in [0,
// kmax], and their rows are among the `rows` that the caller passed.  Every thread of the block calls this; `scratch` is one shared int.
__device__ __forceinline__ int valid_prefix(const int32_t* cu, int B, int kmax, int64_t rows, int upto, int* scratch) {
    if (cu == nullptr) return B;
    if (threadIdx.x == 0) *scratch = B;
    __syncthreads();
    int bad = B;
    for (int b = threadIdx.x; b < upto; b += blockDim.x) {
        const int c0 = *(cu + b), n = *(cu + b + 1) - c0;
        if (n < 0 || n > kmax || (b == 0 && c0 != 0) || (int64_t)c0 + n + b + 1 > rows) {
            bad = b;
            break;
        }
    }
    if (bad < B) atomicMin(scratch, bad);
    __syncthreads();
    return *scratch;
}

// First packed row of stream b's block, and its number of rows (N_b + 1).
__device__ __forceinline__ int64_t first_row(const int32_t* cu, int b, int kmax) {
    return cu == nullptr ? (int64_t)b * (kmax + 1) : (int64_t)*(cu + b) + b;
}
__device__ __forceinline__ int block_rows(const int32_t* cu, int b, int kmax) {
    return cu == nullptr ? kmax + 1 : *(cu + b + 1) - *(cu + b) + 1;
}

}  // namespace sv
