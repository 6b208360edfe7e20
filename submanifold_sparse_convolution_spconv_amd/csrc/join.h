// Sums of partial rows in a fixed order, shared by the gradients that add
// over feature rows.
#pragma once

#include "rowops.h"

namespace spc {

constexpr int kJoinCols = 16;        // columns per workgroup: 64 contiguous bytes of each partial row

// Sum over `rows` rows of column e = block * kJoinCols + threadIdx.x %
// kJoinCols of part (rows x n): SL slices of the rows per column, eight loads
// in flight, slices joined in order.  kJoinCols * SL threads; the result is
// valid in the first kJoinCols lanes (columns past n give 0).
template <int SL>
__device__ __forceinline__ float join_column(const float* part, int64_t rows, int64_t n, int64_t block) {
    __shared__ float s[SL][kJoinCols + 1];
    const int col = threadIdx.x % kJoinCols, sl = threadIdx.x / kJoinCols;
    const int64_t e = block * kJoinCols + col;
    const int64_t per = (rows + SL - 1) / SL, r0 = min(rows, sl * per), r1 = min(rows, r0 + per);
    float v = 0.f;
    if (e < n) {
        for (int64_t r = r0; r < r1; r += 8) {
            float t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = part[min(r + k, r1 - 1) * n + e];
#pragma unroll
            for (int k = 0; k < 8; ++k) v += r + k < r1 ? t[k] : 0.f;
        }
    }
    s[sl][col] = v;
    __syncthreads();
    float t = 0.f;
    if (sl == 0) {
#pragma unroll 8
        for (int k = 0; k < SL; ++k) t += s[k][col];
    }
    return t;
}

}  // namespace spc
