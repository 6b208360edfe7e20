// Sums of partial rows in a fixed order, shared by the gradients that add
// over feature rows.
#pragma once

#include "rowops.h"

namespace spc {

constexpr int kJoinCols = 16;        // lanes along the columns of a partial row

// V consecutive columns: one, or four where the rows' length is a multiple.
template <int V>
struct JoinVec {
    float f[V];
    __device__ __forceinline__ JoinVec& operator+=(const JoinVec& o) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += o.f[i];
        return *this;
    }
};

// Sums over `rows` rows of the V columns from e = V (block * kJoinCols +
// threadIdx.x % kJoinCols) of part (rows x n): SL slices of the rows per
// column, eight loads in flight, slices joined in order.  kJoinCols * SL
// threads; the result is valid in the first kJoinCols lanes (columns past n
// give 0).
template <int SL, int V>
__device__ __forceinline__ JoinVec<V> join_columns(const float* part, int64_t rows, int64_t n, int64_t block) {
    __shared__ JoinVec<V> s[SL][kJoinCols];
    const int col = threadIdx.x % kJoinCols, sl = threadIdx.x / kJoinCols;
    const int64_t e = (block * kJoinCols + col) * V;
    const int64_t per = (rows + SL - 1) / SL, r0 = min(rows, sl * per), r1 = min(rows, r0 + per);
    JoinVec<V> v = {};
    if (e < n) {
        for (int64_t r = r0; r < r1; r += 8) {
            JoinVec<V> t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float* p = part + min(r + k, r1 - 1) * n + e;
                if constexpr (V == 4) {
                    const f32x4r_t q = *(const f32x4r_t*)p;
                    t[k] = {q[0], q[1], q[2], q[3]};
                } else {
                    t[k].f[0] = *p;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r + k < r1) v += t[k];
        }
    }
    s[sl][col] = v;
    __syncthreads();
    JoinVec<V> t = {};
    if (sl == 0) {
#pragma unroll 8
        for (int k = 0; k < SL; ++k) t += s[k][col];
    }
    return t;
}

}  // namespace spc
