// Where a workgroup stands among packed sequences whose offsets are on the
// device, shared by the operators over the rows of a scene.
#pragma once

#include "rowops.h"

namespace spc {

// Tiles of `rows` rows over the sequences without a list of them: sequence b's
// tile i has place floor(offsets[b] per / rows) + b + i, which leaves each
// sequence at least as many places as it has tiles and none to share; some
// places stay empty.  All 64 lanes search together.
struct Place {
    int b, tile;
    int64_t q0, k0;
    int Lq, Lk;       // positions and keys of the sequence
};
__device__ __forceinline__ int64_t clamp_to(int64_t x, int64_t lo, int64_t hi) {
    return x < lo ? lo : x > hi ? hi : x;
}
__device__ __forceinline__ Place find_place(const int32_t* offs, int B, int64_t n, int per, int rows, int64_t item) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int64_t i = (int64_t)lo + (int64_t)(lane + 1) * step;
        const bool below = i < hi && clamp_to(offs[i], 0, n) * per / rows + i <= item;
        const int c = __popcll(__ballot(below));
        lo += c * step;
        hi = min(hi, lo + step);
    }
    lo = __builtin_amdgcn_readfirstlane(min(lo, B - 1));
    Place p;
    p.b = lo;
    const int64_t a = clamp_to(offs[lo], 0, n);
    const int64_t e = clamp_to(offs[lo + 1], a, n);
    p.q0 = a;
    p.Lq = (int)(e - a);
    const int64_t t = item - (a * per / rows + lo);
    p.tile = t < 0 || t * rows >= (int64_t)p.Lq * per ? -1 : (int)t;
    return p;
}

// The row of a position; whatever `order` holds, one of the n rows.
__device__ __forceinline__ int64_t row_of(const int32_t* order, int64_t pos, int64_t n) {
    return order ? (int64_t)min((uint32_t)order[pos], (uint32_t)n - 1) : pos;
}

}  // namespace spc
