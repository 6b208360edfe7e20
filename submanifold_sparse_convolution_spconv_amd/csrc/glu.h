// Shared by the gated linear unit's kernels: arguments, activations, stores.
#pragma once

#include "rowops.h"

namespace spc {

typedef __bf16 bf16x4r_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4r_t lds_bf16x4r_t;

struct GluParams {
    const void* x;
    const void* w;
    const float* bias;
    const void* dout;
    void* h;           // forward
    void* dab;         // (N, 2, F): da, db
    void* dx;
    void* dw;
    float* bpart;      // [row tiles][2][F] partial sums of dbias; or NULL
    float* wpart;      // [splits][C][2 F] partial sums of dw; NULL: one split, into dw
    float* xpart;      // [dx splits][N][C] partial sums of dx; NULL: one split, into dx
    int64_t N;
    int C, F;
    int64_t rows_per_split;
    int dx_splits, dx_per;      // of dx's reduction (2 F), and its length
    int64_t first_block;        // of this launch (tiles: a call may need several)
    bool stream;       // outputs past the caches
};

__device__ __forceinline__ float fast_sigmoid(float a) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896f * a));
}

// act(a) and act'(a).  FINE: to the precision of fp32 outputs, in a GELU's tail
// too.
struct Act {
    float v, d;
};
template <int ACT, bool FINE = false>
__device__ __forceinline__ Act activation(float a) {
    if constexpr (ACT == SPCONV_SILU) {
        const float s = fast_sigmoid(a);
        const float v = a * s;
        // s (1 + a (1 - s)): 1 - s is exact from s = 1/2 on and 0 where s is 1, so
        // that the 1 is not lost next to a large a
        return {v, fmaf(v, 1.f - s, s)};
    } else {
        // The normal distribution from erfc(x) = t P(t) e^(-x^2), t = 1 / (1 + p x);
        // the density needs the same exponential.  For bfloat16 outputs
        // Abramowitz and Stegun 7.1.26, off by 1.5e-7 at most, which in the tail is
        // 5e-5 of the value at a = -3 and 1.5% at -9.  FINE: nine degrees, fitted here
        // by least squares with weights that even out the relative error, to 7e-9 of
        // the value up to where the exponential vanishes (x = 9.4).
        const float x = fabsf(a) * 0.70710678f;
        const float t = __builtin_amdgcn_rcpf(fmaf(FINE ? 0.4f : 0.3275911f, x, 1.f));
        const float e = __builtin_amdgcn_exp2f(-0.72134752f * a * a);
        float q;
        if constexpr (FINE) {
            q = fmaf(-0.0305951991f, t, 0.2034744751f);
            q = fmaf(q, t, -0.5117215136f);
            q = fmaf(q, t, 0.5647543606f);
            q = fmaf(q, t, -0.2988673864f);
            q = fmaf(q, t, 0.2799084512f);
            q = fmaf(q, t, 0.1269454937f);
            q = fmaf(q, t, 0.2155105960f);
            q = fmaf(q, t, 0.2248800748f);
            q = fmaf(q, t, 0.2257106544f);
        } else {
            q = fmaf(1.061405429f, t, -1.453152027f);
            q = fmaf(q, t, 1.421413741f);
            q = fmaf(q, t, -0.284496736f);
            q = fmaf(q, t, 0.254829592f);
        }
        q *= 0.5f * t * e;
        const float cdf = a >= 0.f ? 1.f - q : q;
        return {a * cdf, fmaf(0.39894228f * a, e, cdf)};
    }
}

template <typename T>
struct Four;
template <>
struct Four<__bf16> {
    typedef bf16x4r_t vec;
};
template <>
struct Four<float> {
    typedef f32x4r_t vec;
};
// E (4 or 8) consecutive elements.
template <typename T, int E>
struct Group {
    typedef T vec __attribute__((ext_vector_type(E)));
};
template <typename T>
__device__ __forceinline__ void store_four(T* p, const float (&f)[4]) {
    typename Four<T>::vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)f[i];
    *(typename Four<T>::vec*)p = v;
}

// bfloat16 rows of at most kGluRowC channels: both projections of a row come
// from weights that stay in LDS (glu_rows.hip).
constexpr int kGluRowC = 128;
hipError_t launch_glu_rows(const GluParams& p, int act, hipStream_t st);
hipError_t launch_glu_rows_dx(const GluParams& p, int act, hipStream_t st);
// dw's and dbias' partial sums: `splits` splits of rows_per_split rows; the
// number of splits that fills the card.
int glu_rows_splits(int64_t N, int C, int F);
hipError_t launch_glu_rows_dw(const GluParams& p, int act, int splits, hipStream_t st);

}  // namespace spc
