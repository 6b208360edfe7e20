// Device helpers shared by the row-wise operators (layer norm, gated linear
// unit, gated recurrence): 16-byte pieces of a feature row in either element
// type, and sums over lane groups.
#pragma once

#include "spconv_internal.h"

namespace spc {

typedef __bf16 bf16x8r_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8ru_t __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4r_t __attribute__((ext_vector_type(4)));
typedef float f32x4ru_t __attribute__((ext_vector_type(4), aligned(4)));

// A row is read in pieces of 16 bytes.  Rows need only be aligned to their
// element: gfx950 serves 16-byte global accesses at any element address, so
// odd channel counts keep the wide pieces (the last one is cut).
template <typename T>
struct Piece;
template <>
struct Piece<__bf16> {
    static constexpr int V = 8;
    typedef bf16x8r_t vec;
    typedef bf16x8ru_t uvec;
};
template <>
struct Piece<float> {
    static constexpr int V = 4;
    typedef f32x4r_t vec;
    typedef f32x4ru_t uvec;
};

// The n <= V elements at p (n may be <= 0: nothing is read); the rest are 0.
template <typename T>
__device__ __forceinline__ typename Piece<T>::vec load_piece(const T* p, int n) {
    constexpr int V = Piece<T>::V;
    typename Piece<T>::vec v;
    if (n >= V) {
        v = *(const typename Piece<T>::uvec*)p;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? p[i] : (T)0.f;
    }
    return v;
}

// Outputs larger than this are written past the caches: nothing of them would
// be left there for the next kernel, and they would push out its inputs (half
// of the 256 MB memory-side cache).
constexpr int64_t kStreamBytes = 128 << 20;
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&f)[Piece<T>::V], int n, bool stream) {
    constexpr int V = Piece<T>::V;
    typename Piece<T>::vec v;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (T)f[i];
    if (n >= V) {
        typename Piece<T>::uvec* q = (typename Piece<T>::uvec*)p;
        if (stream)
            __builtin_nontemporal_store((typename Piece<T>::uvec)v, q);
        else
            *q = v;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = v[i];
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Sum over the L consecutive lanes (L a power of two up to 64, groups aligned
// to L); every lane of a group gets the same bits.  Lane moves of the vector
// unit only, no LDS.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
    if constexpr (L >= 2) x += dpp_move<0xB1>(x);        // quad_perm [1,0,3,2]
    if constexpr (L >= 4) x += dpp_move<0x4E>(x);        // quad_perm [2,3,0,1]
    if constexpr (L >= 8) x += dpp_move<0x141>(x);       // row_half_mirror
    if constexpr (L >= 16) x += dpp_move<0x140>(x);      // row_mirror
    if constexpr (L >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (L >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return x;
}

}  // namespace spc
