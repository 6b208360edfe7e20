// Gated linear unit of feature rows and its gradient for gfx950.
//
//   a = x w[0] + b[0],  b = x w[1] + b[1],  h = act(a) b
//
// with w (2, C, F), and from dh the gradient
//
//   da = dh b act'(a),  db = dh act(a),
//   dx = da w[0]^T + db w[1]^T,  dw[s] = x^T (da | db),  dbias[s] = sum_n (da | db)
//
// All products run on the matrix cores with fp32 accumulators, transposed
// (D = W^T x^T), so that a lane ends up with four consecutive features of one
// row: activations, their derivatives and the stores work on 8- or 16-byte
// pieces without a shuffle.  Operands go through LDS; the one whose reduction
// axis is not contiguous in memory is read back with the transposing LDS read
// (bf16) or one word per lane (fp32).
#include "glu.h"
#include "join.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kGluThreads = 256;

// One operand tile in LDS: M outputs x BK of the reduction.  KC: the reduction
// is contiguous in memory and in LDS ([m][k]); else the outputs are ([k][m]).
// The pitches keep the fragment reads free of bank conflicts.
template <typename T, bool KC, int M, int BK>
struct Stage {
    static constexpr bool K_CONTIGUOUS = KC;
    static constexpr int V = Piece<T>::V;
    static constexpr int PER = M * BK / V / kGluThreads;        // pieces per thread
    static constexpr int PITCH = KC ? BK + V : M + (sizeof(T) == 2 ? 8 : 16);
    static constexpr int ELEMS = (KC ? M : BK) * PITCH;
    static_assert(PER >= 1 && M * BK / V % kGluThreads == 0, "whole pieces per thread");
    // piece j of this thread: output m and reduction index k of its first element
    static __device__ __forceinline__ void where(int j, int& m, int& k) {
        const int p = threadIdx.x + kGluThreads * j;
        if constexpr (KC) {
            m = p / (BK / V);
            k = p % (BK / V) * V;
        } else {
            k = p / (M / V);
            m = p % (M / V) * V;
        }
    }
    static __device__ __forceinline__ void put(T* lds, int j, typename Piece<T>::vec v) {
        int m, k;
        where(j, m, k);
        *(typename Piece<T>::vec*)(lds + (KC ? m * PITCH + k : k * PITCH + m)) = v;
    }
};

// 16 x 16 output tiles: fragment of outputs m0 .. m0+15 for one matrix
// instruction (bf16: 32 of the reduction, fp32: 4)
template <typename T>
struct Frag;
template <>
struct Frag<__bf16> {
    static constexpr int K = 32;
    typedef bf16x8r_t type;
    template <class S>
    static __device__ __forceinline__ type read(const __bf16* lds, int m0, int k0) {
        const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        if constexpr (S::K_CONTIGUOUS) {
            return *(const type*)(lds + (m0 + a) * S::PITCH + k0 + 8 * g);
        } else {
            // lane a of group g addresses row 8 g (+ 4) + a / 4, columns
            // 4 (a % 4) ..; it receives column a of the four rows
            const __bf16* p = lds + (k0 + 8 * g + (a >> 2)) * S::PITCH + m0 + 4 * (a & 3);
            const bf16x4r_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4r_t*)p);
            const bf16x4r_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4r_t*)(p + 4 * S::PITCH));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    static __device__ __forceinline__ f32x4r_t mma(type a, type b, f32x4r_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<float> {
    static constexpr int K = 4;
    typedef float type;
    template <class S>
    static __device__ __forceinline__ type read(const float* lds, int m0, int k0) {
        const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        return S::K_CONTIGUOUS ? lds[(m0 + a) * S::PITCH + k0 + g] : lds[(k0 + g) * S::PITCH + m0 + a];
    }
    static __device__ __forceinline__ f32x4r_t mma(type a, type b, f32x4r_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
    }
};

template <typename T>
constexpr int kTileK = sizeof(T) == 2 ? 32 : 16;
constexpr int kTile = 128;     // outputs of each kind per workgroup

// acc += A B over the reduction [k0, k1), both operands staged a BK at a time
// with the next tiles' loads in flight.  load_a / load_b (m, k) give the piece
// at output m and reduction index k (0 outside); m_at / n_at the first output
// of this wave's i-th / j-th 16-wide tile.
template <typename T, bool AKC, bool BKC, class LA, class LB, class MA, class NA>
__device__ __forceinline__ void tile_product(f32x4r_t (&acc)[4][4], int64_t k0, int64_t k1, LA load_a, LB load_b,
                                             MA m_at, NA n_at) {
    constexpr int BK = kTileK<T>;
    using A = Stage<T, AKC, kTile, BK>;
    using B = Stage<T, BKC, kTile, BK>;
    __shared__ __align__(16) T la[A::ELEMS];
    __shared__ __align__(16) T lb[B::ELEMS];
    typename Piece<T>::vec ra[A::PER], rb[B::PER];
    auto fetch = [&](int64_t k) {
        int m, kk;
#pragma unroll
        for (int j = 0; j < A::PER; ++j) {
            A::where(j, m, kk);
            ra[j] = load_a(m, k + kk);
        }
#pragma unroll
        for (int j = 0; j < B::PER; ++j) {
            B::where(j, m, kk);
            rb[j] = load_b(m, k + kk);
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
    fetch(k0);
    for (int64_t k = k0; k < k1; k += BK) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < A::PER; ++j) A::put(la, j, ra[j]);
#pragma unroll
        for (int j = 0; j < B::PER; ++j) B::put(lb, j, rb[j]);
        __syncthreads();
        if (k + BK < k1) fetch(k + BK);
#pragma unroll
        for (int s = 0; s < BK; s += Frag<T>::K) {
            typename Frag<T>::type fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = Frag<T>::template read<A>(la, m_at(i), s);
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j] = Frag<T>::template read<B>(lb, n_at(j), s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = Frag<T>::mma(fa[i], fb[j], acc[i][j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ typename Piece<T>::vec piece_or_zero(const T* p, bool in) {
    typename Piece<T>::vec v;
    if (in) {
        v = *(const typename Piece<T>::vec*)p;
    } else {
#pragma unroll
        for (int i = 0; i < Piece<T>::V; ++i) v[i] = (T)0.f;
    }
    return v;
}

// 128 rows x 64 hidden features, both projections: h, or (GRAD) da and db with
// their sums over the tile's rows.
template <typename T, int ACT, bool GRAD>
__global__ void __launch_bounds__(kGluThreads) k_glu_project(GluParams p) {
    __shared__ float bsum[2][2][64];
    const int wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F;
    const int ft = (F + 63) / 64, f0 = (int)(blockIdx.x % ft) * 64;
    const int64_t tile = blockIdx.x / ft, r0 = tile * kTile;
    const T* x = (const T*)p.x;
    const T* w = (const T*)p.w;
    f32x4r_t acc[4][4];        // [0, 1]: a, [2, 3]: b, of 16 features each
    tile_product<T, false, true>(
        acc, 0, C,
        [&](int m, int64_t k) {
            const int s = m >> 6, f = f0 + (m & 63);
            return piece_or_zero(w + ((int64_t)s * C + k) * F + f, k < C && f < F);
        },
        [&](int n, int64_t k) { return piece_or_zero(x + (r0 + n) * C + k, r0 + n < p.N && k < C); },
        [&](int i) { return 64 * (i >> 1) + 32 * wm + 16 * (i & 1); }, [&](int j) { return 64 * wn + 16 * j; });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int fl = 32 * wm + 16 * i + 4 * g, f = f0 + fl;
        f32x4r_t ba = {0.f, 0.f, 0.f, 0.f}, bb = ba;
        if (p.bias && f < F) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ba[e] = p.bias[f + e];
                bb[e] = p.bias[F + f + e];
            }
        }
        f32x4r_t sa = {0.f, 0.f, 0.f, 0.f}, sb = sa;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 64 * wn + 16 * j + a;
            if (r >= p.N || f >= F) continue;
            const f32x4r_t va = acc[i][j] + ba, vb = acc[i + 2][j] + bb;
            float o[4], q[4];
            if constexpr (!GRAD) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = activation<ACT>(va[e]).v * vb[e];
                store_four((T*)p.h + r * F + f, o);
            } else {
                const typename Four<T>::vec dh = *(const typename Four<T>::vec*)((const T*)p.dout + r * F + f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Act t = activation<ACT>(va[e]);
                    o[e] = (float)dh[e] * vb[e] * t.d;
                    q[e] = (float)dh[e] * t.v;
                    sa[e] += o[e];
                    sb[e] += q[e];
                }
                T* d = (T*)p.dab + r * 2 * F + f;
                store_four(d, o);
                store_four(d + F, q);
            }
        }
        if constexpr (GRAD) {
            if (p.bpart) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = group_sum<16>(sa[e]), v = group_sum<16>(sb[e]);
                    if (a == 0) {
                        bsum[wn][0][fl + e] = u;
                        bsum[wn][1][fl + e] = v;
                    }
                }
            }
        }
    }
    if constexpr (GRAD) {
        if (!p.bpart) return;
        __syncthreads();
        const int s = threadIdx.x >> 6, f = threadIdx.x & 63;
        if (threadIdx.x < 128 && f0 + f < F)
            p.bpart[(tile * 2 + s) * F + f0 + f] = bsum[0][s][f] + bsum[1][s][f];
    }
}

// dx: 128 rows x 128 channels, reduced over both halves of dab.
template <typename T>
__global__ void __launch_bounds__(kGluThreads) k_glu_dx(GluParams p) {
    const int wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F;
    const int ct = (C + kTile - 1) / kTile, c0 = (int)(blockIdx.x % ct) * kTile;
    const int64_t r0 = (int64_t)(blockIdx.x / ct) * kTile;
    const T* w = (const T*)p.w;
    const T* dab = (const T*)p.dab;
    f32x4r_t acc[4][4];
    tile_product<T, true, true>(
        acc, 0, 2 * F,
        [&](int m, int64_t k) {
            const int c = c0 + m;
            const int64_t at = k < F ? (int64_t)c * F + k : (int64_t)(C + c) * F + (k - F);
            return piece_or_zero(w + at, c < C && k < 2 * F);
        },
        [&](int n, int64_t k) { return piece_or_zero(dab + (r0 + n) * 2 * F + k, r0 + n < p.N && k < 2 * F); },
        [&](int i) { return 64 * wm + 16 * i; }, [&](int j) { return 64 * wn + 16 * j; });
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = c0 + 64 * wm + 16 * i + 4 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 64 * wn + 16 * j + a;
            if (r >= p.N || c >= C) continue;
            const float o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            store_four((T*)p.dx + r * C + c, o);
        }
    }
}

// Partial dw of one split of the rows: 128 columns of dab x 128 channels.
template <typename T>
__global__ void __launch_bounds__(kGluThreads) k_glu_dw(GluParams p) {
    const int wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F2 = 2 * p.F;
    const int m0 = blockIdx.x * kTile, c0 = blockIdx.y * kTile;
    const int64_t k0 = (int64_t)blockIdx.z * p.rows_per_split, k1 = min(p.N, k0 + p.rows_per_split);
    const T* x = (const T*)p.x;
    const T* dab = (const T*)p.dab;
    f32x4r_t acc[4][4];
    tile_product<T, false, false>(
        acc, k0, k1,
        [&](int m, int64_t k) { return piece_or_zero(dab + k * F2 + m0 + m, k < k1 && m0 + m < F2); },
        [&](int n, int64_t k) { return piece_or_zero(x + k * C + c0 + n, k < k1 && c0 + n < C); },
        [&](int i) { return 64 * wm + 16 * i; }, [&](int j) { return 64 * wn + 16 * j; });
    float* part = p.wpart + (int64_t)blockIdx.z * C * F2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + 64 * wm + 16 * i + 4 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + 64 * wn + 16 * j + a;
            if (m < F2 && c < C) *(f32x4r_t*)(part + (int64_t)c * F2 + m) = acc[i][j];
        }
    }
}

// dw[s][c][f]: the splits' partials (C, 2 F) added in their order, rounded once.
template <typename T>
__global__ void __launch_bounds__(kJoinCols * 16) k_glu_dw_join(const float* part, int splits, int C, int F, T* dw) {
    const int64_t n = (int64_t)C * 2 * F;
    const float t = join_column<16>(part, splits, n);
    const int64_t e = (int64_t)blockIdx.x * kJoinCols + threadIdx.x;
    if (threadIdx.x >= kJoinCols || e >= n) return;
    const int64_t c = e / (2 * F);
    const int m = (int)(e % (2 * F));
    dw[m < F ? c * F + m : (C + c) * F + (m - F)] = (T)t;
}

__global__ void __launch_bounds__(kJoinCols * 64) k_glu_dbias_join(const float* part, int64_t tiles, int n,
                                                                   float* dbias) {
    const float t = join_column<64>(part, tiles, n);
    const int e = blockIdx.x * kJoinCols + threadIdx.x;
    if (threadIdx.x < kJoinCols && e < n) dbias[e] = t;
}

// Few channels and enough rows to give every CU a block of them: glu_rows.hip.
bool use_rows(int64_t N, int C, int dtype) { return dtype == SPCONV_BF16 && C <= kGluRowC && N >= 32768; }

struct GluLayout {
    size_t dab, bpart, wpart, total;
    int64_t tiles, rows_per_split;
    int splits;
};
GluLayout glu_layout(int64_t N, int C, int F, int dtype) {
    GluLayout l{};
    if (use_rows(N, C, dtype)) {
        const int want = glu_rows_splits(N, F);
        l.rows_per_split = round_up((N + want - 1) / want, 64);
        l.splits = (int)((N + l.rows_per_split - 1) / l.rows_per_split);
        l.tiles = l.splits;
        l.wpart = align_up((size_t)l.splits * 2 * F * 4, 256);
        l.total = l.wpart + align_up((size_t)l.splits * C * 2 * F * 4, 256);
        return l;
    }
    l.tiles = (N + kTile - 1) / kTile;
    // enough workgroups for four per CU, at least 512 rows each
    const int64_t t = (int64_t)((2 * F + kTile - 1) / kTile) * ((C + kTile - 1) / kTile);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>((1024 + t - 1) / t, (N + 511) / 512));
    l.rows_per_split = round_up((N + want - 1) / std::max<int64_t>(want, 1), 32);
    l.splits = l.rows_per_split ? (int)((N + l.rows_per_split - 1) / l.rows_per_split) : 0;
    size_t at = 0;
    l.dab = at;
    at += align_up((size_t)N * 2 * F * (dtype == SPCONV_BF16 ? 2 : 4), 256);
    l.bpart = at;
    at += align_up((size_t)l.tiles * 2 * F * 4, 256);
    l.wpart = at;
    at += align_up((size_t)l.splits * C * 2 * F * 4, 256);
    l.total = at;
    return l;
}

template <typename T>
hipError_t glu_join(const GluParams& p, const GluLayout& l, void* dw, float* dbias, hipStream_t st) {
    const int64_t n = (int64_t)p.C * 2 * p.F;
    k_glu_dw_join<T><<<(unsigned)((n + kJoinCols - 1) / kJoinCols), kJoinCols * 16, 0, st>>>(p.wpart, l.splits, p.C,
                                                                                             p.F, (T*)dw);
    if (dbias)
        k_glu_dbias_join<<<(2 * p.F + kJoinCols - 1) / kJoinCols, kJoinCols * 64, 0, st>>>(p.bpart, l.tiles, 2 * p.F,
                                                                                           dbias);
    return hipGetLastError();
}

template <typename T, int ACT>
hipError_t glu_go(const GluParams& p, bool grad, const GluLayout& l, void* dw, float* dbias, hipStream_t st) {
    // row tiles in the first grid dimension, next to the tiles of their columns
    const unsigned proj = (unsigned)(l.tiles * ((p.F + 63) / 64));
    if (!grad) {
        k_glu_project<T, ACT, false><<<proj, kGluThreads, 0, st>>>(p);
        return hipGetLastError();
    }
    const int ct = (p.C + kTile - 1) / kTile;
    if (p.N > 0) {
        k_glu_project<T, ACT, true><<<proj, kGluThreads, 0, st>>>(p);
        k_glu_dx<T><<<(unsigned)(l.tiles * ct), kGluThreads, 0, st>>>(p);
        k_glu_dw<T><<<dim3((2 * p.F + kTile - 1) / kTile, ct, l.splits), kGluThreads, 0, st>>>(p);
    }
    return glu_join<T>(p, l, dw, dbias, st);
}

}  // namespace

size_t glu_grad_workspace_bytes(int64_t N, int C, int F, int dtype) { return glu_layout(N, C, F, dtype).total; }

hipError_t launch_glu(const GluArgs& a, bool grad, hipStream_t stream) {
    if (a.N == 0 && !grad) return hipSuccess;
    const GluLayout l = glu_layout(a.N, a.C, a.F, a.dtype);
    GluParams p{};
    p.x = a.x;
    p.w = a.w;
    p.bias = a.bias;
    p.dout = a.dout;
    p.h = a.out;
    p.dx = a.out;
    if (grad) {
        char* ws = (char*)a.workspace;
        p.dab = ws + l.dab;
        p.bpart = a.dbias ? (float*)(ws + l.bpart) : nullptr;
        p.wpart = (float*)(ws + l.wpart);
    }
    p.N = a.N;
    p.C = a.C;
    p.F = a.F;
    p.rows_per_split = l.rows_per_split;
    p.stream = a.N * (grad ? a.C : a.F) * (a.dtype == SPCONV_BF16 ? 2 : 4) > kStreamBytes;
    if (use_rows(a.N, a.C, a.dtype)) {
        if (!grad) return launch_glu_rows(p, a.act, stream);
        hipError_t e = launch_glu_rows_dx(p, a.act, stream);
        if (e == hipSuccess) e = launch_glu_rows_dw(p, a.act, l.splits, stream);
        return e == hipSuccess ? glu_join<__bf16>(p, l, a.dw, a.dbias, stream) : e;
    }
    if (a.dtype == SPCONV_BF16)
        return a.act == SPCONV_SILU ? glu_go<__bf16, SPCONV_SILU>(p, grad, l, a.dw, a.dbias, stream)
                                    : glu_go<__bf16, SPCONV_GELU>(p, grad, l, a.dw, a.dbias, stream);
    return a.act == SPCONV_SILU ? glu_go<float, SPCONV_SILU>(p, grad, l, a.dw, a.dbias, stream)
                                : glu_go<float, SPCONV_GELU>(p, grad, l, a.dw, a.dbias, stream);
}

}  // namespace spc
