// Layer norm of feature rows and its gradient for gfx950.
//
//   y[n, c]  = (x[n, c] - mean[n]) * rstd[n] * weight[c] + bias[c]
//   rstd[n]  = 1 / sqrt(mean_c (x - mean)^2 + eps)
//
// and, with xhat = (x - mean) rstd and g = dy weight,
//
//   dx       = rstd (g - mean_c g - xhat mean_c (g xhat))
//   dweight  = sum_n dy xhat,   dbias = sum_n dy
//
// Both are bound by memory: each row is read once and kept in registers, the
// variance is taken from the deviations there (no difference of squares), all
// sums in fp32.  A row belongs to L consecutive lanes that hold NV 16-byte
// pieces each; rows wider than two pieces per lane of a wave belong to a whole
// workgroup (L = 256), whose four waves join their sums through LDS, so that
// a lane never holds more than 16 elements of a row next to its weights.
// Workgroups stay and walk the rows, with the weights in registers.  At
// 1,006,716 x 128 bf16: 107 us forward (4.9 TB/s), 156 us gradient (5.0 TB/s), where
// a large copy reaches 5.4.
#include "join.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;
// Workgroups of the gradient: each writes one partial row of dweight and
// dbias, so their number bounds the second kernel's reading.
constexpr int kNormGradBlocks = 1024;
constexpr int kNormBlocks = 2048;

// Sum over the L lanes of a row; U values at a time.  L = 256: through `red`
// (kNormWaves * U floats; the caller alternates two of them, so one barrier
// per sum is enough).
template <int L, int U>
__device__ __forceinline__ void row_sum(float (&v)[U], float* red) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = group_sum<(L > 64 ? 64 : L)>(v[u]);
    if constexpr (L > 64) {
        const int t = threadIdx.x;
        if ((t & 63) == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) red[u * kNormWaves + (t >> 6)] = v[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kNormWaves; ++k) s += red[u * kNormWaves + k];
            v[u] = s;
        }
    }
}

struct NormParams {
    const void* x;
    const float* weight;
    const float* bias;
    void* y;
    float* mean;
    float* rstd;
    const void* dout;
    float* part;      // [blocks][2][C]
    int64_t N;
    int C;
    float eps;
    bool stream;      // outputs past the caches
};

template <typename T, int L, int NV, int U>
__global__ void __launch_bounds__(kNormThreads) k_norm(NormParams p) {
    constexpr int V = Piece<T>::V;
    constexpr int G = kNormThreads / L;          // rows side by side
    __shared__ float red[2][kNormWaves * U];
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    const int C = p.C;
    const T* x = (const T*)p.x;
    T* y = (T*)p.y;
    const float inv = 1.f / (float)C;
    float wt[NV][V], bs[NV][V];
    int nv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * V;
        nv[j] = C - c;                           // elements from here on (may be <= 0)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wt[j][i] = p.weight && i < nv[j] ? p.weight[c + i] : 1.f;
            bs[j][i] = p.bias && i < nv[j] ? p.bias[c + i] : 0.f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * (G * U);
    for (int64_t r0 = (int64_t)blockIdx.x * (G * U); r0 < p.N; r0 += step) {
        typename Piece<T>::vec raw[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G + g;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                raw[u][j] = load_piece(x + r * C + (j * L + lane) * V, r < p.N ? nv[j] : 0);
        }
        float m[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) m[u] += (float)raw[u][j][i];
        }
        row_sum<L, U>(m, red[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] *= inv;
            s[u] = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = (float)raw[u][j][i] - m[u];
                    s[u] += i < nv[j] ? d * d : 0.f;
                }
        }
        row_sum<L, U>(s, red[1]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G + g;
            if (r >= p.N) continue;
            const float rs = 1.f / sqrtf(s[u] * inv + p.eps);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = ((float)raw[u][j][i] - m[u]) * rs * wt[j][i] + bs[j][i];
                store_piece(y + r * C + (j * L + lane) * V, o, nv[j], p.stream);
            }
            if (p.mean && lane == 0) {
                p.mean[r] = m[u];
                p.rstd[r] = rs;
            }
        }
    }
}

template <typename T, int L, int NV, int U>
__global__ void __launch_bounds__(kNormThreads) k_norm_grad(NormParams p) {
    constexpr int V = Piece<T>::V;
    constexpr int G = kNormThreads / L;
    __shared__ float red[2][kNormWaves * 2 * U];
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    const int C = p.C;
    const T* x = (const T*)p.x;
    const T* dy = (const T*)p.dout;
    T* dx = (T*)p.y;
    const float inv = 1.f / (float)C;
    float wt[NV][V], dw[NV][V], db[NV][V];
    int nv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * V;
        nv[j] = C - c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wt[j][i] = p.weight && i < nv[j] ? p.weight[c + i] : 1.f;
            dw[j][i] = 0.f;
            db[j][i] = 0.f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * (G * U);
    int par = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * (G * U); r0 < p.N; r0 += step) {
        typename Piece<T>::vec rx[U][NV], rd[U][NV];
        float mean[U], rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G + g;
            const bool in = r < p.N;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                rx[u][j] = load_piece(x + r * C + (j * L + lane) * V, in ? nv[j] : 0);
                rd[u][j] = load_piece(dy + r * C + (j * L + lane) * V, in ? nv[j] : 0);
            }
            mean[u] = in ? p.mean[r] : 0.f;
            rs[u] = in ? p.rstd[r] : 0.f;
        }
        float sums[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    // past the row's end dy is 0 and x is 0: nothing is added
                    const float d = (float)rd[u][j][i];
                    const float xh = i < nv[j] ? ((float)rx[u][j][i] - mean[u]) * rs[u] : 0.f;
                    const float gw = d * wt[j][i];
                    dw[j][i] += d * xh;
                    db[j][i] += d;
                    a += gw;
                    b += gw * xh;
                }
            sums[2 * u] = a;
            sums[2 * u + 1] = b;
        }
        row_sum<L, 2 * U>(sums, red[par]);
        par ^= 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G + g;
            if (r >= p.N) continue;
            const float m1 = sums[2 * u] * inv, m2 = sums[2 * u + 1] * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = ((float)rx[u][j][i] - mean[u]) * rs[u];
                    o[i] = ((float)rd[u][j][i] * wt[j][i] - m1 - xh * m2) * rs[u];
                }
                store_piece(dx + r * C + (j * L + lane) * V, o, nv[j], p.stream);
            }
        }
    }
    if (!p.part) return;
    // one partial row per workgroup: its G row groups joined in their order
    float* pw = p.part + (int64_t)blockIdx.x * 2 * C;
    if constexpr (G == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < nv[j]) {
                    const int c = (j * L + lane) * V + i;
                    pw[c] = dw[j][i];
                    pw[C + c] = db[j][i];
                }
    } else {
        __shared__ float join[G][2 * L * V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                join[g][lane * V + i] = dw[j][i];
                join[g][L * V + lane * V + i] = db[j][i];
            }
            __syncthreads();
            for (int e = threadIdx.x; e < 2 * L * V; e += kNormThreads) {
                const int c = j * L * V + e % (L * V);
                if (c < C) {
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < G; ++k) s += join[k][e];
                    pw[(e / (L * V)) * C + c] = s;
                }
            }
        }
    }
}

__global__ void __launch_bounds__(kJoinCols * 64) k_norm_join(const float* part, int blocks, int C, float* dweight,
                                                              float* dbias) {
    const float t = join_columns<64, 1>(part, blocks, 2 * C, blockIdx.x).f[0];
    const int e = blockIdx.x * kJoinCols + threadIdx.x;
    if (threadIdx.x < kJoinCols && e < 2 * C) (e < C ? dweight : dbias - C)[e] = t;
}

// Lanes per row and pieces per lane for rows of C elements: the smallest
// group whose lanes hold at most two pieces, else the workgroup.
struct NormShape {
    int L, NV;
};
NormShape norm_shape(int C, int V) {
    const int pieces = (C + V - 1) / V;
    if (pieces > 128) return {256, pieces > 512 ? 4 : pieces > 256 ? 2 : 1};
    int L = 1;
    while (L < 64 && L < pieces) L *= 2;
    return {L, pieces > L ? 2 : 1};
}
int norm_rows(const NormShape& s) { return kNormThreads / s.L * (s.NV == 1 ? 2 : 1); }

template <typename T, int L, int NV>
hipError_t norm_go(const NormParams& p, bool grad, int blocks, hipStream_t st) {
    constexpr int U = NV == 1 ? 2 : 1;
    if (grad)
        k_norm_grad<T, L, NV, U><<<blocks, kNormThreads, 0, st>>>(p);
    else
        k_norm<T, L, NV, U><<<blocks, kNormThreads, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t norm_dispatch(const NormParams& p, bool grad, int most, hipStream_t st) {
    const NormShape s = norm_shape(p.C, Piece<T>::V);
    const int rows = norm_rows(s);
    const int blocks = (int)std::min<int64_t>((p.N + rows - 1) / rows, most);
    switch (s.L * 8 + s.NV) {
        case 1 * 8 + 1: return norm_go<T, 1, 1>(p, grad, blocks, st);
        case 2 * 8 + 1: return norm_go<T, 2, 1>(p, grad, blocks, st);
        case 4 * 8 + 1: return norm_go<T, 4, 1>(p, grad, blocks, st);
        case 8 * 8 + 1: return norm_go<T, 8, 1>(p, grad, blocks, st);
        case 16 * 8 + 1: return norm_go<T, 16, 1>(p, grad, blocks, st);
        case 32 * 8 + 1: return norm_go<T, 32, 1>(p, grad, blocks, st);
        case 64 * 8 + 1: return norm_go<T, 64, 1>(p, grad, blocks, st);
        case 64 * 8 + 2: return norm_go<T, 64, 2>(p, grad, blocks, st);
        case 256 * 8 + 1: return norm_go<T, 256, 1>(p, grad, blocks, st);
        case 256 * 8 + 2: return norm_go<T, 256, 2>(p, grad, blocks, st);
        default: break;
    }
    if constexpr (Piece<T>::V == 4) return norm_go<T, 256, 4>(p, grad, blocks, st);
    return hipErrorInvalidValue;
}

int norm_grad_blocks(int64_t N, int C, int dtype) {
    const int rows = norm_rows(norm_shape(C, dtype == SPCONV_BF16 ? 8 : 4));
    return (int)std::min<int64_t>((N + rows - 1) / rows, kNormGradBlocks);
}

bool norm_streams(int64_t N, int C, int dtype) { return N * C * (dtype == SPCONV_BF16 ? 2 : 4) > kStreamBytes; }

}  // namespace

size_t norm_grad_workspace_bytes(int64_t N, int C, int dtype) {
    return align_up((size_t)norm_grad_blocks(N, C, dtype) * 2 * C * 4, 256);
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    if (a.N == 0) return hipSuccess;
    const NormParams p{a.x, a.weight, a.bias, a.y, a.mean, a.rstd, nullptr, nullptr, a.N, a.C, a.eps,
                       norm_streams(a.N, a.C, a.dtype)};
    return a.dtype == SPCONV_BF16 ? norm_dispatch<__bf16>(p, false, kNormBlocks, stream)
                                  : norm_dispatch<float>(p, false, kNormBlocks, stream);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream) {
    if (a.N > 0) {
        const NormParams p{a.x, a.weight, nullptr, a.dx, const_cast<float*>(a.mean), const_cast<float*>(a.rstd),
                           a.dout, a.dweight ? (float*)a.workspace : nullptr, a.N, a.C, 0.f,
                           norm_streams(a.N, a.C, a.dtype)};
        const hipError_t e = a.dtype == SPCONV_BF16 ? norm_dispatch<__bf16>(p, true, kNormGradBlocks, stream)
                                                    : norm_dispatch<float>(p, true, kNormGradBlocks, stream);
        if (e != hipSuccess) return e;
    }
    if (!a.dweight) return hipSuccess;
    k_norm_join<<<(2 * a.C + kJoinCols - 1) / kJoinCols, kJoinCols * 64, 0, stream>>>(
        (const float*)a.workspace, norm_grad_blocks(a.N, a.C, a.dtype), a.C, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace spc
