// Group norm with an activation over the rows of each scene, channels last,
// and its gradient, for gfx950.
//
//   xhat = (x - mean) rstd,  z = xhat weight + bias,  y = act(z)
//
// mean and rstd = 1 / sqrt(var + eps) over the rows of a scene and the channels
// of a group.  With dz = dout act'(z):
//
//   dx = rstd (dz weight - m1 - xhat m2),  m1 = mean of dz weight,
//   m2 = mean of dz weight xhat,  dweight = sum dz xhat,  dbias = sum dz
//
// Bound by memory: a scene's statistics are needed before its first output, so
// every input is read twice.  A scene's rows are cut into chunks; a kernel
// writes one partial result per chunk and channel, one joins them per scene
// and group in a fixed order, and one walks the chunks again.  The forward's
// partials are (mean, sum of squared deviations), taken batch by batch in
// registers and joined by counts: no difference of large squares.  The second
// walk goes backwards, over what the first left in the memory-side cache.  At
// 1,006,716 x 128 bf16 in four scenes: 63 + 9 + 89 us forward (4.1 TB/s reading, 5.8
// reading and writing), 112 + 9 + 142 us gradient.
#include "glu.h"
#include "join.h"
#include "places.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kGrpThreads = 256;

struct GroupParams {
    const void* x;
    const void* dout;          // gradient
    const int32_t* offsets;
    const float* weight;       // or NULL
    const float* bias;         // or NULL
    void* y;                   // forward: y; gradient: dx
    float* mean;               // (scenes, groups)
    float* rstd;
    float* m12;                // gradient: (scenes, groups, 2)
    float* part;               // [items][2][C]
    float* dweight;            // or NULL
    float* dbias;
    int64_t N, items;
    int C, G, B, rows;         // rows: per chunk
    int tx;                    // threads along the channels (a power of two)
    int jx;                    // the same for the channels of a group, in the join
    float eps;
    int act;
    bool stream;
};

// A workgroup's chunk of rows and a thread's piece of channels: threads stand
// tx along the channels, the others on rows side by side.
struct Chunk {
    int b;
    int64_t row;          // the chunk's first
    int n;                // its rows
    int64_t of;           // the scene's rows
};
__device__ __forceinline__ Chunk find_chunk(const GroupParams& p, int64_t item) {
    const Place pl = find_place(p.offsets, p.B, p.N, 1, p.rows, item);
    if (pl.tile < 0) return {pl.b, 0, 0, pl.Lq};
    const int64_t at = (int64_t)pl.tile * p.rows;
    return {pl.b, pl.q0 + at, (int)min((int64_t)p.rows, pl.Lq - at), pl.Lq};
}

template <int ACT>
__device__ __forceinline__ Act group_act(float z) {
    if constexpr (ACT == SPCONV_LINEAR)
        return {z, 1.f};
    else
        return activation<ACT, true>(z);
}

// (mean, sum of squared deviations) over n values each.
struct Moments {
    float n, mean, m2;
};

// MODE 0: statistics of the rows (part: mean, m2).  MODE 1: sums of dz and
// dz xhat (part: A, B).
template <typename T, int ACT, int MODE>
__global__ void __launch_bounds__(kGrpThreads) k_group_part(GroupParams p) {
    constexpr int V = Piece<T>::V;
    constexpr int U = MODE == 0 ? 8 : 4;           // rows in flight
    __shared__ float s0[kGrpThreads * V], s1[kGrpThreads * V];
    const int t = threadIdx.x, tx = t & (p.tx - 1), ty = t / p.tx, TY = kGrpThreads / p.tx;
    const int cb = blockIdx.y * p.tx * V;          // the workgroup's first channel
    const int c = cb + tx * V, nv = p.C - c;
    const Chunk ch = find_chunk(p, blockIdx.x);
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.C;
    if (ch.n == 0) {
        // an empty place adds nothing to the sums over all places
        if (MODE == 1 && ty == 0)
            for (int i = 0; i < V; ++i)
                if (i < nv) part[c + i] = part[p.C + c + i] = 0.f;
        return;
    }
    const T* x = (const T*)p.x + ch.row * p.C + c;
    const T* dout = (const T*)p.dout + ch.row * p.C + c;
    float a0[V], a1[V], mu[V], rs[V], wt[V], bs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        a0[i] = a1[i] = 0.f;
        if constexpr (MODE == 1) {
            const int g = i < nv ? (c + i) / (p.C / p.G) : 0;
            mu[i] = p.mean[(int64_t)ch.b * p.G + g];
            rs[i] = p.rstd[(int64_t)ch.b * p.G + g];
            wt[i] = p.weight && i < nv ? p.weight[c + i] : 1.f;
            bs[i] = p.bias && i < nv ? p.bias[c + i] : 0.f;
        }
    }
    float count = 0.f;
    int r = ty;
    for (; r + (U - 1) * TY < ch.n; r += U * TY) {
        typename Piece<T>::vec vx[U], vd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            vx[u] = load_piece(x + (int64_t)(r + u * TY) * p.C, nv);
            if constexpr (MODE == 1) vd[u] = load_piece(dout + (int64_t)(r + u * TY) * p.C, nv);
        }
        if constexpr (MODE == 0) {
            // the batch's own mean and deviations, joined with those before
            const float n = count + U, wb = U / n, wc = count * wb;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float m = 0.f, q = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) m += (float)vx[u][i];
                m *= 1.f / U;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float d = (float)vx[u][i] - m;
                    q = fmaf(d, d, q);
                }
                const float d = m - a0[i];
                a0[i] = fmaf(d, wb, a0[i]);
                a1[i] += fmaf(d * d, wc, q);
            }
            count = n;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = ((float)vx[u][i] - mu[i]) * rs[i];
                    const float dz = (float)vd[u][i] * group_act<ACT>(fmaf(xh, wt[i], bs[i])).d;
                    a0[i] += dz;
                    a1[i] = fmaf(dz, xh, a1[i]);
                }
        }
    }
    for (; r < ch.n; r += TY) {
        const auto vx = load_piece(x + (int64_t)r * p.C, nv);
        if constexpr (MODE == 0) {
            count += 1.f;
            const float w = 1.f / count;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = (float)vx[i] - a0[i];
                a0[i] = fmaf(d, w, a0[i]);
                a1[i] = fmaf(d, (float)vx[i] - a0[i], a1[i]);
            }
        } else {
            const auto vd = load_piece(dout + (int64_t)r * p.C, nv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = ((float)vx[i] - mu[i]) * rs[i];
                const float dz = (float)vd[i] * group_act<ACT>(fmaf(xh, wt[i], bs[i])).d;
                a0[i] += dz;
                a1[i] = fmaf(dz, xh, a1[i]);
            }
        }
    }
    const int W = p.tx * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s0[ty * W + tx * V + i] = a0[i];
        s1[ty * W + tx * V + i] = a1[i];
    }
    __syncthreads();
    // rows side by side, in their order
    for (int e = t; e < W; e += kGrpThreads) {
        if (cb + e >= p.C) continue;
        float r0, r1;
        if constexpr (MODE == 0) {
            Moments m{0.f, 0.f, 0.f};
            for (int k = 0; k < min(TY, ch.n); ++k) {
                const float n = (float)((ch.n - k + TY - 1) / TY), all = m.n + n, d = s0[k * W + e] - m.mean;
                m.mean = fmaf(d, n / all, m.mean);
                m.m2 += fmaf(d * d, m.n * (n / all), s1[k * W + e]);
                m.n = all;
            }
            r0 = m.mean;
            r1 = m.m2;
        } else {
            r0 = r1 = 0.f;
            for (int k = 0; k < min(TY, ch.n); ++k) {
                r0 += s0[k * W + e];
                r1 += s1[k * W + e];
            }
        }
        part[cb + e] = r0;
        part[p.C + cb + e] = r1;
    }
}

// dweight and dbias (kJoinCols of both) from the parts of all places.
__device__ __forceinline__ void group_sums(const float* part, int64_t items, int C, float* dweight, float* dbias,
                                           int block) {
    const float t = join_columns<64, 1>(part, items, 2 * C, block).f[0];
    const int e = block * kJoinCols + threadIdx.x;
    if (threadIdx.x < kJoinCols && e < 2 * C) (e < C ? dbias : dweight - C)[e] = t;
}

// Sum over a workgroup of THR threads, the same bits in every thread.
template <int THR>
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = group_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < THR / 64; ++k) s += red[k];
    return s;
}

// The chunks' parts of one scene and group: its statistics, or its two means
// of the gradient.  Threads stand along the group's channels (a power of two of
// them), the others on chunks side by side; the first few chunks of a thread
// stay in registers.  The gradient's channel sums over all places are further
// workgroups of the same launch (or, where a wave is enough for a scene and
// group, a launch of their own).
constexpr int kGrpKeep = 8;
template <int MODE, int THR>
__global__ void __launch_bounds__(THR) k_group_join(GroupParams p) {
    __shared__ float red[THR / 64];
    const int stats = p.B * p.G;
    if constexpr (MODE == 1 && THR == kJoinCols * 64) {
        if ((int)blockIdx.x >= stats) {
            group_sums(p.part, p.items, p.C, p.dweight, p.dbias, blockIdx.x - stats);
            return;
        }
    }
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G, cg = p.C / p.G;
    const int64_t o0 = clamp_to(p.offsets[b], 0, p.N), len = clamp_to(p.offsets[b + 1], o0, p.N) - o0;
    const int64_t item = o0 / p.rows + b;
    const int chunks = (int)((len + p.rows - 1) / p.rows);
    const float* part = p.part + item * 2 * p.C + g * cg;
    const auto rows_of = [&](int k) { return (float)min((int64_t)p.rows, len - (int64_t)k * p.rows); };
    const float inv = len ? 1.f / ((float)len * cg) : 0.f;
    const int jx = min(p.jx, THR), tc = threadIdx.x & (jx - 1), tk = threadIdx.x / jx, step = THR / jx;
    float q0[kGrpKeep], q1[kGrpKeep], v0 = 0.f, v1 = 0.f;
    // element i of the thread: its channel and chunk
    const int mine = tk < chunks ? (chunks - tk + step - 1) / step : 0, all = mine * ((cg - tc + jx - 1) / jx);
    const auto at = [&](int i, int& c, int& k) {
        if (i < mine) {
            c = tc;
            k = tk + i * step;
        } else {
            const int w = i / mine;
            c = tc + w * jx;
            k = tk + (i - w * mine) * step;
        }
        return part + (int64_t)k * 2 * p.C + c;
    };
    const auto each = [&](auto use) {
#pragma unroll
        for (int i = 0; i < kGrpKeep; ++i)
            if (i < all && tc < cg) {
                int c, k;
                at(i, c, k);
                use(q0[i], q1[i], c, k);
            }
        for (int i = kGrpKeep; i < all && tc < cg; ++i) {
            int c, k;
            const float* q = at(i, c, k);
            use(q[0], q[p.C], c, k);
        }
    };
#pragma unroll
    for (int i = 0; i < kGrpKeep; ++i)
        if (i < all && tc < cg) {
            int c, k;
            const float* q = at(i, c, k);
            q0[i] = q[0];
            q1[i] = q[p.C];
        }
    each([&](float a0, float a1, int c, int k) {
        const float w = MODE == 0 ? rows_of(k) : p.weight ? p.weight[g * cg + c] : 1.f;
        v0 = fmaf(a0, w, v0);
        if constexpr (MODE == 1) v1 = fmaf(a1, w, v1);
    });
    v0 = block_sum<THR>(v0, red) * inv;
    if constexpr (MODE == 0)
        each([&](float a0, float a1, int, int k) {
            const float d = a0 - v0;
            v1 += fmaf(d * d, rows_of(k), a1);
        });
    v1 = block_sum<THR>(v1, red) * inv;
    if (threadIdx.x == 0) {
        if constexpr (MODE == 0) {
            p.mean[blockIdx.x] = v0;
            p.rstd[blockIdx.x] = 1.f / sqrtf(v1 + p.eps);
        } else {
            p.m12[2 * blockIdx.x] = v0;
            p.m12[2 * blockIdx.x + 1] = v1;
        }
    }
}

__global__ void __launch_bounds__(kJoinCols * 64) k_group_sums(const float* part, int64_t items, int C, float* dweight,
                                                               float* dbias) {
    group_sums(part, items, C, dweight, dbias, blockIdx.x);
}

template <typename T, int ACT, bool GRAD>
__global__ void __launch_bounds__(kGrpThreads) k_group_apply(GroupParams p) {
    constexpr int V = Piece<T>::V;
    constexpr int U = 4;
    const int t = threadIdx.x, tx = t & (p.tx - 1), ty = t / p.tx, TY = kGrpThreads / p.tx;
    const int c = (blockIdx.y * p.tx + tx) * V, nv = p.C - c;
    const Chunk ch = find_chunk(p, p.items - 1 - blockIdx.x);
    if (ch.n == 0 || nv <= 0) return;
    const T* x = (const T*)p.x + ch.row * p.C + c;
    const T* dout = (const T*)p.dout + ch.row * p.C + c;
    T* y = (T*)p.y + ch.row * p.C + c;
    float mu[V], rs[V], wt[V], bs[V], m1[V], m2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = (int64_t)ch.b * p.G + (i < nv ? (c + i) / (p.C / p.G) : 0);
        mu[i] = p.mean[g];
        rs[i] = p.rstd[g];
        wt[i] = p.weight && i < nv ? p.weight[c + i] : 1.f;
        bs[i] = p.bias && i < nv ? p.bias[c + i] : 0.f;
        if constexpr (GRAD) {
            m1[i] = p.m12[2 * g];
            m2[i] = p.m12[2 * g + 1];
        }
    }
    for (int r = ty; r < ch.n; r += U * TY) {
        typename Piece<T>::vec vx[U], vd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = r + u * TY < ch.n ? nv : 0;
            vx[u] = load_piece(x + (int64_t)(r + u * TY) * p.C, n);
            if constexpr (GRAD) vd[u] = load_piece(dout + (int64_t)(r + u * TY) * p.C, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + u * TY >= ch.n) continue;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = ((float)vx[u][i] - mu[i]) * rs[i];
                const Act a = group_act<ACT>(fmaf(xh, wt[i], bs[i]));
                if constexpr (GRAD) {
                    // the product is rounded before the mean, a sum of such, is
                    // taken off: a group of one element gives 0
#pragma clang fp contract(off)
                    const float g = (float)vd[u][i] * a.d * wt[i];
                    o[i] = (g - m1[i] - xh * m2[i]) * rs[i];
                } else {
                    o[i] = a.v;
                }
            }
            store_piece(y + (int64_t)(r + u * TY) * p.C, o, nv, p.stream);
        }
    }
}

// Few rows: a workgroup per scene and group keeps the group's elements in
// registers between the statistics and the outputs (kOneElems per thread), a
// launch in place of three.  A thread holds W channels (all of a 16-byte piece,
// where groups and rows are whole numbers of those, else one) of rows one
// stride apart.  The gradient has no such form: with two inputs to hold it took 35.7
// us where three launches took 13.4 (4,096 x 32 in one scene of 8 groups).
constexpr int kOneThreads = 1024, kOneElems = 32;
template <typename T, int W, int ACT>
__global__ void __launch_bounds__(kOneThreads) k_group_one(GroupParams p) {
    constexpr int NE = kOneElems / W;
    typedef T vec __attribute__((ext_vector_type(W)));
    __shared__ float red[kOneThreads / 64];
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G, cg = p.C / p.G, per = cg / W, side = kOneThreads / per;
    const int64_t o0 = clamp_to(p.offsets[b], 0, p.N);
    const int len = (int)(clamp_to(p.offsets[b + 1], o0, p.N) - o0);
    const int t = threadIdx.x, tr = t / per, c = g * cg + (t - tr * per) * W;
    const bool mine = tr < side;
    const int64_t first = (o0 + tr) * p.C + c, step = (int64_t)side * p.C;
    const T* x = (const T*)p.x + first;
    T* y = (T*)p.y + first;
    const float inv = len ? 1.f / ((float)len * cg) : 0.f;
    float wt[W], bs[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        wt[i] = p.weight && mine ? p.weight[c + i] : 1.f;
        bs[i] = p.bias && mine ? p.bias[c + i] : 0.f;
    }
    vec vx[NE];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const bool in = mine && tr + e * side < len;
        vx[e] = in ? *(const vec*)(x + e * step) : vec{};
    }
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int i = 0; i < W; ++i) s0 += (float)vx[e][i];
    const float mean = block_sum<kOneThreads>(s0, red) * inv;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const bool in = mine && tr + e * side < len;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float d = (float)vx[e][i] - mean;
            s1 += in ? d * d : 0.f;
        }
    }
    const float rstd = 1.f / sqrtf(block_sum<kOneThreads>(s1, red) * inv + p.eps);
    if (t == 0) {
        p.mean[blockIdx.x] = mean;
        p.rstd[blockIdx.x] = rstd;
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        if (!mine || tr + e * side >= len) continue;
        vec o;
#pragma unroll
        for (int i = 0; i < W; ++i)
            o[i] = (T)group_act<ACT>(fmaf(((float)vx[e][i] - mean) * rstd, wt[i], bs[i])).v;
        *(vec*)(y + e * step) = o;
    }
}

struct GroupShape {
    int tx, cols, rows;
    int64_t items;
};
// Chunks of about 1 / 2,048 of the rows, but four rows per thread at least.
GroupShape group_shape(int64_t N, int C, int scenes, int dtype) {
    const int V = dtype == SPCONV_BF16 ? 8 : 4, pieces = (C + V - 1) / V;
    GroupShape s;
    s.tx = 1;
    while (s.tx < 64 && s.tx < pieces) s.tx *= 2;
    s.cols = (pieces + s.tx - 1) / s.tx;
    const int64_t batch = kGrpThreads / s.tx * 4;
    s.rows = (int)(std::max<int64_t>(1, (N / 2048 + batch - 1) / batch) * batch);
    s.items = N / s.rows + scenes;
    return s;
}

// Whether a scene's share of a group fits the registers of a workgroup, the
// whole is small enough for workgroups that read parts of rows, and they are as
// many as the card takes at a time (4,096 x 32 fp32, 8 groups, forward, one launch
// against three: 1 scene 7.8 and 12.6 us, 64 scenes 8.3 and 12.9, 128 scenes 14.5
// and 13.6; 2,048 x 128, 32 groups, 1,024 scenes: 389 and 29).
bool group_one(int64_t N, int C, int B, int G, int W) {
    const int per = C / G / W;
    return per <= kOneThreads && N <= (int64_t)(kOneThreads / per) * (kOneElems / W) && N * C <= (1 << 18) &&
           (int64_t)B * G <= 512;
}

// Workgroups of group_sums.
unsigned channel_sums(int C) { return (2 * C + kJoinCols - 1) / kJoinCols; }

template <typename T, int ACT>
hipError_t group_go(const GroupParams& p, bool grad, const GroupShape& s, hipStream_t st) {
    const dim3 grid((unsigned)s.items, s.cols);
    const unsigned stats = (unsigned)(p.B * p.G);
    constexpr int V = Piece<T>::V;
    const bool whole = p.C / p.G % V == 0 && ((uintptr_t)p.x | (uintptr_t)p.y) % 16 == 0;
    if (!grad && group_one(p.N, p.C, p.B, p.G, whole ? V : 1)) {
        (whole ? k_group_one<T, V, ACT> : k_group_one<T, 1, ACT>)<<<stats, kOneThreads, 0, st>>>(p);
        return hipGetLastError();
    }
    // threads that join a scene's parts: a wave where it has a few on average
    constexpr int kMany = kJoinCols * 64;
    const bool many = (p.N / p.B / p.rows + 1) * (p.C / p.G) > 256;
    const unsigned sums = channel_sums(p.C);
    if (!grad) {
        k_group_part<T, ACT, 0><<<grid, kGrpThreads, 0, st>>>(p);
        if (many)
            k_group_join<0, kMany><<<stats, kMany, 0, st>>>(p);
        else
            k_group_join<0, 64><<<stats, 64, 0, st>>>(p);
        k_group_apply<T, ACT, false><<<grid, kGrpThreads, 0, st>>>(p);
        return hipGetLastError();
    }
    k_group_part<T, ACT, 1><<<grid, kGrpThreads, 0, st>>>(p);
    if (many) {
        k_group_join<1, kMany><<<stats + (p.dweight ? sums : 0), kMany, 0, st>>>(p);
    } else {
        k_group_join<1, 64><<<stats, 64, 0, st>>>(p);
        if (p.dweight) k_group_sums<<<sums, kMany, 0, st>>>(p.part, p.items, p.C, p.dweight, p.dbias);
    }
    k_group_apply<T, ACT, true><<<grid, kGrpThreads, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T>
hipError_t group_type(const GroupParams& p, bool grad, const GroupShape& s, hipStream_t st) {
    switch (p.act) {
        case SPCONV_SILU: return group_go<T, SPCONV_SILU>(p, grad, s, st);
        case SPCONV_GELU: return group_go<T, SPCONV_GELU>(p, grad, s, st);
        default: return group_go<T, SPCONV_LINEAR>(p, grad, s, st);
    }
}

size_t stats_bytes(int scenes, int groups) { return align_up((size_t)scenes * groups * 8, 256); }

}  // namespace

bool group_fits(int64_t N, int C, int scenes, int groups, int dtype, bool grad) {
    const GroupShape s = group_shape(N, C, scenes, dtype);
    const int64_t joins = (int64_t)scenes * groups + (grad ? channel_sums(C) : 0);
    return s.items * s.cols * kGrpThreads < (1ll << 32) && joins * kOneThreads < (1ll << 32);
}
size_t group_workspace_bytes(int64_t N, int C, int scenes, int groups, int dtype) {
    return stats_bytes(scenes, groups) + align_up((size_t)group_shape(N, C, scenes, dtype).items * 2 * C * 4, 256);
}

hipError_t launch_group(const GroupArgs& a, bool grad, hipStream_t stream) {
    if (a.scenes == 0) return hipSuccess;
    const GroupShape s = group_shape(a.N, a.C, a.scenes, a.dtype);
    GroupParams p{};
    p.x = a.x;
    p.dout = a.dout;
    p.offsets = a.offsets;
    p.weight = a.weight;
    p.bias = a.bias;
    p.y = a.y;
    // statistics that the caller does not want are the workspace's; so are the gradient's means
    p.mean = a.mean ? a.mean : (float*)a.workspace;
    p.rstd = a.rstd ? a.rstd : (float*)a.workspace + (int64_t)a.scenes * a.groups;
    p.m12 = (float*)a.workspace;
    p.part = (float*)((uint8_t*)a.workspace + stats_bytes(a.scenes, a.groups));
    p.dweight = a.dweight;
    p.dbias = a.dbias;
    p.N = a.N;
    p.items = s.items;
    p.C = a.C;
    p.G = a.groups;
    p.B = a.scenes;
    p.rows = s.rows;
    p.tx = s.tx;
    p.jx = 1;
    while (p.jx < 1024 && p.jx < a.C / a.groups) p.jx *= 2;
    p.eps = a.eps;
    p.act = a.act;
    p.stream = a.N * a.C * (a.dtype == SPCONV_BF16 ? 2 : 4) > kStreamBytes;
    return a.dtype == SPCONV_BF16 ? group_type<__bf16>(p, grad, s, stream) : group_type<float>(p, grad, s, stream);
}

}  // namespace spc
