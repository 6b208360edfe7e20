// Rotary positions of the heads of (N, H, D) rows for gfx950.
//
//   pair i = (a, b) of a head, turned by t = pos[n, i / (P / axes)] freq[i]:
//   (a', b') = gain (a cos t - b sin t, b cos t + a sin t)
//
// for the P pairs of the first 2 P elements; the others are copied.  The
// gradient is the turn the other way, with the same gain.
//
// Bound by memory.  A workgroup takes some rows, works out their cosines and
// sines once for all heads (LDS), then walks the heads in 16-byte pieces, a
// head's on neighbouring lanes of one wave.  A last piece that does not come
// out even starts earlier instead and repeats some of its neighbour's elements
// (in place too: the wave has read both before either is written).  Angles
// are 64-bit turns less whole turns: in 32 bits the angle of position 1e6 would
// be off by 0.06.  1,006,716 rows of 8 heads of 32 bf16: 187 us (5.6 TB/s).
#include "places.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTable = 2048;      // cosines and sines of a workgroup's rows, at least one row's

struct RotParams {
    const uint8_t* x;
    const int32_t* pos;
    const double* freqs;
    uint8_t* y;
    int64_t xs[2], ys[2], ps;        // row and head strides, bytes; positions, elements
    int64_t N;
    int H, D, P, per;                // per: pairs of an axis
    int rows;                        // per workgroup
    int tx;                          // lanes along a head (a power of two)
    int end;                         // elements in pieces that turn (interleaved: copies among them)
    int turn, rest;                  // such pieces, and those that are only copied
    bool repeat;                     // whether a last piece may start earlier
    float gain, sign;
    uint32_t heads_magic;
    bool stream;
};

// x / d and the rest for x < 2^31 (magic = 2^32 / d + 1: off by one at most)
struct Div {
    uint32_t q, r;
};
__device__ __forceinline__ Div divide(uint32_t x, uint32_t d, uint32_t magic) {
    if (d == 1) return {x, 0};
    uint32_t q = __umulhi(x, magic);
    int32_t r = (int32_t)(x - q * d);
    if (r < 0) {
        --q;
        r += d;
    }
    return {q, (uint32_t)r};
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kRotThreads) k_rotary(RotParams p) {
    constexpr int V = Piece<T>::V;
    extern __shared__ float2 table[];
    for (int64_t n0 = (int64_t)blockIdx.x * p.rows; n0 < p.N; n0 += (int64_t)gridDim.x * p.rows) {
        __syncthreads();         // the table of the rows before has been read
        const int rows = (int)min((int64_t)p.rows, p.N - n0);
        for (int e = threadIdx.x; e < rows * p.P; e += kRotThreads) {
            const int r = e / p.P, i = e - r * p.P;
            const double turns = (double)p.pos[(n0 + r) * p.ps + i / p.per] * (p.freqs[i] * 0.15915494309189533577);
            float s, c;
            sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
            table[e] = {c * p.gain, s * p.gain * p.sign};
        }
        __syncthreads();
        const int tx = threadIdx.x & (p.tx - 1), step = kRotThreads / p.tx;
        for (uint32_t e = threadIdx.x / p.tx; e < (uint32_t)rows * p.H; e += step) {
            const Div b = divide(e, p.H, p.heads_magic);
            const T* x = (const T*)(p.x + (n0 + b.q) * p.xs[0] + b.r * p.xs[1]);
            T* y = (T*)(p.y + (n0 + b.q) * p.ys[0] + b.r * p.ys[1]);
            const float2* cs = table + b.q * p.P;
            for (int c = tx; c < p.rest; c += p.tx) {
                const int d = 2 * p.P + c * V;
                const auto v = load_piece(x + d, p.D - d);
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = (float)v[j];
                store_piece(y + d, o, p.D - d, p.stream);
            }
            for (int c = tx; c < p.turn; c += p.tx) {
                const int i = p.repeat ? min(c * V, p.end - V) : c * V, n = p.end - i;
                if constexpr (HALF) {
                    const auto va = load_piece(x + i, n), vb = load_piece(x + p.P + i, n);
                    float oa[V], ob[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float2 w = cs[min(i + j, p.P - 1)];
                        oa[j] = (float)va[j] * w.x - (float)vb[j] * w.y;
                        ob[j] = (float)vb[j] * w.x + (float)va[j] * w.y;
                    }
                    store_piece(y + i, oa, n, p.stream);
                    store_piece(y + p.P + i, ob, n, p.stream);
                } else {
                    const auto v = load_piece(x + i, n);
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const int pair = (i + j) / 2;
                        const float2 w = cs[min(pair, p.P - 1)];
                        const float ra = (float)v[j] * w.x - (float)v[j + 1] * w.y;
                        const float rb = (float)v[j + 1] * w.x + (float)v[j] * w.y;
                        o[j] = pair < p.P ? ra : (float)v[j];
                        o[j + 1] = pair < p.P ? rb : (float)v[j + 1];
                    }
                    store_piece(y + i, o, n, p.stream);
                }
            }
        }
    }
}

uint32_t magic(int d) { return (uint32_t)((1ull << 32) / d + 1); }

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, bool back, hipStream_t stream) {
    if (a.N == 0) return hipSuccess;
    const int es = a.dtype == SPCONV_BF16 ? 2 : 4, V = 16 / es;
    RotParams p{};
    p.x = (const uint8_t*)a.x;
    p.pos = a.positions;
    p.freqs = a.freqs;
    p.y = (uint8_t*)a.y;
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i] * es;
        p.ys[i] = a.ys[i] * es;
    }
    p.ps = a.pos_stride;
    p.N = a.N;
    p.H = a.H;
    p.D = a.D;
    p.P = a.pairs;
    p.per = a.pairs / a.axes;
    const bool half = a.layout == SPCONV_HALF;
    // in place there is nothing to copy; interleaved pairs run on into it, where they can
    const bool in_place = a.x == a.y, through = !half && !in_place && a.D % 2 == 0;
    p.end = half ? a.pairs : through ? a.D : 2 * a.pairs;
    p.turn = (p.end + V - 1) / V;
    p.rest = in_place || through ? 0 : (a.D - 2 * a.pairs + V - 1) / V;
    p.tx = 1;
    while (p.tx < 64 && p.tx < p.turn) p.tx *= 2;
    p.repeat = p.end >= V && p.turn <= p.tx;
    p.rows = std::max(1, std::min(kRotTable / a.pairs, 32));
    // few rows: over as many workgroups as there are rows
    p.rows = (int)std::max<int64_t>(1, std::min<int64_t>(p.rows, a.N / 512));
    p.gain = a.gain;
    p.sign = back ? -1.f : 1.f;
    p.heads_magic = a.H > 1 ? magic(a.H) : 0;
    p.stream = a.N * a.H * a.D * es > kStreamBytes;
    // (a launch's threads are counted in 32 bits: more rows take turns)
    const unsigned blocks = (unsigned)std::min<int64_t>((a.N + p.rows - 1) / p.rows, 1 << 20);
    const size_t lds = (size_t)p.rows * p.P * sizeof(float2);
    if (a.dtype == SPCONV_BF16) {
        if (half)
            k_rotary<__bf16, true><<<blocks, kRotThreads, lds, stream>>>(p);
        else
            k_rotary<__bf16, false><<<blocks, kRotThreads, lds, stream>>>(p);
    } else if (half) {
        k_rotary<float, true><<<blocks, kRotThreads, lds, stream>>>(p);
    } else {
        k_rotary<float, false><<<blocks, kRotThreads, lds, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace spc
