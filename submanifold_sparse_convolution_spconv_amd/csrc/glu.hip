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
//
// With bfloat16, da and db are rounded to it once, since the matrix instructions
// take operands of that type (two-part operands would double the products): the
// gradients' error against 64 bits is 2.3e-3 of their norm where unrounded ones give
// 1.7e-3, the outputs' own rounding.
//
// Gradient of 29,578 rows, 256 -> 680 bf16 (averages of ten): 58 us for da and db (the
// activations), 80 us for both products (513 TFLOP/s; LDS reads take 47% of the time),
// 8 us to join the partial sums.  In fp32 197 us forward (104 TFLOP/s), 705 us gradient.
#include "glu.h"
#include "join.h"

#include <algorithm>
#include <type_traits>

namespace spc {

namespace {

// Tiles of TILE x TILE outputs: WM waves along the first operand, WN along the
// second; a wave holds NM x NN blocks of 16 x 16.  Eight waves share the large
// tile rather than four: with half the accumulators each, four fit on a SIMD,
// and short reductions spend less of their time waiting.
template <int TILE>
struct Shape {
    static constexpr int WM = TILE >= 64 ? 2 : 1, WN = TILE >= 64 ? TILE / 32 : 2, THREADS = 64 * WM * WN;
    static constexpr int NM = TILE / 16 / WM, NN = TILE / 16 / WN;
};

template <typename V>
__device__ __forceinline__ V keep(V v, bool in) {
    uint32_t w[sizeof(V) / 4];
    __builtin_memcpy(w, &v, sizeof v);
#pragma unroll
    for (unsigned i = 0; i < sizeof(V) / 4; ++i) w[i] = in ? w[i] : 0u;
    __builtin_memcpy(&v, w, sizeof v);
    return v;
}

template <typename T>
constexpr int kTileK = sizeof(T) == 2 ? 64 : 32;      // of the reduction per step

// One operand tile in LDS: M outputs x BK of the reduction.  KC: the reduction
// is contiguous in memory and in LDS ([m][k]); else the outputs are ([k][m]).
// The pitches keep the fragment reads free of bank conflicts: 16 rows' 16-byte
// units (KC, bf16: an odd number of units), four rows' four units (bf16), one
// word per lane (fp32).
template <typename T, bool KC, int M>
struct Stage {
    static constexpr bool K_CONTIGUOUS = KC;
    static constexpr int BK = kTileK<T>;
    static constexpr int V = Piece<T>::V;
    static constexpr int THREADS = Shape<M>::THREADS;
    static constexpr int PER = M * BK / V / THREADS;             // pieces per thread
    static constexpr int PITCH = KC ? BK + V : M + (sizeof(T) == 2 ? 32 : 16);
    static constexpr int ELEMS = (KC ? M : BK) * PITCH;
    static_assert(PER >= 1 && M * BK / V % THREADS == 0, "whole pieces per thread");
    // piece j of this thread: output m and reduction index k of its first element
    static __device__ __forceinline__ void where(int j, int& m, int& k) {
        const int p = threadIdx.x + THREADS * j;
        if constexpr (KC) {
            m = p / (BK / V);
            k = p % (BK / V) * V;
        } else {
            k = p / (M / V);
            m = p % (M / V) * V;
        }
    }
};

// One operand of a product on its way to LDS: this thread's pieces of the next
// two steps in registers.  An address is the tile's place at the step (the same
// for the workgroup) and a 32-bit offset of the thread, so a step costs no
// address arithmetic.  Loads stand under no branch that differs between lanes
// (the compiler would wait for all of them at the first use): pieces outside
// read a valid place and become 0 on the way to LDS, on tiles and steps that
// have any.
template <typename T, bool KC, int M>
struct Operand {
    using S = Stage<T, KC, M>;
    static constexpr int NP = KC ? S::PER : 1;                  // outputs per thread
    static constexpr int KSTEP = S::THREADS / (M / S::V);      // !KC: k from piece to piece
    const T* base;        // output 0 at reduction index 0
    int64_t pitch;        // of k, where the outputs are contiguous
    bool full;            // every output of the tile is inside
    int kk;               // k of the first piece
    uint32_t off[NP];     // of the outputs; 0 where outside
    bool in[NP];
    typename Piece<T>::vec raw[2][S::PER];
    // offset(m): elements from output 0 to output m, valid where inside(m)
    template <class O, class I>
    __device__ __forceinline__ Operand(const T* base, O offset, I inside, bool full, int64_t k_pitch)
        : base(base), pitch(k_pitch), full(full) {
        int m;
#pragma unroll
        for (int j = NP - 1; j >= 0; --j) {
            S::where(j, m, kk);
            in[j] = inside(m);
            off[j] = in[j] ? offset(m) : 0;
        }
    }
    // pieces of the step at k; klim: the reduction's end
    template <int SLOT>
    __device__ __forceinline__ void fetch(int64_t k, int64_t klim) {
        if (k >= klim) return;
        const bool tail = k + S::BK > klim;
#pragma unroll
        for (int j = 0; j < S::PER; ++j) {
            const T* p;
            if constexpr (KC) {
                const int kc = tail ? min(kk, (int)(klim - k) - S::V) : kk;
                p = (base + k) + (off[j] + (uint32_t)kc);
            } else {
                const int last = (int)(klim - k) - 1, kj = kk + KSTEP * j;
                if (tail)
                    p = (base + k * pitch) + (off[0] + (uint32_t)min(kj, last) * (uint32_t)pitch);
                else
                    p = (base + (k + KSTEP * j) * pitch) + (off[0] + (uint32_t)kk * (uint32_t)pitch);
            }
            raw[SLOT][j] = *(const typename Piece<T>::vec*)p;
        }
    }
    template <int SLOT>
    __device__ __forceinline__ void put(T* lds, int64_t k, int64_t klim) const {
        const bool all = full && k + S::BK <= klim;
#pragma unroll
        for (int j = 0; j < S::PER; ++j) {
            int m, kj;
            S::where(j, m, kj);
            T* p = lds + (KC ? m * S::PITCH + kj : kj * S::PITCH + m);
            if (all)
                *(typename Piece<T>::vec*)p = raw[SLOT][j];
            else
                *(typename Piece<T>::vec*)p = keep(raw[SLOT][j], in[KC ? j : 0] && k + kj < klim);
        }
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
    // STEP: outputs between one piece of four and the next (4: 16 outputs in
    // a row; 8: with m0 and m0 + 4, 32 in a row, eight of them per lane)
    template <class S, int STEP>
    static __device__ __forceinline__ type read(const __bf16* lds, int m0, int k0) {
        const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        if constexpr (S::K_CONTIGUOUS) {
            return *(const type*)(lds + (m0 + a) * S::PITCH + k0 + 8 * g);
        } else {
            // lane a of group g addresses row 8 g (+ 4) + a / 4, piece a % 4;
            // it receives output a of the four rows
            const __bf16* p = lds + (k0 + 8 * g + (a >> 2)) * S::PITCH + m0 + STEP * (a & 3);
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
    template <class S, int STEP>
    static __device__ __forceinline__ type read(const float* lds, int m0, int k0) {
        const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        return S::K_CONTIGUOUS ? lds[(m0 + a) * S::PITCH + k0 + g]
                               : lds[(k0 + g) * S::PITCH + m0 + STEP * (a >> 2) + (a & 3)];
    }
    static __device__ __forceinline__ f32x4r_t mma(type a, type b, f32x4r_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
    }
};

// LDS of a product: two buffers of both operands.
template <typename T, bool AKC, bool BKC, int TILE>
constexpr size_t kProductBytes = 2 * sizeof(T) * (Stage<T, AKC, TILE>::ELEMS + Stage<T, BKC, TILE>::ELEMS);
template <typename T, int TILE>
constexpr size_t kMostBytes = std::max(kProductBytes<T, false, true, TILE>,
                                       std::max(kProductBytes<T, true, true, TILE>, kProductBytes<T, false, false, TILE>));

// acc += A B over the reduction [k0, k1).  The pieces of the next two steps
// are on their way while this step's are multiplied; two buffers, one barrier
// per step.  m_at /
// n_at: the first output of this wave's i-th / j-th block.  fp32 adds its
// products in runs of 512 of the reduction, so that a long sum is not one
// chain.
template <typename T, bool AKC, bool BKC, int TILE, int ASTEP = 4, class MA, class NA>
__device__ __forceinline__ void tile_product(f32x4r_t (&acc)[Shape<TILE>::NM][Shape<TILE>::NN], Operand<T, AKC, TILE>& A,
                                             Operand<T, BKC, TILE>& B, int64_t k0, int64_t k1, char* smem, MA m_at,
                                             NA n_at) {
    using SA = Stage<T, AKC, TILE>;
    using SB = Stage<T, BKC, TILE>;
    constexpr int BK = kTileK<T>, NM = Shape<TILE>::NM, NN = Shape<TILE>::NN;
    T* la = (T*)smem;
    T* lb = la + 2 * SA::ELEMS;
    f32x4r_t run[sizeof(T) == 4 ? NM : 1][NN];
    if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < NN; ++j) run[sizeof(T) == 4 ? i : 0][j] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
    }
    auto step = [&](auto slot, int64_t k) {
        constexpr int SLOT = decltype(slot)::value;
        A.template put<SLOT>(la + SLOT * SA::ELEMS, k, k1);
        B.template put<SLOT>(lb + SLOT * SB::ELEMS, k, k1);
        __syncthreads();
        A.template fetch<SLOT>(k + 2 * BK, k1);
        B.template fetch<SLOT>(k + 2 * BK, k1);
        const T* pa = la + SLOT * SA::ELEMS;
        const T* pb = lb + SLOT * SB::ELEMS;
#pragma unroll
        for (int s = 0; s < BK; s += Frag<T>::K) {
            typename Frag<T>::type fa[NM], fb[NN];
#pragma unroll
            for (int i = 0; i < NM; ++i) fa[i] = Frag<T>::template read<SA, ASTEP>(pa, m_at(i), s);
#pragma unroll
            for (int j = 0; j < NN; ++j) fb[j] = Frag<T>::template read<SB, 4>(pb, n_at(j), s);
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int j = 0; j < NN; ++j) {
                    if constexpr (sizeof(T) == 4)
                        run[i][j] = Frag<T>::mma(fa[i], fb[j], run[i][j]);
                    else
                        acc[i][j] = Frag<T>::mma(fa[i], fb[j], acc[i][j]);
                }
        }
        if constexpr (sizeof(T) == 4) {
            if (((k - k0) & 511) == 512 - BK || k + BK >= k1) {
#pragma unroll
                for (int i = 0; i < NM; ++i)
#pragma unroll
                    for (int j = 0; j < NN; ++j) {
                        acc[i][j] += run[i][j];
                        run[i][j] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
                    }
            }
        }
    };
    A.template fetch<0>(k0, k1);
    B.template fetch<0>(k0, k1);
    A.template fetch<1>(k0 + BK, k1);
    B.template fetch<1>(k0 + BK, k1);
    for (int64_t k = k0; k < k1; k += 2 * BK) {
        step(std::integral_constant<int, 0>{}, k);
        if (k + BK < k1) step(std::integral_constant<int, 1>{}, k + BK);
    }
    __syncthreads();        // the buffers may be used again
}
template <int NM, int NN>
__device__ __forceinline__ void clear_blocks(f32x4r_t (&acc)[NM][NN]) {
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j) acc[i][j] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
}

// Workgroups go round the 8 XCDs, each of which has its own L2.  Blocks that
// read the same rows (`inner` of them to each of `outer`) stand 8 apart, so
// that they run on one XCD, where there are enough of the outer ones to give
// every XCD several; else in a row.  False: no such block.
constexpr int kXcds = 8;
__host__ __device__ __forceinline__ bool by_xcd(int64_t outer) { return outer >= 2 * kXcds; }
__device__ __forceinline__ bool place_block(int64_t id, int64_t outer, int inner, int64_t& o, int& i) {
    if (by_xcd(outer)) {
        const int64_t k = id / kXcds;
        o = k / inner * kXcds + id % kXcds;
        i = (int)(k % inner);
    } else {
        o = id / inner;
        i = (int)(id % inner);
    }
    return o < outer;
}
int64_t block_count(int64_t outer, int64_t inner) { return (by_xcd(outer) ? round_up(outer, kXcds) : outer) * inner; }

// A launch's threads are counted in 32 bits: at 2^32 it is refused, above it runs
// only what is left of the number.  Calls with more (fp32, h of 137 GB; rows of 8
// channels from 2^30 on) take several launches, of whole rounds of the XCDs.
constexpr int64_t kLaunchThreads = (int64_t)1 << 31;
template <class L>
hipError_t launch_blocks(GluParams& p, int64_t blocks, int threads, L launch) {
    const int64_t most = kLaunchThreads / threads;
    for (p.first_block = 0; p.first_block < blocks; p.first_block += most) {
        launch((unsigned)std::min(most, blocks - p.first_block));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// TILE rows x TILE / 2 hidden features, both projections: h, or (GRAD) da and
// db with their sums over the tile's rows.
template <typename T, int ACT, bool GRAD, int TILE>
__global__ void __launch_bounds__(Shape<TILE>::THREADS, TILE == 128 ? 4 : 3) k_glu_project(GluParams p) {
    constexpr int NM = Shape<TILE>::NM, NN = Shape<TILE>::NN, WN = Shape<TILE>::WN, FT = TILE / 2;
    constexpr int FW = FT / Shape<TILE>::WM;      // features of a wave
    __shared__ __align__(16) char smem[kProductBytes<T, false, true, TILE>];
    __shared__ float bsum[WN][2][FT];
    const int wave = threadIdx.x >> 6, wm = wave % Shape<TILE>::WM, wn = wave / Shape<TILE>::WM;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F;
    int64_t tile;
    int f0;
    if (!place_block(p.first_block + blockIdx.x, (p.N + TILE - 1) / TILE, (F + FT - 1) / FT, tile, f0)) return;
    f0 *= FT;
    const int64_t r0 = tile * TILE;
    const T* x = (const T*)p.x;
    const T* w = (const T*)p.w;
    Operand<T, false, TILE> A(w + f0, [&](int m) { return (uint32_t)(m / FT) * C * F + m % FT; },
                              [&](int m) { return f0 + m % FT < F; }, f0 + FT <= F, F);
    Operand<T, true, TILE> B(x + r0 * C, [&](int n) { return (uint32_t)n * C; },
                             [&](int n) { return r0 + n < p.N; }, r0 + TILE <= p.N, 0);
    // A lane's features: E in a row (of the wave's FW: 4 from each block, 8
    // from each pair of blocks).
    constexpr int PAIR = NM / 2 >= 2 ? 2 : 1, E = 4 * PAIR, NP = NM / 2 / PAIR;
    typedef typename Group<T, E>::vec group;
    f32x4r_t acc[NM][NN];      // gates in the first half of i, values in the second
    int f[NP];
    group dh[GRAD ? NP : 1][NN];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        f[i] = f0 + FW * wm + 16 * PAIR * i + E * g;
#pragma unroll
        for (int q = 0; q < PAIR; ++q) {
            const int at = f[i] < F ? f[i] + 4 * q : 0;
            f32x4r_t ba = {0.f, 0.f, 0.f, 0.f}, bb = ba;
            if (p.bias) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ba[e] = p.bias[at + e];
                    bb[e] = p.bias[F + at + e];
                }
            }
#pragma unroll
            for (int j = 0; j < NN; ++j) {
                acc[PAIR * i + q][j] = ba;
                acc[NM / 2 + PAIR * i + q][j] = bb;
            }
        }
        if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < NN; ++j) {
                const int64_t r = min(r0 + 16 * NN * wn + 16 * j + a, p.N - 1);
                dh[i][j] = *(const group*)((const T*)p.dout + r * F + (f[i] < F ? f[i] : 0));
            }
        }
    }
    tile_product<T, false, true, TILE, 4 * PAIR>(
        acc, A, B, 0, C, smem,
        [&](int i) {
            const int k = i % (NM / 2);
            return FT * (2 * i / NM) + FW * wm + 16 * PAIR * (k / PAIR) + 4 * (k % PAIR);
        },
        [&](int j) { return 16 * NN * wn + 16 * j; });
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float sa[E], sb[E];
#pragma unroll
        for (int e = 0; e < E; ++e) sa[e] = sb[e] = 0.f;
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const int64_t r = r0 + 16 * NN * wn + 16 * j + a;
            if (r >= p.N || f[i] >= F) continue;
            group o, q;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float va = acc[PAIR * i + e / 4][j][e % 4], vb = acc[NM / 2 + PAIR * i + e / 4][j][e % 4];
                const Act t = activation<ACT, sizeof(T) == 4>(va);
                if constexpr (!GRAD) {
                    o[e] = (T)(t.v * vb);
                } else {
                    const float d = (float)dh[i][j][e], u = d * vb * t.d, v = d * t.v;
                    sa[e] += u;
                    sb[e] += v;
                    o[e] = (T)u;
                    q[e] = (T)v;
                }
            }
            if constexpr (!GRAD) {
                *(group*)((T*)p.h + r * F + f[i]) = o;
            } else {
                T* d = (T*)p.dab + r * 2 * F + f[i];
                *(group*)d = o;
                *(group*)(d + F) = q;
            }
        }
        if constexpr (GRAD) {
            if (p.bpart) {
                const int fl = f[i] - f0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
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
        const int s = threadIdx.x / FT, fl = threadIdx.x % FT;
        if (threadIdx.x < 2 * FT && f0 + fl < F) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < WN; ++k) t += bsum[k][s][fl];
            p.bpart[(tile * 2 + s) * F + f0 + fl] = t;
        }
    }
}

// dx: TILE rows x TILE channels, reduced over both halves of dab, or over one
// split of them as a partial sum.
template <typename T, int TILE>
__device__ __forceinline__ void glu_dx_tile(const GluParams& p, int64_t block, char* smem) {
    constexpr int NM = Shape<TILE>::NM, NN = Shape<TILE>::NN;
    const int wave = threadIdx.x >> 6, wm = wave % Shape<TILE>::WM, wn = wave / Shape<TILE>::WM;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F;
    int64_t r0;
    int at;
    const int ct = (C + TILE - 1) / TILE;
    if (!place_block(block, (p.N + TILE - 1) / TILE, ct * p.dx_splits, r0, at)) return;
    r0 *= TILE;
    const int c0 = at % ct * TILE, split = at / ct;
    f32x4r_t acc[NM][NN];
    clear_blocks(acc);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
        const int k0 = max(split * p.dx_per - s * F, 0), k1 = min((split + 1) * p.dx_per - s * F, F);
        if (k0 >= k1) continue;
        Operand<T, true, TILE> A((const T*)p.w + ((int64_t)s * C + c0) * F, [&](int m) { return (uint32_t)m * F; },
                                 [&](int m) { return c0 + m < C; }, c0 + TILE <= C, 0);
        Operand<T, true, TILE> B((const T*)p.dab + r0 * 2 * F + s * F, [&](int n) { return (uint32_t)n * 2 * F; },
                                 [&](int n) { return r0 + n < p.N; }, r0 + TILE <= p.N, 0);
        tile_product<T, true, true, TILE>(acc, A, B, k0, k1, smem, [&](int i) { return 16 * NM * wm + 16 * i; },
                                          [&](int j) { return 16 * NN * wn + 16 * j; });
    }
#pragma unroll
    for (int i = 0; i < NM; ++i) {
        const int c = c0 + 16 * NM * wm + 16 * i + 4 * g;
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const int64_t r = r0 + 16 * NN * wn + 16 * j + a;
            if (r >= p.N || c >= C) continue;
            if (p.xpart) {
                *(f32x4r_t*)(p.xpart + (split * p.N + r) * C + c) = acc[i][j];
            } else {
                const float o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                store_four((T*)p.dx + r * C + c, o);
            }
        }
    }
}

// dw of one split of the rows: TILE columns of dab x TILE channels, as a
// partial sum, or (one split) as it is.
template <typename T, int TILE>
__device__ __forceinline__ void glu_dw_tile(const GluParams& p, int64_t block, char* smem) {
    constexpr int NM = Shape<TILE>::NM, NN = Shape<TILE>::NN;
    const int wave = threadIdx.x >> 6, wm = wave % Shape<TILE>::WM, wn = wave / Shape<TILE>::WM;
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F, F2 = 2 * F;
    const int mt = (F2 + TILE - 1) / TILE, ct = (C + TILE - 1) / TILE;
    int64_t split;
    int at;
    if (!place_block(block, (p.N + p.rows_per_split - 1) / p.rows_per_split, mt * ct, split, at)) return;
    const int m0 = at % mt * TILE, c0 = at / mt * TILE;
    const int64_t k0 = split * p.rows_per_split, k1 = min(p.N, k0 + p.rows_per_split);
    Operand<T, false, TILE> A((const T*)p.dab + m0, [&](int m) { return (uint32_t)m; },
                              [&](int m) { return m0 + m < F2; }, m0 + TILE <= F2, F2);
    Operand<T, false, TILE> B((const T*)p.x + c0, [&](int n) { return (uint32_t)n; },
                              [&](int n) { return c0 + n < C; }, c0 + TILE <= C, C);
    f32x4r_t acc[NM][NN];
    clear_blocks(acc);
    tile_product<T, false, false, TILE>(acc, A, B, k0, k1, smem, [&](int i) { return 16 * NM * wm + 16 * i; },
                                        [&](int j) { return 16 * NN * wn + 16 * j; });
    float* part = p.wpart + split * C * F2;
#pragma unroll
    for (int i = 0; i < NM; ++i) {
        const int m = m0 + 16 * NM * wm + 16 * i + 4 * g;
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const int64_t c = c0 + 16 * NN * wn + 16 * j + a;
            if (m >= F2 || c >= C) continue;
            if (p.wpart) {
                *(f32x4r_t*)(part + c * F2 + m) = acc[i][j];
            } else {
                const float o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                store_four((T*)p.dw + (m < F ? c * F + m : (C + c) * F + (m - F)), o);
            }
        }
    }
}

// Both products of the gradient: they need the same da and db and nothing of
// each other.
template <typename T, int TILE>
__global__ void __launch_bounds__(Shape<TILE>::THREADS, TILE == 128 ? 4 : 3) k_glu_products(GluParams p, int64_t dx_blocks) {
    __shared__ __align__(16) char smem[kMostBytes<T, TILE>];
    const int64_t block = p.first_block + blockIdx.x;
    if (block < dx_blocks)
        glu_dx_tile<T, TILE>(p, block, smem);
    else
        glu_dw_tile<T, TILE>(p, block - dx_blocks, smem);
}

// The partial sums of dw (splits, C, 2 F), dbias (tiles, 2 F) and dx (splits,
// N, C) added in their order and rounded once; the first w_blocks workgroups
// serve dw, the next b_blocks dbias.
template <typename T>
__global__ void __launch_bounds__(kJoinCols * 16) k_glu_join(GluParams p, int splits, int64_t tiles, float* dbias,
                                                             unsigned w_blocks, unsigned b_blocks) {
    if (blockIdx.x >= w_blocks + b_blocks) {
        // few splits: a lane adds four columns by itself
        const int64_t n = p.N * p.C;
        const int64_t e = ((int64_t)(blockIdx.x - w_blocks - b_blocks) * (kJoinCols * 16) + threadIdx.x) * 4;
        if (e >= n) return;
        f32x4r_t t = *(const f32x4r_t*)(p.xpart + e);
#pragma unroll 4
        for (int q = 1; q < p.dx_splits; ++q) t += *(const f32x4r_t*)(p.xpart + q * n + e);
        const float o[4] = {t[0], t[1], t[2], t[3]};
        store_four((T*)p.dx + e, o);
        return;
    }
    const int F = p.F;
    const bool w = blockIdx.x < w_blocks;
    const int64_t n = w ? (int64_t)p.C * 2 * F : 2 * F;
    const int64_t block = blockIdx.x - (w ? 0 : w_blocks);
    const JoinVec<4> t = join_columns<16, 4>(w ? p.wpart : p.bpart, w ? splits : tiles, n, block);
    const int64_t e = (block * kJoinCols + threadIdx.x) * 4;
    if (threadIdx.x >= kJoinCols || e >= n) return;
    if (!w) {
        *(f32x4ru_t*)(dbias + e) = f32x4ru_t{t.f[0], t.f[1], t.f[2], t.f[3]};    // aligned to its elements only
        return;
    }
    const int64_t c = e / (2 * F);
    const int m = (int)(e % (2 * F));
    store_four((T*)p.dw + (m < F ? c * F + m : (p.C + c) * F + (m - F)), t.f);
}

// Few channels and enough rows: glu_rows.hip.  Its blocks have 256 rows and one of
// them fills a CU, so that a call takes the same time up to 65,536 rows, while the
// tiles' time grows with the rows.  The two cross at about 49,152 rows forward and
// 32,768 in the gradient, which reads and writes da and db with tiles.  us, rows
// against tiles:
//                    forward                                 gradient
//   C -> F       32,768       49,152       65,536       24,576       32,768       49,152
//   32 -> 256    11.9/10.3    12.7/13.7    13.5/16.9    29.9/34.9    31.7/41.4    34.2/51.3
//   64 -> 512    21.9/16.9    22.5/22.3    22.8/28.3    52.2/58.9    56.2/66.3    62.1/84.9
//   128 -> 256   17.1/12.0    18.1/16.6    19.3/21.0    50.6/44.5    54.1/53.4    57.9/65.5
//   128 -> 1024  49.8/36.5    51.5/52.5    56.2/68.7   121.1/108.8  129.1/124.4  148.1/187.7
// Weights that take several slabs of LDS (128 -> 344 and wider), loaded again for
// every block, do not turn this: 131,072 rows 128 -> 344 49/52 and 180/218 us,
// 128 -> 1024 117/163 and 324/541.
bool use_rows(int64_t N, int C, int dtype, bool grad) {
    return dtype == SPCONV_BF16 && C <= kGluRowC && N >= (grad ? 32768 : 49152);
}

// Tiles of 128 where they fill the card (the operands are then read half as
// often), of 64 where they would not.
int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }
// (fp32, whose matrix instructions take four times as long as their operands'
// reads, has no use for those.)
int big_tile(bool fills, int dtype) { return fills && dtype == SPCONV_BF16 ? 128 : 64; }

struct GluLayout {
    size_t dab, bpart, wpart, total;
    int64_t tiles, rows_per_split;    // row tiles of the projections; rows per split of dw
    int splits, tile, ptile;          // tile of the products and of the projections
    int dx_splits, dx_per;
    size_t xpart;
    bool rows;
};
GluLayout glu_layout(int64_t N, int C, int F, int dtype, bool grad) {
    GluLayout l{};
    l.rows = use_rows(N, C, dtype, grad);
    if (l.rows) {
        const int want = glu_rows_splits(N, C, F);
        l.rows_per_split = round_up((N + want - 1) / want, 64);
        l.splits = (int)((N + l.rows_per_split - 1) / l.rows_per_split);
        l.tiles = l.splits;
        l.wpart = align_up((size_t)l.splits * 2 * F * 4, 256);
        l.total = l.wpart + align_up((size_t)l.splits * C * 2 * F * 4, 256);
        return l;
    }
    l.ptile = big_tile(tiles_of(N, 128) * tiles_of(F, 64) >= 256, dtype);
    // The projections' reduction is not split (the activations need all of it).
    // In fp32 a tile of 64 is 32 cycles of matrix instructions for each channel:
    // tiles of 32 where those of 64 leave CUs idle (one row, 1024 -> 4096: 32.5
    // -> 23.3 us; a little slower where they do not).
    if (dtype == SPCONV_F32 && tiles_of(N, 64) * tiles_of(F, 32) < 256) l.ptile = 32;
    l.tiles = tiles_of(N, l.ptile);
    l.tile = big_tile(tiles_of(N, 128) * tiles_of(C, 128) >= 192, dtype);
    // enough workgroups for two per CU, at least 128 rows each
    const int64_t t = tiles_of(2 * F, l.tile) * tiles_of(C, l.tile);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>((512 + t - 1) / t, N / 128));
    l.rows_per_split = round_up((N + want - 1) / want, 64);
    l.splits = l.rows_per_split ? (int)((N + l.rows_per_split - 1) / l.rows_per_split) : 0;
    size_t at = 0;
    l.dab = at;
    at += align_up((size_t)N * 2 * F * (dtype == SPCONV_BF16 ? 2 : 4), 256);
    l.bpart = at;
    if (l.tiles > 1) at += align_up((size_t)l.tiles * 2 * F * 4, 256);
    l.wpart = at;
    if (l.splits > 1) at += align_up((size_t)l.splits * C * 2 * F * 4, 256);
    // dx, where its tiles leave most of the card idle and its reduction is long
    // (one row, 1024 -> 4096 fp32: 248 us unsplit): splits of at least four steps,
    // or eight where only dx would need the sums to be joined
    const int bk = dtype == SPCONV_BF16 ? kTileK<__bf16> : kTileK<float>, least = l.splits > 1 ? 4 : 8;
    const int64_t dx = std::max<int64_t>(1, tiles_of(N, l.tile) * tiles_of(C, l.tile)), steps = tiles_of(2 * F, bk);
    l.dx_splits = 1;
    l.dx_per = 2 * F;
    if (dx < 256 && steps >= 3 * least) {
        const int64_t want = std::min<int64_t>((512 + dx - 1) / dx, steps / least);
        l.dx_per = (int)tiles_of(steps, want) * bk;
        l.dx_splits = (int)tiles_of(2 * F, l.dx_per);
    }
    l.xpart = at;
    if (l.dx_splits > 1) at += align_up((size_t)l.dx_splits * N * C * 4, 256);
    l.total = at;
    return l;
}

template <typename T, int ACT>
hipError_t glu_project(GluParams p, bool grad, const GluLayout& l, hipStream_t st) {
    const int64_t blocks = block_count(l.tiles, tiles_of(p.F, l.ptile / 2));
    int threads = Shape<64>::THREADS;
    auto fn = grad ? k_glu_project<T, ACT, true, 64> : k_glu_project<T, ACT, false, 64>;
    if constexpr (sizeof(T) == 2) {
        if (l.ptile == 128) {
            fn = grad ? k_glu_project<T, ACT, true, 128> : k_glu_project<T, ACT, false, 128>;
            threads = Shape<128>::THREADS;
        }
    } else if (l.ptile == 32) {
        fn = grad ? k_glu_project<T, ACT, true, 32> : k_glu_project<T, ACT, false, 32>;
        threads = Shape<32>::THREADS;
    }
    return launch_blocks(p, blocks, threads, [&](unsigned n) { fn<<<n, threads, 0, st>>>(p); });
}

template <typename T>
hipError_t glu_products(GluParams p, const GluLayout& l, hipStream_t st) {
    const int64_t dx = block_count(tiles_of(p.N, l.tile), tiles_of(p.C, l.tile) * l.dx_splits);
    const int64_t dw = block_count(l.splits, tiles_of(2 * p.F, l.tile) * tiles_of(p.C, l.tile));
    const int threads = l.tile == 128 ? Shape<128>::THREADS : Shape<64>::THREADS;
    auto fn = k_glu_products<T, 64>;
    if constexpr (sizeof(T) == 2) {
        if (l.tile == 128) fn = k_glu_products<T, 128>;
    }
    return launch_blocks(p, dx + dw, threads, [&](unsigned n) { fn<<<n, threads, 0, st>>>(p, dx); });
}

template <typename T>
hipError_t glu_go(GluParams p, int act, bool grad, const GluLayout& l, float* dbias, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (l.rows) {
        if constexpr (sizeof(T) == 2) {
            if (!grad) return launch_glu_rows(p, act, st);
            e = launch_glu_rows_dx(p, act, st);
            if (e == hipSuccess) e = launch_glu_rows_dw(p, act, l.splits, st);
        }
    } else if (p.N > 0) {
        e = act == SPCONV_SILU ? glu_project<T, SPCONV_SILU>(p, grad, l, st) : glu_project<T, SPCONV_GELU>(p, grad, l, st);
        if (!grad || e != hipSuccess) return e;
        e = glu_products<T>(p, l, st);
    }
    if (e != hipSuccess) return e;
    // what was not written as it is (no rows: the zeros of both)
    const bool w = p.wpart || p.N == 0, b = dbias && (p.bpart != dbias || p.N == 0);
    const unsigned wb = w ? (unsigned)tiles_of((int64_t)p.C * 2 * p.F, 4 * kJoinCols) : 0;
    const unsigned bb = b ? (unsigned)tiles_of(2 * p.F, 4 * kJoinCols) : 0;
    const unsigned xb = p.xpart ? (unsigned)tiles_of(p.N * p.C, 4 * kJoinCols * 16) : 0;
    if (wb + bb + xb)
        k_glu_join<T><<<wb + bb + xb, kJoinCols * 16, 0, st>>>(p, l.splits, l.tiles, dbias, wb, bb);
    return hipGetLastError();
}

}  // namespace

size_t glu_grad_workspace_bytes(int64_t N, int C, int F, int dtype) { return glu_layout(N, C, F, dtype, true).total; }

hipError_t launch_glu(const GluArgs& a, bool grad, hipStream_t stream) {
    if (a.N == 0 && !grad) return hipSuccess;
    const GluLayout l = glu_layout(a.N, a.C, a.F, a.dtype, grad);
    GluParams p{};
    p.x = a.x;
    p.w = a.w;
    p.bias = a.bias;
    p.dout = a.dout;
    p.h = a.out;
    p.dx = a.out;
    p.dw = a.dw;
    if (grad) {
        // sums of one tile or split are results already
        char* ws = (char*)a.workspace;
        p.dab = ws + l.dab;
        if (a.dbias) p.bpart = l.rows || l.tiles > 1 ? (float*)(ws + l.bpart) : a.dbias;
        if (l.rows || l.splits > 1) p.wpart = (float*)(ws + l.wpart);
        if (l.dx_splits > 1) p.xpart = (float*)(ws + l.xpart);
        p.dx_splits = l.dx_splits;
        p.dx_per = l.dx_per;
    }
    p.N = a.N;
    p.C = a.C;
    p.F = a.F;
    p.rows_per_split = l.rows_per_split;
    p.stream = a.N * (grad ? a.C : a.F) * (a.dtype == SPCONV_BF16 ? 2 : 4) > kStreamBytes;
    return a.dtype == SPCONV_BF16 ? glu_go<__bf16>(p, a.act, grad, l, a.dbias, stream)
                                  : glu_go<float>(p, a.act, grad, l, a.dbias, stream);
}

}  // namespace spc
