// Gated linear unit of bfloat16 rows with at most 128 channels, and its
// gradient, for gfx950.  (Wider rows: glu.hip.)
//
// With few channels the products are short and the rows' traffic is what
// counts: x and dout are read from memory once, and a, b, da and db never
// leave the chip.  The forward and dx keep a slab of the weights in LDS (C x
// 2 x 256 features at 128 channels: 128 KB) and hand each wave rows of its own;
// dw keeps the weights and its sums in registers and hands each wave features
// of its own.  Each of the two gradient kernels computes a and b again: 4 N C F
// operations, where writing da and db and reading them twice would be 12 N F
// bytes, which takes longer below about 300 channels.
//
// 1,006,716 rows, 128 -> 256, silu: 188 to 200 us forward, card by card (3.9 to 4.1
// TB/s), 613 to 636 us gradient (830 to 860 TFLOP/s with what is computed again).  With
// fewer channels the forward's time follows its activations, not its bytes: 100,000
// rows 32 -> 256 take 18 us (3.1 TB/s), 64 -> 512 34 us (3.3).  The gradient's kernels
// are bound by issue:
// vector instructions (the activations) fill 55% of the slots, matrix instructions
// keep their unit busy for 41% of the time, at a clock that the load lowers.
//
// Matrix instructions (16 x 16 x 32) number their outputs so that lanes end up
// with eight consecutive features (channels) of a row: output m of tile t is
// feature 8 (m >> 2) + 4 t + (m & 3) of 32.  That makes 16-byte accesses of h,
// dout and dx, and makes da and db, once rounded, the operand of the next
// product as they are.
#include "glu.h"

#include <algorithm>
#include <type_traits>

namespace spc {

namespace {

// Two waves per SIMD, one workgroup per CU.  (The forward's registers would
// allow three waves; they take 215 us where two take 182 at 1,006,716 rows,
// 128 -> 256, the one width where both were measured: the LDS reads of the weights
// get in each other's way.)
constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int NT = 2;                 // 16-row tiles per wave
constexpr int kWaveRows = 16 * NT;
constexpr int kBlockRows = kRowWaves * kWaveRows;
constexpr int kSlabElems = 65536;     // of w in LDS: 128 KB
constexpr int kCUs = 256;

__device__ __forceinline__ f32x4r_t mma(bf16x8r_t a, bf16x8r_t b, f32x4r_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8r_t join8(bf16x4r_t lo, bf16x4r_t hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// lane a of each 16 addresses four elements of its own and receives element
// a & 3 of the four lanes 4 (a >> 2) .. of the addressing order: the 16 x 4
// transpose of what was addressed as 4 rows of 4 pieces
__device__ __forceinline__ bf16x4r_t read_tr(const __bf16* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4r_t*)p);
}
// the same at byte offset q of LDS, and 16 bytes there
__device__ __forceinline__ bf16x4r_t read_tr(uint32_t q) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4r_t*)(uintptr_t)q);
}
typedef __attribute__((address_space(3))) bf16x8r_t lds_bf16x8r_t;
__device__ __forceinline__ bf16x8r_t read_unit(uint32_t q) { return *(lds_bf16x8r_t*)(uintptr_t)q; }
__device__ __forceinline__ void opaque(uint32_t& v) { asm volatile("" : "+v"(v)); }
// Matrix instructions and LDS reads stay on their sides of this, so that the
// next step's operands are read before this step's products, not after.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x416); }
// Consecutive rows as a buffer: a load's place costs one 32-bit offset (bytes),
// and past the rows it reads zeros.
constexpr uint32_t kOutside = 0x7FFFFFF0u;
struct RowBuffer {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ RowBuffer(const __bf16* p, int elems)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<__bf16*>(p), (short)0, elems * 2, 0x00020000)) {}
    __device__ __forceinline__ bf16x8r_t load8(uint32_t offset, uint32_t step = 0) const {
        const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, offset, step, 0);
        bf16x8r_t v;
        __builtin_memcpy(&v, &w, 16);
        return v;
    }
};
// One activation's instructions stand between four matrix instructions, whose
// operands' reads come first.
__device__ __forceinline__ void interleave() {
    __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x402, 4, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void store_unit(__bf16* p, bf16x8r_t v, bool stream) {
    if (stream)
        __builtin_nontemporal_store(v, (bf16x8r_t*)p);
    else
        *(bf16x8r_t*)p = v;
}
// Rows' loads stand under no branch: a branch between loads makes the compiler
// wait for all of them at the first use of any.  Lanes past the end read a
// valid place instead, and what they got is replaced where it is used.
__device__ __forceinline__ bf16x8r_t load8(const __bf16* p) { return *(const bf16x8r_t*)p; }
__device__ __forceinline__ bf16x8r_t keep(bf16x8r_t v, bool in) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 w;
    __builtin_memcpy(&w, &v, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = in ? w[i] : 0u;
    __builtin_memcpy(&v, &w, 16);
    return v;
}

// Weights in LDS: row c holds the slab's gates and then its values, in 16-byte
// units of 8 features; unit u of row c stands at u ^ swizzle(c): 16 rows' unit u
// (dx) and the four units of four consecutive rows (the projections,
// transposed) lie on different banks.  The slab's size is fixed, so that rows
// and tiles are constant offsets from one address per group of 32 features.
__device__ __forceinline__ int swizzle(int c) { return ((c & 3) << 2) | ((c >> 3) & 3); }
template <int KC>
constexpr int kSlab = kSlabElems / (KC * 32 * 2);       // features

// Features [f0, f0 + kSlab) of w, as far as F goes up to a multiple of 32
// (zeros past F and C).
template <int KC>
__device__ __forceinline__ void load_slab(__bf16* lw, float* lb, const GluParams& p, int f0) {
    constexpr int FS = kSlab<KC>, UNITS = FS / 8;
    const __bf16* w = (const __bf16*)p.w;
    const int n = min((p.F - f0 + 31) / 32 * 4, UNITS);    // units with features
    // eight units at a time, all loads before the first store
    constexpr int B = 8;
    const int total = KC * 32 * 2 * n;
    for (int e0 = threadIdx.x; e0 < total; e0 += B * kRowThreads) {
        bf16x8r_t v[B];
        int at[B];
        bool in[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int e = min(e0 + j * kRowThreads, total - 1);
            const int c = e / (2 * n), u = e - c * 2 * n, s = u >= n, ul = u - s * n, f = f0 + ul * 8;
            in[j] = c < p.C && f < p.F;
            v[j] = load8(w + (in[j] ? ((int64_t)s * p.C + c) * p.F + f : 0));
            at[j] = (c * 2 * UNITS + s * UNITS + (ul ^ swizzle(c))) * 8;
        }
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (e0 + j * kRowThreads < total) *(bf16x8r_t*)(lw + at[j]) = keep(v[j], in[j]);
    }
    for (int e = threadIdx.x; e < 2 * FS; e += kRowThreads) {
        const int s = e >= FS, f = f0 + e - s * FS;
        lb[e] = p.bias && f < p.F ? p.bias[s * p.F + f] : 0.f;
    }
}

// The rows of a wave as operands: x[n][s] holds channels 32 s + 8 g .. of row
// 16 n + a (channel 0 on where those are past C, the last row past the rows).
template <int KC, int ROWS>
__device__ __forceinline__ void load_rows(bf16x8r_t (&x)[ROWS][KC], const GluParams& p, int64_t r0) {
    const int a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int n = 0; n < ROWS; ++n) {
        const __bf16* row = (const __bf16*)p.x + min(r0 + 16 * n + a, p.N - 1) * p.C;
#pragma unroll
        for (int s = 0; s < KC; ++s) x[n][s] = load8(row + (32 * s + 8 * g < p.C ? 32 * s + 8 * g : 0));
    }
}

// The forward, and with DX the input gradient: 32 rows per wave at a time, over
// the slabs of the hidden features.
template <int KC, int ACT, bool DX>
__global__ void __launch_bounds__(kRowThreads) k_glu_rows(GluParams p) {
    extern __shared__ __align__(16) char smem[];
    __bf16* lw = (__bf16*)smem;
    float* lb = (float*)(smem + (size_t)kSlabElems * 2);
    constexpr int FS = kSlab<KC>, PITCH = 2 * FS;        // elements per row
    const int wave = threadIdx.x >> 6, a = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int C = p.C, F = p.F;
    // Byte offsets in LDS.  Projections: row 8 g + (a >> 2) of each 32, piece
    // (a & 3) of the group's units; dx: row 8 (a >> 2) + (a & 3) of each 32,
    // unit g of the group.
    const uint32_t w0 = (uint32_t)(uintptr_t)(lds_bf16x4r_t*)lw;
    const uint32_t w1 = w0 + (8 * g + (a >> 2)) * PITCH * 2;
    const uint32_t x1 = (swizzle(8 * g + (a >> 2)) ^ (a & 3)) * 16;
    const uint32_t w2 = w0 + (8 * (a >> 2) + (a & 3)) * PITCH * 2;
    const uint32_t x2 = (swizzle(8 * (a >> 2) + (a & 3)) ^ g) * 16;
    // The workgroup's tiles of 32 rows, numbered through its blocks.  With one
    // slab its waves take them from a counter: of the two on a SIMD one runs
    // ahead of the other, and with even shares it would leave the SIMD half
    // idle for the last quarter (finishing after 213 us where the other took
    // 294).  Which wave computes a tile does not change it.
    int* taken = (int*)(lb + 2 * FS);
    auto tile_row = [&](int i) {
        return ((int64_t)(i / kRowWaves) * gridDim.x + blockIdx.x) * kBlockRows + i % kRowWaves * kWaveRows;
    };
    const bool whole = FS >= F;
    if (whole) {
        if (threadIdx.x == 0) *taken = kRowWaves;
        load_slab<KC>(lw, lb, p, 0);
        __syncthreads();
    }
    auto next_tile = [&](int i) {
        if (!whole) return i + kRowWaves;
        int t = 0;
        if ((threadIdx.x & 63) == 0) t = atomicAdd(taken, 1);
        return __builtin_amdgcn_readfirstlane(t);
    };
    // The next rows: the forward loads them a whole block ahead; dx, whose sums
    // need the registers, into the operands themselves after their last use.
    bf16x8r_t x[NT][KC], xn[DX ? 1 : NT][KC];
    int tile = wave;
    if constexpr (DX)
        load_rows(x, p, tile_row(tile));
    else
        load_rows(xn, p, tile_row(tile));
    for (;;) {
        const int64_t r0 = tile_row(tile);
        if (whole ? r0 >= p.N : r0 - wave * kWaveRows >= p.N) break;      // (slabs: all waves together)
        tile = next_tile(tile);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int s = 0; s < KC; ++s) x[n][s] = keep(DX ? x[n][s] : xn[DX ? 0 : n][s], 32 * s + 8 * g < C);
        if constexpr (!DX) load_rows(xn, p, tile_row(tile));
        f32x4r_t dx[DX ? 2 * KC : 1][NT];
        if constexpr (DX) {
#pragma unroll
            for (int i = 0; i < 2 * KC; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) dx[i][n] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
        }
        for (int f0 = 0; f0 < F; f0 += FS) {
            if (!whole) {
                __syncthreads();
                load_slab<KC>(lw, lb, p, f0);
                __syncthreads();
            }
            const int fe = min(FS, F - f0);
            bf16x8r_t dn[NT];
            auto load_dout = [&](int fl) {
                const int f = f0 + (fl + 8 * g < fe ? fl + 8 * g : 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    dn[n] = load8((const __bf16*)p.dout + min(r0 + 16 * n + a, p.N - 1) * F + f);
            };
            if constexpr (DX) load_dout(0);
            for (int fl = 0; fl < fe; fl += 32) {
                bf16x8r_t dh[NT];
                if constexpr (DX) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) dh[n] = keep(dn[n], fl + 8 * g < fe);
                    load_dout(fl + 32);
                }
                f32x4r_t pa[2][NT], pb[2][NT];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4r_t ba = *(const f32x4r_t*)(lb + fl + 8 * g + 4 * t);
                    const f32x4r_t bb = *(const f32x4r_t*)(lb + FS + fl + 8 * g + 4 * t);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        pa[t][n] = ba;
                        pb[t][n] = bb;
                    }
                }
                // step i: tile i & 1 of both projections over channels 32 (i / 2) ..
                const uint32_t q1 = w1 + ((fl * 2) ^ x1);
                uint32_t q1h = q1 + 0x10000;         // an offset reaches 64 KB
                opaque(q1h);
                auto read1 = [&](int i, bf16x8r_t (&w)[2]) {
                    const uint32_t at = 8 * (i & 1) + 64 * (i >> 1) * PITCH;
                    const uint32_t q = (at < 0x10000 ? q1 : q1h) + (at & 0xFFFF);
                    w[0] = join8(read_tr(q), read_tr(q + 8 * PITCH));
                    w[1] = join8(read_tr(q + 2 * FS), read_tr(q + 2 * FS + 8 * PITCH));
                };
                constexpr int STEPS = 2 * KC, AHEAD = STEPS < 3 ? STEPS : 3;      // operands on their way
                bf16x8r_t wf[4][2];
#pragma unroll
                for (int i = 0; i < AHEAD - 1; ++i) read1(i, wf[i]);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    if (i + AHEAD - 1 < STEPS) read1(i + AHEAD - 1, wf[(i + AHEAD - 1) % AHEAD]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        pa[i & 1][n] = mma(wf[i % AHEAD][0], x[n][i >> 1], pa[i & 1][n]);
                        pb[i & 1][n] = mma(wf[i % AHEAD][1], x[n][i >> 1], pb[i & 1][n]);
                    }
                    keep_order();
                }
                if (DX && f0 + fl + 32 >= F) load_rows(x, p, tile_row(tile));
                if constexpr (!DX) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        bf16x8r_t o;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = (__bf16)(activation<ACT>(pa[e >> 2][n][e & 3]).v * pb[e >> 2][n][e & 3]);
                        const int64_t r = r0 + 16 * n + a;
                        if (r < p.N && fl + 8 * g < fe)
                            store_unit((__bf16*)p.h + r * F + f0 + fl + 8 * g, o, p.stream);
                    }
                } else {
                    // output m of tile i: channel 32 (i / 2) + 8 (m >> 2) + 4 (i & 1) + (m & 3)
                    const uint32_t q2 = w2 + ((fl * 2) ^ x2);
                    uint32_t q2h = q2 + 0x10000;
                    opaque(q2h);
                    auto read2 = [&](int i, bf16x8r_t (&w)[2]) {
                        const uint32_t at = (32 * (i >> 1) + 4 * (i & 1)) * PITCH * 2;
                        const uint32_t q = (at < 0x10000 ? q2 : q2h) + (at & 0xFFFF);
                        w[0] = read_unit(q);
                        w[1] = read_unit(q + 2 * FS);
                    };
                    // (asked for before the activations)
                    read2(0, wf[0]);
                    read2(1, wf[1]);
                    keep_order();
                    bf16x8r_t da[NT], db[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const Act t = activation<ACT>(pa[e >> 2][n][e & 3]);
                            const float d = (float)dh[n][e];
                            da[n][e] = (__bf16)(d * pb[e >> 2][n][e & 3] * t.d);
                            db[n][e] = (__bf16)(d * t.v);
                        }
                    // two steps at a time: eight products before a sum is needed again
#pragma unroll
                    for (int i = 0; i < STEPS; i += 2) {
                        if (i + 2 < STEPS) {
                            read2(i + 2, wf[(i + 2) % 4]);
                            read2(i + 3, wf[(i + 3) % 4]);
                        }
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int q = i; q < i + 2; ++q)
#pragma unroll
                                for (int n = 0; n < NT; ++n) dx[q][n] = mma(wf[q % 4][s], s ? db[n] : da[n], dx[q][n]);
                        keep_order();
                    }
                }
            }
        }
        if constexpr (DX) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int s = 0; s < KC; ++s) {
                    bf16x8r_t o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = (__bf16)dx[2 * s + (e >> 2)][n][e & 3];
                    const int64_t r = r0 + 16 * n + a;
                    const int c = 32 * s + 8 * g;
                    if (r < p.N && c < C) store_unit((__bf16*)p.dx + r * C + c, o, p.stream);
                }
        }
    }
}

// dw and dbias of one split of the rows and 16 features per wave: 64 rows at a
// time, x shared through LDS, dout (of its own features) per wave.
//
// Here the projections are D = x w: a lane gets four consecutive rows of one
// feature, so da and db, rounded, are the transposed operand of x^T da with
// its reduction (32 rows) numbered 4 g + e (rows of the first 16) and 16 + 4 g
// + e; x is read back transposed in the same order, dout too.
constexpr int kDwWaves = 8;
constexpr int kDwRows = 64;
constexpr int kDwXBytes = kDwRows * 256, kDwDBytes = kDwRows * 32;      // of one buffer; dout: per wave
constexpr int kDwBuffers = 3;
constexpr int kDwLds = kDwBuffers * (kDwXBytes + kDwWaves * kDwDBytes);

// x tile: rows of 256 bytes, 16-byte unit u of row r at u ^ swizzle_row(r):
// conflict-free for 16 rows' unit u and for two units of four consecutive rows
__device__ __forceinline__ int swizzle_row(int r) { return ((r & 7) << 1) | ((r >> 3) & 1); }

template <int KC, int ACT>
__global__ void __launch_bounds__(kDwWaves * 64) k_glu_rows_dw(GluParams p, int slabs, int spread) {
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, a = lane & 15, g = lane >> 4;
    const int C = p.C, F = p.F;
    // the slabs of one split on one XCD (workgroups go round the 8 in turn)
    const int slab = (blockIdx.x >> 3) % slabs;
    const int64_t split = (int64_t)(blockIdx.x >> 3) / slabs * 8 + (blockIdx.x & 7);
    const int64_t k0 = split * p.rows_per_split, k1 = min(p.N, k0 + p.rows_per_split);
    if (k0 >= p.N) return;
    const int f = (slab * spread + wave) * 16;         // this wave's first feature
    const bool works = wave < spread && f < F;         // else it only helps to load x
    const __bf16* w = (const __bf16*)p.w;

    // weights as operands: feature f + a, channels 32 s + 8 g ..
    bf16x8r_t wt[2][KC];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = 32 * k + 8 * g + e;
                const bool in = c < C && f + a < F;
                const __bf16 v = w[in ? ((int64_t)s * C + c) * F + f + a : 0];
                wt[s][k][e] = in ? v : (__bf16)0.f;
            }
    const float ba = p.bias && f + a < F ? p.bias[f + a] : 0.f, bb = p.bias && f + a < F ? p.bias[F + f + a] : 0.f;

    // Byte offsets in LDS, to which buffer, half and tile add constants.  Unit
    // 4 s + g of row a; pieces of four channels of rows 4 g + (a >> 2).
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_bf16x4r_t*)smem;
    uint32_t xa[KC], xt[2 * KC];
#pragma unroll
    for (int s = 0; s < KC; ++s) xa[s] = lds0 + a * 256 + ((4 * s + g) ^ swizzle_row(a)) * 16;
    const int rt = 4 * g + (a >> 2);
#pragma unroll
    for (int i = 0; i < 2 * KC; ++i)
        xt[i] = lds0 + rt * 256 + ((2 * i + ((a & 3) >> 1)) ^ swizzle_row(rt)) * 16 + 8 * (a & 1);
    const uint32_t d0 = lds0 + kDwBuffers * kDwXBytes + wave * kDwBuffers * kDwDBytes;
    const uint32_t dt = d0 + rt * 32 + 8 * (a & 3);

    // x's 64 rows: units of KC * 32 channels, PER of them per thread (half of
    // the threads' for 32 channels); dout's: 16 units of the slab's features,
    // two per thread, a wave's two features' units side by side in LDS
    constexpr int UNITS = KC * 4, PER = (kDwRows * UNITS + kDwWaves * 64 - 1) / (kDwWaves * 64);
    constexpr int RSTEP = kDwWaves * 64 / UNITS;       // rows from unit to unit of a thread
    const int xr = threadIdx.x / UNITS, xu = threadIdx.x % UNITS;
    const bool loads = xr < kDwRows && 8 * xu < C;
    const int dr = threadIdx.x >> 4, du = threadIdx.x & 15, df = slab * spread * 16 + 8 * du;
    bf16x8r_t rx[PER], rd[2];
    uint32_t ox[PER], od[2];                           // bytes from the block's first row
#pragma unroll
    for (int j = 0; j < PER; ++j) ox[j] = loads ? ((xr + RSTEP * j) * C + 8 * xu) * 2 : kOutside;
#pragma unroll
    for (int j = 0; j < 2; ++j) od[j] = df < F ? ((dr + 32 * j) * F + df) * 2 : kOutside;
    // (rows past the split read as zeros)
    auto fetch = [&](int64_t k) {
        const int rows = (int)max((int64_t)0, min((int64_t)kDwRows, k1 - k));
        const RowBuffer bx((const __bf16*)p.x + k * C, rows * C), bd((const __bf16*)p.dout + k * F, rows * F);
#pragma unroll
        for (int j = 0; j < PER; ++j) rx[j] = bx.load8(ox[j]);
#pragma unroll
        for (int j = 0; j < 2; ++j) rd[j] = bd.load8(od[j]);
    };
    // Channels past C were cleared once and are never written; features past F
    // are zero.
    const uint32_t px = lds0 + xr * 256 + (xu ^ swizzle_row(xr)) * 16;
    const uint32_t pd = lds0 + kDwBuffers * kDwXBytes + (du >> 1) * kDwBuffers * kDwDBytes + dr * 32 + (du & 1) * 16;
    auto put = [&](auto buffer) {
        constexpr uint32_t B = decltype(buffer)::value;
        if (loads) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                *(lds_bf16x8r_t*)(uintptr_t)(px + B * kDwXBytes + j * RSTEP * 256) = rx[j];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) *(lds_bf16x8r_t*)(uintptr_t)(pd + B * kDwDBytes + j * 1024) = rd[j];
    };
    f32x4r_t dw[2][2 * KC];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2 * KC; ++i) dw[s][i] = f32x4r_t{0.f, 0.f, 0.f, 0.f};
    // Three things of 32 rows each are under way at once: the projections of
    // the next rows, the activations of these, the products of the last ones
    // with x.  They need nothing of each other, so that a wave's matrix
    // instructions run in the shadow of its activations.
    float sa = 0.f, sb = 0.f;
    f32x4r_t va[2] = {}, vb[2] = {};      // projections, by tile of 16 rows
    bf16x4r_t dh[2] = {};                 // dout of their rows
    bf16x8r_t fa = {}, fb = {};           // da and db of the rows before
    // Both halves of the block in buffer B are projected; what is left of the
    // block before, in buffer P, is finished.
    auto block = [&](auto cur, auto prev) {
        constexpr uint32_t B = decltype(cur)::value, P = decltype(prev)::value;
        if (!works) return;
        constexpr int STEPS = 2 * KC, EACH = 8 / STEPS, AHEAD = 3;
        float ua = 0.f, ub = 0.f;         // this block's sums first: short chains
        // operands of step i: unit s = i / 2 % KC of tile i % 2 of half i / STEPS;
        // channels i % STEPS of the half, transposed
        bf16x8r_t xf[AHEAD], xc[AHEAD];
        auto ask = [&](int i) {
            const int hf = i / STEPS, q = i % STEPS;
            xf[i % AHEAD] = read_unit(xa[q >> 1] + B * kDwXBytes + (32 * hf + 16 * (q & 1)) * 256);
            const uint32_t t = xt[q] + P * kDwXBytes + 32 * hf * 256;
            xc[i % AHEAD] = join8(read_tr(t), read_tr(t + 16 * 256));
        };
#pragma unroll
        for (int i = 0; i < AHEAD - 1; ++i) ask(i);
#pragma unroll
        for (int hf = 0; hf < kDwRows / 32; ++hf) {
            bf16x4r_t dn[2], da[2], db[2];
            f32x4r_t na[2], nb[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                dn[t] = read_tr(dt + B * kDwDBytes + (32 * hf + 16 * t) * 32);
                na[t] = f32x4r_t{ba, ba, ba, ba};
                nb[t] = f32x4r_t{bb, bb, bb, bb};
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int i = hf * STEPS + c / EACH, q = i % STEPS;
                if (c % EACH == 0) {
                    if (i + AHEAD - 1 < 2 * STEPS) ask(i + AHEAD - 1);
                    const bf16x8r_t x1 = xf[i % AHEAD], x0 = xc[i % AHEAD];
                    na[q & 1] = mma(x1, wt[0][q >> 1], na[q & 1]);
                    nb[q & 1] = mma(x1, wt[1][q >> 1], nb[q & 1]);
                    dw[0][q] = mma(fa, x0, dw[0][q]);
                    dw[1][q] = mma(fb, x0, dw[1][q]);
                }
                const int t = c / 4, e = c % 4;
                const Act act = activation<ACT>(va[t][e]);
                const float d = (float)dh[t][e];
                const float u = d * vb[t][e] * act.d, v = d * act.v;
                ua += u;
                ub += v;
                da[t][e] = (__bf16)u;
                db[t][e] = (__bf16)v;
                interleave();
            }
            fa = join8(da[0], da[1]);
            fb = join8(db[0], db[1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                va[t] = na[t];
                vb[t] = nb[t];
                dh[t] = dn[t];
            }
        }
        sa += ua;
        sb += ub;
    };
    for (int e = threadIdx.x; e < kDwBuffers * kDwXBytes / 16; e += kDwWaves * 64)
        *(bf16x8r_t*)(smem + 16 * e) = bf16x8r_t{};
    constexpr std::integral_constant<uint32_t, 0> b0{};
    constexpr std::integral_constant<uint32_t, 1> b1{};
    constexpr std::integral_constant<uint32_t, 2> b2{};
    fetch(k0);
    __syncthreads();
    put(b0);
    // One block past the last row (zeros) finishes the last.  A block is written
    // where the one before the last was: no wave reads that any more.
    const int64_t ke = k1 + kDwRows;
    for (int64_t k = k0;;) {
        auto one = [&](auto cur, auto prev, auto next) {
            fetch(k + kDwRows);
            __syncthreads();
            block(cur, prev);
            put(next);
            k += kDwRows;
            return k < ke;
        };
        if (!one(b0, b2, b1)) break;
        if (!one(b1, b0, b2)) break;
        if (!one(b2, b1, b0)) break;
    }
    if (!works) return;
    // output m = 4 g + e: feature f + m; channel 16 i + a
    float* part = p.wpart + split * C * 2 * F;
#pragma unroll
    for (int i = 0; i < 2 * KC; ++i) {
        const int c = 16 * i + a;
        if (c >= C || f + 4 * g >= F) continue;
        *(f32x4r_t*)(part + (int64_t)c * 2 * F + f + 4 * g) = dw[0][i];
        *(f32x4r_t*)(part + (int64_t)c * 2 * F + F + f + 4 * g) = dw[1][i];
    }
    if (p.bpart) {
        // the four row groups of a feature
        sa += __shfl_xor(sa, 16);
        sb += __shfl_xor(sb, 16);
        sa += __shfl_xor(sa, 32);
        sb += __shfl_xor(sb, 32);
        if (g == 0 && f + a < F) {
            p.bpart[split * 2 * F + f + a] = sa;
            p.bpart[(split * 2 + 1) * F + f + a] = sb;
        }
    }
}

// The features in slabs of at most 8 waves' worth, as even as they go, and the
// splits of the rows that fill the card.
struct DwShape {
    int spread, slabs, splits;
};
DwShape dw_shape(int64_t N, int C, int F) {
    DwShape s;
    const int tiles = (F + 15) / 16;
    s.slabs = (tiles + kDwWaves - 1) / kDwWaves;
    s.spread = (tiles + s.slabs - 1) / s.slabs;
    const int64_t groups = kCUs;      // one workgroup per CU
    s.splits = (int)std::max<int64_t>(1, std::min<int64_t>(groups / s.slabs, (N + kDwRows - 1) / kDwRows));
    return s;
}

template <int KC, int ACT>
hipError_t rows_go(const GluParams& p, int what, int splits, hipStream_t st) {
    if (what == 2) {
        const DwShape s = dw_shape(p.N, p.C, p.F);
        const hipError_t e = hipFuncSetAttribute((const void*)k_glu_rows_dw<KC, ACT>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kDwLds);
        if (e != hipSuccess) return e;
        k_glu_rows_dw<KC, ACT><<<(unsigned)((splits + 7) / 8 * 8 * s.slabs), kDwWaves * 64, kDwLds, st>>>(p, s.slabs,
                                                                                                         s.spread);
        return hipGetLastError();
    }
    const size_t lds = (size_t)kSlabElems * 2 + (size_t)2 * kSlab<KC> * 4 + 16;
    const unsigned grid = (unsigned)std::min<int64_t>((p.N + kBlockRows - 1) / kBlockRows, kCUs);
    const auto fn = what ? k_glu_rows<KC, ACT, true> : k_glu_rows<KC, ACT, false>;
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    fn<<<grid, kRowThreads, lds, st>>>(p);
    return hipGetLastError();
}

template <int ACT>
hipError_t rows_dispatch(const GluParams& p, int what, int splits, hipStream_t st) {
    if (p.C <= 32) return rows_go<1, ACT>(p, what, splits, st);
    if (p.C <= 64) return rows_go<2, ACT>(p, what, splits, st);
    return rows_go<4, ACT>(p, what, splits, st);
}
hipError_t rows_act(const GluParams& p, int act, int what, int splits, hipStream_t st) {
    return act == SPCONV_SILU ? rows_dispatch<SPCONV_SILU>(p, what, splits, st)
                              : rows_dispatch<SPCONV_GELU>(p, what, splits, st);
}

}  // namespace

hipError_t launch_glu_rows(const GluParams& p, int act, hipStream_t st) { return rows_act(p, act, 0, 0, st); }
hipError_t launch_glu_rows_dx(const GluParams& p, int act, hipStream_t st) { return rows_act(p, act, 1, 0, st); }
int glu_rows_splits(int64_t N, int C, int F) { return dw_shape(N, C, F).splits; }
hipError_t launch_glu_rows_dw(const GluParams& p, int act, int splits, hipStream_t st) {
    return rows_act(p, act, 2, splits, st);
}

}  // namespace spc
