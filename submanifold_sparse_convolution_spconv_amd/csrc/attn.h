// Shared by the attention kernels: arguments, matrix instructions of 32 x 32,
// tiles of rows in LDS, and the place of a workgroup among packed sequences.
//
// A sequence's queries of one key head are rows r = (position, head of the
// group), R = Lq G of them: heads that share keys stand next to each other, so
// that a prompt's tile and a single token's are the same thing, keys are read
// once for all of them, and the keys' gradients add over the group by
// themselves.
#pragma once

#include "places.h"

namespace spc {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4a_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4a_t lds_bf16x4a_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

struct AttnParams {
    const uint8_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const int32_t* offsets;
    const int32_t* koffsets;
    const int32_t* order;       // or NULL
    const int32_t* korder;      // or NULL
    uint8_t* out;               // forward: out; gradient: the forward's output, read
    float* lse;                 // (N, H) or NULL
    const uint8_t* dout;
    uint8_t* dq;
    uint8_t* dk;
    uint8_t* dv;
    float* delta;               // (N, H)
    float* part;                // splits: partial sums
    int64_t qs[2], ks[2], vs[2], os[2], dos[2], dqs[2], dks[2], dvs[2];   // row and head strides, bytes
    int64_t N, M;
    int64_t items;              // places of tiles, at most (see Place)
    int H, HK, G, D, B;
    uint32_t magic;             // of a division by G
    int causal;
    int near;                   // 1: rows are below 2 GiB from their tensor's start
    int splits;                 // of the long axis over workgroups
    float scale, scale2;        // of the scores; the same times log2 e, rounded
    float per_lse, per_lse_rest; // scale2 / scale: lse in powers of two
};

AttnParams attn_params(const AttnArgs& a);
// Few queries (attn_few.hip): rows of a workgroup.
constexpr int kFewRows = 16;
hipError_t launch_attn_few(const AttnParams& p, int dtype, hipStream_t st);
// A query's sum from which its reference is taken again (see attn.hip).
constexpr float kAttnMost = 0x1p64f;

__device__ __forceinline__ f32x16_t mfma32(bf16x8r_t a, bf16x8r_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(float a, float b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t zero16() {
    f32x16_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}
// Value i of a lane's 16 in a 32 x 32 result: its row, for lane half h; the
// column is lane & 31.
__device__ __forceinline__ int row16(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// The other half's value (lanes l and l ^ 32).
__device__ __forceinline__ float half_max(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// r / G for r < 2^31: off by one at most before the correction.
struct RowHead {
    int pos, head;
};
__device__ __forceinline__ RowHead split_row(uint32_t r, int G, uint32_t magic) {
    if (G == 1) return {(int)r, 0};
    uint32_t q = __umulhi(r, magic);
    int m = (int)(r - q * (uint32_t)G);
    if (m < 0) {
        --q;
        m += G;
    }
    return {(int)q, m};
}

// A sequence's keys, where they are not the queries' rows.
__device__ __forceinline__ void find_keys(const AttnParams& p, Place& pl) {
    pl.k0 = pl.q0;
    pl.Lk = pl.Lq;
    if (p.koffsets) {
        pl.k0 = clamp_to(p.koffsets[pl.b], 0, p.M);
        pl.Lk = (int)(clamp_to(p.koffsets[pl.b + 1], pl.k0, p.M) - pl.k0);
    }
}

// A wave's COLS query rows, one per column, and the keys they see: each its own
// first `limit`, at most `most` in the wave, and `least` to `longest` over the
// workgroup.  Columns past the sequence repeat its last row.
template <int COLS = 32>
struct QueryRows {
    Place pl;
    int pos, head, limit, least, most, longest;
    uint32_t row;
    bool valid;
    // wave_row: the wave's first row in the tile of tq
    __device__ __forceinline__ bool find(const AttnParams& p, int tq, int wave_row, int hk, int64_t item) {
        pl = find_place(p.offsets, p.B, p.N, p.G, tq, item);
        if (pl.tile < 0) return false;
        find_keys(p, pl);
        const int R = pl.Lq * p.G;
        // a causal sequence's long tiles first
        const int tile = p.causal ? (R - 1) / tq - pl.tile : pl.tile;
        const int first = tile * tq + wave_row, mine = first + (threadIdx.x & (COLS - 1));
        const int past = pl.Lk - pl.Lq + 1;
        const auto sees = [&](int pos) { return p.causal ? min(max(pos + past, 0), pl.Lk) : pl.Lk; };
        const auto pos_of = [&](int r) { return split_row(min(r, R - 1), p.G, p.magic).pos; };
        const RowHead rh = split_row(min(mine, R - 1), p.G, p.magic);
        valid = mine < R;
        pos = rh.pos;
        head = hk * p.G + rh.head;
        row = row_of(p.order, pl.q0 + rh.pos, p.N);
        limit = sees(rh.pos);
        least = sees(pos_of(tile * tq));
        most = first < R ? sees(pos_of(first + COLS - 1)) : 0;
        longest = sees(pos_of(tile * tq + tq - 1));
        return true;
    }
    __device__ __forceinline__ const uint8_t* at(const uint8_t* t, const int64_t (&s)[2]) const {
        return t + row * s[0] + head * s[1];
    }
    __device__ __forceinline__ uint8_t* at(uint8_t* t, const int64_t (&s)[2]) const {
        return t + row * s[0] + head * s[1];
    }
};

// Runs of kRun consecutive places stand on one XCD (a block's XCD is its number
// modulo 8): tiles of one sequence share its L2.
constexpr int kXcds = 8, kRun = 8;
__device__ __forceinline__ int64_t xcd_order(int64_t id) {
    const int64_t xcd = id % kXcds, slot = id / kXcds;
    return (slot / kRun * kXcds + xcd) * kRun + slot % kRun;
}
inline int64_t xcd_blocks(int64_t n) { return (n + kXcds * kRun - 1) / (kXcds * kRun) * (kXcds * kRun); }
// Whether a launch of n places, of 256 threads at most each, stays within the 2^32
// that a launch's threads are counted in.
inline bool attn_threads_fit(int64_t n) { return xcd_blocks(n) * 256 < (1ll << 32); }

// A tile of rows of DP elements in LDS, in 16-byte units.  Units of a row are
// permuted so that both ways of reading are free of bank conflicts (banks repeat
// after 256 bytes, which 16 lanes' units or 32 lanes' half units fill): 16
// consecutive rows' unit u (the operand along the row) lie on 16 different
// units of the banks, and so do the four units side by side of four
// consecutive rows (the transposing read).
template <typename T, int DP>
struct Tile {
    static constexpr int E = 16 / sizeof(T);        // elements per unit
    static constexpr int U = DP / E;                // units per row
    static constexpr int ROWB = DP * (int)sizeof(T);
    static constexpr bool WIDE = U % 8 == 0;        // a row is whole halves of the banks
    static __device__ __forceinline__ int key(int row) {
        if constexpr (WIDE)
            return (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1);
        else
            return (row >> 2) & 3;
    }
    static __device__ __forceinline__ int at(int row, int unit) { return row * ROWB + ((unit ^ key(row)) << 4); }
};

typedef uint32_t u32x4a_t __attribute__((ext_vector_type(4)));

// Rows into a tile by THR threads: each fetches 16-byte units into registers
// while the tile before is worked on, and stores them to consecutive LDS
// addresses; which unit of which row it fetches carries the permutation.
// (Loads past the registers were slower: the compiler has the transposing reads
// wait for all of them.)
constexpr uint32_t kNoUnit = 0x80000000u;      // an offset past every buffer: zeros are read
template <typename T, int DP, int ROWS, int THR>
struct Stager {
    using L = Tile<T, DP>;
    static constexpr int NP = ROWS * L::U / THR;
    static_assert(ROWS * L::U % THR == 0 && THR % 64 == 0);
    static __device__ __forceinline__ int row(int i, int t) { return (i * THR + t) / L::U; }
    // the byte in its row of thread t's unit i
    static __device__ __forceinline__ int byte(int i, int t) {
        const int p = i * THR + t;
        return ((p % L::U) ^ L::key(p / L::U)) * 16;
    }
    static __device__ __forceinline__ void store(const u32x4a_t (&r)[NP], lds_u8* tile, int t) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            *(__attribute__((address_space(3))) u32x4a_t*)(tile + (i * THR + t) * 16) = r[i];
    }
};
__device__ __forceinline__ u32x4a_t fetch16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4a_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
}
__device__ __forceinline__ u32x4a_t fetch16(const uint8_t* p, bool in) {
    u32x4a_t r = {};
    if (in) r = *(const u32x4a_t*)p;
    return r;
}

// Keys' and values' rows of a sequence into tiles.  Rows one after the other
// are a buffer whose start moves with the tile, so that a unit's offset stays
// the same; through korder each row's place is looked up one tile before it
// is fetched (in one buffer, where the tensors are below 2 GiB).  Rows past the
// sequence, zeros or its last one again, are hidden from every query.
template <typename T, int DP, int KT, int THR>
struct KeyStager {
    using St = Stager<T, DP, KT, THR>;
    static constexpr int NP = St::NP;
    const AttnParams& p;
    const uint8_t *k, *v;
    int64_t k0;
    int Lk, t;
    uint32_t ok[NP], ov[NP];
    int row[NP];
    u32x4a_t rk[NP], rv[NP];
    __device__ __forceinline__ KeyStager(const AttnParams& p, const Place& pl, int hk, int t)
        : p(p), k(p.k + hk * p.ks[1]), v(p.v + hk * p.vs[1]), k0(pl.k0), Lk(pl.Lk), t(t) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int by = St::byte(i, t);
            const bool in = by < p.D * (int)sizeof(T);
            ok[i] = !in ? kNoUnit : p.korder ? by : by + St::row(i, t) * (uint32_t)p.ks[0];
            ov[i] = !in ? kNoUnit : p.korder ? by : by + St::row(i, t) * (uint32_t)p.vs[0];
        }
    }
    __device__ __forceinline__ void look_up(int tile) {
        if (!p.korder) return;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            row[i] = p.korder[k0 + min(tile * KT + St::row(i, t), Lk - 1)];
        }
    }
    __device__ __forceinline__ void fetch(int tile) {
        if (p.korder) {
            const auto bk = rows_at(k), bv = rows_at(v);
            const uint32_t last = (uint32_t)p.M - 1;
            if (p.near) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const uint32_t r = min((uint32_t)row[i], last);
                    rk[i] = fetch16(bk, r * (uint32_t)p.ks[0] + ok[i]);
                    rv[i] = fetch16(bv, r * (uint32_t)p.vs[0] + ov[i]);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const uint32_t r = min((uint32_t)row[i], last);
                // (kept from being worked out ahead for all units: registers)
                uint32_t by = ok[i];
                asm volatile("" : "+v"(by));
                rk[i] = fetch16(k + r * p.ks[0] + by, by != kNoUnit);
                rv[i] = fetch16(v + r * p.vs[0] + by, by != kNoUnit);
            }
            return;
        }
        const int64_t at = k0 + (int64_t)tile * KT;
        const auto bk = rows_at(k + at * p.ks[0]), bv = rows_at(v + at * p.vs[0]);
        const int left = Lk - tile * KT;
        if (left >= KT) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                rk[i] = fetch16(bk, ok[i]);
                rv[i] = fetch16(bv, ov[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                rk[i] = fetch16(bk, St::row(i, t) < left ? ok[i] : kNoUnit);
                rv[i] = fetch16(bv, St::row(i, t) < left ? ov[i] : kNoUnit);
            }
        }
    }
    __device__ __forceinline__ void store(lds_u8* kt) const {
        St::store(rk, kt, t);
        St::store(rv, kt + KT * St::L::ROWB, t);
    }
};

// Operands of a matrix instruction from a tile of rows.
// along(row0, c): rows row0 .. row0 + 31 (lane & 31), elements 16 c .. (bf16)
//   or 8 c .. (fp32, four instructions), lane half h its eight / four.
// across(row0, c, d0): the transpose: elements d0 .. d0 + 31 (lane & 31) of the
//   16 (bf16) or 2 (fp32) rows of a 32 x 32 result's values 8 c .. / c that the
//   lane's half holds (row16): such a result is the other operand as it is.
template <typename T, int DP>
struct Operand;

template <int DP>
struct Operand<__bf16, DP> {
    using L = Tile<__bf16, DP>;
    static constexpr int STEPS = DP / 16;     // instructions along a row
    static constexpr int CROSS = 2;           // instructions for 32 rows
    typedef bf16x8r_t frag;
    static __device__ __forceinline__ frag along(const lds_u8* tile, int row0, int s) {
        const int l = threadIdx.x & 63;
        return *(const __attribute__((address_space(3))) bf16x8r_t*)(tile + row0 * L::ROWB +
                                                                     L::at(l & 31, 2 * s + (l >> 5)));
    }
    static __device__ __forceinline__ frag across(const lds_u8* tile, int row0, int c, int dt) {
        const int l = threadIdx.x & 63, a = l & 15, h = l >> 5;
        const int row = 4 * h + (a >> 2);
        const int unit = 4 * dt + 2 * ((l >> 4) & 1) + ((a & 3) >> 1);
        const lds_u8* p = tile + (row0 + 16 * c) * L::ROWB + 8 * (a & 1);
        const bf16x4a_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)(p + L::at(row, unit)));
        const bf16x4a_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)(p + L::at(row + 8, unit)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // the lane's operand for column row `src` (elements 16 s + 8 h ..)
    static __device__ __forceinline__ frag row(const uint8_t* src, int s, int D) {
        const int d = 16 * s + 8 * ((threadIdx.x >> 5) & 1);
        frag f = {};
        if (d < D) f = *(const frag*)(src + 2 * d);
        return f;
    }
    // whether step s has elements of D (fp32: its four instructions are 256 cycles)
    static __device__ __forceinline__ bool wanted(int, int) { return true; }
    // values 8 c .. 8 c + 7 of a result as an operand, rounded
    static __device__ __forceinline__ frag pack(const f32x16_t& p, int c) {
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)p[8 * c + j];
        return f;
    }
    // what that rounding left out, as an operand
    static __device__ __forceinline__ frag pack_rest(const f32x16_t& p, frag b, int c) {
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)(p[8 * c + j] - (float)b[j]);
        return f;
    }
    static __device__ __forceinline__ f32x16_t mma(frag a, frag b, f32x16_t c) { return mfma32(a, b, c); }
    // the rows that the lane's element j of instruction c stands for
    static constexpr int ROWS = 8;
    static __device__ __forceinline__ int index(int c, int j) { return 8 * c + j; }
    // the infinite and NaN elements, the others 0
    static __device__ __forceinline__ frag bad(frag f) {
        u32x4a_t w = __builtin_bit_cast(u32x4a_t, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t top = ((w[j] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;    // exponents of ones
            w[j] &= (top >> 15) * 0xFFFFu;
        }
        return __builtin_bit_cast(frag, w);
    }
    static __device__ __forceinline__ bool any(frag f) {
        const u32x4a_t w = __builtin_bit_cast(u32x4a_t, f);
        return w[0] | w[1] | w[2] | w[3];
    }
    static __device__ __forceinline__ frag without(frag f, frag g) {       // g: some of f's elements
        return __builtin_bit_cast(frag, __builtin_bit_cast(u32x4a_t, f) ^ __builtin_bit_cast(u32x4a_t, g));
    }
    // element j where `mine`, else 0
    static __device__ __forceinline__ frag only(frag f, int j, bool mine) {
        u32x4a_t w = __builtin_bit_cast(u32x4a_t, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = mine && e == (j >> 1) ? w[e] & (0xFFFFu << (16 * (j & 1))) : 0u;
        return __builtin_bit_cast(frag, w);
    }
};

template <int DP>
struct Operand<float, DP> {
    using L = Tile<float, DP>;
    static constexpr int STEPS = DP / 8;
    static constexpr int CROSS = 16;
    typedef f32x4r_t frag4;
    typedef float frag;
    static __device__ __forceinline__ frag4 along(const lds_u8* tile, int row0, int s) {
        const int l = threadIdx.x & 63;
        return *(const __attribute__((address_space(3))) f32x4r_t*)(tile + row0 * L::ROWB +
                                                                    L::at(l & 31, 2 * s + (l >> 5)));
    }
    static __device__ __forceinline__ frag across(const lds_u8* tile, int row0, int c, int dt) {
        const int l = threadIdx.x & 63;
        const int row = row16(c, l >> 5);
        return *(const __attribute__((address_space(3))) float*)(tile + row0 * L::ROWB +
                                                                 L::at(row, 8 * dt + ((l & 31) >> 2)) + 4 * (l & 3));
    }
    static __device__ __forceinline__ frag4 row(const uint8_t* src, int s, int D) {
        const int d = 8 * s + 4 * ((threadIdx.x >> 5) & 1);
        frag4 f = {};
        if (d < D) f = *(const frag4*)(src + 4 * d);
        return f;
    }
    static __device__ __forceinline__ bool wanted(int s, int D) { return 8 * s < D; }
    static __device__ __forceinline__ frag pack(const f32x16_t& p, int c) { return p[c]; }
    static __device__ __forceinline__ f32x16_t mma(frag4 a, frag4 b, f32x16_t c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = mfma32(a[j], b[j], c);
        return c;
    }
    static __device__ __forceinline__ f32x16_t mma(frag a, frag b, f32x16_t c) { return mfma32(a, b, c); }
    static constexpr int ROWS = 1;
    static __device__ __forceinline__ int index(int c, int) { return c; }
    static __device__ __forceinline__ frag bad(frag f) {
        return (__float_as_uint(f) & 0x7F800000u) == 0x7F800000u ? f : 0.f;
    }
    static __device__ __forceinline__ bool any(frag f) { return __float_as_uint(f) != 0; }
    static __device__ __forceinline__ frag without(frag f, frag g) {
        return __uint_as_float(__float_as_uint(f) ^ __float_as_uint(g));
    }
    static __device__ __forceinline__ frag only(frag f, int, bool mine) { return mine ? f : 0.f; }
};
template <typename T>
__device__ __forceinline__ void store_four(uint8_t* p, f32x4r_t v, float f) {
    typedef T vec __attribute__((ext_vector_type(4)));
    vec o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (T)(v[j] * f);
    *(vec*)p = o;
}
// a row's operand has the type of along()
template <typename T, int DP>
using RowFrag = decltype(Operand<T, DP>::row((const uint8_t*)nullptr, 0, 0));

// acc[dt] += (rows' transpose) x w for 32 rows of a tile, w a 32 x 32 result
// whose hidden entries (bit i of `seen` clear) are zero.  A zero times an infinite
// or NaN element of the tile would still be NaN, so masked tiles multiply the
// others only, and where there are some, these are added row by row, to the
// columns that see the row.  FINE (bf16): w in two parts, rounded and rest.
template <typename T, int DP, bool MASKED, bool FINE = false>
__device__ __forceinline__ void add_rows(f32x16_t (&acc)[DP / 32], const lds_u8* tile, int row0, const f32x16_t& w,
                                         uint32_t seen) {
    using O = Operand<T, DP>;
    bool some = false;
#pragma unroll
    for (int c = 0; c < O::CROSS; ++c) {
        const auto b = O::pack(w, c);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) {
            auto a = O::across(tile, row0, c, dt);
            if constexpr (MASKED) {
                const auto x = O::bad(a);
                some |= O::any(x);
                a = O::without(a, x);
            }
            acc[dt] = O::mma(a, b, acc[dt]);
            if constexpr (FINE) acc[dt] = O::mma(a, O::pack_rest(w, b, c), acc[dt]);
        }
    }
    if (MASKED && __builtin_expect(__ballot(some) != 0, 0)) {
        const int h = (threadIdx.x >> 5) & 1;
        // a column's two lane halves see different rows: ask the half that holds it
        const uint32_t other = (uint32_t)__shfl_xor((int)seen, 32);
#pragma unroll
        for (int c = 0; c < O::CROSS; ++c) {
            const auto b = O::pack(w, c);
#pragma unroll 1
            for (int j = 0; j < 2 * O::ROWS; ++j) {
                const int half = j & 1, e = j >> 1;
                const bool see = ((h == half ? seen : other) >> O::index(c, e)) & 1;
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) {
                    const auto x = O::only(O::bad(O::across(tile, row0, c, dt)), e, h == half);
                    const f32x16_t t = O::mma(x, O::only(b, e, h == half), zero16());
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[dt][i] += see ? t[i] : 0.f;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
}

// The lane's 16 values of column `lane & 31` of block dt into a row of outputs.
template <typename T>
__device__ __forceinline__ void store_col(uint8_t* row, const f32x16_t& v, float f, int dt, int D) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = 32 * dt + 8 * i + 4 * h;
        if (d < D) {
            store_four<T>(row + d * (int)sizeof(T), f32x4r_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}, f);
        }
    }
}

// Everything loaded so far has arrived: said before a loop, so that the loop does
// not wait for it (and with it for its own loads) every time.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Between the tiles: the workgroup's waves together, or, where a wave has tiles of
// its own, its own LDS operations (which the hardware keeps in order).
template <bool OWN>
__device__ __forceinline__ void next_tile() {
    if constexpr (OWN)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    else
        __syncthreads();
}

}  // namespace spc
