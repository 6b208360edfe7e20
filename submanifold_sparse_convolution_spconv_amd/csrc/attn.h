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
    int splits;                 // of the long axis over workgroups
    float scale, scale2;        // of the scores; the same times log2 e
};

// What a call's sizes choose: the waves' share (KS, see attn.hip) and the parts
// that the keys (or, in the keys' gradient, the queries) are split into.
struct AttnPlan {
    bool ks;
    int splits;
};
AttnPlan attn_plan(const AttnArgs& a);
AttnParams attn_params(const AttnArgs& a);

// 16 zero bytes: where lanes without a row load from.
static __device__ const uint32_t kAttnZeros[4] = {0, 0, 0, 0};

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

// A wave's 32 query rows, one per lane (both halves), and the keys they see:
// the lane's own first `limit`, and over the wave's and the workgroup's rows.
// Lanes past the sequence repeat its last row.
struct QueryRows {
    Place pl;
    RowHead rh;
    int64_t row;
    int head, limit, least, most, longest;
    bool valid;
    // wave_row: the wave's first row in the tile of tq
    __device__ __forceinline__ bool find(const AttnParams& p, int tq, int wave_row, int hk, int64_t item) {
        pl = find_place(p.offsets, p.B, p.N, p.G, tq, item);
        if (pl.tile < 0) return false;
        find_keys(p, pl);
        const int R = pl.Lq * p.G;
        // a causal sequence's long tiles first
        const int tile = p.causal ? (R - 1) / tq - pl.tile : pl.tile;
        const int first = tile * tq + wave_row, mine = first + (threadIdx.x & 31);
        const int past = pl.Lk - pl.Lq + 1;
        const auto sees = [&](int r) {
            const int pos = split_row(min(r, R - 1), p.G, p.magic).pos;
            return p.causal ? min(max(pos + past, 0), pl.Lk) : pl.Lk;
        };
        valid = mine < R;
        rh = split_row(min(mine, R - 1), p.G, p.magic);
        head = hk * p.G + rh.head;
        row = row_of(p.order, pl.q0 + rh.pos, p.N);
        limit = sees(mine);
        least = sees(first);
        most = first < R ? sees(first + 31) : 0;
        longest = sees(tile * tq + tq - 1);
        return true;
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

// A tile of ROWS rows of DP elements in LDS, in 16-byte units.  Units of a row
// are permuted so that both ways of reading are free of bank conflicts: eight
// consecutive rows' unit u (the operand along the row) lie on eight different
// bank groups, and so do the unit pairs of four consecutive rows (the
// transposing read).
template <typename T, int DP>
struct Tile {
    static constexpr int E = 16 / sizeof(T);        // elements per unit
    static constexpr int U = DP / E;                // units per row
    static constexpr int ROWB = DP * (int)sizeof(T);
    static constexpr bool WIDE = U % 8 == 0;        // a row is whole turns of the banks
    static __device__ __forceinline__ int key(int row) {
        if constexpr (WIDE)
            return ((row & 3) << 1) | ((row >> 2) & 1);
        else
            return (((row >> 1) & 1) << 1) | ((row >> 2) & 1);
    }
    static __device__ __forceinline__ int at(int row, int unit) { return row * ROWB + ((unit ^ key(row)) << 4); }
};

// Rows into a tile, by THR threads, past the registers.  A lane's unit goes to
// consecutive LDS addresses; which unit of which row it fetches carries the
// permutation.
template <typename T, int DP, int ROWS, int THR>
struct Stager {
    using L = Tile<T, DP>;
    static constexpr int NP = ROWS * L::U / THR;
    static_assert(ROWS * L::U % THR == 0 && THR % 64 == 0);
    static __device__ __forceinline__ int row(int i, int t) { return (i * THR + t) / L::U; }
    // the byte in its row of thread t's unit i, or -1 past D
    static __device__ __forceinline__ int byte(int i, int t, int D) {
        const int p = i * THR + t;
        const int u = (p % L::U) ^ L::key(p / L::U);
        return u * L::E < D ? u * 16 : -1;
    }
    static __device__ __forceinline__ void load(const uint8_t* src, lds_u8* tile, int i, int t) {
        __builtin_amdgcn_global_load_lds(src, tile + (i * THR + (t & ~63)) * 16, 16, 0, 0);
    }
};

// Keys' and values' rows of a sequence into tiles, ahead of their use: the rows'
// places are looked up (through korder) one tile before they are loaded.
template <typename T, int DP, int KT, int THR>
struct KeyStager {
    using St = Stager<T, DP, KT, THR>;
    const AttnParams& p;
    const Place& pl;
    const uint8_t *k, *v;
    int t;
    int64_t row[St::NP];
    __device__ __forceinline__ KeyStager(const AttnParams& p, const Place& pl, int hk, int t)
        : p(p), pl(pl), k(p.k + hk * p.ks[1]), v(p.v + hk * p.vs[1]), t(t) {}
    __device__ __forceinline__ void look_up(int tile) {
#pragma unroll
        for (int i = 0; i < St::NP; ++i) {
            const int j = tile * KT + St::row(i, t);
            row[i] = j < pl.Lk ? row_of(p.korder, pl.k0 + j, p.M) : -1;
        }
    }
    __device__ __forceinline__ void load(lds_u8* kt, lds_u8* vt) const {
#pragma unroll
        for (int i = 0; i < St::NP; ++i) {
            const int by = St::byte(i, t, p.D);
            const bool in = row[i] >= 0 && by >= 0;
            St::load(in ? k + row[i] * p.ks[0] + by : (const uint8_t*)kAttnZeros, kt, i, t);
            St::load(in ? v + row[i] * p.vs[0] + by : (const uint8_t*)kAttnZeros, vt, i, t);
        }
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
        const int row = 4 * h + (a >> 2);                     // and 8 rows on, whose key is the same
        const int unit = 4 * dt + 2 * ((l >> 4) & 1) + ((a & 3) >> 1);
        const lds_u8* p = tile + (row0 + 16 * c) * L::ROWB + L::at(row, unit) + 8 * (a & 1);
        const bf16x4a_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)p);
        const bf16x4a_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)(p + 8 * L::ROWB));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // the lane's operand for column row `src` (elements 16 s + 8 h ..)
    static __device__ __forceinline__ frag row(const uint8_t* src, int s, int D) {
        const int d = 16 * s + 8 * ((threadIdx.x >> 5) & 1);
        frag f = {};
        if (d < D) f = *(const frag*)(src + 2 * d);
        return f;
    }
    // values 8 c .. 8 c + 7 of a result as an operand, rounded
    static __device__ __forceinline__ frag pack(const f32x16_t& p, int c) {
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)p[8 * c + j];
        return f;
    }
    static __device__ __forceinline__ f32x16_t mma(frag a, frag b, f32x16_t c) { return mfma32(a, b, c); }
    // the rows that the lane's element j of instruction c stands for
    static constexpr int ROWS = 8;
    static __device__ __forceinline__ int index(int c, int j) { return 8 * c + j; }
    static __device__ __forceinline__ bool bad(frag f) {
        uint32_t w[4], t = 0;
        __builtin_memcpy(w, &f, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) t |= (w[j] & 0x7F807F80u) + 0x00800080u;
        return t & 0x80008000u;
    }
    static __device__ __forceinline__ frag only(frag f, int j, bool mine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = mine && e == j ? f[e] : (__bf16)0.f;
        return f;
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
    static __device__ __forceinline__ frag pack(const f32x16_t& p, int c) { return p[c]; }
    static __device__ __forceinline__ f32x16_t mma(frag4 a, frag4 b, f32x16_t c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = mfma32(a[j], b[j], c);
        return c;
    }
    static __device__ __forceinline__ f32x16_t mma(frag a, frag b, f32x16_t c) { return mfma32(a, b, c); }
    static constexpr int ROWS = 1;
    static __device__ __forceinline__ int index(int c, int) { return c; }
    static __device__ __forceinline__ bool bad(frag f) { return (__float_as_uint(f) & 0x7F800000u) == 0x7F800000u; }
    static __device__ __forceinline__ frag only(frag f, int, bool mine) { return mine ? f : 0.f; }
};
// a row's operand has the type of along()
template <typename T, int DP>
using RowFrag = decltype(Operand<T, DP>::row((const uint8_t*)nullptr, 0, 0));

// acc[dt] += (rows' transpose) x w for 32 rows of a tile, w a 32 x 32 result
// whose hidden entries (bit i of `seen` clear) are zero.  A zero times an infinite
// or NaN element of the tile would still be NaN, so a tile that holds some
// (masked tiles only are looked at) goes row by row: every other row's
// elements zeroed, and the sum taken over only by the columns that see the row.
template <typename T, int DP, bool MASKED>
__device__ __forceinline__ void add_rows(f32x16_t (&acc)[DP / 32], const lds_u8* tile, int row0, const f32x16_t& w,
                                         uint32_t seen) {
    using O = Operand<T, DP>;
    if constexpr (MASKED) {
        bool bad = false;
#pragma unroll
        for (int c = 0; c < O::CROSS; ++c)
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) bad |= O::bad(O::across(tile, row0, c, dt));
        if (__ballot(bad)) {
            const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
            for (int c = 0; c < O::CROSS; ++c)
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) {
                    const auto a = O::across(tile, row0, c, dt);
                    const auto b = O::pack(w, c);
#pragma unroll 1
                    for (int j = 0; j < O::ROWS; ++j)
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            const f32x16_t t = O::mma(O::only(a, j, h == half), O::only(b, j, h == half), acc[dt]);
                            // a column's two lane halves see different rows: ask the half that holds it
                            const uint32_t other = (uint32_t)__shfl_xor((int)seen, 32);
                            const bool see = ((h == half ? seen : other) >> O::index(c, j)) & 1;
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[dt][i] = see ? t[i] : acc[dt][i];
                        }
                }
            return;
        }
    }
#pragma unroll
    for (int c = 0; c < O::CROSS; ++c) {
        const auto b = O::pack(w, c);
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = O::mma(O::across(tile, row0, c, dt), b, acc[dt]);
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
            typedef T vec __attribute__((ext_vector_type(4)));
            vec o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = (T)(v[4 * i + j] * f);
            *(vec*)(row + d * (int)sizeof(T)) = o;
        }
    }
}

// All of this wave's loads into LDS have landed.
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("" ::: "memory");
}
// Every LDS read of this wave has returned.
__device__ __forceinline__ void wait_reads() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}

}  // namespace spc
