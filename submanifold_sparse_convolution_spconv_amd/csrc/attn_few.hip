// Attention of few queries within packed sequences for gfx950: single tokens
// against many keys, and calls too small to fill the card by their queries.
//
// The formulas and the references are attn.hip's.  A workgroup has 16 rows
// (positions and heads that share keys), the columns of 16 x 16 products, so
// that little is lost where there are few; its waves take turns at the keys,
// each with a tile of its own, and join their parts at the end.  With a long
// axis and few workgroups the keys are also split over workgroups, joined by a
// second kernel.  Bound by memory where it is about single tokens: a wave has
// the next 32 keys and values in flight (16 KB at D = 128 bf16) while it works
// on the last.  64 single tokens against 262,144 keys, 8 heads on 2 of 128 bf16:
// 95 us a call (2.8 TB/s; with the 32 columns of the other kernel and half as many
// waves 215).
//
// bf16 weights are the second product's operand in two parts, rounded and rest: its
// instructions are not what bounds these calls, and the outputs then have their own
// rounding only (1.7e-3 of their norm; 2.2e-3 with weights rounded once, at 92 us
// for that call, and 10.7 instead of 11.2 for 4,096 rows in 16 scenes).
#include "attn.h"

#include <algorithm>

namespace spc {

namespace {

typedef float f32x4a_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4a_t mfma16(bf16x8r_t a, bf16x8r_t b, f32x4a_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4a_t mfma16(float a, float b, f32x4a_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Operands of 16 x 16 products.  Lane l has column (or row) l & 15 and, as group
// g = l >> 4, the reduction's part 8 g .. (bf16, of 32) or g (fp32, of 4); of a
// result it has the rows 4 g .. 4 g + 3.  The scores of 32 keys are two results,
// whose eight values v (of keys 16 (v / 4) + 4 g + v % 4) are the second
// product's operand as they lie.
template <typename T, int DP>
struct Operand16;

template <int DP>
struct Operand16<__bf16, DP> {
    using L = Tile<__bf16, DP>;
    using Wide = Operand<__bf16, DP>;
    static constexpr int STEPS = DP / 32;
    static constexpr int CROSS = 1;
    typedef bf16x8r_t frag;
    static __device__ __forceinline__ frag along(const lds_u8* tile, int row0, int s) {
        const int l = threadIdx.x & 63;
        return *(const __attribute__((address_space(3))) bf16x8r_t*)(tile + row0 * L::ROWB +
                                                                     L::at(l & 15, 4 * s + (l >> 4)));
    }
    static __device__ __forceinline__ frag row(const uint8_t* src, int s, int D) {
        const int d = 32 * s + 8 * ((threadIdx.x & 63) >> 4);
        frag f = {};
        if (d < D) f = *(const frag*)(src + 2 * d);
        return f;
    }
    static __device__ __forceinline__ frag across(const lds_u8* tile, int, int dt) {
        const int l = threadIdx.x & 63, a = l & 15;
        const int r = 4 * (l >> 4) + (a >> 2);                   // and 16 rows on, whose key is the same
        const lds_u8* p = tile + L::at(r, 2 * dt + ((a & 3) >> 1)) + 8 * (a & 1);
        const bf16x4a_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)p);
        const bf16x4a_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4a_t*)(p + 16 * L::ROWB));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ frag pack(const float (&w)[8], int) {
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)w[j];
        return f;
    }
    // what that rounding left out, as an operand
    static __device__ __forceinline__ frag pack_rest(const float (&w)[8], frag b, int) {
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (__bf16)(w[j] - (float)b[j]);
        return f;
    }
    static __device__ __forceinline__ f32x4a_t mma(frag a, frag b, f32x4a_t c) { return mfma16(a, b, c); }
    static constexpr int VALUES = 8;          // of a lane's eight that one instruction takes
};

template <int DP>
struct Operand16<float, DP> {
    using L = Tile<float, DP>;
    using Wide = Operand<float, DP>;
    static constexpr int STEPS = DP / 16;
    static constexpr int CROSS = 8;
    typedef f32x4r_t frag4;
    typedef float frag;
    static __device__ __forceinline__ frag4 along(const lds_u8* tile, int row0, int s) {
        const int l = threadIdx.x & 63;
        return *(const __attribute__((address_space(3))) f32x4r_t*)(tile + row0 * L::ROWB +
                                                                    L::at(l & 15, 4 * s + (l >> 4)));
    }
    static __device__ __forceinline__ frag4 row(const uint8_t* src, int s, int D) {
        const int d = 16 * s + 4 * ((threadIdx.x & 63) >> 4);
        frag4 f = {};
        if (d < D) f = *(const frag4*)(src + 4 * d);
        return f;
    }
    static __device__ __forceinline__ frag across(const lds_u8* tile, int c, int dt) {
        const int l = threadIdx.x & 63;
        const int r = 16 * (c >> 2) + 4 * (l >> 4) + (c & 3);
        return *(const __attribute__((address_space(3))) float*)(tile + L::at(r, 4 * dt + ((l & 15) >> 2)) + 4 * (l & 3));
    }
    static __device__ __forceinline__ frag pack(const float (&w)[8], int c) { return w[c]; }
    static __device__ __forceinline__ f32x4a_t mma(frag4 a, frag4 b, f32x4a_t c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = mfma16(a[j], b[j], c);
        return c;
    }
    static __device__ __forceinline__ f32x4a_t mma(frag a, frag b, f32x4a_t c) { return mfma16(a, b, c); }
    static constexpr int VALUES = 1;
};

// Over the four lanes of a column.
__device__ __forceinline__ float column_max(float x) {
    x = half_max(x);
    return fmaxf(x, __shfl_xor(x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x = half_sum(x);
    return x + __shfl_xor(x, 16);
}

// add_rows of attn.h for the 32 rows of a tile and 16 columns.
template <typename T, int DP, bool MASKED>
__device__ __forceinline__ void add_rows16(f32x4a_t (&acc)[DP / 16], const lds_u8* tile, const float (&w)[8],
                                           uint32_t seen) {
    using O = Operand16<T, DP>;
    using W = typename O::Wide;
    bool some = false;
#pragma unroll
    for (int c = 0; c < O::CROSS; ++c) {
        const auto b = O::pack(w, c);
#pragma unroll
        for (int dt = 0; dt < DP / 16; ++dt) {
            auto a = O::across(tile, c, dt);
            if constexpr (MASKED) {
                const auto x = W::bad(a);
                some |= W::any(x);
                a = W::without(a, x);
            }
            acc[dt] = O::mma(a, b, acc[dt]);
            if constexpr (sizeof(T) == 2) acc[dt] = O::mma(a, O::pack_rest(w, b, c), acc[dt]);
        }
    }
    if (MASKED && __builtin_expect(__ballot(some) != 0, 0)) {
        const int l = threadIdx.x & 63;
#pragma unroll
        for (int c = 0; c < O::CROSS; ++c) {
            const auto b = O::pack(w, c);
#pragma unroll 1
            for (int j = 0; j < 4 * O::VALUES; ++j) {
                const int g = j & 3, e = j >> 2;
                const bool see = (__shfl((int)seen, (l & 15) + 16 * g) >> (c * O::VALUES + e)) & 1;
#pragma unroll
                for (int dt = 0; dt < DP / 16; ++dt) {
                    const auto x = W::only(W::bad(O::across(tile, c, dt)), e, l >> 4 == g);
                    const f32x4a_t t = O::mma(x, W::only(b, e, l >> 4 == g), f32x4a_t{});
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[dt][i] += see ? t[i] : 0.f;
                }
            }
        }
    }
}

template <typename T, int DP>
struct FewShape {
    static constexpr int ES = sizeof(T);
    static constexpr int KT = 32, NW = 4;
    static constexpr int TILE = KT * DP * ES;
    static constexpr int WAVE = 2 * TILE;             // keys and values of a wave
    static constexpr int LDS = WAVE * NW;
    static constexpr int OCC = ES == 2 ? (DP == 32 ? 4 : DP == 64 ? 3 : 2) : DP <= 32 ? 2 : 1;
};

template <typename T, int DP>
__global__ void __launch_bounds__((64 * FewShape<T, DP>::NW), (FewShape<T, DP>::OCC)) k_attn_few(AttnParams p) {
    using S = FewShape<T, DP>;
    using O = Operand16<T, DP>;
    constexpr int KT = S::KT, NW = S::NW, NDT = DP / 16;
    extern __shared__ __align__(16) uint8_t smem[];

    const int64_t id = xcd_order(blockIdx.x);
    if (id >= p.items * p.HK * p.splits) return;
    const int split = (int)(id % p.splits);
    const int hk = (int)(id / p.splits / p.items);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    QueryRows<kFewRows> qr;
    if (!qr.find(p, kFewRows, 0, hk, id / p.splits % p.items)) return;
    decltype(O::row((const uint8_t*)nullptr, 0, 0)) qf[O::STEPS];
#pragma unroll
    for (int s = 0; s < O::STEPS; ++s) qf[s] = O::row(qr.at(p.q, p.qs), s, p.D);

    const int nt = (qr.longest + KT - 1) / KT;
    const int t0 = (int)((int64_t)nt * split / p.splits), t1 = (int)((int64_t)nt * (split + 1) / p.splits);
    const int begin = t0 + wave;
    lds_u8* kt = (lds_u8*)smem + wave * S::WAVE;
    lds_u8* vt = kt + S::TILE;
    KeyStager<T, DP, KT, 64> keys(p, qr.pl, hk, lane);

    f32x4a_t acc[NDT];
    // (as in attn.hip; bf16 has less only after a first pass that did not do)
    float ref = -INFINITY, less = 0.f, base = 0.f, sum;
    const auto scores = [&](int tl, auto masked, float(&s)[8], uint32_t& seen) {
        f32x4a_t c0 = {}, c1 = {};
#pragma unroll
        for (int c = 0; c < O::STEPS; ++c) {
            c0 = O::mma(O::along(kt, 0, c), qf[c], c0);
            c1 = O::mma(O::along(kt, 16, c), qf[c], c1);
        }
        seen = 0xFFu;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = c0[i];
            s[4 + i] = c1[i];
        }
        if constexpr (decltype(masked)::value) {
            seen = 0;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const bool see = tl * KT + 16 * (v >> 2) + 4 * g + (v & 3) < qr.limit;
                seen |= (uint32_t)see << v;
                s[v] = see ? s[v] : -INFINITY;
            }
        }
    };
    // One pass over the tiles, or, where its reference does not do, one for the maximum
    // and another with that (columns whose reference did keep it, as in attn.hip).
    enum { kFirst, kMaximum, kAgain } pass = kFirst;
    const auto raise = [&](int tl) {
        uint32_t seen;
        float s[8];
        scores(tl, std::true_type{}, s, seen);
#pragma unroll
        for (int v = 0; v < 8; ++v) ref = fmaxf(ref, s[v]);
    };
    const auto set_base = [&]() {
        ref = column_max(ref);
        less = ref == -INFINITY ? 0.f : ref;
        base = less * p.scale2;
        (S::ES == 4 || pass != kFirst ? base : less) = 0.f;
    };
    const auto compute = [&](int tl, auto masked) {
        uint32_t seen;
        float s[8];
        scores(tl, masked, s, seen);
        float part[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            s[v] = __builtin_amdgcn_exp2f(S::ES == 4 ? (s[v] - less) * p.scale2 : fmaf(s[v] - less, p.scale2, -base));
            part[v & 1] += s[v];
        }
        sum += part[0] + part[1];
        add_rows16<T, DP, decltype(masked)::value>(acc, vt, s, seen);
    };
    bool again = false;
    float kept = 0.f, kept_base = 0.f;
    for (;;) {
        sum = 0.f;
#pragma unroll
        for (int d = 0; d < NDT; ++d) acc[d] = f32x4a_t{};
        if (begin < t1) {
            keys.look_up(begin);
            keys.fetch(begin);
            wait_loads();
            keys.store(kt);
            keys.look_up(begin + NW);
            next_tile<true>();
            if (pass == kFirst) {
                raise(begin);
                set_base();
            }
        }
        for (int tl = begin; tl < t1; tl += NW) {
            if (tl + NW < t1) {
                keys.fetch(tl + NW);
                keys.look_up(tl + 2 * NW);
            }
            if (__builtin_expect(pass == kMaximum, 0))
                raise(tl);
            else if ((tl + 1) * KT <= qr.least)
                compute(tl, std::false_type{});
            else
                compute(tl, std::true_type{});
            // (a wave's LDS operations keep their order)
            if (tl + NW < t1) keys.store(kt);
            next_tile<true>();
        }
        if (pass == kMaximum) {
            set_base();
            if (!again) {
                ref = kept;
                less = S::ES == 4 && ref > -INFINITY ? ref : 0.f;
                base = kept_base;
            }
            pass = kAgain;
            continue;
        }
        sum = column_sum(sum);
        if (pass == kAgain) break;
        // (a column that sees none of the wave's first keys sees none of the others)
        const bool sees = begin < t1 && begin * KT < qr.limit;
        again = sees && (!(sum < kAttnMost && sum > 1.f / kAttnMost) || ref == -INFINITY);
#pragma unroll
        for (int d = 0; d < NDT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) again |= !(fabsf(acc[d][i]) < INFINITY);
        if (__builtin_expect(__ballot(again) == 0, 1)) break;
        again = column_max(again ? 1.f : 0.f) > 0.f;
        kept = ref;
        kept_base = base;
        pass = kMaximum;
    }

    // the waves' parts, in their order: the columns, references and sums
    __syncthreads();
    constexpr int PART = (DP + 2) * 16;       // floats
    static_assert(PART * 4 <= S::WAVE);
    if (wave > 0) {
        float* mine = (float*)(smem + wave * S::WAVE);
#pragma unroll
        for (int d = 0; d < NDT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(16 * d + 4 * g + i) * 16 + (lane & 15)] = acc[d][i];
        if (g == 0) {
            mine[DP * 16 + lane] = ref;
            mine[DP * 16 + 16 + lane] = sum;
        }
    }
    __syncthreads();
    if (wave > 0) return;
    float top = ref;
    for (int w = 1; w < NW; ++w) top = fmaxf(top, ((const float*)(smem + w * S::WAVE))[DP * 16 + (lane & 15)]);
    const float from = top == -INFINITY ? 0.f : top;
    const float f0 = __builtin_amdgcn_exp2f((ref - from) * p.scale2);
    sum *= f0;
#pragma unroll
    for (int d = 0; d < NDT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[d][i] *= f0;
#pragma unroll 1
    for (int w = 1; w < NW; ++w) {
        const float* o = (const float*)(smem + w * S::WAVE);
        const float f = __builtin_amdgcn_exp2f((o[DP * 16 + (lane & 15)] - from) * p.scale2);
        sum = fmaf(o[DP * 16 + 16 + (lane & 15)], f, sum);
#pragma unroll
        for (int d = 0; d < NDT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[d][i] = fmaf(o[(16 * d + 4 * g + i) * 16 + (lane & 15)], f, acc[d][i]);
    }
    if (!qr.valid) return;
    // (no key, or no score above -inf: no weight either)
    const bool none = sum == 0.f;
    float f = 1.f;
    uint8_t* out;
    if (p.splits > 1) {
        const int64_t NH = p.N * p.H, at = (int64_t)split * NH + (qr.pl.q0 + qr.pos) * p.H + qr.head;
        out = (uint8_t*)(p.part + at * p.D);
        if (g == 0) {
            float* m = p.part + p.splits * NH * p.D + at * 2;
            m[0] = top;
            m[1] = sum;
        }
    } else {
        f = none ? 0.f : 1.f / sum;
        out = qr.at(p.out, p.os);
        if (p.lse && g == 0)
            p.lse[(int64_t)qr.row * p.H + qr.head] = none ? -INFINITY : fmaf(top, p.scale, logf(sum));
    }
#pragma unroll
    for (int dt = 0; dt < NDT; ++dt) {
        const int d = 16 * dt + 4 * g;
        if (d >= p.D) continue;
        if (p.splits > 1)
            *(f32x4a_t*)(out + 4 * d) = acc[dt];
        else
            store_four<T>(out + d * S::ES, acc[dt], f);
    }
}

// The splits' parts of one (position, head) each block, added in their order
// by kJoinParts runs of them.
constexpr int kJoinThreads = 256, kJoinQuads = 32;     // lanes along D, four elements each
constexpr int kJoinParts = kJoinThreads / kJoinQuads;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(AttnParams p) {
    __shared__ f32x4r_t so[kJoinParts][kJoinQuads];
    __shared__ float sl[kJoinParts];
    const int64_t pos = blockIdx.x / p.H;
    const int head = blockIdx.x % p.H;
    const int64_t begin = clamp_to(p.offsets[0], 0, p.N);
    if (pos < begin || pos >= clamp_to(p.offsets[p.B], begin, p.N)) return;
    const int64_t NH = p.N * p.H, at = pos * p.H + head;
    const float* ml = p.part + p.splits * NH * p.D + at * 2;
    const int t = threadIdx.x, q = t % kJoinQuads, g = t / kJoinQuads;
    float top = -INFINITY;
    for (int s = t & 63; s < p.splits; s += 64) top = fmaxf(top, ml[s * NH * 2]);
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    const float base = top == -INFINITY ? 0.f : top;
    f32x4r_t o = {};
    float l = 0.f;
    const int per = (p.splits + kJoinParts - 1) / kJoinParts;
#pragma unroll 4
    for (int s = g * per; s < min(p.splits, (g + 1) * per); ++s) {
        const float f = __builtin_amdgcn_exp2f((ml[s * NH * 2] - base) * p.scale2);
        l = fmaf(ml[s * NH * 2 + 1], f, l);
        if (4 * q < p.D) o += *(const f32x4r_t*)(p.part + (s * NH + at) * p.D + 4 * q) * f;
    }
    so[g][q] = o;
    if (q == 0) sl[g] = l;
    __syncthreads();
    if (g) return;
    for (int k = 1; k < kJoinParts; ++k) {
        o += so[k][q];
        l += sl[k];
    }
    const bool none = l == 0.f;
    const int64_t row = row_of(p.order, pos, p.N);
    if (4 * q < p.D) {
        uint8_t* out = p.out + row * p.os[0] + head * p.os[1] + 4 * q * (int)sizeof(T);
        store_four<T>(out, o, none ? 0.f : 1.f / l);
    }
    if (p.lse && q == 0) p.lse[row * p.H + head] = none ? -INFINITY : fmaf(top, p.scale, logf(l));
}

template <typename T, int DP>
hipError_t few_go(AttnParams p, hipStream_t st) {
    using S = FewShape<T, DP>;
    p.items = attn_places(p.N, p.G, kFewRows, p.B);
    const hipError_t e =
        hipFuncSetAttribute((const void*)k_attn_few<T, DP>, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    k_attn_few<T, DP><<<(unsigned)xcd_blocks(p.items * p.HK * p.splits), 64 * S::NW, S::LDS, st>>>(p);
    if (p.splits > 1) k_attn_join<T><<<(unsigned)(p.N * p.H), kJoinThreads, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T>
hipError_t few_type(const AttnParams& p, hipStream_t st) {
    switch ((p.D + 31) / 32) {
        case 1: return few_go<T, 32>(p, st);
        case 2: return few_go<T, 64>(p, st);
        case 3: return few_go<T, 96>(p, st);
        default: return few_go<T, 128>(p, st);
    }
}

}  // namespace

hipError_t launch_attn_few(const AttnParams& p, int dtype, hipStream_t st) {
    return dtype == SPCONV_BF16 ? few_type<__bf16>(p, st) : few_type<float>(p, st);
}

}  // namespace spc
