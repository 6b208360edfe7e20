// Attention within packed sequences of voxels for gfx950.
//
//   out[i] = sum_j p[i, j] v[j],  p[i, :] = softmax over j of scale q[i] k[j],
//   lse[i] = log sum_j exp(scale q[i] k[j]),  j <= i + Lk - Lq where causal
//
// One pass over the keys with a running reference and sum per query.  A wave
// holds 32 queries as the columns of its matrix products: scores come as
// (key, query) tiles, so that a query's softmax is in its own lane (and the lane
// 32 on), the sum needs no exchange until the end, and the scores' layout is
// already that of the second product's operand (rounded to bf16 there; sums and
// references stay fp32).  Values are read transposed from LDS.
//
// The reference that a query's exponentials are taken against is the maximum of
// the first 32 keys, so that the largest weight is 1 at least; larger ones do
// floating point no harm until they leave its range.  No maximum is needed on
// the way, and nothing rescaled (which cost a fifth of the time, most of it in
// copies of the sums around the branch).  Where the sum reaches 2^64, or a
// result is not finite, the tile is done again with the maximum of all keys.
#include "attn.h"

#include <algorithm>

namespace spc {

namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kMost = 0x1p64f;    // a query's sum from which its reference is taken again

// KS: the workgroup's waves take turns at the keys of one tile of 32 queries
// (each with tiles of its own, joined at the end) instead of sharing the
// keys' tiles for 32 queries each.
template <typename T, int DP, bool KS, int NB>
struct FwdShape {
    static constexpr int ES = sizeof(T);
    static constexpr int KT = ES == 2 && !KS ? 64 : 32;             // keys per tile
    static constexpr int NW = KS && ES == 4 && DP > 64 ? 2 : 4;     // waves (LDS holds no more)
    static constexpr int TQ = KS ? 32 : 32 * NB * NW;               // query rows per workgroup
    static constexpr int TILE = KT * DP * ES;
    static constexpr int LDS = 4 * TILE * (KS ? NW : 1);            // two buffers of keys and values
    static constexpr int OCC = ES == 2 && DP <= 64 ? (DP == 32 ? 4 : 3) - (NB == 2) : ES == 2 || DP <= (KS ? 32 : 64) ? 2 : 1;   // waves of a SIMD that registers are for
};

template <typename T, int DP, bool KS, int NB>
__global__ void __launch_bounds__((64 * FwdShape<T, DP, KS, NB>::NW), (FwdShape<T, DP, KS, NB>::OCC)) k_attn(AttnParams p) {
    using S = FwdShape<T, DP, KS, NB>;
    using O = Operand<T, DP>;
    constexpr int KT = S::KT, NW = S::NW, NSUB = KT / 32, NDT = DP / 32;
    extern __shared__ __align__(16) uint8_t smem[];

    const int64_t id = xcd_order(blockIdx.x);
    if (id >= p.items * p.HK * p.splits) return;
    const int split = (int)(id % p.splits);
    const int hk = (int)(id / p.splits / p.items);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), h = lane >> 5;
    QueryRows<NB> qr;
    if (!qr.find(p, S::TQ, KS ? 0 : 32 * NB * wave, hk, id / p.splits % p.items)) return;
    RowFrag<T, DP> qf[NB][O::STEPS];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int s = 0; s < O::STEPS; ++s) qf[n][s] = O::row(qr.at(p.q, p.qs, n), s, p.D);

    const int nt = (qr.longest + KT - 1) / KT;
    const int t0 = (int)((int64_t)nt * split / p.splits), t1 = (int)((int64_t)nt * (split + 1) / p.splits);
    constexpr int STEP = KS ? NW : 1;
    const int begin = t0 + (KS ? wave : 0);
    lds_u8* buf = (lds_u8*)smem + (KS ? wave * 4 * S::TILE : 0);
    KeyStager<T, DP, KT, KS ? 64 : 64 * NW> keys(p, qr.pl, hk, KS ? lane : t);

    f32x16_t acc[NB][NDT];
    // the references of the lane's queries (scores, -inf if they see no key here), and
    // what they take off exponents (in bf16 powers of two)
    float ref[NB], base[NB], sum[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        ref[n] = -INFINITY;
        base[n] = 0.f;
    }

    // scores of 32 keys of a tile
    const auto scores = [&](int tl, int b, int u, auto masked, f32x16_t(&s)[NB], uint32_t(&seen)[NB]) {
        const lds_u8* kt = buf + b * 2 * S::TILE;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            s[n] = zero16();
            seen[n] = 0xFFFFu;
        }
#pragma unroll
        for (int c = 0; c < O::STEPS; ++c) {
            const auto a = O::along(kt, 32 * u, c);
#pragma unroll
            for (int n = 0; n < NB; ++n) s[n] = O::mma(a, qf[n][c], s[n]);
        }
        if constexpr (decltype(masked)::value) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                seen[n] = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool see = tl * KT + 32 * u + row16(i, h) < qr.limit[n];
                    seen[n] |= (uint32_t)see << i;
                    s[n][i] = see ? s[n][i] : -INFINITY;
                }
            }
        }
    };
    const auto raise = [&](int tl, int b, int u) {
        uint32_t seen[NB];
        f32x16_t s[NB];
        scores(tl, b, u, std::true_type{}, s, seen);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) ref[n] = fmaxf(ref[n], s[n][i]);
    };
    const auto set_base = [&]() {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            ref[n] = half_max(ref[n]);
            base[n] = ref[n] == -INFINITY ? 0.f : S::ES == 4 ? ref[n] : ref[n] * p.scale2;
        }
    };
    const auto compute = [&](int tl, int b, auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
        for (int u = 0; u < NSUB; ++u) {
            uint32_t seen[NB];
            f32x16_t s[NB];
            scores(tl, b, u, masked, s, seen);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // fp32: the reference's own weight is 1 to the bit, so that one key's
                    // value comes out as it is; in bf16 the rounding sees to that
                    s[n][i] = __builtin_amdgcn_exp2f(S::ES == 4 ? (s[n][i] - base[n]) * p.scale2
                                                                : fmaf(s[n][i], p.scale2, -base[n]));
                    part[i & 3] += s[n][i];
                }
                sum[n] += (part[0] + part[1]) + (part[2] + part[3]);
            }
            add_rows<T, DP, MASKED, NB>(acc, buf + b * 2 * S::TILE + S::TILE, 32 * u, s, seen);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // all tiles: `first` before them, when the first has arrived; `each` on those
    // that every query sees whole, then on those that some do not
    const auto sweep = [&](auto first, auto each) {
        if (begin < t1) {
            keys.look_up(begin);
            keys.fetch(begin);
            keys.store(buf);
            keys.look_up(begin + STEP);
        }
        wait_loads();
        next_tile<KS>();
        if (begin < t1 && begin * KT < qr.most) first();
        int b = 0, tl = begin;
        const auto run = [&](int end, auto masked) {
            for (; tl < end; tl += STEP, b ^= 1) {
                if (tl + STEP < t1) {
                    keys.fetch(tl + STEP);
                    keys.look_up(tl + 2 * STEP);
                }
                if (tl * KT < qr.most) each(tl, b, masked);
                if (tl + STEP < t1) keys.store(buf + (b ^ 1) * 2 * S::TILE);
                next_tile<KS>();
            }
        };
        run(min(t1, qr.least / KT), std::false_type{});
        run(t1, std::true_type{});
    };
    const auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            sum[n] = 0.f;
#pragma unroll
            for (int d = 0; d < NDT; ++d) acc[n][d] = zero16();
        }
    };
    clear();
    sweep(
        [&]() {
            raise(begin, 0, 0);
            set_base();
        },
        compute);
    bool again = false;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        again |= !(sum[n] < kMost);
#pragma unroll
        for (int d = 0; d < NDT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) again |= !(fabsf(acc[n][d][i]) < INFINITY);
    }
    if (__builtin_expect(KS ? __ballot(again) != 0 : __syncthreads_or(again), 0)) {
        sweep([]() {},
              [&](int tl, int b, auto) {
#pragma unroll 1
                  for (int u = 0; u < NSUB; ++u) raise(tl, b, u);
              });
        set_base();
        clear();
        sweep([]() {}, compute);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) sum[n] = half_sum(sum[n]);

    if constexpr (KS) {
        // the waves' parts, in their order: (sum, reference) and the columns
        __syncthreads();
        constexpr int PART = (DP + 2) * 32;       // floats
        static_assert(PART * 4 <= 4 * S::TILE);
        float* mine = (float*)(smem + wave * 4 * S::TILE);
        if (wave > 0) {
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(32 * d + row16(i, h)) * 32 + (lane & 31)] = acc[0][d][i];
            if (h == 0) {
                mine[DP * 32 + lane] = ref[0];
                mine[DP * 32 + 32 + lane] = sum[0];
            }
        }
        __syncthreads();
        if (wave > 0) return;
        float top = ref[0];
        for (int w = 1; w < NW; ++w) top = fmaxf(top, ((float*)(smem + w * 4 * S::TILE))[DP * 32 + (lane & 31)]);
        const float base = top == -INFINITY ? 0.f : top;
        const float f0 = __builtin_amdgcn_exp2f((ref[0] - base) * p.scale2);
        sum[0] *= f0;
#pragma unroll
        for (int d = 0; d < NDT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[0][d][i] *= f0;
        for (int w = 1; w < NW; ++w) {
            const float* o = (const float*)(smem + w * 4 * S::TILE);
            const float f = __builtin_amdgcn_exp2f((o[DP * 32 + (lane & 31)] - base) * p.scale2);
            sum[0] = fmaf(o[DP * 32 + 32 + (lane & 31)], f, sum[0]);
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[0][d][i] = fmaf(o[(32 * d + row16(i, h)) * 32 + (lane & 31)], f, acc[0][d][i]);
        }
        ref[0] = top;
    }

#pragma unroll
    for (int n = 0; n < NB; ++n) {
        if (!qr.valid[n]) continue;
        const bool sees = qr.limit[n] > 0;
        if (p.splits > 1) {
            const int64_t NH = p.N * p.H, at = (int64_t)split * NH + (qr.pl.q0 + qr.pos[n]) * p.H + qr.head[n];
            float* o = p.part + at * p.D;
#pragma unroll
            for (int d = 0; d < NDT; ++d) store_col<float>((uint8_t*)o, acc[n][d], 1.f, d, p.D);
            if (h == 0) {
                float* m = p.part + p.splits * NH * p.D + at * 2;
                m[0] = ref[n] * p.scale2;
                m[1] = sees ? sum[n] : -1.f;
            }
            continue;
        }
        const float f = sees ? 1.f / sum[n] : 0.f;
        uint8_t* o = qr.at(p.out, p.os, n);
#pragma unroll
        for (int d = 0; d < NDT; ++d) store_col<T>(o, acc[n][d], f, d, p.D);
        if (p.lse && h == 0)
            p.lse[(int64_t)qr.row[n] * p.H + qr.head[n]] = sees ? fmaf(ref[n], p.scale, logf(sum[n])) : -INFINITY;
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
    const bool none = ml[1] < 0.f;
    const float base = top == -INFINITY ? 0.f : top;
    f32x4r_t o = {};
    float l = 0.f;
    const int per = (p.splits + kJoinParts - 1) / kJoinParts;
#pragma unroll 4
    for (int s = g * per; s < min(p.splits, (g + 1) * per); ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[s * NH * 2] - base);
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
    const int64_t row = row_of(p.order, pos, p.N);
    if (4 * q < p.D) {
        typedef T vec __attribute__((ext_vector_type(4)));
        vec r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = (T)(none ? 0.f : o[j] * (1.f / l));
        *(vec*)(p.out + row * p.os[0] + head * p.os[1] + 4 * q * (int)sizeof(T)) = r;
    }
    if (p.lse && q == 0) p.lse[row * p.H + head] = none ? -INFINITY : (top + log2f(l)) * kLn2;
}

template <typename T, int DP, bool KS, int NB>
hipError_t attn_go(AttnParams p, hipStream_t st) {
    using S = FwdShape<T, DP, KS, NB>;
    p.items = attn_places(p.N, p.G, S::TQ, p.B);
    const int64_t blocks = xcd_blocks(p.items * p.HK * p.splits);
    const hipError_t e =
        hipFuncSetAttribute((const void*)k_attn<T, DP, KS, NB>, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    k_attn<T, DP, KS, NB><<<(unsigned)blocks, 64 * S::NW, S::LDS, st>>>(p);
    if (p.splits > 1) k_attn_join<T><<<(unsigned)(p.N * p.H), kJoinThreads, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, int DP>
hipError_t attn_width(const AttnParams& p, bool ks, hipStream_t st) {
    constexpr int NB = 1;
    return ks ? attn_go<T, DP, true, 1>(p, st) : attn_go<T, DP, false, NB>(p, st);
}
template <typename T>
hipError_t attn_type(const AttnParams& p, bool ks, hipStream_t st) {
    switch ((p.D + 31) / 32) {
        case 1: return attn_width<T, 32>(p, ks, st);
        case 2: return attn_width<T, 64>(p, ks, st);
        case 3: return attn_width<T, 96>(p, ks, st);
        default: return attn_width<T, 128>(p, ks, st);
    }
}

}  // namespace

AttnPlan attn_plan(const AttnArgs& a) {
    AttnPlan r;
    const int64_t G = a.H / a.HK;
    // queries per sequence, on average over those that can have any
    const int64_t seqs = std::max<int64_t>(1, std::min<int64_t>(a.B, a.N));
    const int64_t rows = a.N * G / seqs;
    const int64_t shared = attn_places(a.N, G, 128, seqs) * a.HK;
    r.ks = rows <= 32 || shared < 512;
    const int64_t blocks = r.ks ? attn_places(a.N, G, 32, seqs) * a.HK : shared;
    const int64_t keys = a.M / std::max<int64_t>(1, std::min<int64_t>(a.B, a.M));
    int64_t splits = blocks >= 512 ? 1 : std::min((1024 + blocks - 1) / std::max<int64_t>(blocks, 1), keys / 512);
    r.splits = (int)std::max<int64_t>(1, std::min<int64_t>(splits, 256));
    if (attn_places(a.N, G, 32, a.B) * a.HK * r.splits > (1 << 20)) r.splits = 1;     // (many empty sequences)
    return r;
}

bool attn_fits(const AttnArgs& a, bool grad) {
    // most workgroups of 256 threads that any plan launches per sequence and split
    const auto fits = [&](int64_t n, int64_t per) {
        return n * per < (1ll << 31) &&
               (attn_places(n, per, 32, a.B) * a.HK + kXcds * kRun) * 256 < (1ll << 32);
    };
    return fits(a.N, a.H / a.HK) && (!grad || fits(a.M, 1));
}

size_t attn_workspace_bytes(const AttnArgs& a) {
    const AttnPlan r = attn_plan(a);
    return r.splits > 1 ? align_up((size_t)r.splits * a.N * a.H * (a.D + 2) * 4, 256) : 0;
}

AttnParams attn_params(const AttnArgs& a) {
    const int es = a.dtype == SPCONV_BF16 ? 2 : 4;
    AttnParams p{};
    p.q = (const uint8_t*)a.q;
    p.k = (const uint8_t*)a.k;
    p.v = (const uint8_t*)a.v;
    p.offsets = a.offsets;
    p.koffsets = a.koffsets;
    p.order = a.order;
    p.korder = a.koffsets ? a.korder : a.order;
    p.out = (uint8_t*)a.out;
    p.lse = a.lse;
    p.dout = (const uint8_t*)a.dout;
    p.dq = (uint8_t*)a.dq;
    p.dk = (uint8_t*)a.dk;
    p.dv = (uint8_t*)a.dv;
    const auto strides = [es](int64_t (&d)[2], const int64_t (&s)[2]) {
        d[0] = s[0] * es;
        d[1] = s[1] * es;
    };
    strides(p.qs, a.qs);
    strides(p.ks, a.ks);
    strides(p.vs, a.vs);
    strides(p.os, a.os);
    strides(p.dos, a.dos);
    strides(p.dqs, a.dqs);
    strides(p.dks, a.dks);
    strides(p.dvs, a.dvs);
    p.N = a.N;
    p.M = a.M;
    p.H = a.H;
    p.HK = a.HK;
    p.G = a.H / a.HK;
    p.D = a.D;
    p.B = a.B;
    p.magic = (uint32_t)((1ull << 32) / p.G + 1);
    p.causal = a.causal;
    p.splits = 1;
    const auto below = [&](const int64_t(&s)[2]) { return a.M * s[0] * es < (1ll << 31); };
    p.near = below(a.ks) && below(a.vs);
    p.scale = a.scale;
    p.scale2 = a.scale * 1.4426950408889634f;
    return p;
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
    if (a.N == 0) return hipSuccess;
    AttnParams p = attn_params(a);
    const AttnPlan r = attn_plan(a);
    p.splits = r.splits;
    p.part = (float*)a.workspace;
    return a.dtype == SPCONV_BF16 ? attn_type<__bf16>(p, r.ks, stream) : attn_type<float>(p, r.ks, stream);
}

}  // namespace spc
