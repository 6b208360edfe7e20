// Attention within packed sequences of voxels for gfx950.
//
//   out[i] = sum_j p[i, j] v[j],  p[i, :] = softmax over j of scale q[i] k[j],
//   lse[i] = log sum_j exp(scale q[i] k[j]),  j <= i + Lk - Lq where causal
//
// One pass over the keys with a reference and a running sum per query.  A wave
// holds 32 queries as the columns of its matrix products: scores come as
// (key, query) tiles, so that a query's softmax is in its own lane (and the lane
// 32 on), the sum needs no exchange until the end, and the scores' layout is
// already that of the second product's operand (rounded to bf16 there, which
// adds as much error as the output's own rounding; sums and references stay
// fp32.  In two parts, rounded and rest, outputs would have their own rounding
// only, but the calls below would take 1,401 instead of 1,037 us and 805 instead
// of 537).  Values are read transposed from LDS.  Four waves share tiles of 64
// keys (32 in fp32), fetched into registers while the tile before is worked on.
//
// Bound by issue: exponentials at heads of 32 (1,006,716 rows in runs of 1,024
// by order, 4 heads bf16: 1,036 us a call, 509 TFLOP/s), exponentials and matrix
// instructions at 64 (29,578 rows in two causal scenes, 8 heads on 2: 541 us,
// 870 TFLOP/s).
//
// The reference that a query's exponentials are taken against is the maximum of
// the first 32 keys, so that the largest weight is 1 at least; larger ones do
// floating point no harm until they leave its range.  No maximum is needed on
// the way, and nothing rescaled (which cost a fifth of the time, most of it in
// copies of the sums around the branch).  Where a query's sum leaves 2^-64 .. 2^64,
// a result is not finite, or all scores of its first keys are -inf, the tile is
// done again with that query's maximum of all keys.
#include "attn.h"

#include <algorithm>

namespace spc {

namespace {

template <typename T, int DP>
struct FwdShape {
    static constexpr int ES = sizeof(T);
    static constexpr int KT = ES == 2 ? 64 : 32;                    // keys per tile
    static constexpr int NW = 4;                                    // waves
    static constexpr int TQ = 32 * NW;                              // query rows per workgroup
    static constexpr int TILE = KT * DP * ES;
    static constexpr int LDS = 4 * TILE;                            // two buffers of keys and values
    // waves of a SIMD that registers are for
    static constexpr int OCC = ES == 2 && DP <= 64 ? (DP == 32 ? 4 : 3) : ES == 2 || DP <= 64 ? 2 : 1;
};

template <typename T, int DP>
__global__ void __launch_bounds__((64 * FwdShape<T, DP>::NW), (FwdShape<T, DP>::OCC)) k_attn(AttnParams p) {
    using S = FwdShape<T, DP>;
    using O = Operand<T, DP>;
    constexpr int KT = S::KT, NSUB = KT / 32, NDT = DP / 32;
    extern __shared__ __align__(16) uint8_t smem[];

    const int64_t id = xcd_order(blockIdx.x);
    if (id >= p.items * p.HK) return;
    const int hk = (int)(id / p.items);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), h = lane >> 5;
    QueryRows<> qr;
    if (!qr.find(p, S::TQ, 32 * wave, hk, id % p.items)) return;
    RowFrag<T, DP> qf[O::STEPS];
#pragma unroll
    for (int s = 0; s < O::STEPS; ++s) qf[s] = O::row(qr.at(p.q, p.qs), s, p.D);

    const int nt = (qr.longest + KT - 1) / KT;
    lds_u8* buf = (lds_u8*)smem;
    KeyStager<T, DP, KT, 64 * S::NW> keys(p, qr.pl, hk, t);

    f32x16_t acc[NDT];
    // the reference of the lane's query (a score, -inf if it sees no key here), what of
    // it is taken off the scores, and what off their exponents
    float ref = -INFINITY, less = 0.f, base = 0.f, sum;

    // scores of 32 keys of a tile
    const auto scores = [&](int tl, int b, int u, auto masked, uint32_t& seen) {
        const lds_u8* kt = buf + b * 2 * S::TILE;
        f32x16_t s = zero16();
#pragma unroll
        for (int c = 0; c < O::STEPS; ++c)
            if (O::wanted(c, p.D)) s = O::mma(O::along(kt, 32 * u, c), qf[c], s);
        seen = 0xFFFFu;
        if constexpr (decltype(masked)::value) {
            seen = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool see = tl * KT + 32 * u + row16(i, h) < qr.limit;
                seen |= (uint32_t)see << i;
                s[i] = see ? s[i] : -INFINITY;
            }
        }
        return s;
    };
    const auto raise = [&](int tl, int b, int u) {
        uint32_t seen;
        const f32x16_t s = scores(tl, b, u, std::true_type{}, seen);
#pragma unroll
        for (int i = 0; i < 16; ++i) ref = fmaxf(ref, s[i]);
    };
    const auto set_base = [&]() {
        ref = half_max(ref);
        less = ref == -INFINITY ? 0.f : ref;
        base = less * p.scale2;
    };
    const auto compute = [&](int tl, int b, auto masked, auto exact) {
        // the next 32 keys' scores under the exponentials of these
        uint32_t seen[NSUB];
        f32x16_t s[NSUB];
        s[0] = scores(tl, b, 0, masked, seen[0]);
#pragma unroll
        for (int u = 0; u < NSUB; ++u) {
            if (u + 1 < NSUB) s[u + 1] = scores(tl, b, u + 1, masked, seen[u + 1]);
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // fp32: the reference's own weight is 1 to the bit, so that one key's
                // value comes out as it is; in bf16 the rounding sees to that, and
                // base may be off by half a step, the same for all of a query's keys
                s[u][i] = __builtin_amdgcn_exp2f(S::ES == 4 ? (s[u][i] - less) * p.scale2
                                                 : decltype(exact)::value
                                                     ? fmaf(s[u][i] - less, p.scale2, -base)
                                                     : fmaf(s[u][i], p.scale2, -base));
                part[i & 3] += s[u][i];
            }
            sum += (part[0] + part[1]) + (part[2] + part[3]);
            add_rows<T, DP, decltype(masked)::value>(acc, buf + b * 2 * S::TILE + S::TILE, 32 * u, s[u], seen[u]);
        }
    };

    // all tiles: `first` before them, when the first has arrived; `each` on those
    // that every query sees whole, then on those that some do not
    const auto sweep = [&](auto first, auto each) {
        if (nt > 0) {
            keys.look_up(0);
            keys.fetch(0);
            keys.store(buf);
            keys.look_up(1);
        }
        wait_loads();
        next_tile<false>();
        if (qr.most > 0) first();
        int b = 0, tl = 0;
        const auto run = [&](int end, auto masked) {
            for (; tl < end; ++tl, b ^= 1) {
                if (tl + 1 < nt) {
                    keys.fetch(tl + 1);
                    keys.look_up(tl + 2);
                }
                if (tl * KT < qr.most) each(tl, b, masked);
                if (tl + 1 < nt) keys.store(buf + (b ^ 1) * 2 * S::TILE);
                next_tile<false>();
            }
        };
        run(qr.least / KT, std::false_type{});
        run(nt, std::true_type{});
    };
    const auto clear = [&]() {
        sum = 0.f;
#pragma unroll
        for (int d = 0; d < NDT; ++d) acc[d] = zero16();
    };
    clear();
    sweep(
        [&]() {
            raise(0, 0, 0);
            set_base();
        },
        [&](int tl, int b, auto masked) { compute(tl, b, masked, std::false_type{}); });
    sum = half_sum(sum);
    bool again = qr.limit > 0 && (!(sum < kAttnMost && sum > 1.f / kAttnMost) || ref == -INFINITY);
#pragma unroll
    for (int d = 0; d < NDT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) again |= !(fabsf(acc[d][i]) < INFINITY);
    again &= qr.valid;       // (columns past the sequence do not count; a wave of them saw no key)
    // (a pass of its own each: as modes of one loop they cost the first 7%)
    if (__builtin_expect(__syncthreads_or(again), 0)) {
        again = half_max(again ? 1.f : 0.f) > 0.f;
        const float kept = ref, kept_base = base;
        sweep([]() {},
              [&](int tl, int b, auto) {
#pragma unroll 1
                  for (int u = 0; u < NSUB; ++u) raise(tl, b, u);
              });
        set_base();
        // (the reference off the score first: base, of scores like 1e30, is too far from it)
        base = 0.f;
        // the tile's other queries keep what they had, and so their bits: what made this
        // one's reference too small may be hidden from them
        if (!again) {
            ref = kept;
            less = S::ES == 4 && ref > -INFINITY ? ref : 0.f;
            base = kept_base;
        }
        clear();
        sweep([]() {}, [&](int tl, int b, auto masked) { compute(tl, b, masked, std::true_type{}); });
        sum = half_sum(sum);
    }

    if (!qr.valid) return;
    // (no key, or no score above -inf: no weight either)
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    uint8_t* o = qr.at(p.out, p.os);
#pragma unroll
    for (int d = 0; d < NDT; ++d) store_col<T>(o, acc[d], f, d, p.D);
    if (p.lse && h == 0)
        p.lse[(int64_t)qr.row * p.H + qr.head] = sum == 0.f ? -INFINITY : fmaf(ref, p.scale, logf(sum));
}

template <typename T, int DP>
hipError_t attn_go(AttnParams p, hipStream_t st) {
    using S = FwdShape<T, DP>;
    p.items = attn_places(p.N, p.G, S::TQ, p.B);
    const hipError_t e =
        hipFuncSetAttribute((const void*)k_attn<T, DP>, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    k_attn<T, DP><<<(unsigned)xcd_blocks(p.items * p.HK), 64 * S::NW, S::LDS, st>>>(p);
    return hipGetLastError();
}

// What a call's sizes choose: 16 rows a workgroup (attn_few.hip), and the parts
// that the keys are split into; else 128.
//
// Few workgroups of 128 leave the card idle, workgroups of 16 read the keys eight
// times as often.  One scene, 8 heads on 2 of 64, us with 16 and with 128 rows:
//   rows (workgroups of 128)   2,000 (126)   3,000 (188)   4,000 (252)   8,000 (502)
//   bf16, causal                  26, 30        42, 42        61, 55       193, 139
//   bf16, full                    37, 31        64, 43       105, 56       372, 155
//   fp32, causal                  88, 168      168, 248      277, 329      979, 1051
//   fp32, full                   138, 172      290, 251      490, 333     1855, 1088
// One bound for all: 256 workgroups, where causal bf16 changes sides.  Sequences of
// 32 rows at most take 16 whatever their number, for the sake of single tokens and
// long caches (64 tokens against 262,144 keys: 95, 215); many short sequences on their
// own keys lose by it (1,000 of 16 rows, 4 heads of 32 bf16: 37, 23; of 32: 44, 25).
// Averages decide, since offsets are on the device: a long sequence among many
// short ones is treated as they are.
struct Plan {
    bool few;
    int splits;
};
Plan plan(const AttnArgs& a) {
    Plan r{};
    const int64_t G = a.H / a.HK;
    // rows per sequence, on average over those that can have any
    const int64_t seqs = std::max<int64_t>(1, std::min<int64_t>(a.B, a.N));
    const int64_t rows = a.N * G / seqs;
    r.few = rows <= 32 || attn_places(a.N, G, 128, seqs) * a.HK < 256;
    r.splits = 1;
    if (r.few) {
        const int64_t blocks = attn_places(a.N, G, kFewRows, seqs) * a.HK;
        const int64_t keys = a.M / std::max<int64_t>(1, std::min<int64_t>(a.B, a.M));
        if (blocks < 512)
            r.splits = (int)std::max<int64_t>(1, std::min<int64_t>({(1024 + blocks - 1) / blocks, keys / 256, 256}));
        if (attn_places(a.N, G, kFewRows, a.B) * a.HK * r.splits > (1 << 20)) r.splits = 1;     // (many empty sequences)
    }
    return r;
}

template <typename T>
hipError_t attn_type(const AttnParams& p, hipStream_t st) {
    switch ((p.D + 31) / 32) {
        case 1: return attn_go<T, 32>(p, st);
        case 2: return attn_go<T, 64>(p, st);
        case 3: return attn_go<T, 96>(p, st);
        default: return attn_go<T, 128>(p, st);
    }
}

}  // namespace

bool attn_fits(const AttnArgs& a) {
    const Plan r = plan(a);
    return attn_threads_fit(attn_places(a.N, a.H / a.HK, r.few ? kFewRows : 128, a.B) * a.HK * r.splits);
}

size_t attn_workspace_bytes(const AttnArgs& a) {
    const Plan r = plan(a);
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
    // (both directions multiply every score by scale2 as it is rounded; a gradient whose
    // lse went by log2 e instead would have all weights off the same way)
    p.scale2 = a.scale * 1.4426950408889634f;
    const double per_lse = (double)p.scale2 / a.scale;
    p.per_lse = (float)per_lse;
    p.per_lse_rest = (float)(per_lse - p.per_lse);
    return p;
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t stream) {
    if (a.N == 0) return hipSuccess;
    AttnParams p = attn_params(a);
    const Plan r = plan(a);
    p.splits = r.splits;
    p.part = (float*)a.workspace;
    if (r.few) return launch_attn_few(p, a.dtype, stream);
    return a.dtype == SPCONV_BF16 ? attn_type<__bf16>(p, stream) : attn_type<float>(p, stream);
}

}  // namespace spc
