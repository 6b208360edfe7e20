// Gradient of the attention within packed sequences, for gfx950.
//
// With p = exp(scale q k - lse) and delta[i] = dout[i] out[i]:
//   ds[i, j] = p[i, j] (dout[i] v[j] - delta[i])
//   dq[i] = scale sum_j ds[i, j] k[j]
//   dk[j] = scale sum_i ds[i, j] q[i],   dv[j] = sum_i p[i, j] dout[i]
//
// Two kernels, so that every sum has one owner and a fixed order: one over the
// queries (dq, and delta for the other), one over the keys (dk and dv, summed
// over the heads that share them).  Each computes p and ds again: 7 products
// where 5 are needed, against atomics in dq.  As in the forward the results of
// the first products are the operands of the next as they lie in the
// registers: (key, query) tiles for dq, (query, key) tiles for dk and dv; all
// sums are fp32.
//
// Two causal scenes of 29,578 rows, 8 heads on 2 of 64 bf16: 1,803 us a call; under
// the profiler 828 for dq, 1,120 for dk and dv in five parts and 27 for their sums
// (850 and 840 TFLOP/s of executed products), vector issue 43% and matrix unit 44%
// of the time.
//
// In bf16, p and ds are rounded once as operands, which is as much again as the
// results' own rounding (2.4e-3 of a gradient's norm in all, 1.7e-3 without).
// delta suffers from the rounding of out, little where a query sees many keys, but
// where it sees a few dout v - delta cancels (two keys, causal: 1.0e-2).  So a
// tile of queries that see kFineKeys at most works out delta = sum_j p dout v from
// the keys first, and ds and p, also of the keys of such sequences, are taken in two
// parts: their gradients are then off by the results' rounding only, for a third more
// time (120 causal runs of 250, 4 heads on 2 of 64: 92 -> 123 us).
#include "attn.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kFineKeys = 256;

// KS: the waves of a workgroup take turns at the long axis for 32 rows instead
// of sharing its tiles for 32 rows each.
template <typename T, int DP, bool KS>
struct GradShape {
    static constexpr int ES = sizeof(T);
    static constexpr int KT = ES == 2 && !KS ? 64 : 32;             // rows per tile of the long axis
    static constexpr int NW = KS && ES == 4 && DP > 64 ? 2 : 4;
    static constexpr int TR = KS ? 32 : 32 * NW;                    // rows that a workgroup owns
    static constexpr int TILE = KT * DP * ES;
    static constexpr int STATS = 2 * KT * 4;                        // lse and delta of a tile of queries
    static constexpr int WAVE = 4 * TILE + 2 * STATS;               // two buffers
    static constexpr int LDS = WAVE * (KS ? NW : 1);
    static constexpr int DQ_OCC = ES == 2 && DP == 32 ? 4 : DP <= 32 || (DP == 64 && (ES == 2 || !KS)) ? 2 : 1;   // waves of a SIMD that registers are for
    static constexpr int DKV_OCC = DP <= 32 || (DP == 64 && (ES == 2 || !KS)) ? 2 : 1;
};

// lse in powers of two; rows without keys (-inf), and places without a row (inf): p =
// 2^-inf = 0
__device__ __forceinline__ float stat2(const AttnParams& p, float lse) {
    return fabsf(lse) == INFINITY ? INFINITY : fmaf(lse, p.per_lse, lse * p.per_lse_rest);
}

template <typename T, int DP, bool KS>
__global__ void __launch_bounds__((64 * GradShape<T, DP, KS>::NW), (GradShape<T, DP, KS>::DQ_OCC)) k_attn_dq(AttnParams p) {
    using S = GradShape<T, DP, KS>;
    using O = Operand<T, DP>;
    constexpr int KT = S::KT, NW = S::NW, NDT = DP / 32;
    extern __shared__ __align__(16) uint8_t smem[];

    const int64_t id = xcd_order(blockIdx.x);
    if (id >= p.items * p.HK * p.splits) return;
    const int split = (int)(id % p.splits);
    const int hk = (int)(id / p.splits / p.items);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), h = lane >> 5;
    QueryRows<> qr;
    if (!qr.find(p, S::TR, KS ? 0 : 32 * wave, hk, id / p.splits % p.items)) return;
    RowFrag<T, DP> qf[O::STEPS], df[O::STEPS];
    f32x16_t dd = zero16();
#pragma unroll
    for (int s = 0; s < O::STEPS; ++s) {
        qf[s] = O::row(qr.at(p.q, p.qs), s, p.D);
        df[s] = O::row(qr.at(p.dout, p.dos), s, p.D);
        dd = O::mma(O::row(qr.at((const uint8_t*)p.out, p.os), s, p.D), df[s], dd);
    }
    // the diagonal: row16(i, h) = lane & 31
    float delta = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) delta = row16(i, h) == (lane & 31) ? dd[i] : delta;
    const float other = __shfl_xor(delta, 32);
    delta = ((lane >> 2) & 1) == h ? delta : other;
    const float lse2 = stat2(p, p.lse[(int64_t)qr.row * p.H + qr.head]);

    const int nt = (qr.longest + KT - 1) / KT;
    const bool fine = S::ES == 2 && qr.longest <= kFineKeys;
    const int t0 = (int)((int64_t)nt * split / p.splits), t1 = (int)((int64_t)nt * (split + 1) / p.splits);
    constexpr int STEP = KS ? NW : 1;
    const int begin = t0 + (KS ? wave : 0);
    lds_u8* buf = (lds_u8*)smem + (KS ? wave * S::WAVE : 0);
    KeyStager<T, DP, KT, KS ? 64 : 64 * NW> keys(p, qr.pl, hk, KS ? lane : t);

    f32x16_t acc[NDT];
#pragma unroll
    for (int d = 0; d < NDT; ++d) acc[d] = zero16();

    // where the sums of dout v start: -delta
    f32x16_t less;
    const auto probabilities = [&](int tl, int b, int u, auto masked, f32x16_t& e, f32x16_t& dp, uint32_t& seen) {
        const lds_u8* kt = buf + b * 2 * S::TILE;
        const lds_u8* vt = kt + S::TILE;
        e = zero16();
        dp = less;
#pragma unroll
        for (int c = 0; c < O::STEPS; ++c) {
            if (!O::wanted(c, p.D)) continue;
            e = O::mma(O::along(kt, 32 * u, c), qf[c], e);
            dp = O::mma(O::along(vt, 32 * u, c), df[c], dp);
        }
        seen = 0xFFFFu;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            e[i] = __builtin_amdgcn_exp2f(fmaf(e[i], p.scale2, -lse2));
            if constexpr (decltype(masked)::value) {
                const bool see = tl * KT + 32 * u + row16(i, h) < qr.limit;
                seen = see ? seen : seen & ~(1u << i);
                e[i] = see ? e[i] : 0.f;
                dp[i] = see ? dp[i] : 0.f;
            }
        }
    };
    const auto compute = [&](int tl, int b, auto masked, auto two) {
#pragma unroll
        for (int u = 0; u < KT / 32; ++u) {
            uint32_t seen;
            f32x16_t e, dp;
            probabilities(tl, b, u, masked, e, dp, seen);
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] *= dp[i];
            add_rows<T, DP, decltype(masked)::value, decltype(two)::value>(acc, buf + b * 2 * S::TILE, 32 * u, e, seen);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // the tiles from `from` on
    const auto sweep = [&](int from, int to, int whole, auto each, auto rest) {
        if (from < to) {
            keys.look_up(from);
            keys.fetch(from);
            keys.store(buf);
            keys.look_up(from + STEP);
        }
        wait_loads();
        next_tile<KS>();
        int b = 0, tl = from;
        const auto run = [&](int end, auto f) {
            for (; tl < end; tl += STEP, b ^= 1) {
                if (tl + STEP < to) {
                    keys.fetch(tl + STEP);
                    keys.look_up(tl + 2 * STEP);
                }
                if (tl * KT < qr.most) f(tl, b);
                if (tl + STEP < to) keys.store(buf + (b ^ 1) * 2 * S::TILE);
                next_tile<KS>();
            }
        };
        run(min(to, whole), each);
        run(to, rest);
    };
    const auto none = [](int, int) {};
    if constexpr (S::ES == 2)
        if (fine) {
            less = zero16();
            float d = 0.f;
            sweep(KS ? wave : 0, nt, 0, none, [&](int tl, int b) {
#pragma unroll 1
                for (int u = 0; u < KT / 32; ++u) {
                    uint32_t seen;
                    f32x16_t e, dp;
                    probabilities(tl, b, u, std::true_type{}, e, dp, seen);
#pragma unroll
                    for (int i = 0; i < 16; ++i) d = fmaf(e[i], dp[i], d);
                }
            });
            delta = half_sum(d);
            if constexpr (KS) {
                __shared__ float parts[NW][32];
                if (h == 0) parts[wave][lane] = delta;
                __syncthreads();
                delta = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) delta += parts[w][lane & 31];
            }
        }
    if (qr.valid && h == 0 && split == 0 && (!KS || wave == 0)) p.delta[(int64_t)qr.row * p.H + qr.head] = delta;
#pragma unroll
    for (int i = 0; i < 16; ++i) less[i] = -delta;
    const auto masked = [&](int tl, int b) { compute(tl, b, std::true_type{}, std::false_type{}); };
    if (fine) {
        if constexpr (S::ES == 2)
            sweep(begin, t1, 0, none, [&](int tl, int b) { compute(tl, b, std::true_type{}, std::true_type{}); });
    } else {
        // tiles that every query sees whole, then those that some do not
        sweep(begin, t1, qr.least / KT, [&](int tl, int b) { compute(tl, b, std::false_type{}, std::false_type{}); },
              masked);
    }

    if constexpr (KS) {
        __syncthreads();
        if (wave > 0) {
            float* mine = (float*)(smem + wave * S::WAVE);
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(32 * d + row16(i, h)) * 32 + (lane & 31)] = acc[d][i];
        }
        __syncthreads();
        if (wave > 0) return;
        for (int w = 1; w < NW; ++w) {
            const float* o = (const float*)(smem + w * S::WAVE);
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] += o[(32 * d + row16(i, h)) * 32 + (lane & 31)];
        }
    }
    if (!qr.valid) return;
    // (the weight of a single key is 1, whatever its score)
    const float scale = qr.limit > 1 ? p.scale : 0.f;
    if (p.splits > 1) {
        float* o = p.part + ((split * p.N + qr.pl.q0 + qr.pos) * p.H + qr.head) * p.D;
#pragma unroll
        for (int d = 0; d < NDT; ++d) store_col<float>((uint8_t*)o, acc[d], scale, d, p.D);
        return;
    }
    uint8_t* o = qr.at(p.dq, p.dqs);
#pragma unroll
    for (int d = 0; d < NDT; ++d) store_col<T>(o, acc[d], scale, d, p.D);
}

template <typename T, int DP, bool KS>
__global__ void __launch_bounds__((64 * GradShape<T, DP, KS>::NW), (GradShape<T, DP, KS>::DKV_OCC)) k_attn_dkv(AttnParams p) {
    using S = GradShape<T, DP, KS>;
    using O = Operand<T, DP>;
    constexpr int KT = S::KT, NW = S::NW, NDT = DP / 32;
    constexpr int THR = KS ? 64 : 64 * NW;
    using St = Stager<T, DP, KT, THR>;
    extern __shared__ __align__(16) uint8_t smem[];

    const int64_t id = xcd_order(blockIdx.x);
    if (id >= p.items * p.HK * p.splits) return;
    const int split = (int)(id % p.splits);
    const int hk = (int)(id / p.splits / p.items);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), h = lane >> 5;
    const int st = KS ? lane : t;

    // the sequence by its keys
    Place pl = find_place(p.koffsets ? p.koffsets : p.offsets, p.B, p.M, 1, S::TR, id / p.splits % p.items);
    if (pl.tile < 0) return;
    pl.k0 = pl.q0;
    pl.Lk = pl.Lq;
    if (p.koffsets) {
        pl.q0 = clamp_to(p.offsets[pl.b], 0, p.N);
        pl.Lq = (int)(clamp_to(p.offsets[pl.b + 1], pl.q0, p.N) - pl.q0);
    }
    const int R = pl.Lq * p.G;
    const int first = pl.tile * S::TR + (KS ? 0 : 32 * wave);
    const bool valid = first + (lane & 31) < pl.Lk;
    const int key = min(first + (lane & 31), pl.Lk - 1);
    // the first query row that sees a key
    const auto seen_from = [&](int k) {
        const int64_t r = p.causal ? (int64_t)max(0, k - (pl.Lk - pl.Lq)) * p.G : 0;
        return (int)min(r, (int64_t)R);
    };
    const int from = seen_from(key);
    const int wave_first = first < pl.Lk ? seen_from(first) : R;
    const int block_last = seen_from(min((pl.tile + 1) * S::TR, pl.Lk) - 1);
    const int64_t krow = row_of(p.korder, pl.k0 + key, p.M);
    RowFrag<T, DP> kf[O::STEPS], vf[O::STEPS];
#pragma unroll
    for (int s = 0; s < O::STEPS; ++s) {
        kf[s] = O::row(p.k + krow * p.ks[0] + hk * p.ks[1], s, p.D);
        vf[s] = O::row(p.v + krow * p.vs[0] + hk * p.vs[1], s, p.D);
    }

    const int tb = seen_from(pl.tile * S::TR) / KT, nt = (R + KT - 1) / KT - tb;
    const int t0 = tb + (int)((int64_t)nt * split / p.splits), t1 = tb + (int)((int64_t)nt * (split + 1) / p.splits);
    constexpr int STEP = KS ? NW : 1;
    const int begin = t0 + (KS ? wave : 0);
    lds_u8* buf = (lds_u8*)smem + (KS ? wave * S::WAVE : 0);
    float* stats = (float*)(smem + (KS ? wave * S::WAVE : 0) + 4 * S::TILE);

    // The queries' rows.  Where a tile is a whole number of positions, those one after
    // the other and its heads within 31 bits, as the keys are fetched; else each row's
    // place is looked up one tile before.
    constexpr int NP = St::NP;
    const auto close = [&](const int64_t(&s)[2]) { return KT / p.G * s[0] + p.G * s[1] < (1ll << 31); };
    const bool plain = !p.order && KT % p.G == 0 && close(p.qs) && close(p.dos);
    uint32_t oq[NP], od[NP];
    int qrow[NP], qhead[NP];
    u32x4a_t rq[NP], rd[NP];
    float lse = INFINITY, delta = 0.f, lse_next = INFINITY, delta_next = 0.f;
    const uint8_t* qh = p.q + hk * p.G * p.qs[1];
    const uint8_t* dh = p.dout + hk * p.G * p.dos[1];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int by = St::byte(i, st);
        const RowHead rh = plain ? split_row(St::row(i, st), p.G, p.magic) : RowHead{0, 0};
        const bool in = by < p.D * (int)sizeof(T);
        oq[i] = in ? (uint32_t)(by + rh.pos * p.qs[0] + rh.head * p.qs[1]) : kNoUnit;
        od[i] = in ? (uint32_t)(by + rh.pos * p.dos[0] + rh.head * p.dos[1]) : kNoUnit;
    }
    auto look_up = [&](int tl) {
        if (!plain) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = tl * KT + St::row(i, st);
                qrow[i] = -1;
                qhead[i] = 0;
                if (r < R) {
                    const RowHead rh = split_row(r, p.G, p.magic);
                    qrow[i] = (int)row_of(p.order, pl.q0 + rh.pos, p.N);
                    qhead[i] = rh.head;
                }
            }
        }
        if (st < KT) {
            const int r = tl * KT + st;
            lse_next = INFINITY;
            delta_next = 0.f;
            if (r < R) {
                const RowHead rh = split_row(r, p.G, p.magic);
                const int64_t at = row_of(p.order, pl.q0 + rh.pos, p.N) * p.H + hk * p.G + rh.head;
                lse_next = p.lse[at];
                delta_next = p.delta[at];
            }
        }
    };
    auto fetch = [&](int tl) {
        lse = lse_next;
        delta = delta_next;
        if (!plain) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const bool in = qrow[i] >= 0 && oq[i] != kNoUnit;
                rq[i] = fetch16(qh + qrow[i] * p.qs[0] + qhead[i] * p.qs[1] + oq[i], in);
                rd[i] = fetch16(dh + qrow[i] * p.dos[0] + qhead[i] * p.dos[1] + od[i], in);
            }
            return;
        }
        const int64_t at = pl.q0 + (int64_t)tl * (KT / p.G);
        const auto bq = rows_at(qh + at * p.qs[0]), bd = rows_at(dh + at * p.dos[0]);
        const int left = R - tl * KT;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            rq[i] = fetch16(bq, left >= KT || St::row(i, st) < left ? oq[i] : kNoUnit);
            rd[i] = fetch16(bd, left >= KT || St::row(i, st) < left ? od[i] : kNoUnit);
        }
    };
    auto store = [&](int b) {
        lds_u8* qt = buf + b * 2 * S::TILE;
        St::store(rq, qt, st);
        St::store(rd, qt + S::TILE, st);
        if (st < KT) {
            stats[b * 2 * KT + st] = stat2(p, lse);
            stats[b * 2 * KT + KT + st] = -delta;
        }
    };

    f32x16_t dk[NDT], dv[NDT];
#pragma unroll
    for (int d = 0; d < NDT; ++d) dk[d] = dv[d] = zero16();

    const bool fine = S::ES == 2 && pl.Lk <= kFineKeys;
    auto compute = [&](int tl, int b, auto masked, auto two) {
        constexpr bool MASKED = decltype(masked)::value, TWO = decltype(two)::value;
        const lds_u8* qt = buf + b * 2 * S::TILE;
        const lds_u8* dt = qt + S::TILE;
#pragma unroll
        for (int u = 0; u < KT / 32; ++u) {
            const float* l2 = stats + b * 2 * KT + 32 * u;
            f32x16_t s = zero16(), dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] = l2[KT + row16(i, h)];
#pragma unroll
            for (int c = 0; c < O::STEPS; ++c) {
                if (!O::wanted(c, p.D)) continue;
                s = O::mma(O::along(qt, 32 * u, c), kf[c], s);
                dp = O::mma(O::along(dt, 32 * u, c), vf[c], dp);
            }
            uint32_t seen = 0xFFFFu;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(fmaf(s[i], p.scale2, -l2[row16(i, h)]));
                dp[i] *= e;
                s[i] = e;
                if constexpr (MASKED) {
                    const bool see = tl * KT + 32 * u + row16(i, h) >= from;
                    seen = see ? seen : seen & ~(1u << i);
                    s[i] = see ? s[i] : 0.f;
                    dp[i] = see ? dp[i] : 0.f;
                }
            }
            add_rows<T, DP, MASKED, TWO>(dv, dt, 32 * u, s, seen);
            add_rows<T, DP, MASKED, TWO>(dk, qt, 32 * u, dp, seen);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (begin < t1) {
        look_up(begin);
        fetch(begin);
        store(0);
        look_up(begin + STEP);
    }
    wait_loads();
    next_tile<KS>();
    int b = 0, tl = begin;
    const auto sweep = [&](int end, auto masked, auto two) {
        for (; tl < end; tl += STEP, b ^= 1) {
            if (tl + STEP < t1) {
                fetch(tl + STEP);
                look_up(tl + 2 * STEP);
            }
            if ((tl + 1) * KT > wave_first) compute(tl, b, masked, two);
            if (tl + STEP < t1) store(b ^ 1);
            next_tile<KS>();
        }
    };
    if (fine) {
        if constexpr (S::ES == 2) sweep(t1, std::true_type{}, std::true_type{});
    } else {
        // tiles that some keys are hidden from, then those that see every key
        sweep(min(t1, (block_last + KT - 1) / KT), std::true_type{}, std::false_type{});
        sweep(t1, std::false_type{}, std::false_type{});
    }

    if constexpr (KS) {
        static_assert(DP * 32 * 4 * 2 <= 4 * S::TILE);
        __syncthreads();
        if (wave > 0) {
            float* mine = (float*)(smem + wave * S::WAVE);
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    mine[(32 * d + row16(i, h)) * 32 + (lane & 31)] = dk[d][i];
                    mine[(DP + 32 * d + row16(i, h)) * 32 + (lane & 31)] = dv[d][i];
                }
        }
        __syncthreads();
        if (wave > 0) return;
        for (int w = 1; w < NW; ++w) {
            const float* o = (const float*)(smem + w * S::WAVE);
#pragma unroll
            for (int d = 0; d < NDT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    dk[d][i] += o[(32 * d + row16(i, h)) * 32 + (lane & 31)];
                    dv[d][i] += o[(DP + 32 * d + row16(i, h)) * 32 + (lane & 31)];
                }
        }
    }
    if (!valid) return;
    const float scale = pl.Lk > 1 ? p.scale : 0.f;     // (a single key's weight is 1)
    if (p.splits > 1) {
        float* o = p.part + ((split * p.M + pl.k0 + key) * p.HK + hk) * p.D;
        const int64_t all = p.splits * p.M * p.HK * p.D;
#pragma unroll
        for (int d = 0; d < NDT; ++d) {
            store_col<float>((uint8_t*)o, dk[d], scale, d, p.D);
            store_col<float>((uint8_t*)(o + all), dv[d], 1.f, d, p.D);
        }
        return;
    }
#pragma unroll
    for (int d = 0; d < NDT; ++d) {
        store_col<T>(p.dk + krow * p.dks[0] + hk * p.dks[1], dk[d], scale, d, p.D);
        store_col<T>(p.dv + krow * p.dvs[0] + hk * p.dvs[1], dv[d], 1.f, d, p.D);
    }
}

// Sums of the splits' parts in their order: four elements of a (position, head)
// per thread.  A second tensor's parts (dv next to dk) follow the first's.
struct SumOut {
    uint8_t* t;
    int64_t rs, hs;        // bytes from row to row and from head to head
};
template <typename T>
__global__ void __launch_bounds__(256) k_attn_sum(const float* part, int splits, const int32_t* offsets, int B,
                                                  const int32_t* order, int64_t n, int heads, int D, SumOut out0,
                                                  SumOut out1) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = D / 4, all = n * heads * quads;
    if (e >= all) return;
    const int64_t pos = e / quads / heads;
    const int64_t begin = clamp_to(offsets[0], 0, n);
    if (pos < begin || pos >= clamp_to(offsets[B], begin, n)) return;
    const SumOut out = blockIdx.y ? out1 : out0;
    part += blockIdx.y * splits * all * 4;
    f32x4r_t s = {};
#pragma unroll 8
    for (int k = 0; k < splits; ++k) s += *(const f32x4r_t*)(part + 4 * (k * all + e));
    store_four<T>(out.t + row_of(order, pos, n) * out.rs + e / quads % heads * out.hs +
                      e % quads * 4 * (int)sizeof(T),
                  s, 1.f);
}

struct Plan {
    bool ks;
    int splits;
};
// A gradient kernel owns rows (queries or keys) of one axis and sums over the
// other: the waves' share and the splits from both axes' sizes.  Waves that take
// turns serve few rows only (4,097 rows of 2 heads in fp32, keys' gradient: 219
// us, 156 with rows of their own and the queries in parts).
Plan side_plan(int64_t n, int64_t per, int64_t B, int64_t HK, int64_t along) {
    const int64_t seqs = std::max<int64_t>(1, std::min(B, n));
    Plan r;
    const int64_t shared = attn_places(n, per, 128, seqs) * HK;
    r.ks = n * per / seqs <= 32 || shared < 64;
    const int64_t blocks = std::max<int64_t>(1, r.ks ? attn_places(n, per, 32, seqs) * HK : shared);
    const int64_t splits = blocks >= 512 ? 1 : std::min((2048 + blocks - 1) / blocks, along / 128);
    r.splits = (int)std::max<int64_t>(1, std::min<int64_t>(splits, 256));
    if (attn_places(n, per, 32, B) * HK * r.splits > (1 << 20)) r.splits = 1;     // (many empty sequences)
    return r;
}
Plan dq_plan(const AttnArgs& a) {
    return side_plan(a.N, a.H / a.HK, a.B, a.HK, a.M / std::max<int64_t>(1, std::min<int64_t>(a.B, a.M)));
}
Plan dkv_plan(const AttnArgs& a) {
    return side_plan(a.M, 1, a.B, a.HK, a.N * (a.H / a.HK) / std::max<int64_t>(1, std::min<int64_t>(a.B, a.N)));
}
size_t delta_bytes(const AttnArgs& a) { return align_up((size_t)a.N * a.H * 4, 256); }

template <typename T, int DP, bool KS>
hipError_t dq_go(AttnParams p, hipStream_t st) {
    using S = GradShape<T, DP, KS>;
    p.items = attn_places(p.N, p.G, S::TR, p.B);
    hipError_t e = hipFuncSetAttribute((const void*)k_attn_dq<T, DP, KS>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    k_attn_dq<T, DP, KS><<<(unsigned)xcd_blocks(p.items * p.HK * p.splits), 64 * S::NW, S::LDS, st>>>(p);
    return hipGetLastError();
}
template <typename T, int DP, bool KS>
hipError_t dkv_go(AttnParams p, hipStream_t st) {
    using S = GradShape<T, DP, KS>;
    p.items = attn_places(p.M, 1, S::TR, p.B);
    hipError_t e = hipFuncSetAttribute((const void*)k_attn_dkv<T, DP, KS>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    k_attn_dkv<T, DP, KS><<<(unsigned)xcd_blocks(p.items * p.HK * p.splits), 64 * S::NW, S::LDS, st>>>(p);
    return hipGetLastError();
}

template <typename T, int DP>
hipError_t grad_width(const AttnArgs& a, AttnParams p, hipStream_t st) {
    const auto sum = [&](const int32_t* offs, const int32_t* order, int64_t n, int heads, SumOut a, SumOut b) {
        const int64_t quads = n * heads * (p.D / 4);
        k_attn_sum<T><<<dim3((unsigned)((quads + 255) / 256), b.t ? 2 : 1), 256, 0, st>>>(
            p.part, p.splits, offs, p.B, order, n, heads, p.D, a, b);
        return hipGetLastError();
    };
    hipError_t e = hipSuccess;
    if (p.N > 0) {
        const Plan r = dq_plan(a);
        p.splits = r.splits;
        e = r.ks ? dq_go<T, DP, true>(p, st) : dq_go<T, DP, false>(p, st);
        if (e == hipSuccess && r.splits > 1)
            e = sum(p.offsets, p.order, p.N, p.H, {p.dq, p.dqs[0], p.dqs[1]}, {});
        if (e != hipSuccess) return e;
    }
    if (p.M > 0) {
        const Plan r = dkv_plan(a);
        p.splits = r.splits;
        e = r.ks ? dkv_go<T, DP, true>(p, st) : dkv_go<T, DP, false>(p, st);
        if (e == hipSuccess && r.splits > 1)
            e = sum(p.koffsets ? p.koffsets : p.offsets, p.korder, p.M, p.HK, {p.dk, p.dks[0], p.dks[1]},
                    {p.dv, p.dvs[0], p.dvs[1]});
    }
    return e;
}
template <typename T>
hipError_t grad_type(const AttnArgs& a, const AttnParams& p, hipStream_t st) {
    switch ((p.D + 31) / 32) {
        case 1: return grad_width<T, 32>(a, p, st);
        case 2: return grad_width<T, 64>(a, p, st);
        case 3: return grad_width<T, 96>(a, p, st);
        default: return grad_width<T, 128>(a, p, st);
    }
}

}  // namespace

bool attn_grad_fits(const AttnArgs& a) {
    const auto fits = [&](const Plan& r, int64_t n, int64_t per) {
        return attn_threads_fit(attn_places(n, per, r.ks ? 32 : 128, a.B) * a.HK * r.splits);
    };
    return fits(dq_plan(a), a.N, a.H / a.HK) && fits(dkv_plan(a), a.M, 1);
}
size_t attn_grad_workspace_bytes(const AttnArgs& a) {
    const Plan q = dq_plan(a), k = dkv_plan(a);
    size_t part = 0;
    if (q.splits > 1) part = (size_t)q.splits * a.N * a.H * a.D * 4;
    if (k.splits > 1) part = std::max(part, (size_t)k.splits * a.M * a.HK * a.D * 8);
    return delta_bytes(a) + align_up(part, 256);
}

hipError_t launch_attn_grad(const AttnArgs& a, hipStream_t stream) {
    AttnParams p = attn_params(a);
    p.delta = (float*)a.workspace;
    p.part = (float*)((uint8_t*)a.workspace + delta_bytes(a));
    return a.dtype == SPCONV_BF16 ? grad_type<__bf16>(a, p, stream) : grad_type<float>(a, p, stream);
}

}  // namespace spc
