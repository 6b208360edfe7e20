// Gated linear recurrence over the voxels of each scene, in a given order, and
// its gradient, for gfx950.
//
//   h[t] = f[t] h[t-1] + (1 - f[t]) x[t],   f = sigmoid(z)
//
// Each step is the affine map s -> f s + v, and maps compose:
// (F2, V2) after (F1, V1) is (F2 F1, F2 V1 + V2).  So the sequence is cut into
// chunks, one per workgroup, the chunks into segments of consecutive rows that
// one lane walks for four channels; segments are joined by a scan over the
// lanes and waves, chunks through the chain of their maps (see Chain).  A scene's first row forgets what came before: its
// map is marked F = kForget, and composing selects instead of multiplying, so
// infinities and NaN of one scene stay in it.
//
// The gradient runs the same maps backwards: with g[t] the derivative at h[t],
//   y[t] = f[t] g[t]                what row t hands to row t - 1
//   g[t] = dout[t] + y[t+1]         (0 from another scene)
//   dx = (1 - f) g,   dz = g (h[t-1] - x) f (1 - f),   dh0 = y[first]
// i.e. s -> f s + f dout from the last row to the first.
//
// With e = exp(-|z|), the smaller of f and 1 - f is e / (1 + e), in its own
// relative precision, and the larger is one minus it: rounded once and without
// a bias (the reciprocal's would add up over the thousands of steps that an
// open gate remembers).  States, maps and sums are fp32.
#include "rowops.h"

#include <algorithm>
#include <type_traits>

namespace spc {

namespace {

constexpr int kScanThreads = 512;
constexpr int kScanWaves = kScanThreads / 64;
constexpr float kForget = -1.f;      // F of a map that forgets the state; real F are in [0, 1]
constexpr int kScanV = 4;            // channels per lane
// Lanes per row, at most: 128 channels per workgroup.  Four channels per lane
// (8-byte pieces in bfloat16) rather than a full 16 bytes: a lane's registers
// then hold twice the rows, and joining the segments costs half as much for
// each element.
constexpr int kScanGroup = 32;
constexpr int kScanRows = 8;         // rows per lane, forward
constexpr int kScanGradRows = 4;     // and gradient, which holds more of each

struct Step {
    float f, n;      // sigmoid(z), sigmoid(-z)
};
__device__ __forceinline__ Step gate(float z) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896f * fabsf(z));
    const float small = e * __builtin_amdgcn_rcpf(1.f + e), big = 1.f - small;
    return {z >= 0.f ? big : small, z >= 0.f ? small : big};
}

struct Map {
    float F, V;
};
// b after a
__device__ __forceinline__ Map after(Map b, Map a) {
    Map r;
    r.V = b.F < 0.f ? b.V : fmaf(b.F, a.V, b.V);
    r.F = b.F < 0.f || a.F < 0.f ? kForget : b.F * a.F;
    return r;
}
__device__ __forceinline__ float apply(Map m, float s) { return m.F < 0.f ? m.V : fmaf(m.F, s, m.V); }

struct ScanParams {
    const void* x;
    const void* z;
    const void* dout;
    const int32_t* offsets;
    const int32_t* order;
    const float* h0;
    const float* dlast;
    void* h;           // forward: h; gradient: dx
    void* dz;
    float* last;       // forward: the scenes' last states; gradient: dh0
    float* carry;      // gradient: [its chunks][C] state that enters the chunk
    uint64_t* words;   // chunk maps by level (see Chain); NULL: one chunk
    uint32_t* ticket;  // [channel tiles] chunks handed out
    int64_t N;
    int C, scenes;
    int64_t chunks;
};

// Four elements of a row, aligned to their element.
typedef __bf16 bf16x4s_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4su_t __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
struct Quad;
template <>
struct Quad<__bf16> {
    typedef bf16x4s_t vec;
    typedef bf16x4su_t uvec;
};
template <>
struct Quad<float> {
    typedef f32x4r_t vec;
    typedef f32x4ru_t uvec;
};
template <typename T>
__device__ __forceinline__ typename Quad<T>::vec load_quad(const T* p, int n, float other) {
    typename Quad<T>::vec v;
    if (n >= kScanV) {
        v = *(const typename Quad<T>::uvec*)p;
    } else {
#pragma unroll
        for (int i = 0; i < kScanV; ++i) v[i] = i < n ? p[i] : (T)other;
    }
    return v;
}
template <typename T>
__device__ __forceinline__ void store_quad(T* p, const float (&f)[kScanV], int n) {
    typename Quad<T>::vec v;
#pragma unroll
    for (int i = 0; i < kScanV; ++i) v[i] = (T)f[i];
    if (n >= kScanV) {
        *(typename Quad<T>::uvec*)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < kScanV; ++i)
            if (i < n) p[i] = v[i];
    }
}

// ---- the chain ------------------------------------------------------------
// The chunks' maps, in one pass over the rows: each workgroup takes the next
// chunk, publishes the chunk's map, and composes the maps of all chunks before
// it.  So that this is few loads and always the same composition (whichever
// chunks were ready first), every 16 maps of a level are also published
// composed, as one map of the level above, by the workgroup of the last of
// them: chunk i reads the maps before its own on each level, at most 15 per
// level below the top.  A chunk waits only for chunks handed out before it,
// each of which publishes level 0 without waiting, so every wait ends.
// A map is one 64-bit word (F low, V high), written and read whole by relaxed
// device-scope accesses: no fences.  kNoWord, which a kernel before this one
// fills in, marks a word not written yet; its F is a NaN that publishing never
// writes.
constexpr int kChainLog2 = 4;                  // log2 of the maps joined per level
constexpr int kChainMask = (1 << kChainLog2) - 1;
constexpr int kChainLevels = 4;
constexpr uint64_t kNoWord = ~0ull;

__host__ __device__ __forceinline__ int chain_top(int64_t chunks) {
    int k = 0;
    while (k + 1 < kChainLevels && (chunks >> (kChainLog2 * (k + 1))) > 0) ++k;
    return k;
}
// first entry of level k; chain_at(chunks, chain_top + 1): all entries
__host__ __device__ __forceinline__ int64_t chain_at(int64_t chunks, int k) {
    int64_t at = 0;
    for (int j = 0; j < k; ++j) at += chunks >> (kChainLog2 * j);
    return at;
}

__device__ __forceinline__ void publish(uint64_t* w, Map m) {
    const uint32_t F = m.F == m.F ? __float_as_uint(m.F) : 0x7FC00000u;
    __hip_atomic_store(w, ((uint64_t)__float_as_uint(m.V) << 32) | F, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* w) {
    return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The maps w[0], w[stride], ... (n of them) composed after m; waits for those
// not published yet.  Eight loads are in flight at a time.
__device__ __forceinline__ Map compose_words(const uint64_t* w, int64_t stride, int n, Map m) {
    constexpr int B = 8;
    for (int a = 0; a < n; a += B) {
        uint64_t v[B];
#pragma unroll
        for (int k = 0; k < B; ++k) v[k] = a + k < n ? peek(w + (a + k) * stride) : 0;
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (a + k >= n) break;
            while (v[k] == kNoWord) {
                __builtin_amdgcn_s_sleep(1);
                v[k] = peek(w + (a + k) * stride);
            }
            m = after(Map{__uint_as_float((uint32_t)v[k]), __uint_as_float((uint32_t)(v[k] >> 32))}, m);
        }
    }
    return m;
}

// Publishes chunk i's map of channel c, and with it the maps of the groups
// that chunk i completes.
__device__ __forceinline__ void chain_publish(const ScanParams& p, int64_t i, int c, Map m) {
    const int top = chain_top(p.chunks);
    int64_t at = 0, n = p.chunks;
    publish(p.words + i * p.C + c, m);
    for (int k = 0; k < top && (i & kChainMask) == kChainMask; ++k) {
        m = after(m, compose_words(p.words + (at + i - kChainMask) * p.C + c, p.C, kChainMask, {1.f, 0.f}));
        at += n;
        n >>= kChainLog2;
        i >>= kChainLog2;
        publish(p.words + (at + i) * p.C + c, m);
    }
}

// The state that enters chunk i, into state[0 .. CT): the maps before it,
// oldest first (the top level's, then each lower level's within the group),
// shared by the workgroup's lanes of a channel.  Ends with a barrier.
template <int CT>
__device__ __forceinline__ void chain_state(const ScanParams& p, int64_t i, Map* join, float* state) {
    constexpr int P = kScanThreads / CT;
    const int cl = threadIdx.x % CT, part = threadIdx.x / CT;
    const int c = blockIdx.y * CT + cl;
    const int top = chain_top(p.chunks);
    int64_t total = i >> (kChainLog2 * top);
    for (int k = 0; k < top; ++k) total += (i >> (kChainLog2 * k)) & kChainMask;
    const int64_t per = (total + P - 1) / P;
    const int64_t e0 = min(total, part * per), e1 = min(total, e0 + per);
    Map m = {1.f, 0.f};
    if (c < p.C) {
        int64_t seen = 0;
        for (int k = top; k >= 0; --k) {
            const int64_t idx = i >> (kChainLog2 * k);
            const int64_t first = k == top ? 0 : idx & ~(int64_t)kChainMask, count = idx - first;
            const int64_t a = max(e0 - seen, (int64_t)0), b = min(e1 - seen, count);
            if (a < b)
                m = compose_words(p.words + (chain_at(p.chunks, k) + first + a) * p.C + c, p.C, (int)(b - a), m);
            seen += count;
        }
    }
    join[part * CT + cl] = m;
    __syncthreads();
    if (part == 0) {
        float s = 0.f;
        for (int q = 0; q < P; ++q) s = apply(join[q * CT + cl], s);
        state[cl] = s;
    }
    __syncthreads();
}

// Before a chained kernel: no map published, no chunk handed out.
__global__ void __launch_bounds__(256) k_scan_clear(uint64_t* words, int64_t n, uint32_t* ticket, int tiles) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t e = t; e < n; e += (int64_t)gridDim.x * 256) words[e] = kNoWord;
    if (t < tiles) ticket[t] = 0;
}

// The chunk this workgroup takes, in its direction's order.
__device__ __forceinline__ int64_t next_chunk(const ScanParams& p) {
    if (!p.words) return 0;
    __shared__ uint32_t got;
    if (threadIdx.x == 0) got = atomicAdd(p.ticket + blockIdx.y, 1u);
    __syncthreads();
    return got;
}

// ---- scenes ---------------------------------------------------------------
// Which rows of a chunk begin and end a scene, as scene numbers (-1: none).
template <int R>
struct SceneMarks {
    int first[R], last[R];
};

// Marks of the chunk of rows [p0, p0 + R).  Offsets are only compared: a bad
// one marks a wrong row or none, never memory outside the marks.
template <int R>
__device__ __forceinline__ void mark_scenes(SceneMarks<R>& m, const ScanParams& p, int64_t p0) {
    for (int i = threadIdx.x; i < R; i += kScanThreads) m.first[i] = m.last[i] = -1;
    __syncthreads();
    int b0 = 0;
    if (p.scenes > 2 * kScanThreads) {
        // from the last scene that begins before p0
        int lo = 0, hi = p.scenes;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (p.offsets[mid] < p0) lo = mid + 1; else hi = mid;
        }
        b0 = max(lo - 1, 0);
    }
    for (int b = b0 + threadIdx.x; b < p.scenes; b += kScanThreads) {
        const int64_t lo = p.offsets[b], hi = p.offsets[b + 1];
        if (lo >= p0 + R) break;
        if (hi <= lo) continue;
        if (lo >= p0) m.first[lo - p0] = b;
        if (hi > p0 && hi <= p0 + R) m.last[hi - 1 - p0] = b;
    }
    __syncthreads();
}

// Whether some row of this wave's segments begins or ends a scene.
template <int L, int R>
__device__ __forceinline__ bool wave_marks(const SceneMarks<R>& m, int seg) {
    int any = 0;
#pragma unroll
    for (int l = 0; l < L; ++l) any |= (m.first[seg * L + l] >= 0) | (m.last[seg * L + l] >= 0);
    return __any(any);
}

// Scenes without rows: their state is what came in.  The lanes of the grid
// share the scenes; one writes its scene's channels alone (they are few).
__device__ __forceinline__ void empty_scenes(const ScanParams& p, const float* in, float* out, int channels) {
    const int c0 = blockIdx.y * channels, c1 = min(p.C, c0 + channels);
    for (int64_t b = (int64_t)blockIdx.x * kScanThreads + threadIdx.x; b < p.scenes;
         b += (int64_t)gridDim.x * kScanThreads) {
        if (p.offsets[b + 1] > p.offsets[b]) continue;
        for (int c = c0; c < c1; ++c) out[b * p.C + c] = in ? in[b * p.C + c] : 0.f;
    }
}

// ---- rows and segments ----------------------------------------------------
// The caller's rows of a segment's positions; -1 for positions past the end or
// an order value outside the rows (such a row is neither read nor written and
// hands the state on).
template <int L>
__device__ __forceinline__ void segment_rows(const ScanParams& p, int64_t pos, int (&row)[L]) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
        int64_t r = pos + l;
        if (r < p.N && p.order) r = (uint32_t)p.order[r];
        row[l] = r < p.N ? (int)r : -1;
    }
}

// A scan of the lanes' maps over the workgroup's segments.  Within a wave
// here: m becomes the composition of the wave's segments before the lane's own
// (BACK: behind it), the whole wave's goes to wave_maps[wave][channel].
template <int G, bool BACK>
__device__ __forceinline__ void scan_wave(Map (&m)[kScanV], Map* wave_maps) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane % G;
    const int seg = BACK ? 64 / G - 1 - lane / G : lane / G;     // position within the wave's order
#pragma unroll
    for (int d = 1; d < 64 / G; d *= 2) {
#pragma unroll
        for (int i = 0; i < kScanV; ++i) {
            const Map a = {BACK ? __shfl_down(m[i].F, d * G) : __shfl_up(m[i].F, d * G),
                           BACK ? __shfl_down(m[i].V, d * G) : __shfl_up(m[i].V, d * G)};
            const Map r = after(m[i], a);
            if (seg >= d) m[i] = r;
        }
    }
#pragma unroll
    for (int i = 0; i < kScanV; ++i) {
        if (seg == 64 / G - 1) wave_maps[wave * (G * kScanV) + c * kScanV + i] = m[i];
        m[i] = {BACK ? __shfl_down(m[i].F, G) : __shfl_up(m[i].F, G),
                BACK ? __shfl_down(m[i].V, G) : __shfl_up(m[i].V, G)};
        if (seg == 0) m[i] = {1.f, 0.f};
    }
}
// Over the waves, by one lane per channel after a barrier: wave_maps become
// the compositions of the waves before; returns the workgroup's.
template <int CT, bool BACK>
__device__ __forceinline__ Map scan_waves(Map* wave_maps, int c) {
    Map all = {1.f, 0.f};
#pragma unroll
    for (int k = 0; k < kScanWaves; ++k) {
        Map* w = wave_maps + (BACK ? kScanWaves - 1 - k : k) * CT + c;
        const Map m = *w;
        *w = all;
        all = after(m, all);
    }
    return all;
}

// The states.  STATES false: only the states that enter the gradient's chunks
// (two of them to one of these), into carry.
template <typename T, int G, bool STATES>
__global__ void __launch_bounds__(kScanThreads, 4) k_scan(ScanParams p) {
    constexpr int V = kScanV, L = kScanRows, S = kScanThreads / G, R = S * L, CT = G * V;
    __shared__ SceneMarks<R> marks;
    __shared__ Map wave_maps[kScanWaves * CT], join[kScanThreads];
    __shared__ float state[CT];
    const int64_t chunk = next_chunk(p), p0 = chunk * R;
    const int lane = threadIdx.x % G, seg = threadIdx.x / G;
    const int c0 = (blockIdx.y * G + lane) * V, nv = p.C - c0;
    int row[L];
    segment_rows<L>(p, p0 + seg * L, row);
    typename Quad<T>::vec x[L], z[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int64_t at = (int64_t)row[l] * p.C + c0;
        // a row that is not there: f = 1, 1 - f = 0
        z[l] = load_quad((const T*)p.z + at, row[l] >= 0 ? nv : 0, __builtin_inff());
        x[l] = load_quad((const T*)p.x + at, row[l] >= 0 ? nv : 0, 0.f);
    }
    mark_scenes(marks, p, p0);
    const bool marked = wave_marks<L>(marks, seg);
    constexpr int LK = STATES ? L : 1;
    Map m[LK][V], pre[V];       // m[l]: the segment's rows 0 .. l composed
    auto compose = [&](auto mk) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[seg * L + l] : -1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step s = gate((float)z[l][i]);
                const float v = s.n * (float)x[l][i];
                const Map was = l ? m[STATES ? l - 1 : 0][i] : Map{1.f, 0.f};
                Map now;
                if (decltype(mk)::value) {
                    now = after({s.f, v}, was);
                    if (b >= 0) {
                        const float in = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
                        now = {kForget, fmaf(s.f, in, v)};
                    }
                } else {
                    now = l ? Map{s.f * was.F, fmaf(s.f, was.V, v)} : Map{s.f, v};
                }
                m[STATES ? l : 0][i] = now;
            }
        }
    };
    if (marked)
        compose(std::true_type{});
    else
        compose(std::false_type{});
#pragma unroll
    for (int i = 0; i < V; ++i) pre[i] = m[LK - 1][i];
    scan_wave<G, false>(pre, wave_maps);
    __syncthreads();
    if (threadIdx.x < CT) {
        const Map all = scan_waves<CT, false>(wave_maps, threadIdx.x);
        const int c = blockIdx.y * CT + threadIdx.x;
        if (p.words && c < p.C) chain_publish(p, chunk, c, all);
    }
    if (p.words)
        chain_state<CT>(p, chunk, join, state);
    else
        __syncthreads();
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = apply(wave_maps[(threadIdx.x >> 6) * CT + lane * V + i], p.words ? state[lane * V + i] : 0.f);
        s[i] = apply(pre[i], s[i]);
    }
    if constexpr (!STATES) {
        if (seg == 0 || seg == S / 2) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < nv) p.carry[(2 * chunk + (seg ? 1 : 0)) * p.C + c0 + i] = s[i];
        }
        return;
    }
#pragma unroll
    for (int l = 0; l < LK; ++l) {
        float o[V];
        if (marked) {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = apply(m[l][i], s[i]);
            const int e = marks.last[seg * L + l];
            if (e >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < nv) p.last[(int64_t)e * p.C + c0 + i] = o[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf(m[l][i].F, s[i], m[l][i].V);
        }
        if (row[l] >= 0) store_quad((T*)p.h + (int64_t)row[l] * p.C + c0, o, nv);
    }
    empty_scenes(p, p.h0, p.last, CT);
}

// The gradient, from the last chunk to the first, with the states that enter
// the chunks known (carry; NULL: one chunk).
template <typename T, int G>
__global__ void __launch_bounds__(kScanThreads, 4) k_scan_grad(ScanParams p) {
    constexpr int V = kScanV, L = kScanGradRows, S = kScanThreads / G, R = S * L, CT = G * V;
    __shared__ SceneMarks<R> marks;
    __shared__ Map wave_maps[2][kScanWaves * CT], join[kScanThreads];
    __shared__ float state[CT];
    const int64_t back = next_chunk(p), chunk = p.chunks - 1 - back, p0 = chunk * R;
    const int lane = threadIdx.x % G, seg = threadIdx.x / G;
    const int c0 = (blockIdx.y * G + lane) * V, nv = p.C - c0;
    int row[L];
    segment_rows<L>(p, p0 + seg * L, row);
    typename Quad<T>::vec x[L], z[L], d[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int64_t at = (int64_t)row[l] * p.C + c0;
        z[l] = load_quad((const T*)p.z + at, row[l] >= 0 ? nv : 0, __builtin_inff());
        x[l] = load_quad((const T*)p.x + at, row[l] >= 0 ? nv : 0, 0.f);
        d[l] = load_quad((const T*)p.dout + at, row[l] >= 0 ? nv : 0, 0.f);
    }
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = p.carry && i < nv ? p.carry[chunk * p.C + c0 + i] : 0.f;
    mark_scenes(marks, p, p0);
    const bool marked = wave_marks<L>(marks, seg);
    Map m[V], mb[V];
    float f[L][V], n[L][V], dh[L][V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = mb[i] = {1.f, 0.f};
    auto compose = [&](auto mk) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[seg * L + l] : -1;
            const int e = decltype(mk)::value ? marks.last[seg * L + l] : -1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step g = gate((float)z[l][i]);
                const float v = g.n * (float)x[l][i];
                f[l][i] = g.f;
                n[l][i] = g.n;
                float t = (float)d[l][i];
                if (decltype(mk)::value) {
                    if (e >= 0 && p.dlast && i < nv) t += p.dlast[(int64_t)e * p.C + c0 + i];
                    if (b >= 0) {
                        const float in = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
                        m[i] = {kForget, fmaf(g.f, in, v)};
                        mb[i] = after(mb[i], {kForget, 0.f});
                    } else {
                        m[i] = after({g.f, v}, m[i]);
                        mb[i] = after(mb[i], {g.f, g.f * t});
                    }
                } else {
                    mb[i].V = fmaf(m[i].F, g.f * t, mb[i].V);
                    m[i] = {g.f * m[i].F, fmaf(g.f, m[i].V, v)};
                }
                dh[l][i] = t;
            }
        }
        if (!decltype(mk)::value) {
#pragma unroll
            for (int i = 0; i < V; ++i) mb[i].F = m[i].F;
        }
    };
    if (marked)
        compose(std::true_type{});
    else
        compose(std::false_type{});
    scan_wave<G, true>(mb, wave_maps[1]);
    scan_wave<G, false>(m, wave_maps[0]);
    __syncthreads();
    if (threadIdx.x < CT) {
        const Map all = scan_waves<CT, true>(wave_maps[1], threadIdx.x);
        const int c = blockIdx.y * CT + threadIdx.x;
        if (p.words && c < p.C) chain_publish(p, back, c, all);
    } else if (threadIdx.x < 2 * CT) {
        scan_waves<CT, false>(wave_maps[0], threadIdx.x - CT);
    }
    if (p.words)
        chain_state<CT>(p, back, join, state);
    else
        __syncthreads();
    // forward: the states again, and (h[t-1] - x) f (1 - f)
    float y[V], q[L][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = (threadIdx.x >> 6) * CT + lane * V + i;
        s[i] = apply(m[i], apply(wave_maps[0][at], s[i]));
        y[i] = apply(mb[i], apply(wave_maps[1][at], p.words ? state[lane * V + i] : 0.f));
    }
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int b = marked ? marks.first[seg * L + l] : -1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xv = (float)x[l][i];
            if (b >= 0) s[i] = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
            q[l][i] = (s[i] - xv) * (f[l][i] * n[l][i]);
            s[i] = fmaf(f[l][i], s[i], n[l][i] * xv);
        }
    }
#pragma unroll
    for (int l = L - 1; l >= 0; --l) {
        const int b = marked ? marks.first[seg * L + l] : -1;
        float ox[V], oz[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float gt = dh[l][i] + y[i];
            ox[i] = n[l][i] * gt;
            oz[i] = q[l][i] * gt;
            y[i] = f[l][i] * gt;
        }
        if (b >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (p.last && i < nv) p.last[(int64_t)b * p.C + c0 + i] = y[i];
                y[i] = 0.f;
            }
        }
        if (row[l] >= 0) {
            const int64_t at = (int64_t)row[l] * p.C + c0;
            store_quad((T*)p.h + at, ox, nv);
            store_quad((T*)p.dz + at, oz, nv);
        }
    }
    if (p.last) empty_scenes(p, p.dlast, p.last, CT);
}

// Lanes per row: enough for its channels, kScanGroup at most (wider rows take
// several workgroups).
int scan_group(int C) {
    int G = 1;
    while (G < kScanGroup && G * kScanV < C) G *= 2;
    return G;
}
int64_t scan_chunks(int64_t N, int C, bool grad) {
    const int64_t R = (int64_t)(kScanThreads / scan_group(C)) * (grad ? kScanGradRows : kScanRows);
    return std::max<int64_t>(1, (N + R - 1) / R);
}
// Workspace: the words of the longer chain (the gradient runs two, one after
// the other), the tickets, the gradient's entering states.
struct ScanLayout {
    int64_t chunks, gchunks;     // of the forward and of the gradient
    int tiles;
    size_t ticket, carry, total;
};
int64_t chain_entries(int64_t chunks) { return chain_at(chunks, chain_top(chunks) + 1); }
ScanLayout scan_layout(int64_t N, int C, bool grad) {
    static_assert(kScanRows == 2 * kScanGradRows, "two chunks of the gradient to one of the forward");
    ScanLayout l{};
    l.chunks = scan_chunks(N, C, false);
    l.gchunks = scan_chunks(N, C, true);
    l.tiles = (C + scan_group(C) * kScanV - 1) / (scan_group(C) * kScanV);
    const int64_t n = grad ? l.gchunks : l.chunks;
    if (n == 1) return l;
    l.ticket = align_up((size_t)chain_entries(n) * C * 8, 256);
    l.carry = l.ticket + align_up((size_t)l.tiles * 4, 256);
    l.total = l.carry + (grad ? align_up((size_t)2 * l.chunks * C * 4, 256) : 0);
    return l;
}

template <typename T, int G>
hipError_t scan_go(ScanParams p, bool grad, const ScanLayout& l, char* ws, hipStream_t st) {
    auto chain = [&](int64_t chunks) {
        p.chunks = chunks;
        p.words = chunks > 1 ? (uint64_t*)ws : nullptr;
        p.ticket = chunks > 1 ? (uint32_t*)(ws + l.ticket) : nullptr;
        if (chunks == 1) return;
        const int64_t n = chain_entries(chunks) * p.C;
        k_scan_clear<<<(unsigned)std::min<int64_t>((n + 1023) / 1024, 2048), 256, 0, st>>>(p.words, n, p.ticket,
                                                                                           l.tiles);
    };
    if (grad) {
        if (l.gchunks > 1) {
            p.carry = (float*)(ws + l.carry);
            chain(l.chunks);
            k_scan<T, G, false><<<dim3((unsigned)l.chunks, l.tiles), kScanThreads, 0, st>>>(p);
        }
        chain(l.gchunks);
        k_scan_grad<T, G><<<dim3((unsigned)l.gchunks, l.tiles), kScanThreads, 0, st>>>(p);
    } else {
        chain(l.chunks);
        k_scan<T, G, true><<<dim3((unsigned)l.chunks, l.tiles), kScanThreads, 0, st>>>(p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t scan_dispatch(const ScanParams& p, bool grad, char* ws, hipStream_t st) {
    const ScanLayout l = scan_layout(p.N, p.C, grad);
    switch (scan_group(p.C)) {
        case 1: return scan_go<T, 1>(p, grad, l, ws, st);
        case 2: return scan_go<T, 2>(p, grad, l, ws, st);
        case 4: return scan_go<T, 4>(p, grad, l, ws, st);
        case 8: return scan_go<T, 8>(p, grad, l, ws, st);
        case 16: return scan_go<T, 16>(p, grad, l, ws, st);
        default: return scan_go<T, 32>(p, grad, l, ws, st);
    }
}

}  // namespace

size_t scan_workspace_bytes(int64_t N, int C, int, bool grad) { return scan_layout(N, C, grad).total; }

hipError_t launch_scan(const ScanArgs& a, bool grad, hipStream_t stream) {
    ScanParams p{};
    p.x = a.x;
    p.z = a.z;
    p.dout = a.dout;
    p.offsets = a.offsets;
    p.order = a.order;
    p.h0 = a.h0;
    p.dlast = a.dlast;
    p.h = a.out;
    p.dz = a.dz;
    p.last = a.state;
    p.N = a.N;
    p.C = a.C;
    p.scenes = a.scenes;
    char* ws = (char*)a.workspace;
    return a.dtype == SPCONV_BF16 ? scan_dispatch<__bf16>(p, grad, ws, stream) : scan_dispatch<float>(p, grad, ws, stream);
}

}  // namespace spc
