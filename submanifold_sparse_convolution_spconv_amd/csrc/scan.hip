// Gated linear recurrence over the voxels of each scene, in a given order, and
// its gradient, for gfx950.
//
//   h[t] = f[t] h[t-1] + (1 - f[t]) x[t],   f = sigmoid(z)
//
// Each step is the affine map s -> f s + v, and maps compose:
// (F2, V2) after (F1, V1) is (F2 F1, F2 V1 + V2).  So the sequence is cut into
// chunks, one per workgroup, the chunks into segments of consecutive rows that
// one lane walks for four channels; segments are joined by a scan over the
// lanes and waves.  Long sequences take several kernels, none of which waits
// for another workgroup: the chunks' maps, the states that enter the chunks
// (composed from the maps in a fixed order), and the rows again with those
// states.  A scene's first row forgets what came before: its
// map is marked F = kForget, and composing selects instead of multiplying, so
// infinities and NaN of one scene stay in it.  Products of factors above zero
// stay above zero (the smallest number where they would underflow), so that an
// infinite state stays infinite through a composed map as it does step by step.
//
// The gradient runs the same maps backwards: with g[t] the derivative at h[t],
//   y[t] = f[t] g[t]                what row t hands to row t - 1
//   g[t] = dout[t] + y[t+1]         (0 from another scene)
//   dx = (1 - f) g,   dz = g (h[t-1] - x) f (1 - f),   dh0 = y[first]
// i.e. s -> f s + f dout from the last row to the first.
//
// With e = exp(-|z|), the smaller of f and 1 - f is e / (1 + e), in its own
// relative precision, and the larger is one minus it.  That is rounded once, to a
// multiple of 2^-24 below one: over varying gates to either side (a reciprocal's
// error would lean to one), but a gate that stays open at one value repeats its
// error at every step.  Then 1 - f, as the state decays, is off by up to 2^-25: 3%
// of it at z = 15, 44% at 17 (f = 1 - 2^-24), all of it from 17.4 on (f = 1); and a
// state kept for t steps by up to t 2^-24 of itself, the products' rounding
// included (0.5% after 300,000 steps at z = 17).  States, maps and sums are fp32.
//
// Long sequences are bound by memory, at the price of reading the rows twice:
// 1,006,716 x 128 bf16 takes 274 to 288 us forward, card by card (1.29 GB, 4.5 to 4.7
// TB/s), and 472 to 490 us for the gradient (2.06 GB, 4.2 to 4.4 TB/s).  Workgroups that keep their rows and wait for the
// states before them took 323 and 867 us.  Short sequences are a chain of reads:
// 64 scenes of one row, 7.6 us.
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
// Rows per lane, forward: eight, or for short sequences, whose time is a lane's
// own, four where chunks are few (no groups of them, or not two per CU), and two
// where one chunk has all rows (3,000 x 128: 18.5 us with eight, 15.6 with four).  Gradient, which holds more of each: four.
constexpr int kScanRows = 8, kScanRowsShort = 4, kScanRowsOne = 2;
constexpr int kScanGradRows = 4;

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
// b after a.  A product that would round to 0 without a factor of 0 becomes the
// smallest number, 2^-149: 0 times an infinite state would be NaN.
__device__ __forceinline__ Map after(Map b, Map a) {
    Map r;
    r.V = b.F < 0.f ? b.V : fmaf(b.F, a.V, b.V);
    r.F = b.F < 0.f || a.F < 0.f ? kForget : fmaxf(b.F * a.F, fminf(fminf(b.F, a.F), 0x1p-149f));
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
    int64_t N;
    int C, scenes, tiles;
    int64_t chunks;
    bool stream;       // outputs past the caches
    // [directions][chunks][C] maps of the chunks, first to last and (gradient) last to
    // first; the same of groups of chunks; the states that enter the chunks
    Map* maps;
    Map* groups;
    float* carry;
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
// Rows of a multiple of four channels: a lane has four or none.  Of more than
// four: the last lane may have fewer; it reads the row's last four and moves its
// own to the front.  Of fewer than four: one by one.
enum RowEnd { kWholeQuads, kCutQuad, kSingles };
template <typename Q>
__device__ __forceinline__ Q move_down(Q q, int s) {
    if constexpr (sizeof(Q) == 8) {
        uint64_t w;
        __builtin_memcpy(&w, &q, 8);
        w >>= 16 * s;
        __builtin_memcpy(&q, &w, 8);
    } else {
        const Q one = __builtin_shufflevector(q, q, 1, 2, 3, 3);
#pragma unroll
        for (int i = 0; i < kScanV; ++i) q[i] = s & 1 ? one[i] : q[i];
        const Q two = __builtin_shufflevector(q, q, 2, 3, 3, 3);
#pragma unroll
        for (int i = 0; i < kScanV; ++i) q[i] = s & 2 ? two[i] : q[i];
    }
    return q;
}
// The load is the same instruction in every lane (a missing row's or channel's
// reads row 0 or channel 0 instead), so that all of a segment's are in flight
// together; a branch around each would end that.  Channels past the row's end
// get some value.
template <typename T, RowEnd END>
__device__ __forceinline__ typename Quad<T>::vec load_quad(const T* base, int row, int C, int c0) {
    const int n = C - c0;
    const T* p = base + (int64_t)max(row, 0) * C;
    typename Quad<T>::vec v;
    if constexpr (END == kSingles) {
#pragma unroll
        for (int i = 0; i < kScanV; ++i) v[i] = p[min(c0 + i, C - 1)];
    } else {
        v = *(const typename Quad<T>::uvec*)(p + (n > 0 ? min(c0, C - kScanV) : 0));
        if constexpr (END == kCutQuad) v = move_down(v, n > 0 ? max(kScanV - n, 0) : 0);
    }
    return v;
}
template <typename T, RowEnd END>
__device__ __forceinline__ void store_quad(T* base, int row, int C, int c0, const float (&f)[kScanV], bool stream) {
    const int n = row >= 0 ? C - c0 : 0;
    T* p = base + (int64_t)row * C + c0;
    typename Quad<T>::vec v;
#pragma unroll
    for (int i = 0; i < kScanV; ++i) v[i] = (T)f[i];
    if (END != kSingles && n >= kScanV) {
        typename Quad<T>::uvec* q = (typename Quad<T>::uvec*)p;
        if (stream)
            __builtin_nontemporal_store((typename Quad<T>::uvec)v, q);
        else
            *q = v;
    } else if (END != kWholeQuads) {
#pragma unroll
        for (int i = 0; i < kScanV; ++i)
            if (i < n) p[i] = v[i];
    }
}

// The value, as new to the compiler: what was computed from it before is then
// computed again instead of being kept in registers.
template <typename Q>
__device__ __forceinline__ void forget_uses(Q& q) {
    uint32_t w[sizeof(Q) / 4];
    __builtin_memcpy(w, &q, sizeof q);
#pragma unroll
    for (unsigned i = 0; i < sizeof(Q) / 4; ++i) asm volatile("" : "+v"(w[i]));
    __builtin_memcpy(&q, w, sizeof q);
}

// ---- chunks ---------------------------------------------------------------
constexpr int kChunkGroup = 64;       // chunks per group
constexpr int kCarryChannels = 64;    // channels per workgroup of k_scan_groups and k_scan_carry
constexpr int kCarryParts = kScanThreads / kCarryChannels;
constexpr int kCarryPer = kChunkGroup / kCarryParts;

// The maps w[0], w[stride], ... (n of them) composed after m, eight loads at a
// time (the last again where fewer are left: no branch between the loads).
__device__ __forceinline__ Map compose_maps(const Map* w, int64_t stride, int n, Map m) {
    constexpr int B = 8;
    for (int a = 0; a < n; a += B) {
        Map v[B];
#pragma unroll
        for (int k = 0; k < B; ++k) v[k] = w[min(a + k, n - 1) * stride];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const Map r = after(v[k], m);
            if (a + k < n) m = r;
        }
    }
    return m;
}

// The state after the n maps w[0], w[stride], ... from zero, for channel c:
// P lanes of the workgroup compose a share each, joined in order through
// `join` (P * CT maps).  Ends with a barrier; every lane of a channel gets it.
template <int CT>
__device__ __forceinline__ float state_after(const Map* w, int64_t stride, int n, bool live, Map* join) {
    constexpr int P = kScanThreads / CT;
    const int cl = threadIdx.x % CT, part = threadIdx.x / CT;
    const int per = (n + P - 1) / P, a = min(n, part * per), b = min(n, a + per);
    join[part * CT + cl] = live ? compose_maps(w + a * stride, stride, b - a, {1.f, 0.f}) : Map{1.f, 0.f};
    __syncthreads();
    float s = 0.f;
    for (int q = 0; q < P; ++q) s = apply(join[q * CT + cl], s);
    return s;
}

// The chunks of a group as k_scan_groups and k_scan_carry share them: kCarryPer
// for each of the workgroup's parts, all loaded together.
struct CarryChunks {
    Map m[kCarryPer];
    int64_t at, step;      // of the first, from one to the next
    int n;
    __device__ __forceinline__ CarryChunks(const ScanParams& p, bool back, int part, int c, bool live) {
        const int64_t first = (int64_t)blockIdx.x * kChunkGroup;
        const int all = (int)min((int64_t)kChunkGroup, p.chunks - first), a = min(all, part * kCarryPer);
        n = live ? min(kCarryPer, all - a) : 0;
        step = back ? -p.C : p.C;
        at = (back ? p.chunks + first + all - 1 - a : first + a) * p.C + c;
#pragma unroll
        for (int k = 0; k < kCarryPer; ++k) m[k] = k < n ? p.maps[at + k * step] : Map{1.f, 0.f};
    }
    __device__ __forceinline__ Map whole() const {
        Map r = {1.f, 0.f};
#pragma unroll
        for (int k = 0; k < kCarryPer; ++k) r = after(m[k], r);
        return r;
    }
};

// Maps of groups of chunks; blockIdx.z: the direction.
__global__ void __launch_bounds__(kScanThreads) k_scan_groups(ScanParams p) {
    constexpr int CT = kCarryChannels;
    __shared__ Map join[kScanThreads];
    const int cl = threadIdx.x % CT, part = threadIdx.x / CT, c = blockIdx.y * CT + cl;
    const bool back = blockIdx.z;
    join[threadIdx.x] = CarryChunks(p, back, part, c, c < p.C).whole();
    __syncthreads();
    if (part || c >= p.C) return;
    Map m = {1.f, 0.f};
#pragma unroll
    for (int q = 0; q < kCarryParts; ++q) m = after(join[q * CT + cl], m);
    p.groups[((back ? gridDim.x : 0) + blockIdx.x) * (int64_t)p.C + c] = m;
}

// States that enter the chunks of one group: the groups before it, then the
// chunks before each of its own.
__global__ void __launch_bounds__(kScanThreads) k_scan_carry(ScanParams p) {
    constexpr int CT = kCarryChannels;
    __shared__ Map join[kScanThreads], own[kScanThreads];
    const int cl = threadIdx.x % CT, part = threadIdx.x / CT;
    const int c = blockIdx.y * CT + cl;
    const bool back = blockIdx.z, live = c < p.C;
    const Map* g = p.groups + (back ? 2 * (int64_t)gridDim.x - 1 : 0) * p.C + c;
    const int before = back ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x;
    const CarryChunks chunks(p, back, part, c, live);
    own[threadIdx.x] = chunks.whole();
    float s = state_after<CT>(g, back ? -p.C : p.C, before, live, join);
    for (int q = 0; q < part; ++q) s = apply(own[q * CT + cl], s);
#pragma unroll
    for (int k = 0; k < kCarryPer; ++k) {
        if (k < chunks.n) p.carry[chunks.at + k * chunks.step] = s;
        s = apply(chunks.m[k], s);
    }
}

// The state that enters this workgroup's chunk, for its channels: from
// k_scan_carry, or (few chunks: no groups) from the maps.  Ends with a barrier.
template <int CT, bool BACK>
__device__ __forceinline__ void entering_state(const ScanParams& p, int64_t chunk, int tile, Map* join, float* state) {
    const int cl = threadIdx.x % CT, c = tile * CT + cl;
    const int64_t dir = BACK ? p.chunks : 0;
    float s = 0.f;
    if (p.chunks > kChunkGroup) {
        if (threadIdx.x < CT && c < p.C) s = p.carry[(dir + chunk) * p.C + c];
    } else if (p.chunks > 1) {
        const Map* w = p.maps + (dir + (BACK ? p.chunks - 1 : 0)) * p.C + c;
        s = state_after<CT>(w, BACK ? -p.C : p.C, (int)(BACK ? p.chunks - 1 - chunk : chunk), c < p.C, join);
    }
    if (threadIdx.x < CT) state[cl] = s;
    __syncthreads();
}

// The chunk (in the grid's order) and the tile of channels of this workgroup.
// Workgroups go round the 8 XCDs: the tiles of one chunk follow each other on one
// of them, so that the cache lines at their borders are read once (gradient of
// 400,000 x 200 bf16: 519 -> 379 us; of 29,000 x 1,024, whose rows end with their
// lines: 99 -> 106).
struct Place {
    int64_t chunk;
    int tile;
    __device__ __forceinline__ explicit Place(const ScanParams& p) {
        if (p.tiles == 1) {
            chunk = blockIdx.x;
            tile = 0;
        } else {
            // (a quotient is the same in every lane, which the compiler has to be
            // told: as a vector it costs 25 us at 1,006,716 x 128)
            const uint32_t k = blockIdx.x / 8, q = __builtin_amdgcn_readfirstlane(k / p.tiles);
            chunk = (int64_t)q * 8 + blockIdx.x % 8;
            tile = k - q * p.tiles;
        }
    }
};

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

// Scenes without rows: their state is what came in.  A wave looks at 64 scenes
// at once, or at 8 where that reaches all of them, and writes the empty ones.
__device__ __forceinline__ void empty_scenes(const ScanParams& p, Place at, const float* in, float* out, int channels) {
    const int c0 = at.tile * channels, c1 = min(p.C, c0 + channels), lane = threadIdx.x & 63;
    const int64_t waves = p.chunks * kScanWaves;
    const int per = p.scenes <= 8 * waves ? 8 : 64;
    for (int64_t b0 = (at.chunk * kScanWaves + (threadIdx.x >> 6)) * per; b0 < p.scenes; b0 += waves * per) {
        const int64_t b = b0 + lane, i = min(b, (int64_t)p.scenes - 1);
        uint64_t empty = __ballot(lane < per && b < p.scenes && p.offsets[i + 1] <= p.offsets[i]);
        for (; empty; empty &= empty - 1) {
            const int64_t e = b0 + __builtin_ctzll(empty);
            for (int c = c0 + lane; c < c1; c += 64) out[e * p.C + c] = in ? in[e * p.C + c] : 0.f;
        }
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
        const int64_t t = pos + l;
        const uint32_t r = p.order ? (uint32_t)p.order[min(t, p.N - 1)] : (uint32_t)t;
        row[l] = t < p.N && r < p.N ? (int)r : -1;
    }
}

// A row that is not there: f = 1, 1 - f = 0, so the state passes.
template <int L>
__device__ __forceinline__ bool any_missing(const int (&row)[L]) {
    int any = 0;
#pragma unroll
    for (int l = 0; l < L; ++l) any |= row[l];
    return __any(any < 0);
}
template <typename T>
__device__ __forceinline__ void missing_row(int row, typename Quad<T>::vec& z, typename Quad<T>::vec& x) {
    if (row >= 0) return;
#pragma unroll
    for (int i = 0; i < kScanV; ++i) {
        z[i] = (T)__builtin_inff();
        x[i] = (T)0.f;
    }
}

// Whether some gate of a channel is 0 in 32 bits: z below -87.33, where the
// exponential vanishes.  As whole numbers the bits of negative z grow as z falls,
// above those of every other: one maximum for two elements.
template <typename T>
struct Shut {
    typedef std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t> word;
    typedef word vec __attribute__((ext_vector_type(kScanV)));
    static constexpr word kBorder = sizeof(T) == 2 ? (word)0xC2AE : (word)0xC2AEAC50;
    vec most = {};
    __device__ __forceinline__ void add(typename Quad<T>::vec z) {
        vec w;
        __builtin_memcpy(&w, &z, sizeof w);
        most = __builtin_elementwise_max(most, w);
    }
    // Plain products of gates leave 0 for an underflow too: such a factor becomes
    // the smallest number, unless a gate is 0.  True: some factor of the wave was 0.
    __device__ __forceinline__ bool lift(Map (&m)[kScanV]) const {
        int any = 0;
#pragma unroll
        for (int i = 0; i < kScanV; ++i) {
            const bool zero = m[i].F == 0.f;
            any |= zero;
            if (zero && most[i] <= kBorder) m[i].F = 0x1p-149f;
        }
        return __any(any);
    }
};
// Whether a row's gradient met a factor of 0 in the plain products: infinite ones
// have become NaN there.
__device__ __forceinline__ bool any_nan(const Map (&m)[kScanV]) {
    int any = 0;
#pragma unroll
    for (int i = 0; i < kScanV; ++i) any |= m[i].V != m[i].V;
    return __any(any);
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

// Rows whose scenes' states are asked for together (a row at a time, each
// would wait for its own: 64 scenes of one row took 18 us).
template <int L>
constexpr int kSceneRows = L < 4 ? L : 4;

// Rows of a workgroup's chunk, and what its scenes need of them.
template <typename T, int G, int L, RowEnd END>
struct Chunk {
    static constexpr int V = kScanV, S = kScanThreads / G, R = S * L, CT = G * V;
    int lane, seg, c0, nv;
    int64_t p0;
    int row[L];
    __device__ __forceinline__ Chunk(const ScanParams& p, int64_t chunk, int tile) {
        lane = threadIdx.x % G;
        seg = threadIdx.x / G;
        c0 = (tile * G + lane) * V;
        nv = p.C - c0;
        p0 = chunk * R;
        segment_rows<L>(p, p0 + seg * L, row);
    }
    __device__ __forceinline__ typename Quad<T>::vec load(const void* t, int l, int C) const {
        return load_quad<T, END>((const T*)t, row[l], C, c0);
    }
    // The states t of up to four rows' scenes b (0 where a row has none, or
    // without states), all loads in flight together.
    __device__ __forceinline__ void of_scenes(const float* t, const int* b, float (&s)[kSceneRows<L>][V], int C) const {
#pragma unroll
        for (int l = 0; l < kSceneRows<L>; ++l) {
            typename Quad<float>::vec v = {};
            if (t) v = load_quad<float, END>(t, b[l], C, c0);
#pragma unroll
            for (int i = 0; i < V; ++i) s[l][i] = v[i];
        }
    }
};

// Maps of the chunks: first to last, and with GRAD last to first.
template <typename T, int G, int L, RowEnd END, bool GRAD>
__global__ void __launch_bounds__(kScanThreads) k_scan_maps(ScanParams p) {
    using K = Chunk<T, G, L, END>;
    constexpr int V = K::V, SR = kSceneRows<L>;
    __shared__ SceneMarks<K::R> marks;
    __shared__ Map wave_maps[GRAD ? 2 : 1][kScanWaves * K::CT];
    const Place at(p);
    if (at.chunk >= p.chunks) return;
    const int64_t chunk = at.chunk;
    const K k(p, chunk, at.tile);
    typename Quad<T>::vec x[L], z[L], d[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        z[l] = k.load(p.z, l, p.C);
        x[l] = k.load(p.x, l, p.C);
        if constexpr (GRAD) d[l] = k.load(p.dout, l, p.C);
    }
    mark_scenes(marks, p, k.p0);
    if (any_missing(k.row)) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            missing_row<T>(k.row[l], z[l], x[l]);
            if (GRAD && k.row[l] < 0) d[l] = typename Quad<T>::vec{};
        }
    }
    Map m[V], mb[V];
    Shut<T> shut;
    auto compose = [&](auto mk) {
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = mb[i] = {1.f, 0.f};
        float h0[SR][V], dl[SR][V];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[k.seg * L + l] : -1;
            const int e = decltype(mk)::value && GRAD ? marks.last[k.seg * L + l] : -1;
            if (!decltype(mk)::value) shut.add(z[l]);
            if (decltype(mk)::value && l % SR == 0) {
                k.of_scenes(p.h0, marks.first + k.seg * L + l, h0, p.C);
                if (GRAD) k.of_scenes(p.dlast, marks.last + k.seg * L + l, dl, p.C);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step g = gate((float)z[l][i]);
                const float v = g.n * (float)x[l][i];
                float t = GRAD ? (float)d[l][i] : 0.f;
                if (decltype(mk)::value) {
                    if (GRAD && e >= 0) t += dl[l % SR][i];
                    if (b >= 0) {
                        m[i] = {kForget, fmaf(g.f, h0[l % SR][i], v)};
                        if (GRAD) mb[i] = after(mb[i], {kForget, 0.f});
                    } else {
                        m[i] = after({g.f, v}, m[i]);
                        if (GRAD) mb[i] = after(mb[i], {g.f, g.f * t});
                    }
                } else {
                    // (the product of the factors serves both directions)
                    if (GRAD) mb[i].V = fmaf(m[i].F, g.f * t, mb[i].V);
                    m[i] = {g.f * m[i].F, fmaf(g.f, m[i].V, v)};
                }
            }
        }
    };
    bool by_maps = wave_marks<L>(marks, k.seg);
    if (!by_maps) {
        compose(std::false_type{});
        by_maps = shut.lift(m) && GRAD && any_nan(mb);
#pragma unroll
        for (int i = 0; i < V; ++i) mb[i].F = m[i].F;
    }
    if (by_maps) compose(std::true_type{});
    scan_wave<G, false>(m, wave_maps[0]);
    if constexpr (GRAD) scan_wave<G, true>(mb, wave_maps[1]);
    __syncthreads();
    constexpr int CT = K::CT;
    const int dir = threadIdx.x / CT, c = at.tile * CT + threadIdx.x % CT;
    if (dir < (GRAD ? 2 : 1) && c < p.C) {
        const Map all = dir ? scan_waves<CT, true>(wave_maps[GRAD ? 1 : 0], threadIdx.x % CT)
                            : scan_waves<CT, false>(wave_maps[0], threadIdx.x);
        p.maps[(dir * p.chunks + chunk) * p.C + c] = all;
    }
}

// The states, with the chunks' entering states known.  From the last chunk to
// the first: the rows that k_scan_maps read last are still in the memory-side
// cache.
template <typename T, int G, int L, RowEnd END>
__global__ void __launch_bounds__(kScanThreads) k_scan(ScanParams p) {
    using K = Chunk<T, G, L, END>;
    constexpr int V = K::V, CT = K::CT, SR = kSceneRows<L>;
    __shared__ SceneMarks<K::R> marks;
    __shared__ Map wave_maps[kScanWaves * CT], join[kScanThreads];
    __shared__ float state[CT];
    const Place at(p);
    if (at.chunk >= p.chunks) return;
    if (p.N == 0) {              // nothing to read: the scenes' states alone
        empty_scenes(p, at, p.h0, p.last, CT);
        return;
    }
    const int64_t chunk = p.chunks - 1 - at.chunk;
    const K k(p, chunk, at.tile);
    typename Quad<T>::vec x[L], z[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        z[l] = k.load(p.z, l, p.C);
        x[l] = k.load(p.x, l, p.C);
    }
    empty_scenes(p, at, p.h0, p.last, CT);      // (while the rows are on their way)
    entering_state<CT, false>(p, chunk, at.tile, join, state);
    mark_scenes(marks, p, k.p0);
    if (any_missing(k.row)) {
#pragma unroll
        for (int l = 0; l < L; ++l) missing_row<T>(k.row[l], z[l], x[l]);
    }
    const bool marked = wave_marks<L>(marks, k.seg);
    Map pre[V];
    Shut<T> shut;
    auto compose = [&](auto mk) {
#pragma unroll
        for (int i = 0; i < V; ++i) pre[i] = {1.f, 0.f};
        float h0[SR][V];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[k.seg * L + l] : -1;
            if (!decltype(mk)::value) shut.add(z[l]);
            if (decltype(mk)::value && l % SR == 0)
                k.of_scenes(p.h0, marks.first + k.seg * L + l, h0, p.C);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step g = gate((float)z[l][i]);
                const float v = g.n * (float)x[l][i];
                if (decltype(mk)::value)
                    pre[i] = b >= 0 ? Map{kForget, fmaf(g.f, h0[l % SR][i], v)} : after({g.f, v}, pre[i]);
                else
                    pre[i] = {g.f * pre[i].F, fmaf(g.f, pre[i].V, v)};
            }
        }
    };
    if (marked) {
        compose(std::true_type{});
    } else {
        compose(std::false_type{});
        shut.lift(pre);
    }
    scan_wave<G, false>(pre, wave_maps);
    __syncthreads();
    if (threadIdx.x < CT) scan_waves<CT, false>(wave_maps, threadIdx.x);
    __syncthreads();
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        s[i] = apply(pre[i], apply(wave_maps[(threadIdx.x >> 6) * CT + k.lane * V + i], state[k.lane * V + i]));
    // the rows again, from their entering state: the gates cost less than the
    // registers that would keep them (64 for 32 elements)
#pragma unroll
    for (int l = 0; l < L; ++l) {
        forget_uses(z[l]);
        forget_uses(x[l]);
    }
    auto walk = [&](auto mk) {
        float h0[SR][V];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[k.seg * L + l] : -1;
            const int e = decltype(mk)::value ? marks.last[k.seg * L + l] : -1;
            if (decltype(mk)::value && l % SR == 0)
                k.of_scenes(p.h0, marks.first + k.seg * L + l, h0, p.C);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (decltype(mk)::value && b >= 0) s[i] = h0[l % SR][i];
                const Step g = gate((float)z[l][i]);
                s[i] = fmaf(g.f, s[i], g.n * (float)x[l][i]);
                if (decltype(mk)::value && e >= 0 && i < k.nv) p.last[(int64_t)e * p.C + k.c0 + i] = s[i];
            }
            store_quad<T, END>((T*)p.h, k.row[l], p.C, k.c0, s, p.stream);
        }
    };
    if (marked)
        walk(std::true_type{});
    else
        walk(std::false_type{});
}

// The gradient, with the states that enter the chunks known in both
// directions; from the last chunk to the first, like k_scan.
template <typename T, int G, RowEnd END>
__global__ void __launch_bounds__(kScanThreads, 4) k_scan_grad(ScanParams p) {
    constexpr int L = kScanGradRows;
    using K = Chunk<T, G, L, END>;
    constexpr int V = K::V, CT = K::CT, SR = kSceneRows<L>;
    __shared__ SceneMarks<K::R> marks;
    __shared__ Map wave_maps[2][kScanWaves * CT], join[2][kScanThreads];
    __shared__ float state[2][CT];
    const Place at(p);
    if (at.chunk >= p.chunks) return;
    if (p.N == 0) {
        if (p.last) empty_scenes(p, at, p.dlast, p.last, CT);
        return;
    }
    const int64_t chunk = p.chunks - 1 - at.chunk;
    const K k(p, chunk, at.tile);
    typename Quad<T>::vec x[L], z[L], d[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        z[l] = k.load(p.z, l, p.C);
        x[l] = k.load(p.x, l, p.C);
        d[l] = k.load(p.dout, l, p.C);
    }
    if (p.last) empty_scenes(p, at, p.dlast, p.last, CT);
    entering_state<CT, false>(p, chunk, at.tile, join[0], state[0]);
    entering_state<CT, true>(p, chunk, at.tile, join[1], state[1]);
    mark_scenes(marks, p, k.p0);
    if (any_missing(k.row)) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            missing_row<T>(k.row[l], z[l], x[l]);
            if (k.row[l] < 0) d[l] = typename Quad<T>::vec{};
        }
    }
    const bool marked = wave_marks<L>(marks, k.seg);
    Map m[V], mb[V];
    float f[L][V], n[L][V], dh[L][V];
    Shut<T> shut;
    auto compose = [&](auto mk) {
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = mb[i] = {1.f, 0.f};
        float h0[SR][V], dl[SR][V];
        if (decltype(mk)::value) {
            k.of_scenes(p.h0, marks.first + k.seg * L, h0, p.C);
            k.of_scenes(p.dlast, marks.last + k.seg * L, dl, p.C);
        }
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[k.seg * L + l] : -1;
            const int e = decltype(mk)::value ? marks.last[k.seg * L + l] : -1;
            if (!decltype(mk)::value) shut.add(z[l]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step g = gate((float)z[l][i]);
                const float v = g.n * (float)x[l][i];
                f[l][i] = g.f;
                n[l][i] = g.n;
                float t = (float)d[l][i];
                if (decltype(mk)::value) {
                    if (e >= 0) t += dl[l][i];
                    if (b >= 0) {
                        m[i] = {kForget, fmaf(g.f, h0[l][i], v)};
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
    };
    bool by_maps = marked;
    if (!by_maps) {
        compose(std::false_type{});
        by_maps = shut.lift(m) && any_nan(mb);
#pragma unroll
        for (int i = 0; i < V; ++i) mb[i].F = m[i].F;
    }
    if (by_maps) compose(std::true_type{});
    scan_wave<G, false>(m, wave_maps[0]);
    scan_wave<G, true>(mb, wave_maps[1]);
    __syncthreads();
    if (threadIdx.x < CT)
        scan_waves<CT, false>(wave_maps[0], threadIdx.x);
    else if (threadIdx.x < 2 * CT)
        scan_waves<CT, true>(wave_maps[1], threadIdx.x - CT);
    __syncthreads();
    // forward: the states again, and (h[t-1] - x) f (1 - f)
    float s[V], y[V], q[L][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int own = (threadIdx.x >> 6) * CT + k.lane * V + i;
        s[i] = apply(m[i], apply(wave_maps[0][own], state[0][k.lane * V + i]));
        y[i] = apply(mb[i], apply(wave_maps[1][own], state[1][k.lane * V + i]));
    }
    static_assert(L == SR, "one group of rows");
    auto states = [&](auto mk) {
        float h0[SR][V];
        if (decltype(mk)::value) k.of_scenes(p.h0, marks.first + k.seg * L, h0, p.C);
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int b = decltype(mk)::value ? marks.first[k.seg * L + l] : -1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xv = (float)x[l][i];
                if (decltype(mk)::value && b >= 0) s[i] = h0[l][i];
                q[l][i] = (s[i] - xv) * (f[l][i] * n[l][i]);
                s[i] = fmaf(f[l][i], s[i], n[l][i] * xv);
            }
        }
    };
    if (marked)
        states(std::true_type{});
    else
        states(std::false_type{});
#pragma unroll
    for (int l = L - 1; l >= 0; --l) {
        const int b = marked ? marks.first[k.seg * L + l] : -1;
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
                if (p.last && i < k.nv) p.last[(int64_t)b * p.C + k.c0 + i] = y[i];
                y[i] = 0.f;
            }
        }
        store_quad<T, END>((T*)p.h, k.row[l], p.C, k.c0, ox, p.stream);
        store_quad<T, END>((T*)p.dz, k.row[l], p.C, k.c0, oz, p.stream);
    }
}

// Lanes per row: enough for its channels, kScanGroup at most (wider rows take
// several workgroups).
int scan_group(int C) {
    int G = 1;
    while (G < kScanGroup && G * kScanV < C) G *= 2;
    return G;
}
int64_t scan_chunks(int64_t N, int C, int rows) {
    const int64_t R = (int64_t)(kScanThreads / scan_group(C)) * rows;
    return std::max<int64_t>(1, (N + R - 1) / R);
}
int scan_rows(int64_t N, int C, bool grad) {
    if (grad) return kScanGradRows;
    if (scan_chunks(N, C, kScanRowsOne) == 1) return kScanRowsOne;
    const int64_t tiles = (C + scan_group(C) * kScanV - 1) / (scan_group(C) * kScanV);
    return scan_chunks(N, C, kScanRowsShort) <= kChunkGroup || scan_chunks(N, C, kScanRows) * tiles < 512
               ? kScanRowsShort : kScanRows;
}
// Workspace: the chunks' maps, the groups' maps and the entering states, each
// for both directions in the gradient.
struct ScanLayout {
    int64_t chunks, groups;
    int rows, tiles, dirs;
    size_t group_at, carry_at, total;
};
ScanLayout scan_layout(int64_t N, int C, bool grad) {
    ScanLayout l{};
    l.rows = scan_rows(N, C, grad);
    l.chunks = scan_chunks(N, C, l.rows);
    l.groups = (l.chunks + kChunkGroup - 1) / kChunkGroup;
    l.tiles = (C + scan_group(C) * kScanV - 1) / (scan_group(C) * kScanV);
    l.dirs = grad ? 2 : 1;
    if (l.chunks == 1) return l;
    l.group_at = l.total = align_up((size_t)l.dirs * l.chunks * C * sizeof(Map), 256);
    if (l.groups == 1) return l;
    l.carry_at = l.group_at + align_up((size_t)l.dirs * l.groups * C * sizeof(Map), 256);
    l.total = l.carry_at + align_up((size_t)l.dirs * l.chunks * C * 4, 256);
    return l;
}

unsigned scan_blocks(const ScanLayout& l) {
    return (unsigned)(l.tiles > 1 ? round_up(l.chunks, 8) * l.tiles : l.chunks);
}

template <typename T, int G, RowEnd END>
hipError_t scan_go(ScanParams p, bool grad, const ScanLayout& l, char* ws, hipStream_t st) {
    const unsigned grid = scan_blocks(l);
    p.chunks = l.chunks;
    p.tiles = l.tiles;
    p.maps = (Map*)ws;
    p.groups = (Map*)(ws + l.group_at);
    p.carry = (float*)(ws + l.carry_at);
    if (l.chunks > 1) {
        auto maps = k_scan_maps<T, G, kScanGradRows, END, true>;
        if (!grad)
            maps = l.rows == kScanRows ? k_scan_maps<T, G, kScanRows, END, false>
                                       : k_scan_maps<T, G, kScanRowsShort, END, false>;
        maps<<<grid, kScanThreads, 0, st>>>(p);
    }
    if (l.groups > 1) {
        k_scan_groups<<<dim3((unsigned)l.groups, (p.C + kCarryChannels - 1) / kCarryChannels, l.dirs), kScanThreads, 0,
                        st>>>(p);
        k_scan_carry<<<dim3((unsigned)l.groups, (p.C + kCarryChannels - 1) / kCarryChannels, l.dirs), kScanThreads, 0,
                       st>>>(p);
    }
    auto rows = k_scan_grad<T, G, END>;
    if (!grad)
        rows = l.rows == kScanRows        ? k_scan<T, G, kScanRows, END>
               : l.rows == kScanRowsShort ? k_scan<T, G, kScanRowsShort, END>
                                          : k_scan<T, G, kScanRowsOne, END>;
    rows<<<grid, kScanThreads, 0, st>>>(p);
    return hipGetLastError();
}

template <typename T, int G>
hipError_t scan_ends(const ScanParams& p, bool grad, const ScanLayout& l, char* ws, hipStream_t st) {
    if (p.C % kScanV == 0) return scan_go<T, G, kWholeQuads>(p, grad, l, ws, st);
    // (a group of one lane serves up to four channels, a larger one more)
    return scan_go<T, G, G == 1 ? kSingles : kCutQuad>(p, grad, l, ws, st);
}

template <typename T>
hipError_t scan_dispatch(const ScanParams& p, bool grad, char* ws, hipStream_t st) {
    const ScanLayout l = scan_layout(p.N, p.C, grad);
    switch (scan_group(p.C)) {
        case 1: return scan_ends<T, 1>(p, grad, l, ws, st);
        case 2: return scan_ends<T, 2>(p, grad, l, ws, st);
        case 4: return scan_ends<T, 4>(p, grad, l, ws, st);
        case 8: return scan_ends<T, 8>(p, grad, l, ws, st);
        case 16: return scan_ends<T, 16>(p, grad, l, ws, st);
        default: return scan_ends<T, 32>(p, grad, l, ws, st);
    }
}

}  // namespace

bool scan_fits(int64_t N, int C, bool grad) {
    return (uint64_t)scan_blocks(scan_layout(N, C, grad)) * kScanThreads < (uint64_t)1 << 32;
}
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
    p.stream = a.N * a.C * (a.dtype == SPCONV_BF16 ? 2 : 4) > kStreamBytes;
    char* ws = (char*)a.workspace;
    return a.dtype == SPCONV_BF16 ? scan_dispatch<__bf16>(p, grad, ws, stream) : scan_dispatch<float>(p, grad, ws, stream);
}

}  // namespace spc
