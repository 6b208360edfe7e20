// Gated linear recurrence over the voxels of each scene, in a given order, and
// its gradient, for gfx950.
//
//   h[t] = f[t] h[t-1] + (1 - f[t]) x[t],   f = sigmoid(z)
//
// Each step is the affine map s -> f s + v, and maps compose:
// (F2, V2) after (F1, V1) is (F2 F1, F2 V1 + V2).  So the sequence is cut into
// chunks, the chunks into segments of consecutive rows that one lane walks for
// its channels; segments are joined by a scan over the lanes, chunks by a scan
// over their composed maps.  A scene's first row forgets what came before: its
// map is marked F = kForget, and composing selects instead of multiplying, so
// infinities and NaN of one scene stay in it.
//
// The gradient runs the same maps backwards: with g[t] the derivative at h[t],
//   y[t] = f[t] g[t]                what row t hands to row t - 1
//   g[t] = dout[t] + y[t+1]         (0 from another scene)
//   dx = (1 - f) g,   dz = g (h[t-1] - x) f (1 - f),   dh0 = y[first]
// i.e. s -> f s + f dout from the last row to the first.
//
// f = 1 / (1 + e^-z) and 1 - f = 1 / (1 + e^z) come from e = exp(-|z|), so both
// keep their relative precision; states, maps and sums are fp32.
#include "rowops.h"

#include <algorithm>

namespace spc {

namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWaves = kScanThreads / 64;
constexpr float kForget = -1.f;      // F of a map that forgets the state; real F are in [0, 1]
constexpr int kScanGroup = 16;       // lanes per row, at most: 256 bytes of a row per workgroup

struct Step {
    float f, n;      // sigmoid(z), sigmoid(-z)
};
__device__ __forceinline__ Step gate(float z) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896f * fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    const float er = e * r;
    return {z >= 0.f ? r : er, z >= 0.f ? er : r};
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
    float2* agg;       // [chunks][C] maps of the chunks
    float2* aggb;      // the same, last row to first (gradient)
    float* carry;      // [chunks][C] state that enters the chunk
    float* carryb;     // the same, from the chunk behind
    int64_t N;
    int C, scenes;
    int64_t chunks;
};

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
    if (p.scenes > 4 * kScanThreads) {
        // the last scene that begins at or before p0 (several may: the empty ones before it)
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

// The caller's rows of a segment's positions; -1 for positions past the end or
// an order value outside the rows (such a row is neither read nor written and
// hands the state on).
template <int L>
__device__ __forceinline__ void segment_rows(const ScanParams& p, int64_t pos, int64_t (&row)[L]) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
        int64_t r = pos + l;
        if (r < p.N && p.order) r = (uint32_t)p.order[r];
        row[l] = r < p.N ? r : -1;
    }
}

template <typename T>
__device__ __forceinline__ typename Piece<T>::vec load_gate(const T* z, int64_t row, int n) {
    typename Piece<T>::vec v = load_piece(z, row >= 0 ? n : 0);
    if (row < 0) {
#pragma unroll
        for (int i = 0; i < Piece<T>::V; ++i) v[i] = (T)__builtin_inff();   // f = 1, 1 - f = 0
    }
    return v;
}

// Exclusive scan of the lanes' maps over the segments of the workgroup, in
// segment order (BACK: from the last segment to the first).  m: in, the
// segment's map; out, the composed map of the segments before it.  total: the
// map of the whole workgroup, in every lane.
template <int G, int V, bool BACK>
__device__ __forceinline__ void scan_segments(Map (&m)[V], Map (&total)[V], Map* wave_maps) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane % G;
    const int seg = BACK ? 64 / G - 1 - lane / G : lane / G;     // position within the wave's order
#pragma unroll
    for (int d = 1; d < 64 / G; d *= 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Map a = {BACK ? __shfl_down(m[i].F, d * G) : __shfl_up(m[i].F, d * G),
                           BACK ? __shfl_down(m[i].V, d * G) : __shfl_up(m[i].V, d * G)};
            const Map r = after(m[i], a);
            if (seg >= d) m[i] = r;
        }
    }
    if (seg == 64 / G - 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) wave_maps[wave * (G * V) + c * V + i] = m[i];
    }
    Map ex[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (G < 64) {
            ex[i] = {BACK ? __shfl_down(m[i].F, G) : __shfl_up(m[i].F, G),
                     BACK ? __shfl_down(m[i].V, G) : __shfl_up(m[i].V, G)};
            if (seg == 0) ex[i] = {1.f, 0.f};
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        Map before = {1.f, 0.f}, all = {1.f, 0.f};
#pragma unroll
        for (int k = 0; k < kScanWaves; ++k) {
            const int w = BACK ? kScanWaves - 1 - k : k;
            if (w == wave) before = all;
            all = after(wave_maps[w * (G * V) + c * V + i], all);
        }
        m[i] = after(ex[i], before);
        total[i] = all;
    }
}

// Maps of the chunks: forward, and with GRAD backward too.
template <typename T, int G, int L, bool GRAD>
__global__ void __launch_bounds__(kScanThreads) k_scan_maps(ScanParams p) {
    constexpr int V = Piece<T>::V, S = kScanThreads / G, R = S * L;
    __shared__ SceneMarks<R> marks;
    __shared__ Map wave_maps[2][kScanWaves * G * V];
    const int64_t chunk = blockIdx.x, p0 = chunk * R;
    const int lane = threadIdx.x % G, seg = threadIdx.x / G;
    const int c0 = (blockIdx.y * G + lane) * V, nv = p.C - c0;
    int64_t row[L];
    segment_rows<L>(p, p0 + seg * L, row);
    typename Piece<T>::vec x[L], z[L], d[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int64_t at = row[l] * p.C + c0;
        z[l] = load_gate((const T*)p.z + at, row[l], nv);
        x[l] = load_piece((const T*)p.x + at, row[l] >= 0 ? nv : 0);
        if constexpr (GRAD) d[l] = load_piece((const T*)p.dout + at, row[l] >= 0 ? nv : 0);
    }
    mark_scenes(marks, p, p0);
    Map m[V], total[V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = {1.f, 0.f};
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int b = marks.first[seg * L + l];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Step s = gate((float)z[l][i]);
            const float v = s.n * (float)x[l][i];
            if (b >= 0) {
                const float in = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
                m[i] = {kForget, fmaf(s.f, in, v)};
            } else {
                m[i] = after({s.f, v}, m[i]);
            }
        }
    }
    scan_segments<G, V, false>(m, total, wave_maps[0]);
    if (seg == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < nv) p.agg[chunk * p.C + c0 + i] = make_float2(total[i].F, total[i].V);
    }
    if constexpr (GRAD) {
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = {1.f, 0.f};
#pragma unroll
        for (int l = L - 1; l >= 0; --l) {
            const int b = marks.first[seg * L + l], e = marks.last[seg * L + l];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Step s = gate((float)z[l][i]);
                float dh = (float)d[l][i];
                if (e >= 0 && p.dlast && i < nv) dh += p.dlast[(int64_t)e * p.C + c0 + i];
                m[i] = b >= 0 ? Map{kForget, 0.f} : after({s.f, s.f * dh}, m[i]);
            }
        }
        scan_segments<G, V, true>(m, total, wave_maps[1]);
        if (seg == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < nv) p.aggb[chunk * p.C + c0 + i] = make_float2(total[i].F, total[i].V);
        }
    }
}

// States that enter the chunks: the chunks in 64 parts, a lane composes its
// part's maps for one channel, joins the parts before it, and walks its part
// again.  BACK: from the last chunk to the first.
template <bool BACK>
__global__ void __launch_bounds__(256) k_scan_carry(const float2* agg, float* carry, int64_t chunks, int C) {
    __shared__ Map part[64][4];
    const int ch = threadIdx.x & 3, pt = threadIdx.x >> 2;
    const int c = blockIdx.x * 4 + ch;
    const int64_t per = (chunks + 63) / 64;
    const int64_t a = min(chunks, pt * per), e = min(chunks, a + per);
    Map m = {1.f, 0.f};
    if (c < C) {
        for (int64_t k = a; k < e; ++k) {
            const float2 g = agg[(BACK ? chunks - 1 - k : k) * C + c];
            m = after({g.x, g.y}, m);
        }
    }
    part[pt][ch] = m;
    __syncthreads();
    float s = 0.f;
    for (int k = 0; k < pt; ++k) s = apply(part[k][ch], s);
    if (c < C) {
        for (int64_t k = a; k < e; ++k) {
            const int64_t at = (BACK ? chunks - 1 - k : k) * C + c;
            carry[at] = s;
            const float2 g = agg[at];
            s = apply({g.x, g.y}, s);
        }
    }
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

// The forward's states, with the chunks' entering states known (carry NULL:
// one chunk, nothing enters).
template <typename T, int G, int L>
__global__ void __launch_bounds__(kScanThreads) k_scan(ScanParams p) {
    constexpr int V = Piece<T>::V, S = kScanThreads / G, R = S * L;
    __shared__ SceneMarks<R> marks;
    __shared__ Map wave_maps[kScanWaves * G * V];
    const int64_t chunk = blockIdx.x, p0 = chunk * R;
    const int lane = threadIdx.x % G, seg = threadIdx.x / G;
    const int c0 = (blockIdx.y * G + lane) * V, nv = p.C - c0;
    int64_t row[L];
    segment_rows<L>(p, p0 + seg * L, row);
    typename Piece<T>::vec x[L], z[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int64_t at = row[l] * p.C + c0;
        z[l] = load_gate((const T*)p.z + at, row[l], nv);
        x[l] = load_piece((const T*)p.x + at, row[l] >= 0 ? nv : 0);
    }
    mark_scenes(marks, p, p0);
    Map m[L][V], pre[V], total[V];       // m[l]: the segment's rows 0 .. l composed
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int b = marks.first[seg * L + l];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Step s = gate((float)z[l][i]);
            const float v = s.n * (float)x[l][i];
            if (b >= 0) {
                const float in = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
                m[l][i] = {kForget, fmaf(s.f, in, v)};
            } else {
                m[l][i] = l ? after({s.f, v}, m[l - 1][i]) : Map{s.f, v};
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) pre[i] = m[L - 1][i];
    scan_segments<G, V, false>(pre, total, wave_maps);
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = apply(pre[i], p.carry && i < nv ? p.carry[chunk * p.C + c0 + i] : 0.f);
#pragma unroll
    for (int l = 0; l < L; ++l) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = apply(m[l][i], s[i]);
        if (row[l] >= 0) store_piece((T*)p.h + row[l] * p.C + c0, o, nv);
        const int e = marks.last[seg * L + l];
        if (e >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < nv) p.last[(int64_t)e * p.C + c0 + i] = o[i];
        }
    }
    empty_scenes(p, p.h0, p.last, G * V);
}

template <typename T, int G, int L>
__global__ void __launch_bounds__(kScanThreads) k_scan_grad(ScanParams p) {
    constexpr int V = Piece<T>::V, S = kScanThreads / G, R = S * L;
    __shared__ SceneMarks<R> marks;
    __shared__ Map wave_maps[2][kScanWaves * G * V];
    const int64_t chunk = blockIdx.x, p0 = chunk * R;
    const int lane = threadIdx.x % G, seg = threadIdx.x / G;
    const int c0 = (blockIdx.y * G + lane) * V, nv = p.C - c0;
    int64_t row[L];
    segment_rows<L>(p, p0 + seg * L, row);
    typename Piece<T>::vec x[L], z[L], d[L];
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int64_t at = row[l] * p.C + c0;
        z[l] = load_gate((const T*)p.z + at, row[l], nv);
        x[l] = load_piece((const T*)p.x + at, row[l] >= 0 ? nv : 0);
        d[l] = load_piece((const T*)p.dout + at, row[l] >= 0 ? nv : 0);
    }
    mark_scenes(marks, p, p0);
    Map m[V], mb[V], total[V];
    float dh[L][V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = mb[i] = {1.f, 0.f};
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int b = marks.first[seg * L + l], e = marks.last[seg * L + l];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Step s = gate((float)z[l][i]);
            const float v = s.n * (float)x[l][i];
            float t = (float)d[l][i];
            if (e >= 0 && p.dlast && i < nv) t += p.dlast[(int64_t)e * p.C + c0 + i];
            dh[l][i] = t;
            if (b >= 0) {
                const float in = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
                m[i] = {kForget, fmaf(s.f, in, v)};
                mb[i] = after(mb[i], {kForget, 0.f});
            } else {
                m[i] = after({s.f, v}, m[i]);
                mb[i] = after(mb[i], {s.f, s.f * t});
            }
        }
    }
    scan_segments<G, V, false>(m, total, wave_maps[0]);
    scan_segments<G, V, true>(mb, total, wave_maps[1]);
    float s[V], y[V];
    float q[L][V];       // (h[t-1] - x) f (1 - f)
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = apply(m[i], p.carry && i < nv ? p.carry[chunk * p.C + c0 + i] : 0.f);
        y[i] = apply(mb[i], p.carryb && i < nv ? p.carryb[chunk * p.C + c0 + i] : 0.f);
    }
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const int b = marks.first[seg * L + l];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Step g = gate((float)z[l][i]);
            const float xv = (float)x[l][i];
            if (b >= 0) s[i] = p.h0 && i < nv ? p.h0[(int64_t)b * p.C + c0 + i] : 0.f;
            q[l][i] = (s[i] - xv) * (g.f * g.n);
            s[i] = fmaf(g.f, s[i], g.n * xv);
        }
    }
#pragma unroll
    for (int l = L - 1; l >= 0; --l) {
        const int b = marks.first[seg * L + l];
        float ox[V], oz[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Step g = gate((float)z[l][i]);
            const float gt = dh[l][i] + y[i];
            ox[i] = g.n * gt;
            oz[i] = q[l][i] * gt;
            y[i] = g.f * gt;
            if (b >= 0) {
                if (p.last && i < nv) p.last[(int64_t)b * p.C + c0 + i] = y[i];
                y[i] = 0.f;
            }
        }
        if (row[l] >= 0) {
            store_piece((T*)p.h + row[l] * p.C + c0, ox, nv);
            store_piece((T*)p.dz + row[l] * p.C + c0, oz, nv);
        }
    }
    if (p.last) empty_scenes(p, p.dlast, p.last, G * V);
}

// Lanes per row: enough for its pieces, kScanGroup at most (wider rows take
// several workgroups, one for each 256 bytes).
int scan_group(int C, int V) {
    int G = 1;
    while (G < kScanGroup && G * V < C) G *= 2;
    return G;
}
// Rows that a lane walks: 64 elements (forward), 32 (gradient: it holds more
// of each).
constexpr int scan_len(int V, bool grad) { return (grad ? 32 : 64) / V; }
int64_t scan_chunks(int64_t N, int C, int dtype, bool grad) {
    const int V = dtype == SPCONV_BF16 ? 8 : 4;
    const int64_t R = (int64_t)(kScanThreads / scan_group(C, V)) * scan_len(V, grad);
    return std::max<int64_t>(1, (N + R - 1) / R);
}

template <typename T, int G>
hipError_t scan_go(const ScanParams& p, bool grad, hipStream_t st) {
    constexpr int V = Piece<T>::V;
    const dim3 grid((unsigned)p.chunks, (p.C + G * V - 1) / (G * V));
    const unsigned cg = (p.C + 3) / 4;
    if (grad) {
        if (p.chunks > 1) {
            k_scan_maps<T, G, scan_len(V, true), true><<<grid, kScanThreads, 0, st>>>(p);
            k_scan_carry<false><<<cg, 256, 0, st>>>(p.agg, p.carry, p.chunks, p.C);
            k_scan_carry<true><<<cg, 256, 0, st>>>(p.aggb, p.carryb, p.chunks, p.C);
        }
        k_scan_grad<T, G, scan_len(V, true)><<<grid, kScanThreads, 0, st>>>(p);
    } else {
        if (p.chunks > 1) {
            k_scan_maps<T, G, scan_len(V, false), false><<<grid, kScanThreads, 0, st>>>(p);
            k_scan_carry<false><<<cg, 256, 0, st>>>(p.agg, p.carry, p.chunks, p.C);
        }
        k_scan<T, G, scan_len(V, false)><<<grid, kScanThreads, 0, st>>>(p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t scan_dispatch(const ScanParams& p, bool grad, hipStream_t st) {
    switch (scan_group(p.C, Piece<T>::V)) {
        case 1: return scan_go<T, 1>(p, grad, st);
        case 2: return scan_go<T, 2>(p, grad, st);
        case 4: return scan_go<T, 4>(p, grad, st);
        case 8: return scan_go<T, 8>(p, grad, st);
        default: return scan_go<T, 16>(p, grad, st);
    }
}

}  // namespace

size_t scan_workspace_bytes(int64_t N, int C, int dtype, bool grad) {
    const int64_t chunks = scan_chunks(N, C, dtype, grad);
    if (chunks == 1) return 0;
    return align_up((size_t)chunks * C * 12 * (grad ? 2 : 1), 256);
}

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
    p.chunks = scan_chunks(a.N, a.C, a.dtype, grad);
    if (p.chunks > 1) {
        const size_t n = (size_t)p.chunks * a.C;
        p.agg = (float2*)a.workspace;
        p.aggb = grad ? p.agg + n : nullptr;
        p.carry = (float*)(p.agg + (grad ? 2 : 1) * n);
        p.carryb = grad ? p.carry + n : nullptr;
    }
    return a.dtype == SPCONV_BF16 ? scan_dispatch<__bf16>(p, grad, stream) : scan_dispatch<float>(p, grad, stream);
}

}  // namespace spc
