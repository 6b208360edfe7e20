/*
 * spconv_mi355x.h -- C interface of libspconv_mi355x.so: the fused
 * gather-GEMM-accumulate of a submanifold sparse 3D convolution on one
 * AMD Instinct MI355X (gfx950).
 *
 * The operation (page "mlx_backend/sparse_conv_metal.py": module docstring,
 * the kernel body and the `sparse_conv_metal` wrapper docstring):
 *
 *     out[n, co] = bias[co] + sum_k sum_ci feats[nbr[k, n], ci] * w[k, ci, co]
 *
 * nbr is a (K, N) int32 neighbour map, element k*N + n, whose value N marks a
 * missing neighbour (the page's pad row; it contributes nothing).  The (K, N, Ci)
 * gather is never materialised: one kernel accumulates straight from feats and w.
 *
 * Conventions shared by every call:
 *  - Pointers marked (dev) are HIP device memory owned by the caller; the
 *    library never allocates, frees or retains device memory.  Pointers marked
 *    (host) are ordinary host memory.
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Calls enqueue work on it and return without waiting, except where noted.
 *  - Every call returns an int status (SPCONV_OK = 0, negative on error).
 *    Argument checks happen on the host before any launch; a failed check
 *    enqueues nothing.  spconv_last_error() gives a text for the last failure
 *    of the calling thread.
 *  - Device buffers must be 256-byte aligned (arena, workspace) or 16-byte
 *    aligned (coords, feats, w, out, nbr); torch allocations satisfy both.
 */
#ifndef SPCONV_MI355X_H
#define SPCONV_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPCONV_ABI_VERSION 1

enum spconv_status {
    SPCONV_OK = 0,
    SPCONV_E_INVALID = -1,      /* bad argument: null pointer, bad K, bad alignment, ... */
    SPCONV_E_UNSUPPORTED = -2,  /* valid but not implemented (e.g. a channel count)      */
    SPCONV_E_COORD_RANGE = -3,  /* a coordinate outside [-2^20, 2^20)                    */
    SPCONV_E_DUPLICATE = -4,    /* two voxels share a coordinate                          */
    SPCONV_E_WORKSPACE = -5,    /* arena or workspace smaller than required               */
    SPCONV_E_HIP = -6           /* a HIP runtime call failed                              */
};

enum spconv_dtype {
    SPCONV_F32 = 0,             /* feats, w, out float32                                  */
    SPCONV_BF16 = 1             /* feats, w, out bfloat16; accumulation is fp32 either way */
};

enum spconv_act {
    SPCONV_SILU = 0,            /* a sigmoid(a)                                            */
    SPCONV_GELU = 1             /* a (1 + erf(a / sqrt 2)) / 2                             */
};

/* Opaque host-side handle of a built neighbour map.  The map's device data
 * lives in the caller's arena, which must outlive every use of the handle. */
typedef struct spconv_nmap spconv_nmap;

int spconv_abi_version(void);

/* Byte sizes of the persistent arena (the map, its row schedule and block
 * masks: about (4K+4)*N bytes) and of the build-only workspace (sort buffers
 * and brick table: about 24N + 32*2^ceil(log2(2N)) bytes) for N voxels and K
 * offsets.  Host only, pure.  K must be >= 1. */
int spconv_nmap_sizes(int64_t N, int K, size_t* arena_bytes, size_t* workspace_bytes);

/* Build the neighbour map of N active voxels.
 *   coords   (dev) int32 (N, 3): x, y, z of voxel n at 3n..3n+2, each in
 *            [-2^20, 2^20), all distinct.  The caller's order defines n.
 *   K        an odd cube (1, 27, 125, ...): offsets o_k, k = ((a*s)+b)*s + c,
 *            s = cbrt(K), o_k = (a-r, b-r, c-r) * dilation, r = (s-1)/2
 *            (x slowest, z fastest; centre k = (K-1)/2).  The page leaves the
 *            offset numbering to the map's builder; this is the numbering of a
 *            dense 3D cross-correlation with padding r*dilation.
 *   dilation >= 1.
 *   nbr[k, n] = m if coords[m] == coords[n] + o_k, else N  (page: the
 *   `sparse_conv_metal` wrapper docstring gives the (K, N) int32 layout and
 *   the N sentinel).
 * The map is stored in the arena in an internal row order (Morton order of the
 * voxels, refined by sorting rows on their validity masks inside 128-row
 * half tiles); spconv_nmap_export returns it in the caller's order.
 * Waits on `stream` twice: mid-build for the coordinate range check and the
 * number of Morton bits that vary (which fixes the sort passes; the first sort
 * pass is already queued, so the GPU keeps working meanwhile), and at the end
 * (SPCONV_E_DUPLICATE, and the valid-pair count kept in the handle).  Both
 * results arrive in a small pinned host buffer that the kernels write
 * directly; the waits use one HIP event per device.  The buffer (128 bytes)
 * and the events belong to the calling thread and are kept until the process
 * ends: the library never frees them, since at process exit the HIP runtime
 * may already be gone.  The workspace may be reused or freed when this
 * returns.
 * On success *out receives a handle to release with spconv_nmap_destroy. */
int spconv_build_nmap(const int32_t* coords, int64_t N, int K, int dilation,
                      void* arena, size_t arena_bytes,
                      void* workspace, size_t workspace_bytes,
                      void* stream, spconv_nmap** out);

/* spconv_build_nmap for several scenes in one map (batched coordinates; the
 * pages' voxel sets carry no batch field, so this is the library's form):
 *   coords   (dev) int32 (N, 4): b, x, y, z of voxel n at 4n..4n+3, b in
 *            [0, batches); voxels are neighbours only within one batch.
 *   Each batch occupies its own slab of S = 2^21 / B' x-values, B' = batches
 *   rounded up to a power of two: its x must lie in [-S/2 + r*d, S/2 - r*d)
 *   (r*d = the stencil's reach), y and z in [-2^20, 2^20); otherwise
 *   SPCONV_E_COORD_RANGE.  Too many batches for the reach gives
 *   SPCONV_E_UNSUPPORTED.  Arena and workspace sizes, ordering, errors and
 *   synchronisation are those of spconv_build_nmap. */
int spconv_build_nmap_batched(const int32_t* coords, int64_t N, int batches, int K, int dilation,
                              void* arena, size_t arena_bytes,
                              void* workspace, size_t workspace_bytes,
                              void* stream, spconv_nmap** out);

/* Wrap a caller-made (K, N) int32 map (dev, element k*N + n) into a handle, as
 * the page's operator receives one.  Values outside [0, N) are treated as
 * missing.  Rows keep the caller's order apart from the in-tile mask sort.
 * Needs an arena of spconv_nmap_sizes(N, K) bytes, no workspace, no sync. */
int spconv_nmap_wrap(const int32_t* nbr, int64_t N, int K,
                     void* arena, size_t arena_bytes, void* stream, spconv_nmap** out);

/* Copy the map out in the caller's order.
 *   nbr_out   (dev) int32 (K, N), or NULL
 *   order_out (dev) int32 (N): row i of the internal schedule holds voxel
 *             order_out[i]; or NULL
 * Asynchronous on `stream`. */
int spconv_nmap_export(const spconv_nmap* h, int32_t* nbr_out, int32_t* order_out, void* stream);

/* Sizes of a handle; valid_pairs (the number of (k, n) entries != N) is read
 * from the device, which synchronises `stream` the first time.  Any output
 * pointer may be NULL. */
int spconv_nmap_info(const spconv_nmap* h, int64_t* N, int* K, int* dilation,
                     int64_t* valid_pairs, void* stream);

/* The fused forward (page: the kernel body and the wrapper).
 *   feats (dev) (N, Ci) row-major (N+1 rows are accepted; row N is never read)
 *   w     (dev) (K, Ci, Co) row-major, K = the handle's K
 *   bias  (dev) float32 (Co,), or NULL for zero
 *   out   (dev) (N, Co) row-major, written completely
 *   dtype SPCONV_F32 or SPCONV_BF16 for feats, w and out together.
 * Accumulation is fp32 over all K offsets; bias is added in fp32 and the sum
 * is rounded once (round-to-nearest-even) to the output type.  (The page adds
 * the bias after rounding the accumulator to the weight type; one rounding is
 * this library's choice.)
 * Supported: Ci in {32, 64, 128, 256}, Co a multiple of 32 up to 4096.
 * Others return SPCONV_E_UNSUPPORTED.  Asynchronous, no synchronisation:
 * two calls with the same inputs give bit-identical outputs.
 * bfloat16 with Ci = 128 and Co a multiple of 64 runs the kernel over each
 * tile's distinct neighbour rows, which reads w packed: this call packs w
 * into a stream-ordered allocation of K*Ci*Co*2 bytes (hipMallocAsync) that
 * it frees on `stream` after the forward; spconv_forward_packed with a
 * caller's pack gives the same bits without it.  That kernel's workgroups
 * take tiles from atomic counters (which workgroup computes a tile changes
 * from run to run, how it is computed does not) held in a library-owned
 * device array of 8192 counter slots per device: each launch takes Co/128
 * or Co/64 slots in turn and leaves them at zero when it completes, so
 * launches in flight at the same time share counters only if 8192 slots
 * were handed out between their starts.  N = 0 is a no-op. */
int spconv_forward(const void* feats, const spconv_nmap* nmap, const void* w,
                   const float* bias, void* out, int Ci, int Co, int dtype, void* stream);

/* The forward with feats in a dtype of their own (page: the wrapper casts
 * feats to the weights' dtype before the kernel runs).
 *   feats_dtype  SPCONV_F32 or SPCONV_BF16: the element type of feats
 *   dtype        the element type of w and out
 *   wpack        (dev) optional: spconv_pack_weights(w), used where the
 *                bfloat16 forward has a packed form; or NULL
 *   workspace    (dev) optional, 256-byte aligned, of at least
 *                spconv_forward_mixed_workspace_size bytes; or NULL
 * float32 -> bfloat16 rounds to nearest even (NaN stays NaN); bfloat16 ->
 * float32 is exact.  Without a workspace each gathered value is converted as
 * it is loaded.  With one (float32 feats into bfloat16 weights only; the size
 * is 0 for the other pairings and the argument is then ignored), a streaming
 * pass first writes the cast features into it and the bfloat16 forward runs
 * on them: the page's order, and faster at Ci = 128 and 256.  Both give the
 * forward of the cast features up to accumulation order.  With feats_dtype ==
 * dtype this is spconv_forward (same kernels).  Other arguments, limits,
 * errors and ordering are spconv_forward's.  Only the work this call
 * enqueues on `stream` writes and reads the workspace; it may be reused once
 * that work is done. */
int spconv_forward_mixed_workspace_size(int64_t N, int Ci, int feats_dtype, int dtype, size_t* bytes);
int spconv_forward_mixed(const void* feats, int feats_dtype, const spconv_nmap* nmap, const void* w,
                         const void* wpack, const float* bias, void* out, int Ci, int Co, int dtype,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Packed weights: an optional second copy of w (the same size) in the order
 * the bf16 forward reads it, so that the kernel loads each offset's slice with
 * plain 16-byte accesses instead of transposing w again for every tile.
 *   Ci = 128, Co a multiple of 64: fragment order.  16-byte unit
 *     e = (((k (Co/64) + c) 4 + s) 4 + j) 64 + l, lane l = m + 16 q, holds
 *     w[k][32 s + 8 q .. 32 s + 8 q + 7][64 c + 16 (m >> 2) + 4 j + (m & 3)]:
 *     lane l's matrix-core operand of output tile j, input-channel step s.
 *   Ci = 256, or Ci = 128 with other Co: per offset k and tile of BN output
 *     channels, 8 input channels x one output channel per 16-byte unit, output
 *     channels in the order the matrix-core tiles use.
 * The page's operator takes w as is; packing is this library's own
 * acceleration and is computed from w alone.
 *
 * spconv_pack_weights_size: bytes of the packed copy for (K, Ci, Co, dtype);
 * 0 when the forward has no packed form for that configuration (float32, or
 * Ci < 128).  Host only.
 * spconv_pack_weights: writes the packed copy of w (dev, (K, Ci, Co)
 * row-major) into wpack (dev, 16-byte aligned, at least the size above);
 * asynchronous on `stream`; a no-op when the size is 0.  wpack must be
 * repacked whenever w changes. */
int spconv_pack_weights_size(int K, int Ci, int Co, int dtype, size_t* bytes);
int spconv_pack_weights(const void* w, int K, int Ci, int Co, int dtype,
                        void* wpack, size_t wpack_bytes, void* stream);

/* spconv_forward with packed weights: the same operation, arguments and
 * result (bit for bit) as spconv_forward, plus wpack packed from the same w
 * for the handle's K; no allocation.  w is still required: configurations the
 * packed kernels do not serve (Ci = 256 feats of 4 GiB or more) read it
 * directly.  wpack may be NULL only when spconv_pack_weights_size gives 0. */
int spconv_forward_packed(const void* feats, const spconv_nmap* nmap, const void* w,
                          const void* wpack, const float* bias, void* out,
                          int Ci, int Co, int dtype, void* stream);

/* Input gradient of spconv_forward (the adjoint of its linear map in feats;
 * the page gives the forward formula, module docstring of
 * "mlx_backend/sparse_conv_metal.py", and the gradient follows from it):
 *   dfeats[m, ci] = sum over (k, n) with nbr[k, n] == m of
 *                   sum_co dout[n, co] * w[k, ci, co]
 *   dout     (dev) (N, Co), dtype as w;  w (dev) (K, Ci, Co)
 *   dfeats   (dev) (N, Ci) written, dtype as w; no bias term
 *   workspace (dev) spconv_dgrad_workspace_size bytes, 256-byte aligned,
 *            caller-owned, free after the call's work has run
 * The map must come from spconv_build_nmap: a map of a symmetric stencil is
 * its own mirror, nbr[K-1-k, nbr[k, n]] = n, so the gradient is the forward
 * over dout with the weights w'[k] = w[K-1-k]^T, which this call writes into
 * the workspace (and packs there when the bf16 kernel has a packed form)
 * before running the forward kernels with Ci and Co exchanged.  A wrapped map
 * gives SPCONV_E_UNSUPPORTED; so does a (Ci, Co) for which the exchanged
 * forward has no kernel (Co in {32, 64, 128, 256}, Ci a multiple of 32 up to
 * 4096).  Asynchronous on `stream`, no allocation, no synchronisation. */
int spconv_dgrad_workspace_size(int K, int Ci, int Co, int dtype, size_t* bytes);
int spconv_dgrad(const void* dout, const spconv_nmap* nmap, const void* w,
                 void* workspace, size_t workspace_bytes, void* dfeats,
                 int Ci, int Co, int dtype, void* stream);

/* spconv_dgrad without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Same operation, arguments, result and errors as
 * spconv_dgrad; the mirrored and packed weights go into a fixed scratch array
 * of SPCONV_NOALLOC_SCRATCH_BYTES inside the library (one per device, taken
 * at the first call on that device and held until the process ends).
 * Configurations whose spconv_dgrad_workspace_size exceeds it return
 * SPCONV_E_WORKSPACE (K = 27 fits every supported Ci, Co <= 256 in either
 * dtype).  The call allocates nothing.  Every call on one device shares that
 * device's scratch: calls that overlap in time on one device (concurrent
 * streams, other host threads) race and must be serialised by the caller;
 * calls in order on one stream are safe.  Nothing in the scratch needs to
 * start at zero: each call writes all of the part it reads. */
#define SPCONV_NOALLOC_SCRATCH_BYTES (16u << 20)
int spconv_dgrad_noalloc(const void* dout, const spconv_nmap* nmap, const void* w, void* dfeats,
                         int Ci, int Co, int dtype, void* stream);

/* Weight gradient of spconv_forward (its derivative with respect to w,
 * contracted with dout; the page gives the forward formula, module docstring
 * of "mlx_backend/sparse_conv_metal.py"):
 *   dw[k, ci, co] = sum over n with nbr[k, n] present of feats[nbr[k, n], ci] * dout[n, co]
 *   feats    (dev) (N or N+1, Ci) and dout (dev) (N, Co), one dtype
 *   dw       (dev) (K, Ci, Co) written in that dtype (fp32 sums, one rounding)
 *   workspace (dev) spconv_wgrad_workspace_size bytes, 256-byte aligned,
 *            caller-owned: fp32 partial sums of row chunks (a few times
 *            K*Ci*Co*4 bytes), added up in a fixed order, so the result is
 *            deterministic
 * Ci and Co: multiples of 32 up to 4096.  Works with built and wrapped maps.
 * Asynchronous on `stream`, no allocation, no synchronisation, no atomics. */
int spconv_wgrad_workspace_size(int64_t N, int K, int Ci, int Co, int dtype, size_t* bytes);
int spconv_wgrad(const void* feats, const void* dout, const spconv_nmap* nmap,
                 void* workspace, size_t workspace_bytes, void* dw,
                 int Ci, int Co, int dtype, void* stream);

/* ---- Row-wise operators of a voxel block ---------------------------------
 * They take (N, C) feature rows in the caller's order, contiguous, and stand
 * next to the convolution: the norm before it, the recurrence along the map's
 * schedule order, the gated linear unit after it.  All sums and statistics
 * are fp32, each output is rounded once, two calls with the same inputs give
 * bit-identical outputs.  C up to 4096.  Asynchronous on `stream`, no
 * allocation, no synchronisation; N = 0 enqueues nothing but the zeros of
 * outputs that sum over rows.  Outputs do not overlap inputs or the workspace
 * (but spconv_layernorm's y may be x).  The row operators' conventions on errors are
 * the library's. */

/* Layer norm over each row's channels.
 *   y[n, c] = (x[n, c] - mean[n]) * rstd[n] * weight[c] + bias[c]
 *   rstd[n] = 1 / sqrt(mean over c of (x - mean)^2 + eps)
 *   x, y   (dev) (N, C) of dtype, aligned to their elements; y may be x
 *   weight, bias (dev) float32 (C,), or NULL for 1 and 0
 *   mean, rstd   (dev) float32 (N,) written, or both NULL
 *   eps >= 0. */
int spconv_layernorm(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                     int64_t N, int C, float eps, int dtype, void* stream);

/* Gradient of spconv_layernorm, from the statistics that it wrote.  With
 * xhat = (x - mean) rstd and g = dout weight:
 *   dx      = rstd (g - mean_c(g) - xhat mean_c(g xhat))       (N, C), dtype
 *   dweight = sum_n dout xhat,  dbias = sum_n dout             float32 (C,)
 *   weight    (dev) as given to the forward (NULL for 1)
 *   dweight, dbias (dev) written, or both NULL (then no workspace is needed)
 *   workspace (dev) spconv_layernorm_grad_workspace_size bytes, 256-byte
 *             aligned: per-workgroup partial sums, added in a fixed order. */
int spconv_layernorm_grad_workspace_size(int64_t N, int C, int dtype, size_t* bytes);
int spconv_layernorm_grad(const void* dout, const void* x, const float* mean, const float* rstd,
                          const float* weight, void* workspace, size_t workspace_bytes, void* dx, float* dweight,
                          float* dbias, int64_t N, int C, int dtype, void* stream);

/* Gated linear unit of a feed-forward block: both projections, the activation
 * and the product in one pass.
 *   a = x w[0] + bias[0],  b = x w[1] + bias[1],  h = act(a) b
 *   x    (dev) (N, C),  w (dev) (2, C, F) row-major,  h (dev) (N, F) written;
 *        all of dtype and 16-byte aligned
 *   bias (dev) float32 (2, F), or NULL for zero
 *   act  SPCONV_SILU or SPCONV_GELU
 * C and F multiples of 8 up to 4096; others give SPCONV_E_UNSUPPORTED.  a and
 * b stay in fp32; the output is rounded once. */
int spconv_glu(const void* x, const void* w, const float* bias, void* h, int64_t N, int C, int F, int act,
               int dtype, void* stream);

/* Gradient of spconv_glu; a and b are computed again.
 *   da = dout b act'(a),  db = dout act(a)
 *   dx = da w[0]^T + db w[1]^T                     (N, C) of dtype
 *   dw[0] = x^T da,  dw[1] = x^T db                (2, C, F) of dtype
 *   dbias[s] = sum_n (da | db)                     float32 (2, F), or NULL
 * With SPCONV_BF16, da and db are rounded to bfloat16 once as the operands of
 * dx and dw (dbias adds them unrounded); all sums are fp32.
 *   workspace (dev) spconv_glu_grad_workspace_size bytes, 256-byte aligned:
 *             da and db, partial sums (added in a fixed order). */
int spconv_glu_grad_workspace_size(int64_t N, int C, int F, int dtype, size_t* bytes);
int spconv_glu_grad(const void* dout, const void* x, const void* w, const float* bias, void* workspace,
                    size_t workspace_bytes, void* dx, void* dw, float* dbias, int64_t N, int C, int F, int act,
                    int dtype, void* stream);

/* Gated linear recurrence over the voxels of each scene, in a given order
 * (the map's schedule order from spconv_nmap_export follows a space-filling
 * curve, 128 voxels at a time):
 *   h[t] = f[t] h[t-1] + (1 - f[t]) x[t],   f[t] = sigmoid(z[t])
 * per channel, along the positions t = offsets[b] .. offsets[b+1] - 1 of scene
 * b, from h0[b] before the first.
 *   x, z    (dev) (N, C) of dtype, in the caller's row order, aligned to their
 *           elements
 *   offsets (dev) int32 (scenes + 1,): 0 = offsets[0] <= ... <=
 *           offsets[scenes] = N; scenes without positions may stand anywhere
 *   order   (dev) int32 (N,): position t is row order[t], each row once; or
 *           NULL: position t is row t
 *   h0      (dev) float32 (scenes, C), or NULL for zero
 *   h       (dev) (N, C) written, of dtype: row order[t] holds h[t]
 *   last    (dev) float32 (scenes, C) written: each scene's last state (h0 of
 *           a scene without positions)
 *   workspace (dev) spconv_scan_workspace_size bytes, 256-byte aligned (may
 *           be NULL when that is 0)
 * f is a number of 32 bits too: a state kept by a constant open gate is off by
 * up to 2^-24 of itself per step.
 * An infinite state stays infinite until a gate is 0 in 32 bits (z below -87),
 * which makes it NaN; neither leaves its scene and channel.
 * Calls of more than 2^32 threads (the gradient from N C = 3.5e10 at the widths
 * that use their threads least) give SPCONV_E_UNSUPPORTED.
 * The contents of offsets and order are not checked: bad values give wrong
 * states, never an access outside the given arrays. */
int spconv_scan_workspace_size(int64_t N, int C, int dtype, size_t* bytes);
int spconv_scan(const void* x, const void* z, const int32_t* offsets, const int32_t* order, const float* h0,
                void* workspace, size_t workspace_bytes, void* h, float* last, int64_t N, int C, int scenes,
                int dtype, void* stream);

/* Gradient of spconv_scan.  With g[t] = dout[t] + f[t+1] g[t+1] along a scene
 * (dlast[b] added at its last position):
 *   dx[t] = (1 - f[t]) g[t],  dz[t] = g[t] (h[t-1] - x[t]) f[t] (1 - f[t]),
 *   dh0[b] = f[first] g[first]  (dlast[b] of a scene without positions)
 *   dout    (dev) (N, C) of dtype, in the caller's row order
 *   dlast   (dev) float32 (scenes, C): the gradient at `last`, or NULL for 0
 *   dx, dz  (dev) (N, C) written, of dtype, in the caller's row order
 *   dh0     (dev) float32 (scenes, C) written, or NULL
 * The states are computed again; nothing of the forward is needed.  Other
 * arguments, and what is said about them, are spconv_scan's. */
int spconv_scan_grad_workspace_size(int64_t N, int C, int dtype, size_t* bytes);
int spconv_scan_grad(const void* dout, const void* x, const void* z, const int32_t* offsets, const int32_t* order,
                     const float* h0, const float* dlast, void* workspace, size_t workspace_bytes, void* dx,
                     void* dz, float* dh0, int64_t N, int C, int scenes, int dtype, void* stream);

/* Release a handle (host memory only; the arena stays the caller's). */
void spconv_nmap_destroy(spconv_nmap* h);

const char* spconv_status_string(int status);
const char* spconv_last_error(void);
/* The same thread-local text under the name the hot-path boundary proposes
 * for SPCONV_E_HIP failures (it covers every failure, HIP or not). */
const char* spconv_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPCONV_MI355X_H */
