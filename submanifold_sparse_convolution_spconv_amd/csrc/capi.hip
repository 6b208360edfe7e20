// C interface of libspconv_mi355x: argument checks, handle management and
// dispatch to the builder and forward launchers.  Every check runs on the host
// before anything is enqueued.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>

#include "spconv_internal.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return status;
}

int hip_fail(hipError_t e, const char* where) {
    return fail(SPCONV_E_HIP, "%s: %s", where, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The sentinel N has to fit the int32 map (the page's kernel compares
// int nbr >= (int)N).
constexpr int64_t kMaxN = (int64_t)INT32_MAX - 1;
constexpr int kMaxKApi = 1000;

int check_nk(int64_t N, int K) {
    if (N < 0) return fail(SPCONV_E_INVALID, "N must be >= 0 (got %lld)", (long long)N);
    if (N > kMaxN) return fail(SPCONV_E_UNSUPPORTED, "N must be < 2^31-1 (got %lld)", (long long)N);
    if (K < 1 || K > kMaxKApi) return fail(SPCONV_E_INVALID, "K must be in [1, %d] (got %d)", kMaxKApi, K);
    return SPCONV_OK;
}

spconv_nmap* make_handle(int64_t N, int K, int dilation, int wrapped, const spc::ArenaLayout& al,
                         char* arena) {
    spconv_nmap* h = new (std::nothrow) spconv_nmap;
    if (!h) return nullptr;
    h->magic = kNmapMagic;
    h->N = N;
    h->Npad = al.Npad;
    h->ntiles = al.ntiles;
    h->K = K;
    h->dilation = dilation;
    h->wrapped = wrapped;
    h->nbr_m = (int32_t*)(arena + al.nbr_off);
    h->order = (int32_t*)(arena + al.order_off);
    h->blkmask = (uint16_t*)(arena + al.mask_off);
    h->dcount = (uint32_t*)(arena + al.dcount_off);
    h->drow = (int32_t*)(arena + al.drow_off);
    h->smap = (uint16_t*)(arena + al.smap_off);
    h->info = (spc::MapInfo*)(arena + al.info_off);
    h->valid_pairs = (N == 0) ? 0 : -1;
    h->max_distinct = (N == 0) ? 0 : -1;
    return h;
}

bool valid_handle(const spconv_nmap* h) { return h && h->magic == kNmapMagic; }

// Scratch of spconv_dgrad_noalloc: the input gradient's mirrored weights and
// their packed form, for callers that cannot allocate.  Each device holds its
// own copy from the library's first use there until the process ends.  In
// host code `scratch` only names the symbol; its device address comes from
// hipGetSymbolAddress, once per device with that device current, and only
// that address is handed to kernels.
constexpr size_t kNoAllocScratchBytes = SPCONV_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

constexpr int kMaxScratchDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxScratchDevices] = {};

// Device address of `scratch` on the device of `stream` (the current device
// for the null stream).
int scratch_address(void* stream, void** ptr, const char* where) {
    int dev = 0;
    hipError_t e = stream ? hipStreamGetDevice((hipStream_t)stream, &dev) : hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, where);
    if (dev < 0 || dev >= kMaxScratchDevices)
        return fail(SPCONV_E_UNSUPPORTED, "%s: device %d beyond the %d this library serves", where, dev,
                    kMaxScratchDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        int cur = 0;
        e = hipGetDevice(&cur);
        if (e != hipSuccess) return hip_fail(e, where);
        if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess) return hip_fail(e, where);
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (cur != dev) {
            const hipError_t e2 = hipSetDevice(cur);
            if (e == hipSuccess) e = e2;
        }
        if (e != hipSuccess) return hip_fail(e, where);
        if (!p || !aligned(p, 256)) return fail(SPCONV_E_HIP, "%s: scratch address %p not usable", where, p);
        g_scratch_ptr[dev] = p;
    }
    *ptr = g_scratch_ptr[dev];
    return SPCONV_OK;
}

}  // namespace

extern "C" {

int spconv_abi_version(void) { return SPCONV_ABI_VERSION; }

const char* spconv_last_error(void) { return g_last_error; }
const char* spconv_last_hip_error(void) { return g_last_error; }

const char* spconv_status_string(int status) {
    switch (status) {
        case SPCONV_OK: return "ok";
        case SPCONV_E_INVALID: return "invalid argument";
        case SPCONV_E_UNSUPPORTED: return "unsupported configuration";
        case SPCONV_E_COORD_RANGE: return "coordinate out of range [-2^20, 2^20)";
        case SPCONV_E_DUPLICATE: return "duplicate coordinate";
        case SPCONV_E_WORKSPACE: return "arena or workspace too small";
        case SPCONV_E_HIP: return "HIP runtime error";
        default: return "unknown status";
    }
}

int spconv_nmap_sizes(int64_t N, int K, size_t* arena_bytes, size_t* workspace_bytes) {
    int rc = check_nk(N, K);
    if (rc) return rc;
    if (arena_bytes) *arena_bytes = spc::arena_layout(N, K).total;
    if (workspace_bytes) *workspace_bytes = spc::workspace_layout(N).total;
    return SPCONV_OK;
}

static int build_impl(const int32_t* coords, int batches, int64_t N, int K, int dilation, void* arena,
                      size_t arena_bytes, void* workspace, size_t workspace_bytes, void* stream,
                      spconv_nmap** out, const char* name) {
    if (!out) return fail(SPCONV_E_INVALID, "out handle pointer is NULL");
    *out = nullptr;
    int rc = check_nk(N, K);
    if (rc) return rc;
    const int side = spc::cube_side(K);
    if (side < 0) return fail(SPCONV_E_INVALID, "K must be an odd cube 1, 27, 125, ... (got %d)", K);
    if (dilation < 1) return fail(SPCONV_E_INVALID, "dilation must be >= 1 (got %d)", dilation);
    if ((int64_t)dilation * (side - 1) / 2 >= (1 << 20))
        return fail(SPCONV_E_UNSUPPORTED, "dilation * radius must be < 2^20");
    if (batches > 0) {
        if (batches > (1 << 20)) return fail(SPCONV_E_UNSUPPORTED, "at most 2^20 batches (got %d)", batches);
        // each batch's x-slab must be wider than twice the stencil's reach
        const int64_t half = (int64_t)1 << (20 - spc::batch_slab_log2(batches));
        if ((int64_t)dilation * (side - 1) / 2 >= half)
            return fail(SPCONV_E_UNSUPPORTED, "%d batches leave x-slabs of %lld values, too narrow for "
                                              "dilation %d and K=%d", batches, (long long)(2 * half), dilation, K);
    }
    const spc::ArenaLayout al = spc::arena_layout(N, K);
    const spc::WorkspaceLayout wl = spc::workspace_layout(N);
    if (!arena) return fail(SPCONV_E_INVALID, "arena is NULL");
    if (!aligned(arena, 256)) return fail(SPCONV_E_INVALID, "arena must be 256-byte aligned");
    if (arena_bytes < al.total)
        return fail(SPCONV_E_WORKSPACE, "arena has %zu bytes, needs %zu", arena_bytes, al.total);
    if (N > 0) {
        if (!coords) return fail(SPCONV_E_INVALID, "coords is NULL");
        if (!aligned(coords, 4)) return fail(SPCONV_E_INVALID, "coords must be 4-byte aligned");
        if (!workspace) return fail(SPCONV_E_INVALID, "workspace is NULL");
        if (!aligned(workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
        if (workspace_bytes < wl.total)
            return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes,
                        wl.total);
    }
    spconv_nmap* h = make_handle(N, K, dilation, 0, al, (char*)arena);
    if (!h) return fail(SPCONV_E_INVALID, "out of host memory");
    if (N == 0) {
        *out = h;
        return SPCONV_OK;
    }
    spc::BuildFlags flags;
    memset(&flags, 0, sizeof flags);
    hipError_t e = spc::launch_build(coords, batches, N, K, dilation, side, al, (char*)arena, wl,
                                     (char*)workspace, (hipStream_t)stream, &flags);
    if (e != hipSuccess) {
        delete h;
        return hip_fail(e, name);
    }
    if (flags.range_error) {
        delete h;
        if (batches > 0) {
            const int64_t half = (int64_t)1 << (20 - spc::batch_slab_log2(batches));
            const int64_t reach = (int64_t)dilation * (side - 1) / 2;
            return fail(SPCONV_E_COORD_RANGE,
                        "a batch index outside [0, %d), an x outside [%lld, %lld) or a y, z outside [-2^20, 2^20)",
                        batches, (long long)(-half + reach), (long long)(half - reach));
        }
        return fail(SPCONV_E_COORD_RANGE, "a coordinate lies outside [-2^20, 2^20)");
    }
    if (flags.duplicate) {
        delete h;
        return fail(SPCONV_E_DUPLICATE, "two voxels share a coordinate");
    }
    h->valid_pairs = (int64_t)flags.valid_pairs;
    h->max_distinct = flags.max_distinct == spc::kNoDistinct ? (int64_t)spc::kDistinctListCap + 1
                                                              : (int64_t)flags.max_distinct;
    *out = h;
    return SPCONV_OK;
}

int spconv_build_nmap(const int32_t* coords, int64_t N, int K, int dilation, void* arena,
                      size_t arena_bytes, void* workspace, size_t workspace_bytes, void* stream,
                      spconv_nmap** out) {
    return build_impl(coords, 0, N, K, dilation, arena, arena_bytes, workspace, workspace_bytes, stream, out,
                      "spconv_build_nmap");
}

int spconv_build_nmap_batched(const int32_t* coords, int64_t N, int batches, int K, int dilation, void* arena,
                              size_t arena_bytes, void* workspace, size_t workspace_bytes, void* stream,
                              spconv_nmap** out) {
    if (batches < 1) return fail(SPCONV_E_INVALID, "batches must be >= 1 (got %d)", batches);
    return build_impl(coords, batches, N, K, dilation, arena, arena_bytes, workspace, workspace_bytes, stream,
                      out, "spconv_build_nmap_batched");
}

int spconv_nmap_wrap(const int32_t* nbr, int64_t N, int K, void* arena, size_t arena_bytes,
                     void* stream, spconv_nmap** out) {
    if (!out) return fail(SPCONV_E_INVALID, "out handle pointer is NULL");
    *out = nullptr;
    int rc = check_nk(N, K);
    if (rc) return rc;
    const spc::ArenaLayout al = spc::arena_layout(N, K);
    if (!arena) return fail(SPCONV_E_INVALID, "arena is NULL");
    if (!aligned(arena, 256)) return fail(SPCONV_E_INVALID, "arena must be 256-byte aligned");
    if (arena_bytes < al.total)
        return fail(SPCONV_E_WORKSPACE, "arena has %zu bytes, needs %zu", arena_bytes, al.total);
    if (N > 0 && !nbr) return fail(SPCONV_E_INVALID, "nbr is NULL");
    if (N > 0 && !aligned(nbr, 4)) return fail(SPCONV_E_INVALID, "nbr must be 4-byte aligned");
    spconv_nmap* h = make_handle(N, K, 1, 1, al, (char*)arena);
    if (!h) return fail(SPCONV_E_INVALID, "out of host memory");
    if (N > 0) {
        hipError_t e = spc::launch_wrap(nbr, N, K, al, (char*)arena, (hipStream_t)stream);
        if (e != hipSuccess) {
            delete h;
            return hip_fail(e, "spconv_nmap_wrap");
        }
    }
    *out = h;
    return SPCONV_OK;
}

int spconv_nmap_export(const spconv_nmap* h, int32_t* nbr_out, int32_t* order_out, void* stream) {
    if (!valid_handle(h)) return fail(SPCONV_E_INVALID, "invalid handle");
    if ((nbr_out && !aligned(nbr_out, 4)) || (order_out && !aligned(order_out, 4)))
        return fail(SPCONV_E_INVALID, "outputs must be 4-byte aligned");
    if (h->N == 0 || (!nbr_out && !order_out)) return SPCONV_OK;
    hipError_t e = spc::launch_export(h->nbr_m, h->order, h->N, h->Npad, h->K, nbr_out, order_out,
                                      (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_nmap_export");
}

int spconv_nmap_info(const spconv_nmap* h, int64_t* N, int* K, int* dilation, int64_t* valid_pairs,
                     void* stream) {
    if (!valid_handle(h)) return fail(SPCONV_E_INVALID, "invalid handle");
    if (N) *N = h->N;
    if (K) *K = h->K;
    if (dilation) *dilation = h->dilation;
    if (valid_pairs) {
        if (h->valid_pairs < 0) {
            unsigned long long v = 0;
            hipError_t e = hipMemcpyAsync(&v, &h->info->valid_pairs, sizeof v, hipMemcpyDeviceToHost,
                                          (hipStream_t)stream);
            if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
            if (e != hipSuccess) return hip_fail(e, "spconv_nmap_info");
            const_cast<spconv_nmap*>(h)->valid_pairs = (int64_t)v;
        }
        *valid_pairs = h->valid_pairs;
    }
    return SPCONV_OK;
}

static int forward_impl(const void* feats, int feats_dtype, const spconv_nmap* nmap, const void* w,
                        const void* wpack, const float* bias, void* out, int Ci, int Co, int dtype, void* stream,
                        const char* name, void* cast_ws = nullptr) {
    if (!valid_handle(nmap)) return fail(SPCONV_E_INVALID, "invalid handle");
    if (dtype != SPCONV_F32 && dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", dtype);
    if (feats_dtype != SPCONV_F32 && feats_dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "feats_dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", feats_dtype);
    if (Ci < 1 || Co < 1) return fail(SPCONV_E_INVALID, "Ci and Co must be >= 1");
    if (!spc::forward_supported(dtype, Ci, Co))
        return fail(SPCONV_E_UNSUPPORTED,
                    "no kernel for Ci=%d Co=%d (Ci in {32,64,128,256}, Co a multiple of 32 <= 4096)",
                    Ci, Co);
    if (nmap->N == 0) return SPCONV_OK;
    if (!feats || !w || !out) return fail(SPCONV_E_INVALID, "feats, w and out must be non-NULL");
    if (!aligned(feats, 16) || !aligned(w, 16) || !aligned(out, 16))
        return fail(SPCONV_E_INVALID, "feats, w and out must be 16-byte aligned");
    if (bias && !aligned(bias, 4)) return fail(SPCONV_E_INVALID, "bias must be 4-byte aligned");
    if (wpack && spc::packed_weight_bytes(nmap->K, Ci, Co, dtype) == 0) wpack = nullptr;  // no packed form
    if (wpack && !aligned(wpack, 16)) return fail(SPCONV_E_INVALID, "wpack must be 16-byte aligned");
    spc::ForwardArgs a;
    a.feats = feats;
    a.nbr_m = nmap->nbr_m;
    a.order = nmap->order;
    a.blkmask = nmap->blkmask;
    a.dcount = nmap->dcount;
    a.drow = nmap->drow;
    a.smap = nmap->smap;
    a.max_distinct = nmap->max_distinct;
    a.w = w;
    a.wpack = wpack;
    a.bias = bias;
    a.out = out;
    a.N = nmap->N;
    a.Npad = nmap->Npad;
    a.K = nmap->K;
    a.Ci = Ci;
    a.Co = Co;
    a.dtype = dtype;
    a.feats_dtype = feats_dtype;
    a.cast_ws = cast_ws;
    // The tile kernel reads w in its packed form only: without one, pack w
    // into a stream-ordered allocation that is released on the stream after
    // the forward.
    hipStream_t st = (hipStream_t)stream;
    void* tmp = nullptr;
    const int fdt = (feats_dtype == SPCONV_F32 && dtype == SPCONV_BF16 && cast_ws) ? SPCONV_BF16 : feats_dtype;
    if (!wpack && spc::tile_forward(dtype, fdt, Ci, Co)) {
        hipError_t e = hipMallocAsync(&tmp, spc::packed_weight_bytes(nmap->K, Ci, Co, dtype), st);
        if (e != hipSuccess) return hip_fail(e, name);
        e = spc::launch_pack_weights(w, nmap->K, Ci, Co, dtype, tmp, st);
        if (e != hipSuccess) {
            (void)hipFreeAsync(tmp, st);
            return hip_fail(e, name);
        }
        a.wpack = tmp;
    }
    hipError_t e = spc::launch_forward(a, st);
    if (tmp) {
        const hipError_t ef = hipFreeAsync(tmp, st);
        if (e == hipSuccess) e = ef;
    }
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, name);
}

int spconv_forward(const void* feats, const spconv_nmap* nmap, const void* w, const float* bias,
                   void* out, int Ci, int Co, int dtype, void* stream) {
    return forward_impl(feats, dtype, nmap, w, nullptr, bias, out, Ci, Co, dtype, stream, "spconv_forward");
}

int spconv_forward_mixed_workspace_size(int64_t N, int Ci, int feats_dtype, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    if (N < 0 || N > kMaxN) return fail(SPCONV_E_INVALID, "N must be in [0, 2^31-1) (got %lld)", (long long)N);
    if (Ci < 1) return fail(SPCONV_E_INVALID, "Ci must be >= 1");
    if ((feats_dtype != SPCONV_F32 && feats_dtype != SPCONV_BF16) || (dtype != SPCONV_F32 && dtype != SPCONV_BF16))
        return fail(SPCONV_E_INVALID, "feats_dtype and dtype must be SPCONV_F32 or SPCONV_BF16");
    *bytes = spc::cast_workspace_bytes(N, Ci, feats_dtype, dtype);
    return SPCONV_OK;
}

int spconv_forward_mixed(const void* feats, int feats_dtype, const spconv_nmap* nmap, const void* w,
                         const void* wpack, const float* bias, void* out, int Ci, int Co, int dtype,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_handle(nmap)) return fail(SPCONV_E_INVALID, "invalid handle");
    size_t need = 0;
    int rc = spconv_forward_mixed_workspace_size(nmap->N, Ci, feats_dtype, dtype, &need);
    if (rc) return rc;
    if (need == 0 || nmap->N == 0) workspace = nullptr;   // no cast pass for this pairing
    if (workspace) {
        if (!aligned(workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
        if (workspace_bytes < need)
            return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
    return forward_impl(feats, feats_dtype, nmap, w, wpack, bias, out, Ci, Co, dtype, stream,
                        "spconv_forward_mixed", workspace);
}

int spconv_pack_weights_size(int K, int Ci, int Co, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    if (K < 1 || K > kMaxKApi) return fail(SPCONV_E_INVALID, "K must be in [1, %d] (got %d)", kMaxKApi, K);
    if (dtype != SPCONV_F32 && dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", dtype);
    if (!spc::forward_supported(dtype, Ci, Co))
        return fail(SPCONV_E_UNSUPPORTED, "no kernel for Ci=%d Co=%d", Ci, Co);
    *bytes = spc::packed_weight_bytes(K, Ci, Co, dtype);
    return SPCONV_OK;
}

int spconv_pack_weights(const void* w, int K, int Ci, int Co, int dtype, void* wpack, size_t wpack_bytes,
                        void* stream) {
    size_t need = 0;
    int rc = spconv_pack_weights_size(K, Ci, Co, dtype, &need);
    if (rc) return rc;
    if (need == 0) return SPCONV_OK;
    if (!w || !wpack) return fail(SPCONV_E_INVALID, "w and wpack must be non-NULL");
    if (!aligned(w, 16) || !aligned(wpack, 16)) return fail(SPCONV_E_INVALID, "w and wpack must be 16-byte aligned");
    if (wpack_bytes < need) return fail(SPCONV_E_WORKSPACE, "wpack has %zu bytes, needs %zu", wpack_bytes, need);
    hipError_t e = spc::launch_pack_weights(w, K, Ci, Co, dtype, wpack, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_pack_weights");
}


int spconv_forward_packed(const void* feats, const spconv_nmap* nmap, const void* w, const void* wpack,
                          const float* bias, void* out, int Ci, int Co, int dtype, void* stream) {
    if (valid_handle(nmap) && nmap->N > 0 && !wpack && spc::packed_weight_bytes(nmap->K, Ci, Co, dtype) > 0)
        return fail(SPCONV_E_INVALID, "wpack is NULL");
    return forward_impl(feats, dtype, nmap, w, wpack, bias, out, Ci, Co, dtype, stream, "spconv_forward_packed");
}

// Workspace of spconv_dgrad: the mirrored, transposed weights (K x Co x Ci
// elements), then their packed form when the bf16 kernel has one.
static size_t dgrad_wt_bytes(int K, int Ci, int Co, int dtype) {
    return spc::align_up((size_t)K * Ci * Co * (dtype == SPCONV_BF16 ? 2 : 4), 256);
}

int spconv_dgrad_workspace_size(int K, int Ci, int Co, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    if (K < 1 || K > kMaxKApi) return fail(SPCONV_E_INVALID, "K must be in [1, %d] (got %d)", kMaxKApi, K);
    if (dtype != SPCONV_F32 && dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", dtype);
    // the gradient runs the forward with the roles of Ci and Co exchanged
    if (!spc::forward_supported(dtype, Co, Ci))
        return fail(SPCONV_E_UNSUPPORTED,
                    "no input-gradient kernel for Ci=%d Co=%d (Co in {32,64,128,256}, Ci a multiple of 32 <= 4096)",
                    Ci, Co);
    *bytes = dgrad_wt_bytes(K, Ci, Co, dtype) + spc::packed_weight_bytes(K, Co, Ci, dtype);
    return SPCONV_OK;
}

int spconv_dgrad(const void* dout, const spconv_nmap* nmap, const void* w, void* workspace,
                 size_t workspace_bytes, void* dfeats, int Ci, int Co, int dtype, void* stream) {
    if (!valid_handle(nmap)) return fail(SPCONV_E_INVALID, "invalid handle");
    if (nmap->wrapped)
        return fail(SPCONV_E_UNSUPPORTED, "the input gradient needs a map from spconv_build_nmap "
                                          "(a caller-made map need not be its own mirror)");
    size_t need = 0;
    int rc = spconv_dgrad_workspace_size(nmap->K, Ci, Co, dtype, &need);
    if (rc) return rc;
    if (nmap->N == 0) return SPCONV_OK;
    if (!w || !workspace) return fail(SPCONV_E_INVALID, "w and workspace must be non-NULL");
    if (!aligned(w, 16) || !aligned(workspace, 256))
        return fail(SPCONV_E_INVALID, "w must be 16-byte and workspace 256-byte aligned");
    if (workspace_bytes < need)
        return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    void* wt = workspace;
    const size_t pk = spc::packed_weight_bytes(nmap->K, Co, Ci, dtype);
    void* wtpack = pk ? (char*)workspace + dgrad_wt_bytes(nmap->K, Ci, Co, dtype) : nullptr;
    hipError_t e = spc::launch_mirror_weights(w, nmap->K, Ci, Co, dtype, wt, (hipStream_t)stream);
    if (e == hipSuccess && wtpack) e = spc::launch_pack_weights(wt, nmap->K, Co, Ci, dtype, wtpack, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "spconv_dgrad");
    return forward_impl(dout, dtype, nmap, wt, wtpack, nullptr, dfeats, Co, Ci, dtype, stream, "spconv_dgrad");
}

int spconv_dgrad_noalloc(const void* dout, const spconv_nmap* nmap, const void* w, void* dfeats, int Ci, int Co,
                         int dtype, void* stream) {
    if (!valid_handle(nmap)) return fail(SPCONV_E_INVALID, "invalid handle");
    size_t need = 0;
    int rc = spconv_dgrad_workspace_size(nmap->K, Ci, Co, dtype, &need);
    if (rc) return rc;
    if (need > kNoAllocScratchBytes)
        return fail(SPCONV_E_WORKSPACE,
                    "spconv_dgrad_noalloc: K=%d Ci=%d Co=%d needs %zu bytes of scratch, beyond its fixed %zu "
                    "(use spconv_dgrad with a workspace)",
                    nmap->K, Ci, Co, need, kNoAllocScratchBytes);
    if (nmap->N == 0) return spconv_dgrad(dout, nmap, w, nullptr, 0, dfeats, Ci, Co, dtype, stream);
    void* ptr = nullptr;
    rc = scratch_address(stream, &ptr, "spconv_dgrad_noalloc");
    if (rc) return rc;
    return spconv_dgrad(dout, nmap, w, ptr, kNoAllocScratchBytes, dfeats, Ci, Co, dtype, stream);
}

int spconv_wgrad_workspace_size(int64_t N, int K, int Ci, int Co, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    int rc = check_nk(N, K);
    if (rc) return rc;
    if (dtype != SPCONV_F32 && dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", dtype);
    if (!spc::wgrad_supported(dtype, Ci, Co))
        return fail(SPCONV_E_UNSUPPORTED, "no weight-gradient kernel for Ci=%d Co=%d (multiples of 32 up to 4096)",
                    Ci, Co);
    *bytes = spc::wgrad_workspace_bytes(N, K, Ci, Co, dtype);
    return SPCONV_OK;
}

int spconv_wgrad(const void* feats, const void* dout, const spconv_nmap* nmap, void* workspace,
                 size_t workspace_bytes, void* dw, int Ci, int Co, int dtype, void* stream) {
    if (!valid_handle(nmap)) return fail(SPCONV_E_INVALID, "invalid handle");
    size_t need = 0;
    int rc = spconv_wgrad_workspace_size(nmap->N, nmap->K, Ci, Co, dtype, &need);
    if (rc) return rc;
    if (!dw) return fail(SPCONV_E_INVALID, "dw is NULL");
    if (!aligned(dw, 16)) return fail(SPCONV_E_INVALID, "dw must be 16-byte aligned");
    if (nmap->N > 0) {
        if (!feats || !dout || !workspace) return fail(SPCONV_E_INVALID, "feats, dout and workspace must be non-NULL");
        if (!aligned(feats, 16) || !aligned(dout, 16) || !aligned(workspace, 256))
            return fail(SPCONV_E_INVALID, "feats and dout must be 16-byte and workspace 256-byte aligned");
        if (workspace_bytes < need)
            return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
    spc::WgradArgs a;
    a.feats = feats;
    a.dout = dout;
    a.nbr_m = nmap->nbr_m;
    a.order = nmap->order;
    a.blkmask = nmap->blkmask;
    a.dcount = nmap->dcount;
    a.drow = nmap->drow;
    a.smap = nmap->smap;
    a.max_distinct = nmap->max_distinct;
    a.workspace = workspace;
    a.dw = dw;
    a.N = nmap->N;
    a.Npad = nmap->Npad;
    a.K = nmap->K;
    a.Ci = Ci;
    a.Co = Co;
    a.dtype = dtype;
    // with no rows the gradient is zero (written by the kernels; no workspace used)
    hipError_t e = spc::launch_wgrad(a, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_wgrad");
}

// Checks shared by the row-wise operators: rows, channels, element type.
static int check_rows(int64_t N, int C, int dtype, const char* what) {
    if (dtype != SPCONV_F32 && dtype != SPCONV_BF16)
        return fail(SPCONV_E_INVALID, "dtype must be SPCONV_F32 or SPCONV_BF16 (got %d)", dtype);
    if (N < 0) return fail(SPCONV_E_INVALID, "N must be >= 0 (got %lld)", (long long)N);
    if (N > kMaxN) return fail(SPCONV_E_UNSUPPORTED, "N must be < 2^31-1 (got %lld)", (long long)N);
    if (C < 1) return fail(SPCONV_E_INVALID, "%s must be >= 1 (got %d)", what, C);
    if (C > spc::kMaxRowChannels)
        return fail(SPCONV_E_UNSUPPORTED, "%s must be <= %d (got %d)", what, spc::kMaxRowChannels, C);
    return SPCONV_OK;
}
static size_t elem_size(int dtype) { return dtype == SPCONV_BF16 ? 2 : 4; }

int spconv_layernorm(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                     int64_t N, int C, float eps, int dtype, void* stream) {
    int rc = check_rows(N, C, dtype, "C");
    if (rc) return rc;
    if (!(eps >= 0.f)) return fail(SPCONV_E_INVALID, "eps must be >= 0 (got %g)", (double)eps);
    if (!mean != !rstd) return fail(SPCONV_E_INVALID, "mean and rstd must be given together");
    if (N == 0) return SPCONV_OK;
    if (!x || !y) return fail(SPCONV_E_INVALID, "x and y must be non-NULL");
    const size_t es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(y, es)) return fail(SPCONV_E_INVALID, "x and y must be aligned to their elements");
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SPCONV_E_INVALID, "weight, bias, mean and rstd must be 4-byte aligned");
    hipError_t e = spc::launch_norm({x, weight, bias, y, mean, rstd, N, C, eps, dtype}, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_layernorm");
}

int spconv_layernorm_grad_workspace_size(int64_t N, int C, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    int rc = check_rows(N, C, dtype, "C");
    if (rc) return rc;
    *bytes = spc::norm_grad_workspace_bytes(N, C, dtype);
    return SPCONV_OK;
}

int spconv_layernorm_grad(const void* dout, const void* x, const float* mean, const float* rstd,
                          const float* weight, void* workspace, size_t workspace_bytes, void* dx, float* dweight,
                          float* dbias, int64_t N, int C, int dtype, void* stream) {
    size_t need = 0;
    int rc = spconv_layernorm_grad_workspace_size(N, C, dtype, &need);
    if (rc) return rc;
    if (!dweight != !dbias) return fail(SPCONV_E_INVALID, "dweight and dbias must be given together");
    const size_t es = elem_size(dtype);
    if (N > 0) {
        if (!dout || !x || !mean || !rstd || !dx)
            return fail(SPCONV_E_INVALID, "dout, x, mean, rstd and dx must be non-NULL");
        if (!aligned(dout, es) || !aligned(x, es) || !aligned(dx, es))
            return fail(SPCONV_E_INVALID, "dout, x and dx must be aligned to their elements");
        if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(weight, 4))
            return fail(SPCONV_E_INVALID, "mean, rstd and weight must be 4-byte aligned");
        if (dweight) {
            if (!workspace) return fail(SPCONV_E_INVALID, "workspace is NULL");
            if (!aligned(workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
            if (workspace_bytes < need)
                return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
        }
    }
    if (!aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(SPCONV_E_INVALID, "dweight and dbias must be 4-byte aligned");
    // with no rows dweight and dbias are zero (written by the kernel; no workspace used)
    hipError_t e = spc::launch_norm_grad({dout, x, mean, rstd, weight, workspace, dx, dweight, dbias, N, C, dtype},
                                         (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_layernorm_grad");
}

static int check_glu(int64_t N, int C, int F, int act, int dtype) {
    int rc = check_rows(N, C, dtype, "C");
    if (rc) return rc;
    rc = check_rows(N, F, dtype, "F");
    if (rc) return rc;
    if (act != SPCONV_SILU && act != SPCONV_GELU)
        return fail(SPCONV_E_INVALID, "act must be SPCONV_SILU or SPCONV_GELU (got %d)", act);
    if (C % 8 || F % 8) return fail(SPCONV_E_UNSUPPORTED, "no kernel for C=%d F=%d (multiples of 8 up to %d)", C, F,
                                    spc::kMaxRowChannels);
    return SPCONV_OK;
}

int spconv_glu(const void* x, const void* w, const float* bias, void* h, int64_t N, int C, int F, int act,
               int dtype, void* stream) {
    int rc = check_glu(N, C, F, act, dtype);
    if (rc) return rc;
    if (N == 0) return SPCONV_OK;
    if (!x || !w || !h) return fail(SPCONV_E_INVALID, "x, w and h must be non-NULL");
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(h, 16))
        return fail(SPCONV_E_INVALID, "x, w and h must be 16-byte aligned");
    if (!aligned(bias, 4)) return fail(SPCONV_E_INVALID, "bias must be 4-byte aligned");
    hipError_t e = spc::launch_glu({x, w, bias, nullptr, nullptr, h, nullptr, nullptr, N, C, F, act, dtype}, false,
                                   (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_glu");
}

int spconv_glu_grad_workspace_size(int64_t N, int C, int F, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    int rc = check_glu(N, C, F, SPCONV_SILU, dtype);
    if (rc) return rc;
    *bytes = spc::glu_grad_workspace_bytes(N, C, F, dtype);
    return SPCONV_OK;
}

int spconv_glu_grad(const void* dout, const void* x, const void* w, const float* bias, void* workspace,
                    size_t workspace_bytes, void* dx, void* dw, float* dbias, int64_t N, int C, int F, int act,
                    int dtype, void* stream) {
    int rc = check_glu(N, C, F, act, dtype);
    if (rc) return rc;
    const size_t need = spc::glu_grad_workspace_bytes(N, C, F, dtype);
    if (!dw) return fail(SPCONV_E_INVALID, "dw is NULL");
    if (!aligned(dw, 16)) return fail(SPCONV_E_INVALID, "dw must be 16-byte aligned");
    if (!aligned(bias, 4) || !aligned(dbias, 4)) return fail(SPCONV_E_INVALID, "bias and dbias must be 4-byte aligned");
    if (N > 0) {
        if (!dout || !x || !w || !dx || !workspace)
            return fail(SPCONV_E_INVALID, "dout, x, w, dx and workspace must be non-NULL");
        if (!aligned(dout, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(dx, 16) || !aligned(workspace, 256))
            return fail(SPCONV_E_INVALID, "dout, x, w and dx must be 16-byte and workspace 256-byte aligned");
        if (workspace_bytes < need)
            return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
    // with no rows dw and dbias are zero (written by the kernels; no workspace used)
    hipError_t e = spc::launch_glu({x, w, bias, dout, workspace, dx, dw, dbias, N, C, F, act, dtype}, true,
                                   (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "spconv_glu_grad");
}

static int scan_size(int64_t N, int C, int dtype, bool grad, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    int rc = check_rows(N, C, dtype, "C");
    if (rc) return rc;
    if (!spc::scan_fits(N, C, grad))
        return fail(SPCONV_E_UNSUPPORTED, "N=%lld rows of C=%d channels need more than 2^32 threads", (long long)N, C);
    *bytes = spc::scan_workspace_bytes(N, C, dtype, grad);
    return SPCONV_OK;
}

// Checks of both directions; a.out .. a.state are the outputs.
static int scan_impl(const spc::ScanArgs& a, bool grad, size_t workspace_bytes, void* stream, const char* name) {
    size_t need = 0;
    int rc = scan_size(a.N, a.C, a.dtype, grad, &need);
    if (rc) return rc;
    if (a.scenes < 1) return fail(SPCONV_E_INVALID, "scenes must be >= 1 (got %d)", a.scenes);
    if (!a.offsets) return fail(SPCONV_E_INVALID, "offsets is NULL");
    if (!grad && !a.state) return fail(SPCONV_E_INVALID, "last is NULL");
    if (!aligned(a.offsets, 4) || !aligned(a.order, 4) || !aligned(a.h0, 4) || !aligned(a.dlast, 4) ||
        !aligned(a.state, 4))
        return fail(SPCONV_E_INVALID, "offsets, order and the scenes' states must be 4-byte aligned");
    if (a.N > 0) {
        const size_t es = elem_size(a.dtype);
        if (!a.x || !a.z || !a.out || (grad && (!a.dout || !a.dz)))
            return fail(SPCONV_E_INVALID, grad ? "dout, x, z, dx and dz must be non-NULL"
                                               : "x, z and h must be non-NULL");
        if (!aligned(a.x, es) || !aligned(a.z, es) || !aligned(a.out, es) || !aligned(a.dout, es) ||
            !aligned(a.dz, es))
            return fail(SPCONV_E_INVALID, "feature rows must be aligned to their elements");
        if (need) {
            if (!a.workspace) return fail(SPCONV_E_INVALID, "workspace is NULL");
            if (!aligned(a.workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
            if (workspace_bytes < need)
                return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
        }
    }
    hipError_t e = spc::launch_scan(a, grad, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, name);
}

int spconv_scan_workspace_size(int64_t N, int C, int dtype, size_t* bytes) {
    return scan_size(N, C, dtype, false, bytes);
}

int spconv_scan(const void* x, const void* z, const int32_t* offsets, const int32_t* order, const float* h0,
                void* workspace, size_t workspace_bytes, void* h, float* last, int64_t N, int C, int scenes,
                int dtype, void* stream) {
    return scan_impl({x, z, nullptr, offsets, order, h0, nullptr, workspace, h, nullptr, last, N, C, scenes, dtype},
                     false, workspace_bytes, stream, "spconv_scan");
}

int spconv_scan_grad_workspace_size(int64_t N, int C, int dtype, size_t* bytes) {
    return scan_size(N, C, dtype, true, bytes);
}

int spconv_scan_grad(const void* dout, const void* x, const void* z, const int32_t* offsets, const int32_t* order,
                     const float* h0, const float* dlast, void* workspace, size_t workspace_bytes, void* dx,
                     void* dz, float* dh0, int64_t N, int C, int scenes, int dtype, void* stream) {
    return scan_impl({x, z, dout, offsets, order, h0, dlast, workspace, dx, dz, dh0, N, C, scenes, dtype}, true,
                     workspace_bytes, stream, "spconv_scan_grad");
}

int spconv_rotary_freqs(int pairs, int axes, double base, double factor, double original, double* freqs) {
    if (!freqs) return fail(SPCONV_E_INVALID, "freqs is NULL");
    if (axes < 1 || axes > 8 || pairs < 1 || pairs > spc::kMaxRowChannels / 2 || pairs % axes)
        return fail(SPCONV_E_INVALID, "pairs must be a multiple of axes (1..8) up to %d (got %d, %d)",
                    spc::kMaxRowChannels / 2, pairs, axes);
    if (!(base > 1.0) || !(factor >= 1.0) || !(original >= 0.0) || !std::isfinite(base) || !std::isfinite(factor) ||
        !std::isfinite(original))
        return fail(SPCONV_E_INVALID, "base must be > 1, factor >= 1 and original >= 0 (got %g, %g, %g)", base, factor,
                    original);
    const int n = pairs / axes;
    for (int i = 0; i < pairs; ++i) {
        const double f = std::pow(base, -(double)(i % n) / n);
        const double turns = original * f / 6.283185307179586;
        const double keep = original > 0 ? std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0)) : 0.0;
        freqs[i] = f / factor * (1.0 - keep) + f * keep;
    }
    return SPCONV_OK;
}

// Whether an output's rows or heads, D elements each, lie in one another: a stride
// is shorter than D, or the longer one than all that the shorter one spans.
static bool heads_overlap(const int64_t* strides, int64_t rows, int heads, int D) {
    const int64_t r = std::abs(strides[0]), h = std::abs(strides[1]);
    if ((rows > 1 && r < D) || (heads > 1 && h < D)) return true;
    if (rows <= 1 || heads <= 1) return false;
    return (r < h ? rows : heads) - 1 > (std::max(r, h) - D) / std::min(r, h);
}

static int rotary_impl(const void* x, const int32_t* positions, int64_t pos_stride, const double* freqs, void* y,
                       const int64_t* strides, int64_t N, int H, int D, int pairs, int axes, int layout, float gain,
                       int dtype, void* stream, bool back, const char* name) {
    int rc = check_rows(N, D, dtype, "D");
    if (!rc) rc = check_rows(N, H, dtype, "H");
    if (rc) return rc;
    if (axes < 1 || axes > 8 || pairs < 1 || pairs % axes || 2 * (int64_t)pairs > D)
        return fail(SPCONV_E_INVALID, "pairs must be a multiple of axes (1..8) and 2 pairs <= D (got %d, %d, D=%d)",
                    pairs, axes, D);
    if (layout != SPCONV_HALF && layout != SPCONV_INTERLEAVED)
        return fail(SPCONV_E_INVALID, "layout must be SPCONV_HALF or SPCONV_INTERLEAVED (got %d)", layout);
    if (N == 0) return SPCONV_OK;
    if (!x || !positions || !freqs || !y) return fail(SPCONV_E_INVALID, "rows, positions and freqs must be non-NULL");
    const size_t es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(positions, 4) || !aligned(freqs, 8))
        return fail(SPCONV_E_INVALID, "rows, positions and freqs must be aligned to their elements");
    spc::RotaryArgs a{x, positions, pos_stride, freqs, y, {(int64_t)H * D, D}, {(int64_t)H * D, D}, N, H, D,
                      pairs, axes, layout, gain, dtype};
    if (strides) {
        for (int i = 0; i < 2; ++i) {
            a.xs[i] = strides[i];
            a.ys[i] = strides[2 + i];
        }
        if (x == y && (a.xs[0] != a.ys[0] || a.xs[1] != a.ys[1]))
            return fail(SPCONV_E_INVALID, "in place, both strides must be the same");
        if (heads_overlap(a.ys, N, H, D)) return fail(SPCONV_E_INVALID, "rows or heads of the output overlap");
    }
    hipError_t e = spc::launch_rotary(a, back, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, name);
}

int spconv_rotary(const void* x, const int32_t* positions, int64_t pos_stride, const double* freqs, void* y,
                  const int64_t* strides, int64_t N, int H, int D, int pairs, int axes, int layout, float gain,
                  int dtype, void* stream) {
    return rotary_impl(x, positions, pos_stride, freqs, y, strides, N, H, D, pairs, axes, layout, gain, dtype, stream,
                       false, "spconv_rotary");
}

int spconv_rotary_grad(const void* dout, const int32_t* positions, int64_t pos_stride, const double* freqs, void* dx,
                       const int64_t* strides, int64_t N, int H, int D, int pairs, int axes, int layout, float gain,
                       int dtype, void* stream) {
    return rotary_impl(dout, positions, pos_stride, freqs, dx, strides, N, H, D, pairs, axes, layout, gain, dtype,
                       stream, true, "spconv_rotary_grad");
}

// Sizes of a group norm, and the workspace they need.
static int check_group(int64_t N, int C, int scenes, int groups, int dtype, bool grad, size_t* bytes) {
    int rc = check_rows(N, C, dtype, "C");
    if (rc) return rc;
    if (scenes < 1) return fail(SPCONV_E_INVALID, "scenes must be >= 1 (got %d)", scenes);
    if (groups < 1 || C % groups)
        return fail(SPCONV_E_INVALID, "C must be a multiple of groups (got C=%d groups=%d)", C, groups);
    if (!spc::group_fits(N, C, scenes, groups, dtype, grad))
        return fail(SPCONV_E_UNSUPPORTED, "%d scenes of %d groups need more than 2^32 threads", scenes, groups);
    *bytes = spc::group_workspace_bytes(N, C, scenes, groups, dtype);
    return SPCONV_OK;
}

int spconv_groupnorm_workspace_size(int64_t N, int C, int scenes, int groups, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    return check_group(N, C, scenes, groups, dtype, false, bytes);
}

// Checks of both directions.
static int group_impl(const spc::GroupArgs& a, bool grad, size_t workspace_bytes, void* stream, const char* name) {
    size_t need = 0;
    int rc = check_group(a.N, a.C, a.scenes, a.groups, a.dtype, grad, &need);
    if (rc) return rc;
    if (!(a.eps >= 0.f)) return fail(SPCONV_E_INVALID, "eps must be >= 0 (got %g)", (double)a.eps);
    if (a.act != SPCONV_SILU && a.act != SPCONV_GELU && a.act != SPCONV_LINEAR)
        return fail(SPCONV_E_INVALID, "act must be SPCONV_SILU, SPCONV_GELU or SPCONV_LINEAR (got %d)", a.act);
    if (grad ? !a.mean || !a.rstd : !a.mean != !a.rstd)
        return fail(SPCONV_E_INVALID, "mean and rstd must be given%s", grad ? "" : " together");
    if (!a.dweight != !a.dbias) return fail(SPCONV_E_INVALID, "dweight and dbias must be given together");
    if (!a.offsets) return fail(SPCONV_E_INVALID, "offsets is NULL");
    if (!a.workspace) return fail(SPCONV_E_INVALID, "workspace is NULL");
    if (a.N > 0 && (!a.x || !a.y || (grad && !a.dout)))
        return fail(SPCONV_E_INVALID, "feature rows must be non-NULL");
    const size_t es = elem_size(a.dtype);
    if (!aligned(a.x, es) || !aligned(a.y, es) || !aligned(a.dout, es))
        return fail(SPCONV_E_INVALID, "feature rows must be aligned to their elements");
    if (!aligned(a.offsets, 4) || !aligned(a.weight, 4) || !aligned(a.bias, 4) || !aligned(a.mean, 4) ||
        !aligned(a.rstd, 4) || !aligned(a.dweight, 4) || !aligned(a.dbias, 4))
        return fail(SPCONV_E_INVALID, "offsets, weights and statistics must be 4-byte aligned");
    if (!aligned(a.workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
        return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    hipError_t e = spc::launch_group(a, grad, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, name);
}

int spconv_groupnorm(const void* x, const int32_t* offsets, const float* weight, const float* bias, void* workspace,
                     size_t workspace_bytes, void* y, float* mean, float* rstd, int64_t N, int C, int scenes,
                     int groups, float eps, int act, int dtype, void* stream) {
    return group_impl({x, nullptr, offsets, weight, bias, workspace, y, mean, rstd, nullptr, nullptr, N, C, scenes,
                       groups, eps, act, dtype},
                      false, workspace_bytes, stream, "spconv_groupnorm");
}

int spconv_groupnorm_grad(const void* dout, const void* x, const int32_t* offsets, const float* mean,
                          const float* rstd, const float* weight, const float* bias, void* workspace,
                          size_t workspace_bytes, void* dx, float* dweight, float* dbias, int64_t N, int C,
                          int scenes, int groups, int act, int dtype, void* stream) {
    return group_impl({x, dout, offsets, weight, bias, workspace, dx, const_cast<float*>(mean),
                       const_cast<float*>(rstd), dweight, dbias, N, C, scenes, groups, 0.f, act, dtype},
                      true, workspace_bytes, stream, "spconv_groupnorm_grad");
}

// Sizes of an attention: rows, sequences, heads.
static int check_attention(const spc::AttnArgs& a, bool grad) {
    int rc = check_rows(a.N, a.H, a.dtype, "H");
    if (!rc) rc = check_rows(a.M, a.HK, a.dtype, "HK");
    if (rc) return rc;
    if (a.B < 1) return fail(SPCONV_E_INVALID, "B must be >= 1 (got %d)", a.B);
    if (a.H % a.HK) return fail(SPCONV_E_INVALID, "H must be a multiple of HK (got %d and %d)", a.H, a.HK);
    if (a.D < 1) return fail(SPCONV_E_INVALID, "D must be >= 1 (got %d)", a.D);
    if (a.D % 8 || a.D > spc::kMaxHeadDim)
        return fail(SPCONV_E_UNSUPPORTED, "no kernel for D=%d (multiples of 8 up to %d)", a.D, spc::kMaxHeadDim);
    if (a.N * (a.H / a.HK) > spc::kMaxAttnRows || a.M > spc::kMaxAttnRows)
        return fail(SPCONV_E_UNSUPPORTED, "no more than %lld rows N H / HK and keys M (got N=%lld M=%lld H=%d HK=%d)",
                    (long long)spc::kMaxAttnRows, (long long)a.N, (long long)a.M, a.H, a.HK);
    if (!(grad ? spc::attn_grad_fits(a) : spc::attn_fits(a)))
        return fail(SPCONV_E_UNSUPPORTED, "N=%lld M=%lld B=%d H=%d HK=%d need more than 2^32 threads",
                    (long long)a.N, (long long)a.M, a.B, a.H, a.HK);
    return SPCONV_OK;
}
static spc::AttnArgs attention_sizes(int64_t N, int64_t M, int B, int H, int HK, int D, int dtype) {
    spc::AttnArgs a{};
    a.N = N;
    a.M = M;
    a.B = B;
    a.H = H;
    a.HK = HK;
    a.D = D;
    a.dtype = dtype;
    return a;
}

int spconv_attention_workspace_size(int64_t N, int64_t M, int B, int H, int HK, int D, int dtype, size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    const spc::AttnArgs a = attention_sizes(N, M, B, H, HK, D, dtype);
    int rc = check_attention(a, false);
    if (rc) return rc;
    *bytes = spc::attn_workspace_bytes(a);
    return SPCONV_OK;
}

int spconv_attention_grad_workspace_size(int64_t N, int64_t M, int B, int H, int HK, int D, int dtype,
                                         size_t* bytes) {
    if (!bytes) return fail(SPCONV_E_INVALID, "bytes pointer is NULL");
    const spc::AttnArgs a = attention_sizes(N, M, B, H, HK, D, dtype);
    int rc = check_attention(a, true);
    if (rc) return rc;
    *bytes = spc::attn_grad_workspace_bytes(a);
    return SPCONV_OK;
}

// Checks of both directions, after the sizes; fills in the strides.
static int attention_impl(spc::AttnArgs& a, bool grad, const int64_t* strides, size_t workspace_bytes, void* stream,
                          const char* name) {
    int rc = check_attention(a, grad);
    if (rc) return rc;
    if (!(a.scale > 0.f) || !std::isfinite(a.scale))
        return fail(SPCONV_E_INVALID, "scale must be > 0 and finite (got %g)", (double)a.scale);
    if (!a.offsets) return fail(SPCONV_E_INVALID, "offsets is NULL");
    if (!a.koffsets && (a.M != a.N || a.korder))
        return fail(SPCONV_E_INVALID, "without koffsets the keys are the queries' rows: M = N, no korder");
    if (!aligned(a.offsets, 4) || !aligned(a.koffsets, 4) || !aligned(a.order, 4) || !aligned(a.korder, 4) ||
        !aligned(a.lse, 4))
        return fail(SPCONV_E_INVALID, "offsets, orders and lse must be 4-byte aligned");
    if (a.N > 0 && (!a.q || !a.out || (grad && (!a.dout || !a.lse || !a.dq))))
        return fail(SPCONV_E_INVALID, "%s must be non-NULL", grad ? "q, out, lse, dout and dq" : "q and out");
    if (a.M > 0 && (!a.k || !a.v || (grad && (!a.dk || !a.dv))))
        return fail(SPCONV_E_INVALID, "%s must be non-NULL", grad ? "k, v, dk and dv" : "k and v");
    struct {
        const void* t;
        int64_t* s;
        int heads;
    } const tensors[] = {{a.q, a.qs, a.H},     {a.k, a.ks, a.HK},   {a.v, a.vs, a.HK},   {a.out, a.os, a.H},
                         {a.dout, a.dos, a.H}, {a.dq, a.dqs, a.H}, {a.dk, a.dks, a.HK}, {a.dv, a.dvs, a.HK}};
    const int unit = a.dtype == SPCONV_BF16 ? 8 : 4;
    for (int i = 0; i < (grad ? 8 : 4); ++i) {
        tensors[i].s[0] = strides ? strides[2 * i] : (int64_t)tensors[i].heads * a.D;
        tensors[i].s[1] = strides ? strides[2 * i + 1] : a.D;
        if (!aligned(tensors[i].t, 16) || tensors[i].s[0] % unit || tensors[i].s[1] % unit)
            return fail(SPCONV_E_INVALID, "rows and heads must start at 16-byte addresses");
        if (tensors[i].s[0] < 0 || tensors[i].s[1] < 0) return fail(SPCONV_E_INVALID, "strides must be >= 0");
        if (tensors[i].s[0] * (16 / unit) > spc::kMaxRowStride)
            return fail(SPCONV_E_UNSUPPORTED, "rows must be at most %lld bytes apart", (long long)spc::kMaxRowStride);
        const int64_t rows = tensors[i].s == a.dks || tensors[i].s == a.dvs ? a.M : a.N;
        if ((grad ? i > 4 : i == 3) && heads_overlap(tensors[i].s, rows, tensors[i].heads, a.D))
            return fail(SPCONV_E_INVALID, "rows or heads of an output overlap");
    }
    const size_t need = grad ? spc::attn_grad_workspace_bytes(a) : spc::attn_workspace_bytes(a);
    if (need) {
        if (!a.workspace) return fail(SPCONV_E_INVALID, "workspace is NULL");
        if (!aligned(a.workspace, 256)) return fail(SPCONV_E_INVALID, "workspace must be 256-byte aligned");
        if (workspace_bytes < need)
            return fail(SPCONV_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
    hipError_t e = grad ? spc::launch_attn_grad(a, (hipStream_t)stream) : spc::launch_attn(a, (hipStream_t)stream);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, name);
}

int spconv_attention(const void* q, const void* k, const void* v, const int32_t* offsets, const int32_t* koffsets,
                     const int32_t* order, const int32_t* korder, const int64_t* strides, void* workspace,
                     size_t workspace_bytes, void* out, float* lse, int64_t N, int64_t M, int B, int H, int HK, int D,
                     float scale, int causal, int dtype, void* stream) {
    spc::AttnArgs a = attention_sizes(N, M, B, H, HK, D, dtype);
    a.q = q;
    a.k = k;
    a.v = v;
    a.offsets = offsets;
    a.koffsets = koffsets;
    a.order = order;
    a.korder = korder;
    a.workspace = workspace;
    a.out = out;
    a.lse = lse;
    a.scale = scale;
    a.causal = causal != 0;
    return attention_impl(a, false, strides, workspace_bytes, stream, "spconv_attention");
}

int spconv_attention_grad(const void* dout, const void* q, const void* k, const void* v, const void* out,
                          const float* lse, const int32_t* offsets, const int32_t* koffsets, const int32_t* order,
                          const int32_t* korder, const int64_t* strides, void* workspace, size_t workspace_bytes,
                          void* dq, void* dk, void* dv, int64_t N, int64_t M, int B, int H, int HK, int D, float scale,
                          int causal, int dtype, void* stream) {
    spc::AttnArgs a = attention_sizes(N, M, B, H, HK, D, dtype);
    a.q = q;
    a.k = k;
    a.v = v;
    a.offsets = offsets;
    a.koffsets = koffsets;
    a.order = order;
    a.korder = korder;
    a.dout = dout;
    a.workspace = workspace;
    a.out = const_cast<void*>(out);
    a.lse = const_cast<float*>(lse);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.causal = causal != 0;
    return attention_impl(a, true, strides, workspace_bytes, stream, "spconv_attention_grad");
}

void spconv_nmap_destroy(spconv_nmap* h) {
    if (valid_handle(h)) {
        h->magic = 0;
        delete h;
    }
}

}  // extern "C"
