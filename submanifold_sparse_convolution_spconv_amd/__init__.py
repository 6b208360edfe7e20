"""Submanifold sparse 3D convolution on AMD Instinct MI355X (gfx950).

Thin ctypes binding over ``libspconv_mi355x.so`` (declared in
``include/spconv_mi355x.h``).  Every step of the computation runs in the HIP
library; this module only checks tensor metadata, allocates the caller-owned
device buffers with PyTorch and passes pointers and the current HIP stream.
There is no fallback: if the library cannot be loaded, calls raise.

Operation (page "mlx_backend/sparse_conv_metal.py"):
    out[n, co] = bias[co] + sum_k sum_ci feats[nbr[k, n], ci] * w[k, ci, co]
with nbr a (K, N) int32 map whose value N marks a missing neighbour.

Functions carry the C entry points' names:
    spconv_nmap_sizes(N, K) -> (arena_bytes, workspace_bytes)
    spconv_build_nmap(coords, K=27, dilation=1) -> NMap
    spconv_nmap_wrap(nbr) -> NMap
    spconv_nmap_export(nmap) -> (nbr (K,N) int32, order (N,) int32)
    spconv_nmap_info(nmap) -> dict(N, K, dilation, valid_pairs)
    spconv_forward(feats, nmap, w, bias=None, out=None) -> out
    spconv_pack_weights_size(K, Ci, Co, dtype) -> bytes
    spconv_pack_weights(w) -> wpack (uint8 tensor; empty when there is no packed form)
    spconv_forward_packed(feats, nmap, w, wpack, bias=None, out=None) -> out
    spconv_forward_mixed(feats, nmap, w, bias=None, out=None) -> out  (feats cast to w's dtype)
    spconv_build_nmap_batched(coords (N,4) b,x,y,z, batches, K=27, dilation=1) -> NMap
    spconv_dgrad(dout, nmap, w) -> dfeats
    spconv_dgrad_noalloc(dout, nmap, w, out) -> out  (no workspace: a fixed scratch in the library)
    spconv_wgrad(feats, dout, nmap) -> dw
Row-wise operators of a voxel block, on (N, C) feature rows:
    spconv_layernorm(x, weight=None, bias=None, eps=1e-5, stats=False) -> y, or (y, mean, rstd)
    spconv_layernorm_grad(dout, x, mean, rstd, weight=None, sums=None) -> (dx, dweight, dbias)
    spconv_glu(x, w, bias=None, act="silu") -> h
    spconv_glu_grad(dout, x, w, bias=None, act="silu") -> (dx, dw, dbias)
    spconv_scan(x, z, offsets, order=None, h0=None) -> (h, last)
    spconv_scan_grad(dout, x, z, offsets, order=None, h0=None, dlast=None) -> (dx, dz, dh0)
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "SpconvError", "NMap", "load_library", "library_path",
    "spconv_nmap_sizes", "spconv_build_nmap", "spconv_nmap_wrap", "spconv_nmap_export",
    "spconv_nmap_info", "spconv_forward", "spconv_nmap_destroy",
    "spconv_pack_weights_size", "spconv_pack_weights", "spconv_forward_packed", "spconv_forward_mixed",
    "spconv_forward_mixed_workspace_size",
    "spconv_build_nmap_batched", "spconv_dgrad_workspace_size", "spconv_dgrad", "spconv_dgrad_noalloc",
    "SPCONV_NOALLOC_SCRATCH_BYTES",
    "spconv_wgrad_workspace_size", "spconv_wgrad",
    "spconv_layernorm", "spconv_layernorm_grad_workspace_size", "spconv_layernorm_grad",
    "spconv_glu", "spconv_glu_grad_workspace_size", "spconv_glu_grad", "SPCONV_SILU", "SPCONV_GELU",
    "spconv_scan_workspace_size", "spconv_scan", "spconv_scan_grad_workspace_size", "spconv_scan_grad",
    "SPCONV_F32", "SPCONV_BF16", "STATUS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# SPCONV_LIB may name another build of the library (the host-sanitized one)
_LIB_PATH = os.environ.get("SPCONV_LIB") or os.path.join(_PKG, "libspconv_mi355x.so")

SPCONV_F32 = 0
SPCONV_BF16 = 1
SPCONV_SILU = 0
SPCONV_GELU = 1
STATUS = {0: "SPCONV_OK", -1: "SPCONV_E_INVALID", -2: "SPCONV_E_UNSUPPORTED",
          -3: "SPCONV_E_COORD_RANGE", -4: "SPCONV_E_DUPLICATE", -5: "SPCONV_E_WORKSPACE",
          -6: "SPCONV_E_HIP"}

_lib = None


class SpconvError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}: {detail}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the HIP library, building it first only if no build exists."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        from . import build as _build
        _build.build()
    lib = ctypes.CDLL(_LIB_PATH)
    vp, sz, i64, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
    lib.spconv_abi_version.argtypes = []
    lib.spconv_abi_version.restype = i32
    lib.spconv_nmap_sizes.argtypes = [i64, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.spconv_build_nmap.argtypes = [vp, i64, i32, i32, vp, sz, vp, sz, vp, ctypes.POINTER(vp)]
    lib.spconv_build_nmap_batched.argtypes = [vp, i64, i32, i32, i32, vp, sz, vp, sz, vp, ctypes.POINTER(vp)]
    lib.spconv_nmap_wrap.argtypes = [vp, i64, i32, vp, sz, vp, ctypes.POINTER(vp)]
    lib.spconv_nmap_export.argtypes = [vp, vp, vp, vp]
    lib.spconv_nmap_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i32),
                                     ctypes.POINTER(i32), ctypes.POINTER(i64), vp]
    lib.spconv_forward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp]
    lib.spconv_forward_mixed.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
    lib.spconv_forward_mixed_workspace_size.argtypes = [i64, i32, i32, i32, ctypes.POINTER(sz)]
    lib.spconv_forward_mixed_workspace_size.restype = i32
    for f in (lib.spconv_nmap_sizes, lib.spconv_build_nmap, lib.spconv_build_nmap_batched, lib.spconv_nmap_wrap,
              lib.spconv_nmap_export, lib.spconv_nmap_info, lib.spconv_forward, lib.spconv_forward_mixed):
        f.restype = i32
    lib.spconv_pack_weights_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.spconv_pack_weights_size.restype = i32
    lib.spconv_pack_weights.argtypes = [vp, i32, i32, i32, i32, vp, sz, vp]
    lib.spconv_pack_weights.restype = i32
    lib.spconv_forward_packed.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]
    lib.spconv_forward_packed.restype = i32
    lib.spconv_dgrad_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.spconv_dgrad_workspace_size.restype = i32
    lib.spconv_dgrad.argtypes = [vp, vp, vp, vp, sz, vp, i32, i32, i32, vp]
    lib.spconv_dgrad.restype = i32
    lib.spconv_dgrad_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
    lib.spconv_dgrad_noalloc.restype = i32
    lib.spconv_wgrad_workspace_size.argtypes = [i64, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.spconv_wgrad_workspace_size.restype = i32
    lib.spconv_wgrad.argtypes = [vp, vp, vp, vp, sz, vp, i32, i32, i32, vp]
    lib.spconv_wgrad.restype = i32
    f32, szp = ctypes.c_float, ctypes.POINTER(sz)
    lib.spconv_layernorm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, f32, i32, vp]
    lib.spconv_layernorm_grad_workspace_size.argtypes = [i64, i32, i32, szp]
    lib.spconv_layernorm_grad.argtypes = [vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, i64, i32, i32, vp]
    lib.spconv_glu.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i32, vp]
    lib.spconv_glu_grad_workspace_size.argtypes = [i64, i32, i32, i32, szp]
    lib.spconv_glu_grad.argtypes = [vp, vp, vp, vp, vp, sz, vp, vp, vp, i64, i32, i32, i32, i32, vp]
    lib.spconv_scan_workspace_size.argtypes = [i64, i32, i32, szp]
    lib.spconv_scan.argtypes = [vp, vp, vp, vp, vp, vp, sz, vp, vp, i64, i32, i32, i32, vp]
    lib.spconv_scan_grad_workspace_size.argtypes = [i64, i32, i32, szp]
    lib.spconv_scan_grad.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, i64, i32, i32, i32, vp]
    for f in (lib.spconv_glu, lib.spconv_glu_grad_workspace_size, lib.spconv_glu_grad,
              lib.spconv_scan_workspace_size, lib.spconv_scan, lib.spconv_scan_grad_workspace_size,
              lib.spconv_scan_grad, lib.spconv_layernorm, lib.spconv_layernorm_grad_workspace_size, lib.spconv_layernorm_grad):
        f.restype = i32
    lib.spconv_nmap_destroy.argtypes = [vp]
    lib.spconv_nmap_destroy.restype = None
    lib.spconv_status_string.argtypes = [i32]
    lib.spconv_status_string.restype = ctypes.c_char_p
    lib.spconv_last_error.argtypes = []
    lib.spconv_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int, where: str):
    if rc != 0:
        raise SpconvError(rc, where, load_library().spconv_last_error().decode())


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def spconv_nmap_sizes(N: int, K: int):
    a, w = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().spconv_nmap_sizes(N, K, ctypes.byref(a), ctypes.byref(w)),
           "spconv_nmap_sizes")
    return a.value, w.value


class NMap:
    """A built (or wrapped) neighbour map: the C handle plus the arena tensor
    that holds its device data."""

    def __init__(self, handle, arena, N, K, dilation, device):
        self._h = handle
        self.arena = arena
        self.N, self.K, self.dilation, self.device = N, K, dilation, device

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("neighbour map already destroyed")
        return self._h

    def destroy(self):
        if self._h is not None and _lib is not None:
            _lib.spconv_nmap_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def valid_pairs(self) -> int:
        return spconv_nmap_info(self)["valid_pairs"]

    def export(self):
        return spconv_nmap_export(self)


def spconv_build_nmap(coords, K: int = 27, dilation: int = 1, workspace=None) -> NMap:
    """coords: int32 CUDA tensor (N, 3).  Returns an NMap (arena owned by it)."""
    import torch
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 3 or not coords.is_cuda:
        raise ValueError("coords must be an int32 CUDA tensor of shape (N, 3)")
    coords = coords.contiguous()
    N = coords.shape[0]
    lib = load_library()
    arena_b, ws_b = spconv_nmap_sizes(N, K)
    dev = coords.device
    arena = torch.empty(arena_b, dtype=torch.uint8, device=dev)
    ws = workspace
    if ws is None or ws.numel() < ws_b:
        ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    h = ctypes.c_void_p()
    with torch.cuda.device(dev):
        rc = lib.spconv_build_nmap(_ptr(coords), N, K, dilation, _ptr(arena), arena_b,
                                   _ptr(ws), ws.numel(), _stream(dev), ctypes.byref(h))
    _check(rc, "spconv_build_nmap")
    return NMap(h, arena, N, K, dilation, dev)


def spconv_build_nmap_batched(coords, batches: int, K: int = 27, dilation: int = 1, workspace=None) -> NMap:
    """coords: int32 CUDA tensor (N, 4) of (b, x, y, z), b in [0, batches);
    voxels are neighbours only within one batch.  Returns an NMap."""
    import torch
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 4 or not coords.is_cuda:
        raise ValueError("coords must be an int32 CUDA tensor of shape (N, 4)")
    coords = coords.contiguous()
    N = coords.shape[0]
    lib = load_library()
    arena_b, ws_b = spconv_nmap_sizes(N, K)
    dev = coords.device
    arena = torch.empty(arena_b, dtype=torch.uint8, device=dev)
    ws = workspace
    if ws is None or ws.numel() < ws_b:
        ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    h = ctypes.c_void_p()
    with torch.cuda.device(dev):
        rc = lib.spconv_build_nmap_batched(_ptr(coords), N, batches, K, dilation, _ptr(arena), arena_b,
                                           _ptr(ws), ws.numel(), _stream(dev), ctypes.byref(h))
    _check(rc, "spconv_build_nmap_batched")
    return NMap(h, arena, N, K, dilation, dev)


def spconv_nmap_wrap(nbr) -> NMap:
    """nbr: int32 CUDA tensor (K, N), element [k, n], sentinel N."""
    import torch
    if nbr.dtype != torch.int32 or nbr.dim() != 2 or not nbr.is_cuda:
        raise ValueError("nbr must be an int32 CUDA tensor of shape (K, N)")
    nbr = nbr.contiguous()
    K, N = nbr.shape
    lib = load_library()
    arena_b, _ = spconv_nmap_sizes(N, K)
    dev = nbr.device
    arena = torch.empty(arena_b, dtype=torch.uint8, device=dev)
    h = ctypes.c_void_p()
    with torch.cuda.device(dev):
        rc = lib.spconv_nmap_wrap(_ptr(nbr), N, K, _ptr(arena), arena_b, _stream(dev), ctypes.byref(h))
    _check(rc, "spconv_nmap_wrap")
    return NMap(h, arena, N, K, 1, dev)


def spconv_nmap_export(nmap: NMap):
    """(nbr (K, N) int32, order (N,) int32) on the map's device, caller order."""
    import torch
    nbr = torch.empty((nmap.K, nmap.N), dtype=torch.int32, device=nmap.device)
    order = torch.empty((nmap.N,), dtype=torch.int32, device=nmap.device)
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_nmap_export(nmap.handle, _ptr(nbr), _ptr(order), _stream(nmap.device))
    _check(rc, "spconv_nmap_export")
    return nbr, order


def spconv_nmap_info(nmap: NMap) -> dict:
    import torch
    N, vp = ctypes.c_int64(), ctypes.c_int64()
    K, d = ctypes.c_int(), ctypes.c_int()
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_nmap_info(nmap.handle, ctypes.byref(N), ctypes.byref(K),
                                             ctypes.byref(d), ctypes.byref(vp), _stream(nmap.device))
    _check(rc, "spconv_nmap_info")
    return {"N": N.value, "K": K.value, "dilation": d.value, "valid_pairs": vp.value}


def spconv_nmap_destroy(nmap: NMap):
    nmap.destroy()


def _forward_args(feats, nmap: NMap, w, bias, out, mixed=False):
    import torch
    dt = {torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16}.get(w.dtype)
    if dt is None or feats.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("feats and w must be float32 or bfloat16")
    if not mixed and feats.dtype != w.dtype:
        raise ValueError("feats and w must both be float32 or both bfloat16")
    if w.dim() != 3 or w.shape[0] != nmap.K or feats.dim() != 2 or feats.shape[1] != w.shape[1]:
        raise ValueError("expected feats (N, Ci) and w (K, Ci, Co) matching the map")
    if feats.shape[0] not in (nmap.N, nmap.N + 1):
        raise ValueError("feats must have N or N+1 rows")
    for t in (feats, w):
        if not t.is_cuda or t.device != nmap.device:
            raise ValueError("tensors must live on the map's device")
    Co = w.shape[2]
    feats = feats.contiguous()
    w = w.contiguous()
    if bias is not None:
        if bias.dtype != torch.float32 or bias.shape != (Co,) or bias.device != nmap.device:
            raise ValueError("bias must be float32 (Co,) on the map's device")
        bias = bias.contiguous()
    if out is None:
        out = torch.empty((nmap.N, Co), dtype=w.dtype, device=nmap.device)
    elif out.shape != (nmap.N, Co) or out.dtype != w.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous (N, Co) tensor of w's dtype")
    return feats, w, bias, out, dt


def spconv_forward(feats, nmap: NMap, w, bias=None, out=None):
    """feats (N or N+1, Ci), w (K, Ci, Co): both float32 or both bfloat16, CUDA.
    bias: float32 (Co,) or None.  Returns out (N, Co) in w's dtype."""
    import torch
    feats, w, bias, out, dt = _forward_args(feats, nmap, w, bias, out)
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_forward(_ptr(feats), nmap.handle, _ptr(w), _ptr(bias), _ptr(out),
                                           w.shape[1], w.shape[2], dt, _stream(nmap.device))
    _check(rc, "spconv_forward")
    return out


def spconv_forward_mixed_workspace_size(N: int, Ci: int, feats_dtype: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().spconv_forward_mixed_workspace_size(N, Ci, feats_dtype, dtype, ctypes.byref(n)),
           "spconv_forward_mixed_workspace_size")
    return n.value


def spconv_forward_mixed(feats, nmap: NMap, w, bias=None, out=None, workspace=None, wpack=None):
    """spconv_forward with feats float32 or bfloat16 independently of w: feats
    are converted to w's dtype (fp32 -> bf16 rounds to nearest even).  With a
    uint8 device ``workspace`` of spconv_forward_mixed_workspace_size bytes,
    fp32 feats are cast by a separate pass first; without one, in the gather.
    ``wpack`` (spconv_pack_weights(w)) is optional.  Returns out (N, Co) in
    w's dtype."""
    import torch
    feats, w, bias, out, dt = _forward_args(feats, nmap, w, bias, out, mixed=True)
    fdt = SPCONV_F32 if feats.dtype == torch.float32 else SPCONV_BF16
    if wpack is not None:
        if wpack.dtype != torch.uint8 or wpack.device != nmap.device:
            raise ValueError("wpack must be the uint8 tensor from spconv_pack_weights on the map's device")
        if wpack.numel() < spconv_pack_weights_size(nmap.K, w.shape[1], w.shape[2], dt):
            raise ValueError("wpack is smaller than spconv_pack_weights_size")
    ws, wsb = None, 0
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != nmap.device:
            raise ValueError("workspace must be a contiguous uint8 tensor on the map's device")
        ws, wsb = workspace, workspace.numel()
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_forward_mixed(_ptr(feats), fdt, nmap.handle, _ptr(w),
                                                 _ptr(wpack) if wpack is not None and wpack.numel() else None,
                                                 _ptr(bias), _ptr(out), w.shape[1], w.shape[2], dt, _ptr(ws), wsb,
                                                 _stream(nmap.device))
    _check(rc, "spconv_forward_mixed")
    return out


def spconv_pack_weights_size(K: int, Ci: int, Co: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().spconv_pack_weights_size(K, Ci, Co, dtype, ctypes.byref(n)),
           "spconv_pack_weights_size")
    return n.value


def spconv_pack_weights(w, out=None):
    """Packed copy of w (K, Ci, Co) for spconv_forward_packed: a uint8 device
    tensor, empty when the forward has no packed form for this configuration."""
    import torch
    dt = {torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16}.get(w.dtype)
    if dt is None or w.dim() != 3 or not w.is_cuda:
        raise ValueError("w must be a float32 or bfloat16 (K, Ci, Co) CUDA tensor")
    w = w.contiguous()
    K, Ci, Co = w.shape
    n = spconv_pack_weights_size(K, Ci, Co, dt)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w.device)
    elif out.dtype != torch.uint8 or out.numel() < n or out.device != w.device:
        raise ValueError("out must be a uint8 tensor of at least spconv_pack_weights_size bytes")
    with torch.cuda.device(w.device):
        rc = load_library().spconv_pack_weights(_ptr(w), K, Ci, Co, dt, _ptr(out) if n else None, n,
                                                _stream(w.device))
    _check(rc, "spconv_pack_weights")
    return out


def spconv_forward_packed(feats, nmap: NMap, w, wpack, bias=None, out=None):
    """spconv_forward with wpack = spconv_pack_weights(w)."""
    import torch
    feats, w, bias, out, dt = _forward_args(feats, nmap, w, bias, out)
    if wpack.dtype != torch.uint8 or wpack.device != nmap.device:
        raise ValueError("wpack must be the uint8 tensor from spconv_pack_weights on the map's device")
    if wpack.numel() < spconv_pack_weights_size(nmap.K, w.shape[1], w.shape[2], dt):
        raise ValueError("wpack is smaller than spconv_pack_weights_size")
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_forward_packed(_ptr(feats), nmap.handle, _ptr(w),
                                                  _ptr(wpack) if wpack.numel() else None, _ptr(bias),
                                                  _ptr(out), w.shape[1], w.shape[2], dt, _stream(nmap.device))
    _check(rc, "spconv_forward_packed")
    return out


def spconv_dgrad_workspace_size(K: int, Ci: int, Co: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().spconv_dgrad_workspace_size(K, Ci, Co, dtype, ctypes.byref(n)),
           "spconv_dgrad_workspace_size")
    return n.value


def spconv_dgrad(dout, nmap: NMap, w, out=None, workspace=None):
    """Input gradient of spconv_forward: dout (N, Co) and w (K, Ci, Co), both
    float32 or both bfloat16, CUDA; returns dfeats (N, Ci) in w's dtype.  The
    map must come from spconv_build_nmap.  workspace: a uint8 tensor of at least
    spconv_dgrad_workspace_size bytes (allocated when None)."""
    import torch
    dt = {torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16}.get(w.dtype)
    if dt is None or dout.dtype != w.dtype:
        raise ValueError("dout and w must both be float32 or both bfloat16")
    if w.dim() != 3 or w.shape[0] != nmap.K or dout.dim() != 2 or dout.shape != (nmap.N, w.shape[2]):
        raise ValueError("expected dout (N, Co) and w (K, Ci, Co) matching the map")
    for t in (dout, w):
        if not t.is_cuda or t.device != nmap.device:
            raise ValueError("tensors must live on the map's device")
    K, Ci, Co = w.shape
    dout = dout.contiguous()
    w = w.contiguous()
    n = spconv_dgrad_workspace_size(K, Ci, Co, dt)
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=nmap.device)
    elif workspace.dtype != torch.uint8 or workspace.numel() < n or workspace.device != nmap.device:
        raise ValueError("workspace must be a uint8 tensor of at least spconv_dgrad_workspace_size bytes")
    if out is None:
        out = torch.empty((nmap.N, Ci), dtype=w.dtype, device=nmap.device)
    elif out.shape != (nmap.N, Ci) or out.dtype != w.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous (N, Ci) tensor of w's dtype")
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_dgrad(_ptr(dout), nmap.handle, _ptr(w), _ptr(workspace), workspace.numel(),
                                         _ptr(out), Ci, Co, dt, _stream(nmap.device))
    _check(rc, "spconv_dgrad")
    return out


SPCONV_NOALLOC_SCRATCH_BYTES = 16 << 20


def spconv_dgrad_noalloc(dout, nmap: NMap, w, out):
    """spconv_dgrad without a workspace: the library's fixed per-device scratch
    (SPCONV_NOALLOC_SCRATCH_BYTES) holds the mirrored weights, so the C call
    allocates nothing.  ``out`` (N, Ci) in w's dtype is required, so this
    function allocates nothing either.  Calls that overlap in time on one
    device race on the scratch."""
    import torch
    dt = {torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16}.get(w.dtype)
    if dt is None or dout.dtype != w.dtype:
        raise ValueError("dout and w must both be float32 or both bfloat16")
    if w.dim() != 3 or w.shape[0] != nmap.K or dout.dim() != 2 or dout.shape != (nmap.N, w.shape[2]):
        raise ValueError("expected dout (N, Co) and w (K, Ci, Co) matching the map")
    if not (dout.is_contiguous() and w.is_contiguous()):
        raise ValueError("dout and w must be contiguous (no copies are made)")
    K, Ci, Co = w.shape
    if out is None or out.shape != (nmap.N, Ci) or out.dtype != w.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous (N, Ci) tensor of w's dtype")
    for t in (dout, w, out):
        if not t.is_cuda or t.device != nmap.device:
            raise ValueError("tensors must live on the map's device")
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_dgrad_noalloc(_ptr(dout), nmap.handle, _ptr(w), _ptr(out), Ci, Co, dt,
                                                 _stream(nmap.device))
    _check(rc, "spconv_dgrad_noalloc")
    return out


def spconv_wgrad_workspace_size(N: int, K: int, Ci: int, Co: int, dtype: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().spconv_wgrad_workspace_size(N, K, Ci, Co, dtype, ctypes.byref(n)),
           "spconv_wgrad_workspace_size")
    return n.value


def spconv_wgrad(feats, dout, nmap: NMap, out=None, workspace=None):
    """Weight gradient of spconv_forward: feats (N or N+1, Ci) and dout (N, Co),
    both float32 or both bfloat16, CUDA; returns dw (K, Ci, Co) in their dtype.
    workspace: a uint8 tensor of at least spconv_wgrad_workspace_size bytes
    (allocated when None)."""
    import torch
    dt = {torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16}.get(feats.dtype)
    if dt is None or dout.dtype != feats.dtype:
        raise ValueError("feats and dout must both be float32 or both bfloat16")
    if feats.dim() != 2 or dout.dim() != 2 or feats.shape[0] not in (nmap.N, nmap.N + 1) or dout.shape[0] != nmap.N:
        raise ValueError("expected feats (N or N+1, Ci) and dout (N, Co) matching the map")
    for t in (feats, dout):
        if not t.is_cuda or t.device != nmap.device:
            raise ValueError("tensors must live on the map's device")
    Ci, Co = feats.shape[1], dout.shape[1]
    feats = feats.contiguous()
    dout = dout.contiguous()
    n = spconv_wgrad_workspace_size(nmap.N, nmap.K, Ci, Co, dt)
    if workspace is None:
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=nmap.device)
    elif workspace.dtype != torch.uint8 or workspace.numel() < n or workspace.device != nmap.device:
        raise ValueError("workspace must be a uint8 tensor of at least spconv_wgrad_workspace_size bytes")
    if out is None:
        out = torch.empty((nmap.K, Ci, Co), dtype=feats.dtype, device=nmap.device)
    elif out.shape != (nmap.K, Ci, Co) or out.dtype != feats.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous (K, Ci, Co) tensor of feats' dtype")
    with torch.cuda.device(nmap.device):
        rc = load_library().spconv_wgrad(_ptr(feats), _ptr(dout), nmap.handle, _ptr(workspace), workspace.numel(),
                                         _ptr(out), Ci, Co, dt, _stream(nmap.device))
    _check(rc, "spconv_wgrad")
    return out


# The row operators' calls are short (a single voxel's takes a few microseconds
# on the GPU), so what stands around them here is kept short too: addresses as
# plain integers, torch looked up once, a device guard only where another device
# is current, outputs made like the inputs.
_torch = None
_row_codes = {}
_current_device = _raw_stream = None


def _load_torch():
    global _torch, _current_device, _raw_stream
    import torch
    _row_codes.update({torch.float32: SPCONV_F32, torch.bfloat16: SPCONV_BF16})
    # torch's own short cuts, where this torch has them
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
    _torch = torch


def _row_dtype(x, name="x"):
    """The dtype code of a feature tensor (N, C)."""
    if _torch is None:
        _load_torch()
    dt = _row_codes.get(x.dtype)
    if dt is None or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a float32 or bfloat16 (N, C) CUDA tensor")
    return dt


def _at(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """The C function on the current stream of dev."""
    fn = getattr(_lib or load_library(), name)
    index = dev.index
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with _torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(rc, name)


def _size(name, *args):
    n = ctypes.c_size_t(0)
    rc = getattr(_lib or load_library(), name)(*args, ctypes.byref(n))
    if rc:
        _check(rc, name)
    return n.value


def _like(t, shape, dtype, device, name):
    """t, contiguous, checked against what an input has to be; None stays."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on the features' device")
    return t.contiguous()


def _out(out, shape, like, name):
    """The output of this shape, of like's type and device: the caller's,
    checked, or a new one."""
    if out is None:
        return _torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    if out.shape != shape or out.dtype != like.dtype or out.device != like.device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} {tuple(shape)} tensor on the features' device")
    return out


def _workspace(workspace, n, device, size_name):
    """The workspace and its bytes: the caller's, checked, or one of n bytes
    (none for 0)."""
    if workspace is None:
        return (_torch.empty(n, dtype=_torch.uint8, device=device) if n else None), n
    if workspace.dtype != _torch.uint8 or workspace.numel() < n or workspace.device != device \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {size_name} bytes")
    return workspace, workspace.numel()


def spconv_layernorm(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = False, out=None):
    """Layer norm over each row's channels: x (N, C) float32 or bfloat16, CUDA,
    C <= 4096; weight, bias float32 (C,) or None.  Returns y in x's dtype, with
    ``stats`` (y, mean, rstd), float32 (N,) each, for the gradient."""
    dt = _row_dtype(x)
    N, C = x.shape
    dev = x.device
    x = x.contiguous()
    weight = _like(weight, (C,), _torch.float32, dev, "weight")
    bias = _like(bias, (C,), _torch.float32, dev, "bias")
    y = _out(out, x.shape, x, "out")
    mean = _torch.empty(N, dtype=_torch.float32, device=dev) if stats else None
    rstd = _torch.empty(N, dtype=_torch.float32, device=dev) if stats else None
    _call("spconv_layernorm", dev, _at(x), _at(weight), _at(bias), _at(y), _at(mean), _at(rstd), N, C, eps, dt)
    return (y, mean, rstd) if stats else y


def spconv_layernorm_grad_workspace_size(N: int, C: int, dtype: int) -> int:
    return _size("spconv_layernorm_grad_workspace_size", N, C, dtype)


def spconv_layernorm_grad(dout, x, mean, rstd, weight=None, out=None, workspace=None, sums=None):
    """Gradient of spconv_layernorm: dout and x (N, C), the statistics that the
    forward returned, its weight.  ``sums``: whether dweight and dbias are wanted
    (None: where weight is given; True also serves a norm with a bias and no
    weight).  Returns (dx, dweight, dbias), dweight and dbias float32 (C,), or
    None both.  workspace: a uint8 tensor of at least
    spconv_layernorm_grad_workspace_size bytes (allocated when None)."""
    dt = _row_dtype(x)
    N, C = x.shape
    dev = x.device
    x = x.contiguous()
    dout = _like(dout, (N, C), x.dtype, dev, "dout")
    mean = _like(mean, (N,), _torch.float32, dev, "mean")
    rstd = _like(rstd, (N,), _torch.float32, dev, "rstd")
    if dout is None or mean is None or rstd is None:
        raise ValueError("dout, mean and rstd must be given")
    weight = _like(weight, (C,), _torch.float32, dev, "weight")
    dx = _out(out, x.shape, x, "out")
    ws = dweight = dbias = None
    n = 0
    if weight is not None if sums is None else sums:
        ws, n = _workspace(workspace, spconv_layernorm_grad_workspace_size(N, C, dt), dev,
                           "spconv_layernorm_grad_workspace_size")
        dweight = _torch.empty(C, dtype=_torch.float32, device=dev)
        dbias = _torch.empty(C, dtype=_torch.float32, device=dev)
    _call("spconv_layernorm_grad", dev, _at(dout), _at(x), _at(mean), _at(rstd), _at(weight), _at(ws), n, _at(dx),
          _at(dweight), _at(dbias), N, C, dt)
    return dx, dweight, dbias


_ACTS = {"silu": SPCONV_SILU, "gelu": SPCONV_GELU}


def _glu_args(x, w, bias, act):
    dt = _row_dtype(x)
    N, C = x.shape
    dev = x.device
    if w is None or w.dtype != x.dtype or w.dim() != 3 or w.shape[0] != 2 or w.shape[1] != C or w.device != dev:
        raise ValueError("w must be (2, C, F) of x's dtype on its device")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    F = w.shape[2]
    bias = _like(bias, (2, F), _torch.float32, dev, "bias")
    return dt, N, C, F, dev, x.contiguous(), w.contiguous(), bias, _ACTS[act]


def spconv_glu(x, w, bias=None, act: str = "silu", out=None):
    """Gated linear unit h = act(x w[0] + bias[0]) * (x w[1] + bias[1]): x (N, C)
    and w (2, C, F), both float32 or both bfloat16, CUDA; bias float32 (2, F) or
    None; act "silu" or "gelu" (erf); C and F multiples of 8 up to 4096.  Like
    the convolution's operands, x, w and out start at 16-byte addresses; others
    (contiguous views into a buffer) raise SpconvError, SPCONV_E_INVALID.
    Returns h (N, F) in their dtype."""
    dt, N, C, F, dev, x, w, bias, a = _glu_args(x, w, bias, act)
    h = _out(out, (N, F), x, "out")
    _call("spconv_glu", dev, _at(x), _at(w), _at(bias), _at(h), N, C, F, a, dt)
    return h


def spconv_glu_grad_workspace_size(N: int, C: int, F: int, dtype: int) -> int:
    return _size("spconv_glu_grad_workspace_size", N, C, F, dtype)


def spconv_glu_grad(dout, x, w, bias=None, act: str = "silu", workspace=None):
    """Gradient of spconv_glu: dout (N, F), at a 16-byte address like x and w, the
    forward's inputs.  Returns (dx
    (N, C), dw (2, C, F), dbias float32 (2, F), or None where bias is None).
    workspace: a uint8 tensor of at least spconv_glu_grad_workspace_size bytes
    (allocated when None)."""
    dt, N, C, F, dev, x, w, bias, a = _glu_args(x, w, bias, act)
    dout = _like(dout, (N, F), x.dtype, dev, "dout")
    if dout is None:
        raise ValueError("dout must be given")
    dx = _torch.empty_like(x)
    dw = _torch.empty_like(w)
    dbias = _torch.empty_like(bias) if bias is not None else None
    ws, n = _workspace(workspace, spconv_glu_grad_workspace_size(N, C, F, dt), dev, "spconv_glu_grad_workspace_size")
    _call("spconv_glu_grad", dev, _at(dout), _at(x), _at(w), _at(bias), _at(ws), n, _at(dx), _at(dw), _at(dbias), N,
          C, F, a, dt)
    return dx, dw, dbias


def _scan_args(x, z, offsets, order, h0):
    dt = _row_dtype(x)
    N, C = x.shape
    dev = x.device
    if z is None or offsets is None:
        raise ValueError("z and offsets must be given")
    if offsets.dtype != _torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or offsets.device != dev:
        raise ValueError("offsets must be an int32 (scenes + 1,) tensor on the features' device")
    B = offsets.numel() - 1
    x = x.contiguous()
    z = _like(z, (N, C), x.dtype, dev, "z")
    order = _like(order, (N,), _torch.int32, dev, "order")
    h0 = _like(h0, (B, C), _torch.float32, dev, "h0")
    return dt, N, C, B, dev, x, z, offsets.contiguous(), order, h0


def spconv_scan_workspace_size(N: int, C: int, dtype: int) -> int:
    return _size("spconv_scan_workspace_size", N, C, dtype)


def spconv_scan(x, z, offsets, order=None, h0=None, out=None, workspace=None):
    """Gated linear recurrence h[t] = f h[t-1] + (1 - f) x[t], f = sigmoid(z[t]),
    along each scene: x, z (N, C) float32 or bfloat16, CUDA, C <= 4096; offsets
    int32 (scenes + 1,), the scenes' positions; order int32 (N,), the row of
    each position (None: rows in order); h0 float32 (scenes, C), the states to
    start from (None: zero).  Returns (h (N, C) in the caller's row order, last
    (scenes, C) float32: each scene's last state).  workspace: a uint8 tensor of
    at least spconv_scan_workspace_size bytes (allocated when None)."""
    dt, N, C, B, dev, x, z, offsets, order, h0 = _scan_args(x, z, offsets, order, h0)
    h = _out(out, x.shape, x, "out")
    last = _torch.empty((B, C), dtype=_torch.float32, device=dev)
    ws, n = _workspace(workspace, spconv_scan_workspace_size(N, C, dt), dev, "spconv_scan_workspace_size")
    _call("spconv_scan", dev, _at(x), _at(z), _at(offsets), _at(order), _at(h0), _at(ws), n, _at(h), _at(last), N, C,
          B, dt)
    return h, last


def spconv_scan_grad_workspace_size(N: int, C: int, dtype: int) -> int:
    return _size("spconv_scan_grad_workspace_size", N, C, dtype)


def spconv_scan_grad(dout, x, z, offsets, order=None, h0=None, dlast=None, workspace=None):
    """Gradient of spconv_scan: dout (N, C) at h, dlast float32 (scenes, C) at
    the last states (None: zero), the forward's inputs.  Returns (dx, dz, dh0),
    dh0 float32 (scenes, C), or None where h0 is None.  workspace: a uint8
    tensor of at least spconv_scan_grad_workspace_size bytes (allocated when
    None)."""
    dt, N, C, B, dev, x, z, offsets, order, h0 = _scan_args(x, z, offsets, order, h0)
    dout = _like(dout, (N, C), x.dtype, dev, "dout")
    if dout is None:
        raise ValueError("dout must be given")
    dlast = _like(dlast, (B, C), _torch.float32, dev, "dlast")
    dx = _torch.empty_like(x)
    dz = _torch.empty_like(x)
    dh0 = _torch.empty_like(h0) if h0 is not None else None
    ws, n = _workspace(workspace, spconv_scan_grad_workspace_size(N, C, dt), dev, "spconv_scan_grad_workspace_size")
    _call("spconv_scan_grad", dev, _at(dout), _at(x), _at(z), _at(offsets), _at(order), _at(h0), _at(dlast), _at(ws),
          n, _at(dx), _at(dz), _at(dh0), N, C, B, dt)
    return dx, dz, dh0
