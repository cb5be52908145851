"""ctypes binding of libdpclip.so: the C ABI of include/dpclip.h, one Python function per entry.

This module only marshals arguments.  It turns torch tensors into device pointers and shapes,
and the current torch stream into a ``cudaStream_t``.  Every step of the computation runs in
the CUDA library.  When the library is missing this module raises; it never falls back to
other code.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdpclip.so")
# The same library built with -DDPCLIP_DEBUG: device-side index checks (see dp_workspace_status).
DEBUG_LIB_PATH = os.path.join(PKG, "libdpclip_debug.so")

(DP_OK, DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_WORKSPACE, DP_ERR_CUDA, DP_ERR_TIMEOUT,
 DP_ERR_DEVICE_CHECK) = range(7)
DP_F32, DP_BF16 = 0, 1
DP_I32, DP_I64 = 0, 1
DP_NORM_AUTO, DP_NORM_GHOST, DP_NORM_EXPLICIT, DP_NORM_ONCE = 0, 1, 2, 3
METHODS = {"auto": DP_NORM_AUTO, "ghost": DP_NORM_GHOST, "explicit": DP_NORM_EXPLICIT,
           "once": DP_NORM_ONCE}
METHOD_NAMES = {v: k for k, v in METHODS.items()}

_c_void_p, _c_int, _c_float = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_c_size_t, _c_ll, _c_ull, _c_uint = ctypes.c_size_t, ctypes.c_longlong, ctypes.c_ulonglong, ctypes.c_uint

class DpLayer(ctypes.Structure):
    """Mirror of the C struct dp_layer (include/dpclip.h)."""
    _fields_ = [("X", ctypes.c_void_p), ("dY", ctypes.c_void_p), ("d_in", ctypes.c_int),
                ("d_out", ctypes.c_int), ("layer_id", ctypes.c_uint), ("C", ctypes.c_float),
                ("G_out", ctypes.c_void_p), ("norms_out", ctypes.c_void_p), ("P", ctypes.c_void_p),
                ("r", ctypes.c_int)]


DP_CLIP_PER_LAYER, DP_CLIP_FLAT = 0, 1
CLIP_MODES = {"per_layer": DP_CLIP_PER_LAYER, "flat": DP_CLIP_FLAT}

SIGNATURES = {
    "dp_workspace_size": (_c_size_t, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "dp_workspace_size_for": (_c_size_t, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "dp_per_sample_norms": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                     _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_clip_accumulate": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_void_p, _c_float, _c_void_p, _c_void_p,
                                    _c_size_t, _c_void_p]),
    "dp_add_noise": (_c_int, [_c_void_p, _c_ll, _c_ll, _c_float, _c_ull, _c_ull, _c_uint, _c_void_p]),
    "dp_projection_matrix": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_ull, _c_uint, _c_void_p]),
    "dp_linear_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                _c_int, _c_int, _c_float, _c_float, _c_ull, _c_ull, _c_uint, _c_int,
                                _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_linear_step_dev_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                         _c_int, _c_int, _c_float, _c_float, _c_ull, _c_void_p, _c_uint,
                                         _c_int, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_workspace_status": (_c_int, [_c_void_p, _c_void_p]),
    "dp_selftest_wait_timeout": (_c_int, [_c_void_p, _c_ull, _c_void_p]),
    "dp_selftest_fail_launches": (_c_int, [_c_ll, _c_ll, _c_int]),
    "dp_per_sample_norms_static": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                            _c_int, _c_void_p, _c_void_p]),
    "dp_philox_blocks": (_c_int, [_c_void_p, _c_ull, _c_ull, _c_ull, _c_uint, _c_uint, _c_void_p]),
    "dp_box_muller": (_c_int, [_c_void_p, _c_ll, _c_void_p, _c_void_p]),
    "dp_auto_norm_method": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "dp_status_string": (ctypes.c_char_p, [_c_int]),
    "dp_last_cuda_error": (ctypes.c_char_p, []),
    "dp_block_workspace_size": (_c_size_t, [ctypes.POINTER(DpLayer), _c_int, _c_int, _c_int, _c_int,
                                            _c_int, _c_int]),
    "dp_block_step": (_c_int, [ctypes.POINTER(DpLayer), _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                               _c_float, _c_ull, _c_ull, _c_int, _c_void_p, _c_void_p, _c_size_t,
                               _c_void_p]),
    "dp_block_step_dev_step": (_c_int, [ctypes.POINTER(DpLayer), _c_int, _c_int, _c_int, _c_int, _c_int,
                                        _c_float, _c_float, _c_ull, _c_void_p, _c_int, _c_void_p, _c_void_p,
                                        _c_size_t, _c_void_p]),
    "dp_adam_workspace_size": (_c_size_t, [_c_int, _c_int]),
    "dp_projected_adam_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int,
                                        _c_int, _c_int, _c_float, _c_float, _c_float, _c_float, _c_float,
                                        _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "dp_embedding_lookup": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_float, _c_ll, _c_int, _c_int,
                                     _c_void_p, _c_int, _c_void_p]),
    "dp_embedding_workspace_size": (_c_size_t, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "dp_embedding_per_sample_norms": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                               _c_int, _c_float, _c_ll, _c_void_p, _c_void_p, _c_size_t,
                                               _c_void_p]),
    "dp_embedding_clip_accumulate": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                              _c_int, _c_float, _c_ll, _c_void_p, _c_float, _c_void_p,
                                              _c_void_p, _c_size_t, _c_void_p]),
    "dp_embedding_step": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _c_float, _c_ll, _c_float, _c_float, _c_ull, _c_ull, _c_uint, _c_void_p,
                                   _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_embedding_step_dev_step": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                            _c_int, _c_float, _c_ll, _c_float, _c_float, _c_ull, _c_void_p,
                                            _c_uint, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_rmsnorm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_ll, _c_int, _c_float, _c_void_p,
                            _c_void_p, _c_void_p]),
    "dp_rmsnorm_workspace_size": (_c_size_t, [_c_int, _c_int, _c_int, _c_int]),
    "dp_rmsnorm_backward": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int,
                                     _c_int, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                     _c_void_p]),
    "dp_rmsnorm_clip_accumulate": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_float, _c_void_p,
                                            _c_void_p]),
    "dp_rmsnorm_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                 _c_float, _c_float, _c_float, _c_ull, _c_ull, _c_uint, _c_void_p, _c_void_p,
                                 _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_rmsnorm_step_dev_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int,
                                          _c_int, _c_float, _c_float, _c_float, _c_ull, _c_void_p, _c_uint,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "dp_muon_workspace_size": (_c_size_t, [_c_int, _c_int]),
    "dp_orthogonalize": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_size_t,
                                  _c_void_p]),
    "dp_muon_step": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_float, _c_float, _c_int, _c_float,
                              _c_float, _c_float, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "dp_profiling_enable": (_c_int, [_c_int]),
    "dp_profiling_kinds": (_c_int, []),
    "dp_profiling_kind_name": (ctypes.c_char_p, [_c_int]),
    "dp_profiling_collect": (_c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_c_ll)]),
    "dp_kernel_launches": (_c_ll, []),
}

_lib = None
_debug_lib = None


def load(path):
    """A ctypes handle of the library at ``path`` with every entry point's signature set."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m sample_gradient_clipping_b200.build` (nvcc, sm_100a)")
    handle = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def debug_lib():
    """The checked build of the library (libdpclip_debug.so), loaded beside the normal one."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = load(DEBUG_LIB_PATH)
    return _debug_lib


class using:
    """Context manager: the functions of this module call ``handle`` (e.g. debug_lib())
    instead of the normal library while it is active."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        global _lib
        lib()
        self.saved, _lib = _lib, self.handle
        return self.handle

    def __exit__(self, *exc):
        global _lib
        _lib = self.saved
        return False


class DPError(RuntimeError):
    def __init__(self, status, what):
        detail = lib().dp_last_cuda_error().decode() if status == DP_ERR_CUDA else ""
        msg = f"{what}: {lib().dp_status_string(status).decode()}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


def check(status, what):
    if status != DP_OK:
        raise DPError(status, what)


_DTYPE_CODES = {}   # torch dtype -> dp_dtype, filled on the first use (torch is imported lazily)


def _dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        import torch

        _DTYPE_CODES.update({torch.bfloat16: DP_BF16, torch.float32: DP_F32})
        code = _DTYPE_CODES.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _stream(stream):
    import torch

    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bt_dims(X, dY):
    if X.dim() != 3 or dY.dim() != 3 or X.shape[:2] != dY.shape[:2]:
        raise ValueError("X must be [B, T, d_in] and dY [B, T, d_out]")
    if not (X.is_contiguous() and dY.is_contiguous()):
        raise ValueError("X and dY must be contiguous")
    if X.dtype != dY.dtype:
        raise ValueError("X and dY must share a dtype")
    return int(X.shape[0]), int(X.shape[1]), int(X.shape[2]), int(dY.shape[2])


def _holds_fp32(t, name, count):
    """The library writes or reads ``count`` fp32 values at t's pointer."""
    import torch

    if t is not None and (t.dtype != torch.float32 or t.numel() < count or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {torch.float32} of {count} elements, got {t.dtype} {list(t.shape)}")


def _projection_width(P, X, d_out):
    """r of a projection P [d_out, r] in X's dtype, 0 without one."""
    if P is None:
        return 0
    if P.dim() != 2 or P.shape[0] != d_out or P.dtype != X.dtype or not P.is_contiguous():
        raise ValueError(f"P must be contiguous {X.dtype} of shape [{d_out}, r], got {P.dtype} {list(P.shape)}")
    return int(P.shape[1])


def workspace_size(B, T, d_in, d_out, r=0, dtype_code=DP_BF16, method="auto"):
    return int(lib().dp_workspace_size_for(B, T, d_in, d_out, r, dtype_code, METHODS[method]))


def _workspace(X, dY, r, workspace, method="auto"):
    import torch

    B, T, d_in, d_out = _bt_dims(X, dY)
    need = workspace_size(B, T, d_in, d_out, r, _dtype_code(X), method)
    if need == 0:
        raise DPError(DP_ERR_INVALID_ARG, "workspace size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    return workspace


def dp_per_sample_norms(X, dY, P=None, method="auto", norms=None, workspace=None, stream=None):
    """Per-sample norms n_i (fp32 [B]) of X_i^T dY_i [P]."""
    import torch

    B, T, d_in, d_out = _bt_dims(X, dY)
    r = _projection_width(P, X, d_out)
    _holds_fp32(norms, "norms", B)
    ws = _workspace(X, dY, r, workspace)
    if norms is None:
        norms = torch.empty(B, dtype=torch.float32, device=X.device)
    check(lib().dp_per_sample_norms(_ptr(X), _ptr(dY), _ptr(P), r, _dtype_code(X), B, T, d_in, d_out,
                                    METHODS[method], _ptr(norms), _ptr(ws), ws.numel(), _stream(stream)),
          "dp_per_sample_norms")
    return norms


def dp_clip_accumulate(X, dY, norms, C, G_sum, P=None, workspace=None, stream=None):
    """G_sum += sum_i c_i X_i^T dY_i [P] with c_i = min(1, C / norms[i])."""
    B, T, d_in, d_out = _bt_dims(X, dY)
    r = _projection_width(P, X, d_out)
    _holds_fp32(norms, "norms", B)
    _holds_fp32(G_sum, "G_sum", d_in * (r or d_out))
    ws = _workspace(X, dY, r, workspace)
    check(lib().dp_clip_accumulate(_ptr(X), _ptr(dY), _ptr(P), r, _dtype_code(X), B, T, d_in, d_out,
                                   _ptr(norms), float(C), _ptr(G_sum), _ptr(ws), ws.numel(),
                                   _stream(stream)),
          "dp_clip_accumulate")
    return G_sum


def dp_add_noise(G, std, seed, step, layer_id, stream=None):
    """G += std * z (Philox stream 0 at (seed, step, layer_id)), in place."""
    rows = int(G.shape[0])
    cols = int(G.numel() // max(rows, 1))
    check(lib().dp_add_noise(_ptr(G), rows, cols, float(std), int(seed), int(step), int(layer_id),
                             _stream(stream)),
          "dp_add_noise")
    return G


def dp_projection_matrix(P, seed, layer_id, stream=None):
    """Fills P[d_out, r] with z / sqrt(r) from Philox stream 1 at (seed, layer_id)."""
    check(lib().dp_projection_matrix(_ptr(P), _dtype_code(P), int(P.shape[0]), int(P.shape[1]),
                                     int(seed), int(layer_id), _stream(stream)),
          "dp_projection_matrix")
    return P


def _device_step(step):
    """A device tensor holding the step (int64/uint64, one element), or None for a number."""
    import torch

    if not isinstance(step, torch.Tensor):
        return None
    if step.numel() != 1 or step.dtype not in (torch.int64, torch.uint64) or not step.is_cuda:
        raise ValueError("a device step must be a one-element int64 CUDA tensor")
    return step


def dp_linear_step(X, dY, C, sigma, seed, step, layer_id, P=None, r=0, method="auto",
                   norms_out=None, G_out=None, workspace=None, stream=None):
    """One privatised step; returns (G_out, norms_out).

    ``step`` is a number, or a one-element int64 CUDA tensor read when the kernels run
    (dp_linear_step_dev_step), so that a CUDA graph of this call serves every step.
    """
    import torch

    B, T, d_in, d_out = _bt_dims(X, dY)
    if P is not None:
        r = _projection_width(P, X, d_out)
    width = r if r else d_out
    _holds_fp32(G_out, "G_out", d_in * width)
    _holds_fp32(norms_out, "norms_out", B)
    ws = _workspace(X, dY, r, workspace, method)
    if G_out is None:
        G_out = torch.empty(d_in, width, dtype=torch.float32, device=X.device)
    if norms_out is None:
        norms_out = torch.empty(B, dtype=torch.float32, device=X.device)
    dstep = _device_step(step)
    if dstep is not None:
        check(lib().dp_linear_step_dev_step(_ptr(X), _ptr(dY), _ptr(P), r, _dtype_code(X), B, T, d_in, d_out,
                                            float(C), float(sigma), int(seed), _ptr(dstep), int(layer_id),
                                            METHODS[method], _ptr(norms_out), _ptr(G_out), _ptr(ws),
                                            ws.numel(), _stream(stream)),
              "dp_linear_step_dev_step")
    else:
        check(lib().dp_linear_step(_ptr(X), _ptr(dY), _ptr(P), r, _dtype_code(X), B, T, d_in, d_out,
                                   float(C), float(sigma), int(seed), int(step), int(layer_id),
                                   METHODS[method], _ptr(norms_out), _ptr(G_out), _ptr(ws), ws.numel(),
                                   _stream(stream)),
              "dp_linear_step")
    return G_out, norms_out


def dp_philox_blocks(nblocks, seed, step, layer_id, stream_id, out=None, device="cuda", stream=None):
    """Raw Philox4x32-10 words [nblocks, 4] (int32 tensor holding the uint32 bits)."""
    import torch

    if out is None:
        out = torch.empty(int(nblocks), 4, dtype=torch.int32, device=device)
    check(lib().dp_philox_blocks(_ptr(out), int(nblocks), int(seed), int(step), int(layer_id),
                                 int(stream_id), _stream(stream)),
          "dp_philox_blocks")
    return out


def dp_box_muller(words, out=None, stream=None):
    """The noise's Box-Muller transform of word pairs: words int32/uint32 [n, 2] on the device
    (the uint32 bits) -> fp64 [n, 2] (z_even, z_odd) before the sigma*C scaling."""
    import torch

    n = int(words.shape[0])
    if out is None:
        out = torch.empty(n, 2, dtype=torch.float64, device=words.device)
    check(lib().dp_box_muller(_ptr(words), n, _ptr(out), _stream(stream)), "dp_box_muller")
    return out


def dp_workspace_status(workspace, stream=None):
    return lib().dp_workspace_status(_ptr(workspace), _stream(stream))


def auto_norm_method(B, T, d_in, d_out, r=0, dtype_code=DP_BF16):
    return METHOD_NAMES[lib().dp_auto_norm_method(B, T, d_in, d_out, r, dtype_code)]


def kernel_launches():
    """Kernels launched by the library so far in this process."""
    return int(lib().dp_kernel_launches())


def profiling_enable(on=True):
    check(lib().dp_profiling_enable(1 if on else 0), "dp_profiling_enable")


def profiling_collect():
    """{kernel kind: (device ms, launches)} for the launches recorded since the last collect."""
    n = int(lib().dp_profiling_kinds())
    ms = (ctypes.c_double * n)()
    cnt = (_c_ll * n)()
    check(lib().dp_profiling_collect(ms, cnt), "dp_profiling_collect")
    return {lib().dp_profiling_kind_name(k).decode(): (ms[k], cnt[k]) for k in range(n) if cnt[k]}


def dp_block_step(layers, mode="per_layer", C=1.0, sigma=0.0, seed=0, step=0, method="auto",
                  flat_norms_out=None, workspace=None, stream=None):
    """One step for a block of linears sharing the batch.

    ``layers``: dicts with X, dY, layer_id, C (per-layer bound), and optional G_out, norms_out and
    P (a [d_out, r] projection: the layer then clips and noises G_i P).
    ``step``: a number, or a one-element int64 CUDA tensor read when the kernels run.
    Returns (list of G_out, list of norms_out or None, flat_norms_out or None).
    """
    import torch

    first = layers[0]
    B, T = int(first["X"].shape[0]), int(first["X"].shape[1])
    dt = _dtype_code(first["X"])
    arr = (DpLayer * len(layers))()
    outs, norms = [], []
    for k, l in enumerate(layers):
        _, _, d_in, d_out = _bt_dims(l["X"], l["dY"])
        P = l.get("P")
        r = _projection_width(P, l["X"], d_out)
        G = l.get("G_out")
        if G is None:
            G = torch.empty(d_in, r or d_out, dtype=torch.float32, device=l["X"].device)
        n = l.get("norms_out")
        _holds_fp32(G, "G_out", d_in * (r or d_out))
        _holds_fp32(n, "norms_out", B)
        arr[k] = DpLayer(_ptr(l["X"]), _ptr(l["dY"]), d_in, d_out, int(l["layer_id"]), float(l.get("C", C)),
                         _ptr(G), _ptr(n), _ptr(P), r)
        outs.append(G)
        norms.append(n)
    need = int(lib().dp_block_workspace_size(arr, len(layers), B, T, dt, CLIP_MODES[mode], METHODS[method]))
    if need == 0:
        raise DPError(DP_ERR_INVALID_ARG, "dp_block_workspace_size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=first["X"].device)
    if mode == "flat" and flat_norms_out is None:
        flat_norms_out = torch.empty(B, dtype=torch.float32, device=first["X"].device)
    dstep = _device_step(step)
    if dstep is not None:
        check(lib().dp_block_step_dev_step(arr, len(layers), dt, B, T, CLIP_MODES[mode], float(C), float(sigma),
                                           int(seed), _ptr(dstep), METHODS[method], _ptr(flat_norms_out),
                                           _ptr(workspace), workspace.numel(), _stream(stream)),
              "dp_block_step_dev_step")
    else:
        check(lib().dp_block_step(arr, len(layers), dt, B, T, CLIP_MODES[mode], float(C), float(sigma),
                                  int(seed), int(step), METHODS[method], _ptr(flat_norms_out),
                                  _ptr(workspace), workspace.numel(), _stream(stream)),
              "dp_block_step")
    return outs, norms, flat_norms_out


def dp_projected_adam_step(W, R, m, v, P, lr, t, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0,
                           workspace=None, stream=None):
    """One projected Adam update: W -= lr * U P^T with Adam moments m, v kept in r-space."""
    import torch

    d_in, d_out = int(W.shape[0]), int(W.shape[1])
    r = int(R.shape[1])
    if workspace is None:
        workspace = torch.empty(int(lib().dp_adam_workspace_size(d_in, r)), dtype=torch.uint8, device=W.device)
    check(lib().dp_projected_adam_step(_ptr(W), _ptr(R), _ptr(m), _ptr(v), _ptr(P), _dtype_code(P), d_in, d_out,
                                       r, float(lr), float(beta1), float(beta2), float(eps), float(grad_scale),
                                       int(t), _ptr(workspace), workspace.numel(), _stream(stream)),
          "dp_projected_adam_step")
    return W, m, v


# ---------------------------------------------------------------- embedding, RMS norm, Muon
class _Launch:
    """The stream one call is enqueued on.  Every tensor given (the first is not None) must be
    contiguous and on one CUDA device; while the object is entered, that device and the call's
    stream are current, so that what the binding allocates for the call belongs to that stream.
    Entering gives the stream's handle.  ``names``: the tensors' names, for the errors."""

    __slots__ = ("index", "ctx")

    def __init__(self, stream, names, *tensors):
        import torch

        index = self.index = tensors[0].get_device()
        ok = index >= 0
        for t in tensors:
            if t is not None and (t.get_device() != index or not t.is_contiguous()):
                ok = False
        if not ok:
            self._complain(names, tensors)
        self.ctx = None
        if stream is not None:   # also makes the stream's device current
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=tensors[0].device)
            if stream.device != tensors[0].device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {tensors[0].device}")
            self.ctx = torch.cuda.stream(stream)
        elif index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(index)

    @staticmethod
    def _complain(names, tensors):
        for name, t in zip(names.split(), tensors):
            if t is not None:
                if not t.is_cuda:
                    raise ValueError(f"{name} must be a CUDA tensor")
                if t.device != tensors[0].device:
                    raise ValueError(f"{name} is on {t.device}, the first tensor on {tensors[0].device}")
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return False


_short_stream = None


def _raw_stream(index):
    """The handle of the device's current stream (the short way to it where torch has one: a
    Stream object costs 3 us, a third of a small call)."""
    global _short_stream
    if _short_stream is None:
        import torch

        _short_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _short_stream(index)


def _expect(t, name, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, got {t.dtype} {list(t.shape)}")


def _scratch(workspace, need, device, what):
    import torch

    if need == 0:
        raise DPError(DP_ERR_INVALID_ARG, what)
    return torch.empty(need, dtype=torch.uint8, device=device) if workspace is None else workspace


def _ws_bytes(ws):
    return ws.numel() * ws.element_size()


def _index_code(ids):
    import torch

    if ids.dtype == torch.int64:
        return DP_I64
    if ids.dtype == torch.int32:
        return DP_I32
    raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")


def dp_embedding_lookup(W, ids, scale=1.0, out=None, out_dtype=None, stream=None):
    """scale * W[ids] ([*ids.shape, d]); ids outside the table give rows of zeros."""
    import torch

    if W.dim() != 2:
        raise ValueError("W must be [V, d]")
    V, d = W.shape
    dtype = out.dtype if out is not None else (out_dtype or W.dtype)
    shape = (*ids.shape, d)
    _expect(out, "out", shape, dtype)
    with _Launch(stream, "W ids out", W, ids, out) as s:
        Y = torch.empty(shape, dtype=dtype, device=W.device) if out is None else out
        if ids.numel():
            check(lib().dp_embedding_lookup(_ptr(W), _dtype_code(W), _ptr(ids), _index_code(ids), float(scale),
                                            ids.numel(), V, d, _ptr(Y), _dtype_code(Y), s),
                  "dp_embedding_lookup")
    return Y


def _embedding_dims(ids, dY):
    if dY.dim() == 3:
        B, T, d = dY.shape
        if ids.shape == (B, T):
            return B, T, d
    raise ValueError("ids must be [B, T] and dY [B, T, d]")


# The sizes depend on their arguments alone, and a call through ctypes costs a microsecond.
@functools.lru_cache(maxsize=1024)
def embedding_workspace_size(B, T, V, d, dtype_code=DP_BF16):
    return int(lib().dp_embedding_workspace_size(B, T, V, d, dtype_code))


def _padding(padding_idx):
    return -1 if padding_idx is None else int(padding_idx)


def dp_embedding_per_sample_norms(ids, dY, V, scale=1.0, padding_idx=None, norms=None, workspace=None, stream=None):
    """Per-sample norms (fp32 [B]) of the gradient of an embedding table of V rows."""
    import torch

    B, T, d = _embedding_dims(ids, dY)
    _expect(norms, "norms", (B,), torch.float32)
    with _Launch(stream, "dY ids norms workspace", dY, ids, norms, workspace) as s:
        ws = _scratch(workspace, embedding_workspace_size(B, T, int(V), d, _dtype_code(dY)), dY.device,
                      "dp_embedding_workspace_size")
        if norms is None:
            norms = torch.empty(B, dtype=torch.float32, device=dY.device)
        check(lib().dp_embedding_per_sample_norms(_ptr(ids), _index_code(ids), _ptr(dY), _dtype_code(dY), B, T,
                                                  int(V), d, float(scale), _padding(padding_idx), _ptr(norms),
                                                  _ptr(ws), _ws_bytes(ws), s),
              "dp_embedding_per_sample_norms")
    return norms


def dp_embedding_clip_accumulate(ids, dY, norms, C, G_sum, scale=1.0, padding_idx=None, workspace=None, stream=None):
    """G_sum[V, d] += sum_i c_i G_i for given norms; rows that no token names are not touched."""
    import torch

    B, T, d = _embedding_dims(ids, dY)
    if G_sum.dim() != 2:
        raise ValueError("G_sum must be [V, d]")
    V = int(G_sum.shape[0])
    _expect(G_sum, "G_sum", (V, d), torch.float32)
    _expect(norms, "norms", (B,), torch.float32)
    with _Launch(stream, "dY ids norms G_sum workspace", dY, ids, norms, G_sum, workspace) as s:
        ws = _scratch(workspace, embedding_workspace_size(B, T, V, d, _dtype_code(dY)), dY.device,
                      "dp_embedding_workspace_size")
        check(lib().dp_embedding_clip_accumulate(_ptr(ids), _index_code(ids), _ptr(dY), _dtype_code(dY), B, T, V, d,
                                                 float(scale), _padding(padding_idx), _ptr(norms), float(C),
                                                 _ptr(G_sum), _ptr(ws), _ws_bytes(ws), s),
              "dp_embedding_clip_accumulate")
    return G_sum


def dp_embedding_step(ids, dY, V, C, sigma, seed, step, layer_id, scale=1.0, padding_idx=None, norms_out=None,
                      G_out=None, workspace=None, stream=None):
    """The privatised gradient of an embedding table of V rows; returns (G_out [V, d], norms_out).

    ``ids`` [B, T] int32 or int64, ``dY`` [B, T, d]; ``step`` as in dp_linear_step.
    An id >= V is recorded in the workspace's status word, so a caller who wants to know brings the
    workspace (embedding_workspace_size) and asks dp_workspace_status.
    """
    import torch

    B, T, d = _embedding_dims(ids, dY)
    V = int(V)
    _expect(G_out, "G_out", (V, d), torch.float32)
    _expect(norms_out, "norms_out", (B,), torch.float32)
    dstep = _device_step(step)
    with _Launch(stream, "dY ids norms_out G_out workspace step", dY, ids, norms_out, G_out, workspace, dstep) as s:
        ws = _scratch(workspace, embedding_workspace_size(B, T, V, d, _dtype_code(dY)), dY.device,
                      "dp_embedding_workspace_size")
        if G_out is None:
            G_out = torch.empty(V, d, dtype=torch.float32, device=dY.device)
        if norms_out is None:
            norms_out = torch.empty(B, dtype=torch.float32, device=dY.device)
        entry = lib().dp_embedding_step if dstep is None else lib().dp_embedding_step_dev_step
        check(entry(_ptr(ids), _index_code(ids), _ptr(dY), _dtype_code(dY), B, T, V, d, float(scale),
                    _padding(padding_idx), float(C), float(sigma), int(seed),
                    int(step) if dstep is None else _ptr(dstep), int(layer_id), _ptr(norms_out), _ptr(G_out),
                    _ptr(ws), _ws_bytes(ws), s),
              "dp_embedding_step")
    return G_out, norms_out


def dp_rmsnorm(X, gain, eps=1e-6, residual=None, H_out=None, Y=None, stream=None):
    """(y, h): h = X + residual (X itself without one), y = h / rms(h) * gain, over the last axis."""
    import torch

    shape, dtype = X.shape, X.dtype
    d = shape[-1]
    _expect(gain, "gain", (d,), torch.float32)
    _expect(residual, "residual", shape, dtype)
    _expect(H_out, "H_out", shape, dtype)
    _expect(Y, "Y", shape, dtype)
    if residual is None and H_out is not None:
        raise ValueError("H_out needs a residual: without one h is X itself")
    with _Launch(stream, "X gain residual H_out Y", X, gain, residual, H_out, Y) as s:
        Y = torch.empty_like(X) if Y is None else Y
        H = X
        if residual is not None:
            H = torch.empty_like(X) if H_out is None else H_out
        if X.numel():
            check(lib().dp_rmsnorm(_ptr(X), _ptr(residual), _ptr(gain), _dtype_code(X), X.numel() // d, d, float(eps),
                                   _ptr(H) if residual is not None else None, _ptr(Y), s), "dp_rmsnorm")
    return Y, H


@functools.lru_cache(maxsize=1024)
def rmsnorm_workspace_size(B, T, d, dtype_code=DP_BF16):
    return int(lib().dp_rmsnorm_workspace_size(B, T, d, dtype_code))


def _norm_dims(H, dY, gain, residual_grad, dX):
    import torch

    shape, dtype = H.shape, H.dtype
    if len(shape) != 3:
        raise ValueError("H must be [B, T, d]")
    B, T, d = shape
    _expect(dY, "dY", shape, dtype)
    _expect(gain, "gain", (d,), torch.float32)
    _expect(residual_grad, "residual_grad", shape, dtype)
    _expect(dX, "dX", shape, dtype)
    return B, T, d


def dp_rmsnorm_backward(H, gain, dY, eps=1e-6, residual_grad=None, dX=None, per_sample=None, norms=None,
                        workspace=None, stream=None):
    """(dX, per-sample gain gradients fp32 [B, d], their norms fp32 [B]); nothing is clipped yet."""
    import torch

    B, T, d = _norm_dims(H, dY, gain, residual_grad, dX)
    _expect(per_sample, "per_sample", (B, d), torch.float32)
    _expect(norms, "norms", (B,), torch.float32)
    with _Launch(stream, "H gain dY residual_grad dX per_sample norms workspace", H, gain, dY, residual_grad, dX,
                 per_sample, norms, workspace) as s:
        ws = _scratch(workspace, rmsnorm_workspace_size(B, T, d, _dtype_code(H)), H.device,
                      "dp_rmsnorm_workspace_size")
        dX = torch.empty_like(H) if dX is None else dX
        if per_sample is None:
            per_sample = torch.empty(B, d, dtype=torch.float32, device=H.device)
        if norms is None:
            norms = torch.empty(B, dtype=torch.float32, device=H.device)
        check(lib().dp_rmsnorm_backward(_ptr(H), _ptr(gain), _ptr(dY), _ptr(residual_grad), _dtype_code(H), B, T, d,
                                        float(eps), _ptr(dX), _ptr(per_sample), _ptr(norms), _ptr(ws), _ws_bytes(ws),
                                        s), "dp_rmsnorm_backward")
    return dX, per_sample, norms


def dp_rmsnorm_clip_accumulate(per_sample, norms, C, G_sum, stream=None):
    """G_sum[d] += sum_i min(1, C / norms[i]) per_sample[i]."""
    import torch

    if per_sample.dim() != 2:
        raise ValueError("per_sample must be [B, d]")
    B, d = int(per_sample.shape[0]), int(per_sample.shape[1])
    _expect(per_sample, "per_sample", (B, d), torch.float32)
    _expect(norms, "norms", (B,), torch.float32)
    _expect(G_sum, "G_sum", (d,), torch.float32)
    with _Launch(stream, "per_sample norms G_sum", per_sample, norms, G_sum) as s:
        check(lib().dp_rmsnorm_clip_accumulate(_ptr(per_sample), _ptr(norms), B, d, float(C), _ptr(G_sum), s),
              "dp_rmsnorm_clip_accumulate")
    return G_sum


def dp_rmsnorm_step(H, gain, dY, C, sigma, seed, step, layer_id, eps=1e-6, residual_grad=None, dX=None,
                    norms_out=None, G_out=None, workspace=None, stream=None):
    """The backward of dp_rmsnorm with the gain's privatised gradient: (dX, G_out [d], norms_out).

    ``H`` is the h of the forward, ``residual_grad`` the gradient that reaches h past the norm;
    ``step`` as in dp_linear_step.
    """
    import torch

    B, T, d = _norm_dims(H, dY, gain, residual_grad, dX)
    _expect(G_out, "G_out", (d,), torch.float32)
    _expect(norms_out, "norms_out", (B,), torch.float32)
    dstep = _device_step(step)
    with _Launch(stream, "H gain dY residual_grad dX norms_out G_out workspace step", H, gain, dY, residual_grad, dX,
                 norms_out, G_out, workspace, dstep) as s:
        ws = _scratch(workspace, rmsnorm_workspace_size(B, T, d, _dtype_code(H)), H.device,
                      "dp_rmsnorm_workspace_size")
        dX = torch.empty_like(H) if dX is None else dX
        if G_out is None:
            G_out = torch.empty(d, dtype=torch.float32, device=H.device)
        if norms_out is None:
            norms_out = torch.empty(B, dtype=torch.float32, device=H.device)
        entry = lib().dp_rmsnorm_step if dstep is None else lib().dp_rmsnorm_step_dev_step
        check(entry(_ptr(H), _ptr(gain), _ptr(dY), _ptr(residual_grad), _dtype_code(H), B, T, d, float(eps), float(C),
                    float(sigma), int(seed), int(step) if dstep is None else _ptr(dstep), int(layer_id), _ptr(dX),
                    _ptr(norms_out), _ptr(G_out), _ptr(ws), _ws_bytes(ws), s),
              "dp_rmsnorm_step")
    return dX, G_out, norms_out


@functools.lru_cache(maxsize=1024)
def muon_workspace_size(rows, cols):
    return int(lib().dp_muon_workspace_size(rows, cols))


def dp_orthogonalize(G, steps=5, U=None, workspace=None, stream=None):
    """G [rows, cols] (fp32 or bf16) orthogonalised by `steps` Newton-Schulz products, in bf16."""
    import torch

    if G.dim() != 2:
        raise ValueError("G must be [rows, cols]")
    rows, cols = int(G.shape[0]), int(G.shape[1])
    _expect(U, "U", (rows, cols), torch.bfloat16)
    with _Launch(stream, "G U workspace", G, U, workspace) as s:
        ws = _scratch(workspace, muon_workspace_size(rows, cols), G.device, "dp_muon_workspace_size")
        U = torch.empty(rows, cols, dtype=torch.bfloat16, device=G.device) if U is None else U
        check(lib().dp_orthogonalize(_ptr(G), _dtype_code(G), rows, cols, int(steps), _ptr(U), _ptr(ws),
                                     _ws_bytes(ws), s), "dp_orthogonalize")
    return U


def dp_muon_step(W, R, M, lr, momentum=0.95, nesterov=True, weight_decay=0.0, grad_scale=1.0, update_scale=1.0,
                 steps=5, workspace=None, stream=None):
    """One Muon update of W [d_in, d_out] with the privatised gradient R and the momentum M, both
    W and M in place (fp32); returns (W, M)."""
    import torch

    if W.dim() != 2:
        raise ValueError("W must be [d_in, d_out]")
    for name, t in (("W", W), ("R", R), ("M", M)):
        _expect(t, name, W.shape, torch.float32)
    d_in, d_out = int(W.shape[0]), int(W.shape[1])
    with _Launch(stream, "W R M workspace", W, R, M, workspace) as s:
        ws = _scratch(workspace, muon_workspace_size(d_in, d_out), W.device, "dp_muon_workspace_size")
        check(lib().dp_muon_step(_ptr(W), _ptr(R), _ptr(M), d_in, d_out, float(lr), float(momentum),
                                 1 if nesterov else 0, float(weight_decay), float(grad_scale), float(update_scale),
                                 int(steps), _ptr(ws), _ws_bytes(ws), s), "dp_muon_step")
    return W, M
