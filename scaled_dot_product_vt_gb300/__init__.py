"""Python binding of the vt_attn C ABI (include/vt_attn.h): argument marshalling only.

Every step of the attention forward runs in the CUDA kernels of ``libvt_attn.so``;
this module only converts arguments and calls the C entry points through ctypes.
There is no fallback: if the library is missing or cannot be loaded, every call
raises.  PyTorch is used for device memory and the current stream.
"""

from __future__ import annotations

import ctypes
import os
import numbers
import struct

from ._build import LIB, LIB_DEBUG, build  # noqa: F401

VT_F32, VT_BF16 = 0, 1
VT_OPT_TEST_STALL = 1
VT_OPT_TEST_BOUNDS = 2
VT_MASK_NONE, VT_MASK_CAUSAL, VT_MASK_WINDOW, VT_MASK_WINDOW_COMPLEMENT = 0, 1, 2, 3
MASKS = {"none": VT_MASK_NONE, "causal": VT_MASK_CAUSAL, "window": VT_MASK_WINDOW,
         "window_complement": VT_MASK_WINDOW_COMPLEMENT}

STATUS = {
    0: "VT_OK", 1: "VT_ERR_INVALID_ARG", 2: "VT_ERR_UNSUPPORTED", 3: "VT_ERR_MISALIGNED",
    4: "VT_ERR_CUDA", 5: "VT_ERR_DEVICE_TIMEOUT", 6: "VT_ERR_DEVICE_BOUNDS",
}

# Every symbol the header declares.
EXPORTS = ("vt_attn_fwd", "vt_attn_fwd_strided", "vt_attn_fwd_ex", "vt_attn_fwd_splitkv",
           "vt_attn_splitkv_workspace_size", "vt_attn_splitkv_choose", "vt_attn_fwd_splitkv_noalloc",
           "vt_attn_fwd_general", "vt_qk_rope_fwd", "vt_qk_rope_bwd", "vt_qk_rope_bwd_workspace_size",
           "vt_attn_fwd_prefix", "vt_attn_prefix_workspace_size", "vt_attn_fwd_tree",
           "vt_attn_tree_workspace_size",
           "vt_attn_fwd_packed", "vt_attn_bwd_packed", "vt_attn_bwd_packed_workspace_size",
           "vt_status_str", "vt_last_device_status")


class VtError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class vt_attn_opts(ctypes.Structure):
    _fields_ = [("wait_timeout_ns", ctypes.c_uint64), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class vt_attn_mask(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("offset", ctypes.c_int64),
                ("window", ctypes.c_int64)]


_lib = None


def load(path: str | None = None):
    """Load libvt_attn.so (it must have been built; see ``build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: run scaled_dot_product_vt_gb300.build() (the CUDA path has no fallback)")
    lib = ctypes.CDLL(p)
    i64, vp, f, i, u = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_uint
    st3 = ctypes.POINTER(ctypes.c_int64)
    lib.vt_attn_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f, i, i, vp]
    lib.vt_attn_fwd.restype = i
    lib.vt_attn_fwd_strided.argtypes = [vp, st3, vp, st3, vp, st3, vp, st3, i64, i64, i64, i64, i64, i64, f, i, i, vp]
    lib.vt_attn_fwd_strided.restype = i
    lib.vt_attn_fwd_ex.argtypes = [vp, st3, vp, st3, vp, st3, vp, st3, i64, i64, i64, i64, i64, i64, f, i, i,
                                   ctypes.POINTER(vt_attn_opts), vp]
    lib.vt_attn_fwd_ex.restype = i
    sz = ctypes.c_size_t
    lib.vt_attn_fwd_splitkv.argtypes = [vp, st3, vp, st3, vp, st3, vp, st3, i64, i64, i64, i64, i64, i64, f, i, i,
                                        i, vp, sz, vp]
    lib.vt_attn_fwd_splitkv.restype = i
    lib.vt_attn_splitkv_workspace_size.argtypes = [i64, i64, i64, i64, i]
    lib.vt_attn_splitkv_workspace_size.restype = sz
    lib.vt_attn_splitkv_choose.argtypes = [i64, i64, i64, i64, i, i]
    lib.vt_attn_splitkv_choose.restype = i
    lib.vt_attn_fwd_splitkv_noalloc.argtypes = [vp, st3, vp, st3, vp, st3, vp, st3, i64, i64, i64, i64, i64, i64,
                                                f, i, i, i, vp]
    lib.vt_attn_fwd_splitkv_noalloc.restype = i
    lib.vt_attn_fwd_general.argtypes = [vp, st3, vp, st3, vp, st3, vp, st3, vp, i64, i64, i64, i64, i64, i64, i64, f,
                                        i, ctypes.POINTER(vt_attn_mask), i, vp, sz, ctypes.POINTER(vt_attn_opts), vp]
    lib.vt_attn_fwd_general.restype = i
    lib.vt_qk_rope_fwd.argtypes = [ctypes.c_char_p, vp]
    lib.vt_qk_rope_fwd.restype = i
    lib.vt_qk_rope_bwd.argtypes = [ctypes.c_char_p, vp, st3, vp, st3, vp, vp, vp, sz, vp]
    lib.vt_qk_rope_bwd.restype = i
    lib.vt_qk_rope_bwd_workspace_size.argtypes = [i64]
    lib.vt_qk_rope_bwd_workspace_size.restype = sz
    lib.vt_attn_fwd_prefix.argtypes = [ctypes.c_char_p, vp]
    lib.vt_attn_fwd_prefix.restype = i
    lib.vt_attn_fwd_tree.argtypes = [ctypes.c_char_p, vp, vp]
    lib.vt_attn_fwd_tree.restype = i
    lib.vt_attn_prefix_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, i64, i64, i]
    lib.vt_attn_prefix_workspace_size.restype = sz
    lib.vt_attn_tree_workspace_size.argtypes = lib.vt_attn_prefix_workspace_size.argtypes
    lib.vt_attn_tree_workspace_size.restype = sz
    lib.vt_attn_fwd_packed.argtypes = [ctypes.c_char_p, vp]
    lib.vt_attn_fwd_packed.restype = i
    lib.vt_attn_bwd_packed.argtypes = [ctypes.c_char_p, ctypes.c_char_p, vp]
    lib.vt_attn_bwd_packed.restype = i
    lib.vt_attn_bwd_packed_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, i64, i]
    lib.vt_attn_bwd_packed_workspace_size.restype = sz
    lib.vt_status_str.argtypes = [i]
    lib.vt_status_str.restype = ctypes.c_char_p
    lib.vt_last_device_status.argtypes = [vp]
    lib.vt_last_device_status.restype = i
    if path is None:
        _lib = lib
    return lib


def load_debug():
    """Load libvt_attn_debug.so: the same entry points, with device index checks (VT_DEBUG) that report
    VT_ERR_DEVICE_BOUNDS.  Returns a separate handle; the module-level wrappers keep using the release
    library."""
    return load(LIB_DEBUG)


def _stride3(s):
    if s is None:
        return None
    return (ctypes.c_int64 * 3)(*[int(x) for x in s])


def vt_attn_fwd(Q, K, V, O, B, H, S_q, S_k, D_qk, D_v, scale, causal, dtype, stream) -> int:
    """The C entry point with raw device addresses (ints); returns the vt_status code."""
    return load().vt_attn_fwd(Q, K, V, O, B, H, S_q, S_k, D_qk, D_v, scale, int(causal), dtype, stream)


def vt_attn_fwd_strided(Q, q_stride, K, k_stride, V, v_stride, O, o_stride,
                        B, H, S_q, S_k, D_qk, D_v, scale, causal, dtype, stream) -> int:
    return load().vt_attn_fwd_strided(Q, _stride3(q_stride), K, _stride3(k_stride), V, _stride3(v_stride),
                                      O, _stride3(o_stride), B, H, S_q, S_k, D_qk, D_v, scale, int(causal),
                                      dtype, stream)


def vt_attn_fwd_ex(Q, q_stride, K, k_stride, V, v_stride, O, o_stride,
                   B, H, S_q, S_k, D_qk, D_v, scale, causal, dtype, opts, stream) -> int:
    return load().vt_attn_fwd_ex(Q, _stride3(q_stride), K, _stride3(k_stride), V, _stride3(v_stride),
                                 O, _stride3(o_stride), B, H, S_q, S_k, D_qk, D_v, scale, int(causal), dtype,
                                 ctypes.byref(opts) if opts is not None else None, stream)


def vt_attn_fwd_splitkv(Q, q_stride, K, k_stride, V, v_stride, O, o_stride, B, H, S_q, S_k, D_qk, D_v,
                        scale, causal, dtype, n_split, workspace, workspace_bytes, stream) -> int:
    return load().vt_attn_fwd_splitkv(Q, _stride3(q_stride), K, _stride3(k_stride), V, _stride3(v_stride),
                                      O, _stride3(o_stride), B, H, S_q, S_k, D_qk, D_v, scale, int(causal), dtype,
                                      int(n_split), workspace, int(workspace_bytes), stream)


def vt_attn_splitkv_workspace_size(B, H, S_q, D_v, n_split) -> int:
    return int(load().vt_attn_splitkv_workspace_size(B, H, S_q, D_v, int(n_split)))


def vt_attn_splitkv_choose(B, H, S_q, S_k, causal, dtype) -> int:
    return int(load().vt_attn_splitkv_choose(B, H, S_q, S_k, int(causal), dtype))


def vt_attn_fwd_splitkv_noalloc(Q, q_stride, K, k_stride, V, v_stride, O, o_stride, B, H, S_q, S_k, D_qk, D_v,
                                scale, causal, dtype, n_split, stream) -> int:
    """Split-KV forward whose scratch is the library's fixed 32 MiB device array: for callers that
    may not allocate device memory.  Raw device addresses (ints); returns the vt_status code."""
    return load().vt_attn_fwd_splitkv_noalloc(Q, _stride3(q_stride), K, _stride3(k_stride), V, _stride3(v_stride),
                                              O, _stride3(o_stride), B, H, S_q, S_k, D_qk, D_v, scale, int(causal),
                                              dtype, int(n_split), stream)


def vt_attn_fwd_general(Q, q_stride, K, k_stride, V, v_stride, O, o_stride, lse, B, H, H_kv, S_q, S_k, D_qk, D_v,
                        scale, dtype, mask, n_split, workspace, workspace_bytes, opts, stream) -> int:
    """The general C entry point with raw device addresses (ints; lse and workspace may be None);
    ``mask`` is a vt_attn_mask or None.  Returns the vt_status code."""
    return load().vt_attn_fwd_general(Q, _stride3(q_stride), K, _stride3(k_stride), V, _stride3(v_stride), O,
                                      _stride3(o_stride), lse, B, H, H_kv, S_q, S_k, D_qk, D_v, scale, dtype,
                                      ctypes.byref(mask) if mask is not None else None, int(n_split), workspace,
                                      int(workspace_bytes), ctypes.byref(opts) if opts is not None else None, stream)


# vt_qk_rope_args in field order (every field is aligned without padding): its size and the addresses, then the rest
_QK_ROPE_PTRS = struct.Struct("=12Q")
_QK_ROPE_REST = struct.Struct("=8q4ifi21q128s")
_QK_ROPE_BYTES = _QK_ROPE_PTRS.size + _QK_ROPE_REST.size


def vt_qk_rope_fwd(args: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_qk_rope_args; returns the vt_status code."""
    return load().vt_qk_rope_fwd(args, stream)


def vt_qk_rope_bwd(args: bytes, dq_out, dq_out_stride, dk_out, dk_out_stride, dq_weight, dk_weight, workspace,
                   workspace_bytes, stream) -> int:
    return load().vt_qk_rope_bwd(args, dq_out, _stride3(dq_out_stride), dk_out, _stride3(dk_out_stride), dq_weight,
                                 dk_weight, workspace, int(workspace_bytes), stream)


def vt_qk_rope_bwd_workspace_size(D) -> int:
    return int(load().vt_qk_rope_bwd_workspace_size(D))


# vt_attn_prefix_args in field order (every field is aligned without padding): its size, the addresses and the
# workspace's size, then the rest
_ATTN_PREFIX_PTRS = struct.Struct("=11Q")
_ATTN_PREFIX_REST = struct.Struct("=8qif16q")
_ATTN_PREFIX_BYTES = _ATTN_PREFIX_PTRS.size + _ATTN_PREFIX_REST.size


def vt_attn_fwd_prefix(args: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_attn_prefix_args; returns the vt_status code."""
    return load().vt_attn_fwd_prefix(args, stream)


def vt_attn_tree_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype) -> int:
    return int(load().vt_attn_tree_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype))


def vt_attn_fwd_tree(args: bytes, parents, stream) -> int:
    """The C entry point: ``args`` is a packed vt_attn_prefix_args; returns the vt_status code."""
    return load().vt_attn_fwd_tree(args, parents, stream)


def vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype) -> int:
    return int(load().vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype))


# vt_attn_packed_args and vt_attn_packed_grads in field order (every field is aligned without padding): the size and the
# addresses (and the workspace's size), then the rest
_ATTN_PACKED_PTRS = struct.Struct("=8Q")
_ATTN_PACKED_REST = struct.Struct("=8qifii8q")
_ATTN_PACKED_BYTES = _ATTN_PACKED_PTRS.size + _ATTN_PACKED_REST.size
_PACKED_GRADS_PTRS = struct.Struct("=8Q")
_PACKED_GRADS_REST = struct.Struct("=8q")
_PACKED_GRADS_BYTES = _PACKED_GRADS_PTRS.size + _PACKED_GRADS_REST.size


def vt_attn_fwd_packed(args: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_attn_packed_args; returns the vt_status code."""
    return load().vt_attn_fwd_packed(args, stream)


def vt_attn_bwd_packed(args: bytes, grads: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_attn_packed_args and ``grads`` a packed vt_attn_packed_grads; returns
    the vt_status code."""
    return load().vt_attn_bwd_packed(args, grads, stream)


def vt_attn_bwd_packed_workspace_size(N, H, H_kv, T_q, T_k, D_qk, D_v, dtype) -> int:
    return int(load().vt_attn_bwd_packed_workspace_size(N, H, H_kv, T_q, T_k, D_qk, D_v, dtype))


def vt_status_str(code: int) -> str:
    return load().vt_status_str(code).decode()


def vt_last_device_status(stream=None) -> int:
    return load().vt_last_device_status(_stream_handle(stream))


# ---------------------------------------------------------------- torch conveniences

def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return VT_BF16
    if t.dtype == torch.float32:
        return VT_F32
    raise TypeError(f"vt_attn supports bfloat16 and float32 tensors, got {t.dtype}")


def _bhs_strides(t):
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("tensors are [B, H, S, D] with the last dimension contiguous")
    return (t.stride(0), t.stride(1), t.stride(2))


def attn_fwd(q, k, v, scale: float | None = None, causal: bool = False, out=None, stream=None, opts=None):
    """O = softmax(scale * q k^T) v for CUDA tensors q [B,H,S_q,D_qk], k [B,H,S_k,D_qk], v [B,H,S_k,D_v].

    Strided inputs are passed as they are (last dimension contiguous).  ``out`` may be a
    preallocated (possibly strided) [B,H,S_q,D_v] tensor; otherwise one is allocated.
    """
    import torch
    B, H, S_q, D_qk = q.shape
    S_k, D_v = k.shape[2], v.shape[3]
    if k.shape != (B, H, S_k, D_qk) or v.shape != (B, H, S_k, D_v):
        raise ValueError("shape mismatch between q, k and v")
    code = _dtype_code(q)
    if _dtype_code(k) != code or _dtype_code(v) != code:
        raise TypeError("q, k and v must share one dtype")
    if scale is None:
        scale = float(D_qk) ** -0.5
    if out is None:
        out = torch.empty((B, H, S_q, D_v), dtype=q.dtype, device=q.device)
    rc = vt_attn_fwd_ex(q.data_ptr(), _bhs_strides(q), k.data_ptr(), _bhs_strides(k), v.data_ptr(),
                        _bhs_strides(v), out.data_ptr(), _bhs_strides(out), B, H, S_q, S_k, D_qk, D_v,
                        float(scale), causal, code, opts, _stream_handle(stream))
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd")
    return out


def attn_fwd_splitkv(q, k, v, scale: float | None = None, causal: bool = False, n_split: int | None = None,
                     out=None, workspace=None, stream=None):
    """Split-KV forward for CUDA tensors (bf16 or fp32).  ``n_split=None`` uses the
    library's choice; ``workspace`` may be a preallocated uint8 CUDA tensor of at least
    ``vt_attn_splitkv_workspace_size`` bytes (allocated here otherwise)."""
    import torch
    B, H, S_q, D_qk = q.shape
    S_k, D_v = k.shape[2], v.shape[3]
    if k.shape != (B, H, S_k, D_qk) or v.shape != (B, H, S_k, D_v):
        raise ValueError("shape mismatch between q, k and v")
    code = _dtype_code(q)
    if _dtype_code(k) != code or _dtype_code(v) != code:
        raise TypeError("q, k and v must share one dtype")
    if scale is None:
        scale = float(D_qk) ** -0.5
    if n_split is None:
        n_split = vt_attn_splitkv_choose(B, H, S_q, S_k, causal, code)
    if out is None:
        out = torch.empty((B, H, S_q, D_v), dtype=q.dtype, device=q.device)
    need = vt_attn_splitkv_workspace_size(B, H, S_q, D_v, n_split)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = vt_attn_fwd_splitkv(q.data_ptr(), _bhs_strides(q), k.data_ptr(), _bhs_strides(k), v.data_ptr(),
                             _bhs_strides(v), out.data_ptr(), _bhs_strides(out), B, H, S_q, S_k, D_qk, D_v,
                             float(scale), causal, code, n_split, ws_ptr, ws_bytes, _stream_handle(stream))
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd_splitkv")
    return out


def attn_fwd_general(q, k, v, scale: float | None = None, mask: str = "none", offset: int = 0, window: int = 0,
                     return_lse: bool = False, n_split: int = 1, out=None, lse=None, workspace=None, stream=None,
                     opts=None):
    """General forward for CUDA tensors: q [B,H,S_q,D_qk], k [B,H_kv,S_k,D_qk], v [B,H_kv,S_k,D_v] with H a
    multiple of H_kv (grouped heads), ``mask`` one of ``MASKS`` with ``offset`` and ``window`` (see
    include/vt_attn.h).  Returns O, or (O, LSE) with ``return_lse`` (LSE: float32 [B,H,S_q], natural log).
    ``n_split`` > 1 runs the split-KV form; its workspace is allocated here unless given."""
    import torch
    B, H, S_q, D_qk = q.shape
    H_kv, S_k, D_v = k.shape[1], k.shape[2], v.shape[3]
    if k.shape != (B, H_kv, S_k, D_qk) or v.shape != (B, H_kv, S_k, D_v):
        raise ValueError("shape mismatch between q, k and v")
    code = _dtype_code(q)
    if _dtype_code(k) != code or _dtype_code(v) != code:
        raise TypeError("q, k and v must share one dtype")
    if scale is None:
        scale = float(D_qk) ** -0.5
    if out is None:
        out = torch.empty((B, H, S_q, D_v), dtype=q.dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * S_q):
        raise ValueError("lse must be a contiguous float32 tensor of B*H*S_q elements")
    need = vt_attn_splitkv_workspace_size(B, H, S_q, D_v, n_split)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    m = vt_attn_mask(MASKS[mask], 0, int(offset), int(window))
    rc = vt_attn_fwd_general(q.data_ptr(), _bhs_strides(q), k.data_ptr(), _bhs_strides(k), v.data_ptr(),
                             _bhs_strides(v), out.data_ptr(), _bhs_strides(out),
                             lse.data_ptr() if lse is not None else None, B, H, H_kv, S_q, S_k, D_qk, D_v,
                             float(scale), code, m, n_split, ws_ptr, ws_bytes, opts, _stream_handle(stream))
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd_general")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------- token preparation

# The wrappers below check a call and pack the fixed part of its arguments once per combination of shapes, strides,
# types, devices and options (a plan, which holds no address), and add the addresses per call.  What they read of each
# tensor is written out: it is most of what a small call costs on the host, and a function for it half as much again.

_MOST_PLANS = 4096
_rope_plans, _rope_bwd_plans, _prefix_plans, _packed_plans, _packed_bwd_plans = {}, {}, {}, {}, {}


def _keep(plans, key, plan):
    if len(plans) >= _MOST_PLANS:
        plans.clear()
    plans[key] = plan
    return plan


def _elsewhere(fn, first, stream, args, kw):
    """Run a wrapper on another stream (a torch stream or a raw handle) or for tensors of another device than the
    current one: what it allocates is then allocated on that stream, and that device is current."""
    import torch
    if not first.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        with torch.cuda.device(first.device):
            return fn(*args, **kw)
    if not isinstance(stream, torch.cuda.Stream):
        # (torch takes an external stream of handle 0 for no handle, and makes a new stream)
        stream = (torch.cuda.ExternalStream(int(stream), device=first.device) if int(stream)
                  else torch.cuda.default_stream(first.device))
    if stream.device != first.device:
        raise ValueError("the stream must be of the tensors' device")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _here(t) -> bool:
    """The tensor is on the current CUDA device."""
    import torch
    return t.is_cuda and t.get_device() == torch.cuda.current_device()


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _workspace_bytes(workspace, first) -> int:
    if workspace is None:
        return 0
    if workspace.get_device() != first.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the other tensors")
    return workspace.numel() * workspace.element_size()


def _check(name, meta, dev, dtype, shape=None, dims=4):
    """Strides of a tensor of `dims` indices whose last one is contiguous, without the last."""
    t_shape, stride, t_dtype, t_dev = meta
    if t_dev != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    if len(t_shape) != dims or (stride[-1] != 1 and t_shape[-1] != 1):
        raise ValueError(f"{name} must have {dims} dimensions, the last one contiguous")
    if shape is not None and tuple(t_shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t_shape)}")
    if t_dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t_dtype}")
    return stride[:-1]


def _check_vector(name, meta, dev, dtype, n):
    shape, stride, t_dtype, t_dev = meta
    if t_dev != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    if t_dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t_dtype}")
    if len(shape) != 1 or (n is not None and shape[0] != n) or (shape[0] > 1 and stride[0] != 1):
        raise ValueError(f"{name} must be a contiguous vector" + (f" of {n} elements" if n is not None else ""))


def _contiguous(shape, strides) -> bool:
    """Whether elements of this shape lie behind each other (any strides do where there is none)."""
    want = 1
    for n, st in zip(reversed(shape), reversed(strides)):
        if n > 1 and st != want:
            return 0 in shape
        want *= n
    return True


def _new_rows(shape, dtype, device):
    """A new [B, H, S, D] tensor; rows that are no multiple of 16 bytes are padded to one (a view is returned)."""
    import torch
    over = shape[3] % (16 // dtype.itemsize)
    if over == 0:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty((*shape[:3], shape[3] - over + 16 // dtype.itemsize), dtype=dtype, device=device)[..., :shape[3]]


def _new_strides(shape, dtype):
    """Strides of _new_rows(shape, dtype)."""
    step = 16 // dtype.itemsize
    row = (shape[3] + step - 1) // step * step
    return (shape[1] * shape[2] * row, shape[2] * row, row)


def _pair_axis_bytes(pair_axis, pairs: int, axes: int) -> bytes:
    if pair_axis is None:
        if axes != 1:
            raise ValueError("pair_axis is required with more than one position axis")
        pair_axis = (0,) * pairs
    if not all(isinstance(a, numbers.Integral) for a in pair_axis):
        raise TypeError("pair_axis must hold whole numbers")
    if len(pair_axis) != pairs or any(not 0 <= a < axes for a in pair_axis):
        raise ValueError(f"pair_axis must name one of the {axes} axes for each of the {pairs} pairs")
    return bytes(pair_axis).ljust(128, b"\0")


_NO3 = (0, 0, 0)


def _rope_plan(q, k, freqs, positions, q_weight, k_weight, q_out, k_out, kv_len, v, v_out, pair_axis, interleaved, eps):
    """Checks of a qk_rope call from its tensors' metadata; the packed fixed part of its arguments."""
    import torch
    q_shape, _, dt, dev = q
    code = VT_BF16 if dt == torch.bfloat16 else VT_F32 if dt == torch.float32 else None
    if code is None:
        raise TypeError(f"qk_rope supports bfloat16 and float32 tensors, got {dt}")
    sq = _check("q", q, dev, dt)
    B, H, S, D = q_shape
    _check_vector("freqs", freqs, dev, torch.float32, None)
    pairs = freqs[0][0]
    if not 1 <= pairs <= 128:
        raise ValueError("freqs must have 1 to 128 entries")
    if positions[3] != dev or positions[2] != torch.int32:
        raise TypeError("positions must be int32, on the device of the other tensors")
    p_shape, p_stride = positions[0], positions[1]
    if len(p_shape) not in (2, 3) or tuple(p_shape[-2:]) != (B, S):
        raise ValueError("positions must be [B, S] or [axes, B, S]")
    axes, pos_st = (1, (0, *p_stride)) if len(p_shape) == 2 else (p_shape[0], p_stride)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check_vector(name, w, dev, dt, D)
    sqo = _check("q_out", q_out, dev, dt, q_shape) if q_out is not None else _new_strides(q_shape, dt)
    sk = sko = sv = svo = _NO3
    H_kv = cap = D_v = 0
    if k is not None:
        sk = _check("k", k, dev, dt)
        H_kv = k[0][1]
        if tuple(k[0]) != (B, H_kv, S, D):
            raise ValueError("shape mismatch between q and k")
    if kv_len is not None:
        if k is None or k_out is None or (v is None) != (v_out is None):
            raise ValueError("an append needs k and its cache k_out, and v only with its cache v_out")
        _check_vector("kv_len", kv_len, dev, torch.int32, B)
        cap = k_out[0][2] if len(k_out[0]) == 4 else 0
        sko = _check("k_out", k_out, dev, dt, (B, H_kv, cap, D))
        if v is not None:
            D_v = v[0][3] if len(v[0]) == 4 else 0
            sv = _check("v", v, dev, dt, (B, H_kv, S, D_v))
            svo = _check("v_out", v_out, dev, dt, (B, H_kv, cap, D_v))
    elif v is not None or v_out is not None:
        raise ValueError("v is appended with kv_len only")
    elif k is not None:
        sko = _check("k_out", k_out, dev, dt, k[0]) if k_out is not None else _new_strides(k[0], dt)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    return _QK_ROPE_REST.pack(B, H, H_kv, S, D, 2 * pairs, cap, D_v, code, interleaved, eps is not None, axes,
                              eps or 0.0, 0, *sq, *sk, *sqo, *sko, *sv, *svo, *pos_st,
                              _pair_axis_bytes(pair_axis, pairs, axes))


def qk_rope(q, k, freqs, positions, *, pair_axis=None, interleaved: bool = False, eps: float | None = None,
            q_weight=None, k_weight=None, q_out=None, k_out=None, kv_len=None, v=None, v_out=None, stream=None):
    """Norm (with ``eps``) and rotation of the rows of q [B,H,S,D] and k [B,H_kv,S,D] (or None) in one pass: see
    vt_qk_rope_fwd in include/vt_attn.h.  Returns (q_out, k_out).

    ``freqs`` (float32) holds the angle per position of each of the R/2 rotated pairs, ``positions`` (int32) is
    [B,S] or [axes,B,S], and ``pair_axis`` (a tuple) names the axis of every pair.  ``eps=None`` leaves the norm out.
    ``q_out=q`` and ``k_out=k`` work in place.  With ``kv_len`` (int32 [B]: the lengths after these tokens), k_out
    is a cache [B,H_kv,cap,D] that K's rows are appended to, and v [B,H_kv,S,D_v] is appended to v_out.
    ``stream`` may name another stream than the current one (a torch stream or a raw handle).  Nothing is recorded for
    autograd: the results are detached, and ``qk_rope_bwd`` gives the gradients."""
    if stream is not None or not _here(q):
        return _elsewhere(qk_rope, q, stream, (q, k, freqs, positions), dict(
            pair_axis=pair_axis, interleaved=interleaved, eps=eps, q_weight=q_weight, k_weight=k_weight, q_out=q_out,
            k_out=k_out, kv_len=kv_len, v=v, v_out=v_out))
    import torch
    if pair_axis is not None and type(pair_axis) is not tuple:
        pair_axis = tuple(pair_axis)
    if eps is not None and type(eps) is not float:
        eps = float(eps)  # (a plan is kept by values: a tensor's may change)
    key = ((q.shape, q.stride(), q.dtype, q.get_device()),
           None if k is None else (k.shape, k.stride(), k.dtype, k.get_device()),
           (freqs.shape, freqs.stride(), freqs.dtype, freqs.get_device()),
           (positions.shape, positions.stride(), positions.dtype, positions.get_device()),
           None if q_weight is None else (q_weight.shape, q_weight.stride(), q_weight.dtype, q_weight.get_device()),
           None if k_weight is None else (k_weight.shape, k_weight.stride(), k_weight.dtype, k_weight.get_device()),
           None if q_out is None else (q_out.shape, q_out.stride(), q_out.dtype, q_out.get_device()),
           None if k_out is None else (k_out.shape, k_out.stride(), k_out.dtype, k_out.get_device()),
           None if kv_len is None else (kv_len.shape, kv_len.stride(), kv_len.dtype, kv_len.get_device()),
           None if v is None else (v.shape, v.stride(), v.dtype, v.get_device()),
           None if v_out is None else (v_out.shape, v_out.stride(), v_out.dtype, v_out.get_device()),
           pair_axis, bool(interleaved), eps)
    rest = _rope_plans.get(key)
    if rest is None:
        rest = _keep(_rope_plans, key, _rope_plan(*key))
    if q_out is None:
        q_out = _new_rows(q.shape, q.dtype, q.device)
    if k_out is None and k is not None:
        k_out = _new_rows(k.shape, q.dtype, q.device)
    args = _QK_ROPE_PTRS.pack(_QK_ROPE_BYTES, q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), freqs.data_ptr(),
                              positions.data_ptr(), q_out.data_ptr(), _ptr(k_out), _ptr(kv_len), _ptr(v),
                              _ptr(v_out)) + rest
    rc = load().vt_qk_rope_fwd(args, torch._C._cuda_getCurrentRawStream(q.get_device()))
    if rc != 0:
        raise VtError(rc, "vt_qk_rope_fwd")
    return q_out, k_out


def _rope_bwd_plan(gq, gk, freqs, positions, q, k, q_weight, k_weight, dq, dk, pair_axis, interleaved, eps):
    """Checks of a qk_rope_bwd call from its tensors' metadata: (packed fixed part of its arguments, strides of dq_out,
    strides of dk_out)."""
    if eps is not None and (q is None or (k is None) != (gk is None)):
        raise ValueError("the norm's gradients need the forward's inputs q and k")
    # the forward's fields, with dq and dk for its outputs
    x, y = (q, k) if eps is not None else (gq, gk)
    if q is not None and tuple(q[0]) != tuple(gq[0]) or k is not None and (gk is None or tuple(k[0]) != tuple(gk[0])):
        raise ValueError("q and k must have the shapes of dq_out and dk_out")
    rest = _rope_plan(x, y, freqs, positions, q_weight, k_weight, dq, dk, None, None, None, pair_axis, interleaved, eps)
    dt, dev = x[2], x[3]
    sgq = _check("dq_out", gq, dev, dt)
    sgk = _check("dk_out", gk, dev, dt) if gk is not None else None
    c3 = ctypes.c_int64 * 3
    return rest, c3(*sgq), c3(*sgk) if sgk is not None else None


def qk_rope_bwd(dq_out, dk_out, freqs, positions, *, q=None, k=None, pair_axis=None, interleaved: bool = False,
                eps: float | None = None, q_weight=None, k_weight=None, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of ``qk_rope`` (without the append): see vt_qk_rope_bwd in include/vt_attn.h.  dq_out, dk_out are
    the gradients of its outputs; q, k its inputs (needed with ``eps``).  Returns (dq, dk, dq_weight, dk_weight); the
    weights' gradients are float32 [D], and None without ``eps`` (or, for K's, without dk_out).  ``dq=dq_out`` and
    ``dk=dk_out`` work in place.  ``workspace`` may be a preallocated uint8 CUDA tensor of at least
    ``vt_qk_rope_bwd_workspace_size`` bytes, ``stream`` another stream than the current one."""
    if stream is not None or not _here(dq_out):
        return _elsewhere(qk_rope_bwd, dq_out, stream, (dq_out, dk_out, freqs, positions), dict(
            q=q, k=k, pair_axis=pair_axis, interleaved=interleaved, eps=eps, q_weight=q_weight, k_weight=k_weight,
            dq=dq, dk=dk, workspace=workspace))
    import torch
    if pair_axis is not None and type(pair_axis) is not tuple:
        pair_axis = tuple(pair_axis)
    if eps is not None and type(eps) is not float:
        eps = float(eps)  # (a plan is kept by values: a tensor's may change)
    key = ((dq_out.shape, dq_out.stride(), dq_out.dtype, dq_out.get_device()),
           None if dk_out is None else (dk_out.shape, dk_out.stride(), dk_out.dtype, dk_out.get_device()),
           (freqs.shape, freqs.stride(), freqs.dtype, freqs.get_device()),
           (positions.shape, positions.stride(), positions.dtype, positions.get_device()),
           None if q is None else (q.shape, q.stride(), q.dtype, q.get_device()),
           None if k is None else (k.shape, k.stride(), k.dtype, k.get_device()),
           None if q_weight is None else (q_weight.shape, q_weight.stride(), q_weight.dtype, q_weight.get_device()),
           None if k_weight is None else (k_weight.shape, k_weight.stride(), k_weight.dtype, k_weight.get_device()),
           None if dq is None else (dq.shape, dq.stride(), dq.dtype, dq.get_device()),
           None if dk is None else (dk.shape, dk.stride(), dk.dtype, dk.get_device()),
           pair_axis, bool(interleaved), eps)
    plan = _rope_bwd_plans.get(key)
    if plan is None:
        plan = _keep(_rope_bwd_plans, key, _rope_bwd_plan(*key))
    rest, sgq, sgk = plan
    dt, dev = dq_out.dtype, dq_out.device
    if dq is None:
        dq = _new_rows(dq_out.shape, dt, dev)
    if dk is None and dk_out is not None:
        dk = _new_rows(dk_out.shape, dt, dev)
    dqw = dkw = None
    ws_bytes = 0
    lib = load()
    if eps is not None:
        D = dq_out.shape[3]
        dqw = torch.empty(D, dtype=torch.float32, device=dev)
        if dk_out is not None:
            dkw = torch.empty(D, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(lib.vt_qk_rope_bwd_workspace_size(D), dtype=torch.uint8, device=dev)
        ws_bytes = _workspace_bytes(workspace, dq_out)
    args = _QK_ROPE_PTRS.pack(_QK_ROPE_BYTES, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), freqs.data_ptr(),
                              positions.data_ptr(), dq.data_ptr(), _ptr(dk), 0, 0, 0) + rest
    rc = lib.vt_qk_rope_bwd(args, dq_out.data_ptr(), sgq, _ptr(dk_out), sgk, _ptr(dqw), _ptr(dkw), _ptr(workspace),
                            ws_bytes, torch._C._cuda_getCurrentRawStream(dq_out.get_device()))
    if rc != 0:
        raise VtError(rc, "vt_qk_rope_bwd")
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- attention behind a shared prefix

def _prefix_plan(q, k_prefix, v_prefix, k_cache, v_cache, parents, kv_len, out, lse, scale):
    """Checks of an attn_fwd_prefix or attn_fwd_tree call from its tensors' metadata: (packed fixed part of its arguments, shape of O,
    bytes of workspace)."""
    import torch
    q_shape, _, dt, dev = q
    code = VT_BF16 if dt == torch.bfloat16 else VT_F32 if dt == torch.float32 else None
    if code is None:
        raise TypeError(f"attn_fwd_prefix supports bfloat16 and float32 tensors, got {dt}")
    if (k_prefix is None) != (v_prefix is None) or (k_cache is None) != (v_cache is None):
        raise ValueError("K and V of the prefix, and of the cache, come together")
    if k_prefix is None and k_cache is None:
        raise ValueError("a prefix or a cache is required")
    sq = _check("q", q, dev, dt)
    B, H, S_q, D_qk = q_shape
    some_k, some_v = (k_prefix, v_prefix) if k_prefix is not None else (k_cache, v_cache)
    if len(some_k[0]) < 3 or len(some_v[0]) < 3:
        raise ValueError("the prefix is [H_kv, S, D] and the cache [B, H_kv, S, D]")
    H_kv, D_v = some_k[0][-3], some_v[0][-1]
    S_p = S_c = 0
    skp = svp = (0, 0)
    skc = svc = _NO3
    if k_prefix is not None:
        S_p = k_prefix[0][-2]
        skp = _check("k_prefix", k_prefix, dev, dt, (H_kv, S_p, D_qk), 3)
        svp = _check("v_prefix", v_prefix, dev, dt, (H_kv, S_p, D_v), 3)
    if k_cache is not None:
        S_c = k_cache[0][-2]
        skc = _check("k_cache", k_cache, dev, dt, (B, H_kv, S_c, D_qk))
        svc = _check("v_cache", v_cache, dev, dt, (B, H_kv, S_c, D_v))
    if kv_len is not None:
        _check_vector("kv_len", kv_len, dev, torch.int32, B)
    if parents is not None and (parents[3] != dev or parents[2] != torch.int32 or tuple(parents[0]) != (B, S_q)
                                or not _contiguous(*parents[:2])):
        raise ValueError("parents must be a contiguous int32 [B, S_q] tensor on the device of the other tensors")
    o_shape = (B, H, S_q, D_v)
    so = _check("out", out, dev, dt, o_shape) if out is not None else _new_strides(o_shape, dt)
    if lse is not None and (lse[3] != dev or lse[2] != torch.float32 or tuple(lse[0]) != (B, H, S_q)
                            or not _contiguous(*lse[:2])):
        raise ValueError("lse must be a contiguous float32 [B, H, S_q] tensor on the device of the other tensors")
    if scale is None:
        scale = float(D_qk) ** -0.5
    size = vt_attn_prefix_workspace_size if parents is None else vt_attn_tree_workspace_size
    need = size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, code)
    rest = _ATTN_PREFIX_REST.pack(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, code, scale, *sq, *skp, *svp, *skc, *svc, *so)
    return rest, o_shape, need


def attn_fwd_prefix(q, k_prefix, v_prefix, k_cache, v_cache, kv_len=None, *, scale: float | None = None,
                    return_lse: bool = False, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [B,H,S_q,D_qk] over a prefix that all sequences share, k_prefix [H_kv,S_p,D_qk] and v_prefix
    [H_kv,S_p,D_v], and over each sequence's own cache, k_cache [B,H_kv,S_c,D_qk] and v_cache [B,H_kv,S_c,D_v], up to
    its length kv_len (int32 [B], counting these S_q tokens; None: S_c): see vt_attn_fwd_prefix in include/vt_attn.h.
    Prefix or cache may be None.  Returns O, or (O, LSE) with ``return_lse``.  ``workspace`` may be a preallocated
    uint8 CUDA tensor of at least ``vt_attn_prefix_workspace_size`` bytes, ``stream`` another stream than the
    current one."""
    return _prefix_call(q, k_prefix, v_prefix, k_cache, v_cache, None, kv_len, scale, return_lse, out, lse, workspace,
                        stream)


def attn_fwd_tree(q, k_prefix, v_prefix, k_cache, v_cache, parents, kv_len=None, *, scale: float | None = None,
                  return_lse: bool = False, out=None, lse=None, workspace=None, stream=None):
    """``attn_fwd_prefix`` for trees of drafted tokens: the S_q <= 64 tokens of each sequence that its last cache rows hold
    are nodes, and parents (int32 [B,S_q], contiguous, on the device) names the earlier node that each continues, or -1.
    A node sees the prefix, the cache before the tree, its ancestors and itself: see vt_attn_fwd_tree in
    include/vt_attn.h.  The other arguments are those of ``attn_fwd_prefix``; a given ``workspace`` has
    ``vt_attn_tree_workspace_size`` bytes."""
    if parents is None:
        raise ValueError("parents is required")
    return _prefix_call(q, k_prefix, v_prefix, k_cache, v_cache, parents, kv_len, scale, return_lse, out, lse, workspace,
                        stream)


def _prefix_call(q, k_prefix, v_prefix, k_cache, v_cache, parents, kv_len, scale, return_lse, out, lse, workspace, stream):
    if stream is not None or not _here(q):
        return _elsewhere(_prefix_call, q, stream, (q, k_prefix, v_prefix, k_cache, v_cache, parents, kv_len, scale,
                                                    return_lse, out, lse, workspace, None), {})
    import torch
    if scale is not None and type(scale) is not float:
        scale = float(scale)  # (a plan is kept by values: a tensor's may change)
    key = ((q.shape, q.stride(), q.dtype, q.get_device()),
           None if k_prefix is None else (k_prefix.shape, k_prefix.stride(), k_prefix.dtype, k_prefix.get_device()),
           None if v_prefix is None else (v_prefix.shape, v_prefix.stride(), v_prefix.dtype, v_prefix.get_device()),
           None if k_cache is None else (k_cache.shape, k_cache.stride(), k_cache.dtype, k_cache.get_device()),
           None if v_cache is None else (v_cache.shape, v_cache.stride(), v_cache.dtype, v_cache.get_device()),
           None if parents is None else (parents.shape, parents.stride(), parents.dtype, parents.get_device()),
           None if kv_len is None else (kv_len.shape, kv_len.stride(), kv_len.dtype, kv_len.get_device()),
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()),
           None if lse is None else (lse.shape, lse.stride(), lse.dtype, lse.get_device()),
           scale)
    plan = _prefix_plans.get(key)
    if plan is None:
        plan = _keep(_prefix_plans, key, _prefix_plan(*key))
    rest, o_shape, need = plan
    dev = q.device
    if out is None:
        out = _new_rows(o_shape, q.dtype, dev)
    if return_lse and lse is None:
        lse = torch.empty(o_shape[:3], dtype=torch.float32, device=dev)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    args = _ATTN_PREFIX_PTRS.pack(_ATTN_PREFIX_BYTES, q.data_ptr(), _ptr(k_prefix), _ptr(v_prefix), _ptr(k_cache),
                                  _ptr(v_cache), _ptr(kv_len), out.data_ptr(), _ptr(lse), _ptr(workspace),
                                  _workspace_bytes(workspace, q)) + rest
    raw = torch._C._cuda_getCurrentRawStream(q.get_device())
    rc = load().vt_attn_fwd_prefix(args, raw) if parents is None else load().vt_attn_fwd_tree(args, parents.data_ptr(), raw)
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd_prefix" if parents is None else "vt_attn_fwd_tree")
    return (out, lse) if return_lse else out


def attn_prefix_step(q, k, v, freqs, positions, k_prefix, v_prefix, k_cache, v_cache, kv_len, *, pair_axis=None,
                     interleaved: bool = False, eps: float | None = None, q_weight=None, k_weight=None,
                     scale: float | None = None, return_lse: bool = False, out=None, lse=None, workspace=None,
                     stream=None):
    """One step of a batch behind a shared prefix, from the projections of its new tokens: norm and rotate q and k,
    append k and v to the caches at the end of each sequence (``kv_len`` counts the new tokens already), and attend
    to the prefix and to the caches.  ``qk_rope`` and ``attn_fwd_prefix`` in one call, with their arguments; q and k
    are left as they are."""
    q_rot, _ = qk_rope(q, k, freqs, positions, pair_axis=pair_axis, interleaved=interleaved, eps=eps,
                       q_weight=q_weight, k_weight=k_weight, k_out=k_cache, kv_len=kv_len, v=v, v_out=v_cache,
                       stream=stream)
    return attn_fwd_prefix(q_rot, k_prefix, v_prefix, k_cache, v_cache, kv_len, scale=scale, return_lse=return_lse,
                           out=out, lse=lse, workspace=workspace, stream=stream)


# ---------------------------------------------------------------- attention over packed sequences

def _new_tokens(shape, dtype, device):
    """A new [H, T, D] tensor, token by token in memory ([T, H, D], as projections leave and take rows); rows that are no
    multiple of 16 bytes are padded to one (a view is returned)."""
    import torch
    H, T, D = shape
    row, token = _new_token_strides(shape, dtype)
    return torch.empty_strided((H, T, D), (row, token, 1), dtype=dtype, device=device)


def _new_token_strides(shape, dtype):
    """Strides of _new_tokens(shape, dtype)."""
    step = 16 // dtype.itemsize
    row = (shape[2] + step - 1) // step * step
    return (row, shape[0] * row)


def _check_lse(name, meta, dev, shape):
    if meta[3] != dev or meta[2] != _float32() or tuple(meta[0]) != shape or not _contiguous(*meta[:2]):
        raise ValueError(f"{name} must be a contiguous float32 [H, T_q] tensor on the device of the other tensors")


def _float32():
    import torch
    return torch.float32


def _packed_plan(q, k, v, cu_q, cu_k, out, lse, scale, mask, window):
    """Checks of an attn_fwd_packed call from its tensors' metadata: (packed fixed part of its arguments, shape of O)."""
    import torch
    q_shape, _, dt, dev = q
    code = VT_BF16 if dt == torch.bfloat16 else VT_F32 if dt == torch.float32 else None
    if code is None:
        raise TypeError(f"attention over packed sequences supports bfloat16 and float32 tensors, got {dt}")
    sq = _check("q", q, dev, dt, dims=3)
    H, T_q, D_qk = q_shape
    if len(k[0]) != 3 or len(v[0]) != 3:
        raise ValueError("k and v must have 3 dimensions")
    H_kv, T_k, D_v = k[0][0], k[0][1], v[0][2]
    sk = _check("k", k, dev, dt, (H_kv, T_k, D_qk), 3)
    sv = _check("v", v, dev, dt, (H_kv, T_k, D_v), 3)
    _check_vector("cu_q", cu_q, dev, torch.int32, None)
    N = cu_q[0][0] - 1
    if N < 0:
        raise ValueError("cu_q must hold the first row of every sequence and the end of the last")
    _check_vector("cu_k", cu_k, dev, torch.int32, N + 1)
    o_shape = (H, T_q, D_v)
    so = _check("out", out, dev, dt, o_shape, 3) if out is not None else _new_token_strides(o_shape, dt)
    if lse is not None:
        _check_lse("lse", lse, dev, (H, T_q))
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {tuple(MASKS)}")
    if scale is None:
        scale = float(D_qk) ** -0.5
    rest = _ATTN_PACKED_REST.pack(N, H, H_kv, T_q, T_k, D_qk, D_v, window, code, scale, MASKS[mask], 0, *sq, *sk, *sv, *so)
    return rest, o_shape


def attn_fwd_packed(q, k, v, cu_q, cu_k=None, *, scale: float | None = None, mask: str = "causal", window: int = 0,
                    return_lse: bool = False, out=None, lse=None, stream=None):
    """Attention of sequences of different lengths that lie behind each other: q [H,T_q,D_qk], k [H_kv,T_k,D_qk] and
    v [H_kv,T_k,D_v], with sequence n's queries in rows cu_q[n] to cu_q[n + 1] and its keys in rows cu_k[n] to cu_k[n + 1]
    (int32 [N + 1] on the device; cu_k may be left out where it is cu_q): see vt_attn_fwd_packed in include/vt_attn.h.
    The queries are the last of their sequence's positions; ``mask`` is one of ``MASKS`` with ``window``.

    Returns O [H,T_q,D_v], or (O, LSE) with ``return_lse`` (float32 [H,T_q], natural log).  Rows of no sequence are not
    written.  A new O lies token by token ([T_q,H,D_v] in memory).  ``stream`` may name another stream than the current
    one.  Nothing is recorded for autograd; ``attn_bwd_packed`` gives the gradients."""
    if stream is not None or not _here(q):
        return _elsewhere(attn_fwd_packed, q, stream, (q, k, v, cu_q, cu_k), dict(
            scale=scale, mask=mask, window=window, return_lse=return_lse, out=out, lse=lse))
    import torch
    if cu_k is None:
        cu_k = cu_q
    if scale is not None and type(scale) is not float:
        scale = float(scale)  # (a plan is kept by values: a tensor's may change)
    if type(window) is not int:
        window = int(window)
    key = ((q.shape, q.stride(), q.dtype, q.get_device()), (k.shape, k.stride(), k.dtype, k.get_device()),
           (v.shape, v.stride(), v.dtype, v.get_device()), (cu_q.shape, cu_q.stride(), cu_q.dtype, cu_q.get_device()),
           (cu_k.shape, cu_k.stride(), cu_k.dtype, cu_k.get_device()),
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()),
           None if lse is None else (lse.shape, lse.stride(), lse.dtype, lse.get_device()), scale, mask, window)
    plan = _packed_plans.get(key)
    if plan is None:
        plan = _keep(_packed_plans, key, _packed_plan(*key))
    rest, o_shape = plan
    if out is None:
        out = _new_tokens(o_shape, q.dtype, q.device)
    if return_lse and lse is None:
        lse = torch.empty(o_shape[:2], dtype=torch.float32, device=q.device)
    args = _ATTN_PACKED_PTRS.pack(_ATTN_PACKED_BYTES, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
                                  cu_k.data_ptr(), out.data_ptr(), _ptr(lse)) + rest
    rc = load().vt_attn_fwd_packed(args, torch._C._cuda_getCurrentRawStream(q.get_device()))
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd_packed")
    return (out, lse) if return_lse else out


def _packed_bwd_plan(do, q, k, v, cu_q, cu_k, o, lse, dlse, dq, dk, dv, scale, mask, window):
    """Checks of an attn_bwd_packed call from its tensors' metadata: (packed fixed parts of its two structs, bytes of
    workspace)."""
    if lse is None:
        raise ValueError("lse must be the forward's")
    rest, o_shape = _packed_plan(q, k, v, cu_q, cu_k, o, lse, scale, mask, window)
    dt, dev = q[2], q[3]
    if dlse is not None:
        _check_lse("dlse", dlse, dev, tuple(o_shape[:2]))
    strides = [_check("do", do, dev, dt, o_shape, 3)]
    for name, meta, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        strides.append(_check(name, meta, dev, dt, like[0], 3) if meta is not None else _new_token_strides(like[0], dt))
    H, T_q, D_qk = q[0]
    H_kv, T_k, D_v = v[0]
    need = vt_attn_bwd_packed_workspace_size(cu_q[0][0] - 1, H, H_kv, T_q, T_k, D_qk, D_v,
                                             VT_BF16 if dt.itemsize == 2 else VT_F32)
    return rest, _PACKED_GRADS_REST.pack(*(x for st in strides for x in st)), need


def attn_bwd_packed(do, q, k, v, o, lse, cu_q, cu_k=None, *, scale: float | None = None, mask: str = "causal",
                    window: int = 0, dlse=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of ``attn_fwd_packed``: see vt_attn_bwd_packed in include/vt_attn.h.  ``do`` [H,T_q,D_v] is the gradient
    of O (and ``dlse``, float32 [H,T_q], that of LSE), ``o`` and ``lse`` are the forward's results and the other arguments
    its own.  Returns (dq, dk, dv); new ones lie token by token, and given ones may lie beside each other in one tensor.
    ``workspace`` may be a preallocated uint8 CUDA tensor of at least ``vt_attn_bwd_packed_workspace_size`` bytes,
    ``stream`` another stream than the current one."""
    if stream is not None or not _here(q):
        return _elsewhere(attn_bwd_packed, q, stream, (do, q, k, v, o, lse, cu_q, cu_k), dict(
            scale=scale, mask=mask, window=window, dlse=dlse, dq=dq, dk=dk, dv=dv, workspace=workspace))
    import torch
    if cu_k is None:
        cu_k = cu_q
    if scale is not None and type(scale) is not float:
        scale = float(scale)  # (a plan is kept by values: a tensor's may change)
    if type(window) is not int:
        window = int(window)
    key = ((do.shape, do.stride(), do.dtype, do.get_device()), (q.shape, q.stride(), q.dtype, q.get_device()),
           (k.shape, k.stride(), k.dtype, k.get_device()), (v.shape, v.stride(), v.dtype, v.get_device()),
           (cu_q.shape, cu_q.stride(), cu_q.dtype, cu_q.get_device()),
           (cu_k.shape, cu_k.stride(), cu_k.dtype, cu_k.get_device()), (o.shape, o.stride(), o.dtype, o.get_device()),
           None if lse is None else (lse.shape, lse.stride(), lse.dtype, lse.get_device()),
           None if dlse is None else (dlse.shape, dlse.stride(), dlse.dtype, dlse.get_device()),
           None if dq is None else (dq.shape, dq.stride(), dq.dtype, dq.get_device()),
           None if dk is None else (dk.shape, dk.stride(), dk.dtype, dk.get_device()),
           None if dv is None else (dv.shape, dv.stride(), dv.dtype, dv.get_device()), scale, mask, window)
    plan = _packed_bwd_plans.get(key)
    if plan is None:
        plan = _keep(_packed_bwd_plans, key, _packed_bwd_plan(*key))
    rest, grads_rest, need = plan
    dev = q.device
    if dq is None:
        dq = _new_tokens(q.shape, q.dtype, dev)
    if dk is None:
        dk = _new_tokens(k.shape, q.dtype, dev)
    if dv is None:
        dv = _new_tokens(v.shape, q.dtype, dev)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    args = _ATTN_PACKED_PTRS.pack(_ATTN_PACKED_BYTES, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
                                  cu_k.data_ptr(), o.data_ptr(), lse.data_ptr()) + rest
    grads = _PACKED_GRADS_PTRS.pack(_PACKED_GRADS_BYTES, do.data_ptr(), _ptr(dlse), dq.data_ptr(), dk.data_ptr(),
                                    dv.data_ptr(), _ptr(workspace), _workspace_bytes(workspace, q)) + grads_rest
    rc = load().vt_attn_bwd_packed(args, grads, torch._C._cuda_getCurrentRawStream(q.get_device()))
    if rc != 0:
        raise VtError(rc, "vt_attn_bwd_packed")
    return dq, dk, dv
