"""Python binding of the vt_attn C ABI (include/vt_attn.h): argument marshalling only.

Every step of the attention forward runs in the CUDA kernels of ``libvt_attn.so``;
this module only converts arguments and calls the C entry points through ctypes.
There is no fallback: if the library is missing or cannot be loaded, every call
raises.  PyTorch is used for device memory and the current stream.
"""

from __future__ import annotations

import ctypes
import functools
import os
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
           "vt_attn_fwd_prefix", "vt_attn_prefix_workspace_size",
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
    lib.vt_attn_prefix_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64, i64, i64, i]
    lib.vt_attn_prefix_workspace_size.restype = sz
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


# vt_qk_rope_args, packed in field order (every field is aligned without padding)
_QK_ROPE_ARGS = struct.Struct("=Q6q4ifi2Q6q2QQQ3q2Q6qQ2q2Q6q128s")


def vt_qk_rope_fwd(args: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_qk_rope_args; returns the vt_status code."""
    return load().vt_qk_rope_fwd(args, stream)


def vt_qk_rope_bwd(args: bytes, dq_out, dq_out_stride, dk_out, dk_out_stride, dq_weight, dk_weight, workspace,
                   workspace_bytes, stream) -> int:
    return load().vt_qk_rope_bwd(args, dq_out, _stride3(dq_out_stride), dk_out, _stride3(dk_out_stride), dq_weight,
                                 dk_weight, workspace, int(workspace_bytes), stream)


def vt_qk_rope_bwd_workspace_size(D) -> int:
    return int(load().vt_qk_rope_bwd_workspace_size(D))


# vt_attn_prefix_args, packed in field order (every field is aligned without padding)
_ATTN_PREFIX_ARGS = struct.Struct("=Q8qifQ3q2Q4q2Q6q2Q3q3Q")


def vt_attn_fwd_prefix(args: bytes, stream) -> int:
    """The C entry point: ``args`` is a packed vt_attn_prefix_args; returns the vt_status code."""
    return load().vt_attn_fwd_prefix(args, stream)


def vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype) -> int:
    return int(load().vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, dtype))


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

def _on_stream(fn):
    """Run a wrapper on its ``stream=`` (a torch stream or a raw handle; None: the current stream of the first
    tensor's device).  What the wrapper allocates is then allocated on that stream, and that device is current."""

    @functools.wraps(fn)
    def call(first, *args, stream=None, **kw):
        import torch
        if not first.is_cuda:
            raise ValueError("the tensors must be CUDA tensors")
        dev = first.device
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            with torch.cuda.stream(stream):
                return fn(first, *args, **kw)
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return fn(first, *args, **kw)
        return fn(first, *args, **kw)

    return call


def _same_place(what, first, *tensors):
    """Every tensor given (not None) lives on the first one's device."""
    dev = first.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{what}: all tensors must be on {dev}")


def _bhsd(name, t, shape=None, dtype=None):
    """(address, strides) of a [B, H, S, D] tensor with its last dimension contiguous."""
    if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] != 1):
        raise ValueError(f"{name} must be [B, H, S, D] with the last dimension contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr(), t.stride()[:3]


@functools.lru_cache(maxsize=64)
def _pair_axis_bytes(pair_axis, pairs: int, axes: int) -> bytes:
    if pair_axis is None:
        if axes != 1:
            raise ValueError("pair_axis is required with more than one position axis")
        pair_axis = (0,) * pairs
    if len(pair_axis) != pairs or any(not 0 <= a < axes for a in pair_axis):
        raise ValueError(f"pair_axis must name one of the {axes} axes for each of the {pairs} pairs")
    return bytes(pair_axis).ljust(128, b"\0")


def _rope_form(q, k, freqs, positions, pair_axis, q_weight, k_weight):
    """The fields the two directions share: (dims, weights, freqs and positions, pair axes)."""
    import torch
    B, H, S, D = q.shape
    if k is not None and (k.dim() != 4 or k.shape[0] != B or k.shape[2] != S or k.shape[3] != D):
        raise ValueError("shape mismatch between q and k")
    if freqs.dtype != torch.float32 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float32 vector")
    pairs = freqs.shape[0]
    if not 1 <= pairs <= 128:
        raise ValueError("freqs must have 1 to 128 entries")
    if positions.dtype != torch.int32:
        raise TypeError(f"positions must be int32, got {positions.dtype}")
    if positions.dim() == 2:
        axes, pos_stride = 1, (0, *positions.stride())
    elif positions.dim() == 3:
        axes, pos_stride = positions.shape[0], positions.stride()
    else:
        raise ValueError("positions must be [B, S] or [axes, B, S]")
    if positions.shape[-2:] != (B, S):
        raise ValueError("positions must be [B, S] or [axes, B, S]")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != q.dtype or w.shape != (D,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous vector of {D} elements of q's dtype")
    if pair_axis is not None and not isinstance(pair_axis, tuple):
        pair_axis = tuple(pair_axis)
    return (B, H, k.shape[1] if k is not None else 0, S, D, 2 * pairs, axes,
            q_weight.data_ptr() if q_weight is not None else 0, k_weight.data_ptr() if k_weight is not None else 0,
            freqs.data_ptr(), positions.data_ptr(), pos_stride, _pair_axis_bytes(pair_axis, pairs, axes))


_NO_TENSOR = (0, (0, 0, 0))


def _new_rows(B, H, S, D, dtype, device):
    """A new [B, H, S, D] tensor; rows that are no multiple of 16 bytes are padded to one (a view is returned)."""
    import torch
    step = 16 // dtype.itemsize
    if D % step == 0:
        return torch.empty((B, H, S, D), dtype=dtype, device=device)
    return torch.empty((B, H, S, D + -D % step), dtype=dtype, device=device)[..., :D]


@_on_stream
def qk_rope(q, k, freqs, positions, *, pair_axis=None, interleaved: bool = False, eps: float | None = None,
            q_weight=None, k_weight=None, q_out=None, k_out=None, kv_len=None, v=None, v_out=None):
    """Norm (with ``eps``) and rotation of the rows of q [B,H,S,D] and k [B,H_kv,S,D] (or None) in one pass: see
    vt_qk_rope_fwd in include/vt_attn.h.  Returns (q_out, k_out).

    ``freqs`` (float32) holds the angle per position of each of the R/2 rotated pairs, ``positions`` (int32) is
    [B,S] or [axes,B,S], and ``pair_axis`` names the axis of every pair.  ``eps=None`` leaves the norm out.
    ``q_out=q`` and ``k_out=k`` work in place.  With ``kv_len`` (int32 [B]: the lengths after these tokens), k_out
    is a cache [B,H_kv,cap,D] that K's rows are appended to, and v [B,H_kv,S,D_v] is appended to v_out.
    ``stream`` may name another stream than the current one."""
    import torch
    (B, H, H_kv, S, D, R, axes, qw, kw, fr, pos, pos_st, axis) = _rope_form(q, k, freqs, positions, pair_axis,
                                                                           q_weight, k_weight)
    code = _dtype_code(q)
    _same_place("qk_rope", q, k, freqs, positions, q_weight, k_weight, q_out, k_out, kv_len, v, v_out)
    if q_out is None:
        q_out = _new_rows(B, H, S, D, q.dtype, q.device)
    pq, sq = _bhsd("q", q)
    pqo, sqo = _bhsd("q_out", q_out, q.shape, q.dtype)
    (pk, sk), (pko, sko), (pv, sv), (pvo, svo) = _NO_TENSOR, _NO_TENSOR, _NO_TENSOR, _NO_TENSOR
    lens, cap, D_v = 0, 0, 0
    if kv_len is not None:
        if k is None or k_out is None or (v is None) != (v_out is None):
            raise ValueError("an append needs k and its cache k_out, and v only with its cache v_out")
        if kv_len.dtype != torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
            raise ValueError("kv_len must be a contiguous int32 vector of B entries")
        lens, cap = kv_len.data_ptr(), k_out.shape[2]
        pko, sko = _bhsd("k_out", k_out, (B, H_kv, cap, D), q.dtype)
        if v is not None:
            D_v = v.shape[3]
            pv, sv = _bhsd("v", v, (B, H_kv, S, D_v), q.dtype)
            pvo, svo = _bhsd("v_out", v_out, (B, H_kv, cap, D_v), q.dtype)
    elif v is not None or v_out is not None:
        raise ValueError("v is appended with kv_len only")
    elif k is not None:
        if k_out is None:
            k_out = _new_rows(B, H_kv, S, D, q.dtype, q.device)
        pko, sko = _bhsd("k_out", k_out, k.shape, q.dtype)
    if k is not None:
        pk, sk = _bhsd("k", k, None, q.dtype)
    args = _QK_ROPE_ARGS.pack(_QK_ROPE_ARGS.size, B, H, H_kv, S, D, R, code, bool(interleaved), eps is not None, axes,
                              eps or 0.0, 0, pq, pk, *sq, *sk, qw, kw, fr, pos, *pos_st, pqo, pko, *sqo, *sko, lens,
                              cap, D_v, pv, pvo, *sv, *svo, axis)
    rc = load().vt_qk_rope_fwd(args, torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise VtError(rc, "vt_qk_rope_fwd")
    return q_out, k_out


@_on_stream
def qk_rope_bwd(dq_out, dk_out, freqs, positions, *, q=None, k=None, pair_axis=None, interleaved: bool = False,
                eps: float | None = None, q_weight=None, k_weight=None, dq=None, dk=None, workspace=None):
    """Gradients of ``qk_rope`` (without the append): see vt_qk_rope_bwd in include/vt_attn.h.  dq_out, dk_out are
    the gradients of its outputs; q, k its inputs (needed with ``eps``).  Returns (dq, dk, dq_weight, dk_weight); the
    weights' gradients are float32 [D], and None without ``eps`` (or, for K's, without dk_out).  ``dq=dq_out`` and
    ``dk=dk_out`` work in place."""
    import torch
    (B, H, H_kv, S, D, R, axes, qw, kw, fr, pos, pos_st, axis) = _rope_form(dq_out, dk_out, freqs, positions, pair_axis,
                                                                           q_weight, k_weight)
    code = _dtype_code(dq_out)
    _same_place("qk_rope_bwd", dq_out, dk_out, freqs, positions, q, k, q_weight, k_weight, dq, dk, workspace)
    dt, dev = dq_out.dtype, dq_out.device
    (pq, sq), (pk, sk), (pdk, sdk), (pgk, sgk) = _NO_TENSOR, _NO_TENSOR, _NO_TENSOR, _NO_TENSOR
    if dq is None:
        dq = _new_rows(B, H, S, D, dt, dev)
    pgq, sgq = _bhsd("dq_out", dq_out)
    pdq, sdq = _bhsd("dq", dq, dq_out.shape, dt)
    if dk_out is not None:
        if dk is None:
            dk = _new_rows(B, H_kv, S, D, dt, dev)
        pgk, sgk = _bhsd("dk_out", dk_out, None, dt)
        pdk, sdk = _bhsd("dk", dk, dk_out.shape, dt)
    dqw = dkw = None
    ws_ptr, ws_bytes = None, 0
    if eps is not None:
        if q is None or (k is None) != (dk_out is None):
            raise ValueError("the norm's gradients need the forward's inputs q and k")
        pq, sq = _bhsd("q", q, dq_out.shape, dt)
        dqw = torch.empty(D, dtype=torch.float32, device=dev)
        if k is not None:
            pk, sk = _bhsd("k", k, dk_out.shape, dt)
            dkw = torch.empty(D, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(load().vt_qk_rope_bwd_workspace_size(D), dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    args = _QK_ROPE_ARGS.pack(_QK_ROPE_ARGS.size, B, H, H_kv, S, D, R, code, bool(interleaved), eps is not None, axes,
                              eps or 0.0, 0, pq, pk, *sq, *sk, qw, kw, fr, pos, *pos_st, pdq, pdk, *sdq, *sdk, 0, 0, 0,
                              0, 0, 0, 0, 0, 0, 0, 0, axis)
    rc = vt_qk_rope_bwd(args, pgq, sgq, pgk, sgk, dqw.data_ptr() if dqw is not None else None,
                        dkw.data_ptr() if dkw is not None else None, ws_ptr, ws_bytes,
                        torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise VtError(rc, "vt_qk_rope_bwd")
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- attention behind a shared prefix

def _kv(name, t, H_kv, S, D, dtype):
    """(address, strides) of a prefix tensor [H_kv, S, D] with its last dimension contiguous."""
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] != 1):
        raise ValueError(f"{name} must be [H_kv, S, D] with the last dimension contiguous")
    if t.shape != (H_kv, S, D):
        raise ValueError(f"{name} must have shape {(H_kv, S, D)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr(), t.stride()[:2]


@_on_stream
def attn_fwd_prefix(q, k_prefix, v_prefix, k_cache, v_cache, kv_len=None, *, scale: float | None = None,
                    return_lse: bool = False, out=None, lse=None, workspace=None):
    """Attention of q [B,H,S_q,D_qk] over a prefix that all sequences share, k_prefix [H_kv,S_p,D_qk] and v_prefix
    [H_kv,S_p,D_v], and over each sequence's own cache, k_cache [B,H_kv,S_c,D_qk] and v_cache [B,H_kv,S_c,D_v], up to
    its length kv_len (int32 [B], counting these S_q tokens; None: S_c): see vt_attn_fwd_prefix in include/vt_attn.h.
    Prefix or cache may be None.  Returns O, or (O, LSE) with ``return_lse``.  ``workspace`` may be a preallocated
    uint8 CUDA tensor of at least ``vt_attn_prefix_workspace_size`` bytes; ``stream`` may name another stream than the
    current one."""
    import torch
    B, H, S_q, D_qk = q.shape
    if (k_prefix is None) != (v_prefix is None) or (k_cache is None) != (v_cache is None):
        raise ValueError("K and V of the prefix, and of the cache, come together")
    if k_prefix is None and k_cache is None:
        raise ValueError("a prefix or a cache is required")
    some_k, some_v = (k_prefix, v_prefix) if k_prefix is not None else (k_cache, v_cache)
    H_kv, D_v = some_k.shape[-3], some_v.shape[-1]
    code, dt = _dtype_code(q), q.dtype
    _same_place("attn_fwd_prefix", q, k_prefix, v_prefix, k_cache, v_cache, kv_len, out, lse, workspace)
    if scale is None:
        scale = float(D_qk) ** -0.5
    S_p = S_c = 0
    pkp = pvp = pkc = pvc = lens = plse = 0
    skp = svp = (0, 0)
    skc = svc = (0, 0, 0)
    pq, sq = _bhsd("q", q)
    if k_prefix is not None:
        S_p = k_prefix.shape[1]
        pkp, skp = _kv("k_prefix", k_prefix, H_kv, S_p, D_qk, dt)
        pvp, svp = _kv("v_prefix", v_prefix, H_kv, S_p, D_v, dt)
    if k_cache is not None:
        S_c = k_cache.shape[2]
        pkc, skc = _bhsd("k_cache", k_cache, (B, H_kv, S_c, D_qk), dt)
        pvc, svc = _bhsd("v_cache", v_cache, (B, H_kv, S_c, D_v), dt)
    if kv_len is not None:
        if kv_len.dtype != torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
            raise ValueError("kv_len must be a contiguous int32 vector of B entries")
        lens = kv_len.data_ptr()
    if out is None:
        out = _new_rows(B, H, S_q, D_v, dt, q.device)
    po, so = _bhsd("out", out, (B, H, S_q, D_v), dt)
    if return_lse and lse is None:
        lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    if lse is not None:
        if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != (B, H, S_q):
            raise ValueError("lse must be a contiguous float32 [B, H, S_q] tensor")
        plse = lse.data_ptr()
    lib = load()
    ws_ptr = ws_bytes = 0
    if workspace is None:
        need = lib.vt_attn_prefix_workspace_size(B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, code)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    args = _ATTN_PREFIX_ARGS.pack(_ATTN_PREFIX_ARGS.size, B, H, H_kv, S_q, S_p, S_c, D_qk, D_v, code, scale, pq, *sq,
                                  pkp, pvp, *skp, *svp, pkc, pvc, *skc, *svc, lens, po, *so, plse, ws_ptr, ws_bytes)
    rc = lib.vt_attn_fwd_prefix(args, torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise VtError(rc, "vt_attn_fwd_prefix")
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
