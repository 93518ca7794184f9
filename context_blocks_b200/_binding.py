"""ctypes binding of ``libpa_attn.so`` (the C ABI in ``include/pa_attn.h``).

Argument marshalling only: tensors are checked for dtype, device, layout and
shape, their device pointers and sizes are handed to the C entry points, and
a non-zero status becomes a :class:`PaError`.  Every step of the attention
and the merge runs in the library's CUDA kernels.  There is no fallback: if
the library is missing or does not load, every call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libpa_attn.so")

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_MISALIGNED = -3
PA_ERR_CUDA = -4
PA_ERR_TIMEOUT = -5
PA_ERR_BAD_INPUT = -6
PA_ACCUM_FIRST = 1
PA_ACCUM_FINAL = 2

# (name, restype, argtypes) for every symbol declared in include/pa_attn.h.
_VP, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "pa_attn_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP]),
    "pa_attn_fwd_accum": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _I, _VP]),
    "pa_attn_fwd_fp8": (_I, [_VP, _VP, _VP, _F, _F, _F, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP]),
    "pa_attn_fwd_fp8_dev": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP]),
    "pa_quantize_e4m3": (_I, [_VP, ctypes.c_longlong, _VP, _VP, _VP]),
    "pa_attn_fwd_chunks": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _F, _VP]),
    "pa_attn_merge": (_I, [_VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _VP]),
    "pa_attn_chunks_noalloc": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _F, _VP]),
    "pa_attn_fwd_mod": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _F, _VP, _VP]),
    "pa_attn_shared_prefix": (_I, [_VP] * 8 + [_I] * 7 + [_VP, _F, _F, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_attn_shared_prefix_workspace": (ctypes.c_size_t, [_I] * 7),
    "pa_gate_residual_norm": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP]),
    "pa_residual_diff": (_I, [_VP, _VP, ctypes.c_longlong, _VP, _VP]),
    "pa_status_string": (ctypes.c_char_p, [_I]),
    "pa_last_error": (ctypes.c_char_p, []),
    "pa_poll_device_status": (_I, []),
    "pa_selftest_timeout": (_I, [_I, _VP]),
    "pa_set_wait_limit_ms": (_I, [_I]),
    "pa_version": (_I, []),
}


class ScoreMod(ctypes.Structure):
    """``pa_score_mod`` of include/pa_attn.h."""

    _fields_ = [("softcap", _F), ("causal", _I), ("slopes", _VP), ("prefix_lens", _VP), ("doc_offsets", _VP),
                ("n_docs", _I), ("q_offset", _I)]


class BlockNorm(ctypes.Structure):
    """``pa_block_norm`` of include/pa_attn.h."""

    _fields_ = [("post", _I), ("norm", _I), ("post_weight", _VP), ("norm_weight", _VP), ("gate", _VP), ("scale", _VP),
                ("shift", _VP), ("gate_stride", ctypes.c_longlong), ("scale_stride", ctypes.c_longlong),
                ("shift_stride", ctypes.c_longlong), ("residual_scale", _F), ("eps", _F)]


_Strides12, _Strides10 = ctypes.c_longlong * 12, ctypes.c_longlong * 10
_nullcontext = contextlib.nullcontext()
PA_NORM = {"none": 0, "rms": 1, "layer": 2}


class PaError(RuntimeError):
    """A non-zero status from the C library."""

    def __init__(self, code: int, where: str, detail: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({detail})" if detail else
                         f"{where}: {status_string(code)}")


_lib = None
_lock = threading.Lock()


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load (once) and return the library; raises if it is not built."""
    global _lib
    if path is None and _lib is not None:  # the common case, without the lock
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m context_blocks_b200.build`")
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(code: int) -> str:
    return load_library().pa_status_string(int(code)).decode()


def last_error() -> str:
    return load_library().pa_last_error().decode()


def version() -> int:
    return int(load_library().pa_version())


def _check(rc: int, where: str, check: bool = False) -> None:
    """Raise on a non-zero status.  With ``check`` also wait for the device
    and raise on an error the kernels recorded (a bounded wait that gave up,
    a bad value read on the device): this synchronises, so it is for
    debugging and tests, not for a hot loop."""
    if rc != PA_OK:
        raise PaError(rc, where, last_error())
    if check:
        import torch
        torch.cuda.synchronize()
        code = poll_device_status()
        if code != PA_OK:
            raise PaError(code, where, "reported by the device after the call")


_raw_stream = None  # torch's current-stream handle getter, looked up once


def _stream_handle(stream, device) -> int:
    """cudaStream_t of `stream`, or of torch's current stream on `device`."""
    global _raw_stream
    import torch
    if stream is None:
        if _raw_stream is None:
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", False)
        if _raw_stream:  # the handle alone, without building a Stream object
            index = device.index if isinstance(device, torch.device) else device
            return int(_raw_stream(torch.cuda.current_device() if index is None else int(index)))
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check_bf16(name, t, ndim):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16 (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def attn_fwd(q, k, v, scale: Optional[float] = None, out=None, lse=None, stream=None, check: bool = False):
    """Attention of q [B,H,Nq,d] against one K/V chunk k, v [B,H,Nk,d].

    Returns (o [B,H,Nq,d] bf16, lse [B,H,Nq] fp32, natural log), written into
    ``out`` / ``lse`` when given.  ``scale`` defaults to 1/sqrt(d).
    ``check=True`` synchronises and raises on a device-side error.
    """
    _check_bf16("q", q, 4)
    _check_bf16("k", k, 4)
    _check_bf16("v", v, 4)
    B, H, Nq, d = q.shape
    kB, kH, Nk, kd = k.shape
    if kB != B or kH != H or kd != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse)
    rc = load_library().pa_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                     B, H, Nq, Nk, d, float(scale), _stream_handle(stream, q.device))
    _check(rc, "pa_attn_fwd", check)
    return out, lse


def attn_fwd_accum(q, k, v, o_acc, lse_acc, first: bool = False, final: bool = False, out=None,
                   scale: Optional[float] = None, stream=None, check: bool = False):
    """Fold the attention of q over one more K/V chunk into the running state
    (``pa_attn_fwd_accum``): o_acc [B,H,Nq,d] fp32 and lse_acc [B,H,Nq] fp32,
    updated in place.  ``first`` ignores their incoming contents.  With
    ``final`` the result goes to ``out`` (bf16, allocated when None) instead
    of o_acc, and that tensor is returned; otherwise o_acc is returned.
    Returns (o, lse_acc)."""
    import torch
    _check_bf16("q", q, 4)
    _check_bf16("k", k, 4)
    _check_bf16("v", v, 4)
    B, H, Nq, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    for name, t, shape in (("o_acc", o_acc, (B, H, Nq, d)), ("lse_acc", lse_acc, (B, H, Nq))):
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape
                or not t.is_contiguous() or t.device != q.device):
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on q's device")
    if final:
        if out is None:
            out = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q.device)
        else:
            _check_bf16("out", out, 4)
            if tuple(out.shape) != (B, H, Nq, d):
                raise ValueError("out must have q's shape")
    elif out is not None:
        raise ValueError("out is written only by the final fold")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    flags = (PA_ACCUM_FIRST if first else 0) | (PA_ACCUM_FINAL if final else 0)
    rc = load_library().pa_attn_fwd_accum(q.data_ptr(), k.data_ptr(), v.data_ptr(), o_acc.data_ptr(),
                                           lse_acc.data_ptr(), out.data_ptr() if final else None, B, H, Nq,
                                           k.shape[2], d, float(scale), flags, _stream_handle(stream, q.device))
    _check(rc, "pa_attn_fwd_accum", check)
    return (out if final else o_acc), lse_acc


def attn_fwd_fp8(q, k, v, q_scale: float, k_scale: float, v_scale: float, scale: Optional[float] = None,
                 out=None, lse=None, stream=None, check: bool = False):
    """Attention over e4m3 inputs (``pa_attn_fwd_fp8``): q [B,H,Nq,128],
    k, v [B,H,Nk,128] of dtype torch.float8_e4m3fn, whose real values are the
    tensors times their scales.  Returns (o bf16, lse fp32) like attn_fwd."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float8_e4m3fn:
            raise TypeError(f"{name} must be a torch.float8_e4m3fn tensor")
        if t.device.type != "cuda" or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-d CUDA tensor")
    B, H, Nq, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse)
    scales = (q_scale, k_scale, v_scale)
    if all(isinstance(x, torch.Tensor) for x in scales):
        # device-resident scales (as pa_quantize_e4m3 writes them)
        for x in scales:
            if x.dtype != torch.float32 or x.numel() != 1 or x.device != q.device:
                raise ValueError("device scales must be one-element float32 tensors on q's device")
        rc = load_library().pa_attn_fwd_fp8_dev(q.data_ptr(), k.data_ptr(), v.data_ptr(), *[x.data_ptr() for x in scales],
                                                out.data_ptr(), lse.data_ptr(), B, H, Nq, k.shape[2], d, float(scale),
                                                _stream_handle(stream, q.device))
        _check(rc, "pa_attn_fwd_fp8_dev", check)
        return out, lse
    rc = load_library().pa_attn_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), float(q_scale), float(k_scale),
                                        float(v_scale), out.data_ptr(), lse.data_ptr(), B, H, Nq, k.shape[2], d,
                                        float(scale), _stream_handle(stream, q.device))
    _check(rc, "pa_attn_fwd_fp8", check)
    return out, lse


def quantize_e4m3(x, out=None, scale=None, stream=None, check: bool = False):
    """Per-tensor e4m3 quantisation of a bf16 tensor on the device
    (``pa_quantize_e4m3``): returns (q torch.float8_e4m3fn of x's shape,
    scale one-element float32 device tensor) with x ~= scale * q."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.device.type != "cuda" \
            or not x.is_contiguous():
        raise TypeError("x must be a contiguous bfloat16 CUDA tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    elif out.dtype != torch.float8_e4m3fn or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous float8_e4m3fn tensor of x's shape")
    if scale is None:
        scale = torch.empty((1,), dtype=torch.float32, device=x.device)
    elif scale.dtype != torch.float32 or scale.numel() != 1:
        raise ValueError("scale must be a one-element float32 tensor")
    rc = load_library().pa_quantize_e4m3(x.data_ptr(), x.numel(), out.data_ptr(), scale.data_ptr(),
                                         _stream_handle(stream, x.device))
    _check(rc, "pa_quantize_e4m3", check)
    return out, scale


def residual_diff(cur, prev, out=None, stream=None, check: bool = False):
    """First Block Cache's residual difference (``pa_residual_diff``):
    sum |cur - prev| / sum |prev| over two bf16 CUDA tensors of the same
    shape, as a one-element float32 device tensor (no host synchronisation;
    compare it with the threshold on the device or read it when needed)."""
    import torch
    for name, t in (("cur", cur), ("prev", prev)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device.type != "cuda" \
                or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    if cur.shape != prev.shape:
        raise ValueError(f"shape mismatch: cur {tuple(cur.shape)}, prev {tuple(prev.shape)}")
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=cur.device)
    elif out.dtype != torch.float32 or out.numel() != 1 or out.device != cur.device:
        raise ValueError("out must be a one-element float32 tensor on cur's device")
    rc = load_library().pa_residual_diff(cur.data_ptr(), prev.data_ptr(), cur.numel(), out.data_ptr(),
                                         _stream_handle(stream, cur.device))
    _check(rc, "pa_residual_diff", check)
    return out


def _on_stream(stream, device):
    """A context in which buffers are allocated for the stream the kernels run
    on, so that the allocator hands their memory on only behind those kernels."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _refuse_rows(name, t, ndim, index):
    """Raise what is wrong with an operand that must be a bf16 tensor with a
    contiguous last dimension on CUDA device ``index``."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16 (got {t.dtype})")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must live on {'a CUDA device' if index is None else f'cuda:{index}'}")
    raise ValueError(f"{name} must be a {ndim}-d tensor with a contiguous last dimension")


class _Torch:
    """torch and what of it the calls below need on every call, looked up on the
    first one (importing this package alone does not import torch)."""

    def __getattr__(self, name):
        import torch
        self.torch, self.bf16, self.f32, self.i32 = torch, torch.bfloat16, torch.float32, torch.int32
        self.empty_like = torch.empty_like
        return self.__dict__[name]


_t = _Torch()


def _check_rows(name, t, ndim, index=None):
    """A bf16 CUDA tensor (on device ``index``, where given) whose last
    dimension is contiguous; returns its device index.  On the way of every
    call: only cheap accessors."""
    try:
        at = t.get_device()
        if (t.dtype is _t.bf16 and at >= 0 and (index is None or at == index) and t.dim() == ndim
                and (t.is_contiguous() or t.stride(-1) == 1 or t.shape[-1] <= 1)):
            return at
    except AttributeError:
        pass
    _refuse_rows(name, t, ndim, index)


def _check_vector(name, t, dtype, shape, index):
    """The address of a contiguous tensor of this type and shape on device
    ``index``; None for None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")


def attn_fwd_mod(q, k, v, scale: Optional[float] = None, softcap: float = 0.0, slopes=None, causal: bool = False,
                 prefix_lens=None, doc_offsets=None, q_offset: Optional[int] = None, out=None, lse=None, stream=None,
                 check: bool = False):
    """Attention with capped and biased scores and interval masks
    (``pa_attn_fwd_mod``): q [B,Hq,Nq,d], k, v [B,Hkv,Nk,d] bf16, Hq a multiple
    of Hkv, any strides that are multiples of 8 elements with the last
    dimension contiguous.

    ``softcap`` c > 0 turns a score s into c*tanh(s/c); ``slopes`` [Hq] float32
    subtracts slopes[h] * |p_i - j|.  Row i stands at p_i = i + ``q_offset``
    (default Nk - Nq: the queries are the last keys).  ``causal`` hides keys
    behind p_i, except the first ``prefix_lens`` keys ([B] int32; of each
    document [B,n_docs] with documents).  ``doc_offsets`` [B,n_docs+1] int32
    cuts the keys into documents; a row sees its own only.  Rows that see
    nothing get o = 0 and lse = -inf.  Returns (o, lse) like attn_fwd; o has
    q's layout.  With very few query rows use ``attn_shared_prefix``, which
    splits the keys over the GPU.
    """
    index = _check_rows("q", q, 4)
    _check_rows("k", k, 4, index)
    _check_rows("v", v, 4, index)
    B, Hq, Nq, d = q_shape = q.shape
    kB, Hkv, Nk, kd = k_shape = k.shape
    if kB != B or kd != d or v.shape != k_shape or Hkv < 1 or Hq % Hkv:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    n_docs = 0
    if doc_offsets is not None:
        if doc_offsets.dim() != 2 or doc_offsets.shape[1] < 2:
            raise ValueError("doc_offsets must be [B, n_docs + 1] with n_docs >= 1")
        n_docs = doc_offsets.shape[1] - 1
    if q_offset is None:
        q_offset = Nk - Nq
    elif not -(1 << 30) <= q_offset <= 1 << 30:  # as a C int it would wrap round
        raise ValueError(f"|q_offset| must be <= 2^30 (got {q_offset})")
    mod = ScoreMod(softcap, 1 if causal else 0, _check_vector("slopes", slopes, _t.f32, (Hq,), index), None,
                   _check_vector("doc_offsets", doc_offsets, _t.i32, (B, n_docs + 1), index), n_docs, q_offset)
    if prefix_lens is not None:
        shape = (B, n_docs) if n_docs else (B, 1) if prefix_lens.dim() == 2 else (B,)
        mod.prefix_lens = _check_vector("prefix_lens", prefix_lens, _t.i32, shape, index)
    fresh = out is None
    lse_at = None if lse is None else _check_vector("lse", lse, _t.f32, (B, Hq, Nq), index)
    if fresh or lse is None:
        with _nullcontext if stream is None else _on_stream(stream, q.device):
            if out is None:
                out = _t.empty_like(q)  # keeps a dense layout such as [B, Nq, Hq, d]
                if out.stride(-1) != 1:
                    out = q.new_empty(q_shape)
            if lse is None:
                lse = q.new_empty((B, Hq, Nq), dtype=_t.f32)
                lse_at = lse.data_ptr()
    if not fresh:
        _check_rows("out", out, 4, index)
        if out.shape != q_shape:
            raise ValueError("out must have q's shape")
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        strides = _Strides12(*q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *out.stride()[:3])
    rc = load_library().pa_attn_fwd_mod(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_at, B, Hq, Hkv,
                                        Nq, Nk, d, strides, 1.0 / math.sqrt(d) if scale is None else scale,
                                        ctypes.byref(mod), _stream_handle(stream, index))
    if rc or check:
        _check(rc, "pa_attn_fwd_mod", check)
    return out, lse


def shared_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Np: int, Nt: int, d: int) -> int:
    """Bytes of workspace ``attn_shared_prefix`` needs for these sizes."""
    return int(load_library().pa_attn_shared_prefix_workspace(B, Hq, Hkv, Nq, Np, Nt, d))


# A function of the sizes alone, asked for in every decoding step.
_workspace_bytes = functools.lru_cache(maxsize=256)(shared_prefix_workspace_bytes)


def attn_shared_prefix(q, k_prefix, v_prefix, k_tail, v_tail, tail_lens, scale: Optional[float] = None,
                       softcap: float = 0.0, slopes=None, out=None, lse=None, workspace=None, stream=None,
                       check: bool = False):
    """A decoding step of B requests that share a prefix
    (``pa_attn_shared_prefix``): q [B,Hq,Nq,d] (contiguous) against the prefix
    k_prefix, v_prefix [Hkv,Np,d], read once for all requests, and each
    request's own k_tail, v_tail [B,Hkv,Nt,d] up to tail_lens [B] int32, the
    new tokens' own keys being the last Nq of them.  ``softcap`` and ``slopes``
    as in ``attn_fwd_mod``.  ``workspace`` (at least
    ``shared_prefix_workspace_bytes``) is allocated when not given; two calls
    that may overlap on the GPU need one each.  Returns (o, lse).
    """
    index = _check_rows("q", q, 4)
    _check_rows("k_prefix", k_prefix, 3, index)
    _check_rows("v_prefix", v_prefix, 3, index)
    _check_rows("k_tail", k_tail, 4, index)
    _check_rows("v_tail", v_tail, 4, index)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    B, Hq, Nq, d = q_shape = q.shape
    Hkv, Np, pd = p_shape = k_prefix.shape
    tB, tH, Nt, td = t_shape = k_tail.shape
    if (pd != d or v_prefix.shape != p_shape or tB != B or tH != Hkv or td != d or v_tail.shape != t_shape or Hkv < 1
            or Hq % Hkv):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, prefix {tuple(k_prefix.shape)} and "
                         f"{tuple(v_prefix.shape)}, tail {tuple(k_tail.shape)} and {tuple(v_tail.shape)}")
    lens = _check_vector("tail_lens", tail_lens, _t.i32, (B,), index)
    sl = _check_vector("slopes", slopes, _t.f32, (Hq,), index)
    lib = load_library()
    fresh, own_space = out is None, workspace is None
    lse_at = None if lse is None else _check_vector("lse", lse, _t.f32, (B, Hq, Nq), index)
    if fresh or own_space or lse is None:
        with _nullcontext if stream is None else _on_stream(stream, q.device):
            if out is None:
                out = _t.empty_like(q)
            if lse is None:
                lse = q.new_empty((B, Hq, Nq), dtype=_t.f32)
                lse_at = lse.data_ptr()
            if own_space:
                # in bf16 elements of q: one allocation without a type to look up
                workspace = q.new_empty((_workspace_bytes(B, Hq, Hkv, Nq, Np, Nt, d) // 2,))
    if not fresh:
        _check_rows("out", out, 4, index)
        if out.shape != q_shape or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor of q's shape")
    if not own_space and (not isinstance(workspace, _t.torch.Tensor) or workspace.get_device() != index
                          or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on q's device")
    strides = None
    if not (k_prefix.is_contiguous() and v_prefix.is_contiguous() and k_tail.is_contiguous()
            and v_tail.is_contiguous()):
        strides = _Strides10(*k_prefix.stride()[:2], *v_prefix.stride()[:2], *k_tail.stride()[:3],
                             *v_tail.stride()[:3])
    rc = lib.pa_attn_shared_prefix(q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k_tail.data_ptr(),
                                   v_tail.data_ptr(), lens, out.data_ptr(), lse_at, B, Hq, Hkv, Nq, Np, Nt, d,
                                   strides, 1.0 / math.sqrt(d) if scale is None else scale, softcap, sl,
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream_handle(stream, index))
    if rc or check:
        _check(rc, "pa_attn_shared_prefix", check)
    return out, lse


def gate_residual_norm(y, x, gate=None, post: str = "none", post_weight=None, norm: str = "rms", norm_weight=None,
                       scale=None, shift=None, residual_scale: float = 1.0, eps: float = 1e-6, x_out=None, out=None,
                       stream=None, check: bool = False):
    """A block's gated residual update with the norms around it
    (``pa_gate_residual_norm``), in one pass over the data:

        x_new = residual_scale * x + gate * post(y) * post_weight
        h = norm(x_new) * norm_weight * (1 + scale) + shift

    y [B,N,D] bf16, x [B,N,D] bf16 or float32 (the residual stream), gate,
    scale, shift [B,D] bf16 (slices of one wider modulation tensor are taken as
    they are), weights [D] bf16; ``post`` and ``norm`` are "none", "rms" or
    "layer".  Returns (x_new, h); x_new has x's type and goes to ``x_out``, which
    may be x itself, h (bf16, None with norm="none") to ``out``."""
    index = _check_rows("y", y, 3)
    B, N, D = shape = y.shape
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    if (not isinstance(x, _t.torch.Tensor) or x.dtype not in (_t.bf16, _t.f32) or x.shape != shape
            or not x.is_contiguous() or x.get_device() != index):
        raise ValueError("x must be a contiguous bfloat16 or float32 tensor of y's shape on its device")
    if post not in PA_NORM or norm not in PA_NORM:
        raise ValueError(f"post and norm must be one of {sorted(PA_NORM)} (got {post!r}, {norm!r})")
    cfg = BlockNorm(PA_NORM[post], PA_NORM[norm], _check_vector("post_weight", post_weight, _t.bf16, (D,), index),
                    _check_vector("norm_weight", norm_weight, _t.bf16, (D,), index), None, None, None, 0, 0, 0,
                    residual_scale, eps)
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
        if t is None:
            continue
        _check_rows(name, t, 2, index)
        if t.shape != (B, D):
            raise ValueError(f"{name} must be [B, D] = {(B, D)} (got {tuple(t.shape)})")
        setattr(cfg, name, t.data_ptr())
        setattr(cfg, name + "_stride", t.stride(0))
    if norm == "none" and out is not None:
        raise ValueError("out is written only with a norm")
    if x_out is None or (out is None and norm != "none"):
        with _nullcontext if stream is None else _on_stream(stream, y.device):
            if x_out is None:
                x_out = _t.empty_like(x)
            if out is None and norm != "none":
                out = _t.empty_like(y)
    if x_out.dtype != x.dtype or x_out.shape != shape or not x_out.is_contiguous() or x_out.get_device() != index:
        raise ValueError("x_out must be a contiguous tensor of x's type and shape on its device")
    if out is not None:
        _check_rows("out", out, 3, index)
        if out.shape != shape or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor of y's shape")
    rc = load_library().pa_gate_residual_norm(y.data_ptr(), x.data_ptr(), x_out.data_ptr(),
                                               None if out is None else out.data_ptr(), B, N, D,
                                               1 if x.dtype == _t.f32 else 0, ctypes.byref(cfg),
                                               _stream_handle(stream, index))
    if rc or check:
        _check(rc, "pa_gate_residual_norm", check)
    return x_out, out


def attn_merge(o_parts, lse_parts, out=None, lse=None, stream=None, check: bool = False):
    """Merge n partial results o_parts [n,B,H,N,d] bf16, lse_parts [n,B,H,N]
    fp32 (over disjoint key chunks) into (o [B,H,N,d], lse [B,H,N])."""
    import torch
    _check_bf16("o_parts", o_parts, 5)
    n, B, H, N, d = o_parts.shape
    if (lse_parts.dtype != torch.float32 or tuple(lse_parts.shape) != (n, B, H, N)
            or not lse_parts.is_contiguous() or lse_parts.device != o_parts.device):
        raise ValueError("lse_parts must be a contiguous float32 [n,B,H,N] tensor on o_parts' device")
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=o_parts.device)
    else:
        _check_bf16("out", out, 4)
        if tuple(out.shape) != (B, H, N, d):
            raise ValueError(f"out must be [B,H,N,d] = {(B, H, N, d)} (got {tuple(out.shape)})")
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=o_parts.device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B,H,N] tensor")
    rc = load_library().pa_attn_merge(o_parts.data_ptr(), lse_parts.data_ptr(), n, out.data_ptr(),
                                      lse.data_ptr(), B, H, N, d,
                                      _stream_handle(stream, o_parts.device))
    _check(rc, "pa_attn_merge", check)
    return out, lse


def _outputs(q, out, lse):
    """(out, lse) for a query tensor q [B,H,Nq,d]: allocated when None,
    otherwise checked for dtype, shape and layout."""
    import torch
    B, H, Nq, d = q.shape
    if out is None:
        out = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q.device)
    else:
        _check_bf16("out", out, 4)
        if tuple(out.shape) != (B, H, Nq, d):
            raise ValueError("out must have q's shape")
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B,H,Nq] tensor")
    return out, lse


def _chunk_arrays(q, k_chunks, v_chunks):
    B, H, Nq, d = q.shape
    n = len(k_chunks)
    if n < 1 or len(v_chunks) != n:
        raise ValueError("need at least one chunk and as many V chunks as K chunks")
    for kc, vc in zip(k_chunks, v_chunks):
        _check_bf16("k chunk", kc, 4)
        _check_bf16("v chunk", vc, 4)
        if kc.shape != vc.shape or kc.shape[:2] != (B, H) or kc.shape[3] != d:
            raise ValueError("chunk shapes must be [B, H, n_c, d] matching q")
    kp = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc in k_chunks])
    vp = (ctypes.c_void_p * n)(*[vc.data_ptr() for vc in v_chunks])
    nk = (ctypes.c_int * n)(*[kc.shape[2] for kc in k_chunks])
    return kp, vp, nk, n


def attn_fwd_chunks(q, k_chunks, v_chunks, scale: Optional[float] = None, out=None, lse=None, stream=None,
                    check: bool = False):
    """Attention of q over the concatenation of the K/V chunks (up to 8) in a
    single launch (``pa_attn_fwd_chunks``); no partial results are written."""
    _check_bf16("q", q, 4)
    B, H, Nq, d = q.shape
    kp, vp, nk, n = _chunk_arrays(q, k_chunks, v_chunks)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse)
    rc = load_library().pa_attn_fwd_chunks(q.data_ptr(), kp, vp, nk, n, out.data_ptr(), lse.data_ptr(),
                                           B, H, Nq, d, float(scale), _stream_handle(stream, q.device))
    _check(rc, "pa_attn_fwd_chunks", check)
    return out, lse


def attn_chunks_noalloc(q, k_chunks, v_chunks, scale: Optional[float] = None, out=None, lse=None, stream=None,
                        check: bool = False):
    """Attention of q over the concatenation of the K/V chunks through
    ``pa_attn_chunks_noalloc``: the library keeps the per-chunk partials in
    its fixed static array instead of allocating them (see the header for the
    size limit and the sharing rules).  Outputs are allocated here only when
    not given."""
    _check_bf16("q", q, 4)
    B, H, Nq, d = q.shape
    kp, vp, nk, n = _chunk_arrays(q, k_chunks, v_chunks)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse)
    rc = load_library().pa_attn_chunks_noalloc(q.data_ptr(), kp, vp, nk, n, out.data_ptr(), lse.data_ptr(),
                                               B, H, Nq, d, float(scale), _stream_handle(stream, q.device))
    _check(rc, "pa_attn_chunks_noalloc", check)
    return out, lse


def poll_device_status() -> int:
    """Read and clear the device status word (synchronising).  Returns the
    status code (0 = no device-side error since the last poll)."""
    return int(load_library().pa_poll_device_status())


def set_wait_limit_ms(ms: int) -> None:
    """Limit of every device-side barrier wait for later launches
    (``pa_set_wait_limit_ms``; default 5000 ms)."""
    _check(load_library().pa_set_wait_limit_ms(int(ms)), "pa_set_wait_limit_ms")


def selftest_timeout(limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self-test kernel (see pa_selftest_timeout)."""
    import torch
    rc = load_library().pa_selftest_timeout(int(limit_us),
                                            _stream_handle(stream, torch.cuda.current_device()))
    _check(rc, "pa_selftest_timeout")
