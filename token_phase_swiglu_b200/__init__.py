"""Python binding of libfmlp.so, the B200 fused gated-MLP library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/fmlp.h``.  Tensors are torch
CUDA tensors (torch provides device memory and streams); the functions pass
their device pointers and sizes through ctypes and raise ``FmlpError`` on any
status other than FMLP_OK.  There is no fallback: if the shared library has
not been built, importing this package raises ImportError.
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "FmlpError", "FMLP_OK", "FMLP_ERR_INVALID_ARG", "FMLP_ERR_UNSUPPORTED", "FMLP_ERR_CUDA",
    "FMLP_ERR_TIMEOUT", "LIB_PATH", "lib", "fmlp_pack", "fmlp_workspace_bytes", "fmlp_forward",
    "fmlp_gate_up_swiglu", "fmlp_down_proj", "fmlp_device_status", "fmlp_status_string",
    "fmlp_last_cuda_error", "fmlp_kernel_launch_count", "fmlp_set_wait_timeout_ns", "fmlp_set_fault_injection",
    "fmlp_forward_noalloc", "NOALLOC_SCRATCH_BYTES", "EXPORTED_SYMBOLS", "fmlp_forward_bf16",
    "fmlp_sum_partials", "fmlp_quantize_q8", "fmlp_forward_q8", "Q8_GROUP",
    "fmlp_attn_workspace_bytes", "fmlp_attn_decode", "FmlpRope", "CONTROL_BYTES", "fmlp_rope_append",
    "fmlp_rope_append_q8", "fmlp_kv_read_q8", "fmlp_prefill_workspace_bytes", "fmlp_attn_prefill",
    "fmlp_attn_q8_workspace_bytes", "fmlp_attn_decode_q8",
]

FMLP_OK, FMLP_ERR_INVALID_ARG, FMLP_ERR_UNSUPPORTED, FMLP_ERR_CUDA, FMLP_ERR_TIMEOUT = range(5)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfmlp.so")

_i64, _sz, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float

_i32 = ctypes.c_int


class _Rope(ctypes.Structure):   # fmlp_rope in include/fmlp.h
    _fields_ = [("theta", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("amplitude", ctypes.c_double), ("original_ctx", _i64),
                ("rotary_dim", _i32), ("interleaved", _i32), ("scaling", _i32)]


_ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}


class FmlpRope:
    """How q and k are rotated (fmlp_rope in include/fmlp.h): the base, the values of a
    head that turn, their pairing, and the scaling of the frequencies for long contexts
    ("none", "linear", "bands" or "yarn")."""

    def __init__(self, theta: float, rotary_dim: int, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                 original_ctx: int = 1, amplitude: float = 1.0):
        if scaling not in _ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}, got {scaling!r}")
        self._c = _Rope(theta, factor, low, high, amplitude, original_ctx, rotary_dim,
                        int(interleaved), _ROPE_SCALINGS[scaling])


# name -> (restype, argtypes); mirrors include/fmlp.h
_SIGNATURES = {
    "fmlp_pack": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _vp]),
    "fmlp_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fmlp_forward": (_int, [_vp, _i64, _vp, _f32, _vp, _int, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "fmlp_gate_up_swiglu": (_int, [_vp, _i64, _vp, _f32, _vp, _int, _i64, _i64, _vp, _vp, _sz, _vp]),
    "fmlp_down_proj": (_int, [_vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "fmlp_device_status": (_int, [_vp, _vp]),
    "fmlp_status_string": (ctypes.c_char_p, [_int]),
    "fmlp_last_cuda_error": (_int, []),
    "fmlp_kernel_launch_count": (ctypes.c_uint64, []),
    "fmlp_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "fmlp_set_fault_injection": (None, [_int]),
    "fmlp_forward_noalloc": (_int, [_vp, _i64, _vp, _f32, _vp, _int, _vp, _i64, _i64, _vp, _vp, _vp]),
    "fmlp_forward_bf16": (_int, [_vp, _i64, _vp, _f32, _vp, _int, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "fmlp_sum_partials": (_int, [ctypes.POINTER(_vp), _int, _i64, _i64, _vp, _vp, _int, _vp]),
    "fmlp_quantize_q8": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "fmlp_forward_q8": (_int, [_vp, _i64, _vp, _f32, _vp, _vp, _int, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "fmlp_attn_workspace_bytes": (_sz, [_i64, _int, _int, _int]),
    "fmlp_attn_decode": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _i64, _i64, _f32,
                                _vp, _vp, _sz, _vp]),
    "fmlp_rope_append": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _int, _int, _int,
                                ctypes.POINTER(_Rope), _vp, _vp, _f32, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "fmlp_rope_append_q8": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _int, _int, _int,
                                   ctypes.POINTER(_Rope), _vp, _vp, _f32, _vp, _vp, _vp, _vp, _vp, _i64, _vp,
                                   _sz, _vp]),
    "fmlp_prefill_workspace_bytes": (_sz, [_i64, _i64, _int, _int, _int]),
    "fmlp_attn_prefill": (_int, [_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _int, _i64, _f32, _vp, _vp,
                                 _sz, _vp]),
    "fmlp_attn_q8_workspace_bytes": (_sz, [_i64, _int, _int, _int]),
    "fmlp_attn_decode_q8": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _int, _i64, _f32, _vp, _vp, _sz,
                                   _vp]),
    "fmlp_kv_read_q8": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _int, _int, _i64, _vp, _vp, _vp, _sz, _vp]),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(nvcc, sm_100a). There is no non-CUDA implementation.")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()


class FmlpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.fmlp_status_string(status).decode()
        if status == FMLP_ERR_CUDA:
            msg += f" (cudaError {lib.fmlp_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


def _check_status(status: int, where: str) -> None:
    if status != FMLP_OK:
        raise FmlpError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libfmlp must be contiguous")
    return t.data_ptr()


# The current stream's handle without the Stream object around it (CPU-only builds of
# torch do not have it; no tensor is on a device there).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if torch.cuda.is_initialized() and _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _bf16(t, name):
    if t is not None and t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")


def _check(t, name, dtype, shape=None, optional=False):
    """Check one tensor argument before its pointer goes to the library: the
    dtype (TypeError), the exact shape and contiguity (ValueError).  Together
    with _on_device (the library launches on the current device), nothing
    malformed reaches the C ABI."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(**tensors):
    """Every given tensor lives on the current CUDA device (checked after the
    dtypes and shapes of all of them)."""
    current = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if current is None:
            current = torch.cuda.current_device()
        if t.get_device() != current:
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{current}")


def _check_workspace(ws, need: int):
    _check(ws, "workspace", None)
    if ws.nbytes < need:
        raise ValueError(f"workspace holds {ws.nbytes} bytes, {need} needed")


def _dims2(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _check_forward_args(x, gamma, packed, W_down, out, residual):
    """Shapes of the MLP block's tensors: (M, d, I)."""
    _bf16(x, "x")
    M, d = _dims2(x, "x")
    _bf16(W_down, "W_down")
    d2, I = _dims2(W_down, "W_down")
    if d2 != d:
        raise ValueError(f"W_down has {d2} rows, x has {d} columns")
    _check(x, "x", torch.bfloat16, (M, d))
    _check(gamma, "gamma", torch.bfloat16, (d,))
    _check(packed, "packed", torch.bfloat16, (2 * I, d))
    _check(W_down, "W_down", torch.bfloat16, (d, I))
    _check(residual, "residual", torch.bfloat16, (M, d), optional=True)
    return M, d, I


def fmlp_status_string(status: int) -> str:
    return lib.fmlp_status_string(status).decode()


def fmlp_last_cuda_error() -> int:
    return lib.fmlp_last_cuda_error()


def fmlp_kernel_launch_count() -> int:
    return int(lib.fmlp_kernel_launch_count())


def fmlp_set_wait_timeout_ns(ns: int) -> None:
    """Deadline of the kernels' bounded waits (0 = default, one second)."""
    lib.fmlp_set_wait_timeout_ns(int(ns))


def fmlp_set_fault_injection(mode: int) -> None:
    """Testing aid: nonzero makes kernels withhold their last stage (bounded waits expire)."""
    lib.fmlp_set_fault_injection(int(mode))


def fmlp_workspace_bytes(M: int, d: int, I: int) -> int:
    return int(lib.fmlp_workspace_bytes(M, d, I))


def fmlp_pack(W_gate, W_up, tile_T: int, packed, stream=None) -> None:
    """packed [2I x d] <- rows of W_gate / W_up [I x d] interleaved at tile tile_T."""
    _bf16(W_gate, "W_gate"); _bf16(W_up, "W_up"); _bf16(packed, "packed")
    I, d = _dims2(W_gate, "W_gate")
    _check(W_gate, "W_gate", torch.bfloat16, (I, d))
    _check(W_up, "W_up", torch.bfloat16, (I, d))
    _check(packed, "packed", torch.bfloat16, (2 * I, d))
    _on_device(W_gate=W_gate, W_up=W_up, packed=packed)
    _check_status(lib.fmlp_pack(_ptr(W_gate), _ptr(W_up), d, I, tile_T, _ptr(packed),
                                _stream(stream)), "fmlp_pack")


def fmlp_forward(x, gamma, eps: float, packed, tile_T: int, W_down, out, workspace,
                 residual=None, stream=None) -> None:
    """out [M x d] (f32) <- RMSNorm + gated MLP (+ residual) of x [M x d]."""
    M, d, I = _check_forward_args(x, gamma, packed, W_down, out, residual)
    _check(out, "out", torch.float32, (M, d))
    _check_workspace(workspace, fmlp_workspace_bytes(M, d, I))
    _on_device(x=x, gamma=gamma, packed=packed, W_down=W_down, residual=residual, out=out,
               workspace=workspace)
    _check_status(lib.fmlp_forward(_ptr(x), M, _ptr(gamma), eps, _ptr(packed), tile_T,
                                   _ptr(W_down), d, I, _ptr(residual), _ptr(out), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
                  "fmlp_forward")


def fmlp_forward_bf16(x, gamma, eps: float, packed, tile_T: int, W_down, out, workspace,
                      residual=None, stream=None) -> None:
    """out [M x d] (bf16) <- bf16(RMSNorm + gated MLP of x + residual): the output
    chained layers feed to each other.  out may be x or residual itself."""
    M, d, I = _check_forward_args(x, gamma, packed, W_down, out, residual)
    _check(out, "out", torch.bfloat16, (M, d))
    _check_workspace(workspace, fmlp_workspace_bytes(M, d, I))
    _on_device(x=x, gamma=gamma, packed=packed, W_down=W_down, residual=residual, out=out,
               workspace=workspace)
    _check_status(lib.fmlp_forward_bf16(_ptr(x), M, _ptr(gamma), eps, _ptr(packed), tile_T,
                                        _ptr(W_down), d, I, _ptr(residual), _ptr(out),
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)),
                  "fmlp_forward_bf16")


def fmlp_sum_partials(partials, out, residual=None, stream=None) -> None:
    """out [M x d] <- sum of the f32 partial outputs [M x d] (+ residual), out f32 or
    bf16: the reduction of a tensor-parallel MLP block (partials may be peer memory)."""
    if not partials:
        raise ValueError("at least one partial output is needed")
    M, d = _dims2(partials[0], "partials[0]")
    for r, t in enumerate(partials):
        _check(t, f"partials[{r}]", torch.float32, (M, d))
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out must be float32 or bfloat16, got {out.dtype}")
    _check(out, "out", out.dtype, (M, d))
    _check(residual, "residual", torch.bfloat16, (M, d), optional=True)
    _on_device(out=out, residual=residual)
    arr = (_vp * len(partials))(*[t.data_ptr() for t in partials])
    _check_status(lib.fmlp_sum_partials(arr, len(partials), M, d, _ptr(residual), _ptr(out),
                                        int(out.dtype == torch.bfloat16), _stream(stream)),
                  "fmlp_sum_partials")


Q8_GROUP = 64   # elements per scale of the int8 weight format (include/fmlp.h)


def fmlp_quantize_q8(W, q, scales, stream=None) -> None:
    """q int8 [rows x K], scales f32 [rows x K/64] <- the int8 format of W bf16 [rows x K]."""
    _bf16(W, "W")
    rows, K = _dims2(W, "W")
    _check(W, "W", torch.bfloat16, (rows, K))
    _check(q, "q", torch.int8, (rows, K))
    _check(scales, "scales", torch.float32, (rows, K // Q8_GROUP))
    _on_device(W=W, q=q, scales=scales)
    _check_status(lib.fmlp_quantize_q8(_ptr(W), rows, K, _ptr(q), _ptr(scales), _stream(stream)),
                  "fmlp_quantize_q8")


def fmlp_forward_q8(x, gamma, eps: float, packed_q, packed_scales, tile_T: int, W_down_q,
                    W_down_scales, out, workspace, residual=None, stream=None) -> None:
    """out [M x d] (f32) <- the MLP block of x on int8 weights (fmlp_quantize_q8's)."""
    _bf16(x, "x")
    M, d = _dims2(x, "x")
    d2, I = _dims2(W_down_q, "W_down_q")
    if d2 != d:
        raise ValueError(f"W_down_q has {d2} rows, x has {d} columns")
    _check(x, "x", torch.bfloat16, (M, d))
    _check(gamma, "gamma", torch.bfloat16, (d,))
    _check(packed_q, "packed_q", torch.int8, (2 * I, d))
    _check(packed_scales, "packed_scales", torch.float32, (2 * I, d // Q8_GROUP))
    _check(W_down_q, "W_down_q", torch.int8, (d, I))
    _check(W_down_scales, "W_down_scales", torch.float32, (d, I // Q8_GROUP))
    _check(residual, "residual", torch.bfloat16, (M, d), optional=True)
    _check(out, "out", torch.float32, (M, d))
    _check_workspace(workspace, fmlp_workspace_bytes(M, d, I))
    _on_device(x=x, gamma=gamma, packed_q=packed_q, packed_scales=packed_scales,
               W_down_q=W_down_q, W_down_scales=W_down_scales, residual=residual, out=out,
               workspace=workspace)
    _check_status(lib.fmlp_forward_q8(_ptr(x), M, _ptr(gamma), eps, _ptr(packed_q),
                                      _ptr(packed_scales), tile_T, _ptr(W_down_q),
                                      _ptr(W_down_scales), d, I, _ptr(residual), _ptr(out),
                                      _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream)),
                  "fmlp_forward_q8")


def fmlp_attn_workspace_bytes(B: int, H: int, H_kv: int, D: int) -> int:
    n = lib.fmlp_attn_workspace_bytes(B, H, H_kv, D)
    if n == 0:
        raise FmlpError(FMLP_ERR_INVALID_ARG, "fmlp_attn_workspace_bytes: shape not taken")
    return n


def fmlp_attn_decode(q, k_new, v_new, k_cache, v_cache, pos, n_ctx: int, theta: float, out,
                     workspace, stream=None) -> None:
    """One token-phase attention step (RoPE, in-place KV append, attention over
    the cache rows 0..pos); see include/fmlp.h for the layouts."""
    _bf16(q, "q")
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, H, D] and the caches [B, H_kv, n_max, D]")
    B, H, D = q.shape
    H_kv, n_max = k_cache.shape[1], k_cache.shape[2]
    _check(q, "q", torch.bfloat16, (B, H, D))
    _check(k_new, "k_new", torch.bfloat16, (B, H_kv, D))
    _check(v_new, "v_new", torch.bfloat16, (B, H_kv, D))
    _check(k_cache, "k_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check(v_cache, "v_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check(pos, "pos", torch.int32, (B,))
    _check(out, "out", torch.float32, (B, H, D))
    _check_workspace(workspace, fmlp_attn_workspace_bytes(B, H, H_kv, D))
    _on_device(q=q, k_new=k_new, v_new=v_new, k_cache=k_cache, v_cache=v_cache, pos=pos, out=out,
               workspace=workspace)
    _check_status(lib.fmlp_attn_decode(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(pos), B, H, H_kv, D, n_max, n_ctx,
                                       theta, _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream)),
                  "fmlp_attn_decode")


CONTROL_BYTES = 256   # FMLP_CONTROL_BYTES in include/fmlp.h


def _check_rows(t, name, heads=None, D=None):
    """A packed batch's rows [T, heads, D]: bf16, every token's heads contiguous, tokens
    any stride apart (a column range of a projection's output); returns that stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    _bf16(t, name)
    if t.dim() != 3 or (heads is not None and t.shape[1:] != (heads, D)):
        raise ValueError(f"{name} must have shape [tokens, {heads or 'heads'}, {D or 'D'}], got {tuple(t.shape)}")
    T, h, d = t.shape
    if T == 0:
        return h * d
    stride, head, one = t.stride()
    if one != 1 or (h > 1 and head != d):
        raise ValueError(f"the heads of a token must be contiguous in {name}")
    if T == 1:
        return h * d
    if stride < h * d:
        raise ValueError(f"tokens overlap in {name}")
    return stride


def _check_batch(cu_seqlens, kv_len):
    if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1:
        raise ValueError("kv_len must be a 1-D tensor, one entry a sequence")
    B = kv_len.shape[0]
    _check(kv_len, "kv_len", torch.int32, (B,))
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    return B


def _append_args(q, k, v, cu_seqlens, kv_len, rope, q_out, k_cache, v_cache, workspace, q_gamma, k_gamma,
                 cache_dtype):
    q_stride = _check_rows(q, "q")
    T, H, D = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("the caches must be [B, H_kv, n_max, D]")
    B = _check_batch(cu_seqlens, kv_len)
    H_kv, n_max = k_cache.shape[1], k_cache.shape[2]
    k_stride, v_stride = _check_rows(k, "k", H_kv, D), _check_rows(v, "v", H_kv, D)
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q has {T} tokens, k {k.shape[0]} and v {v.shape[0]}")
    if not isinstance(rope, FmlpRope):
        raise TypeError(f"rope must be an FmlpRope, got {type(rope).__name__}")
    _check(k_cache, "k_cache", cache_dtype, (B, H_kv, n_max, D))
    _check(v_cache, "v_cache", cache_dtype, (B, H_kv, n_max, D))
    _check(q_out, "q_out", torch.bfloat16, (T, H, D))
    _check(q_gamma, "q_gamma", torch.bfloat16, (D,), optional=True)
    _check(k_gamma, "k_gamma", torch.bfloat16, (D,), optional=True)
    _check_workspace(workspace, CONTROL_BYTES)
    return q_stride, k_stride, v_stride, T, B, H, H_kv, D, n_max


def fmlp_rope_append(q, k, v, cu_seqlens, kv_len, rope, q_out, k_cache, v_cache, workspace, q_gamma=None,
                     k_gamma=None, eps: float = 1e-6, stream=None) -> None:
    """q_out [T, H, D] <- the (normed and) rotated queries of a packed batch's T new tokens; their (normed
    and) rotated keys and their values into rows kv_len[b] - n_b .. kv_len[b] - 1 of the caches
    [B, H_kv, n_max, D].  See include/fmlp.h."""
    qs, ks, vs, T, B, H, H_kv, D, n_max = _append_args(q, k, v, cu_seqlens, kv_len, rope, q_out, k_cache, v_cache,
                                                       workspace, q_gamma, k_gamma, torch.bfloat16)
    _on_device(q=q, k=k, v=v, cu_seqlens=cu_seqlens, kv_len=kv_len, q_gamma=q_gamma, k_gamma=k_gamma, q_out=q_out,
               k_cache=k_cache, v_cache=v_cache, workspace=workspace)
    _check_status(lib.fmlp_rope_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, cu_seqlens.data_ptr(),
                                       kv_len.data_ptr(), B, H, H_kv, D, ctypes.byref(rope._c), _ptr(q_gamma),
                                       _ptr(k_gamma), eps, q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), n_max,
                                       workspace.data_ptr(), workspace.nbytes,
                                       _stream(stream)),
                  "fmlp_rope_append")


def fmlp_rope_append_q8(q, k, v, cu_seqlens, kv_len, rope, q_out, k_q, k_s, v_q, v_s, workspace, q_gamma=None,
                        k_gamma=None, eps: float = 1e-6, stream=None) -> None:
    """fmlp_rope_append into an int8 cache: codes k_q, v_q int8 [B, H_kv, n_max, D] and one scale a row,
    k_s, v_s f32 [B, H_kv, n_max]."""
    qs, ks, vs, T, B, H, H_kv, D, n_max = _append_args(q, k, v, cu_seqlens, kv_len, rope, q_out, k_q, v_q, workspace,
                                                       q_gamma, k_gamma, torch.int8)
    _check(k_s, "k_s", torch.float32, (B, H_kv, n_max))
    _check(v_s, "v_s", torch.float32, (B, H_kv, n_max))
    _on_device(q=q, k=k, v=v, cu_seqlens=cu_seqlens, kv_len=kv_len, q_gamma=q_gamma, k_gamma=k_gamma, q_out=q_out,
               k_q=k_q, k_s=k_s, v_q=v_q, v_s=v_s, workspace=workspace)
    _check_status(lib.fmlp_rope_append_q8(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, cu_seqlens.data_ptr(),
                                          kv_len.data_ptr(), B, H, H_kv, D, ctypes.byref(rope._c), _ptr(q_gamma),
                                          _ptr(k_gamma), eps, q_out.data_ptr(), k_q.data_ptr(), k_s.data_ptr(), v_q.data_ptr(),
                                          v_s.data_ptr(), n_max, workspace.data_ptr(),
                                          workspace.nbytes, _stream(stream)),
                  "fmlp_rope_append_q8")


def _check_q8_cache(k_q, k_s, v_q, v_s, B):
    if not isinstance(k_q, torch.Tensor) or k_q.dim() != 4:
        raise ValueError("the caches must be [B, H_kv, n_max, D]")
    _, H_kv, n_max, D = k_q.shape
    for t, name in ((k_q, "k_q"), (v_q, "v_q")):
        _check(t, name, torch.int8, (B, H_kv, n_max, D))
    for t, name in ((k_s, "k_s"), (v_s, "v_s")):
        _check(t, name, torch.float32, (B, H_kv, n_max))
    return H_kv, n_max, D


def fmlp_kv_read_q8(k_q, k_s, v_q, v_s, kv_len, k_cache, v_cache, workspace, stream=None) -> None:
    """Rows 0 .. kv_len[b] - 1 of bf16 caches [B, H_kv, n_max, D] <- codes times scales of an int8 cache."""
    B = _check_batch(None, kv_len)
    H_kv, n_max, D = _check_q8_cache(k_q, k_s, v_q, v_s, B)
    _check(k_cache, "k_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check(v_cache, "v_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check_workspace(workspace, CONTROL_BYTES)
    _on_device(k_q=k_q, k_s=k_s, v_q=v_q, v_s=v_s, kv_len=kv_len, k_cache=k_cache, v_cache=v_cache,
               workspace=workspace)
    _check_status(lib.fmlp_kv_read_q8(k_q.data_ptr(), k_s.data_ptr(), v_q.data_ptr(), v_s.data_ptr(), kv_len.data_ptr(), B, H_kv, D, n_max,
                                      k_cache.data_ptr(), v_cache.data_ptr(), workspace.data_ptr(),
                                      workspace.nbytes, _stream(stream)),
                  "fmlp_kv_read_q8")


def fmlp_prefill_workspace_bytes(T: int, B: int, H: int, H_kv: int, D: int) -> int:
    n = lib.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D)
    if n == 0:
        raise FmlpError(FMLP_ERR_INVALID_ARG, "fmlp_prefill_workspace_bytes: shape not taken")
    return n


def fmlp_attn_prefill(q, k_cache, v_cache, cu_seqlens, kv_len, scale: float, out, workspace, stream=None) -> None:
    """out [T, H, D] (bf16) <- causal attention of a packed batch's new tokens (queries q [T, H, D], already
    rotated) over rows 0 .. position of the caches [B, H_kv, n_max, D].  See include/fmlp.h."""
    q_stride = _check_rows(q, "q")
    T, H, D = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("the caches must be [B, H_kv, n_max, D]")
    B = _check_batch(cu_seqlens, kv_len)
    H_kv, n_max = k_cache.shape[1], k_cache.shape[2]
    _check(k_cache, "k_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check(v_cache, "v_cache", torch.bfloat16, (B, H_kv, n_max, D))
    _check(out, "out", torch.bfloat16, (T, H, D))
    _check_workspace(workspace, fmlp_prefill_workspace_bytes(T, B, H, H_kv, D))
    _on_device(q=q, k_cache=k_cache, v_cache=v_cache, cu_seqlens=cu_seqlens, kv_len=kv_len, out=out,
               workspace=workspace)
    _check_status(lib.fmlp_attn_prefill(q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), cu_seqlens.data_ptr(),
                                        kv_len.data_ptr(), T, B, H, H_kv, D, n_max, scale, out.data_ptr(), workspace.data_ptr(),
                                        workspace.nbytes, _stream(stream)),
                  "fmlp_attn_prefill")


def fmlp_attn_q8_workspace_bytes(B: int, H: int, H_kv: int, D: int) -> int:
    n = lib.fmlp_attn_q8_workspace_bytes(B, H, H_kv, D)
    if n == 0:
        raise FmlpError(FMLP_ERR_INVALID_ARG, "fmlp_attn_q8_workspace_bytes: shape not taken")
    return n


def fmlp_attn_decode_q8(q, k_q, k_s, v_q, v_s, kv_len, scale: float, out, workspace, stream=None) -> None:
    """out [B, H, D] (f32) <- attention of one token a sequence (queries q [B, H, D] bf16, already rotated) over
    rows 0 .. kv_len[b] - 1 of an int8 cache (codes [B, H_kv, n_max, D], scales [B, H_kv, n_max])."""
    B = _check_batch(None, kv_len)
    H_kv, n_max, D = _check_q8_cache(k_q, k_s, v_q, v_s, B)
    _bf16(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [B, H, D], got {tuple(q.shape)}")
    H = q.shape[1]
    _check(q, "q", torch.bfloat16, (B, H, D))
    _check(out, "out", torch.float32, (B, H, D))
    _check_workspace(workspace, fmlp_attn_q8_workspace_bytes(B, H, H_kv, D))
    _on_device(q=q, k_q=k_q, k_s=k_s, v_q=v_q, v_s=v_s, kv_len=kv_len, out=out, workspace=workspace)
    _check_status(lib.fmlp_attn_decode_q8(q.data_ptr(), k_q.data_ptr(), k_s.data_ptr(), v_q.data_ptr(), v_s.data_ptr(), kv_len.data_ptr(), B, H,
                                          H_kv, D, n_max, scale, out.data_ptr(), workspace.data_ptr(),
                                          workspace.nbytes, _stream(stream)),
                  "fmlp_attn_decode_q8")


NOALLOC_SCRATCH_BYTES = 8 << 20   # FMLP_NOALLOC_SCRATCH_BYTES in include/fmlp.h


def fmlp_forward_noalloc(x, gamma, eps: float, packed, tile_T: int, W_down, out, residual=None,
                         stream=None) -> None:
    """fmlp_forward without a workspace, for callers that cannot allocate device
    memory (the library's own fixed scratch buffer is used; see include/fmlp.h)."""
    M, d, I = _check_forward_args(x, gamma, packed, W_down, out, residual)
    _check(out, "out", torch.float32, (M, d))
    _on_device(x=x, gamma=gamma, packed=packed, W_down=W_down, residual=residual, out=out)
    _check_status(lib.fmlp_forward_noalloc(_ptr(x), M, _ptr(gamma), eps, _ptr(packed), tile_T,
                                           _ptr(W_down), d, I, _ptr(residual), _ptr(out),
                                           _stream(stream)),
                  "fmlp_forward_noalloc")


def fmlp_gate_up_swiglu(x, gamma, eps: float, packed, tile_T: int, a, workspace,
                        stream=None) -> None:
    """a [M x I] (bf16) <- SiLU(gate) * up of RMSNorm(x) against packed gate/up rows."""
    _bf16(x, "x"); _bf16(a, "a")
    M, d = _dims2(x, "x")
    _, I = _dims2(a, "a")
    _check(x, "x", torch.bfloat16, (M, d))
    _check(gamma, "gamma", torch.bfloat16, (d,))
    _check(packed, "packed", torch.bfloat16, (2 * I, d))
    _check(a, "a", torch.bfloat16, (M, I))
    _check_workspace(workspace, fmlp_workspace_bytes(M, d, I))
    _on_device(x=x, gamma=gamma, packed=packed, a=a, workspace=workspace)
    _check_status(lib.fmlp_gate_up_swiglu(_ptr(x), M, _ptr(gamma), eps, _ptr(packed), tile_T, d,
                                          I, _ptr(a), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream)),
                  "fmlp_gate_up_swiglu")


def fmlp_down_proj(a, W_down, out, workspace, residual=None, stream=None) -> None:
    """out [M x d] (f32) <- a [M x I] W_down^T (+ residual)."""
    _bf16(a, "a"); _bf16(W_down, "W_down")
    M, I = _dims2(a, "a")
    d, _ = _dims2(W_down, "W_down")
    _check(a, "a", torch.bfloat16, (M, I))
    _check(W_down, "W_down", torch.bfloat16, (d, I))
    _check(residual, "residual", torch.bfloat16, (M, d), optional=True)
    _check(out, "out", torch.float32, (M, d))
    _check_workspace(workspace, fmlp_workspace_bytes(M, d, I))
    _on_device(a=a, W_down=W_down, residual=residual, out=out, workspace=workspace)
    _check_status(lib.fmlp_down_proj(_ptr(a), M, _ptr(W_down), d, I, _ptr(residual), _ptr(out),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)),
                  "fmlp_down_proj")


def fmlp_device_status(workspace, stream=None) -> int:
    """Synchronise, read and clear the workspace's device status word; returns the status."""
    _check(workspace, "workspace", None)
    _on_device(workspace=workspace)
    return int(lib.fmlp_device_status(_ptr(workspace), _stream(stream)))
