"""ctypes binding of libgdn.so (declared in include/gdn.h): argument marshalling only.

Each function has the C entry point's name, takes torch tensors on a CUDA device,
checks shapes/dtypes/strides, passes raw pointers and the current torch stream, and
raises ``GDNError`` on a non-OK status. Every step of the computation runs in the CUDA
library; there is no CPU or PyTorch fallback. If the library is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, GDN_ERR_TIMEOUT = range(6)
GDN_F32, GDN_BF16 = 0, 1

# name -> (restype, argtypes); mirrors include/gdn.h
_P, _I32, _I64, _F32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "gdn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gdn_last_error": (ctypes.c_char_p, []),
    "gdn_version": (ctypes.c_char_p, []),
    "gdn_conv1d_silu": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, _I32, _I64, _I32, _P, _P, _P]),
    "gdn_chunk_prefill_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32, _I32, ctypes.c_int]),
    "gdn_chunk_prefill": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I32, _I32,
                                          _I32, _I32, _I64, _I64, _P, _I32, _P, _P, _F32, _I32,
                                          _P, _SZ, _P]),
    "gdn_chunk_prefill_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I32, _I32,
                                             _I32, _I32, _I64, _I64, _P, _I32, _P, _P, ctypes.c_int,
                                             _F32, _I32, _I32, _P, _P, _I64, _P, _SZ, _P]),
    "gdn_prefill_status": (ctypes.c_int, [_P, _P]),
    "gdn_prefill_noalloc_status": (ctypes.c_int, [_P]),
    "gdn_decode_step": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _I32, _I32,
                                        _I32, _I32, _I32, _F32, _P]),
    "gdn_decode_tokens": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _I32, _I32, _I32,
                                         _I32, _I32, _I32, _F32, _P]),
    "gdn_decode_step_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.c_int,
                                          _I32, _I32, _I32, _I32, _I32, _F32, _P]),
    "gdn_decode_tokens_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.c_int,
                                            _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P]),
    "gdn_chunk_prefill_path": (_I32, [ctypes.c_int, _I32, _I32, _I32, _I32, _I32]),
    "gdn_chunk_prefill_launches": (_I32, [_I64, _I32, _I32, _I32, _I32, _I32, ctypes.c_int, _I32, _I32]),
    "gdn_chunk_prefill_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I32,
                                                  _I32, _I32, _I32, _I64, _I64, _P, _I32, _P, _P,
                                                  _F32, _I32, _P]),
    "gdn_decode_paged": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _P, _I64, ctypes.c_int, _I32, _P, _P,
                                        _P, _P, _P, _P, _I64, _P, _F32, _P, ctypes.c_int, _I32, _I32,
                                        _I32, _I32, _I32, _I32, _F32, _P]),
    "gdn_pages_copy": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P]),
    "gdn_pages_take": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P]),
    "gdn_pages_ref": (ctypes.c_int, [_P, _I32, _P, _I32, _I32, _P]),
    "gdn_pages_plan": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _P, _P, _P]),
    "gdn_pages_fork": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _I32, _P]),
    "gdn_pages_compact": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _P, _P, _P, _I32, _P]),
    "gdn_gated_norm": (ctypes.c_int, [_P, _P, _I64, _P, _F32, _P, ctypes.c_int, _I64, _I32, _I32, _P]),
    "gdn_gated_norm_bwd": (ctypes.c_int, [_P, _P, _I64, _P, _F32, _P, _P, _P, _I64, _P, ctypes.c_int,
                                          _I64, _I32, _I32, _P, _SZ, _P]),
    "gdn_add_norm": (ctypes.c_int, [_P, _P, _P, _F32, _F32, _F32, _P, ctypes.c_int, _P, ctypes.c_int,
                                    _I64, _I32, _P]),
    "gdn_add_norm_bwd": (ctypes.c_int, [_P, _P, _P, _P, _F32, _F32, _F32, _P, ctypes.c_int, _P, _P,
                                        ctypes.c_int, _I64, _I32, _P, _SZ, _P]),
    "gdn_norm_bwd_workspace_size": (_SZ, [_I32]),
}



class _PagePool(ctypes.Structure):      # gdn_page_pool_t
    _fields_ = [("src", _P), ("dst", _P), ("page_bytes", _I64), ("src_page_stride", _I64),
                ("src_layer_stride", _I64), ("dst_page_stride", _I64), ("dst_layer_stride", _I64),
                ("layers", _I32)]


_lib = None


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {detail}")


def lib() -> ctypes.CDLL:
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgdn.so is not built ({LIB_PATH}); run "
                               "`python -m gated_deltanet_mixer_causal_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdn_status_string(status).decode()


def _check(status: int, where: str):
    if status != GDN_OK:
        raise GDNError(status, where, lib().gdn_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: Optional[torch.Tensor], name: str, shape=None, dtype=None, device=None, dense=True):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gdn_conv1d_silu(x: torch.Tensor, w: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                    conv_state_in: Optional[torch.Tensor] = None,
                    conv_state_out: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Width-4 causal conv + SiLU: x [T, Cc] -> y [T, Cc] (see include/gdn.h)."""
    T, Cc = x.shape
    dev = x.device
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(x, "x", device=dev)
    _need(w, "w", (Cc, 4), x.dtype, dev)
    _need(cu_seqlens, "cu_seqlens", dtype=torch.int32, device=dev)
    _need(conv_state_in, "conv_state_in", (n_seq, 3, Cc), x.dtype, dev)
    _need(conv_state_out, "conv_state_out", (n_seq, 3, Cc), x.dtype, dev)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", (T, Cc), x.dtype, dev)
    _check(lib().gdn_conv1d_silu(_ptr(x), _ptr(y), _dtype_code(x), _ptr(w), _ptr(cu_seqlens),
                                 n_seq, T, Cc, _ptr(conv_state_in), _ptr(conv_state_out),
                                 _stream(dev)), "gdn_conv1d_silu")
    return y


def gdn_chunk_prefill_workspace_size(T: int, n_seq: int, Hk: int, Hv: int, dk: int, dv: int,
                                     dtype: torch.dtype) -> int:
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    n = lib().gdn_chunk_prefill_workspace_size(T, n_seq, Hk, Hv, dk, dv, code)
    if n == ctypes.c_size_t(-1).value:
        raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_chunk_prefill_workspace_size", "unsupported shape")
    return int(n)


PATH_NAMES = {0: "recurrent", 1: "chunked_tc"}


def gdn_chunk_prefill_path(dtype: torch.dtype, Hk: int, Hv: int, dk: int, dv: int,
                           qk_l2norm: bool = True) -> str:
    """Which kernels gdn_chunk_prefill runs for these arguments: "chunked_tc" (the chunked
    form on tcgen05 tensor cores) or "recurrent" (the token-by-token fp32 kernel)."""
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    p = lib().gdn_chunk_prefill_path(code, Hk, Hv, dk, dv, int(bool(qk_l2norm)))
    if p < 0:
        raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_chunk_prefill_path", "unsupported shape")
    return PATH_NAMES[p]


def gdn_chunk_prefill_launches(T: int, n_seq: int, Hk: int, Hv: int, dk: int, dv: int,
                               dtype: torch.dtype, num_sms: int, qk_l2norm: bool = True) -> int:
    """How many of this library's kernels one gdn_chunk_prefill call with these sizes enqueues
    on a GPU of num_sms SMs (host-only, no GPU needed)."""
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    n = lib().gdn_chunk_prefill_launches(T, n_seq, Hk, Hv, dk, dv, code, int(bool(qk_l2norm)), num_sms)
    if n < 0:
        raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_chunk_prefill_launches", "unsupported arguments")
    return int(n)


def _row_view(t: torch.Tensor, name: str):
    """[T, H, d] with unit inner stride and dense heads; returns the token stride."""
    if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError(f"{name} must be [T, H, d] with dense heads (strides (*, d, 1)), "
                         f"got strides {t.stride()}")
    if t.shape[0] > 1 and t.stride(0) == 0:      # 0 stands for a dense tensor in the C ABI
        raise ValueError(f"{name}: tokens must not share memory (expanded), got strides {t.stride()}")
    return t.stride(0)


def gdn_chunk_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                      beta: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                      initial_state: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None, scale: float = 1.0,
                      qk_l2norm: bool = True, o: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, block_tokens: int = 0,
                      block_states: Optional[torch.Tensor] = None,
                      block_rows: Optional[torch.Tensor] = None, check: bool = False) -> torch.Tensor:
    """Gated delta rule over packed sequences (see include/gdn.h). Returns o [T, Hv, dv].

    q, k: [T, Hk, dk] and v: [T, Hv, dv] may be token-strided views (e.g. of the conv
    output). ``final_state`` ([N, Hv, dv, dk]) is written when given. States are fp32, or
    bf16 storage (fp32 math): the dtype of ``initial_state`` / ``final_state`` /
    ``block_states``, which must agree. With ``block_tokens`` > 0 (a multiple of 64) the
    state after every block_tokens tokens of sequence n goes to ``block_states``
    ([R, Hv, dv, dk]) rows block_rows[n], +1, ...
    ``check``: wait for the call and raise GDNError if a bounded device-side wait gave up.
    """
    T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    dev = q.device
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    qs = _row_view(q, "q"); ks = _row_view(k, "k"); vs = _row_view(v, "v")
    if k.shape != q.shape or ks != qs:
        raise ValueError("k must match q in shape and token stride")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dtype=q.dtype, device=dev, dense=False)
    _need(g, "g", (T, Hv), torch.float32, dev)
    _need(beta, "beta", (T, Hv), torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", dtype=torch.int32, device=dev)
    st_dtype = next((t.dtype for t in (initial_state, final_state, block_states if block_tokens else None)
                     if t is not None), torch.float32)
    if st_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"states must be fp32 or bf16, got {st_dtype}")
    _need(initial_state, "initial_state", (n_seq, Hv, dv, dk), st_dtype, dev)
    _need(final_state, "final_state", (n_seq, Hv, dv, dk), st_dtype, dev)
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)
    _need(o, "o", (T, Hv, dv), q.dtype, dev)
    need = gdn_chunk_prefill_workspace_size(T, n_seq, Hk, Hv, dk, dv, q.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    n_rows = 0
    if block_tokens:
        if block_states is None or block_rows is None:
            raise ValueError("block_tokens needs block_states and block_rows")
        _need(block_states, "block_states", dtype=st_dtype, device=dev)
        if tuple(block_states.shape[1:]) != (Hv, dv, dk):
            raise ValueError(f"block_states has shape {tuple(block_states.shape)}, expected [R, {Hv}, {dv}, {dk}]")
        _need(block_rows, "block_rows", (n_seq,), torch.int32, dev)
        n_rows = block_states.shape[0]
    _check(lib().gdn_chunk_prefill_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), _dtype_code(q), T, Hk, Hv, dk, dv,
        qs, vs, _ptr(cu_seqlens), n_seq, _ptr(initial_state), _ptr(final_state),
        GDN_BF16 if st_dtype == torch.bfloat16 else GDN_F32, float(scale),
        int(bool(qk_l2norm)), int(block_tokens), _ptr(block_states if block_tokens else None),
        _ptr(block_rows if block_tokens else None), n_rows, _ptr(workspace), ws_bytes,
        _stream(dev)), "gdn_chunk_prefill")
    if check and workspace is not None:
        gdn_prefill_status(workspace)
    return o


def gdn_prefill_status(workspace: torch.Tensor) -> None:
    """Wait for the last prefill that used ``workspace`` and raise GDNError(GDN_ERR_TIMEOUT)
    if one of its bounded device-side waits gave up (its outputs are then invalid)."""
    _check(lib().gdn_prefill_status(_ptr(workspace), _stream(workspace.device)), "gdn_prefill_status")


def gdn_prefill_noalloc_status(device: Optional[torch.device] = None) -> None:
    """gdn_prefill_status for gdn_chunk_prefill_noalloc's static scratch on ``device``."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().gdn_prefill_noalloc_status(_stream(dev)), "gdn_prefill_noalloc_status")


def gdn_chunk_prefill_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              g: torch.Tensor, beta: torch.Tensor,
                              cu_seqlens: Optional[torch.Tensor] = None,
                              initial_state: Optional[torch.Tensor] = None,
                              final_state: Optional[torch.Tensor] = None, scale: float = 1.0,
                              qk_l2norm: bool = True, o: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gdn_chunk_prefill with the library's static scratch instead of a workspace, for
    callers that cannot allocate device memory (see include/gdn.h for the size limit and
    the rule that overlapping calls race). Pass ``o`` to keep this call allocation-free
    on the Python side as well."""
    T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    dev = q.device
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    qs = _row_view(q, "q"); ks = _row_view(k, "k"); vs = _row_view(v, "v")
    if k.shape != q.shape or ks != qs:
        raise ValueError("k must match q in shape and token stride")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dtype=q.dtype, device=dev, dense=False)
    _need(g, "g", (T, Hv), torch.float32, dev)
    _need(beta, "beta", (T, Hv), torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", dtype=torch.int32, device=dev)
    _need(initial_state, "initial_state", (n_seq, Hv, dv, dk), torch.float32, dev)
    _need(final_state, "final_state", (n_seq, Hv, dv, dk), torch.float32, dev)
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)
    _need(o, "o", (T, Hv, dv), q.dtype, dev)
    # the scratch array is per device: make the tensors' device current for the call
    with torch.cuda.device(dev):
        _check(lib().gdn_chunk_prefill_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), _dtype_code(q), T, Hk, Hv,
            dk, dv, qs, vs, _ptr(cu_seqlens), n_seq, _ptr(initial_state), _ptr(final_state),
            float(scale), int(bool(qk_l2norm)), _stream(dev)), "gdn_chunk_prefill_noalloc")
    return o


def gdn_decode_step(x: torch.Tensor, conv_w: torch.Tensor, conv_state: torch.Tensor,
                    g: torch.Tensor, beta: torch.Tensor, state: torch.Tensor, Hk: int,
                    o: Optional[torch.Tensor] = None, scale: float = 1.0) -> torch.Tensor:
    """One decode token per sequence; conv_state and state are updated in place. The state
    is fp32, or bf16 (stored in bf16, updated in fp32)."""
    B, Cc = x.shape
    _, Hv, dv, dk = state.shape
    dev = x.device
    if Cc != 2 * Hk * dk + Hv * dv:
        raise ValueError(f"x has {Cc} channels, expected 2*Hk*dk + Hv*dv = {2 * Hk * dk + Hv * dv}")
    _need(x, "x", device=dev)
    _need(conv_w, "conv_w", (Cc, 4), x.dtype, dev)
    _need(conv_state, "conv_state", (B, 3, Cc), x.dtype, dev)
    _need(g, "g", (B, Hv), torch.float32, dev)
    _need(beta, "beta", (B, Hv), torch.float32, dev)
    _need(state, "state", (B, Hv, dv, dk), None, dev)
    if o is None:
        o = torch.empty((B, Hv, dv), dtype=x.dtype, device=dev)
    _need(o, "o", (B, Hv, dv), x.dtype, dev)
    _check(lib().gdn_decode_step_ex(_ptr(x), _ptr(conv_w), _ptr(conv_state), _ptr(g), _ptr(beta),
                                    _ptr(state), _dtype_code(state), _ptr(o), _dtype_code(x), B,
                                    Hk, Hv, dk, dv, float(scale), _stream(dev)), "gdn_decode_step")
    return o


def gdn_decode_tokens(x: torch.Tensor, conv_w: torch.Tensor, conv_state: torch.Tensor,
                      g: torch.Tensor, beta: torch.Tensor, state: torch.Tensor, Hk: int,
                      o: Optional[torch.Tensor] = None, scale: float = 1.0) -> torch.Tensor:
    """n_tok (1..8) consecutive tokens per sequence, x [B, n_tok, Cc]; conv_state and state
    (fp32, or bf16 storage) are updated in place. Returns o [B, n_tok, Hv, dv]."""
    B, n_tok, Cc = x.shape
    _, Hv, dv, dk = state.shape
    dev = x.device
    if Cc != 2 * Hk * dk + Hv * dv:
        raise ValueError(f"x has {Cc} channels, expected 2*Hk*dk + Hv*dv = {2 * Hk * dk + Hv * dv}")
    _need(x, "x", device=dev)
    _need(conv_w, "conv_w", (Cc, 4), x.dtype, dev)
    _need(conv_state, "conv_state", (B, 3, Cc), x.dtype, dev)
    _need(g, "g", (B, n_tok, Hv), torch.float32, dev)
    _need(beta, "beta", (B, n_tok, Hv), torch.float32, dev)
    _need(state, "state", (B, Hv, dv, dk), None, dev)
    if o is None:
        o = torch.empty((B, n_tok, Hv, dv), dtype=x.dtype, device=dev)
    _need(o, "o", (B, n_tok, Hv, dv), x.dtype, dev)
    _check(lib().gdn_decode_tokens_ex(_ptr(x), _ptr(conv_w), _ptr(conv_state), _ptr(g), _ptr(beta),
                                      _ptr(state), _dtype_code(state), _ptr(o), _dtype_code(x), B,
                                      n_tok, Hk, Hv, dk, dv, float(scale), _stream(dev)),
           "gdn_decode_tokens")
    return o


# ------------------------------------------------------- paged decode, pages, norms around a block
#
# These calls take a few microseconds on the GPU for a decode batch, so their checks are kept
# cheap: one comparison per tensor where it is as expected, and the reason worked out only where
# it is not.

def _device_of(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _want(t: torch.Tensor, name: str, shape, dtype, device):
    """t is a dense tensor of this shape (a tuple), type and CUDA device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
        return
    _need(t, name, shape, dtype, device)


def _want_view(t: torch.Tensor, name: str, shape, dtype, device):
    """The same without the demand that it is dense."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device.index:
        return
    _need(t, name, shape, dtype, device, dense=False)


_current_stream = torch._C._cuda_getCurrentRawStream      # torch.cuda.current_stream(d).cuda_stream
_functions = {}


def _call(device: torch.device, name: str, *args):
    """lib().<name>(*args, stream) with the tensors' device current, and its status checked."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, _current_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(device.index))
    if status != GDN_OK:
        _check(status, name)


def _int32(n: int, name: str) -> int:
    """n where the C ABI takes 32 bits; ctypes would drop those above without a word."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} = {n} does not fit 32 bits")
    return n


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dense_from(t: torch.Tensor, name: str, dim: int, what: str) -> int:
    """Elements of the dimensions from ``dim`` on, which must be dense."""
    shape, strides, inner = t.shape, t.stride(), 1
    for i in range(len(shape) - 1, dim - 1, -1):
        if shape[i] != 1 and strides[i] != inner:
            raise ValueError(f"{name}: {what} must be dense, got strides {strides}")
        inner *= shape[i]
    return inner


def _apart(t: torch.Tensor, name: str, stride: int, row: int, what: str) -> int:
    """``stride``, which must cover a row: what an expanded tensor repeats has no rows of its own,
    and its stride of 0 would stand for a dense one."""
    if stride < row:
        raise ValueError(f"{name}: {what} must not share memory (expanded or overlapping), got strides {t.stride()}")
    return stride


def _token_rows(t: torch.Tensor, name: str, lead: int) -> int:
    """The token stride of t, whose first ``lead`` (1 or 2) dimensions count tokens that follow
    one another at one stride; the dimensions behind them must be dense. 0 stands for a dense t."""
    if t.is_contiguous():
        return 0
    inner = _dense_from(t, name, lead, "the dimensions behind the tokens")
    shape, strides = t.shape, t.stride()
    if lead == 1:
        return inner if shape[0] <= 1 else _apart(t, name, strides[0], inner, "tokens")
    if shape[1] <= 1:
        return inner if shape[0] <= 1 else _apart(t, name, strides[0], inner, "tokens")
    if shape[0] > 1 and strides[0] != strides[1] * shape[1]:
        raise ValueError(f"{name}: tokens must follow one another at one stride, got strides {strides}")
    return _apart(t, name, strides[1], inner, "tokens")


def _page_stride(t: torch.Tensor, name: str) -> int:
    """The stride in elements between the dense pages of pool t; 0 stands for a dense pool."""
    if t.is_contiguous():
        return 0
    page = _dense_from(t, name, 1, "pages")
    return page if t.shape[0] <= 1 else _apart(t, name, t.stride(0), page, "pages")


def gdn_decode_paged(x: torch.Tensor, conv_w: torch.Tensor, conv_pool: torch.Tensor, state_pool: torch.Tensor,
                     read_pages: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, Hk: int,
                     write_pages: Optional[torch.Tensor] = None, n_valid: Optional[torch.Tensor] = None,
                     z: Optional[torch.Tensor] = None, norm_w: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, o: Optional[torch.Tensor] = None, scale: float = 1.0) -> torch.Tensor:
    """n_tok (1..8) tokens for each of B sequences whose taps and states lie in pages of
    ``conv_pool`` [P, 3, Cc] and ``state_pool`` [P, Hv, dv, dk] (fp32 or bf16 storage): sequence b
    starts from page ``read_pages[b]`` (-1: from zeros); the state after its token t goes to page
    ``write_pages[b, t]`` (-1: nowhere), or without ``write_pages`` the last one back to the page
    it read. x [B, n_tok, Cc] (tokens may be strided, not expanded), g, beta [B, n_tok, Hv]. ``n_valid`` [B]
    limits each sequence's tokens; rows of ``o`` behind them stay as they were (in an ``o`` made
    here they are not defined). With the gate ``z`` [B, n_tok, Hv, dv] and ``norm_w`` [dv] the
    output is gated and normalised as by ``gdn_gated_norm``. A page that one sequence writes must
    not be read or written by another in the same call. Returns o [B, n_tok, Hv, dv]."""
    if x.dim() != 3 or state_pool.dim() != 4:
        raise ValueError("x must be [B, n_tok, Cc] and state_pool [P, Hv, dv, dk]")
    dev, dt = _device_of(x, "x"), x.dtype
    B, n_tok, Cc = x.shape
    P, Hv, dv, dk = state_pool.shape
    if Cc != 2 * Hk * dk + Hv * dv:
        raise ValueError(f"x has {Cc} channels, expected 2*Hk*dk + Hv*dv = {2 * Hk * dk + Hv * dv}")
    f32, i32 = torch.float32, torch.int32
    _want(conv_w, "conv_w", (Cc, 4), dt, dev)
    _want_view(conv_pool, "conv_pool", (P, 3, Cc), dt, dev)
    _want_view(state_pool, "state_pool", (P, Hv, dv, dk), state_pool.dtype, dev)
    _want(read_pages, "read_pages", (B,), i32, dev)
    _want(g, "g", (B, n_tok, Hv), f32, dev)
    _want(beta, "beta", (B, n_tok, Hv), f32, dev)
    if write_pages is not None:
        _want(write_pages, "write_pages", (B, n_tok), i32, dev)
    if n_valid is not None:
        _want(n_valid, "n_valid", (B,), i32, dev)
    if (z is None) != (norm_w is None):
        raise ValueError("z and norm_w come together")
    z_stride = 0
    if z is not None:
        _want_view(z, "z", (B, n_tok, Hv, dv), dt, dev)
        _want(norm_w, "norm_w", (dv,), dt, dev)
        z_stride = _token_rows(z, "z", 2)
    if o is None:
        o = torch.empty((B, n_tok, Hv, dv), dtype=dt, device=dev)
    else:
        _want(o, "o", (B, n_tok, Hv, dv), dt, dev)
    _call(dev, "gdn_decode_paged", x.data_ptr(), _token_rows(x, "x", 2), conv_w.data_ptr(), conv_pool.data_ptr(),
          _page_stride(conv_pool, "conv_pool"), state_pool.data_ptr(), _page_stride(state_pool, "state_pool"),
          _dtype_code(state_pool), P, read_pages.data_ptr(), _addr(write_pages), _addr(n_valid), g.data_ptr(),
          beta.data_ptr(), _addr(z), z_stride, _addr(norm_w), eps, o.data_ptr(), _dtype_code(x), B, n_tok, Hk, Hv,
          dk, dv, scale)
    return o


def _pool_layout(t: torch.Tensor, name: str, page_dim: int):
    """(pages, layers, page bytes, page stride, layer stride) in bytes of a pool [P, page..]
    (page_dim 0) or [layers, P, page..] (page_dim 1)."""
    shape = t.shape
    if len(shape) < page_dim + 2:
        raise ValueError(f"{name} has {len(shape)} dimensions, too few for page_dim = {page_dim}")
    es, strides = t.element_size(), t.stride()
    pages, layers = _int32(shape[page_dim], "pages"), _int32(shape[0], "layers") if page_dim else 1
    if pages > 1 and t.is_contiguous():
        page = strides[page_dim] * es
    else:
        page = _dense_from(t, name, page_dim + 1, "pages") * es
        if pages > 1:
            _apart(t, name, strides[page_dim] * es, page, "pages")
        if layers > 1:
            _apart(t, name, strides[0] * es, page, "layers")
    return pages, layers, page, strides[page_dim] * es if pages > 1 else page, strides[0] * es if layers > 1 else 0


def _describe(froms, tos, page_dim: int, device: torch.device):
    """The pools of a copy as gdn_pages_copy takes them: (array, source pages, destination pages)."""
    if page_dim not in (0, 1):
        raise ValueError(f"page_dim must be 0 or 1, got {page_dim}")
    if not 1 <= len(froms) <= 4 or len(tos) != len(froms):
        raise ValueError(f"expected 1 to 4 pools and as many destinations, got {len(froms)} and {len(tos)}")
    desc = (_PagePool * len(froms))()
    sp = dp = None
    for d, a, b in zip(desc, froms, tos):
        pages, layers, size, stride, layer = _pool_layout(a, "src_pool", page_dim)
        d.src, d.page_bytes, d.src_page_stride, d.src_layer_stride, d.layers = a.data_ptr(), size, stride, layer, layers
        bad = size <= 0 or (size | stride | layer | a.data_ptr()) & 15
        to_pages = pages
        if b is not a:
            to_pages, to_layers, to_size, stride, layer = _pool_layout(b, "dst_pool", page_dim)
            if b.dtype != a.dtype or to_layers != layers or to_size != size:
                raise ValueError("source and destination pools must agree in dtype, layers and page size")
            bad |= (stride | layer | b.data_ptr()) & 15
        d.dst, d.dst_page_stride, d.dst_layer_stride = b.data_ptr(), stride, layer
        if bad:
            raise ValueError("pages must begin at, and be, multiples of 16 bytes")
        if a.device != device or b.device != device or sp not in (None, pages) or dp not in (None, to_pages):
            raise ValueError("all pools must be on the lists' device and agree in their number of pages")
        sp, dp = pages, to_pages
    return desc, sp, dp


def _pool_list(pools):
    return [pools] if isinstance(pools, torch.Tensor) else list(pools)


def _describe_counted(refs: torch.Tensor, pools, page_dim: int):
    """_describe for pools whose pages ``refs`` counts."""
    pools = _pool_list(pools)
    desc, pages, _ = _describe(pools, pools, page_dim, _device_of(refs, "refs"))
    if pages != refs.numel():
        raise ValueError(f"the pools have {pages} pages, refs has {refs.numel()}")
    return desc, pages


def gdn_pages_copy(src_pool, src: torch.Tensor, dst: torch.Tensor, dst_pool=None, page_dim: int = 0,
                   plain: bool = False) -> None:
    """Page src[i] of ``src_pool`` to page dst[i] of ``dst_pool`` (default: the same pool) for
    every entry of the int32 lists, as if all were read before any is written; the last entry of
    a repeated destination counts, entries that are not pages are skipped. Pools are [P, page..],
    or [layers, P, page..] with ``page_dim`` = 1 (every layer is copied); a list of up to four
    pools with equal P is copied by one call. ``plain``: no destination is named twice or is
    another entry's source (faster)."""
    froms = _pool_list(src_pool)
    n, dev = _int32(src.numel(), "n"), _device_of(src, "src")
    _want(src, "src", (n,), torch.int32, dev)
    _want(dst, "dst", (n,), torch.int32, dev)
    desc, sp, dp = _describe(froms, froms if dst_pool is None else _pool_list(dst_pool), page_dim, dev)
    _call(dev, "gdn_pages_copy", ctypes.addressof(desc), len(desc), sp, dp, src.data_ptr(), dst.data_ptr(), n,
          int(bool(plain)))


def gdn_pages_take(refs: torch.Tensor, n: Optional[int] = None, src: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Take the lowest free pages (count 0 in ``refs`` [P] int32), whose counts become 1: ``n`` of
    them, or one for each entry of ``src`` that is a page in use. Returns them (int32, -1: none)."""
    if (n is None) == (src is None):
        raise ValueError("give either n or src")
    n = _int32(n if src is None else src.numel(), "n")
    dev, P = _device_of(refs, "refs"), _int32(refs.numel(), "pages")
    _want(refs, "refs", (P,), torch.int32, dev)
    if src is not None:
        _want(src, "src", (n,), torch.int32, dev)
    if out is None:
        out = torch.empty((n,), dtype=torch.int32, device=dev)
    else:
        _want(out, "out", (n,), torch.int32, dev)
    _call(dev, "gdn_pages_take", refs.data_ptr(), P, _addr(src), n, out.data_ptr())
    return out


def gdn_pages_ref(refs: torch.Tensor, pages: torch.Tensor, delta: int) -> None:
    """refs[p] += delta for every entry p of ``pages`` that is a page, not below 0: 1 shares
    pages, -1 frees them."""
    delta = _int32(int(delta), "delta")
    dev, P, n = _device_of(refs, "refs"), _int32(refs.numel(), "pages"), _int32(pages.numel(), "n")
    _want(refs, "refs", (P,), torch.int32, dev)
    _want(pages, "pages", (n,), torch.int32, dev)
    _call(dev, "gdn_pages_ref", refs.data_ptr(), P, pages.data_ptr(), n, delta)


def gdn_pages_fork(refs: torch.Tensor, src: torch.Tensor, pools, page_dim: int = 0,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A new page for each entry of ``src`` (see ``gdn_pages_take``), holding a copy of page
    src[i] in each pool of ``pools``. Returns the new pages. A refused call changes nothing."""
    desc, P = _describe_counted(refs, pools, page_dim)
    dev, n = refs.device, _int32(src.numel(), "n")
    _want(refs, "refs", (P,), torch.int32, dev)
    _want(src, "src", (n,), torch.int32, dev)
    if out is None:
        out = torch.empty((n,), dtype=torch.int32, device=dev)
    else:
        _want(out, "out", (n,), torch.int32, dev)
    _call(dev, "gdn_pages_fork", refs.data_ptr(), P, src.data_ptr(), n, out.data_ptr(), ctypes.addressof(desc), len(desc))
    return out


def _plan_lists(refs: torch.Tensor, table: Optional[torch.Tensor]):
    """What gdn_pages_plan writes, src | dst | map | n_live in one tensor, and the call's arguments."""
    dev, P = _device_of(refs, "refs"), _int32(refs.numel(), "pages")
    _want(refs, "refs", (P,), torch.int32, dev)
    if table is not None:
        _want(table, "table", table.shape, torch.int32, dev)
    half = P // 2
    lists = torch.empty((2 * half + P + 1,), dtype=torch.int32, device=dev)
    at = lists.data_ptr()
    return lists, half, (refs.data_ptr(), P, _addr(table), 0 if table is None else _int32(table.numel(), "table entries"),
                         at, at + 4 * half, at + 8 * half, at + 8 * half + 4 * P)


def gdn_pages_plan(refs: torch.Tensor, table: Optional[torch.Tensor] = None):
    """The moves that bring the live pages (count > 0) to the front: (src, dst, map, n_live), the
    lists padded with -1; refs and the page numbers in ``table`` (any shape) are rewritten."""
    lists, half, args = _plan_lists(refs, table)
    _call(refs.device, "gdn_pages_plan", *args)
    return lists[:half], lists[half:2 * half], lists[2 * half:-1], lists[-1:]


def gdn_pages_compact(refs: torch.Tensor, table: Optional[torch.Tensor], pools, page_dim: int = 0):
    """Bring the live pages to the front of every pool: ``refs`` and ``table`` are rewritten.
    Returns (map [P]: each live page's new place, -1 for free ones; n_live [1]), on the device.
    A refused call changes nothing."""
    desc, _ = _describe_counted(refs, pools, page_dim)
    lists, half, args = _plan_lists(refs, table)
    _call(refs.device, "gdn_pages_compact", *args, ctypes.addressof(desc), len(desc))
    return lists[2 * half:-1], lists[-1:]


@functools.lru_cache(maxsize=None)
def gdn_norm_bwd_workspace_size(D: int) -> int:
    """Bytes of workspace the norms' backward passes need for rows of D values."""
    return int(lib().gdn_norm_bwd_workspace_size(D))


def _norm_workspace(D: int, workspace: Optional[torch.Tensor], device):
    if workspace is None:
        need = gdn_norm_bwd_workspace_size(D)
        return torch.empty(need, dtype=torch.uint8, device=device), need
    _need(workspace, "workspace", device=device)
    return workspace, workspace.numel() * workspace.element_size()


def _check_gate(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor, eps: float) -> None:
    """Raises what gdn_gated_norm(o, z, w, eps, y=o) would raise, and launches nothing."""
    dev, dt, shape = _device_of(o, "o"), o.dtype, o.shape
    T, Hv, dv = shape
    _want(o, "o", shape, dt, dev)
    _want_view(z, "z", shape, dt, dev)
    _want(w, "w", (dv,), dt, dev)
    stride = _token_rows(z, "z", 1)
    _call(dev, "gdn_gated_norm", o.data_ptr(), z.data_ptr(), stride, w.data_ptr(), eps, o.data_ptr(), _dtype_code(o), 0,
          Hv, dv)                                                # a call of no tokens checks all but overlaps
    es, row, at = o.element_size(), Hv * dv, o.data_ptr()
    for name, t, size in (("z", z, (T - 1) * (stride or row) + row), ("w", w, dv)):
        if T > 0 and at < t.data_ptr() + size * es and t.data_ptr() < at + T * row * es:
            raise GDNError(GDN_ERR_INVALID_ARG, "gdn_gated_norm", f"o overlaps {name}")


def gdn_gated_norm(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor, eps: float = 1e-6,
                   y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o / sqrt(mean(o^2) + eps) * w * SiLU(z) over the last dimension: o [T, Hv, dv], z the same
    (tokens may be strided, not expanded), w [dv]. ``y`` may be ``o``."""
    dev, dt, shape = _device_of(o, "o"), o.dtype, o.shape
    T, Hv, dv = shape
    _int32(Hv, "Hv")
    _want(o, "o", shape, dt, dev)
    _want_view(z, "z", shape, dt, dev)
    _want(w, "w", (dv,), dt, dev)
    if y is None:
        y = torch.empty_like(o)
    else:
        _want(y, "y", shape, dt, dev)
    _call(dev, "gdn_gated_norm", o.data_ptr(), z.data_ptr(), _token_rows(z, "z", 1), w.data_ptr(), eps, y.data_ptr(),
          _dtype_code(o), T, Hv, dv)
    return y


def gdn_gated_norm_bwd(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, eps: float = 1e-6,
                       do: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                       dw: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Backward of ``gdn_gated_norm``: (do, dz, dw [dv] fp32). ``do`` may be ``dy``; ``dz`` may be
    a token-strided view."""
    dev, dt, shape = _device_of(o, "o"), o.dtype, o.shape
    T, Hv, dv = shape
    _int32(Hv, "Hv")
    do = torch.empty_like(o) if do is None else do
    dz = torch.empty(shape, dtype=dt, device=dev) if dz is None else dz
    dw = torch.empty((dv,), dtype=torch.float32, device=dev) if dw is None else dw
    _want(o, "o", shape, dt, dev)
    _want_view(z, "z", shape, dt, dev)
    _want(w, "w", (dv,), dt, dev)
    _want(dy, "dy", shape, dt, dev)
    _want(do, "do", shape, dt, dev)
    _want_view(dz, "dz", shape, dt, dev)
    _want(dw, "dw", (dv,), torch.float32, dev)
    workspace, ws_bytes = _norm_workspace(dv, workspace, dev)
    _call(dev, "gdn_gated_norm_bwd", o.data_ptr(), z.data_ptr(), _token_rows(z, "z", 1), w.data_ptr(), eps,
          dy.data_ptr(), do.data_ptr(), dz.data_ptr(), _token_rows(dz, "dz", 1), dw.data_ptr(), _dtype_code(o), T, Hv,
          dv, workspace.data_ptr(), ws_bytes)
    return do, dz, dw


def gdn_add_norm(x: torch.Tensor, residual: torch.Tensor, w: torch.Tensor, scale: float = 1.0, w_add: float = 0.0,
                 eps: float = 1e-6, h: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None):
    """h = residual + scale * x and its norm n = h / sqrt(mean(h^2) + eps) * (w + w_add), over the
    last of two dimensions. h has the residual's dtype and may be ``residual``; n has x's.
    Returns (n, h)."""
    dev, dt, shape, res = _device_of(x, "x"), x.dtype, x.shape, residual.dtype
    T, D = shape
    _int32(D, "D")
    h = torch.empty_like(residual) if h is None else h
    n = torch.empty_like(x) if n is None else n
    _want(x, "x", shape, dt, dev)
    _want(residual, "residual", shape, res, dev)
    _want(w, "w", (D,), dt, dev)
    _want(h, "h", shape, res, dev)
    _want(n, "n", shape, dt, dev)
    _call(dev, "gdn_add_norm", x.data_ptr(), residual.data_ptr(), w.data_ptr(), scale, w_add, eps, h.data_ptr(),
          _dtype_code(residual), n.data_ptr(), _dtype_code(x), T, D)
    return n, h


def gdn_add_norm_bwd(h: torch.Tensor, w: torch.Tensor, dn: torch.Tensor, dh: Optional[torch.Tensor] = None,
                     scale: float = 1.0, w_add: float = 0.0, eps: float = 1e-6,
                     dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                     dw: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Backward of ``gdn_add_norm`` at the h it stored: from dn and dh (the gradient that reaches
    h on its own way, or None) the gradients (dx, dres, dw [D] fp32) of x, the residual and w.
    ``dres`` may be ``dh``; dx has dn's dtype (x, w, n and dx share it)."""
    dev, dt, shape, res = _device_of(h, "h"), dn.dtype, h.shape, h.dtype
    T, D = shape
    _int32(D, "D")
    dres = torch.empty_like(h) if dres is None else dres
    dx = torch.empty_like(dn) if dx is None else dx
    dw = torch.empty((D,), dtype=torch.float32, device=dev) if dw is None else dw
    _want(h, "h", shape, res, dev)
    _want(w, "w", (D,), dt, dev)
    _want(dn, "dn", shape, dt, dev)
    if dh is not None:
        _want(dh, "dh", shape, res, dev)
    _want(dres, "dres", shape, res, dev)
    _want(dx, "dx", shape, dt, dev)
    _want(dw, "dw", (D,), torch.float32, dev)
    workspace, ws_bytes = _norm_workspace(D, workspace, dev)
    _call(dev, "gdn_add_norm_bwd", h.data_ptr(), w.data_ptr(), dn.data_ptr(), _addr(dh), scale, w_add, eps,
          dres.data_ptr(), _dtype_code(h), dx.data_ptr(), dw.data_ptr(), _dtype_code(dn), T, D, workspace.data_ptr(),
          ws_bytes)
    return dx, dres, dw
