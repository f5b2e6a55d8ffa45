"""Python binding of the ditattn C ABI (include/ditattn.h): argument marshalling only.

Every step of attention runs in the library's CUDA kernels; this module checks
shapes/dtypes, allocates outputs with PyTorch when the caller does not pass
them, and hands raw pointers plus the current CUDA stream to the C entry
points.  There is no CPU fallback: without the built library or a CUDA device
every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

from . import build as _build

DIT_OK, DIT_ERR_INVALID_ARG, DIT_ERR_UNSUPPORTED, DIT_ERR_CUDA, DIT_ERR_TIMEOUT = range(5)
DIT_F32, DIT_BF16 = 0, 1

EXPORTED_SYMBOLS = ("dit_attn_fwd", "dit_attn_fwd_strided", "dit_attn_chunk_fwd", "dit_attn_chunks_fwd",
                    "dit_attn_chunk_fwd_accumulate", "dit_attn_lse_merge", "dit_layout_copy",
                    "dit_attn_stale_kv_fwd", "dit_attn_chunk_fwd_splitkv",
                    "dit_attn_splitkv_workspace_bytes", "dit_attn_splitkv_suggest",
                    "dit_attn_chunk_fwd_splitkv_noalloc",
                    "dit_qk_norm_rope", "dit_paged_plan", "dit_paged_kv_write", "dit_paged_attn_fwd",
                    "dit_paged_attn_workspace_bytes", "dit_paged_prefill_fwd",
                    "dit_paged_prefill_workspace_bytes", "dit_paged_page_mass", "dit_paged_evict",
                    "dit_paged_evict_workspace_bytes", "dit_paged_select",
                    "dit_paged_select_workspace_bytes", "dit_attn_check", "dit_test_inject_stall", "dit_test_set_grid_limit",
                    "dit_status_string", "dit_version")


class Strides(ctypes.Structure):
    """dit_strides: element strides (b, h, n) of a [B, H, N, D] view with contiguous D."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("n", ctypes.c_longlong)]

_lib = None


class DitError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libditattn.so (built in-tree by __graft_entry__.build()); raises if it is missing."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(path)
        P, I, LL, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        L.dit_attn_fwd.restype = I
        L.dit_attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, F, I, P]
        SP = ctypes.POINTER(Strides)
        L.dit_attn_fwd_strided.restype = I
        L.dit_attn_fwd_strided.argtypes = [P, SP, P, SP, P, SP, P, SP, P, I, I, I, I, I, F, I, P]
        L.dit_attn_stale_kv_fwd.restype = I
        L.dit_attn_stale_kv_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P,
                                            ctypes.c_size_t, P]
        L.dit_attn_chunk_fwd_splitkv.restype = I
        L.dit_attn_chunk_fwd_splitkv.argtypes = [P, P, P, P, P, I, I, I, I, I, LL, F, I, I, P,
                                                 ctypes.c_size_t, P]
        L.dit_attn_chunk_fwd_splitkv_noalloc.restype = I
        L.dit_attn_chunk_fwd_splitkv_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, LL, F, I,
                                                         I, P]
        L.dit_attn_splitkv_workspace_bytes.restype = ctypes.c_size_t
        L.dit_attn_splitkv_workspace_bytes.argtypes = [I, I, I, I, I]
        L.dit_attn_splitkv_suggest.restype = I
        L.dit_attn_splitkv_suggest.argtypes = [I, I, I, I]
        L.dit_layout_copy.restype = I
        L.dit_layout_copy.argtypes = [P, SP, P, SP, I, I, I, I, I, P]
        L.dit_attn_chunk_fwd.restype = I
        L.dit_attn_chunk_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, LL, F, I, P]
        L.dit_attn_chunks_fwd.restype = I
        L.dit_attn_chunks_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, LL, I, ctypes.POINTER(I), F,
                                          I, P]
        L.dit_attn_chunk_fwd_accumulate.restype = I
        L.dit_attn_chunk_fwd_accumulate.argtypes = [P, P, P, P, P, I, I, I, I, I, LL, F, P]
        L.dit_attn_lse_merge.restype = I
        L.dit_attn_lse_merge.argtypes = [P, P, I, P, P, I, I, I, I, I, I, P]
        L.dit_qk_norm_rope.restype = I
        L.dit_qk_norm_rope.argtypes = [P, SP, P, SP, I, P, SP, P, SP, I, I, F, P, P, I, P, ctypes.POINTER(I), I, I, F, P, LL,
                                       LL, P, P, I, I, I, I, P]
        L.dit_paged_plan.restype = I
        L.dit_paged_plan.argtypes = [P, P, P, LL, P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.dit_paged_kv_write.restype = I
        L.dit_paged_kv_write.argtypes = [P, SP, P, SP, P, P, SP, P, SP, P, I, I, I, I, I, P]
        L.dit_paged_attn_fwd.restype = I
        L.dit_paged_attn_fwd.argtypes = [P, SP, P, SP, P, SP, P, LL, P, P, I, P, P, I, I, I, I, I, I,
                                         I, F, I, P, ctypes.c_size_t, P]
        L.dit_paged_attn_workspace_bytes.restype = ctypes.c_size_t
        L.dit_paged_attn_workspace_bytes.argtypes = [I, I, I, I, I, I]
        L.dit_paged_prefill_fwd.restype = I
        L.dit_paged_prefill_fwd.argtypes = [P, SP, P, SP, P, SP, P, LL, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I,
                                            P, ctypes.c_size_t, P]
        L.dit_paged_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.dit_paged_prefill_workspace_bytes.argtypes = [I, I, I]
        L.dit_paged_page_mass.restype = I
        L.dit_paged_page_mass.argtypes = [P, SP, P, P, SP, P, LL, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P]
        L.dit_paged_evict.restype = I
        L.dit_paged_evict.argtypes = [P, P, LL, P, LL, P, P, P, P, P, I, I, I, I, I, I, I, I, P, ctypes.c_size_t, P]
        L.dit_paged_evict_workspace_bytes.restype = ctypes.c_size_t
        L.dit_paged_evict_workspace_bytes.argtypes = [I, I]
        L.dit_paged_select.restype = I
        L.dit_paged_select.argtypes = [P, SP, P, P, LL, P, P, I, I, I, I, I, I, I, I, P,
                                       ctypes.c_size_t, P]
        L.dit_paged_select_workspace_bytes.restype = ctypes.c_size_t
        L.dit_paged_select_workspace_bytes.argtypes = [I, I, I]
        L.dit_attn_check.restype = I
        L.dit_attn_check.argtypes = [P]
        L.dit_test_inject_stall.restype = None
        L.dit_test_inject_stall.argtypes = [I, LL]
        L.dit_test_set_grid_limit.restype = None
        L.dit_test_set_grid_limit.argtypes = [I]
        L.dit_status_string.restype = ctypes.c_char_p
        L.dit_status_string.argtypes = [I]
        L.dit_version.restype = I
        L.dit_version.argtypes = []
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().dit_status_string(int(status)).decode()


def _dt(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return DIT_F32
    if dtype == torch.bfloat16:
        return DIT_BF16
    raise TypeError(f"unsupported output dtype {dtype}; use torch.float32 or torch.bfloat16")


def _stream(device: torch.device, stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, H, N, D]")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous [B, H, N, D]")


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _check_out(out, lse, shape, device, out_name="out", lse_name="lse", contiguous=True):
    """Caller-provided outputs: `out` a [shape] fp32 or bf16 tensor and `lse` a contiguous fp32
    [shape[:-1]] tensor, both on `device` (the C ABI cannot see buffer sizes, so a wrong shape,
    dtype, layout or device must be stopped here).  `contiguous=False` lets `out` be any view
    whose last dimension is contiguous (the strided entry point checks the strides itself)."""
    shape = tuple(int(x) for x in shape)
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.device != device:
            raise ValueError(f"{out_name} must be a tensor on {device}")
        if tuple(out.shape) != shape:
            raise ValueError(f"{out_name} must have shape {list(shape)}, got {list(out.shape)}")
        if out.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"{out_name} must be float32 or bfloat16, got {out.dtype}")
        if contiguous and not out.is_contiguous():
            raise ValueError(f"{out_name} must be contiguous")
        if not contiguous and out.stride(-1) != 1:
            raise ValueError(f"{out_name} must have a contiguous last dimension")
    if lse is not None:
        if not isinstance(lse, torch.Tensor) or lse.device != device:
            raise ValueError(f"{lse_name} must be a tensor on {device}")
        if tuple(lse.shape) != shape[:-1]:
            raise ValueError(f"{lse_name} must have shape {list(shape[:-1])}, "
                             f"got {list(lse.shape)}")
        if lse.dtype != torch.float32:
            raise ValueError(f"{lse_name} must be float32, got {lse.dtype}")
        if not lse.is_contiguous():
            raise ValueError(f"{lse_name} must be contiguous")


def attn_fwd(q, k, v, out=None, lse=None, scale=None, out_dtype=torch.float32, stream=None,
             with_lse=True):
    """Fused attention over all keys.  q, k, v: CUDA bf16 [B, H, N, D] contiguous.

    Returns (out [B, H, N, D] of out_dtype, lse fp32 [B, H, N]); with_lse=False skips the
    LSE (the library gets NULL) and returns (out, None).
    """
    _check_qkv(q, k, v)
    if not (k.is_contiguous() and v.is_contiguous()) or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("k and v must be contiguous with q's shape")
    B, H, N, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check_out(out, lse, (B, H, N, D), q.device)
    if out is None:
        out = torch.empty((B, H, N, D), device=q.device, dtype=out_dtype)
    if lse is None and with_lse:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        st = lib().dit_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                _ptr(lse) if with_lse else None, B, H, N, D, scale,
                                _dt(out.dtype), _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_fwd")
    return out, (lse if with_lse else None)


def view_strides(x: torch.Tensor) -> Strides:
    """dit_strides of a [B, H, N, D] tensor view whose last dimension is contiguous (e.g. a
    token-major [B, N, H, D] tensor passed as x.transpose(1, 2))."""
    if x.dim() != 4 or x.stride(3) != 1:
        raise ValueError("expected a [B, H, N, D] view with contiguous last dimension")
    return Strides(*(int(s) for s in x.stride()[:3]))


def attn_fwd_strided(q, k, v, out=None, lse=None, scale=None, out_dtype=torch.float32,
                     stream=None):
    """Attention over arbitrary strided [B, H, N, D] views (last dimension contiguous): q is
    [B, H, N_q, D], k and v [B, H, n_kv, D].  A BSND tensor x ([B, N, H, D] in memory) is passed as
    x.transpose(1, 2), and `out` may be such a view too.  Returns (out, lse fp32 [B, H, N_q])."""
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4:
            raise ValueError("q, k, v must be 4-D bf16 CUDA tensor views")
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v must be [B, H, n_kv, D] matching q")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, H, Nq, D), device=q.device, dtype=out_dtype)
    _check_out(out, lse, (B, H, Nq, D), q.device, contiguous=False)
    if lse is None:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    qs, ks, vs, os_ = (view_strides(t) for t in (q, k, v, out))
    with torch.cuda.device(q.device):
        st = lib().dit_attn_fwd_strided(_ptr(q), ctypes.byref(qs), _ptr(k), ctypes.byref(ks),
                                        _ptr(v), ctypes.byref(vs), _ptr(out), ctypes.byref(os_),
                                        _ptr(lse), B, H, Nq, k.shape[2], D, scale, _dt(out.dtype),
                                        _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_fwd_strided")
    return out, lse


def layout_copy(src, dst, stream=None):
    """dst[...] = src[...] for two [B, H, N, D] views of the same shape and dtype (bf16 or fp32,
    last dimension contiguous), by the library's strided copy kernel.  Returns dst."""
    if not (src.is_cuda and dst.is_cuda) or src.device != dst.device:
        raise ValueError("src and dst must be CUDA tensors on one device")
    if src.shape != dst.shape or src.dtype != dst.dtype or src.dim() != 4:
        raise ValueError("src and dst must be [B, H, N, D] views of one shape and dtype")
    B, H, N, D = src.shape
    ss, ds = view_strides(src), view_strides(dst)
    with torch.cuda.device(src.device):
        st = lib().dit_layout_copy(_ptr(src), ctypes.byref(ss), _ptr(dst), ctypes.byref(ds), B, H,
                                   N, D, _dt(src.dtype), _stream(src.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_layout_copy")
    return dst


def bsnd_to_bhnd(x, out=None, stream=None):
    """Token-major [B, N, H, D] -> contiguous head-major [B, H, N, D]."""
    B, N, H, D = x.shape
    if out is None:
        out = torch.empty((B, H, N, D), device=x.device, dtype=x.dtype)
    layout_copy(x.transpose(1, 2), out, stream=stream)
    return out


def bhnd_to_bsnd(x, out=None, stream=None):
    """Head-major [B, H, N, D] -> contiguous token-major [B, N, H, D]."""
    B, H, N, D = x.shape
    if out is None:
        out = torch.empty((B, N, H, D), device=x.device, dtype=x.dtype)
    layout_copy(x, out.transpose(1, 2), stream=stream)
    return out


def ulysses_pack(x_local, p, out=None, stream=None):
    """Send buffers of one rank's Ulysses all-to-all: its token shard x_local [B, N/p, H, D]
    (token-major) split by head groups into out [p, B, N/p, H/p, D], out[r] = the heads
    r*H/p .. (r+1)*H/p that rank r will own.  One strided copy per destination rank."""
    B, n, H, D = x_local.shape
    if H % p:
        raise ValueError("Ulysses needs the head count divisible by the degree")
    hp = H // p
    if out is None:
        out = torch.empty((p, B, n, hp, D), device=x_local.device, dtype=x_local.dtype)
    for r in range(p):
        layout_copy(x_local[:, :, r * hp:(r + 1) * hp].transpose(1, 2), out[r].transpose(1, 2),
                    stream=stream)
    return out


def ulysses_unpack(recv, out=None, stream=None):
    """Receive side: recv [p, B, N/p, H/p, D], recv[r] = the token shard of rank r for this
    rank's head group, assembled into all tokens of those heads, out [B, N, H/p, D]
    (token-major; pass out.transpose(1, 2) to the attention as a [B, H/p, N, D] view)."""
    p, B, n, hp, D = recv.shape
    if out is None:
        out = torch.empty((B, p * n, hp, D), device=recv.device, dtype=recv.dtype)
    for r in range(p):
        layout_copy(recv[r].transpose(1, 2), out[:, r * n:(r + 1) * n].transpose(1, 2),
                    stream=stream)
    return out


def splitkv_plan(B, H, n_q, n_kv, D, device, splits=None, workspace=None):
    """(splits, workspace) for a split-KV call: the library's suggestion when splits is None,
    and a fresh torch workspace of the required size unless one is given."""
    with torch.cuda.device(device):
        if splits is None:
            splits = int(lib().dit_attn_splitkv_suggest(B, H, n_q, n_kv))
        need = int(lib().dit_attn_splitkv_workspace_bytes(B, H, n_q, D, splits))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if need and (workspace.numel() * workspace.element_size() < need or not workspace.is_cuda):
        raise ValueError(f"workspace must be a CUDA buffer of at least {need} bytes")
    return splits, workspace


def attn_chunk_fwd_splitkv(q, k, v, out=None, lse=None, scale=None, out_dtype=torch.float32,
                           splits=None, workspace=None, stream=None):
    """dit_attn_chunk_fwd with each (head, Q pair) split over key ranges into fp32 partials in
    `workspace` and merged (for few queries against many keys).  splits=None asks the library;
    the workspace is allocated with torch unless given.  Returns (out, lse)."""
    _check_qkv(q, k, v)
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v chunk must be [B, H, n_kv, D] matching q")
    hs = kv_head_stride(k)
    if kv_head_stride(v) != hs:
        raise ValueError("k and v chunks must have the same head stride")
    n_kv = k.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check_out(out, lse, (B, H, Nq, D), q.device)
    if out is None:
        out = torch.empty((B, H, Nq, D), device=q.device, dtype=out_dtype)
    if lse is None:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    splits, workspace = splitkv_plan(B, H, Nq, n_kv, D, q.device, splits, workspace)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with torch.cuda.device(q.device):
        st = lib().dit_attn_chunk_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H,
                                              Nq, n_kv, D, hs, scale, _dt(out.dtype), splits,
                                              ws_ptr, ws_bytes, _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_chunk_fwd_splitkv")
    return out, lse


def attn_chunk_fwd_splitkv_noalloc(q, k, v, out, lse, scale=None, splits=None, stream=None):
    """Split-KV attention into the caller's out / lse with the library's fixed device scratch:
    no allocation on this path (out and lse are required).  splits=None asks the library.
    Calls overlapping in time race on the one scratch array."""
    _check_qkv(q, k, v)
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v chunk must be [B, H, n_kv, D] matching q")
    hs = kv_head_stride(k)
    if kv_head_stride(v) != hs:
        raise ValueError("k and v chunks must have the same head stride")
    n_kv = k.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None or lse is None:
        raise ValueError("out and lse are required: this path allocates nothing")
    _check_out(out, lse, (B, H, Nq, D), q.device)
    with torch.cuda.device(q.device):
        if splits is None:
            splits = int(lib().dit_attn_splitkv_suggest(B, H, Nq, n_kv))
        st = lib().dit_attn_chunk_fwd_splitkv_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                                      _ptr(lse), B, H, Nq, n_kv, D, hs, scale,
                                                      _dt(out.dtype), splits,
                                                      _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_chunk_fwd_splitkv_noalloc")
    return out, lse


def stale_kv_attention(q, k_new, v_new, k_buf, v_buf, row0, out=None, lse=None, scale=None,
                       out_dtype=torch.float32, splits=1, workspace=None, stream=None):
    """One patch of displaced patch parallelism: the patch's fresh K/V rows [row0, row0 + m)
    overwrite their stale rows of the KV buffers (in place), then its m queries attend to all N
    buffer rows.  q, k_new, v_new [B, H, m, D]; k_buf, v_buf [B, H, N, D]; all bf16, contiguous.
    splits: key ranges of the attention (1: none; None: the library's suggestion).
    Returns (out [B, H, m, D], lse fp32 [B, H, m])."""
    for t in (q, k_new, v_new, k_buf, v_buf):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError("q, k_new, v_new, k_buf, v_buf must be contiguous 4-D bf16 CUDA tensors")
    B, H, m, D = q.shape
    N = k_buf.shape[2]
    if k_new.shape != q.shape or v_new.shape != q.shape or v_buf.shape != k_buf.shape \
            or tuple(k_buf.shape[:2]) != (B, H) or k_buf.shape[3] != D:
        raise ValueError("shape mismatch between the patch and the KV buffers")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check_out(out, lse, (B, H, m, D), q.device)
    if out is None:
        out = torch.empty((B, H, m, D), device=q.device, dtype=out_dtype)
    if lse is None:
        lse = torch.empty((B, H, m), device=q.device, dtype=torch.float32)
    splits, workspace = splitkv_plan(B, H, m, N, D, q.device, splits, workspace)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with torch.cuda.device(q.device):
        st = lib().dit_attn_stale_kv_fwd(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_buf),
                                         _ptr(v_buf), _ptr(out), _ptr(lse), B, H, m, N, D,
                                         int(row0), scale, _dt(out.dtype), splits, ws_ptr,
                                         ws_bytes, _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_stale_kv_fwd")
    return out, lse


def kv_head_stride(k: torch.Tensor) -> int:
    """Elements between consecutive (b, h) heads of a [B, H, n, D] K/V view (rows D apart)."""
    B, H, n, D = k.shape
    if k.stride(3) != 1 or (n > 1 and k.stride(2) != D):
        raise ValueError("K/V rows must be contiguous and D elements apart")
    if B > 1 and H > 1:
        if k.stride(0) != H * k.stride(1):
            raise ValueError("K/V heads must be evenly spaced across the batch")
        return k.stride(1)
    if H > 1:
        return k.stride(1)
    if B > 1:
        return k.stride(0)
    return n * D  # a single head: the stride is never used


def attn_chunk_fwd(q, k, v, out=None, lse=None, scale=None, out_dtype=torch.float32, stream=None):
    """Attention of q against one KV chunk (a view such as k[:, :, s:s+n] or a packed buffer).

    Returns (partial out [B, H, N_q, D] of out_dtype, lse fp32 [B, H, N_q]).
    """
    _check_qkv(q, k, v)
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v chunk must be [B, H, n_kv, D] matching q")
    hs = kv_head_stride(k)
    if kv_head_stride(v) != hs:
        raise ValueError("k and v chunks must have the same head stride")
    n_kv = k.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check_out(out, lse, (B, H, Nq, D), q.device)
    if out is None:
        out = torch.empty((B, H, Nq, D), device=q.device, dtype=out_dtype)
    if lse is None:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        st = lib().dit_attn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq,
                                      n_kv, D, hs, scale, _dt(out.dtype),
                                      _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_chunk_fwd")
    return out, lse


def _chunk_plan(q, k, v, chunks, partials, lses, partial_dtype):
    """Shared argument handling of the all-chunks-in-one-launch calls: (hs, starts, partials,
    lses) with the host chunk-start table and the partial buffers (allocated unless given)."""
    _check_qkv(q, k, v)
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v must be [B, H, n_kv, D] matching q")
    if any(int(n) < 1 for n in chunks) or sum(int(n) for n in chunks) > k.shape[2]:
        raise ValueError("chunk lengths must be positive and fit in the keys")
    hs = kv_head_stride(k)
    if kv_head_stride(v) != hs:
        raise ValueError("k and v must have the same head stride")
    p = len(chunks)
    starts = (ctypes.c_int * (p + 1))()
    acc = 0
    for c, n in enumerate(chunks):
        starts[c] = acc
        acc += int(n)
    starts[p] = acc
    _check_out(partials, lses, (p, B, H, Nq, D), q.device, "partials", "lses")
    if partials is None:
        partials = torch.empty((p, B, H, Nq, D), device=q.device, dtype=partial_dtype)
    if lses is None:
        lses = torch.empty((p, B, H, Nq), device=q.device, dtype=torch.float32)
    return hs, starts, partials, lses


def attn_chunks_fwd(q, k, v, chunks, partials=None, lses=None, scale=None,
                    partial_dtype=torch.float32, stream=None):
    """Every chunk's partial (O_c, lse_c) of the ring decomposition in one launch
    (dit_attn_chunks_fwd): chunk c is keys [s_c, s_c + chunks[c]) of k / v, s_c the sum of the
    earlier lengths.  Returns (partials [p, B, H, N_q, D] of partial_dtype, lses [p, B, H, N_q])."""
    hs, starts, partials, lses = _chunk_plan(q, k, v, chunks, partials, lses, partial_dtype)
    B, H, Nq, D = q.shape
    p = len(chunks)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with torch.cuda.device(q.device):
        st = lib().dit_attn_chunks_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(partials), _ptr(lses), B, H,
                                       Nq, k.shape[2], D, hs, p, starts, scale, _dt(partials.dtype),
                                       _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_chunks_fwd")
    return partials, lses


def attn_chunk_fwd_accumulate(q, k, v, o_run, lse_run, scale=None, stream=None):
    """One ring hop with the merge fused in: the attention of q against one KV chunk (a view such
    as k[:, :, s:s+n] or a packed buffer) merged in place into the running o_run (fp32
    [B, H, N_q, D]) and lse_run (fp32 [B, H, N_q]).  Rows with lse_run = -inf are empty: their
    o_run is not read.  Returns (o_run, lse_run)."""
    _check_qkv(q, k, v)
    B, H, Nq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != D:
        raise ValueError("k/v chunk must be [B, H, n_kv, D] matching q")
    hs = kv_head_stride(k)
    if kv_head_stride(v) != hs:
        raise ValueError("k and v chunks must have the same head stride")
    if (o_run.dtype != torch.float32 or tuple(o_run.shape) != (B, H, Nq, D)
            or not o_run.is_contiguous() or o_run.device != q.device):
        raise ValueError("o_run must be a contiguous fp32 [B, H, N_q, D] tensor on q's device")
    if (lse_run.dtype != torch.float32 or tuple(lse_run.shape) != (B, H, Nq)
            or not lse_run.is_contiguous() or lse_run.device != q.device):
        raise ValueError("lse_run must be a contiguous fp32 [B, H, N_q] tensor on q's device")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with torch.cuda.device(q.device):
        st = lib().dit_attn_chunk_fwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(o_run),
                                                 _ptr(lse_run), B, H, Nq, k.shape[2], D, hs, scale,
                                                 _stream(q.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_chunk_fwd_accumulate")
    return o_run, lse_run


def attn_lse_merge(partials, lses, out=None, lse=None, out_dtype=torch.float32, stream=None):
    """Merge p partials [p, B, H, N, D] (fp32 or bf16) with lses fp32 [p, B, H, N]."""
    if not partials.is_cuda or partials.dim() != 5 or not partials.is_contiguous():
        raise ValueError("partials must be a contiguous CUDA tensor [p, B, H, N, D]")
    if lses.dtype != torch.float32 or tuple(lses.shape) != tuple(partials.shape[:4]) \
            or not lses.is_contiguous():
        raise ValueError("lses must be contiguous fp32 [p, B, H, N]")
    p, B, H, N, D = partials.shape
    _check_out(out, lse, (B, H, N, D), partials.device)
    if out is None:
        out = torch.empty((B, H, N, D), device=partials.device, dtype=out_dtype)
    if lse is None:
        lse = torch.empty((B, H, N), device=partials.device, dtype=torch.float32)
    with torch.cuda.device(partials.device):
        st = lib().dit_attn_lse_merge(_ptr(partials), _ptr(lses), p, _ptr(out), _ptr(lse), B, H, N,
                                      D, _dt(partials.dtype), _dt(out.dtype),
                                      _stream(partials.device, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_lse_merge")
    return out, lse


def check(device=None, stream=None):
    """Synchronise and raise DitError if a kernel reported a timed-out wait."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    with torch.cuda.device(dev):
        st = lib().dit_attn_check(_stream(dev, stream))
    if st != DIT_OK:
        raise DitError(st, "dit_attn_check")


def inject_stall(enable: bool, wait_limit_cycles: int = 0):
    """TEST ONLY: make later attention launches time out on their first K/V wait (see header)."""
    lib().dit_test_inject_stall(1 if enable else 0, int(wait_limit_cycles))


def set_grid_limit(max_ctas: int):
    """TEST ONLY: cap the persistent attention grid (0 restores one CTA per SM)."""
    lib().dit_test_set_grid_limit(int(max_ctas))
    _attn_need.cache_clear()  # with a cap, no call takes the launch that needs no workspace


def chunk_attention(q, k, v, chunks, scale=None, out_dtype=torch.float32,
                    partial_dtype=torch.float32, partials=None, lses=None, stream=None,
                    batched=False):
    """Ring decomposition on one GPU: one dit_attn_chunk_fwd per KV chunk (virtual rank), or
    with batched=True all chunks in one dit_attn_chunks_fwd launch (bitwise the same partials),
    then one dit_attn_lse_merge.  `chunks` lists the chunk lengths (sum = N_kv).  Returns
    (out, lse)."""
    B, H, Nq, D = q.shape
    if sum(chunks) != k.shape[2]:
        raise ValueError("chunk lengths must sum to the number of keys")
    p = len(chunks)
    if partials is None:
        partials = torch.empty((p, B, H, Nq, D), device=q.device, dtype=partial_dtype)
    if lses is None:
        lses = torch.empty((p, B, H, Nq), device=q.device, dtype=torch.float32)
    if batched:
        attn_chunks_fwd(q, k, v, chunks, partials=partials, lses=lses, scale=scale, stream=stream)
    else:
        s = 0
        for c, n in enumerate(chunks):
            attn_chunk_fwd(q, k[:, :, s:s + n], v[:, :, s:s + n], out=partials[c], lse=lses[c],
                           scale=scale, stream=stream)
            s += n
    return attn_lse_merge(partials, lses, out_dtype=out_dtype, stream=stream)


def ring_attention(q, k, v, chunks, scale=None, o_run=None, lse_run=None, stream=None):
    """Ring decomposition on one GPU with the merge fused into each hop: the running (o_run,
    lse_run) starts empty (lse_run = -inf) and every KV chunk (virtual rank) is folded in by one
    dit_attn_chunk_fwd_accumulate.  `chunks` lists the chunk lengths (sum = N_kv).  Returns
    (o_run fp32, lse_run)."""
    B, H, Nq, D = q.shape
    if sum(chunks) != k.shape[2] or any(n < 1 for n in chunks):
        raise ValueError("chunk lengths must be positive and sum to the number of keys")
    if o_run is None:
        o_run = torch.empty((B, H, Nq, D), device=q.device, dtype=torch.float32)
    if lse_run is None:
        lse_run = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    lse_run.fill_(float("-inf"))
    s = 0
    for n in chunks:
        attn_chunk_fwd_accumulate(q, k[:, :, s:s + n], v[:, :, s:s + n], o_run, lse_run,
                                  scale=scale, stream=stream)
        s += n
    return o_run, lse_run


def head_groups(n_heads, groups=5):
    """Split n_heads heads into consecutive groups for host pipelining: small first and last
    groups (so that the first compute starts, and the last copy-back ends, early) around a
    large middle one.  groups=5 (the default) gives about 1/12, 1/6, 1/2, 1/6, 1/12 of the
    heads (2, 4, 12, 4, 2 for 24 heads: the fastest end-to-end split measured for the Wan2.2
    shape among eight tried); groups=3 gives about 1/6, 2/3, 1/6.  Returns [(h0, h1), ...]."""
    if groups >= 5 and n_heads >= 5:
        e1, e2 = max(1, n_heads // 12), max(1, n_heads // 6)
        sizes = [e1, e2, n_heads - 2 * (e1 + e2), e2, e1]
    elif groups >= 3 and n_heads >= 3:
        edge = max(1, n_heads // 6)
        sizes = [edge, n_heads - 2 * edge, edge]
    elif groups >= 2 and n_heads >= 2:
        sizes = [n_heads // 2, n_heads - n_heads // 2]
    else:
        sizes = [n_heads]
    out, h = [], 0
    for n in sizes:
        out.append((h, h + n))
        h += n
    return out


_PIPE_STREAMS = {}


def _pipeline_streams(dev: torch.device):
    """Upload and download streams of host_pipeline, created once per device."""
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    if key not in _PIPE_STREAMS:
        _PIPE_STREAMS[key] = (torch.cuda.Stream(dev), torch.cuda.Stream(dev))
    return _PIPE_STREAMS[key]


def host_pipeline(fn, inputs, outputs, groups, device=None):
    """Runs fn over head groups with host<->device copies overlapped with compute.

    inputs / outputs: host tensors (pinned for the copies to overlap) whose first dimension is
    the flattened (batch, head) index; groups: [(h0, h1), ...] ranges of it.  For each group,
    its input slices are copied to the device on one stream, fn(*device_input_slices) runs on
    the current stream and returns device tensors shaped like the output slices, and those are
    copied back on a third stream: group g+1's upload and group g-1's download overlap group g's
    compute.  Returns outputs once every copy has landed.  (Alternating the groups over two
    compute streams, so that one group's kernels fill the previous group's last wave, measured
    slower.)"""
    dev = torch.device("cuda") if device is None else torch.device(device)
    comp = torch.cuda.current_stream(dev)
    up, down = _pipeline_streams(dev)
    d_in = [torch.empty(t.shape, dtype=t.dtype, device=dev) for t in inputs]
    up.wait_stream(comp)  # the device buffers were allocated on the compute stream
    keep = []
    for h0, h1 in groups:
        with torch.cuda.stream(up):
            for dt, ht in zip(d_in, inputs):
                dt[h0:h1].copy_(ht[h0:h1], non_blocking=True)
        comp.wait_stream(up)
        res = fn(*(dt[h0:h1] for dt in d_in))
        down.wait_stream(comp)
        with torch.cuda.stream(down):
            for ht, r in zip(outputs, res):
                ht[h0:h1].copy_(r, non_blocking=True)
        keep.append(res)  # device results stay alive until their copies are done
    down.synchronize()
    return outputs


def attention(q, k, v, scale=None, chunks=None, out_dtype=torch.float32,
              partial_dtype=torch.float32, device=None, accumulate=False, with_lse=True):
    """User-level call.  Accepts CUDA tensors, or CPU tensors (pinned for the copies to overlap)
    that are processed in head groups through host_pipeline, results returned in pinned host
    memory.  chunks=None runs the fused pass; a list of chunk lengths runs the p-chunk ring
    decomposition, merged by a separate LSE-merge pass or, with accumulate=True, hop by hop
    inside each chunk pass (fp32 output).  with_lse=False (fused pass on device tensors only)
    skips the LSE and returns (out, None)."""
    if not with_lse and (chunks is not None or not q.is_cuda):
        raise ValueError("with_lse=False applies to the fused pass on device tensors")
    if not q.is_cuda:
        # Host tensors: pipelined over head groups (uploads, compute and downloads overlap).
        B, H, Nq, D = q.shape
        o_dtype = torch.float32 if (accumulate and chunks is not None) else out_dtype
        out_h = torch.empty((B * H, Nq, D), dtype=o_dtype, pin_memory=True)
        lse_h = torch.empty((B * H, Nq), dtype=torch.float32, pin_memory=True)

        def per_group(qg, kg, vg):
            o, l = attention(qg.unsqueeze(0), kg.unsqueeze(0), vg.unsqueeze(0), scale=scale,
                             chunks=chunks, out_dtype=out_dtype, partial_dtype=partial_dtype,
                             accumulate=accumulate)
            return o[0], l[0]

        flat = [t.reshape(B * H, *t.shape[2:]) for t in (q, k, v)]
        host_pipeline(per_group, flat, [out_h, lse_h], head_groups(B * H), device)
        return out_h.view(B, H, Nq, D), lse_h.view(B, H, Nq)
    if chunks is None:
        out, lse = attn_fwd(q, k, v, scale=scale, out_dtype=out_dtype, with_lse=with_lse)
    elif accumulate:
        if out_dtype != torch.float32:
            raise ValueError("the hop-by-hop ring accumulates in fp32")
        out, lse = ring_attention(q, k, v, chunks, scale=scale)
    else:
        out, lse = chunk_attention(q, k, v, chunks, scale=scale, out_dtype=out_dtype,
                                   partial_dtype=partial_dtype)
    return out, lse


# ------------------------------------------------------------------ norms and rotary positions


def rope_freqs(rot, theta=10000.0, scaling=None, factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0,
               device="cuda"):
    """The frequencies of qk_norm_rope for `rot` rotated channels, f_i = theta^(-2 i / rot): (freqs fp32 [n], axis_pairs,
    rot_scale).  `rot` is a number, or the channels of each position axis (a video's frame, row and column: 44, 42, 42 of
    128), each with frequencies of its own.  For contexts `factor` times as long as original_len, `scaling`:
      None      as they are
      "linear"  every position divided by factor
      "ntk"     a larger base, theta * factor^(rot / (rot - 2)): the slowest pair stretched by factor, the fastest not
      "yarn"    pairs that turn less than beta_slow times in original_len positions divided by factor, those that
                turn more than beta_fast times left, in between in proportion to the turns; rot_scale = 0.1 ln(factor) + 1
    (Many released models ramp in proportion to the pair's index instead: give their tables as freqs.)  rot_scale is 1
    but for "yarn", and a call that leaves it out attends at another temperature.  Computed in 64 bits on the host."""
    dims = [int(rot)] if isinstance(rot, int) else [int(r) for r in rot]
    if any(r < 2 or r % 2 for r in dims) or not dims:
        raise ValueError("each axis has a positive, even number of channels")
    if scaling not in (None, "linear", "ntk", "yarn") or not factor >= 1 or not theta > 0:
        raise ValueError("scaling is None, 'linear', 'ntk' or 'yarn', factor at least 1, theta positive")
    out = []
    for r in dims:
        i = torch.arange(r // 2, dtype=torch.float64)
        base = theta * factor ** (r / (r - 2)) if scaling == "ntk" and r > 2 else theta
        f = base ** (-2 * i / r)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            turns = original_len * f / (2 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
            f = f * (keep + (1 - keep) / factor)
        out.append(f)
    return (torch.cat(out).float().to(device), [r // 2 for r in dims],
            0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def _rope_view(t, name, index):
    """(B, H, N, D) and strides (b, h, n) of a [B, H, N, D] or a packed [T, H, D] bf16 view."""
    try:  # the usual case, as in _check_tensor
        shape, stride = t.shape, t.stride()
        usual = t.dtype is torch.bfloat16 and stride[-1] == 1 and t.get_device() == index
    except (AttributeError, IndexError):
        usual, shape = False, (None,) * 4
    if not usual or len(shape) not in (3, 4):
        _check_tensor(t, name, torch.bfloat16, (None,) * (3 if len(shape) == 3 else 4), index, rows=True)
    if len(shape) == 3:
        return (1, shape[1], shape[0], shape[2]), Strides(shape[2], stride[1], stride[0])
    return shape, Strides(*stride[:3])


@functools.lru_cache(maxsize=64)
def _int_array(values):
    """The values as a C array (read by the library alone)."""
    return (ctypes.c_int * len(values))(*values)


def qk_norm_rope(q, k=None, positions=None, freqs=None, axis_pairs=None, interleaved=False, rot_scale=1.0, eps=None,
                 q_weight=None, k_weight=None, cu_new=None, start_lens=None, q_out=None, k_out=None, stream=None):
    """dit_qk_norm_rope: RMS norms of each head of q and k by itself (eps None: none; weights [D], bf16 or fp32, or None) and rotary
    positions (freqs None: none), in one pass.  q, k: bf16 views [B, H, N, D], or [T, H, D] of packed tokens.

    freqs (fp32 [n]), axis_pairs and rot_scale are rope_freqs'; axis_pairs None: one axis.  Positions, int32: [N] or
    [axes, N] for all of the batch, or [axes, B, N]; or, of packed requests, cu_new [R + 1] (paged_plan's) and
    start_lens [R], the position of each request's first token: tokens of no request are then left as they are.

    Returns (q_out, k_out or None), contiguous in the inputs' shapes unless given; in place: q_out=q, k_out=k."""
    dev, index = _check_rows(q, "q", q.dim() if isinstance(q, torch.Tensor) and q.dim() in (3, 4) else 4)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return qk_norm_rope(q, k, positions, freqs, axis_pairs, interleaved, rot_scale, eps, q_weight, k_weight, cu_new,
                                start_lens, q_out, k_out)
    (B, Hq, N, D), qs = _rope_view(q, "q", index)
    Hk, ks, kos = 0, None, None
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
            raise ValueError("k must have as many dimensions as q")
        (Bk, Hk, Nk, Dk), ks = _rope_view(k, "k", index)
        if (Bk, Nk, Dk) != (B, N, D):
            raise ValueError("q and k must be of the same tokens and head size")
        if k_out is None:
            k_out = torch.empty(k.shape, device=dev, dtype=torch.bfloat16)
        elif k_out is not k:
            _check_tensor(k_out, "k_out", torch.bfloat16, k.shape, index, rows=True)
        kos = ks if k_out is k else _rope_view(k_out, "k_out", index)[1]
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    if q_out is None:
        q_out = torch.empty(q.shape, device=dev, dtype=torch.bfloat16)
    elif q_out is not q:
        _check_tensor(q_out, "q_out", torch.bfloat16, q.shape, index, rows=True)
    qos = qs if q_out is q else _rope_view(q_out, "q_out", index)[1]
    wdt = torch.bfloat16
    if q_weight is not None or k_weight is not None:
        wdt = getattr(k_weight if q_weight is None else q_weight, "dtype", None)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _check_tensor(w, name, wdt, (D,), index)
    axes, pairs, pos_b, pos_axis, requests = 0, None, 0, 0, 0
    if freqs is None:
        if positions is not None or cu_new is not None or start_lens is not None:
            raise ValueError("positions need freqs")
    else:
        _check_tensor(freqs, "freqs", torch.float32, (None,), index)
        n = freqs.shape[0]
        pairs = (n,) if axis_pairs is None else tuple(int(x) for x in axis_pairs)
        axes = len(pairs)
        if sum(pairs) != n:
            raise ValueError(f"axis_pairs must add up to the {n} frequencies")
        if positions is not None:
            if cu_new is not None or start_lens is not None:
                raise ValueError("positions, or cu_new and start_lens")
            shape = {1: (N,), 2: (axes, N), 3: (axes, B, N)}.get(getattr(positions, "dim", int)(), (axes, B, N))
            if len(shape) == 1 and axes != 1:
                raise ValueError(f"positions must have shape [{axes}, {N}]")
            _check_tensor(positions, "positions", torch.int32, shape, index)
            pos_b, pos_axis = (N if len(shape) == 3 else 0), (B * N if len(shape) == 3 else N)
        else:
            if cu_new is None or start_lens is None or not isinstance(start_lens, torch.Tensor) or start_lens.dim() != 1:
                raise ValueError("freqs need positions, or cu_new and start_lens")
            requests = start_lens.shape[0]
            _check_tensor(start_lens, "start_lens", torch.int32, (requests,), index)
            _check_tensor(cu_new, "cu_new", torch.int32, (requests + 1,), index)
        pairs = _int_array(pairs)
    st = lib().dit_qk_norm_rope(
        q.data_ptr(), qs, q_out.data_ptr(), qos, Hq, None if k is None else k.data_ptr(), ks,
        None if k is None else k_out.data_ptr(), kos, Hk, 0 if eps is None else 1, 0.0 if eps is None else float(eps),
        None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), _dt(wdt),
        None if freqs is None else freqs.data_ptr(), pairs, axes, 1 if interleaved else 0, float(rot_scale),
        None if positions is None else positions.data_ptr(), pos_b, pos_axis, None if cu_new is None else cu_new.data_ptr(),
        None if start_lens is None else start_lens.data_ptr(), requests, B, N, D,
        torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_qk_norm_rope")
    return q_out, k_out


# ------------------------------------------------------------------ paged key/value caches
# One step of a batch of requests whose keys and values live in pages of one pool:
#   lens, n_free, cu, slots = paged_plan(...)         pages and slots for the step's tokens
#   q, k = qk_norm_rope(q, k, ..., cu_new=cu, start_lens=...)    norms and positions
#   paged_kv_write(k, v, slots, k_cache, v_cache, summary)
#   out, lse = paged_prefill_fwd(q, k_cache, v_cache, table, lens, cu)   new tokens, or one of each request:
#   selected = paged_select(q, summary, table, lens, ...)        (sparse attention only)
#   out, lse = paged_attn_fwd(q, k_cache, v_cache, table, lens, selected=selected)
#   paged_page_mass(...); paged_evict(...)            (caches with a budget) least used pages back to the pool
# k_cache and v_cache are [n_pages, H_kv, page_size, D] views (a token-major cache
# [n_pages, page_size, H_kv, D] is passed as x.transpose(1, 2), the halves of one that holds keys and
# values in turn as x[:, 0] and x[:, 1]); block_table is int32
# [B, max_pages], seq_lens int32 [B].


def _elsewhere(device, stream):
    """The context a paged call has to run in, or None where the current device and stream are the
    ones asked for.  The call runs itself again inside it, so that what it allocates belongs to the
    stream that uses it."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() != device.index:
        return torch.cuda.device(device)
    return None


def _check_tensor(t, name, dtype, shape, index, rows=False):
    """Raises unless `t` is a `dtype` tensor of `shape` (None: any extent) on CUDA device `index`,
    contiguous, or (rows=True) with a contiguous last dimension."""
    try:  # one cheap test for the usual case: these calls are bound by the host at small sizes
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(e is not None and e != x for e, x in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if not rows and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if rows and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _check_rows(t, name, dims):
    """(device, CUDA device number) of a bf16 view of `dims` dimensions with a contiguous last one."""
    try:
        index = t.get_device()
        if index >= 0 and t.dtype is torch.bfloat16 and t.dim() == dims and t.stride(-1) == 1:
            return t.device, index
    except (AttributeError, IndexError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _check_tensor(t, name, torch.bfloat16, (None,) * dims, t.get_device(), rows=True)
    return t.device, t.get_device()


def _check_caches(k_cache, v_cache, index):
    """(n_pages, H_kv, page_size, D) of the two caches."""
    try:
        shape = k_cache.shape
        if (k_cache.dtype is torch.bfloat16 and v_cache.dtype is torch.bfloat16 and v_cache.shape == shape
                and len(shape) == 4 and k_cache.get_device() == index and v_cache.get_device() == index
                and k_cache.stride(3) == 1 and v_cache.stride(3) == 1):
            return shape
    except AttributeError:
        pass
    _check_tensor(k_cache, "k_cache", torch.bfloat16, (None,) * 4, index, rows=True)
    _check_tensor(v_cache, "v_cache", torch.bfloat16, k_cache.shape, index, rows=True)
    return k_cache.shape


def _check_table(block_table, seq_lens, B, index):
    """(max_pages, table_stride) of the batch's block table."""
    _check_tensor(seq_lens, "seq_lens", torch.int32, (B,), index)
    try:
        rows, max_pages = block_table.shape
        stride, last = block_table.stride()
        if (last == 1 and rows == B and block_table.dtype is torch.int32
                and block_table.get_device() == index):
            return max_pages, (stride if B > 1 else max_pages)
    except (AttributeError, ValueError):
        pass
    _check_tensor(block_table, "block_table", torch.int32, (B, None), index, rows=True)
    max_pages = block_table.shape[1]
    return max_pages, (block_table.stride(0) if B > 1 else max_pages)


@functools.lru_cache(maxsize=4096)
def _attn_need(index, B, Hq, Hkv, D, page_size, pages):
    """dit_paged_attn_workspace_bytes on the current device, number `index`."""
    return lib().dit_paged_attn_workspace_bytes(B, Hq, Hkv, D, page_size, pages)


@functools.lru_cache(maxsize=4096)
def _select_need(index, B, Hkv, max_pages):
    """dit_paged_select_workspace_bytes on the current device, number `index`."""
    return lib().dit_paged_select_workspace_bytes(B, Hkv, max_pages)


@functools.lru_cache(maxsize=4096)
def _evict_need(B, max_pages):
    """dit_paged_evict_workspace_bytes."""
    return lib().dit_paged_evict_workspace_bytes(B, max_pages)


@functools.lru_cache(maxsize=4096)
def _prefill_need(index, D, page_size, max_pages):
    """dit_paged_prefill_workspace_bytes on the current device, number `index`."""
    return lib().dit_paged_prefill_workspace_bytes(D, page_size, max_pages)


def _workspace(workspace, need, device):
    """(buffer or None, its address or None, bytes) of a call's workspace: the caller's, or a new one."""
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    size = workspace.numel() * workspace.element_size()
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous() or size < need:
        raise ValueError(f"workspace must be a contiguous buffer of at least {need} bytes on {device}")
    return workspace, workspace.data_ptr(), size


def paged_plan(new_lens, seq_lens, block_table, free_pages, n_free, page_size, n_pages, max_tokens,
               seq_lens_out=None, n_free_out=None, cu_new=None, slots=None, stream=None):
    """dit_paged_plan: grants the pages that new_lens [B] more tokens of each request need (from the
    top of the stack free_pages[:n_free], into block_table in place) and maps the step's tokens
    (packed in request order, at most max_tokens) to their slots.  All int32 but slots (int64).

    Returns (seq_lens_out [B], n_free_out [1], cu_new [B + 1], slots [max_tokens]); seq_lens_out may
    be seq_lens and n_free_out may be n_free (updated in place)."""
    if not isinstance(new_lens, torch.Tensor) or not new_lens.is_cuda:
        raise ValueError("new_lens must be a CUDA tensor")
    dev, index = new_lens.device, new_lens.get_device()
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_plan(new_lens, seq_lens, block_table, free_pages, n_free, page_size, n_pages,
                              max_tokens, seq_lens_out, n_free_out, cu_new, slots)
    i32 = torch.int32
    _check_tensor(new_lens, "new_lens", i32, new_lens.shape[:1] or (None,), index)
    B = new_lens.shape[0]
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    if not isinstance(free_pages, torch.Tensor):
        raise ValueError("free_pages must be a CUDA tensor")
    _check_tensor(free_pages, "free_pages", i32, free_pages.shape[:1] or (None,), index)
    _check_tensor(n_free, "n_free", i32, (1,), index)
    max_tokens = int(max_tokens)
    if seq_lens_out is None:
        seq_lens_out = torch.empty(B, dtype=i32, device=dev)
    else:
        _check_tensor(seq_lens_out, "seq_lens_out", i32, (B,), index)
    if n_free_out is None:
        n_free_out = torch.empty(1, dtype=i32, device=dev)
    else:
        _check_tensor(n_free_out, "n_free_out", i32, (1,), index)
    if cu_new is None:
        cu_new = torch.empty(B + 1, dtype=i32, device=dev)
    else:
        _check_tensor(cu_new, "cu_new", i32, (B + 1,), index)
    if slots is None:
        slots = torch.empty(max(0, max_tokens), dtype=torch.int64, device=dev)
    else:
        _check_tensor(slots, "slots", torch.int64, (max_tokens,), index)
    st = lib().dit_paged_plan(new_lens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                              stride, free_pages.data_ptr(), n_free.data_ptr(),
                              seq_lens_out.data_ptr(), n_free_out.data_ptr(), cu_new.data_ptr(),
                              slots.data_ptr(), B, max_pages, page_size, n_pages,
                              free_pages.shape[0], max_tokens, torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_plan")
    return seq_lens_out, n_free_out, cu_new, slots


def paged_kv_write(k_new, v_new, slots, k_cache, v_cache, summary=None, stream=None):
    """dit_paged_kv_write: k_new, v_new bf16 [T, H_kv, D] views (slices of a fused projection need no
    copy) into the slots (int64 [T], below 0: skipped) of the caches; with `summary` (bf16
    [n_pages, H_kv, 2, D]) each touched page's channel minimum and maximum is kept up to date."""
    dev, index = _check_rows(k_new, "k_new", 3)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_kv_write(k_new, v_new, slots, k_cache, v_cache, summary)
    T, H, D = k_new.shape
    _check_tensor(v_new, "v_new", torch.bfloat16, (T, H, D), index, rows=True)
    n_pages, Hc, P, Dc = _check_caches(k_cache, v_cache, index)
    if Hc != H or Dc != D:
        raise ValueError(f"the caches hold {Hc} heads of {Dc}, the new rows {H} of {D}")
    _check_tensor(slots, "slots", torch.int64, (T,), index)
    if summary is not None:
        _check_tensor(summary, "summary", torch.bfloat16, (n_pages, H, 2, D), index)
    kn, kh, _ = k_new.stride()
    vn, vh, _ = v_new.stride()
    st = lib().dit_paged_kv_write(k_new.data_ptr(), Strides(D, kh, kn), v_new.data_ptr(), Strides(D, vh, vn),
                                  slots.data_ptr(), k_cache.data_ptr(), Strides(*k_cache.stride()[:3]),
                                  v_cache.data_ptr(), Strides(*v_cache.stride()[:3]),
                                  None if summary is None else summary.data_ptr(), T, H, D, P,
                                  n_pages, torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_kv_write")


def paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, selected=None, out=None, lse=None,
                   scale=None, out_dtype=torch.float32, workspace=None, stream=None, with_lse=True):
    """dit_paged_attn_fwd: one query token of each request, q bf16 [B, H_q, D] (a view with contiguous
    D), over the request's seq_lens[b] cached tokens; H_q is a multiple of the caches' H_kv.
    `selected` (int32 [B, H_kv, n], paged_select's form) restricts each key/value head to the listed
    pages.  The workspace is allocated with torch unless given.

    Returns (out [B, H_q, D] of out_dtype, lse fp32 [B, H_q]); with_lse=False returns (out, None)."""
    dev, index = _check_rows(q, "q", 3)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, selected, out, lse, scale,
                                  out_dtype, workspace, None, with_lse)
    B, Hq, D = q.shape
    n_pages, Hkv, P, Dc = _check_caches(k_cache, v_cache, index)
    if Dc != D:
        raise ValueError(f"the caches hold heads of {Dc}, q of {D}")
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    if selected is not None:
        _check_tensor(selected, "selected", torch.int32, (B, Hkv, selected.shape[-1]), index)
    if out is not None or lse is not None:
        _check_out(out, lse, (B, Hq, D), dev)
    if out is None:
        out = torch.empty((B, Hq, D), device=dev, dtype=out_dtype)
    if not with_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((B, Hq), device=dev, dtype=torch.float32)
    pages = max_pages if selected is None else selected.shape[2]
    workspace, ws, size = _workspace(workspace, _attn_need(index, B, Hq, Hkv, D, P, pages), dev)
    qb, qh, _ = q.stride()
    st = lib().dit_paged_attn_fwd(
        q.data_ptr(), Strides(qb, qh, D), k_cache.data_ptr(), Strides(*k_cache.stride()[:3]),
        v_cache.data_ptr(), Strides(*v_cache.stride()[:3]), block_table.data_ptr(), stride,
        seq_lens.data_ptr(), None if selected is None else selected.data_ptr(),
        0 if selected is None else selected.shape[2], out.data_ptr(),
        None if lse is None else lse.data_ptr(), B, Hq, Hkv, D, P, n_pages, max_pages,
        1.0 / math.sqrt(D) if scale is None else float(scale), _dt(out.dtype), ws, size,
        torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_attn_fwd")
    return out, lse


def _batch_of(seq_lens):
    """The number of requests, from their lengths."""
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be a CUDA tensor of one dimension")
    return seq_lens.shape[0]


def paged_prefill_fwd(q, k_cache, v_cache, block_table, seq_lens, cu_new, start_lens=None, causal=True, out=None,
                      lse=None, scale=None, out_dtype=torch.float32, workspace=None, stream=None, with_lse=True):
    """dit_paged_prefill_fwd: the step's new tokens, q bf16 [T, H_q, D] (a view with contiguous D) packed in
    request order (cu_new int32 [B + 1], paged_plan's), over the requests' seq_lens[b] cached tokens, their own
    among them; `causal` False: every token sees all of them.  start_lens (int32 [B]): the position of each
    request's first new token, by default such that they are its last.  Rows of no request are left as
    they are.  The workspace is allocated with torch unless given.  The attention's weights are rounded to bf16 whatever the
    output's type, as the dense attention's are (outputs are off by about 1e-3 of their size; paged_attn_fwd holds all of
    them with fp32 output).

    Returns (out [T, H_q, D] of out_dtype, lse fp32 [T, H_q]); with_lse=False returns (out, None)."""
    dev, index = _check_rows(q, "q", 3)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_prefill_fwd(q, k_cache, v_cache, block_table, seq_lens, cu_new, start_lens, causal, out, lse,
                                     scale, out_dtype, workspace, None, with_lse)
    T, Hq, D = q.shape
    n_pages, Hkv, P, Dc = _check_caches(k_cache, v_cache, index)
    if Dc != D:
        raise ValueError(f"the caches hold heads of {Dc}, q of {D}")
    B = _batch_of(seq_lens)
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    _check_tensor(cu_new, "cu_new", torch.int32, (B + 1,), index)
    if start_lens is not None:
        _check_tensor(start_lens, "start_lens", torch.int32, (B,), index)
    if out is not None or lse is not None:
        _check_out(out, lse, (T, Hq, D), dev)
    if out is None:
        out = torch.empty((T, Hq, D), device=dev, dtype=out_dtype)
    if not with_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((T, Hq), device=dev, dtype=torch.float32)
    workspace, ws, size = _workspace(workspace, _prefill_need(index, D, P, max_pages), dev)
    qn, qh, _ = q.stride()
    st = lib().dit_paged_prefill_fwd(
        q.data_ptr(), Strides(D, qh, qn), k_cache.data_ptr(), Strides(*k_cache.stride()[:3]), v_cache.data_ptr(),
        Strides(*v_cache.stride()[:3]), block_table.data_ptr(), stride, seq_lens.data_ptr(), cu_new.data_ptr(),
        None if start_lens is None else start_lens.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        T, B, Hq, Hkv, D, P, n_pages, max_pages, 1 if causal else 0, 1.0 / math.sqrt(D) if scale is None else float(scale),
        _dt(out.dtype), ws, size, torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_prefill_fwd")
    return out, lse


def paged_page_mass(q, lse, k_cache, block_table, seq_lens, mass, cu_new=None, start_lens=None, window=0, mass_out=None,
                    scale=None, stream=None):
    """dit_paged_page_mass: adds to each page's drawn weight, mass fp32 [n_pages, H_kv], what the step's queries
    q bf16 [T, H_q, D] gave it, from their attention's lse fp32 [T, H_q]; pages whose first key is new start from
    nothing.  cu_new (int32 [B + 1]): packed new tokens, of which the last `window` (0: all) of each request count;
    None: one token of each request (T = B).  In place unless mass_out is given, of which only the pages of requests
    with new tokens are written.  Called in every step, it drops what a page's former owner left; a program that skips steps
    clears the weights of the pages that they handed out.  The lse is of all pages, not of selected ones.  Returns mass_out."""
    dev, index = _check_rows(q, "q", 3)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_page_mass(q, lse, k_cache, block_table, seq_lens, mass, cu_new, start_lens, window, mass_out, scale)
    T, Hq, D = q.shape
    n_pages, Hkv, P, Dc = _check_caches(k_cache, k_cache, index)
    if Dc != D:
        raise ValueError(f"the cache holds heads of {Dc}, q of {D}")
    B = _batch_of(seq_lens)
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    _check_tensor(lse, "lse", torch.float32, (T, Hq), index)
    _check_tensor(mass, "mass", torch.float32, (n_pages, Hkv), index)
    if mass_out is None:
        mass_out = mass
    else:
        _check_tensor(mass_out, "mass_out", torch.float32, (n_pages, Hkv), index)
    if cu_new is not None:
        _check_tensor(cu_new, "cu_new", torch.int32, (B + 1,), index)
    if start_lens is not None:
        _check_tensor(start_lens, "start_lens", torch.int32, (B,), index)
    qn, qh, _ = q.stride()
    st = lib().dit_paged_page_mass(
        q.data_ptr(), Strides(D, qh, qn), lse.data_ptr(), k_cache.data_ptr(), Strides(*k_cache.stride()[:3]),
        block_table.data_ptr(), stride, seq_lens.data_ptr(), None if cu_new is None else cu_new.data_ptr(),
        None if start_lens is None else start_lens.data_ptr(), mass.data_ptr(), mass_out.data_ptr(), T, B, Hq, Hkv, D, P,
        n_pages, max_pages, int(window), 1.0 / math.sqrt(D) if scale is None else float(scale),
        torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_page_mass")
    return mass_out


def paged_evict(mass, block_table, seq_lens, free_pages, n_free, page_size, keep, recent=1, table_out=None,
                seq_lens_out=None, n_free_out=None, workspace=None, stream=None):
    """dit_paged_evict: requests of more than `keep` pages keep the newest `recent` and, of the others, those that drew
    most weight (mass fp32 [n_pages, H_kv], paged_page_mass's); the others' numbers go onto the stack free_pages.  The table
    changes in place unless table_out [B, max_pages] is given.  The workspace is allocated with torch unless given.

    Returns (seq_lens_out [B], n_free_out [1]); they may be seq_lens and n_free (updated in place)."""
    if not isinstance(mass, torch.Tensor) or not mass.is_cuda:
        raise ValueError("mass must be a CUDA tensor")
    dev, index = mass.device, mass.get_device()
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_evict(mass, block_table, seq_lens, free_pages, n_free, page_size, keep, recent, table_out,
                               seq_lens_out, n_free_out, workspace)
    i32 = torch.int32
    _check_tensor(mass, "mass", torch.float32, (None, None), index)
    n_pages, Hkv = mass.shape
    B = _batch_of(seq_lens)
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    if table_out is None:
        table_out, out_stride = block_table, stride
    else:
        _check_tensor(table_out, "table_out", i32, (B, max_pages), index, rows=True)
        out_stride = table_out.stride(0) if B > 1 else max_pages
    if not isinstance(free_pages, torch.Tensor):
        raise ValueError("free_pages must be a CUDA tensor")
    _check_tensor(free_pages, "free_pages", i32, free_pages.shape[:1] or (None,), index)
    _check_tensor(n_free, "n_free", i32, (1,), index)
    if seq_lens_out is None:
        seq_lens_out = torch.empty(B, dtype=i32, device=dev)
    else:
        _check_tensor(seq_lens_out, "seq_lens_out", i32, (B,), index)
    if n_free_out is None:
        n_free_out = torch.empty(1, dtype=i32, device=dev)
    else:
        _check_tensor(n_free_out, "n_free_out", i32, (1,), index)
    workspace, ws, size = _workspace(workspace, _evict_need(B, max_pages), dev)
    st = lib().dit_paged_evict(mass.data_ptr(), block_table.data_ptr(), stride, table_out.data_ptr(), out_stride,
                               seq_lens.data_ptr(), seq_lens_out.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(),
                               n_free_out.data_ptr(), B, Hkv, page_size, n_pages, max_pages, free_pages.shape[0],
                               int(keep), int(recent), ws, size, torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_evict")
    return seq_lens_out, n_free_out


def paged_select(q, summary, block_table, seq_lens, page_size, top_k, selected=None, workspace=None,
                 stream=None):
    """dit_paged_select: for each request and key/value head the newest page and the top_k - 1 others
    whose summaries (bf16 [n_pages, H_kv, 2, D]) bound the highest scores for q bf16 [B, H_q, D].

    Returns selected, int32 [B, H_kv, top_k]: table columns in ascending order, then -1."""
    dev, index = _check_rows(q, "q", 3)
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_select(q, summary, block_table, seq_lens, page_size, top_k, selected, workspace)
    B, Hq, D = q.shape
    if not isinstance(summary, torch.Tensor):
        raise ValueError("summary must be a CUDA tensor")
    n_pages, Hkv = summary.shape[:2]
    _check_tensor(summary, "summary", torch.bfloat16, (n_pages, Hkv, 2, D), index)
    max_pages, stride = _check_table(block_table, seq_lens, B, index)
    top_k = int(top_k)
    if selected is None:
        selected = torch.empty((B, Hkv, max(0, top_k)), device=dev, dtype=torch.int32)
    else:
        _check_tensor(selected, "selected", torch.int32, (B, Hkv, top_k), index)
    workspace, ws, size = _workspace(workspace, _select_need(index, B, Hkv, max_pages), dev)
    qb, qh, _ = q.stride()
    st = lib().dit_paged_select(q.data_ptr(), Strides(qb, qh, D), summary.data_ptr(), block_table.data_ptr(),
                            stride, seq_lens.data_ptr(), selected.data_ptr(), B, Hq, Hkv, D, page_size,
                            n_pages, max_pages, top_k, ws, size,
                            torch._C._cuda_getCurrentRawStream(index))
    if st != DIT_OK:
        raise DitError(st, "dit_paged_select")
    return selected
