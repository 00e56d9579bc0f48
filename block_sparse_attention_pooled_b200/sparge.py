"""Python binding of the C ABI in include/sparge.h (argument marshalling only).

Importing this module loads ``libsparge.so`` from the package directory and
raises ImportError when it is missing: there is no fallback implementation.
Tensors are torch CUDA tensors; every call is enqueued on the current torch
stream (or the stream given) and returns without synchronising.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsparge.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m block_sparse_attention_pooled_b200.build`")
_lib = ctypes.CDLL(_LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT = range(6)
OP_MASK, OP_ATTN, OP_SLA2, OP_ATTN_Q8, OP_MASK_ROUTER, OP_ATTN_BWD, OP_SLA2_BWD = 0, 1, 2, 3, 4, 5, 6
OP_WINDOW_FWD, OP_WINDOW_BWD = 7, 8
CACHE_BF16, CACHE_E4M3 = 0, 1

# Kernel launches per call of each entry point (for launch accounting).
MASK_LAUNCHES, ATTN_LAUNCHES, SLA2_LAUNCHES, Q8_LAUNCHES, ROUTER_LAUNCHES, BWD_LAUNCHES = 3, 1, 4, 3, 5, 4
# sla2_attn_bwd: summaries + reduce, linear_out, sparse forward, row pass, dalpha, gradient summaries
# + reduce, transposed mask, dQ, dK/dV sparse part, dK/dV linear part (the memset is not a kernel).
# The attention, SLA2 and low-bit forward calls and both backward calls add order_launches(shape).
SLA2_BWD_LAUNCHES = 12

# Every symbol the header declares.
EXPORTS = ("sparge_workspace_bytes", "sparge_mask", "sparge_attn_fwd", "sla2_attn_fwd",
           "sparge_device_status", "sparge_status_string", "sparge_mask_noalloc", "sparge_attn_fwd_q8",
           "sparge_mask_router", "sparge_attn_bwd", "sla2_attn_bwd", "sparge_selftest_wait",
           "sparge_window_workspace_bytes", "sparge_window_fwd", "sparge_window_bwd", "sparge_cache_write",
           "sparge_cache_read", "sparge_cache_attn_workspace_bytes", "sparge_cache_attn")


def order_launches(shape) -> int:
    """Launches of the tile-order kernel per attention call for this shape (launch accounting):
    1 when at least two heads' K and V (4 N d bytes each) fit in 64 MB, else 0."""
    return 1 if min(shape.B * shape.H, (64 << 20) // (4 * shape.N * shape.d)) >= 2 else 0


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "N", "d", "bq", "bk")]


class WindowShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "Hkv", "N", "d")]


class Window(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("left", "right", "sinks", "unit")]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp")] + [
        (n, ctypes.c_int32) for n in ("pages", "Hkv", "page", "d", "type")]


class CacheBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("page_table", "first", "cu")] + [
        (n, ctypes.c_int32) for n in ("B", "max_pages", "tokens")]


_vp, _sz, _dbl = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_double
_lib.sparge_workspace_bytes.argtypes = [ctypes.c_int, ctypes.POINTER(Shape)]
_lib.sparge_workspace_bytes.restype = _sz
_lib.sparge_mask.argtypes = [_vp, _vp, ctypes.POINTER(Shape), _dbl, _dbl, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparge_mask_router.argtypes = [_vp, _vp, ctypes.POINTER(Shape), _vp, _vp, ctypes.c_int, _dbl, _dbl, _vp, _vp,
                                     _vp, _vp, _vp, _sz, _vp]
_lib.sparge_mask_noalloc.argtypes = [_vp, _vp, ctypes.POINTER(Shape), _dbl, _dbl, _vp, _vp, _vp, _vp, _vp]
_lib.sparge_mask_noalloc.restype = ctypes.c_int
_lib.sparge_attn_fwd.argtypes = [_vp, _vp, _vp, ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sla2_attn_fwd.argtypes = [_vp, _vp, _vp, ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparge_attn_fwd_q8.argtypes = [_vp, _vp, _vp, ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparge_attn_bwd.argtypes = [_vp, _vp, _vp, ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _sz, _vp]
_lib.sla2_attn_bwd.argtypes = [_vp, _vp, _vp, ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]
_lib.sparge_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
_lib.sparge_selftest_wait.argtypes = [ctypes.c_int32, _vp, _vp]
_lib.sparge_status_string.argtypes = [ctypes.c_int]
_lib.sparge_status_string.restype = ctypes.c_char_p
_i32, _i64 = ctypes.c_int32, ctypes.c_int64
_lib.sparge_window_workspace_bytes.argtypes = [ctypes.c_int, _vp, _vp]
_lib.sparge_window_workspace_bytes.restype = _sz
_lib.sparge_window_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparge_window_bwd.argtypes = [_vp] * 13 + [_sz, _vp]
_lib.sparge_cache_write.argtypes = [_vp, _vp, _vp, _i64, _vp, _i64, _vp]
_lib.sparge_cache_read.argtypes = [_vp, _vp, _vp, _vp, _vp]
_lib.sparge_cache_attn_workspace_bytes.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp]
_lib.sparge_cache_attn_workspace_bytes.restype = _sz
_lib.sparge_cache_attn.argtypes = [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]
for _f in ("sparge_window_fwd", "sparge_window_bwd", "sparge_cache_write", "sparge_cache_read", "sparge_cache_attn"):
    getattr(_lib, _f).restype = ctypes.c_int
for _f in ("sparge_mask", "sparge_mask_router", "sparge_attn_bwd", "sla2_attn_bwd", "sparge_attn_fwd", "sla2_attn_fwd", "sparge_device_status", "sparge_attn_fwd_q8",
           "sparge_selftest_wait"):
    getattr(_lib, _f).restype = ctypes.c_int


class SpargeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {_lib.sparge_status_string(code).decode()} (status {code})")
        self.code = code


def lib_path() -> str:
    return _LIB_PATH


def raw() -> ctypes.CDLL:
    """The loaded library (for callers that marshal pointers themselves)."""
    return _lib


def _check(code: int, where: str):
    if code != OK:
        raise SpargeError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_shape(Q: torch.Tensor, bq: int, bk: int) -> Shape:
    B, H, N, d = Q.shape
    return Shape(B, H, N, d, bq, bk)


def workspace_bytes(op: int, shape: Shape) -> int:
    return int(_lib.sparge_workspace_bytes(op, ctypes.byref(shape)))


def _workspace(op: int, shape: Shape, device) -> Tuple[Optional[torch.Tensor], int]:
    n = workspace_bytes(op, shape)
    if n == 0:
        return None, 0
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _check_qkv(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("Q/K/V/O must be contiguous bf16 CUDA tensors of shape [B,H,N,d]")


def sparge_mask(Q, K, bq: int, bk: int, topk: float, topp: float, kv_idx=None, kv_cnt=None,
                row_thresh=None, probs=None, workspace=None, stream=None):
    """Hybrid Top-k / Top-p block mask. Returns (kv_idx, kv_cnt)."""
    _check_qkv(Q, K)
    shape = make_shape(Q, bq, bk)
    B, H, N, _ = Q.shape
    nqb, nkb = -(-N // bq), -(-N // bk)
    if kv_idx is None:
        kv_idx = torch.empty((B, H, nqb, nkb), dtype=torch.int32, device=Q.device)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, H, nqb), dtype=torch.int32, device=Q.device)
    if workspace is None:
        workspace, nws = _workspace(OP_MASK, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sparge_mask(_ptr(Q), _ptr(K), ctypes.byref(shape), float(topk), float(topp), _ptr(kv_idx),
                            _ptr(kv_cnt), _ptr(row_thresh), _ptr(probs), _ptr(workspace), nws, _stream(stream)),
           "sparge_mask")
    return kv_idx, kv_cnt


def sparge_mask_router(Q, K, Wq, Wk, bq: int, bk: int, topk: float, topp: float, kv_idx=None, kv_cnt=None,
                       row_thresh=None, probs=None, workspace=None, stream=None):
    """Block mask scored through the learnt router projections Wq, Wk (fp32 [H, d, dr]).
    Returns (kv_idx, kv_cnt)."""
    _check_qkv(Q, K)
    H, d = Q.shape[1], Q.shape[3]
    for W in (Wq, Wk):
        if W.dtype != torch.float32 or not W.is_cuda or not W.is_contiguous() or W.dim() != 3 \
                or W.shape[0] != H or W.shape[1] != d or W.shape != Wq.shape:
            raise ValueError("Wq/Wk must be contiguous fp32 CUDA tensors of shape [H, d, dr]")
    shape = make_shape(Q, bq, bk)
    B, _, N, _ = Q.shape
    nqb, nkb = -(-N // bq), -(-N // bk)
    if kv_idx is None:
        kv_idx = torch.empty((B, H, nqb, nkb), dtype=torch.int32, device=Q.device)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, H, nqb), dtype=torch.int32, device=Q.device)
    if workspace is None:
        workspace, nws = _workspace(OP_MASK_ROUTER, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sparge_mask_router(_ptr(Q), _ptr(K), ctypes.byref(shape), _ptr(Wq), _ptr(Wk), int(Wq.shape[2]),
                                   float(topk), float(topp), _ptr(kv_idx), _ptr(kv_cnt), _ptr(row_thresh),
                                   _ptr(probs), _ptr(workspace), nws, _stream(stream)), "sparge_mask_router")
    return kv_idx, kv_cnt


def sparge_attn_fwd(Q, K, V, kv_idx, kv_cnt, bq: int, bk: int, O=None, lse=None, workspace=None, stream=None):
    """Block-sparse attention over the kept blocks. Returns O (and fills lse if given)."""
    _check_qkv(Q, K, V)
    shape = make_shape(Q, bq, bk)
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace, nws = _workspace(OP_ATTN, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sparge_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), ctypes.byref(shape), _ptr(kv_idx), _ptr(kv_cnt), _ptr(O),
                                _ptr(lse), _ptr(workspace), nws, _stream(stream)), "sparge_attn_fwd")
    return O


def sparge_attn_bwd(Q, K, V, kv_idx, kv_cnt, O, lse, dO, bq: int, bk: int, dQ=None, dK=None, dV=None,
                    workspace=None, stream=None):
    """Gradients of sparge_attn_fwd (O and lse from that call) for dL/dO = dO. Returns (dQ, dK, dV)."""
    _check_qkv(Q, K, V, O, dO)
    if lse is None or lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be the forward's contiguous float32 CUDA log-sum-exp [B,H,N]")
    shape = make_shape(Q, bq, bk)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    if workspace is None:
        workspace, nws = _workspace(OP_ATTN_BWD, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sparge_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), ctypes.byref(shape), _ptr(kv_idx), _ptr(kv_cnt), _ptr(O),
                                _ptr(lse), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace), nws,
                                _stream(stream)), "sparge_attn_bwd")
    return dQ, dK, dV


def sla2_attn_bwd(Q, K, V, kv_idx, kv_cnt, alpha, dO, bq: int, bk: int, dQ=None, dK=None, dV=None, dalpha=None,
                  workspace=None, stream=None):
    """Gradients of sla2_attn_fwd for dL/dO = dO. Returns (dQ, dK, dV, dalpha)."""
    _check_qkv(Q, K, V, dO)
    if alpha.dtype != torch.float32 or not alpha.is_cuda or alpha.numel() != Q.shape[1]:
        raise ValueError("alpha must be a float32 CUDA tensor with one value per head")
    shape = make_shape(Q, bq, bk)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    dalpha = torch.empty(Q.shape[1], dtype=torch.float32, device=Q.device) if dalpha is None else dalpha
    if workspace is None:
        workspace, nws = _workspace(OP_SLA2_BWD, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sla2_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), ctypes.byref(shape), _ptr(kv_idx), _ptr(kv_cnt),
                              _ptr(alpha), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dalpha), _ptr(workspace), nws,
                              _stream(stream)), "sla2_attn_bwd")
    return dQ, dK, dV, dalpha


def sparge_attn_fwd_q8(Q, K, V, kv_idx, kv_cnt, bq: int, bk: int, O=None, workspace=None, stream=None):
    """Low-bit block-sparse attention (int8 Q/K codes, e4m3 P and V codes). Returns O."""
    _check_qkv(Q, K, V)
    shape = make_shape(Q, bq, bk)
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace, nws = _workspace(OP_ATTN_Q8, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sparge_attn_fwd_q8(_ptr(Q), _ptr(K), _ptr(V), ctypes.byref(shape), _ptr(kv_idx), _ptr(kv_cnt),
                                   _ptr(O), _ptr(workspace), nws, _stream(stream)), "sparge_attn_fwd_q8")
    return O


def quant_q8_workspace_views(workspace, shape):
    """(q8, k8, v8, sq, sk, sv) views into a sparge_attn_fwd_q8 workspace, in the
    library's layout (codes [B,H,N,128] int8 / e4m3 bytes; scales fp32)."""
    B, H, N, d, bq, bk = shape.B, shape.H, shape.N, shape.d, shape.bq, shape.bk
    nqb, nkb = -(-N // bq), -(-N // bk)
    a256 = lambda n: (n + 255) // 256 * 256  # noqa: E731
    codes = a256(B * H * N * d)
    off_q8, off_k8, off_v8 = 0, codes, 2 * codes
    off_sq = 3 * codes
    off_sk = off_sq + a256(B * H * nqb * 4)
    off_sv = off_sk + a256(B * H * nkb * 4)
    w = workspace.view(torch.uint8)
    q8 = w[off_q8:off_q8 + B * H * N * d].view(torch.int8).view(B, H, N, d)
    k8 = w[off_k8:off_k8 + B * H * N * d].view(torch.int8).view(B, H, N, d)
    v8 = w[off_v8:off_v8 + B * H * N * d].view(B, H, N, d)
    sq = w[off_sq:off_sq + B * H * nqb * 4].view(torch.float32).view(B, H, nqb)
    sk = w[off_sk:off_sk + B * H * nkb * 4].view(torch.float32).view(B, H, nkb)
    sv = w[off_sv:off_sv + B * H * d * 4].view(torch.float32).view(B, H, d)
    return q8, k8, v8, sq, sk, sv


def sla2_attn_fwd(Q, K, V, kv_idx, kv_cnt, alpha, bq: int, bk: int, O=None, workspace=None, stream=None):
    """alpha * sparse + (1 - alpha) * linear (phi = elu + 1 over the blocks not kept). Returns O."""
    _check_qkv(Q, K, V)
    shape = make_shape(Q, bq, bk)
    if O is None:
        O = torch.empty_like(Q)
    if workspace is None:
        workspace, nws = _workspace(OP_SLA2, shape, Q.device)
    else:
        nws = workspace.numel() * workspace.element_size()
    _check(_lib.sla2_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), ctypes.byref(shape), _ptr(kv_idx), _ptr(kv_cnt),
                              _ptr(alpha), _ptr(O), _ptr(workspace), nws, _stream(stream)), "sla2_attn_fwd")
    return O


SITE_SELFTEST = 0xF00


def selftest_wait(limit_us: int, gave_up=None, stream=None) -> None:
    """Launches the bounded-wait self-test kernel (it waits on a barrier that
    nothing arrives on and gives up after limit_us microseconds)."""
    _check(_lib.sparge_selftest_wait(int(limit_us), _ptr(gave_up), _stream(stream)), "sparge_selftest_wait")


def device_status(stream=None) -> int:
    """Synchronises the stream, returns and clears the device error word (0 = none)."""
    code = ctypes.c_int32(0)
    rc = _lib.sparge_device_status(_stream(stream), ctypes.byref(code))
    if rc not in (OK, ERR_DEVICE_TIMEOUT):
        raise SpargeError(rc, "sparge_device_status")
    return int(code.value)


# ---------------------------------------------------------------------------
# Windowed attention and the paged cache. A single token's call takes a few
# microseconds on the GPU, so these bindings look at each argument once, pack
# the C structs in one go and hand plain addresses over.
# ---------------------------------------------------------------------------
_pack_wshape = struct.Struct("5i").pack
_pack_window = struct.Struct("4i").pack
_pack_cache = struct.Struct("4P5i4x").pack
_pack_batch = struct.Struct("3P3i4x").pack
_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The current stream's handle without an object for it.
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(fn, args, device, stream, made):
    """Calls fn(*args, stream handle) with the tensors' device current. `made`: tensors taken here; on a stream that is
    not the current one, their memory is not handed out again before that stream is done with them."""
    index = device.index
    handle = _current_handle(index)
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("the stream belongs to another device than the tensors")
        if stream.cuda_stream != handle:
            handle = stream.cuda_stream
            for t in made:
                t.record_stream(stream)
    if _get_device() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        raise SpargeError(rc, fn.__name__)


def _want(t, name, dtype, shape, device):
    if t.dtype is not dtype or t.get_device() != device.index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


def _window_args(Q, K, V, left, right, sinks, unit, lens):
    qs, ks, device = Q.shape, K.shape, Q.device
    index = device.index
    if (Q.dtype is not _BF16 or K.dtype is not _BF16 or V.dtype is not _BF16 or not Q.is_cuda or len(qs) != 4
            or len(ks) != 4 or ks != V.shape or ks[0] != qs[0] or ks[2:] != qs[2:] or K.get_device() != index
            or V.get_device() != index or not Q.is_contiguous() or not K.is_contiguous() or not V.is_contiguous()):
        raise ValueError("Q, K, V must be contiguous bf16 CUDA tensors of shape [B,H,N,d] and [B,Hkv,N,d]")
    B, H, N, d = qs
    plens = None if lens is None else _want(lens, "lens", _I32, (B,), device)
    return _pack_wshape(B, H, ks[1], N, d), _pack_window(left, right, sinks, unit), plens, device


def sparge_window_fwd(Q, K, V, left: int, right: int, sinks: int = 0, unit: int = 1, lens=None, O=None, lse=None,
                      workspace=None, stream=None):
    """Attention with a sliding window and sinks over [B,H,N,d] (K, V: [B,Hkv,N,d]); left and right count units of
    `unit` tokens, -1 for no limit; lens: int32 [B] lengths of a padded batch. Returns O (and fills lse if given).
    It needs no workspace."""
    shape, window, plens, device = _window_args(Q, K, V, left, right, sinks, unit, lens)
    made = ()
    if O is None:
        O = torch.empty_like(Q)
        made = (O,)
    else:
        _want(O, "O", _BF16, Q.shape, device)
    plse = None if lse is None else _want(lse, "lse", _F32, Q.shape[:3], device)
    _launch(_lib.sparge_window_fwd, (Q.data_ptr(), K.data_ptr(), V.data_ptr(), shape, window, plens, O.data_ptr(), plse,
                                     None, 0), device, stream, made)
    return O


def _space(workspace, n, like, made):
    """Address and bytes of the workspace: the caller's, or n bytes taken here, as `like`'s type, and added to `made`."""
    if workspace is None:
        if n == 0:
            return None, 0
        workspace = like.new_empty(-(-n // like.element_size()))
        made.append(workspace)
        return workspace.data_ptr(), n
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def sparge_window_bwd(Q, K, V, O, lse, dO, left: int, right: int, sinks: int = 0, unit: int = 1, lens=None, dQ=None,
                      dK=None, dV=None, workspace=None, stream=None):
    """Gradients of sparge_window_fwd (O and lse from that call) for dL/dO = dO. Returns (dQ, dK, dV)."""
    shape, window, plens, device = _window_args(Q, K, V, left, right, sinks, unit, lens)
    pO, pdO = _want(O, "O", _BF16, Q.shape, device), _want(dO, "dO", _BF16, Q.shape, device)
    plse = _want(lse, "lse", _F32, Q.shape[:3], device)
    made = []
    out = []
    for t, like, name in ((dQ, Q, "dQ"), (dK, K, "dK"), (dV, V, "dV")):
        if t is None:
            t = torch.empty_like(like)
            made.append(t)
        else:
            _want(t, name, _BF16, like.shape, device)
        out.append(t)
    n = _lib.sparge_window_workspace_bytes(OP_WINDOW_BWD, shape, window) if workspace is None else 0
    ws, nws = _space(workspace, n, lse, made)
    _launch(_lib.sparge_window_bwd, (Q.data_ptr(), K.data_ptr(), V.data_ptr(), shape, window, plens, pO, plse, pdO,
                                     out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws, nws), device, stream,
            made)
    return tuple(out)


def _cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu, tokens):
    """The two C structs of a paged cache and a batch of its sequences, and the device."""
    device, dtype, shape = k_pages.device, k_pages.dtype, k_pages.shape
    index = device.index
    if (not k_pages.is_cuda or len(shape) != 4 or v_pages.dtype is not dtype or v_pages.shape != shape
            or v_pages.get_device() != index or not k_pages.is_contiguous() or not v_pages.is_contiguous()):
        raise ValueError("the cache's pages must be contiguous CUDA tensors of one type and of shape [pages, Hkv, page, d]")
    if dtype is _BF16:
        kind, ek, ev = CACHE_BF16, 0, 0
        if k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache has no exponents")
    elif dtype is _E4M3:
        if k_exp is None or v_exp is None:
            raise ValueError("an e4m3 cache needs k_exp and v_exp")
        kind = CACHE_E4M3
        ek, ev = _want(k_exp, "k_exp", _U8, shape[:3], device), _want(v_exp, "v_exp", _U8, shape[:3], device)
    else:
        raise ValueError("a cache holds bfloat16 or float8_e4m3fn")
    table = page_table.shape
    B = table[0] if len(table) == 2 else -1
    if (B < 0 or page_table.dtype is not _I32 or first.dtype is not _I32 or cu.dtype is not _I32 or first.shape != (B,)
            or cu.shape != (B + 1,) or page_table.get_device() != index or first.get_device() != index
            or cu.get_device() != index or not page_table.is_contiguous() or not first.is_contiguous()
            or not cu.is_contiguous()):
        raise ValueError(f"page_table [B, max_pages], first [B] and cu [B + 1] must be contiguous int32 tensors on {device}")
    return (_pack_cache(k_pages.data_ptr(), v_pages.data_ptr(), ek, ev, *shape, kind),
            _pack_batch(page_table.data_ptr(), first.data_ptr(), cu.data_ptr(), B, table[1], tokens), device)


def _token_rows(t, name, heads, d, device):
    """Address and token stride of packed tokens [T, heads, d]: heads and channels contiguous, tokens any stride."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is not _BF16 or t.get_device() != device.index or len(shape) != 3 or shape[1] != heads or shape[2] != d
            or (shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != d)))):
        raise ValueError(f"{name} must be a bf16 tensor of shape [tokens, {heads}, {d}] on {device}, contiguous within a token")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * d


def sparge_cache_write(k, v, k_pages, v_pages, page_table, first, cu_new, k_exp=None, v_exp=None, stream=None) -> None:
    """Writes new tokens' k, v (bf16 [T,Hkv,d], any token stride) into the paged cache at positions first[b], ..."""
    T = k.shape[0]
    cache, batch, device = _cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu_new, T)
    _, Hkv, _, d = k_pages.shape
    pk, sk = _token_rows(k, "k", Hkv, d, device)
    pv, sv = _token_rows(v, "v", Hkv, d, device)
    if v.shape[0] != T:
        raise ValueError("k and v must hold the same tokens")
    _launch(_lib.sparge_cache_write, (cache, batch, pk, sk, pv, sv), device, stream, ())


def sparge_cache_read(k_pages, v_pages, page_table, first, cu, tokens: int, k_exp=None, v_exp=None, K=None, V=None,
                      stream=None):
    """The batch's positions first[b], ... (cu[b+1] - cu[b] of them, `tokens` rows in all) as bf16 (K, V) [tokens,Hkv,d]."""
    cache, batch, device = _cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu, tokens)
    shape = (tokens, k_pages.shape[1], k_pages.shape[3])
    made = []
    out = []
    for t, name in ((K, "K"), (V, "V")):
        if t is None:
            t = k_pages.new_empty(shape) if k_exp is None else torch.empty(shape, dtype=_BF16, device=device)
            made.append(t)
        else:
            _want(t, name, _BF16, shape, device)
        out.append(t)
    _launch(_lib.sparge_cache_read, (cache, batch, out[0].data_ptr(), out[1].data_ptr()), device, stream, made)
    return out[0], out[1]


def sparge_cache_attn(Q, k_pages, v_pages, page_table, first, cu_new, max_new: int, max_len: int, left: int = -1,
                      right: int = 0, sinks: int = 0, unit: int = 1, k_exp=None, v_exp=None, O=None, lse=None,
                      workspace=None, stream=None):
    """Attention of the new tokens Q (bf16 [T,H,d], any token stride), which stand at positions first[b], ... of their
    sequences, over the paged cache that holds those positions already. max_new and max_len bound a sequence's new
    tokens and its length. Returns O [T,H,d] (and fills lse [T,H] if given)."""
    T, H, d = Q.shape
    cache, batch, device = _cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu_new, T)
    pq, sq = _token_rows(Q, "Q", H, k_pages.shape[3], device)
    made = []
    if O is None:
        O = Q.new_empty((T, H, d))
        made.append(O)
    else:
        _want(O, "O", _BF16, Q.shape, device)
    plse = None if lse is None else _want(lse, "lse", _F32, (T, H), device)
    window = _pack_window(left, right, sinks, unit)
    n = 0
    if workspace is None:
        n = _lib.sparge_cache_attn_workspace_bytes(cache, batch, H, max_new, max_len, window)
    ws, nws = _space(workspace, n, page_table, made)
    _launch(_lib.sparge_cache_attn, (cache, batch, pq, sq, H, max_new, max_len, window, O.data_ptr(), plse, ws, nws),
            device, stream, made)
    return O
