"""ctypes binding of libbpa.so: the C entry points under the same names.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libbpa.  Tensors are torch CUDA tensors (PyTorch supplies device
memory and streams); their data pointers and strides are passed through the
C ABI declared in include/bpa.h.  There is no fallback: if the library is
missing or a call fails, a ``BpaError`` is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

BPA_OK, BPA_ERR_INVALID_ARG, BPA_ERR_UNSUPPORTED, BPA_ERR_WORKSPACE = 0, 1, 2, 3
BPA_ERR_CUDA, BPA_ERR_TIMEOUT, BPA_ERR_DEVICE_CHECK = 4, 5, 6
BPA_BF16, BPA_FP32 = 0, 1
BPA_OP_FWD, BPA_OP_BWD = 0, 1


class BpaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class bpa_attn_desc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("S", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_strides", ctypes.c_int64 * 3), ("k_strides", ctypes.c_int64 * 3),
        ("v_strides", ctypes.c_int64 * 3),
        ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
        ("window_left", ctypes.c_int32), ("window_right", ctypes.c_int32),
        ("bias", ctypes.c_void_p), ("bias_strides", ctypes.c_int64 * 4),
        ("query_chunk", ctypes.c_int32), ("key_chunk", ctypes.c_int32),
        ("ring_size", ctypes.c_int32), ("ring_step_begin", ctypes.c_int32),
        ("ring_step_end", ctypes.c_int32),
        ("block_idx", ctypes.c_void_p), ("sel_block", ctypes.c_int32),
        ("top_n", ctypes.c_int32), ("local_window", ctypes.c_int32),
        ("dv", ctypes.c_int32), ("o_strides", ctypes.c_int64 * 3),
        ("seqlens_q", ctypes.c_void_p), ("seqlens_kv", ctypes.c_void_p),
        ("bottom_right", ctypes.c_int32),
        ("sink", ctypes.c_void_p), ("dsink", ctypes.c_void_p),
        ("deterministic", ctypes.c_int32),
        ("dropout_threshold", ctypes.c_uint32), ("dropout_reserved", ctypes.c_uint32),
        ("dropout_seed", ctypes.c_uint64),
    ]


class bpa_cache_desc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_cache_strides", ctypes.c_int64 * 3), ("v_cache_strides", ctypes.c_int64 * 3),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class bpa_cache_batch(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("R", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("max_q", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("q_strides", ctypes.c_int64 * 2), ("o_strides", ctypes.c_int64 * 2),
        ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
        ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
        ("window_left", ctypes.c_int32), ("window_right", ctypes.c_int32),
        ("sink", ctypes.c_void_p),
        ("tree", ctypes.c_void_p), ("tree_words", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class bpa_rope_desc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("S", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("q_strides", ctypes.c_int64 * 3), ("k_strides", ctypes.c_int64 * 3),
        ("qo_strides", ctypes.c_int64 * 3), ("ko_strides", ctypes.c_int64 * 3),
        ("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
    ]


_CACHE_SIZE, _BATCH_SIZE = ctypes.sizeof(bpa_cache_desc), ctypes.sizeof(bpa_cache_batch)
_TWO_PACK = struct.Struct("@2q").pack

_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded libbpa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise BpaError(BPA_ERR_CUDA, f"{path} is missing: build it with ring_attention_gb300.build.build()")
        L = ctypes.CDLL(path)
        P, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        dp = ctypes.POINTER(bpa_attn_desc)
        L.bpa_workspace_size.argtypes, L.bpa_workspace_size.restype = [i32, dp], sz
        L.bpa_fwd.argtypes, L.bpa_fwd.restype = [dp, P, P, P, P, sz, P], ctypes.c_int
        L.bpa_bwd.argtypes, L.bpa_bwd.restype = [dp, P, P, P, P, P, P, P, P, sz, P], ctypes.c_int
        L.bpa_select_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.bpa_select_workspace_size.restype = sz
        L.bpa_select_blocks.argtypes = [P, P, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int64),
                                        ctypes.POINTER(ctypes.c_int64), i32, i32, P, P, sz, P]
        L.bpa_select_blocks.restype = ctypes.c_int
        L.bpa_check.argtypes, L.bpa_check.restype = [P], ctypes.c_int
        L.bpa_status_string.argtypes, L.bpa_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        L.bpa_last_error.argtypes, L.bpa_last_error.restype = [], ctypes.c_char_p
        L.bpa_version.argtypes, L.bpa_version.restype = [], i32
        L.bpa_debug_wait_timeout.argtypes = [P, sz, ctypes.c_uint64, P]
        L.bpa_debug_wait_timeout.restype = ctypes.c_int
        L.bpa_select_noalloc_max_bytes.argtypes, L.bpa_select_noalloc_max_bytes.restype = [], sz
        L.bpa_select_blocks_noalloc.argtypes = [P, P, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int64),
                                                ctypes.POINTER(ctypes.c_int64), i32, i32, P, P]
        L.bpa_select_blocks_noalloc.restype = ctypes.c_int
        L.bpa_set_phase_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i32]
        L.bpa_set_phase_events.restype = None
        # descriptors and strides of the cache calls: a pointer, byref(...) or packed bytes
        L.bpa_cache_plan.argtypes = [i32] * 5 + [P] * 12 + [sz, P]
        L.bpa_cache_plan.restype = ctypes.c_int
        L.bpa_cache_append.argtypes = [P, P, P, P, P, P, i32, i32, P, sz, P]
        L.bpa_cache_append.restype = ctypes.c_int
        L.bpa_cache_attn_workspace_size.argtypes, L.bpa_cache_attn_workspace_size.restype = [P, P], sz
        L.bpa_cache_attn.argtypes = [P, P, P, P, P, P, sz, P]
        L.bpa_cache_attn.restype = ctypes.c_int
        L.bpa_cache_tree.argtypes, L.bpa_cache_tree.restype = [i32, i32, i32, P, P, P, P, P, P, sz, P], ctypes.c_int
        L.bpa_cache_tree_window.argtypes, L.bpa_cache_tree_window.restype = [i32] * 4 + [P] * 6 + [sz, P], ctypes.c_int
        L.bpa_cache_keep.argtypes = [P, i32, i32, i32, P, i32, P, P, P, P, P, sz, P]
        L.bpa_cache_keep.restype = ctypes.c_int
        L.bpa_cache_fork.argtypes, L.bpa_cache_fork.restype = [i32] * 5 + [P] * 12 + [sz, P], ctypes.c_int
        L.bpa_cache_release.argtypes, L.bpa_cache_release.restype = [i32] * 4 + [P] * 9 + [sz, P], ctypes.c_int
        L.bpa_cache_copy.argtypes, L.bpa_cache_copy.restype = [P, i32, P, P, P, sz, P], ctypes.c_int
        L.bpa_rope_fwd.argtypes, L.bpa_rope_fwd.restype = [P, P, P, P], ctypes.c_int
        L.bpa_rope_workspace_size.argtypes, L.bpa_rope_workspace_size.restype = [P], sz
        L.bpa_rope_bwd.argtypes, L.bpa_rope_bwd.restype = [P, P, P, P, P, P, P, P, sz, P], ctypes.c_int
        _lib = L
    return _lib


def _raise_if(status: int, what: str):
    if status != BPA_OK:
        L = lib()
        raise BpaError(status, f"{what}: {L.bpa_status_string(status).decode()}: {L.bpa_last_error().decode()}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BPA_BF16
    if t.dtype == torch.float32:
        return BPA_FP32
    raise TypeError(f"tensors must be bfloat16 or float32, got {t.dtype}")


def _bshd_strides(t: torch.Tensor, name: str):
    if t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D BSHD tensor")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return (t.stride(0), t.stride(1), t.stride(2))


def _stream_ptr(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def make_desc(q, k, v, *, o=None, causal=False, window=(-1, -1), scale=None, bias=None, query_chunk=0,
              key_chunk=0, ring_size=1, ring_steps=None, block_idx=None, sel_block=0, top_n=0,
              local_window=0, seqlens_q=None, seqlens_kv=None, bottom_right=False, sink=None,
              dsink=None, deterministic=False, dropout_p=0.0, dropout_seed=0) -> bpa_attn_desc:
    """Fill a bpa_attn_desc from torch tensors (no data is touched).  The value head dim
    is v's last dim; o (the output, or dout, which shares its strides) sets o_strides."""
    B, S, Hq, d = q.shape
    Hkv = k.shape[2]
    D = bpa_attn_desc()
    D.struct_size = ctypes.sizeof(bpa_attn_desc)
    D.dtype = _dtype_code(q)
    D.B, D.S, D.Hq, D.Hkv, D.d = B, S, Hq, Hkv, d
    D.q, D.k, D.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    D.q_strides[:] = _bshd_strides(q, "q")
    D.k_strides[:] = _bshd_strides(k, "k")
    D.v_strides[:] = _bshd_strides(v, "v")
    D.dv = v.shape[3]
    if o is not None:
        if o.shape[:3] != q.shape[:3] or o.shape[3] != v.shape[3]:
            raise ValueError("o / dout must be [B, S, Hq, dv]")
        D.o_strides[:] = _bshd_strides(o, "o")
    D.scale = 0.0 if scale is None else float(scale)
    D.causal = int(bool(causal))
    wl, wr = (-1, -1) if window is None else window
    D.window_left, D.window_right = int(wl), int(wr)
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() != 4:
            raise ValueError("bias must be a 4-D float32 tensor [B|1, Hq|1, S|1, S|1]")
        D.bias = bias.data_ptr()
        D.bias_strides[:] = [0 if bias.shape[i] == 1 else bias.stride(i) for i in range(4)]
    D.query_chunk, D.key_chunk = int(query_chunk), int(key_chunk)
    D.ring_size = int(ring_size)
    if ring_steps is not None:
        D.ring_step_begin, D.ring_step_end = int(ring_steps[0]), int(ring_steps[1])
    if block_idx is not None:
        if block_idx.dtype != torch.int32 or not block_idx.is_contiguous():
            raise ValueError("block_idx must be a contiguous int32 tensor")
        D.block_idx = block_idx.data_ptr()
        D.sel_block, D.top_n, D.local_window = int(sel_block), int(top_n), int(local_window)
    for name, lens in (("seqlens_q", seqlens_q), ("seqlens_kv", seqlens_kv)):
        if lens is not None:
            if lens.dtype != torch.int32 or lens.shape != (B,) or not lens.is_contiguous() or lens.device != q.device:
                raise ValueError(f"{name} must be a contiguous int32 [B] tensor on q's device")
            setattr(D, name, lens.data_ptr())
    D.bottom_right = int(bool(bottom_right))
    for name, t in (("sink", sink), ("dsink", dsink)):
        if t is not None:
            if t.dtype != torch.float32 or t.shape != (Hq,) or not t.is_contiguous() or t.device != q.device:
                raise ValueError(f"{name} must be a contiguous float32 [Hq] tensor on q's device")
            setattr(D, name, t.data_ptr())
    D.deterministic = int(bool(deterministic))
    D.dropout_threshold = dropout_threshold(dropout_p)
    D.dropout_seed = int(dropout_seed) & (2 ** 64 - 1)
    return D


def dropout_threshold(p: float) -> int:
    """The descriptor's dropout threshold for drop probability p: round(p * 2^32), at most
    2^32 - 1 (entries whose 32-bit draw is below it are dropped)."""
    p = float(p)
    if not 0.0 <= p < 1.0:
        raise ValueError("dropout_p must be in [0, 1)")
    return min(int(round(p * 4294967296.0)), 4294967295)


def bpa_workspace_size(op: int, desc: bpa_attn_desc) -> int:
    return int(lib().bpa_workspace_size(op, ctypes.byref(desc)))


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device buffer of at least nbytes, 256-byte aligned (torch's allocator aligns to 512)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def bpa_fwd(q, k, v, *, o=None, m=None, l=None, workspace_buf=None, stream=None, **kw):
    """Forward pass.  Returns (o, m, l): o [B, S, Hq, dv] (v's head dim); m and l are
    float32 [B, Hq, S]."""
    B, S, Hq, _ = q.shape
    if o is None:
        if v.shape[3] == q.shape[3]:
            o = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
        else:
            o = torch.empty(q.shape[:3] + (v.shape[3],), dtype=q.dtype, device=q.device)
    D = make_desc(q, k, v, o=o, **kw)
    if m is None:
        m = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    if l is None:
        l = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    if o.dtype != q.dtype:
        raise ValueError("o must have the dtype of q")
    need = bpa_workspace_size(BPA_OP_FWD, D)
    if need == 0:
        _raise_if(BPA_ERR_INVALID_ARG, "bpa_workspace_size")
    ws = workspace(need, q.device) if workspace_buf is None else workspace_buf
    st = lib().bpa_fwd(ctypes.byref(D), o.data_ptr(), m.data_ptr(), l.data_ptr(), ws.data_ptr(),
                       ws.numel(), _stream_ptr(stream))
    _raise_if(st, "bpa_fwd")
    return o, m, l


def bpa_bwd(q, k, v, o, dout, m, l, *, dq=None, dk=None, dv=None, workspace_buf=None, stream=None, **kw):
    """Backward pass.  Returns (dq, dk, dv) with the dtypes and strides of q, k, v;
    o and dout are [B, S, Hq, dv] with common strides."""
    D = make_desc(q, k, v, o=o, **kw)
    dq = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device) if dq is None else dq
    dk = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device) if dk is None else dk
    dv = torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device=v.device) if dv is None else dv
    for name, a, b in (("o", o, q), ("dout", dout, o), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if name == "o":
            if a.dtype != b.dtype:
                raise ValueError("o must have the dtype of q")
            continue
        if a.stride() != b.stride() or a.dtype != b.dtype:
            raise ValueError(f"{name} must share dtype and strides with its input")
    need = bpa_workspace_size(BPA_OP_BWD, D)
    if need == 0:
        _raise_if(BPA_ERR_INVALID_ARG, "bpa_workspace_size")
    ws = workspace(need, q.device) if workspace_buf is None else workspace_buf
    st = lib().bpa_bwd(ctypes.byref(D), o.data_ptr(), dout.data_ptr(), m.data_ptr(), l.data_ptr(),
                       dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), ws.numel(),
                       _stream_ptr(stream))
    _raise_if(st, "bpa_bwd")
    return dq, dk, dv


def bpa_select_blocks(q, k, *, block_size=32, top_n=8, out=None, workspace_buf=None, stream=None):
    """Exact top-n block selection: int32 [B, H, S/block_size, top_n]."""
    B, S, H, d = q.shape
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("q and k must share shape and dtype")
    qs = (ctypes.c_int64 * 3)(*_bshd_strides(q, "q"))
    ks = (ctypes.c_int64 * 3)(*_bshd_strides(k, "k"))
    nblk = S // block_size if block_size > 0 else 0
    if out is None:
        out = torch.empty((B, H, nblk, top_n), dtype=torch.int32, device=q.device)
    need = int(lib().bpa_select_workspace_size(B, S, H, d, block_size))
    if need == 0:
        raise BpaError(BPA_ERR_INVALID_ARG, "bpa_select_workspace_size: invalid sizes")
    ws = workspace(need, q.device) if workspace_buf is None else workspace_buf
    st = lib().bpa_select_blocks(q.data_ptr(), k.data_ptr(), _dtype_code(q), B, S, H, d, qs, ks,
                                 block_size, top_n, out.data_ptr(), ws.data_ptr(), ws.numel(),
                                 _stream_ptr(stream))
    _raise_if(st, "bpa_select_blocks")
    return out


def bpa_select_blocks_noalloc(q, k, *, block_size=32, top_n=8, out=None, stream=None):
    """bpa_select_blocks without a workspace: the library's built-in scratch buffer is used."""
    B, S, H, d = q.shape
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("q and k must share shape and dtype")
    qs = (ctypes.c_int64 * 3)(*_bshd_strides(q, "q"))
    ks = (ctypes.c_int64 * 3)(*_bshd_strides(k, "k"))
    nblk = S // block_size if block_size > 0 else 0
    if out is None:
        out = torch.empty((B, H, nblk, top_n), dtype=torch.int32, device=q.device)
    st = lib().bpa_select_blocks_noalloc(q.data_ptr(), k.data_ptr(), _dtype_code(q), B, S, H, d, qs, ks,
                                         block_size, top_n, out.data_ptr(), _stream_ptr(stream))
    _raise_if(st, "bpa_select_blocks_noalloc")
    return out


def bpa_check(workspace_buf: torch.Tensor) -> None:
    """Raises BpaError if a kernel of the last call on this workspace reported a fault."""
    _raise_if(lib().bpa_check(workspace_buf.data_ptr()), "bpa_check")


def bpa_set_phase_events(events) -> None:
    """Record these torch.cuda.Event objects at the phase boundaries of the next
    bpa_fwd / bpa_bwd call on this thread (None clears the hook)."""
    if events is None:
        lib().bpa_set_phase_events(None, 0)
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    lib().bpa_set_phase_events(arr, len(events))


def bpa_debug_wait_timeout(workspace_buf: torch.Tensor, limit_ns: int, stream=None) -> None:
    st = lib().bpa_debug_wait_timeout(workspace_buf.data_ptr(), workspace_buf.numel(), int(limit_ns),
                                      _stream_ptr(stream))
    _raise_if(st, "bpa_debug_wait_timeout")


# ---- paged 8-bit key / value cache --------------------------------------------------------------
# A generation step is a few microseconds of device time, so these calls marshal leanly: descriptors
# are packed in one go (the layouts of bpa_cache_desc and bpa_cache_batch) and each tensor is looked
# at once.  stream (of any of them): a torch stream of the tensors' device instead of torch's current one;
# as for torch's own operators, the caller orders it behind the writers of the tensors passed in and in
# front of the readers of what comes back.
_CACHE_PACK = struct.Struct("@I7iPP6qPP").pack
_BATCH_PACK = struct.Struct("@I5iP4qPPPf3iPP2i").pack
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_CODES = {torch.bfloat16: BPA_BF16, torch.float32: BPA_FP32}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_empty, _current_device = torch.empty, torch.cuda.current_device


def _i32_buffer(t, name, shape, dev):
    """The address of a contiguous int32 tensor of this shape on device number dev (-1: the CPU)."""
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor, got {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors, got {t.device}")
    return t.data_ptr()


def _int32(x, name):
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must lie in [-2^31, 2^31), got {x}")
    return x


def _check_workspace(t, dev):
    if t is not None and (t.dtype is not _U8 or not t.is_contiguous() or t.get_device() != dev):
        raise ValueError("workspace_buf must be a contiguous uint8 tensor on the device of the other tensors")


def _enter(dev, stream):
    """(guard, stream pointer, other) for device number dev: what to leave again (None: nothing), the
    stream of the call (``stream``, or torch's current one) and whether that is not torch's current one.
    It is then made current for the call: torch's allocator orders memory by the stream that it was
    asked for on, so what the call makes must come from the stream whose kernels use it."""
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream must be one of the tensors' device {dev}, got one of {stream.device}")
    ptr = torch._C._cuda_getCurrentRawStream(dev)
    other = stream is not None and stream.cuda_stream != ptr
    guard = None
    if other:
        guard, ptr = torch.cuda.stream(stream), stream.cuda_stream
    elif dev != _current_device():
        guard = torch.cuda.device(dev)
    if guard is not None:
        guard.__enter__()
    return guard, ptr, other


def _leave(guard, other, dev, outs):
    """Undoes _enter; outputs made on another stream than torch's current one are marked for that one,
    where the caller may use and drop them."""
    if guard is not None:
        guard.__exit__(None, None, None)
    if other:
        for t in outs:
            t.record_stream(torch.cuda.current_stream(dev))


def _ints(device, outs, shapes, ws, made):
    """The workspace; int32 tensors in the place of the None of outs.  (Parts of one buffer instead of tensors of their
    own: measured, splitting it costs more than the allocations.)  The caller holds the workspace until it has launched."""
    for i, t in enumerate(outs):
        if t is None:
            outs[i] = t = _empty(shapes[i], dtype=_I32, device=device)
            made.append(t)
    return _empty(256, dtype=_U8, device=device) if ws is None else ws


def _masks(tree):
    return 0 if tree is None else tree.data_ptr()


def _pack_cache(k_cache, v_cache, k_scale, v_scale, dtype):
    """(packed bpa_cache_desc, Hkv, d, dv, device number) of the cache's tensors."""
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"tensors must be bfloat16 or float32, got {dtype}")
    ks, vs, kst, vst = k_cache.shape, v_cache.shape, k_cache.stride(), v_cache.stride()
    for name, c, sh, st in (("k_cache", k_cache, ks, kst), ("v_cache", v_cache, vs, vst)):
        if c.dtype not in _E4M3 or len(sh) != 4 or (st[3] != 1 and sh[3] != 1):
            raise ValueError(f"{name} must be a 4-D [pages, Hkv, page_size, channels] tensor of uint8 or "
                             "float8_e4m3fn with contiguous channels")
    pages, Hkv, P, d = ks
    pages_v, Hkv_v, P_v, dv = vs
    if pages_v != pages or Hkv_v != Hkv or P_v != P:
        raise ValueError("k_cache and v_cache must share pages, heads and page size")
    dev, per_page = k_cache.get_device(), (pages, Hkv)
    for name, c in (("k_scale", k_scale), ("v_scale", v_scale)):
        if c.dtype is not _F32 or c.shape != per_page or not c.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [{pages}, {Hkv}] tensor")
    if v_cache.get_device() != dev or k_scale.get_device() != dev or v_scale.get_device() != dev:
        raise ValueError("the cache's tensors must be on one device")
    return _CACHE_PACK(_CACHE_SIZE, code, Hkv, d, dv, P, pages, 0, k_cache.data_ptr(), v_cache.data_ptr(), kst[0],
                       kst[1], kst[2], vst[0], vst[1], vst[2], k_scale.data_ptr(), v_scale.data_ptr()), Hkv, d, dv, dev


def make_cache_desc(k_cache, v_cache, k_scale, v_scale, dtype) -> bpa_cache_desc:
    """A bpa_cache_desc of the cache's tensors (no data is touched): k_cache [pages, Hkv, page_size,
    d], v_cache [pages, Hkv, page_size, dv] (uint8 or float8_e4m3fn, last dim contiguous; a [pages,
    page_size, Hkv, d] cache is passed as its transpose(1, 2)), scales float32 [pages, Hkv].
    dtype: of the tensors beside the cache."""
    return bpa_cache_desc.from_buffer_copy(_pack_cache(k_cache, v_cache, k_scale, v_scale, dtype)[0])


def _rows_strides(t, name, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on the device of the cache, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    st = t.stride()
    if st[2] != 1 and shape[2] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return st


def bpa_cache_plan(ctx_lens, new_lens, page_table, free_pages, free_count, *, page_size, T, ctx_lens_out=None,
                   free_count_out=None, kv_lens=None, cu_q=None, slot_map=None, positions=None, workspace_buf=None,
                   stream=None):
    """Block tables and slot maps of one step: page_table [R, max_pages] gets the new pages' ids
    (from the end of free_pages [num_pages], of which free_count [1] are free), and returned are
    (kv_lens [R], cu_q [R + 1], slot_map [T], positions [T], ctx_lens_out [R], free_count_out [1]),
    all int32.  ctx_lens_out=ctx_lens and free_count_out=free_count update in place."""
    if ctx_lens.dim() != 1 or page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("ctx_lens must be [R], page_table [R, max_pages], free_pages [num_pages]")
    dev, R, T, page_size = ctx_lens.get_device(), ctx_lens.shape[0], _int32(T, "T"), _int32(page_size, "page_size")
    rows, max_pages = page_table.shape
    if rows != R:
        raise ValueError(f"page_table has {rows} rows for {R} requests")
    num_pages, each, one = free_pages.shape[0], (R,), (1,)
    ins = (_i32_buffer(ctx_lens, "ctx_lens", each, dev), _i32_buffer(new_lens, "new_lens", each, dev),
           _i32_buffer(free_pages, "free_pages", (num_pages,), dev), _i32_buffer(free_count, "free_count", one, dev),
           _i32_buffer(page_table, "page_table", (R, max_pages), dev))
    outs = [kv_lens, cu_q, slot_map, positions, ctx_lens_out, free_count_out]
    shapes = (each, (R + 1,), (T,), (T,), each, one)
    for t, name, shape in zip(outs, ("kv_lens", "cu_q", "slot_map", "positions", "ctx_lens_out", "free_count_out"), shapes):
        if t is not None:
            _i32_buffer(t, name, shape, dev)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    made = []
    try:
        where = ctx_lens.device
        for i in range(6):
            if outs[i] is None:
                outs[i] = _empty(shapes[i], dtype=_I32, device=where)
                made.append(outs[i])
        if workspace_buf is None:
            workspace_buf = _empty(256, dtype=_U8, device=where)
        st = lib().bpa_cache_plan(R, T, page_size, num_pages, max_pages, *ins, *[t.data_ptr() for t in outs],
                                  workspace_buf.data_ptr(), workspace_buf.numel(), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_cache_plan")
    return tuple(outs)


def bpa_cache_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, *, max_new=0, workspace_buf=None,
                     stream=None):
    """Write rows k [T, Hkv, d], v [T, Hkv, dv] into the cache's slots slot_map [T] (-1: skipped),
    updating k_cache, v_cache, k_scale, v_scale in place."""
    dtype = k.dtype
    cache, Hkv, d, dv, dev = _pack_cache(k_cache, v_cache, k_scale, v_scale, dtype)
    T = k.shape[0]
    ks = _rows_strides(k, "k", (T, Hkv, d), dtype, dev)
    vs = _rows_strides(v, "v", (T, Hkv, dv), dtype, dev)
    slots, max_new = _i32_buffer(slot_map, "slot_map", (T,), dev), _int32(max_new, "max_new")
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    try:
        if workspace_buf is None:
            workspace_buf = _empty(256, dtype=_U8, device=k.device)
        st = lib().bpa_cache_append(cache, k.data_ptr(), v.data_ptr(), _TWO_PACK(ks[0], ks[1]), _TWO_PACK(vs[0], vs[1]),
                                    slots, T, max_new, workspace_buf.data_ptr(), workspace_buf.numel(), ptr)
    finally:
        _leave(guard, other, dev, ())
    if st:
        _raise_if(st, "bpa_cache_append")


def _pack_batch(q, o_row, o_head, page_table, kv_lens, cu_q, max_q, causal, window, scale, sink, tree):
    """Packed bpa_cache_batch; o_row, o_head: the output's strides."""
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q must be [T, Hq, d], page_table [R, max_pages]")
    shape, dev, (R, max_pages) = q.shape, q.get_device(), page_table.shape
    T, Hq, _ = shape
    st = _rows_strides(q, "q", shape, q.dtype, dev)
    if sink is not None and (sink.dtype is not _F32 or sink.shape != (Hq,) or not sink.is_contiguous() or
                             sink.get_device() != dev):
        raise ValueError("sink must be a contiguous float32 [Hq] tensor on q's device")
    words = 0
    if tree is not None:
        if tree.dtype is not _I32 or tree.dim() != 2 or tree.shape[0] != T or not tree.is_contiguous() or tree.get_device() != dev:
            raise ValueError("tree must be a contiguous int32 [T, words] tensor on q's device")
        words = tree.shape[1]
        if words < 1:                      # torch gives such a tensor no address, and NULL is no tree
            raise ValueError("tree must have a word a row")
    wl, wr = (-1, -1) if window is None else window
    return _BATCH_PACK(_BATCH_SIZE, R, T, Hq, max_pages, _int32(max_q, "max_q"), q.data_ptr(), st[0], st[1], o_row, o_head,
                       _i32_buffer(page_table, "page_table", (R, max_pages), dev), _i32_buffer(kv_lens, "kv_lens", (R,), dev),
                       _i32_buffer(cu_q, "cu_q", (R + 1,), dev), 0.0 if scale is None else float(scale),
                       1 if causal else 0, _int32(wl, "window"), _int32(wr, "window"), 0 if sink is None else sink.data_ptr(),
                       _masks(tree), words, 0)


def make_cache_batch(q, page_table, kv_lens, cu_q, *, max_q=0, causal=True, window=(-1, -1), scale=None,
                     sink=None, tree=None) -> bpa_cache_batch:
    """A bpa_cache_batch (all but o_strides) of the step's tensors (no data is touched); keywords as
    bpa_cache_attn's."""
    return bpa_cache_batch.from_buffer_copy(_pack_batch(q, 0, 0, page_table, kv_lens, cu_q, max_q, causal, window, scale,
                                                        sink, tree))


def bpa_cache_attn_workspace_size(cache: bpa_cache_desc, batch: bpa_cache_batch) -> int:
    return int(lib().bpa_cache_attn_workspace_size(ctypes.byref(cache), ctypes.byref(batch)))


def bpa_cache_attn(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, cu_q, *, max_q=0, causal=True,
                   window=(-1, -1), scale=None, sink=None, tree=None, o=None, m=None, l=None, workspace_buf=None, stream=None):
    """Attention of packed rows q [T, Hq, d] over the cache.  Returns (o, m, l): o [T, Hq, dv]; m and
    l float32 [Hq, T].  Rows behind cu_q[R] are left as they are.  max_q: the most rows of a
    request (0: unknown, and single tokens then take half as long again), guides the choice of kernel.
    tree: int32 [T, words] masks of drafted trees (bpa_cache_tree's for the same window, or the caller's)."""
    dtype = q.dtype
    cache, _, d, dv, dev = _pack_cache(k_cache, v_cache, k_scale, v_scale, dtype)
    if q.dim() != 3 or q.shape[2] != d or q.get_device() != dev:
        raise ValueError("q must be [T, Hq, d] with k_cache's head dim and device")
    T, Hq, _ = q.shape
    stats = (Hq, T)
    for t, name in ((m, "m"), (l, "l")):
        if t is not None and (t.dtype is not _F32 or t.shape != stats or not t.is_contiguous() or t.get_device() != dev):
            raise ValueError(f"{name} must be a contiguous float32 [Hq, T] tensor on q's device")
    st = (Hq * dv, dv) if o is None else _rows_strides(o, "o", (T, Hq, dv), dtype, dev)
    batch = _pack_batch(q, st[0], st[1], page_table, kv_lens, cu_q, max_q, causal, window, scale, sink, tree)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    made = []
    try:
        L, where = lib(), q.device
        if o is None:
            o = _empty((T, Hq, dv), dtype=dtype, device=where)
            made.append(o)
        if m is None:
            m = _empty(stats, dtype=_F32, device=where)
            made.append(m)
        if l is None:
            l = _empty(stats, dtype=_F32, device=where)
            made.append(l)
        if workspace_buf is None:
            need = L.bpa_cache_attn_workspace_size(cache, batch)
            if need == 0:
                _raise_if(BPA_ERR_INVALID_ARG, "bpa_cache_attn_workspace_size")
            workspace_buf = _empty(need, dtype=_U8, device=where)
        st = L.bpa_cache_attn(cache, batch, o.data_ptr(), m.data_ptr(), l.data_ptr(), workspace_buf.data_ptr(),
                              workspace_buf.numel(), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_cache_attn")
    return o, m, l


def bpa_cache_tree(parents, kv_lens, cu_q, *, words, window=(-1, -1), tree=None, positions=None, workspace_buf=None, stream=None):
    """Masks of drafted trees: parents [T] names each packed row's parent among its request's rows (-1: the
    context).  Returns (tree [T, words], positions [T]), int32: a row's own bit and its ancestors', and its place
    in the sequence.  words: of 32 rows each, for the largest request.  window: of the bpa_cache_attn that the masks are for
    (its right bound says nothing under a tree): ancestors further up than its left bound are left out."""
    if parents.dim() != 1 or kv_lens.dim() != 1:
        raise ValueError("parents must be [T], kv_lens [R]")
    dev, T, R, words = parents.get_device(), parents.shape[0], kv_lens.shape[0], _int32(words, "words")
    wl, wr = (-1, -1) if window is None else window
    wl, wr = _int32(wl, "window"), _int32(wr, "window")
    if wl < -1 or wr < -1:
        raise ValueError(f"window bounds must be >= -1, got {window}")
    ins = (_i32_buffer(parents, "parents", (T,), dev), _i32_buffer(kv_lens, "kv_lens", (R,), dev),
           _i32_buffer(cu_q, "cu_q", (R + 1,), dev))
    if tree is None and not 1 <= words <= 32:
        raise ValueError(f"words must lie in [1, 32], got {words}")
    for t, name, shape in ((tree, "tree", (T, words)), (positions, "positions", (T,))):
        if t is not None:
            _i32_buffer(t, name, shape, dev)
    _check_workspace(workspace_buf, dev)
    outs, made = [tree, positions], []
    guard, ptr, other = _enter(dev, stream)
    try:
        ws = _ints(parents.device, outs, ((T, words), (T,)), workspace_buf, made)
        rest = (*ins, outs[0].data_ptr(), outs[1].data_ptr(), ws.data_ptr(), ws.numel(), ptr)
        st = lib().bpa_cache_tree(R, T, words, *rest) if wl < 0 else lib().bpa_cache_tree_window(R, T, words, wl, *rest)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_cache_tree")
    return outs[0], outs[1]


def bpa_cache_keep(keep, keep_count, kv_lens, cu_q, page_table, k_cache, v_cache, k_scale, v_scale, *, workspace_buf=None,
                   stream=None):
    """Keep the accepted tokens keep [R, max_keep] (ascending indexes of a request's new rows, the first
    keep_count [R] of them) at the end of the context, in place in k_cache, v_cache, k_scale, v_scale.
    kv_lens, cu_q: of the step that appended them."""
    cache, _, _, _, dev = _pack_cache(k_cache, v_cache, k_scale, v_scale, torch.bfloat16)
    if keep.dim() != 2 or page_table.dim() != 2:
        raise ValueError("keep must be [R, max_keep], page_table [R, max_pages]")
    (R, max_keep), max_pages = keep.shape, page_table.shape[1]
    ins = (_i32_buffer(keep_count, "keep_count", (R,), dev), _i32_buffer(kv_lens, "kv_lens", (R,), dev),
           _i32_buffer(cu_q, "cu_q", (R + 1,), dev), _i32_buffer(page_table, "page_table", (R, max_pages), dev))
    rows = _i32_buffer(keep, "keep", (R, max_keep), dev)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    try:
        if workspace_buf is None:
            workspace_buf = _empty(256, dtype=_U8, device=keep.device)
        st = lib().bpa_cache_keep(cache, R, 1 << 30, max_pages, rows, max_keep, *ins, workspace_buf.data_ptr(), workspace_buf.numel(),
                                  ptr)
    finally:
        _leave(guard, other, dev, ())
    if st:
        _raise_if(st, "bpa_cache_keep")


def bpa_cache_fork(src, dst, ctx_lens, page_table, page_refs, free_pages, free_count, *, page_size, copy_src=None, copy_dst=None,
                   ctx_lens_out=None, free_count_out=None, workspace_buf=None, stream=None):
    """Requests dst [N] become holders of what src [N] hold: full pages are shared (page_table and page_refs
    [num_pages] updated in place), a last page that is not full gets one off the free list.  Returns
    (copy_src [N], copy_dst [N], ctx_lens_out [R], free_count_out [1]), int32, the first two for
    bpa_cache_copy.  ctx_lens_out=ctx_lens and free_count_out=free_count update in place."""
    if src.dim() != 1 or ctx_lens.dim() != 1 or page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("src must be [N], ctx_lens [R], page_table [R, max_pages], free_pages [num_pages]")
    dev, N, R, page_size = src.get_device(), src.shape[0], ctx_lens.shape[0], _int32(page_size, "page_size")
    max_pages, num_pages = page_table.shape[1], free_pages.shape[0]
    ins = (_i32_buffer(src, "src", (N,), dev), _i32_buffer(dst, "dst", (N,), dev), _i32_buffer(ctx_lens, "ctx_lens", (R,), dev),
           _i32_buffer(page_table, "page_table", (R, max_pages), dev), _i32_buffer(page_refs, "page_refs", (num_pages,), dev),
           _i32_buffer(free_pages, "free_pages", (num_pages,), dev), _i32_buffer(free_count, "free_count", (1,), dev))
    outs, shapes, made = [copy_src, copy_dst, ctx_lens_out, free_count_out], ((N,), (N,), (R,), (1,)), []
    for t, name, shape in zip(outs, ("copy_src", "copy_dst", "ctx_lens_out", "free_count_out"), shapes):
        if t is not None:
            _i32_buffer(t, name, shape, dev)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    try:
        ws = _ints(src.device, outs, shapes, workspace_buf, made)
        st = lib().bpa_cache_fork(N, R, page_size, num_pages, max_pages, *ins, *[t.data_ptr() for t in outs], ws.data_ptr(), ws.numel(), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_cache_fork")
    return tuple(outs)


def bpa_cache_copy(src, dst, k_cache, v_cache, k_scale, v_scale, *, workspace_buf=None, stream=None):
    """Copy pages src [N] to pages dst [N] with their scales (-1, -1: skipped)."""
    cache, _, _, _, dev = _pack_cache(k_cache, v_cache, k_scale, v_scale, torch.bfloat16)
    if src.dim() != 1:
        raise ValueError("src must be [N]")
    N = src.shape[0]
    a, b = _i32_buffer(src, "src", (N,), dev), _i32_buffer(dst, "dst", (N,), dev)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    try:
        if workspace_buf is None:
            workspace_buf = _empty(256, dtype=_U8, device=src.device)
        st = lib().bpa_cache_copy(cache, N, a, b, workspace_buf.data_ptr(), workspace_buf.numel(), ptr)
    finally:
        _leave(guard, other, dev, ())
    if st:
        _raise_if(st, "bpa_cache_copy")


def bpa_cache_release(ctx_lens, keep_lens, page_table, page_refs, free_pages, free_count, *, page_size, ctx_lens_out=None,
                      free_count_out=None, workspace_buf=None, stream=None):
    """Requests of ctx_lens [R] tokens keep the first keep_lens [R]; pages that no request holds any more go
    to the end of free_pages, ascending (free_pages and page_refs updated in place).  Returns (ctx_lens_out [R],
    free_count_out [1]); ctx_lens_out=ctx_lens and free_count_out=free_count update in place."""
    if ctx_lens.dim() != 1 or page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("ctx_lens must be [R], page_table [R, max_pages], free_pages [num_pages]")
    dev, R, page_size = ctx_lens.get_device(), ctx_lens.shape[0], _int32(page_size, "page_size")
    max_pages, num_pages = page_table.shape[1], free_pages.shape[0]
    ins = (_i32_buffer(ctx_lens, "ctx_lens", (R,), dev), _i32_buffer(keep_lens, "keep_lens", (R,), dev),
           _i32_buffer(page_table, "page_table", (R, max_pages), dev), _i32_buffer(page_refs, "page_refs", (num_pages,), dev),
           _i32_buffer(free_pages, "free_pages", (num_pages,), dev), _i32_buffer(free_count, "free_count", (1,), dev))
    outs, shapes, made = [ctx_lens_out, free_count_out], ((R,), (1,)), []
    for t, name, shape in zip(outs, ("ctx_lens_out", "free_count_out"), shapes):
        if t is not None:
            _i32_buffer(t, name, shape, dev)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    try:
        ws = _ints(ctx_lens.device, outs, shapes, workspace_buf, made)
        st = lib().bpa_cache_release(R, page_size, num_pages, max_pages, *ins, *[t.data_ptr() for t in outs], ws.data_ptr(), ws.numel(), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_cache_release")
    return tuple(outs)


# ---- norms of q and k with the position rotation ---------------------------------------------------
# The same lean marshalling (one packed bpa_rope_desc) and the same meaning of stream as above.
_ROPE_PACK = struct.Struct("@I9ifiPP12qPPPP").pack
_ROPE_SIZE = ctypes.sizeof(bpa_rope_desc)


def _heads_of(t, name, shape, dtype, dev):
    """(b, s, h) strides of a [B, S, H, d] or packed [T, H, d] tensor."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on the device of the others, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return st[:3] if len(shape) == 4 else (0, st[0], st[1])


def _pack_rope(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved, q_like, k_like):
    """Packed bpa_rope_desc; q_like, k_like: the tensors that give the strides behind norm and rotation."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    shape, dtype, dev = first.shape, first.dtype, first.get_device()
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"tensors must be bfloat16 or float32, got {dtype}")
    if len(shape) not in (3, 4):
        raise ValueError("q and k must be [B, S, H, d] or packed [T, H, d]")
    rows, d = shape[:-2], shape[-1]
    B, S = rows if len(rows) == 2 else (1, rows[0])
    sides = []
    for t, like, name in ((q, q_like, "q"), (k, k_like, "k")):
        if t is None:
            sides.append((0, 0, (0, 0, 0), (0, 0, 0)))
            continue
        if t.dim() != len(shape) or t.shape[:-2] != rows or t.shape[-1] != d:
            raise ValueError("q and k must share rows and head dim")
        st = _heads_of(t, name, t.shape, dtype, dev)
        sides.append((t.shape[-2], t.data_ptr(), st, st if like is None else _heads_of(like, name + "'s output or its gradient",
                                                                                      t.shape, dtype, dev)))
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or inv_freq.get_device() != dev:
            raise ValueError("inv_freq must be a contiguous float32 [rot / 2] tensor on the device of the others")
        rot = 2 * inv_freq.shape[0]
    for w, t, name in ((q_weight, q, "q_weight"), (k_weight, k, "k_weight")):
        if w is not None and (w.dtype is not _F32 or w.shape != (d,) or not w.is_contiguous() or w.get_device() != dev):
            raise ValueError(f"{name} must be a contiguous float32 [d] tensor on the device of the others")
        if w is not None and t is None:
            raise ValueError(f"{name} without its tensor")
    pos = 0 if positions is None else _i32_buffer(positions, "positions", rows, dev)
    (Hq, qp, qs, qo), (Hkv, kp, ks, ko) = sides
    return _ROPE_PACK(_ROPE_SIZE, code, B, S, Hq, Hkv, d, rot, 1 if interleaved else 0, 1 if norm else 0, float(eps), 0, qp, kp,
                      *qs, *ks, *qo, *ko, pos, 0 if inv_freq is None else inv_freq.data_ptr(),
                      0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr()), dev


def make_rope_desc(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, *, norm=True, eps=1e-6, interleaved=False,
                   q_out=None, k_out=None) -> bpa_rope_desc:
    """A bpa_rope_desc of the tensors (no data is touched); arguments as bpa_rope_fwd's."""
    return bpa_rope_desc.from_buffer_copy(_pack_rope(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved,
                                                     q_out, k_out)[0])


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def bpa_rope_fwd(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, *, norm=True, eps=1e-6, interleaved=False,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q [B, S, Hq, d] and k [B, S, Hkv, d] (or packed [T, H, d]; one of them
    may be None) and the rotation of its first 2 len(inv_freq) channels by positions [B, S] or [T] (int32; None:
    0, 1, ..).  Returns (q_out, k_out); q_out=q and k_out=k work in place.  Rows of negative position are
    left as they are."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    for t, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if t is None and out is not None:
            raise ValueError(f"{name} without its tensor")
    dev = first.get_device()
    guard, ptr, other = _enter(dev, stream)
    made = []
    try:
        if q is not None and q_out is None:
            q_out = _empty(q.shape, dtype=q.dtype, device=q.device)
            made.append(q_out)
        if k is not None and k_out is None:
            k_out = _empty(k.shape, dtype=k.dtype, device=k.device)
            made.append(k_out)
        desc, _ = _pack_rope(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved, q_out, k_out)
        st = lib().bpa_rope_fwd(desc, _ptr(q_out), _ptr(k_out), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_rope_fwd")
    return q_out, k_out


def bpa_rope_workspace_size(desc: bpa_rope_desc) -> int:
    return int(lib().bpa_rope_workspace_size(ctypes.byref(desc)))


def bpa_rope_bwd(q, k, dq_out, dk_out, positions=None, inv_freq=None, q_weight=None, k_weight=None, *, norm=True, eps=1e-6,
                 interleaved=False, dq=None, dk=None, workspace_buf=None, stream=None):
    """Backward of bpa_rope_fwd: q, k its inputs, dq_out, dk_out the gradients of its outputs.  Returns
    (dq, dk, dq_weight, dk_weight): dq, dk with the strides of q, k (made dense where q, k are); the weights'
    float32 [d] gradients, None without norm or tensor.  dq may be q or dq_out where the strides agree."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    dev = first.get_device()
    for t, g, out, name in ((q, dq_out, dq, "dq"), (k, dk_out, dk, "dk")):
        if (t is None) != (g is None) or (t is None and out is not None):
            raise ValueError(f"{name}_out and {name} go with their tensor")
        if out is not None:
            a, b = _heads_of(out, name, t.shape, t.dtype, dev), _heads_of(t, name[1:], t.shape, t.dtype, dev)
            # a dimension of one never steps
            if any(x != y and n > 1 for x, y, n in zip(a, b, ((1,) + tuple(t.shape))[-4:])):
                raise ValueError(f"{name} must share the strides of its input")
    desc, _ = _pack_rope(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved, dq_out, dk_out)
    _check_workspace(workspace_buf, dev)
    guard, ptr, other = _enter(dev, stream)
    made = []
    try:
        L, grads, weights = lib(), [dq, dk], [None, None]
        for i, t in enumerate((q, k)):
            if t is None:
                continue
            if grads[i] is None:
                grads[i] = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
                made.append(grads[i])
            if norm:
                weights[i] = _empty((t.shape[-1],), dtype=_F32, device=t.device)
                made.append(weights[i])
        if workspace_buf is None:
            need = L.bpa_rope_workspace_size(desc)
            if need == 0:
                _raise_if(BPA_ERR_INVALID_ARG, "bpa_rope_workspace_size")
            workspace_buf = _empty(need, dtype=_U8, device=first.device)
        st = L.bpa_rope_bwd(desc, _ptr(dq_out), _ptr(dk_out), _ptr(grads[0]), _ptr(grads[1]), _ptr(weights[0]), _ptr(weights[1]),
                            workspace_buf.data_ptr(), workspace_buf.numel(), ptr)
    finally:
        _leave(guard, other, dev, made)
    if st:
        _raise_if(st, "bpa_rope_bwd")
    return grads[0], grads[1], weights[0], weights[1]
