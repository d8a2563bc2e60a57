"""ctypes binding of libhils.so (argument marshalling only).

Every function takes torch tensors that already live on the GPU, checks their
dtype, shape and contiguity, and passes raw pointers to the C ABI declared in
include/hils.h.  All arithmetic happens in the CUDA kernels; there is no
fallback: if the library is missing or the tensors are on the CPU, the call
raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhils.so")

HILS_F32, HILS_BF16 = 0, 1
OP_SELECT, OP_ATTEND, OP_DECODE, OP_ATTEND_SELECTED, OP_BACKWARD = 0, 1, 2, 3, 4
OP_DECODE_DENSE, OP_APPEND = 5, 6
STATUS = {
    0: "HILS_OK", 1: "HILS_ERR_INVALID_ARG", 2: "HILS_ERR_UNSUPPORTED", 3: "HILS_ERR_WORKSPACE",
    4: "HILS_ERR_CUDA", 5: "HILS_ERR_DEVICE_CHECK", 6: "HILS_ERR_DEVICE_TIMEOUT",
}


class HilsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class Shape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("seq_len", ctypes.c_int32), ("chunk", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32),
        ("window", ctypes.c_int32),
    ]


_SHAPES = {}


def _shape_of(*key):
    """make_shape's struct for these arguments, made once (the C side only reads it)."""
    s = _SHAPES.get(key)
    if s is None:
        if len(_SHAPES) > 4096:
            _SHAPES.clear()
        s = _SHAPES[key] = make_shape(*key)
    return s


_lib = None
_P = ctypes.c_void_p


def lib():
    """Loads libhils.so once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libhils.so not built ({LIB_PATH}); run "
                           "`python -m chunk_wise_hierarchical_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    S = ctypes.POINTER(Shape)
    i32, sz = ctypes.c_int32, ctypes.c_size_t
    sig = {
        "hils_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hils_abi_version": (i32, []),
        "hils_workspace_size": (i32, [S, i32, ctypes.POINTER(sz)]),
        "hils_summarize": (i32, [S, _P, _P, _P, _P, _P]),
        "hils_summarize_paged": (i32, [S, _P, _P, _P, i32, i32, _P, _P, _P]),
        "hils_select": (i32, [S, _P, _P, _P, _P, _P, _P, sz, _P]),
        "hils_attend": (i32, [S, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "hils_attend_selected": (i32, [S, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "hils_decode": (i32, [S, _P, _P, _P, _P, _P, _P, i32, _P, i32, _P, _P, _P, sz, _P]),
        "hils_summarize_paged_ex": (i32, [S, _P, _P, _P, i32, i32, _P, i32, _P, _P]),
        "hils_decode_ex": (i32, [S, _P, _P, _P, _P, i32, _P, _P, i32, _P, i32, _P, _P, _P, sz, _P]),
        "hils_decode_static": (i32, [S, _P, _P, _P, _P, _P, _P, i32, _P, i32, _P, _P, _P, _P]),
        "hils_device_status": (i32, [_P, _P]),
        "hils_set_wait_limit": (ctypes.c_uint32, [ctypes.c_uint32]),
        "hils_backward": (i32, [S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]),
        "hils_rotate": (i32, [S, _P, _P, _P, _P, ctypes.c_int64, i32, _P, _P, i32, _P]),
        "hils_append_paged": (i32, [S, _P, _P, _P, _P, i32, _P, _P, _P, _P, i32, i32, _P, _P, _P, _P, _P, sz, _P]),
        "hils_decode_dense": (i32, [S, _P, _P, _P, _P, i32, _P, i32, _P, _P, _P, sz, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


EXPORTED = ["hils_abi_version", "hils_append_paged", "hils_attend", "hils_attend_selected", "hils_backward",
            "hils_decode", "hils_decode_dense", "hils_decode_ex", "hils_decode_static", "hils_device_status",
            "hils_rotate", "hils_summarize_paged_ex", "hils_select", "hils_set_wait_limit",
            "hils_status_string", "hils_summarize", "hils_summarize_paged", "hils_workspace_size"]

DEFAULT_WAIT_LIMIT = 1 << 26  # HILS_DEFAULT_WAIT_LIMIT


def set_wait_limit(polls: int) -> int:
    """Polls of an ordinary bounded device wait before a tensor-core kernel gives up
    (process-wide; 0 gives up at once).  Returns the previous limit."""
    return int(lib().hils_set_wait_limit(int(polls)))


def device_status(ws, stream=None) -> int:
    """Reads and clears the error word of a workspace (hils_device_status)."""
    return int(lib().hils_device_status(_ptr(ws), _stream(stream)))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return HILS_BF16
    if t.dtype == torch.float32:
        return HILS_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _expect(t, shape, dtypes, name):
    """Raises unless tensor t has exactly this shape and one of these dtypes: the kernels
    read every tensor at the extent the shape implies."""
    if t is not None and t.shape == shape and (dtypes is None or t.dtype in dtypes):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _same_device(ref, *ts):
    dev = ref.device
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("every tensor must be on q's device")


def check_prefill_args(shape, q, k, v, landmark, out=None):
    """The prefill inputs against the shape: q [b,h,N,d]; k, v [b,g,N,d] and landmark
    [b,h,N//64,d] in q's dtype; out (if given) like q."""
    s = shape
    _expect(q, (s.batch, s.heads_q, s.seq_len, s.head_dim), (torch.bfloat16, torch.float32), "q")
    if _dt(q) != s.dtype:
        raise TypeError("q's dtype does not match the prepared shape")
    kv = (s.batch, s.heads_kv, s.seq_len, s.head_dim)
    _expect(k, kv, (q.dtype,), "k")
    _expect(v, kv, (q.dtype,), "v")
    if landmark is not None:
        _expect(landmark, (s.batch, s.heads_q, s.seq_len // s.chunk, s.head_dim), (q.dtype,), "landmark")
    if out is not None:
        _expect(out, q.shape, (q.dtype,), "out")
    _same_device(q, k, v, landmark, out)


def check_decode_args(shape, q, k_pages, v_pages, kbar_pages, hbias_pages, seq_lens, out=None, topk_idx=None):
    """The decode inputs against the shape: q [b,h,d]; k/v pages [P,g,64,d] in q's dtype;
    kbar pages [P,h,d] fp32 (or bf16, the compact cache); hbias pages [P,h] fp32; seq_lens
    [b] int32; topk_idx (if given) int32 with at least b*g*K entries; out (if given) like q."""
    s = shape
    _expect(q, (s.batch, s.heads_q, s.head_dim), (torch.bfloat16, torch.float32), "q")
    if _dt(q) != s.dtype:
        raise TypeError("q's dtype does not match the prepared shape")
    P = k_pages.shape[0] if k_pages.dim() == 4 else -1
    _expect(k_pages, (P, s.heads_kv, s.chunk, s.head_dim), (q.dtype,), "k_pages")
    _expect(v_pages, (P, s.heads_kv, s.chunk, s.head_dim), (q.dtype,), "v_pages")
    _expect(kbar_pages, (P, s.heads_q, s.head_dim), (torch.float32, torch.bfloat16), "kbar_pages")
    _expect(hbias_pages, (P, s.heads_q), (torch.float32,), "hbias_pages")
    _expect(seq_lens, (s.batch,), (torch.int32,), "seq_lens")
    if topk_idx is not None and (topk_idx.dtype != torch.int32 or topk_idx.numel() < s.batch * s.heads_kv * s.top_k):
        raise TypeError("topk_idx must be an int32 tensor of at least batch * heads_kv * top_k entries")
    if out is not None:
        _expect(out, q.shape, (q.dtype,), "out")
    _same_device(q, k_pages, v_pages, kbar_pages, hbias_pages, seq_lens, out, topk_idx)


def _check(st: int, where: str):
    if st != 0:
        raise HilsError(st, where)


def make_shape(batch, heads_q, heads_kv, head_dim, seq_len, top_k, dtype, chunk=64, scale=0.0, window=0):
    return Shape(batch, heads_q, heads_kv, head_dim, seq_len, chunk, top_k, float(scale or 0.0), dtype,
                 int(window or 0))


def workspace_size(shape: Shape, op: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hils_workspace_size(ctypes.byref(shape), op, ctypes.byref(out)), "hils_workspace_size")
    return out.value


def new_workspace(shape: Shape, op: int, device) -> torch.Tensor:
    """Zero-filled workspace (the error word must start cleared)."""
    n = workspace_size(shape, op)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def summarize(k, landmark, scale=None, stream=None):
    """kbar [b,h,C,d] fp32, hbias [b,h,C] fp32 of every complete chunk."""
    b, g, n, d = k.shape
    h = landmark.shape[1]
    c = n // 64
    if landmark.shape != (b, h, c, d) or landmark.dtype != k.dtype:
        raise ValueError("landmark must be [b, h, seq_len // 64, d] with k's dtype")
    sh = make_shape(b, h, g, d, n, 0, _dt(k), scale=scale or 0.0)
    kbar = torch.empty((b, h, c, d), dtype=torch.float32, device=k.device)
    hb = torch.empty((b, h, c), dtype=torch.float32, device=k.device)
    _check(lib().hils_summarize(ctypes.byref(sh), _ptr(k), _ptr(landmark), _ptr(kbar), _ptr(hb),
                                _stream(stream)), "hils_summarize")
    return kbar, hb


def summarize_paged(k_pages, landmark_pages, page_ids, kbar_pages, hbias_pages, scale=None, stream=None):
    """Writes the summaries of the listed pages into kbar_pages (fp32, or bf16 for the
    compact cache) / hbias_pages (fp32)."""
    n_pages, g, chunk, d = k_pages.shape
    h = landmark_pages.shape[1]
    if page_ids.dtype != torch.int32:
        raise TypeError("page_ids must be int32")
    _expect(landmark_pages, (n_pages, h, d), (k_pages.dtype,), "landmark_pages")
    _expect(kbar_pages, (n_pages, h, d), (torch.float32, torch.bfloat16), "kbar_pages")
    _expect(hbias_pages, (n_pages, h), (torch.float32,), "hbias_pages")
    _same_device(k_pages, landmark_pages, page_ids, kbar_pages, hbias_pages)
    sh = make_shape(0, h, g, d, 0, 0, _dt(k_pages), chunk=chunk, scale=scale or 0.0)
    _check(lib().hils_summarize_paged_ex(ctypes.byref(sh), _ptr(k_pages), _ptr(landmark_pages), _ptr(page_ids),
                                         int(page_ids.numel()), int(n_pages), _ptr(kbar_pages), _dt(kbar_pages),
                                         _ptr(hbias_pages), _stream(stream)), "hils_summarize_paged_ex")


def select(q, kbar, hbias, top_k, heads_kv, scale=None, stream=None, with_scores=True, window=0, ws=None):
    """topk_idx [b,g,N,K] int32 and (optionally) topk_score [b,h,N,K] fp32; `ws`, if
    given, is the workspace whose error word the kernels report into."""
    b, h, n, d = q.shape
    sh = make_shape(b, h, heads_kv, d, n, top_k, _dt(q), scale=scale or 0.0, window=window)
    _expect(kbar, (b, h, n // 64, d), (torch.float32,), "kbar")
    _expect(hbias, (b, h, n // 64), (torch.float32,), "hbias")
    _same_device(q, kbar, hbias, ws)
    idx = torch.empty((b, heads_kv, n, top_k), dtype=torch.int32, device=q.device)
    sc = torch.empty((b, h, n, top_k), dtype=torch.float32, device=q.device) if with_scores else None
    if ws is None:
        ws = new_workspace(sh, OP_SELECT, q.device)
    _check(lib().hils_select(ctypes.byref(sh), _ptr(q), _ptr(kbar), _ptr(hbias), _ptr(idx), _ptr(sc),
                             _ptr(ws), ws.numel(), _stream(stream)), "hils_select")
    return idx, sc


class Prefill:
    """Reusable prefill call: holds the workspace for one shape."""

    def __init__(self, batch, heads_q, heads_kv, seq_len, head_dim, top_k, dtype, scale=None, device="cuda",
                 window=0):
        self.shape = make_shape(batch, heads_q, heads_kv, head_dim, seq_len, top_k,
                                HILS_BF16 if dtype in (torch.bfloat16, "bf16") else HILS_F32,
                                scale=scale or 0.0, window=window)
        self.ws = new_workspace(self.shape, OP_ATTEND, device)

    def __call__(self, q, k, v, landmark, out=None, topk_idx=None, stream=None, lse=None):
        s = self.shape
        check_prefill_args(s, q, k, v, landmark, out)
        _same_device(q, lse, topk_idx, self.ws)
        if out is None:
            out = torch.empty_like(q)
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:3]):
            raise ValueError("lse must be fp32 [b, h, seq_len]")
        if topk_idx is not None and (topk_idx.dtype != torch.int32 or
                                     topk_idx.shape != (s.batch, s.heads_kv, s.seq_len, s.top_k)):
            raise ValueError("topk_idx must be int32 [b, heads_kv, seq_len, top_k]")
        _check(lib().hils_attend(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(landmark), _ptr(out),
                                 _ptr(lse), _ptr(topk_idx), _ptr(self.ws), self.ws.numel(), _stream(stream)),
               "hils_attend")
        return out

    def device_status(self, stream=None):
        return lib().hils_device_status(_ptr(self.ws), _stream(stream))


def attend(q, k, v, landmark, top_k, scale=None, stream=None, return_idx=False, q_score=None, window=0,
           return_lse=False):
    """HiLS prefill forward; returns out, then topk_idx and lse [b,h,N] (log Zhat)
    when asked.

    q_score: a separate scoring query (the Q-Cal interface): summaries, then
    hils_select with q_score, then hils_attend_selected with q.  window: 0 (the
    own-chunk local branch) or a multiple of 64 (a chunk-aligned sliding window)."""
    b, h, n, d = q.shape
    g = k.shape[1]
    lse = torch.empty((b, h, n), dtype=torch.float32, device=q.device) if return_lse else None
    if q_score is not None:
        if q_score.shape != q.shape or q_score.dtype != q.dtype:
            raise ValueError("q_score must match q's shape and dtype")
        kbar, hb = summarize(k, landmark, scale=scale, stream=stream)
        idx, sc = select(q_score, kbar, hb, top_k, g, scale=scale, stream=stream, window=window)
        out = attend_selected(q, k, v, idx, sc, scale=scale, stream=stream, window=window, lse=lse)
    else:
        call = Prefill(b, h, g, n, d, top_k, q.dtype, scale=scale, device=q.device, window=window)
        idx = torch.empty((b, g, n, top_k), dtype=torch.int32, device=q.device) if return_idx else None
        out = call(q, k, v, landmark, topk_idx=idx, stream=stream, lse=lse)
    res = (out,) + ((idx,) if return_idx else ()) + ((lse,) if return_lse else ())
    return res if len(res) > 1 else out


def attend_selected(q, k, v, topk_idx, topk_score, scale=None, out=None, ws=None, stream=None, window=0,
                    lse=None):
    """Attention + fusion for a given selection (topk_idx [b,g,N,K], topk_score [b,h,N,K]);
    lse, if given (fp32 [b,h,N]), receives log Zhat."""
    b, h, n, d = q.shape
    g = k.shape[1]
    K = topk_idx.shape[-1]
    sh = make_shape(b, h, g, d, n, K, _dt(q), scale=scale or 0.0, window=window)
    if topk_idx.dtype != torch.int32 or topk_score.dtype != torch.float32:
        raise TypeError("topk_idx must be int32 and topk_score fp32")
    if topk_idx.shape != (b, g, n, K) or topk_score.shape != (b, h, n, K):
        raise ValueError("topk_idx must be [b, heads_kv, N, K] and topk_score [b, heads_q, N, K]")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (b, h, n)):
        raise ValueError("lse must be fp32 [b, h, N]")
    check_prefill_args(sh, q, k, v, None, out)
    _same_device(q, topk_idx, topk_score, lse, ws)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = new_workspace(sh, OP_ATTEND_SELECTED, q.device)
    _check(lib().hils_attend_selected(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(topk_idx),
                                      _ptr(topk_score), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                      _stream(stream)),
           "hils_attend_selected")
    return out


class Decode:
    """Reusable decode call for a paged cache of `max_chunks` chunks per sequence."""

    def __init__(self, batch, heads_q, heads_kv, head_dim, max_chunks, top_k, dtype, scale=None,
                 device="cuda", window=0):
        self.max_chunks = max_chunks
        self.shape = make_shape(batch, heads_q, heads_kv, head_dim, max_chunks * 64, top_k,
                                HILS_BF16 if dtype in (torch.bfloat16, "bf16") else HILS_F32,
                                scale=scale or 0.0, window=window)
        self.ws = new_workspace(self.shape, OP_DECODE, device)

    def __call__(self, q, k_pages, v_pages, kbar_pages, hbias_pages, block_table, seq_lens, out=None,
                 topk_idx=None, stream=None):
        s = self.shape
        if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
            raise TypeError("block_table and seq_lens must be int32")
        if block_table.shape != (s.batch, self.max_chunks):
            raise ValueError("block_table must be [batch, max_chunks]")
        check_decode_args(s, q, k_pages, v_pages, kbar_pages, hbias_pages, seq_lens, out, topk_idx)
        _same_device(q, block_table, self.ws)
        if out is None:
            out = torch.empty_like(q)
        _check(lib().hils_decode_ex(ctypes.byref(s), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kbar_pages),
                                    _dt(kbar_pages), _ptr(hbias_pages), _ptr(block_table), self.max_chunks,
                                    _ptr(seq_lens), int(k_pages.shape[0]), _ptr(out), _ptr(topk_idx), _ptr(self.ws),
                                    self.ws.numel(), _stream(stream)), "hils_decode_ex")
        return out

    def device_status(self, stream=None):
        return lib().hils_device_status(_ptr(self.ws), _stream(stream))


def decode(q, k_pages, v_pages, kbar_pages, hbias_pages, block_table, seq_lens, top_k, scale=None,
           stream=None, return_idx=False, window=0):
    b, h, d = q.shape
    g = k_pages.shape[1]
    call = Decode(b, h, g, d, block_table.shape[1], top_k, q.dtype, scale=scale, device=q.device, window=window)
    idx = torch.empty((b, g, top_k), dtype=torch.int32, device=q.device) if return_idx else None
    out = call(q, k_pages, v_pages, kbar_pages, hbias_pages, block_table, seq_lens, topk_idx=idx,
               stream=stream)
    return (out, idx) if return_idx else out


DECODE_STATIC_SCRATCH_BYTES = 4 << 20


def decode_static(q, k_pages, v_pages, kbar_pages, hbias_pages, block_table, seq_lens, top_k,
                  scale=None, out=None, topk_idx=None, status_word=None, stream=None):
    """hils_decode_static: decode without a workspace (the library's own
    scratch array is used).  Calls on one device must not overlap in time."""
    b, h, d = q.shape
    g = k_pages.shape[1]
    max_chunks = block_table.shape[1]
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if status_word is not None and (status_word.dtype != torch.int32 or status_word.numel() < 1):
        raise TypeError("status_word must be an int32 device tensor")
    # the entry point reads fp32 summaries only (it has no summary-dtype argument)
    if kbar_pages.dtype != torch.float32 or hbias_pages.dtype != torch.float32:
        raise TypeError("decode_static needs fp32 kbar_pages and hbias_pages (use decode() for a bf16 cache)")
    if kbar_pages.shape != (k_pages.shape[0], h, d) or hbias_pages.shape != (k_pages.shape[0], h):
        raise ValueError("kbar_pages must be [n_pages, heads_q, d] and hbias_pages [n_pages, heads_q]")
    if topk_idx is not None and (topk_idx.dtype != torch.int32 or topk_idx.numel() < b * g * top_k):
        raise TypeError("topk_idx must be an int32 tensor of at least batch * heads_kv * top_k entries")
    for t in (q, k_pages, v_pages, kbar_pages, hbias_pages, block_table, seq_lens, topk_idx, status_word, out):
        if t is not None and t.device != q.device:
            raise ValueError("every tensor must be on q's device")
    sh = make_shape(b, h, g, d, max_chunks * 64, top_k, _dt(q), scale=scale or 0.0)
    if out is None:
        out = torch.empty_like(q)
    _check(lib().hils_decode_static(ctypes.byref(sh), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kbar_pages),
                                    _ptr(hbias_pages), _ptr(block_table), max_chunks, _ptr(seq_lens),
                                    int(k_pages.shape[0]), _ptr(out), _ptr(topk_idx), _ptr(status_word),
                                    _stream(stream)), "hils_decode_static")
    return out


def backward(q, k, v, landmark, out, lse, topk_idx, topk_score, dout, scale=None, window=0, stream=None,
             ws=None):
    """hils_backward: fp32 (dq, dk, dv, dlandmark) for the forward that produced out,
    lse (log Zhat), topk_idx and topk_score on these bf16 inputs."""
    b, h, n, d = q.shape
    g = k.shape[1]
    K = topk_idx.shape[-1]
    if q.dtype != torch.bfloat16:
        raise TypeError("hils_backward takes bf16 inputs")
    for t in (k, v, landmark, out, dout):
        if t.dtype != torch.bfloat16:
            raise TypeError("q, k, v, landmark, out and dout must be bf16")
    if out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("out and dout must have q's shape")
    if lse.dtype != torch.float32 or lse.shape != (b, h, n):
        raise ValueError("lse must be fp32 [b, h, N]")
    if topk_idx.dtype != torch.int32 or topk_idx.shape != (b, g, n, K):
        raise ValueError("topk_idx must be int32 [b, heads_kv, N, K]")
    if topk_score.dtype != torch.float32 or topk_score.shape != (b, h, n, K):
        raise ValueError("topk_score must be fp32 [b, heads_q, N, K]")
    sh = make_shape(b, h, g, d, n, K, HILS_BF16, scale=scale or 0.0, window=window)
    check_prefill_args(sh, q, k, v, landmark, out)
    _same_device(q, lse, topk_idx, topk_score, dout, ws)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((b, h, n, d), **f32)
    dk = torch.empty((b, g, n, d), **f32)
    dv = torch.empty((b, g, n, d), **f32)
    dl = torch.zeros(landmark.shape, **f32)
    if ws is None:
        ws = new_workspace(sh, OP_BACKWARD, q.device)
    _check(lib().hils_backward(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(landmark), _ptr(out), _ptr(lse),
                               _ptr(topk_idx), _ptr(topk_score), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(dl), _ptr(ws), ws.numel(), _stream(stream)), "hils_backward")
    return dq, dk, dv, dl


# ---- the paged cache around the method: rotation, appended tokens, dense layers ----

_FLOATS = (torch.bfloat16, torch.float32)
# The device and stream that a launch finds, without the Python objects around them: these
# calls come once per decoded token.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _on:
    """Makes the device of tensor t current (kernels launch on the current device) and, if
    `stream` is given, that stream (so that what the call allocates belongs to it); gives
    the raw stream to launch on.  The tensor must be on a GPU."""

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if stream is not None and stream.device != t.device:
            raise ValueError("stream must be of the tensors' device")
        self.stream = stream
        self.dev = t.device.index
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
            return self.stream.cuda_stream
        self.prev = torch.cuda.current_device()
        if self.prev != self.dev:
            torch.cuda.set_device(self.dev)
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        elif self.prev != self.dev:
            torch.cuda.set_device(self.prev)
        return False


def _own_workspace(shape, op, device, ws):
    """ws checked, or a new workspace whose zeroes are in place before any stream uses it."""
    if ws is not None:
        if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < max(256, workspace_size(shape, op)):
            raise ValueError("ws must be a contiguous uint8 tensor of workspace_size bytes")
        return ws
    ws = new_workspace(shape, op, device)
    if ws.is_cuda and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(ws.device).synchronize()
    return ws


def _dtype_of(shape):
    return torch.bfloat16 if shape.dtype == HILS_BF16 else torch.float32


def _dense_shape(batch, heads_q, heads_kv, head_dim, max_chunks, dtype, scale=None, window=0):
    if max_chunks * 64 >= 1 << 31:
        raise ValueError("max_chunks * 64 must stay below 2**31")
    return make_shape(batch, heads_q, heads_kv, head_dim, max_chunks * 64, 0,
                      HILS_BF16 if dtype in (torch.bfloat16, "bf16") else HILS_F32, scale=scale or 0.0, window=window)


def _launch(fn, args, t, dev, stream, where):
    """fn(*args, stream) on device dev, tensor t's, and, unless `stream` is given, its current
    stream."""
    if stream is None and dev >= 0 and _current_device() == dev:
        st = fn(*args, _raw_stream(dev))
    else:
        with _on(t, stream) as raw:
            st = fn(*args, raw)
    if st != 0:
        raise HilsError(st, where)


def _empty(shape, dtype, t, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=t.device)
    with _on(t, stream):
        return torch.empty(shape, dtype=dtype, device=t.device)


# hils_rows and hils_rope structs as bytes, which ctypes passes by address: several times
# cheaper to make than ctypes structures.
_pack_rows = struct.Struct("4q").pack
_pack_rope = struct.Struct("qii").pack


def _rope_bytes(inv_freq, interleaved, d):
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float32 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous fp32 vector")
    r = 2 * inv_freq.numel()
    if r == 0 or r > d or r % 16:
        raise ValueError(f"inv_freq must have a multiple of 8 entries, at most head_dim / 2; got {r // 2}")
    return _pack_rope(inv_freq.data_ptr(), r, 1 if interleaved else 0)


def _rows4(t):
    """[b, heads, n, d] as hils_rows."""
    a, b, c, e = t.stride()
    if e != 1:
        raise ValueError("the last dimension of q, k, v and their outputs must be contiguous")
    return _pack_rows(t.data_ptr(), a, b, c)


def _not_contiguous():
    raise ValueError("tensors other than the rows of q, k, v and their outputs must be contiguous")


def check_rotate_args(q, inv_freq, k=None, positions=None, q_out=None, k_out=None):
    """The tensors of rotate against one another; returns the stride of positions over the
    batch (0: shared).  Strides, alignment and overlaps are checked where the rows are packed and
    by hils_rotate."""
    if q.dim() != 4:
        raise ValueError("q must be [b, heads_q, n, d]")
    b, _, n, d = q.shape
    if q.dtype not in _FLOATS:
        raise TypeError(f"q must be bf16 or fp32, got {q.dtype}")
    if inv_freq is None:
        raise ValueError("inv_freq is required")
    if q_out is not None:
        _expect(q_out, q.shape, _FLOATS, "q_out")
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [b, heads_kv, n, d]")
        _expect(k, (b, k.shape[1], n, d), (q.dtype,), "k")
        if k_out is not None:
            _expect(k_out, k.shape, (q.dtype if q_out is None else q_out.dtype,), "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _same_device(q, inv_freq, k, positions, q_out, k_out)
    if positions is None:
        return 0
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        raise TypeError("positions must be contiguous int32")
    if positions.shape == (n,):
        return 0
    if positions.shape != (b, n):
        raise ValueError("positions must be [n] or [b, n]")
    return n


def rotate(q, inv_freq, k=None, positions=None, inverse=False, interleaved=False, q_out=None, k_out=None,
           stream=None):
    """Position rotation of q [b,h,n,d] (and k [b,g,n,d]); returns q_out, or (q_out, k_out).

    inv_freq [rotary_dim / 2] fp32: frequency f turns pair f by position * inv_freq[f]; pair f
    is (f, f + rotary_dim / 2), or (2f, 2f + 1) when interleaved; elements from rotary_dim on
    are copied.  positions: None (token i at position i), int32 [n], or int32 [b, n].
    inverse: the opposite rotation, which takes the gradients of the rotated q and k (backward's
    dq and dk) to those of the unrotated ones.  The tensors may have any strides whose rows are
    contiguous and 16-byte aligned; an output may be its input (in place), and may be bf16 or
    fp32 whatever the input is."""
    qs, dt, dev = q.shape, q.dtype, q.get_device()
    ks = None if k is None else k.shape
    # the call as it mostly comes, in one expression; any other goes through the full check,
    # which says what is wrong
    if (ks is not None and len(qs) == 4 and len(ks) == 4 and dt in _FLOATS and k.dtype is dt and
            ks[0] == qs[0] and ks[2] == qs[2] and ks[3] == qs[3] and k.get_device() == dev and
            inv_freq is not None and inv_freq.get_device() == dev and
            (positions is None or positions.shape == (qs[0], qs[2]) and positions.dtype is torch.int32 and
             positions.get_device() == dev and positions.is_contiguous()) and
            (q_out is None or q_out.shape == qs and q_out.dtype is dt and q_out.get_device() == dev) and
            (k_out is None or q_out is not None and k_out.shape == ks and k_out.dtype is dt and
             k_out.get_device() == dev)):
        pstride = 0 if positions is None else qs[2]
    else:
        pstride = check_rotate_args(q, inv_freq, k, positions, q_out, k_out)
    b, h, n, d = qs
    rope = _rope_bytes(inv_freq, interleaved, d)
    if q_out is None:
        q_out = _empty(qs, dt, q, stream)
    if ks is not None and k_out is None:
        k_out = _empty(ks, q_out.dtype, q, stream)
    g = h if ks is None else ks[1]
    if b * n * h * g:
        bf16, out_bf16 = 1 if dt is torch.bfloat16 else 0, 1 if q_out.dtype is torch.bfloat16 else 0
        _launch(lib().hils_rotate,
                (_shape_of(b, h, g, d, n, 0, bf16), _rows4(q), None if ks is None else _rows4(k), rope,
                 None if positions is None else positions.data_ptr(), pstride, 1 if inverse else 0, _rows4(q_out),
                 None if ks is None else _rows4(k_out), out_bf16), q, dev, stream, "hils_rotate")
    elif b * n and h + g:
        raise ValueError("q and k must have heads, both or neither")
    return q_out if ks is None else (q_out, k_out)


def _rows_single(t):
    """[b, heads, d], one token each, as hils_rows."""
    a, b, e = t.stride()
    if e != 1:
        raise ValueError("the last dimension of q, k, v and their outputs must be contiguous")
    return _pack_rows(t.data_ptr(), a, b, 0)


def _rows_packed(t):
    """[tokens, heads, d] as hils_rows."""
    a, b, e = t.stride()
    if e != 1:
        raise ValueError("the last dimension of q, k, v and their outputs must be contiguous")
    return _pack_rows(t.data_ptr(), 0, b, a)


def append_slots(batch, tokens):
    """Entries of Append's full_pages for a call of `tokens` rows in all (batch * n for
    [b, heads, n, d])."""
    return batch + tokens // 64


def check_append_args(shape, k, v, k_pages, v_pages, block_table, max_chunks, seq_lens, q=None, q_out=None,
                      cu_new=None, new_lens=None, full_pages=None):
    """The tensors of an append against the shape (see Append.__call__).  Strides, alignment and
    overlaps are checked where the rows are packed and by hils_append_paged."""
    b, h, g, d = shape.batch, shape.heads_q, shape.heads_kv, shape.head_dim
    dts = (_dtype_of(shape),)
    if k.dim() == 3:
        n = tokens = k.shape[0]
        rows, qrows = (n, g, d), (n, h, d)
        if cu_new is not None:
            _expect(cu_new, (b + 1,), (torch.int32,), "cu_new")
        elif n != b:
            raise ValueError("packed tokens need cu_new unless there is one per sequence")
        if new_lens is not None:
            raise ValueError("new_lens goes with [b, heads, n, d] tokens")
    elif k.dim() == 4:
        n = k.shape[2]
        tokens = b * n
        rows, qrows = (b, g, n, d), (b, h, n, d)
        if cu_new is not None:
            raise ValueError("cu_new goes with packed [tokens, heads, d] rows")
        if new_lens is not None:
            _expect(new_lens, (b,), (torch.int32,), "new_lens")
    else:
        raise ValueError("k must be [b, heads_kv, n, d] or [tokens, heads_kv, d]")
    _expect(k, rows, dts, "k")
    _expect(v, rows, dts, "v")
    P = k_pages.shape[0] if k_pages.dim() == 4 else -1
    _expect(k_pages, (P, g, 64, d), dts, "k_pages")
    _expect(v_pages, (P, g, 64, d), dts, "v_pages")
    _expect(block_table, (b, max_chunks), (torch.int32,), "block_table")
    _expect(seq_lens, (b,), (torch.int32,), "seq_lens")
    if q is not None:
        _expect(q, qrows, dts, "q")
        if q_out is not None:
            _expect(q_out, qrows, dts, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if full_pages is not None:
        _expect(full_pages, (append_slots(b, tokens),), (torch.int32,), "full_pages")
    _same_device(k, v, q, q_out, k_pages, v_pages, block_table, seq_lens, cu_new, new_lens, full_pages)


class Append:
    """Reusable call that writes new tokens into a paged cache of `max_chunks` chunks per
    sequence; holds the rotation (inv_freq, see rotate; None: no rotation) and the error
    word (`ws`: the caller's own zero-filled workspace)."""

    def __init__(self, batch, heads_q, heads_kv, head_dim, max_chunks, dtype, inv_freq=None, interleaved=False,
                 device="cuda", ws=None):
        self.max_chunks = max_chunks
        self.shape = _dense_shape(batch, heads_q, heads_kv, head_dim, max_chunks, dtype)
        self.inv_freq = inv_freq
        self.rope = None if inv_freq is None else _rope_bytes(inv_freq, interleaved, head_dim)
        self.ws = _own_workspace(self.shape, OP_APPEND, device, ws)
        _same_device(self.ws, inv_freq)
        self._dims = (batch, heads_q, heads_kv, head_dim, _dtype_of(self.shape), self.ws.get_device())

    def __call__(self, k, v, k_pages, v_pages, block_table, seq_lens, q=None, q_out=None, cu_new=None, new_lens=None,
                 full_pages=None, stream=None):
        """Writes k, v into k_pages, v_pages [P,g,64,d] (the keys rotated by their position);
        returns q_out, the rotated queries, or None.

        k, v [b,g,n,d] with q [b,h,n,d]: n tokens per sequence, of which new_lens [b] int32 may
        take only the first ones (right padding).  k, v [tokens,g,d] with q [tokens,h,d]: packed;
        cu_new [b+1] int32 gives each sequence's rows, or None: one token per sequence.
        seq_lens [b] int32 are the lengths after the call.  full_pages: int32
        [append_slots(b, tokens)], receives the pages filled by the call, else -1: it can go to
        summarize_paged as it is.  q_out may be q itself."""
        b, h, g, d, dt, dev = self._dims
        i32, ks, ps = torch.int32, k.shape, k_pages.shape
        if len(ks) == 3:
            n = tokens = ks[0]
            rows, qrows, ragged, entries = (n, g, d), (n, h, d), cu_new, b + 1
            right = new_lens is None and (cu_new is not None or n == b)
        else:
            n = ks[2] if len(ks) == 4 else 0
            tokens, rows, qrows, ragged, entries = b * n, (b, g, n, d), (b, h, n, d), new_lens, b
            right = cu_new is None
        # what makes the call right, in one expression; where it does not hold, the full check
        # says what is wrong
        if not (right and ks == rows and v.shape == ks and k.dtype is dt and v.dtype is dt and
                k.get_device() == dev and v.get_device() == dev and
                (ragged is None or
                 ragged.shape == (entries,) and ragged.dtype is i32 and ragged.get_device() == dev) and
                len(ps) == 4 and ps[1] == g and ps[2] == 64 and ps[3] == d and v_pages.shape == ps and
                k_pages.dtype is dt and v_pages.dtype is dt and
                k_pages.get_device() == dev and v_pages.get_device() == dev and
                block_table.shape == (b, self.max_chunks) and block_table.dtype is i32 and
                block_table.get_device() == dev and
                seq_lens.shape == (b,) and seq_lens.dtype is i32 and seq_lens.get_device() == dev and
                (q_out is None if q is None else
                 q.shape == qrows and q.dtype is dt and q.get_device() == dev and
                 (q_out is None or q_out.shape == qrows and q_out.dtype is dt and q_out.get_device() == dev)) and
                (full_pages is None or full_pages.shape == (b + tokens // 64,) and full_pages.dtype is i32 and
                 full_pages.get_device() == dev)):
            check_append_args(self.shape, k, v, k_pages, v_pages, block_table, self.max_chunks, seq_lens, q, q_out,
                              cu_new, new_lens, full_pages)
            _same_device(k, self.ws)
        if not (k_pages.is_contiguous() and v_pages.is_contiguous() and block_table.is_contiguous() and
                seq_lens.is_contiguous() and (ragged is None or ragged.is_contiguous()) and
                (full_pages is None or full_pages.is_contiguous())):
            _not_contiguous()
        if q is not None and q_out is None:
            q_out = _empty(q.shape, dt, k, stream)
        pack = _rows4 if len(ks) == 4 else _rows_packed if cu_new is not None else _rows_single
        _launch(lib().hils_append_paged,
                (self.shape, pack(k), pack(v), None if q is None else pack(q), None if q is None else pack(q_out),
                 1 if pack is _rows_single else n, None if cu_new is None else cu_new.data_ptr(),
                 None if new_lens is None else new_lens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                 self.max_chunks, ps[0], self.rope, k_pages.data_ptr(), v_pages.data_ptr(),
                 None if full_pages is None else full_pages.data_ptr(), self.ws.data_ptr(), self.ws.numel()),
                k, dev, stream, "hils_append_paged")
        return q_out

    def device_status(self, stream=None):
        with _on(self.ws, stream) as st:
            return lib().hils_device_status(_ptr(self.ws), st)


def append_paged(k, v, k_pages, v_pages, block_table, seq_lens, inv_freq=None, interleaved=False, q=None, q_out=None,
                 cu_new=None, new_lens=None, full_pages=None, stream=None):
    """Append for one call (see Append.__call__); device-side errors are not reported."""
    b, max_chunks = block_table.shape
    g, d = k_pages.shape[1], k_pages.shape[3]
    with _on(k, stream):
        sh = _dense_shape(b, g if q is None else q.shape[1], g, d, max_chunks, k_pages.dtype)
        call = Append(b, sh.heads_q, g, d, max_chunks, k_pages.dtype, inv_freq=inv_freq, interleaved=interleaved,
                      ws=new_workspace(sh, OP_APPEND, k.device))
        return call(k, v, k_pages, v_pages, block_table, seq_lens, q=q, q_out=q_out, cu_new=cu_new,
                    new_lens=new_lens, full_pages=full_pages)


def check_dense_args(shape, q, k_pages, v_pages, block_table, max_chunks, seq_lens, out=None, lse=None):
    """The tensors of a dense decode against the shape: q [b,h,d]; k/v pages [P,g,64,d] in q's
    dtype; block_table [b, max_chunks] and seq_lens [b] int32; out like q; lse [b,h] fp32."""
    b, h, d = shape.batch, shape.heads_q, shape.head_dim
    dts = (_dtype_of(shape),)
    _expect(q, (b, h, d), dts, "q")
    pages = (k_pages.shape[0] if k_pages.dim() == 4 else -1, shape.heads_kv, 64, d)
    _expect(k_pages, pages, dts, "k_pages")
    _expect(v_pages, pages, dts, "v_pages")
    _expect(block_table, (b, max_chunks), (torch.int32,), "block_table")
    _expect(seq_lens, (b,), (torch.int32,), "seq_lens")
    if out is not None:
        _expect(out, (b, h, d), dts, "out")
    if lse is not None:
        _expect(lse, (b, h), (torch.float32,), "lse")
    _same_device(q, k_pages, v_pages, block_table, seq_lens, out, lse)


class DenseDecode:
    """Reusable decode call of a dense layer (every key, or a sliding window of chunks) for a
    paged cache of `max_chunks` chunks per sequence; holds the workspace, which serves one
    call at a time (`ws`: the caller's own, zero-filled before it serves another shape)."""

    def __init__(self, batch, heads_q, heads_kv, head_dim, max_chunks, dtype, scale=None, device="cuda", window=0,
                 ws=None):
        self.max_chunks = max_chunks
        self.shape = _dense_shape(batch, heads_q, heads_kv, head_dim, max_chunks, dtype, scale, window)
        self.ws = _own_workspace(self.shape, OP_DECODE_DENSE, device, ws)
        self._dims = (batch, heads_q, heads_kv, head_dim, _dtype_of(self.shape), self.ws.get_device())

    def __call__(self, q, k_pages, v_pages, block_table, seq_lens, out=None, lse=None, stream=None):
        """out [b,h,d] (q's dtype); lse, if given (fp32 [b,h]), receives log sum exp(logit)."""
        b, h, g, d, dt, dev = self._dims
        i32, qs, ps = torch.int32, q.shape, k_pages.shape
        # what makes the call right, in one expression; where it does not hold, the full check
        # says what is wrong
        if not (qs == (b, h, d) and q.dtype is dt and q.get_device() == dev and
                len(ps) == 4 and ps[1] == g and ps[2] == 64 and ps[3] == d and v_pages.shape == ps and
                k_pages.dtype is dt and v_pages.dtype is dt and
                k_pages.get_device() == dev and v_pages.get_device() == dev and
                block_table.shape == (b, self.max_chunks) and block_table.dtype is i32 and
                block_table.get_device() == dev and
                seq_lens.shape == (b,) and seq_lens.dtype is i32 and seq_lens.get_device() == dev and
                (out is None or out.shape == qs and out.dtype is dt and out.get_device() == dev) and
                (lse is None or lse.shape == (b, h) and lse.dtype is torch.float32 and lse.get_device() == dev)):
            check_dense_args(self.shape, q, k_pages, v_pages, block_table, self.max_chunks, seq_lens, out, lse)
            _same_device(q, self.ws)
        if out is None:
            out = _empty(qs, dt, q, stream)
        if not (q.is_contiguous() and k_pages.is_contiguous() and v_pages.is_contiguous() and
                block_table.is_contiguous() and seq_lens.is_contiguous() and out.is_contiguous() and
                (lse is None or lse.is_contiguous())):
            _not_contiguous()
        _launch(lib().hils_decode_dense,
                (self.shape, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                 self.max_chunks, seq_lens.data_ptr(), ps[0], out.data_ptr(), None if lse is None else lse.data_ptr(),
                 self.ws.data_ptr(), self.ws.numel()), q, dev, stream, "hils_decode_dense")
        return out

    def device_status(self, stream=None):
        with _on(self.ws, stream) as st:
            return lib().hils_device_status(_ptr(self.ws), st)


def decode_dense(q, k_pages, v_pages, block_table, seq_lens, scale=None, window=0, return_lse=False, stream=None):
    """Attention of one new token per sequence over every key of its pages (window 0), or the
    last window / 64 chunks; returns out [b,h,d], then lse [b,h] when asked."""
    b, h, d = q.shape
    with _on(q, stream):
        sh = _dense_shape(b, h, k_pages.shape[1], d, block_table.shape[1], q.dtype, scale, window)
        call = DenseDecode(b, h, k_pages.shape[1], d, block_table.shape[1], q.dtype, scale=scale, window=window,
                           ws=new_workspace(sh, OP_DECODE_DENSE, q.device))
        lse = torch.empty((b, h), dtype=torch.float32, device=q.device) if return_lse else None
        out = call(q, k_pages, v_pages, block_table, seq_lens, lse=lse)
    return (out, lse) if return_lse else out
