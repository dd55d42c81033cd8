"""Attention half of a decoder layer, for PyTorch tensors: a paged key/value cache
held in 4 bits, attention over it, and causal attention over packed prompts
(``include/moe_attention.h``; argument checks and marshalling only, every step runs
in the library's CUDA kernels).

All calls are stream-ordered on ``stream`` (default: PyTorch's current stream),
allocate only their outputs, and do not wait for the GPU.  Token tensors are
``[tokens, heads, head_dim]`` with a contiguous last dimension; other strides are
free as long as base and strides are whole multiples of 16 bytes (slices of a
fused projection's output are).  Index tensors are contiguous int32 on the GPU;
their contents are checked by the kernels: see ``status_message``.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MoeError, _check, lib

MOE_KV_BAD_PAGE = 1
MOE_KV_BAD_LENGTH = 2
MOE_KV_BAD_POSITION = 4
MOE_KV_TIMED_OUT = 8
MOE_KV_COUNTER_BYTES = 4096

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class MoeKvCache(ctypes.Structure):
    """moe_kv_cache"""
    _fields_ = [("pages", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("status", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_seqs", ctypes.c_int32), ("table_width", ctypes.c_int32)]


class MoeTensor(ctypes.Structure):
    """moe_tensor"""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        pc, pt = ctypes.POINTER(MoeKvCache), ctypes.POINTER(MoeTensor)
        L.moe_kv_page_bytes.restype = i64
        L.moe_kv_page_bytes.argtypes = [i32, i32, i32]
        L.moe_kv_append.argtypes = [pc, vp, vp, i32, pt, i32, pt, pt, vp, vp, i32, i32, i32, vp, vp, i32, vp]
        L.moe_kv_read.argtypes = [pc, vp, vp, i32, vp, vp, i32, vp]
        L.moe_kv_attention_workspace.restype = i64
        L.moe_kv_attention_workspace.argtypes = [i32, i32, i32, i32]
        L.moe_kv_attention.argtypes = [pc, vp, pt, i32, i32, f32, i32, vp, vp, i32, vp, i64, vp]
        L.moe_prompt_attention.argtypes = [pt, i32, i32, pt, pt, i32, i32, i32, vp, vp, i32, f32, i32, vp, vp, i32, vp, vp]
        _bound = L
    return _bound


def _refuse(what: str, code: int = MOE_ERR_INVALID_ARG):
    err = MoeError(code, what)
    raise err


def _index(t, name, n, device):
    if t.dtype != torch.int32 or t.device != device or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor of {n} entries on {device}")
    return t.data_ptr()


def _tokens(t, name, n, heads, dim, dtype, device):
    if t.dim() != 3 or t.dtype != dtype or t.device != device or t.stride(2) != 1 or t.shape[2] != dim \
            or (heads is not None and t.shape[1] != heads) or (n is not None and t.shape[0] != n):
        _refuse(f"{name} must be {dtype} [{n if n is not None else 'tokens'}, {heads or 'heads'}, {dim}] on {device} "
                "with a contiguous last dimension")
    return MoeTensor(t.data_ptr(), t.stride(0), t.stride(1))


def _output(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _device(t):
    d = t.device
    if d.type != "cuda" or d.index != torch.cuda.current_device():
        _refuse("tensors must be on the current CUDA device")
    return d


class _On:
    """The stream of a call as a handle; outputs are allocated for that stream."""

    def __init__(self, stream):
        self.ctx = None
        if stream is None:
            self.handle = torch.cuda.current_stream().cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        self.handle = stream.cuda_stream
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *a):
        if self.ctx is not None:
            self.ctx.__exit__(*a)


def kv_page_bytes(n_kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of one page; MoeError for sizes that are not supported."""
    n = int(_lib().moe_kv_page_bytes(n_kv_heads, head_dim, page_size))
    if n == 0:
        _refuse("n_kv_heads >= 1, head_dim 64, 128 or 256 and a page_size of whole 32-token tiles are supported",
                MOE_ERR_UNSUPPORTED)
    return n


def kv_pages(n_pages: int, n_kv_heads: int, head_dim: int, page_size: int, device="cuda"):
    """An empty cache: uint8 [n_pages, page_bytes]."""
    return torch.zeros(n_pages, kv_page_bytes(n_kv_heads, head_dim, page_size), dtype=torch.uint8, device=device)


def rope_table(n_positions: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """cos and sin [n_positions, rot_dim / 2] fp32 of the angles p theta^(-2i / rot_dim), formed in 64 bits
    (an angle of a far position loses its fraction in 32)."""
    f = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float(), a.sin().float()


def _cache(pages, page_table, page_size, n_kv_heads, head_dim, status, device):
    if pages.dtype != torch.uint8 or pages.dim() != 2 or pages.device != device or pages.stride(1) != 1:
        _refuse("pages must be uint8 [n_pages, page_bytes] on the GPU, rows contiguous")
    if pages.shape[1] < kv_page_bytes(n_kv_heads, head_dim, page_size):
        _refuse("a row of pages is shorter than a page")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.device != device \
            or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        _refuse("page_table must be int32 [n_seqs, width] on the GPU, rows contiguous")
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != device):
        _refuse("status must be one int32 on the GPU")
    width = page_table.shape[1]
    return MoeKvCache(pages.data_ptr(), pages.stride(0), page_table.data_ptr(), max(page_table.stride(0), width),
                      0 if status is None else status.data_ptr(), pages.shape[0], page_size, n_kv_heads, head_dim,
                      page_table.shape[0], width)


def kv_append(pages, page_table, starts, cu_tokens, k, v, *, page_size, q=None, cos=None, sin=None,
              interleaved=False, q_out=None, k_out=None, status=None, stream=None):
    """Append new tokens to the cache, rotating their keys and queries (moe_kv_append).

    Tokens [cu_tokens[s], cu_tokens[s+1]) go to positions starts[s], starts[s] + 1, ... of sequence s.
    cos, sin [n_positions, rot_dim / 2] (``rope_table``); None: no rotation.  Returns the rotated queries
    (None without q) and the rotated keys, both contiguous in the inputs' type; the cache holds the keys
    quantised from their fp32 values."""
    dev = _device(k)
    if k.dtype not in _DTYPES or k.dim() != 3:
        _refuse("k must be float32, bfloat16 or float16 [tokens, heads, head_dim]")
    T, hkv, d = k.shape
    c = _cache(pages, page_table, page_size, hkv, d, status, dev)
    tk, tv = _tokens(k, "k", T, hkv, d, k.dtype, dev), _tokens(v, "v", T, hkv, d, k.dtype, dev)
    ps, pc = _index(starts, "starts", c.n_seqs, dev), _index(cu_tokens, "cu_tokens", c.n_seqs + 1, dev)
    rot = n_pos = 0
    cp = sp = None
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape or cos.dtype != torch.float32 \
                or sin.dtype != torch.float32 or cos.device != dev or sin.device != dev \
                or not cos.is_contiguous() or not sin.is_contiguous():
            _refuse("cos and sin must be contiguous float32 [n_positions, rot_dim / 2] on the GPU")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        cp, sp = cos.data_ptr(), sin.data_ptr()
    with _On(stream) as h:
        tq, hq = None, 0
        if q is not None:
            tq = _tokens(q, "q", T, None, d, k.dtype, dev)
            hq = q.shape[1]
            q_out = _output(q_out, "q_out", (T, hq, d), k.dtype, dev)
        k_out = _output(k_out, "k_out", (T, hkv, d), k.dtype, dev)
        _check(_lib().moe_kv_append(ctypes.byref(c), ps, pc, T, None if tq is None else ctypes.byref(tq), hq,
                                    ctypes.byref(tk), ctypes.byref(tv), cp, sp, rot, n_pos, int(interleaved),
                                    None if q is None else q_out.data_ptr(), k_out.data_ptr(), _DTYPES[k.dtype], h),
               "moe_kv_append")
    return (None if q is None else q_out), k_out


def kv_read(pages, page_table, starts, cu_tokens, n_tokens, *, page_size, n_kv_heads, head_dim,
            dtype=torch.bfloat16, status=None, stream=None):
    """The values of cached tokens starts[s] + (i - cu_tokens[s]): keys and values [n_tokens, n_kv_heads,
    head_dim] (moe_kv_read)."""
    dev = _device(pages)
    if dtype not in _DTYPES:
        _refuse("dtype must be float32, bfloat16 or float16")
    c = _cache(pages, page_table, page_size, n_kv_heads, head_dim, status, dev)
    ps, pc = _index(starts, "starts", c.n_seqs, dev), _index(cu_tokens, "cu_tokens", c.n_seqs + 1, dev)
    with _On(stream) as h:
        k = torch.empty((n_tokens, n_kv_heads, head_dim), dtype=dtype, device=dev)
        v = torch.empty_like(k)
        _check(_lib().moe_kv_read(ctypes.byref(c), ps, pc, n_tokens, k.data_ptr(), v.data_ptr(), _DTYPES[dtype], h),
               "moe_kv_read")
    return k, v


_workspaces = {}


def kv_attention_workspace(n_q_heads, n_kv_heads, head_dim, q_tokens=1, device="cuda"):
    """A workspace for kv_attention, to be used by one stream (or one captured graph) at a time."""
    n = int(_lib().moe_kv_attention_workspace(n_q_heads, n_kv_heads, head_dim, q_tokens))
    if n <= 0:
        _refuse("kv_attention_workspace: unsupported sizes", MOE_ERR_UNSUPPORTED)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:MOE_KV_COUNTER_BYTES].zero_()
    return ws


def _workspace(hq, hkv, d, q_tokens, handle, dev):
    # one per stream, as calls on one stream follow each other; a capture gets its own, which its graph keeps
    if torch.cuda.is_current_stream_capturing():
        return kv_attention_workspace(hq, hkv, d, q_tokens, dev)
    key = (dev.index, handle, d)
    ws = _workspaces.get(key)
    if ws is None:
        ws = _workspaces[key] = kv_attention_workspace(hq, hkv, d, q_tokens, dev)
    return ws


def kv_attention(q, pages, page_table, seq_lens, *, page_size, n_kv_heads, q_tokens=1, scale=None, window=0,
                 return_lse=False, out=None, workspace=None, status=None, stream=None):
    """Attention of every sequence's last q_tokens tokens over the cache (moe_kv_attention).

    q [n_seqs * q_tokens, n_q_heads, head_dim] bfloat16 or float16; seq_lens int32 [n_seqs] counts the cached
    tokens, the queried ones among them.  window > 0: a token sees itself and the window - 1 tokens before it.
    Returns [n_seqs * q_tokens, n_q_heads, head_dim], and the log of the sums of exponentials (fp32) with
    return_lse.  Without `workspace` a module-level one per stream is used (inside a graph capture: one of the
    capture's own); graphs that may run at the same time need their own."""
    dev = _device(q)
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    n, hq, d = q.shape
    c = _cache(pages, page_table, page_size, n_kv_heads, d, status, dev)
    if n != c.n_seqs * q_tokens or hq % n_kv_heads:
        _refuse("q must hold q_tokens tokens of every sequence, its heads a multiple of n_kv_heads")
    tq = _tokens(q, "q", n, hq, d, q.dtype, dev)
    pl = _index(seq_lens, "seq_lens", c.n_seqs, dev)
    with _On(stream) as h:
        out = _output(out, "out", (n, hq, d), q.dtype, dev)
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if return_lse else None
        if n:
            ws = _workspace(hq, n_kv_heads, d, q_tokens, h, dev) if workspace is None else workspace
            _check(_lib().moe_kv_attention(ctypes.byref(c), pl, ctypes.byref(tq), hq, q_tokens,
                                           1.0 / math.sqrt(d) if scale is None else scale, window, out.data_ptr(),
                                           lse.data_ptr() if return_lse else None, _DTYPES[q.dtype], ws.data_ptr(),
                                           ws.numel(), h), "moe_kv_attention")
    return (out, lse) if return_lse else out


def prompt_attention(q, k, v, cu_q, cu_k=None, *, scale=None, window=0, return_lse=False, out=None, status=None,
                     stream=None):
    """Causal attention over packed prompts (moe_prompt_attention).

    q [n_q_tokens, n_q_heads, head_dim], k and v [n_k_tokens, n_kv_heads, head_dim], bfloat16 or float16;
    cu_q, cu_k int32 [n_seqs + 1] (cu_k None: cu_q).  With more keys than queries a sequence's queries are its
    last tokens.  window > 0: a token sees itself and the window - 1 tokens before it.  Returns q's shape, and
    the log of the sums of exponentials (fp32 [n_q_tokens, n_q_heads]) with return_lse."""
    dev = _device(q)
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    n, hq, d = q.shape
    tq, tk = _tokens(q, "q", n, hq, d, q.dtype, dev), _tokens(k, "k", None, None, d, q.dtype, dev)
    tv = _tokens(v, "v", k.shape[0], k.shape[1], d, q.dtype, dev)
    cu_k = cu_q if cu_k is None else cu_k
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        _refuse("cu_q must hold n_seqs + 1 offsets")
    n_cu = cu_q.shape[0]
    pq, pk = _index(cu_q, "cu_q", n_cu, dev), _index(cu_k, "cu_k", n_cu, dev)
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != dev):
        _refuse("status must be one int32 on the GPU")
    with _On(stream) as h:
        out = _output(out, "out", (n, hq, d), q.dtype, dev)
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if return_lse else None
        _check(_lib().moe_prompt_attention(ctypes.byref(tq), n, hq, ctypes.byref(tk), ctypes.byref(tv), k.shape[0],
                                           k.shape[1], d, pq, pk, n_cu - 1, 1.0 / math.sqrt(d) if scale is None else scale,
                                           window, out.data_ptr(), lse.data_ptr() if return_lse else None,
                                           _DTYPES[q.dtype], None if status is None else status.data_ptr(), h),
               "moe_prompt_attention")
    return (out, lse) if return_lse else out


def status_message(status) -> str:
    """What the bits of a status word say (reads it: waits for the GPU); empty when nothing is wrong."""
    bits = int(status.item())
    names = ((MOE_KV_BAD_PAGE, "a page number outside the cache"),
             (MOE_KV_BAD_LENGTH, "a length or offset outside the page table or the tensor"),
             (MOE_KV_BAD_POSITION, "a position past the rotation table"),
             (MOE_KV_TIMED_OUT, "a device wait gave up"))
    return "; ".join(text for bit, text in names if bits & bit)
