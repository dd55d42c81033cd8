"""Attention half of a decoder layer, for PyTorch tensors: a paged key/value cache
held in 4 bits, attention over it, and causal attention over packed prompts
(``include/moe_attention.h``; argument checks and marshalling only, every step runs
in the library's CUDA kernels).

All calls are stream-ordered on ``stream`` (default: PyTorch's current stream),
allocate only their outputs, and do not wait for the GPU.  The caller orders that
stream after the work that makes the inputs.  Of a ``torch.cuda.Stream`` the tensors
given may be dropped once the call returns: they are recorded on it.  Of a raw handle
or a ``torch.cuda.ExternalStream``, which may be gone before they are, the caller keeps
them until the work is done.  Token tensors are
``[tokens, heads, head_dim]`` with a contiguous last dimension; other strides are
free as long as base and strides are whole multiples of 16 bytes (slices of a
fused projection's output are).  Index tensors are contiguous int32 on the GPU;
their contents are checked by the kernels: see ``status_message``.
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch

from . import MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MoeError, _check, lib

MOE_KV_BAD_PAGE = 1
MOE_KV_BAD_LENGTH = 2
MOE_KV_BAD_POSITION = 4
MOE_KV_TIMED_OUT = 8
MOE_ROUTE_BAD_LOGIT = 16
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


# the same, packed: a call builds them for itself, and a Structure instance takes several times as long
_CACHE = struct.Struct("@qqqqqiiiiii")
_TENSOR = struct.Struct("@qqq")

_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        L.moe_kv_page_bytes.restype = i64
        L.moe_kv_page_bytes.argtypes = [i32, i32, i32]
        L.moe_kv_append.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp]
        L.moe_kv_append_at.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp]
        L.moe_kv_read.argtypes = [vp, vp, vp, i32, vp, vp, i32, vp]
        L.moe_kv_attention_workspace.restype = i64
        L.moe_kv_attention_workspace.argtypes = [i32, i32, i32, i32]
        L.moe_kv_attention.argtypes = [vp, vp, vp, i32, i32, f32, i32, vp, vp, i32, vp, i64, vp]
        L.moe_prompt_attention.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, i32, f32, i32, vp, vp, i32, vp, vp]
        L.moe_prompt_attention_workspace.restype = i64
        L.moe_prompt_attention_workspace.argtypes = [i32] * 7
        L.moe_prompt_attention_shared.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, i32, f32, i32, vp, vp, i32, vp,
                                                  vp, i64, vp]
        _bound = L
    return _bound


def _refuse(what: str, code: int = MOE_ERR_INVALID_ARG):
    raise MoeError(code, what)


_WIDEST = 2147483647


def _window(window):
    # (ctypes keeps the low 32 bits of a number; no sequence is longer than the widest window)
    return _WIDEST if window > _WIDEST else window if window >= 0 else -1


def _index(t, name, n, dev):
    if t.dtype is not torch.int32 or t.get_device() != dev or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor of {n} entries on the GPU")
    return t.data_ptr()


def _tokens(t, name, n, heads, dim, dtype, dev):
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype is not dtype or t.get_device() != dev or stride[2] != 1 or shape[2] != dim \
            or (heads is not None and shape[1] != heads) or (n is not None and shape[0] != n):
        _refuse(f"{name} must be {dtype} [{n if n is not None else 'tokens'}, {heads or 'heads'}, {dim}] on the GPU "
                "with a contiguous last dimension")
    # a dimension of one has no stride to speak of
    return _TENSOR.pack(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0)


def _output(t, name, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=_cuda(dev))
    if tuple(t.shape) != tuple(shape) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the GPU")
    return t


def _word(t, dev):
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.numel() != 1 or t.get_device() != dev:
        _refuse("status must be one int32 on the GPU")
    return t.data_ptr()


def _device(t):
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse("tensors must be on the current CUDA device")
    return dev


_cuda_devices = {}


def _cuda(dev):
    d = _cuda_devices.get(dev)
    if d is None:
        d = _cuda_devices[dev] = torch.device("cuda", dev)
    return d


def _call(stream, dev, run, *tensors):
    """run(handle of the stream), its outputs allocated for that stream; tensors: what it reads and writes."""
    if stream is None:
        return run(torch._C._cuda_getCurrentRawStream(dev))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    elif not isinstance(stream, torch.cuda.ExternalStream):
        for t in tensors:
            if t is not None and t.is_cuda:  # (an output that is not is refused below)
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return run(stream.cuda_stream)


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


def _cache(pages, page_table, page_size, n_kv_heads, head_dim, status, dev):
    shape, table, stride = pages.shape, page_table.shape, page_table.stride()
    if pages.dtype is not torch.uint8 or len(shape) != 2 or pages.get_device() != dev or pages.stride(1) != 1:
        _refuse("pages must be uint8 [n_pages, page_bytes] on the GPU, rows contiguous")
    if shape[1] < n_kv_heads * page_size * head_dim * 9 // 8:
        _refuse("a row of pages is shorter than a page")
    if page_table.dtype is not torch.int32 or len(table) != 2 or page_table.get_device() != dev \
            or (table[1] > 1 and stride[1] != 1):
        _refuse("page_table must be int32 [n_seqs, width] on the GPU, rows contiguous")
    n, width = table
    return _CACHE.pack(pages.data_ptr(), pages.stride(0) if shape[0] > 1 else shape[1], page_table.data_ptr(),
                       stride[0] if n > 1 else width, 0 if status is None else _word(status, dev), shape[0], page_size,
                       n_kv_heads, head_dim, n, width), n


def kv_append(pages, page_table, starts, cu_tokens, k, v, *, page_size, q=None, cos=None, sin=None,
              interleaved=False, q_out=None, k_out=None, positions=None, status=None, stream=None):
    """Append new tokens to the cache, rotating their keys and queries (moe_kv_append).

    Tokens [cu_tokens[s], cu_tokens[s+1]) go to positions starts[s], starts[s] + 1, ... of sequence s; with `positions` (int32
    [n_seqs], moe_kv_append_at) they are rotated by positions[s], positions[s] + 1, ... instead.
    cos, sin [n_positions, rot_dim / 2] (``rope_table``); None: no rotation.  Returns the rotated queries
    (None without q) and the rotated keys, both contiguous in the inputs' type; the cache holds the keys
    quantised from their fp32 values."""
    dev, dtype = _device(k), k.dtype
    if dtype not in _DTYPES or k.dim() != 3:
        _refuse("k must be float32, bfloat16 or float16 [tokens, heads, head_dim]")
    T, hkv, d = k.shape
    c, n_seqs = _cache(pages, page_table, page_size, hkv, d, status, dev)
    tk, tv = _tokens(k, "k", T, hkv, d, dtype, dev), _tokens(v, "v", T, hkv, d, dtype, dev)
    ps, pc = _index(starts, "starts", n_seqs, dev), _index(cu_tokens, "cu_tokens", n_seqs + 1, dev)
    pp = None if positions is None else _index(positions, "positions", n_seqs, dev)
    tq, hq, rot, n_pos, cp, sp = None, 0, 0, 0, None, None
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        tq = _tokens(q, "q", T, None, d, dtype, dev)
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape or cos.dtype is not torch.float32 \
                or sin.dtype is not torch.float32 or cos.get_device() != dev or sin.get_device() != dev \
                or not cos.is_contiguous() or not sin.is_contiguous():
            _refuse("cos and sin must be contiguous float32 [n_positions, rot_dim / 2] on the GPU")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        cp, sp = cos.data_ptr(), sin.data_ptr()

    def run(handle):
        qo = None if tq is None else _output(q_out, "q_out", (T, hq, d), dtype, dev)
        ko = _output(k_out, "k_out", (T, hkv, d), dtype, dev)
        if pp is None:
            rc = _lib().moe_kv_append(c, ps, pc, T, tq, hq, tk, tv, cp, sp, rot, n_pos, int(interleaved),
                                      None if qo is None else qo.data_ptr(), ko.data_ptr(), _DTYPES[dtype], handle)
        else:
            rc = _lib().moe_kv_append_at(c, ps, pp, pc, T, tq, hq, tk, tv, cp, sp, rot, n_pos, int(interleaved),
                                         None if qo is None else qo.data_ptr(), ko.data_ptr(), _DTYPES[dtype], handle)
        if rc:
            _check(rc, "moe_kv_append")
        return qo, ko
    return _call(stream, dev, run, pages, page_table, starts, cu_tokens, q, k, v, cos, sin, q_out, k_out, positions, status)


def kv_read(pages, page_table, starts, cu_tokens, n_tokens, *, page_size, n_kv_heads, head_dim,
            dtype=torch.bfloat16, status=None, stream=None):
    """The values of cached tokens starts[s] + (i - cu_tokens[s]): keys and values [n_tokens, n_kv_heads,
    head_dim] (moe_kv_read)."""
    dev = _device(pages)
    if dtype not in _DTYPES or n_tokens < 0:
        _refuse("dtype must be float32, bfloat16 or float16, and n_tokens not negative")
    c, n_seqs = _cache(pages, page_table, page_size, n_kv_heads, head_dim, status, dev)
    ps, pc = _index(starts, "starts", n_seqs, dev), _index(cu_tokens, "cu_tokens", n_seqs + 1, dev)

    def run(handle):
        shape = (n_tokens, n_kv_heads, head_dim)
        k, v = _output(None, "k", shape, dtype, dev), _output(None, "v", shape, dtype, dev)
        rc = _lib().moe_kv_read(c, ps, pc, n_tokens, k.data_ptr(), v.data_ptr(), _DTYPES[dtype], handle)
        if rc:
            _check(rc, "moe_kv_read")
        return k, v
    return _call(stream, dev, run, pages, page_table, starts, cu_tokens, status)


_workspaces = {}
_workspaces_lock = threading.Lock()
# Workspaces kept at most, 6 to 20 MB each: a program that goes on making streams would keep one or two of each.  The
# oldest goes first; work that still uses it is on the stream whose later allocations alone can have its memory.
_MOST_KEPT = 32
_PER_THREAD_STREAM = 2  # cudaStreamPerThread: one handle, another stream in every thread
# prompts of at most so many keys or of more rows (tokens times heads) never use a workspace
_FEW_KEYS, _FEW_ROWS = 256, 131072


def kv_attention_workspace(n_q_heads, n_kv_heads, head_dim, q_tokens=1, device="cuda"):
    """A workspace for kv_attention, to be used by one stream (or one captured graph) at a time."""
    n = int(_lib().moe_kv_attention_workspace(n_q_heads, n_kv_heads, head_dim, q_tokens))
    if n <= 0:
        _refuse("kv_attention_workspace: unsupported sizes", MOE_ERR_UNSUPPORTED)
    return _zero_counters(n, device)


def _zero_counters(n, device):
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:MOE_KV_COUNTER_BYTES].zero_()
    return ws


def _kept(key, make):
    # one per stream, as calls on one stream follow each other; a capture gets its own, which its graph keeps
    if torch.cuda.is_current_stream_capturing():
        return make()
    if key[1] == _PER_THREAD_STREAM:
        key += (threading.get_ident(),)
    ws = _workspaces.get(key)
    if ws is None:
        ws = make()
        with _workspaces_lock:
            while len(_workspaces) >= _MOST_KEPT:
                del _workspaces[next(iter(_workspaces))]
            _workspaces[key] = ws
    return ws


def _workspace(hq, hkv, d, q_tokens, handle, dev):
    return _kept((dev, handle, d), lambda: kv_attention_workspace(hq, hkv, d, q_tokens, _cuda(dev)))


def kv_attention(q, pages, page_table, seq_lens, *, page_size, n_kv_heads, q_tokens=1, scale=None, window=0,
                 return_lse=False, out=None, workspace=None, status=None, stream=None):
    """Attention of every sequence's last q_tokens tokens over the cache (moe_kv_attention).

    q [n_seqs * q_tokens, n_q_heads, head_dim] bfloat16 or float16; seq_lens int32 [n_seqs] counts the cached
    tokens, the queried ones among them.  window > 0: a token sees itself and the window - 1 tokens before it.
    Returns [n_seqs * q_tokens, n_q_heads, head_dim], and the log of the sums of exponentials (fp32) with
    return_lse.  Without `workspace` a module-level one per stream is used (inside a graph capture: one of the
    capture's own); graphs that may run at the same time need their own."""
    dev, dtype = _device(q), q.dtype
    if q.dim() != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    shape = q.shape
    n, hq, d = shape
    c, n_seqs = _cache(pages, page_table, page_size, n_kv_heads, d, status, dev)
    if n != n_seqs * q_tokens or n_kv_heads <= 0 or hq % n_kv_heads:
        _refuse("q must hold q_tokens tokens of every sequence, its heads a multiple of n_kv_heads")
    tq = _tokens(q, "q", n, hq, d, dtype, dev)
    pl = _index(seq_lens, "seq_lens", n_seqs, dev)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        _refuse("workspace must be a contiguous tensor on the GPU")

    window = _window(window)

    def run(handle):
        o = _output(out, "out", shape, dtype, dev)
        lse = torch.empty((n, hq), dtype=torch.float32, device=_cuda(dev)) if return_lse else None
        if n:
            ws = _workspace(hq, n_kv_heads, d, q_tokens, handle, dev) if workspace is None else workspace
            rc = _lib().moe_kv_attention(c, pl, tq, hq, q_tokens, d ** -0.5 if scale is None else scale, window,
                                         o.data_ptr(), lse.data_ptr() if return_lse else None, _DTYPES[dtype],
                                         ws.data_ptr(), ws.numel() * ws.element_size(), handle)
            if rc:
                _check(rc, "moe_kv_attention")
        return (o, lse) if return_lse else o
    return _call(stream, dev, run, q, pages, page_table, seq_lens, out, workspace, status)


def prompt_attention_workspace(n_q_tokens, n_q_heads, n_k_tokens, n_kv_heads, head_dim, n_seqs, window=0, device="cuda"):
    """A workspace for prompt_attention, to be used by one stream (or one captured graph) at a time; None where a call
    of these sizes would not use one."""
    n = int(_lib().moe_prompt_attention_workspace(n_q_tokens, n_q_heads, n_k_tokens, n_kv_heads, head_dim, n_seqs,
                                                  _window(window)))
    return _zero_counters(n, device) if n > 0 else None


def prompt_attention(q, k, v, cu_q, cu_k=None, *, scale=None, window=0, return_lse=False, out=None, workspace=None,
                     status=None, stream=None):
    """Causal attention over packed prompts (moe_prompt_attention).

    q [n_q_tokens, n_q_heads, head_dim], k and v [n_k_tokens, n_kv_heads, head_dim], bfloat16 or float16;
    cu_q, cu_k int32 [n_seqs + 1] (cu_k None: cu_q); rows that no sequence holds give NaN, and a status.  With more keys
    than queries a sequence's queries are its last tokens.  window > 0: a token sees itself and the window - 1 tokens
    before it.  Returns q's shape, and the log of the sums of exponentials (fp32 [n_q_tokens, n_q_heads]) with
    return_lse.  Few queries of many keys use a workspace: without `workspace` a module-level one per stream (inside a
    graph capture: one of the capture's own); graphs that may run at the same time need their own."""
    dev, dtype = _device(q), q.dtype
    if q.dim() != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    shape = q.shape
    n, hq, d = shape
    tq, tk = _tokens(q, "q", n, hq, d, dtype, dev), _tokens(k, "k", None, None, d, dtype, dev)
    nk, hkv = k.shape[0], k.shape[1]
    tv = _tokens(v, "v", nk, hkv, d, dtype, dev)
    if cu_q.dim() != 1 or cu_q.shape[0] < (2 if n else 1):
        _refuse("cu_q must hold n_seqs + 1 offsets, of one sequence at least where there are tokens")
    n_cu = cu_q.shape[0]
    pq = _index(cu_q, "cu_q", n_cu, dev)
    pk = pq if cu_k is None else _index(cu_k, "cu_k", n_cu, dev)
    word = _word(status, dev)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        _refuse("workspace must be a contiguous tensor on the GPU")

    window = _window(window)

    def run(handle):
        o = _output(out, "out", shape, dtype, dev)
        lse = torch.empty((n, hq), dtype=torch.float32, device=_cuda(dev)) if return_lse else None
        L, ws = _lib(), workspace
        if ws is None and nk > _FEW_KEYS and n * hq <= _FEW_ROWS:
            # (its size depends on the head size alone, once it is not 0)
            if L.moe_prompt_attention_workspace(n, hq, nk, hkv, d, n_cu - 1, window) > 0:
                ws = _kept((dev, handle, "prompt", d),
                           lambda: prompt_attention_workspace(n, hq, nk, hkv, d, n_cu - 1, window, _cuda(dev)))
        factor, po, pl = d ** -0.5 if scale is None else scale, o.data_ptr(), lse.data_ptr() if return_lse else None
        if ws is None:
            rc = L.moe_prompt_attention(tq, n, hq, tk, tv, nk, hkv, d, pq, pk, n_cu - 1, factor, window, po, pl,
                                        _DTYPES[dtype], word, handle)
        else:
            rc = L.moe_prompt_attention_shared(tq, n, hq, tk, tv, nk, hkv, d, pq, pk, n_cu - 1, factor, window, po, pl,
                                               _DTYPES[dtype], word, ws.data_ptr(), ws.numel() * ws.element_size(), handle)
        if rc:
            _check(rc, "moe_prompt_attention")
        return (o, lse) if return_lse else o
    return _call(stream, dev, run, q, k, v, cu_q, cu_k, out, workspace, status)


def status_message(status) -> str:
    """What the bits of a status word say (reads it: waits for the GPU); empty when nothing is wrong."""
    bits = int(status.item())
    names = ((MOE_KV_BAD_PAGE, "a page number outside the cache"),
             (MOE_KV_BAD_LENGTH, "a length or offset outside the page table or the tensor"),
             (MOE_KV_BAD_POSITION, "a position past the rotation table"),
             (MOE_KV_TIMED_OUT, "a device wait gave up"),
             (MOE_ROUTE_BAD_LOGIT, "a logit that is NaN or +infinity, or a bias that is not finite"))
    return "; ".join(text for bit, text in names if bits & bit)
