"""A cache of bounded size, for PyTorch tensors: the attention weight that cached tokens
receive, and keeping those with most of it (``include/moe_attention.h``; argument checks
and marshalling only).

Totals are float32 ``[n_pages, n_kv_heads, page_size]``, of the same pages as the cache's
tokens.  Streams, outputs and errors are as for the attention operators; a page belongs
to one sequence, once.
"""
from __future__ import annotations

import ctypes

import torch

from . import MOE_ERR_UNSUPPORTED, _check, lib
from .attention import _DTYPES, _cache, _call, _cuda, _device, _index, _refuse, _tokens, _window, _word

_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        L.moe_kv_weigh.argtypes = [vp, vp, vp, i32, i32, f32, i32, vp, vp, i32, i32, vp]
        L.moe_kv_evict_workspace.restype = ctypes.c_int64
        L.moe_kv_evict_workspace.argtypes = [vp]
        L.moe_kv_evict.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, ctypes.c_int64, vp]
        L.moe_prompt_weigh.argtypes = [vp, i32, i32, vp, i32, i32, i32, vp, vp, i32, f32, i32, vp, vp, ctypes.c_int64, i32, i32,
                                       i32, vp, i32, i32, vp, vp]
        _bound = L
    return _bound


def kv_totals(n_pages: int, n_kv_heads: int, page_size: int, device="cuda"):
    """Totals of an empty cache: zeros, float32 [n_pages, n_kv_heads, page_size]."""
    return torch.zeros(n_pages, n_kv_heads, page_size, dtype=torch.float32, device=device)


def _totals(t, n_pages, hkv, page_size, dev):
    if t.dtype is not torch.float32 or tuple(t.shape) != (n_pages, hkv, page_size) or t.get_device() != dev \
            or not t.is_contiguous():
        _refuse(f"totals must be a contiguous float32 tensor [{n_pages}, {hkv}, {page_size}] on the GPU")
    return t.data_ptr()


def _lse(t, n, hq, dev):
    if t.dtype is not torch.float32 or tuple(t.shape) != (n, hq) or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"lse must be a contiguous float32 tensor [{n}, {hq}] on the GPU")
    return t.data_ptr()


def kv_weigh(q, pages, page_table, seq_lens, lse, *, totals, page_size, n_kv_heads, q_tokens=1, scale=None, window=0,
             restart=False, status=None, stream=None):
    """Adds the attention weights of every sequence's last q_tokens tokens to the totals of the tokens that they see
    (moe_kv_weigh).

    The arguments are those of ``kv_attention``, lse what it returns with return_lse.  The queried tokens are new: their
    totals begin at 0; with restart all tokens' of the sequences do.  Returns totals, written in place."""
    dev, dtype = _device(q), q.dtype
    if q.dim() != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    n, hq, d = q.shape
    c, n_seqs = _cache(pages, page_table, page_size, n_kv_heads, d, status, dev)
    if n != n_seqs * q_tokens or n_kv_heads <= 0 or hq % n_kv_heads:
        _refuse("q must hold q_tokens tokens of every sequence, its heads a multiple of n_kv_heads")
    tq = _tokens(q, "q", n, hq, d, dtype, dev)
    pl = _index(seq_lens, "seq_lens", n_seqs, dev)
    pe, pt = _lse(lse, n, hq, dev), _totals(totals, pages.shape[0], n_kv_heads, page_size, dev)
    window = _window(window)

    def run(handle):
        if n:
            rc = _lib().moe_kv_weigh(c, pl, tq, hq, q_tokens, d ** -0.5 if scale is None else scale, window, pe, pt,
                                     bool(restart), _DTYPES[dtype], handle)
            if rc:
                _check(rc, "moe_kv_weigh")
        return totals
    return _call(stream, dev, run, q, pages, page_table, seq_lens, lse, totals, status)


def prompt_weigh(q, k, lse, cu_q, cu_k=None, *, totals, page_table, scale=None, window=0, restart=False, status=None,
                 stream=None):
    """Adds the attention weights of whole prompts' queries, packed one after another, to the totals of the tokens that they
    see (moe_prompt_weigh).

    The arguments are those of ``prompt_attention``, lse what it returns with return_lse; key i of a sequence is its cached
    token i, whose total is found by page_table int32 [n_seqs, width].  The queried tokens, a sequence's last ones, are
    new: their totals begin at 0; with restart all tokens' of the sequences do.  Returns totals, written in place."""
    dev, dtype = _device(q), q.dtype
    if q.dim() != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        _refuse("q must be bfloat16 or float16 [tokens, heads, head_dim]", MOE_ERR_UNSUPPORTED)
    n, hq, d = q.shape
    tq, tk = _tokens(q, "q", n, hq, d, dtype, dev), _tokens(k, "k", None, None, d, dtype, dev)
    nk, hkv = k.shape[0], k.shape[1]
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        _refuse("cu_q must hold n_seqs + 1 offsets")
    n_cu = cu_q.shape[0]
    pq = _index(cu_q, "cu_q", n_cu, dev)
    pk = pq if cu_k is None else _index(cu_k, "cu_k", n_cu, dev)
    if page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n_cu - 1 \
            or page_table.get_device() != dev or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        _refuse("page_table must be int32 [n_seqs, width] on the GPU, rows contiguous")
    if totals.dim() != 3:
        _refuse("totals must be float32 [n_pages, n_kv_heads, page_size]")
    n_pages, _, page_size = totals.shape
    pe, pt = _lse(lse, n, hq, dev), _totals(totals, n_pages, hkv, page_size, dev)
    width = page_table.shape[1]
    row = page_table.stride(0) if n_cu > 2 else width
    word, window = _word(status, dev), _window(window)

    def run(handle):
        rc = _lib().moe_prompt_weigh(tq, n, hq, tk, nk, hkv, d, pq, pk, n_cu - 1, d ** -0.5 if scale is None else scale, window, pe,
                                     page_table.data_ptr(), row, width, n_pages, page_size, pt, bool(restart), _DTYPES[dtype],
                                     word, handle)
        if rc:
            _check(rc, "moe_prompt_weigh")
        return totals
    return _call(stream, dev, run, q, k, lse, cu_q, cu_k, totals, page_table, status)


def kv_evict(pages, page_table, seq_lens, budget, *, totals, page_size, n_kv_heads, head_dim, first=0, recent=0, status=None,
             stream=None):
    """Keeps budget tokens of every sequence that has more (moe_kv_evict): per head its first `first` and last `recent`
    tokens and the heaviest by totals of those between, moved together in place, in their order.

    Returns the new lengths int32 [n_seqs] and the slots that the kept tokens had, int32 [n_seqs, n_kv_heads, budget]
    (ascending; -1 past a shorter sequence's tokens).  pages and totals are written in place; the totals of the slots given
    free become 0.  A kept key stays as it was rotated: tokens appended from then on need ``positions`` of their own
    (``kv_append``).  A window counts places: of w tokens, the last w kept ones."""
    dev = _device(pages)
    c, n_seqs = _cache(pages, page_table, page_size, n_kv_heads, head_dim, status, dev)
    pl = _index(seq_lens, "seq_lens", n_seqs, dev)
    pt = _totals(totals, pages.shape[0], n_kv_heads, page_size, dev)
    if not 0 <= budget <= 2 ** 30 or first < 0 or recent < 0 or first + recent > budget:
        _refuse("budget must be at least first + recent and at most 2^30, none of them negative")

    def run(handle):
        d = _cuda(dev)
        new_lens = torch.empty(n_seqs, dtype=torch.int32, device=d)
        kept = torch.empty((n_seqs, n_kv_heads, budget), dtype=torch.int32, device=d)
        if n_seqs:
            L = _lib()
            size = L.moe_kv_evict_workspace(c)
            if size <= 0:
                _refuse("kv_evict: unsupported sizes", MOE_ERR_UNSUPPORTED)
            ws = torch.empty(size, dtype=torch.uint8, device=d)
            rc = L.moe_kv_evict(c, pl, pt, budget, first, recent, new_lens.data_ptr(), kept.data_ptr(), ws.data_ptr(), size,
                                handle)
            if rc:
                _check(rc, "moe_kv_evict")
        return new_lens, kept
    return _call(stream, dev, run, pages, page_table, seq_lens, totals, status)
