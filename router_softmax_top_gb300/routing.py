"""Routing of tokens to experts, for PyTorch tensors (``include/moe_route.h``; argument
checks and marshalling only): scores by softmax or sigmoid, a bias for balance, groups
of experts, renormalised weights.  ``MoECache.forward_routed`` takes the choice.

Streams, outputs and errors are as for the attention operators.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import MOE_ERR_UNSUPPORTED, _check, lib
from .attention import _DTYPES, MOE_ROUTE_BAD_LOGIT, _call, _device, _output, _refuse, _word  # noqa: F401

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


class MoeRouting(ctypes.Structure):
    """moe_routing"""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_experts", "top_k", "score", "n_groups", "top_groups", "group_score",
                                              "renormalise")] + [("scale", ctypes.c_float)]


_ROUTING = struct.Struct("@iiiiiiif")
_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [vp, vp, i64, i32, vp, vp, vp, i32, vp, vp]
        _bound = L
    return _bound


def route(logits, top_k, *, score="softmax", bias=None, n_groups=1, top_groups=None, group_score="top2",
          renormalise=False, scale=1.0, ids_out=None, weights_out=None, status=None, stream=None):
    """The top_k experts of every token and their weights (moe_route).

    logits [tokens, experts] float32, bfloat16 or float16 with contiguous rows.  score "softmax" or "sigmoid"; bias float32
    [experts] is added to the scores for the choice alone; of n_groups groups of neighbouring experts the top_groups (None:
    all) with the largest group_score ("max": of a member, "top2": sum of its two largest) are chosen from; weights are
    scale times the scores, over their sum with renormalise.  Returns ids int32 and weights float32, both [tokens, top_k],
    in descending order of score plus bias, ties to the lower expert.  A logit of -infinity closes an expert; a row with a
    NaN or +infinity, or with a bias that is not finite, has NaN weights."""
    dev, dtype = _device(logits), logits.dtype
    shape, stride = logits.shape, logits.stride()
    if dtype not in _DTYPES or len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        _refuse("logits must be float32, bfloat16 or float16 [tokens, experts] with contiguous rows")
    n, e = shape
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        _refuse("score is 'softmax' or 'sigmoid', group_score 'max' or 'top2'")
    if bias is not None and (bias.dtype is not torch.float32 or bias.dim() != 1 or bias.shape[0] != e
                             or bias.get_device() != dev or not bias.is_contiguous()):
        _refuse("bias must be a contiguous float32 tensor of an entry per expert on the GPU")
    if top_groups is None:
        top_groups = n_groups
    if max(e, top_k, n_groups, top_groups) > 1024:  # (past 32 bits they could not be passed on)
        _refuse("at most 1024 experts, top_k 32 and 32 groups", MOE_ERR_UNSUPPORTED)
    if min(top_k, n_groups, top_groups) < 1:
        _refuse("top_k, n_groups and top_groups are at least 1")
    if not abs(scale) <= 3.4e38:
        _refuse("scale must be a number that fp32 holds")
    r = _ROUTING.pack(e, top_k, _SCORES[score], n_groups, top_groups, _GROUP_SCORES[group_score], bool(renormalise), scale)
    word = _word(status, dev)

    def run(handle):
        ids = _output(ids_out, "ids_out", (n, top_k), torch.int32, dev)
        weights = _output(weights_out, "weights_out", (n, top_k), torch.float32, dev)
        rc = _lib().moe_route(r, logits.data_ptr(), stride[0], n, None if bias is None else bias.data_ptr(),
                              ids.data_ptr(), weights.data_ptr(), _DTYPES[dtype], word, handle)
        if rc:
            _check(rc, "moe_route")
        return ids, weights
    return _call(stream, dev, run, logits, bias, ids_out, weights_out, status)
