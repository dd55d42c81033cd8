"""Weights of routing as small as fp32 holds, under scales that show them.

Tolerance as in tests/test_gpu_route.py, and below the normal numbers, where steps are 2^-149: two of the exponential and a
half each of the sum and the quotient, three in all, times the scale."""
import numpy as np
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import route_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_small_scores_under_a_large_scale(score, bias):
    scale = 1e38
    low = torch.tensor([-80.0, -87.0, -88.0, -88.5, -88.8, -89.0, -92.0, -96.5, -100.0, -103.0])
    x = low.repeat(4, 1)
    if score == "softmax":
        x[:, 0] = 0.0
    x[1], x[2, 1:], x[3, 3] = x[1].flip(0), -float("inf"), -float("inf")
    b = torch.zeros(10) if bias else None
    ids, w = moe.route(x.cuda(), 10, score=score, bias=b.cuda() if bias else None, scale=scale)
    rid, rw, span = R.route(x.double().numpy(), 10, score, b.double().numpy() if bias else None, 1, 1, "max", False,
                            float(np.float32(scale)))
    assert np.array_equal(ids.cpu().numpy(), rid)
    tol = np.abs(rw) * (64 + span[:, None]) * 2.0 ** -24 + 3 * 2.0 ** -149 * scale
    assert (np.abs(w.cpu().double().numpy() - rw) <= tol).all(), float((np.abs(w.cpu().double().numpy() - rw) / tol).max())
