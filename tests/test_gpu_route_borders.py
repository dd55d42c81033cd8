"""Routing with a bias where the border between chosen and not is crowded: equal values at the border with another just
beside them, saturated scores, and values whose errors in 32 bits differ (against the 64-bit statement, like
tests/test_gpu_route.py; gaps are at least 1e-13 there, or ties)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 8, 32])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
@pytest.mark.parametrize("bias", [0.0, 0.25])
def test_equal_values_at_the_border_and_one_beside_them(score, k, groups, kept, bias):
    # (near 0 fp32 holds logits whose scores 32 bits do not tell apart)
    b = torch.full((128,), bias).cuda()
    for beside in (1e-8, -1e-8, 5e-7, -5e-7, 0.0):
        for n_equal in (k + 1, k + 5):
            rows = []
            for at in (0, n_equal // 2, n_equal, 63):
                x = torch.full((128,), -2.0)
                x[:n_equal + 1] = 1e-9
                x[at] = 1e-9 + beside
                rows.append(x)
                y = x.clone()                            # the same a group further on
                y[32:96] = x[:64]
                y[:32] = -2.0
                rows.append(y)
            check(torch.stack(rows).cuda(), k, score, b, groups, kept, "max")


def test_saturated_scores_that_32_bits_do_not_tell_apart():
    x = torch.full((1, 32), -2.0)
    x[0, :9], x[0, 20] = 17.0, 17.125
    for dt in (torch.float32, torch.bfloat16):
        ids, _ = check(x.to(dt).cuda(), 8, "sigmoid", torch.zeros(32).cuda())
        assert ids[0].tolist() == [20, 0, 1, 2, 3, 4, 5, 6]
    ids, _ = check(torch.tensor([[0.0, 0.0, 1e-8]]).cuda(), 1, "sigmoid", torch.zeros(3).cuda())
    assert ids.item() == 2


@pytest.mark.parametrize("k", [1, 8, 32])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 4)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_many_saturated_scores(k, groups, kept, group_score):
    g = torch.Generator().manual_seed(k)
    x = torch.randn(160, 256, generator=g)
    for t in range(160):
        x[t, torch.randperm(256, generator=g)[:24 + t % 40]] += 12 + 8 * torch.rand(1, generator=g)
    x = x.clamp(max=20).bfloat16()
    for b in (torch.zeros(256), torch.full((256,), 0.3), (torch.randint(-1, 2, (256,), generator=g) * 2.0 ** -20)):
        check(x.cuda(), k, "sigmoid", b.float().cuda(), groups, kept, group_score)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(40, 1), (200, 8), (1024, 32), (1000, 3)])
def test_duplicates_among_near_values(dt, score, E, k):
    # few distinct logits with tiny steps, so that every row has ties and near values at its border
    g = torch.Generator().manual_seed(E + k)
    steps = torch.randint(0, 12, (60, E), generator=g).float()
    x = 0.5 + steps * (2.0 ** -23 if dt is torch.float32 else 2.0 ** -8)
    for b in (torch.zeros(E), (torch.randint(0, 3, (E,), generator=g) * 2.0 ** -24).float()):
        check(x.to(dt).cuda(), k, score, b.cuda())


def test_all_values_equal():
    for E, k in ((32, 8), (256, 8), (1024, 32)):
        for score in ("softmax", "sigmoid"):
            ids, _ = check(torch.full((5, E), 1.5).cuda(), k, score, torch.full((E,), 0.25).cuda())
            assert torch.equal(ids[0].cpu(), torch.arange(k, dtype=torch.int32))


@pytest.mark.parametrize("k", [1, 2])
def test_a_large_score_beside_small_ones(k):
    # Scores far apart have errors far apart: expert 0's score is nearly all of the softmax's sum, and 31 terms of just over
    # half a step of 1 make that sum come out 2e-6 too large in 32 bits; its value is then below those of two experts of
    # tiny scores, which in 64 bits it is above.
    E = 1024
    x = np.full(E, np.float32(np.log(1.02 * 2.0 ** -24)), np.float32)
    x[0] = 0.0
    p = np.exp(x.astype(np.float64))
    p /= p.sum()
    b = np.full(E, -10.0)
    b[0] = -0.5
    c0 = p[0] - 0.5
    for below in ((7.5e-7, 1.15e-6), (7.5e-7, 7.5e-7), (-7.5e-7, -3e-7), (1.15e-6, 3e-6)):
        b[500], b[501] = c0 - below[0] - p[500], c0 - below[1] - p[501]
        ids, _ = check(torch.from_numpy(x)[None].cuda(), k, "softmax", torch.from_numpy(b.astype(np.float32)).cuda())
        assert (ids[0, 0].item() == 0) == (min(below) > 0)
