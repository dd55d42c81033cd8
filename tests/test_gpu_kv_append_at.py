"""Appending with positions of their own: the rotation of one place, the cache of another."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests.test_gpu_kv_cache import i32, make_table

pytestmark = pytest.mark.gpu


def append(lens, starts, positions, q, k, v, cos, sin, ps=32, status=None, inter=False):
    n_pages = sum(-(-(a + n) // ps) for a, n in zip(starts, lens)) + 1
    table = make_table([a + n for a, n in zip(starts, lens)], ps, n_pages).cuda()
    pages = moe.kv_pages(n_pages, k.shape[1], k.shape[2], ps)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    qo, ko = moe.kv_append(pages, table, i32(starts), i32(cu), k, v, page_size=ps, q=q, cos=cos, sin=sin, interleaved=inter,
                           positions=None if positions is None else i32(positions), status=status)
    kc, vc = moe.kv_read(pages, table, i32(starts), i32(cu), cu[-1], page_size=ps, n_kv_heads=k.shape[1], head_dim=k.shape[2],
                         dtype=torch.float32)
    return qo, ko, kc, vc


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 64, True), (256, 256, False)])
def test_rotated_by_positions_placed_by_starts(d, rot, inter):
    lens, starts, positions = [3, 0, 40, 1], [5, 9, 0, 31], [100, 7, 333, 0]
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.randn(44, h, d, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    cos, sin = moe.rope_table(400, rot)
    got = append(lens, starts, positions, q, k, v, cos, sin, inter=inter)
    # what an append at those places of a longer cache gives
    want = append(lens, positions, None, q, k, v, cos, sin, inter=inter)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    own = append(lens, starts, starts, q, k, v, cos, sin, inter=inter)
    assert all(torch.equal(a, b) for a, b in zip(own, append(lens, starts, None, q, k, v, cos, sin, inter=inter)))


def test_positions_that_make_no_sense():
    lens, starts = [2, 3], [4, 0]
    q, k, v = (torch.randn(5, 2, 64, device="cuda") for _ in range(3))
    cos, sin = moe.rope_table(10, 64)
    want = append(lens, starts, [1, 2], q, k, v, cos, sin)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1, 9, 1 << 30, -(1 << 31)):
        status.zero_()
        got = append(lens, starts, [bad, 2], q, k, v, cos, sin, status=status)
        assert int(status) == moe.MOE_KV_BAD_POSITION
        lost = 1 if bad == 9 else 0          # position 9 is the table's last
        assert bool(got[0][lost:2].isnan().all()) and bool(got[1][lost:2].isnan().all())
        for a, b in zip(got, want):
            assert torch.equal(a[2:], b[2:])
    # without a rotation they are not looked at
    status.zero_()
    append(lens, starts, [-1, 1 << 30], q, k, v, None, None, status=status)
    assert int(status) == 0
    with pytest.raises(moe.MoeError):
        moe.kv_append(moe.kv_pages(2, 2, 64, 32), i32([[0], [1]]), i32(starts), i32([0, 2, 5]), k, v, page_size=32, positions=i32([1]))
