"""Prompt attention over offsets and windows at the edges of what they can say."""
import pytest
import torch

import router_softmax_top_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seeded():
    torch.manual_seed(23)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(n, *heads, d=64, dt=torch.bfloat16):
    return [torch.randn(n, h, d, device="cuda").to(dt) for h in heads]


def test_overlapping_sequences_leave_a_shared_workspace_ready():
    # Offsets that go back and forth hold far more tile groups than the tokens do; were they all taken, the parts of a
    # group would not all have a CTA, and its count would be left for the next call.
    n = 1024
    q, k, v = rows(n, 1, 1, 1, d=128)
    bad, good = i32([0, n] * 16 + [0]), i32([0] * 32 + [n])
    ws = moe.prompt_attention_workspace(n, 1, n, 1, 128, 32)
    assert ws is not None
    want, lse = moe.prompt_attention(q, k, v, good, return_lse=True, workspace=ws)
    assert not bool(ws[:moe.MOE_KV_COUNTER_BYTES].any())
    status = i32([0])
    got = moe.prompt_attention(q, k, v, bad, workspace=ws, status=status)
    assert int(status) == moe.MOE_KV_BAD_LENGTH
    assert not bool(ws[:moe.MOE_KV_COUNTER_BYTES].any())
    near = 4 * 2.0 ** -8      # (the first of them is taken; its keys may be shared otherwise)
    assert bool(((got.float() - want.float()).abs() <= near * (1 + want.float().abs())).all())
    for _ in range(3):
        again, lse2 = moe.prompt_attention(q, k, v, good, return_lse=True, workspace=ws)
        assert torch.equal(again, want) and torch.equal(lse2, lse)
    assert not bool(ws[:moe.MOE_KV_COUNTER_BYTES].any())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,cu,held", [
    (12, [3, 10], range(3, 10)),
    (12, [0, 5, 5, 10], range(10)),
    (12, [0, 0], []),
    (40, [0, 20, 50], range(20)),                      # the second one ends past the tokens
    (40, [-1, 20, 40], range(20, 40)),
    (40, [0, 30, 10, 40], range(30)),                  # the third one begins inside the first
    (40, [20, 40, 0, 10], range(20, 40)),
    (700, [100 + i for i in range(80)] + [400, 300, 500], range(100, 400)),
    (5000, [4000, 4100], range(4000, 4100))])
def test_rows_that_no_sequence_holds_are_nan(d, dtype, n, cu, held):
    q, k, v = rows(n, 4, 2, 2, d=d, dt=dtype)
    seen = torch.zeros(n, dtype=torch.bool, device="cuda")
    seen[list(held)] = True
    out, status = torch.full_like(q, 7.0), i32([0])
    got, lse = moe.prompt_attention(q, k, v, i32(cu), i32([max(0, min(x, n)) for x in cu]), out=out, status=status,
                                    return_lse=True)
    assert int(status) == moe.MOE_KV_BAD_LENGTH
    assert got is out
    assert bool(torch.isnan(out[~seen]).all()) and bool(torch.isnan(lse[~seen]).all())
    assert bool(torch.isfinite(out[seen]).all()) and bool(torch.isfinite(lse[seen]).all())


def test_rows_held_beside_rows_that_are_not():
    q, k, v = rows(100, 4, 2, 2)
    clean = moe.prompt_attention(q[20:70].contiguous(), k[20:70].contiguous(), v[20:70].contiguous(), i32([0, 50]))
    got = moe.prompt_attention(q, k, v, i32([20, 70]))
    assert torch.equal(got[20:70], clean)


def test_tokens_without_sequences_are_refused():
    q, k, v = rows(5, 4, 2, 2)
    with pytest.raises(moe.MoeError):
        moe.prompt_attention(q, k, v, i32([0]))
    assert moe.prompt_attention(q[:0], k, v, i32([0])).shape == (0, 4, 64)


def test_full_offsets_set_no_status():
    q, k, v = rows(300, 4, 2, 2)
    for cu in ([0, 300], [0, 0, 100, 100, 300], list(range(0, 301, 3))):
        status = i32([0])
        out = moe.prompt_attention(q, k, v, i32(cu), status=status)
        assert int(status) == 0 and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("nq,nk", [(50, 20), (300, 10), (7, 200)])
def test_the_widest_window_is_no_window(d, nq, nk):
    # with more queries than keys the first ones stand before position 0: that less the window passes 32 bits
    q, _ = rows(nq, 4, 2, d=d)
    k, v = rows(nk, 2, 2, d=d)
    want, lse = moe.prompt_attention(q, k, v, i32([0, nq]), i32([0, nk]), return_lse=True)
    for window in (2147483647, 2147483640):
        got, l = moe.prompt_attention(q, k, v, i32([0, nq]), i32([0, nk]), window=window, return_lse=True)
        assert torch.equal(got, want) and torch.equal(l, lse)
