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
