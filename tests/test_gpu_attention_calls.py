"""How the attention operators are called: streams, sizes of nothing, arguments at their ends."""
import pytest
import torch

import router_softmax_top_gb300 as moe

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def some_cache(n, ps=32, hkv=2, d=64):
    pages = moe.kv_pages(-(-n // ps), hkv, d, ps)
    table = torch.arange(pages.shape[0], dtype=torch.int32, device="cuda")[None]
    k, v = [torch.randn(n, hkv, d, device="cuda").bfloat16() for _ in range(2)]
    moe.kv_append(pages, table, i32([0]), i32([0, n]), k, v, page_size=ps)
    return pages, table


@pytest.mark.parametrize("rot", [0, 32, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_without_a_place_are_nan_whatever_is_rotated(rot, interleaved):
    x = torch.randn(6, 2, 64, device="cuda")
    cos, sin = moe.rope_table(34, rot) if rot else (None, None)
    for starts, cu, bit, dead in (([-1], [0, 6], moe.MOE_KV_BAD_LENGTH, range(6)),
                                  ([0], [0, 4], moe.MOE_KV_BAD_LENGTH, [4, 5]),
                                  ([30], [0, 6], moe.MOE_KV_BAD_POSITION, [4, 5])):
        if not rot and bit == moe.MOE_KV_BAD_POSITION:
            continue
        pages, status = moe.kv_pages(2, 2, 64, 32), i32([0])
        q, k = moe.kv_append(pages, i32([[0, 1]]), i32(starts), i32(cu), x, x, page_size=32, q=x, cos=cos, sin=sin,
                             interleaved=interleaved, status=status)
        assert int(status) == bit
        gone = torch.zeros(6, dtype=torch.bool, device="cuda")
        gone[list(dead)] = True
        for y in (q, k):
            assert bool(torch.isnan(y[gone]).all()) and bool(torch.isfinite(y[~gone]).all())


def test_a_step_of_no_sequences():
    pages = moe.kv_pages(1, 2, 64, 32)
    table, none, cu = i32([[0]])[:0], i32([]), i32([0])
    q, k = [torch.zeros(0, h, 64, device="cuda", dtype=torch.bfloat16) for h in (4, 2)]
    a, b = moe.kv_append(pages, table, none, cu, k, k, page_size=32, q=q)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    for t in moe.kv_read(pages, table, none, cu, 0, page_size=32, n_kv_heads=2, head_dim=64):
        assert t.shape == (0, 2, 64)
    assert moe.kv_attention(q, pages, table, none, page_size=32, n_kv_heads=2).shape == (0, 4, 64)
    assert moe.prompt_attention(q, k, k, cu).shape == (0, 4, 64)
    one = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):       # tokens without a sequence
        moe.kv_append(pages, table, none, cu, one, one, page_size=32)
    with pytest.raises(moe.MoeError):
        moe.kv_read(pages, table, none, cu, 1, page_size=32, n_kv_heads=2, head_dim=64)


def test_inputs_given_up_after_a_call_on_another_stream_keep_their_memory():
    n = 300
    pages, table = some_cache(n)
    lens, cu, ks = i32([n]), i32([0, n]), i32([0])
    q1 = torch.randn(1, 4, 64, device="cuda").bfloat16()
    q, k, v = [torch.randn(n, h, 64, device="cuda").bfloat16() for h in (4, 2, 2)]
    cos, sin = moe.rope_table(n, 64)
    calls = {
        "decode": (lambda q, s: moe.kv_attention(q, pages, table, lens, page_size=32, n_kv_heads=2, stream=s), [q1]),
        "prompt": (lambda q, k, v, s: moe.prompt_attention(q, k, v, cu, stream=s), [q, k, v]),
        "append": (lambda q, k, v, s: moe.kv_append(torch.zeros_like(pages) if s is None else scratch, table, ks, cu, k, v,
                                                    page_size=32, q=q, cos=cos, sin=sin, stream=s), [q, k, v]),
        "read": (lambda t, s: moe.kv_read(pages, t, ks, cu, n, page_size=32, n_kv_heads=2, head_dim=64, stream=s), [table])}
    side = torch.cuda.Stream()
    scratch = torch.zeros_like(pages)
    for name, (call, inputs) in calls.items():
        want = call(*inputs, None)
        given = [t.clone() for t in inputs]
        at = [t.data_ptr() for t in given]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)     # the call has to wait behind this
        got = call(*given, side)
        given = None
        # memory of the same sizes, asked for on this stream, and written
        new = [torch.zeros_like(t) for t in inputs]
        reused = [t.data_ptr() in at for t in new]
        torch.cuda.synchronize()
        want, got = [x if isinstance(x, tuple) else (x,) for x in (want, got)]
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        assert not any(reused), name


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 5, (1 << 63) - 1, 10 ** 30])
def test_windows_past_32_bits_are_no_window(window):
    n = 200
    pages, table = some_cache(n)
    q, k, v = [torch.randn(n, h, 64, device="cuda").bfloat16() for h in (4, 2, 2)]
    assert torch.equal(moe.prompt_attention(q, k, v, i32([0, n]), window=window), moe.prompt_attention(q, k, v, i32([0, n])))
    args = (q[:1], pages, table, i32([n]))
    assert torch.equal(moe.kv_attention(*args, page_size=32, n_kv_heads=2, window=window),
                       moe.kv_attention(*args, page_size=32, n_kv_heads=2))


@pytest.mark.parametrize("window", [-1, -(1 << 31), 5 - (1 << 32)])
def test_negative_windows_are_refused(window):
    pages, table = some_cache(40)
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    with pytest.raises(moe.MoeError):
        moe.kv_attention(q, pages, table, i32([40]), page_size=32, n_kv_heads=2, window=window)
    with pytest.raises(moe.MoeError):
        moe.prompt_attention(q, q[:, :2], q[:, :2], i32([0, 1]), window=window)


def test_outputs_that_are_refused_are_refused_on_any_stream():
    pages, table = some_cache(40)
    q, k = [torch.randn(1, h, 64, device="cuda").bfloat16() for h in (4, 2)]
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        with pytest.raises(moe.MoeError):
            moe.kv_attention(q, pages, table, i32([40]), page_size=32, n_kv_heads=2, out=q.cpu(), stream=stream)
        with pytest.raises(moe.MoeError):
            moe.prompt_attention(q, k, k, i32([0, 1]), out=q.cpu(), stream=stream)
        with pytest.raises(moe.MoeError):
            moe.kv_append(pages, table, i32([0]), i32([0, 1]), k, k, page_size=32, k_out=k.cpu(), stream=stream)
