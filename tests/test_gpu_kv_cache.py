"""The paged 4-bit cache on the GPU: append, read back and attention over it, against
plain 64-bit statements (tests/attention_ref.py).

Tolerances.  Append and read: none; rotation and quantisation round every 32-bit
operation as the statement does.  Attention: with p the weights, A = sum p |v| / sum p
and Z = max_j scale sum_d |q_d k_jd| of a row, the kernel rounds p and p d to fp16
(2^-11 each, on at most 2^-24 of the largest weight's scale more), forms scores in
fp32 over D + 8 terms' products (2^-18 Z covers them at D = 256) and rounds the result
once; so |error| <= A (2^-10 + 2^-12 + 2^-17 Z) + half a step of the result.  Where nearly all the
weight is one key's and its value is 0, A says nothing about the rounding that is not
relative: p and p d below fp16's normal numbers are off by at most 2^-25 each.  With d
at most D and the reference at most 2^7 or 16 / D below the largest weight, n such keys
contribute at most n 8 2^-25 (1 + D) max(2^-7, D / 16): test_one_score_far_above_the_others."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seeded():
    torch.manual_seed(20)


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_table(lens, ps, n_pages, seed=0, width=None):
    """A page table over shuffled pages; entries past a sequence's tokens are -1."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(n_pages, generator=g).tolist()
    w = max([1] + [-(-n // ps) for n in lens]) if width is None else width
    t = torch.full((len(lens), w), -1, dtype=torch.int32)
    for s, n in enumerate(lens):
        for i in range(-(-n // ps)):
            t[s, i] = order.pop()
    return t


def filled(lens, ps, hkv, d, seed, k_size=1.0, v_size=1.0):
    """A cache of random tokens written through moe.kv_append (fp32 values, no rotation); returns pages, table."""
    n_pages = sum(-(-n // ps) for n in lens) + 2
    table = make_table(lens, ps, n_pages, seed)
    pages = moe.kv_pages(n_pages, hkv, d, ps)
    pages.fill_(0xFF)   # what was never written is NaN scales
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    if cu[-1]:
        k = torch.randn(cu[-1], hkv, d, generator=g, device="cuda") * k_size
        v = torch.randn(cu[-1], hkv, d, generator=g, device="cuda") * v_size
        moe.kv_append(pages, table.cuda(), i32([0] * len(lens)), i32(cu), k, v, page_size=ps)
    return pages, table


def check(q, pages, table, lens, ps, hkv, q_tokens=1, window=0, scale=None, tiny=0.0, **kw):
    d, hq = q.shape[2], q.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, lse = moe.kv_attention(q, pages, table.cuda(), i32(lens), page_size=ps, n_kv_heads=hkv, q_tokens=q_tokens,
                                window=window, scale=scale, return_lse=True, **kw)
    o, l, host = out.cpu().double(), lse.cpu().double(), pages.cpu()
    qd = q.cpu().double()
    for s, n in enumerate(lens):
        k, v = R.sequence(host, table[s], n, ps, hkv, d)
        rows = slice(s * q_tokens, (s + 1) * q_tokens)
        at = [n - q_tokens + j for j in range(q_tokens)]
        ro, rl, mag, z = R.attend(qd[rows], k, v, at, n, scale, window)
        tol = mag * (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -17 * z[..., None]) + R.EPS[q.dtype] * ro.abs() + 1e-30 + tiny
        err = (o[rows] - ro).abs()
        assert bool((err <= tol).all()), (s, n, float((err / tol).max()))
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(l[rows]) & (l[rows] < 0), empty)
        bad = (l[rows] - rl).abs()[~empty] > (2.0 ** -17 * z + 2.0 ** -20 * (1 + rl.abs()))[~empty]
        assert not bool(bad.any()), (s, n)
    return out, lse


# ------------------------------------------------------------------- append and read
@pytest.mark.parametrize("d,hq,hkv,rot,ps,dtype,inter,lens,starts", [
    (128, 16, 8, 128, 64, "bf16", False, [1], [0]),
    (128, 6, 2, 128, 32, "bf16", False, [1, 0, 3, 1], [31, 7, 62, 0]),
    (64, 3, 1, 32, 96, "f16", True, [5, 40], [94, 1]),
    (64, 1, 1, 64, 32, "f32", False, [33], [0]),
    (256, 5, 5, 256, 128, "f32", True, [2, 2], [127, 300]),
    (256, 4, 2, 128, 32, "bf16", False, [65, 1, 2], [0, 5, 31]),
    (128, 0, 3, 0, 64, "f16", False, [7], [60]),
    (64, 8, 4, 16, 32, "bf16", True, [0, 0, 9, 0], [0, 0, 0, 3])])
def test_append_writes_exactly_the_quantised_values(d, hq, hkv, rot, ps, dtype, inter, lens, starts):
    dt, T = DT[dtype], sum(lens)
    g = torch.Generator().manual_seed(d + T)
    heads = hq + 2 * hkv
    x = (torch.randn(T, heads, d, generator=g) * 2).to(dt)
    qkv = x.cuda()
    q, k, v = (qkv[:, :hq] if hq else None), qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    ends = [a + n for a, n in zip(starts, lens)]
    cos, sin = moe.rope_table(max(ends), rot, device="cpu") if rot else (None, None)
    n_pages = sum(-(-n // ps) for n in ends) + 1
    table = make_table(ends, ps, n_pages)
    before = torch.randint(0, 256, (n_pages, moe.kv_page_bytes(hkv, d, ps)), generator=g, dtype=torch.uint8)
    pages, status = before.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    rope = {} if not rot else dict(cos=cos.cuda(), sin=sin.cuda())
    qr, kr = moe.kv_append(pages, table.cuda(), i32(starts), i32(cu), k, v, page_size=ps, q=q, interleaved=inter,
                           status=status, **rope)
    kb, vb = moe.kv_read(pages, table.cuda(), i32(starts), i32(cu), T, page_size=ps, n_kv_heads=hkv, head_dim=d,
                         dtype=torch.float32, status=status)
    assert moe.status_message(status) == ""
    seq = [s for s, n in enumerate(lens) for _ in range(n)]
    pos = torch.tensor([starts[s] + j for s, n in enumerate(lens) for j in range(n)])
    k32 = x[:, hq:hq + hkv].float()
    if rot:
        k32 = R.rotate(k32, pos, cos, sin, inter, torch.float32)
        if hq:
            assert torch.equal(qr.cpu(), R.rotate(x[:, :hq].float(), pos, cos, sin, inter, torch.float32).to(dt))
    assert torch.equal(kr.cpu(), k32.to(dt))
    ref = R.Cache(n_pages, hkv, d, ps)
    ref.pages = before.clone()
    for value, src, back in ((0, k32, kb), (1, x[:, hq + hkv:].float(), vb)):
        codes, scales = R.quantise(src)
        for i in range(T):
            page = int(table[seq[i], int(pos[i]) // ps])
            for h in range(hkv):
                ref.put(page, int(pos[i]) % ps, h, value, codes[i, h], scales[i, h])
        assert torch.equal(back.cpu().double(), R.values(codes, scales))
    assert torch.equal(pages.cpu(), ref.pages)      # and nothing else was touched


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_read_rounds_to_each_type(dtype):
    pages, table = filled([70], 32, 2, 64, 3)
    a = moe.kv_read(pages, table.cuda(), i32([0]), i32([0, 70]), 70, page_size=32, n_kv_heads=2, head_dim=64,
                    dtype=torch.float32)
    b = moe.kv_read(pages, table.cuda(), i32([5]), i32([0, 60]), 60, page_size=32, n_kv_heads=2, head_dim=64,
                    dtype=DT[dtype])
    for x, y in zip(a, b):
        assert torch.equal(x[5:65].to(DT[dtype]), y)


def test_append_in_place_and_into_given_outputs():
    T, hq, hkv, d = 9, 4, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, hq, d, generator=g, device="cuda").bfloat16()
    k, v = [torch.randn(T, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    cos, sin = moe.rope_table(64, d)
    res = []
    for inplace in (False, True):
        pages = moe.kv_pages(1, hkv, d, 32)
        qq, kk = q.clone(), k.clone()
        kw = dict(q_out=qq, k_out=kk) if inplace else {}
        r = moe.kv_append(pages, i32([[0]]), i32([4]), i32([0, T]), kk, v, page_size=32, q=qq, cos=cos, sin=sin, **kw)
        if inplace:
            assert r[0] is qq and r[1] is kk
        res.append((r[0], r[1], pages))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_blocks_that_cannot_be_quantised():
    d, hkv = 64, 1
    x = torch.zeros(6, hkv, d)
    x[0, 0, 3] = float("nan")
    x[1, 0, 40] = float("-inf")
    x[2, 0] = 0.0
    x[3, 0, 7] = 1e-44                  # d underflows: codes of 8
    x[4, 0, :32] = 3e38                 # d past fp16: limited
    x[5, 0, 1], x[5, 0, 2] = -5.0, 5.0  # a tie takes the positive value
    pages = moe.kv_pages(1, hkv, d, 32)
    xd = x.cuda()
    moe.kv_append(pages, i32([[0]]), i32([0]), i32([0, 6]), xd, xd, page_size=32)
    k, v = moe.kv_read(pages, i32([[0]]), i32([0]), i32([0, 6]), 6, page_size=32, n_kv_heads=1, head_dim=d,
                       dtype=torch.float32)
    want = R.values(*R.quantise(x))
    for got in (k, v):
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.cpu().double()), torch.nan_to_num(want))
    assert float(k[5, 0, 2]) == 5.0 and float(k[5, 0, 1]) == -4.375
    assert float(k[4, 0, 0]) == 8 * 65504.0


def test_bad_pages_and_positions_are_reported_and_nothing_is_written():
    d, hkv, ps = 64, 2, 32
    x = torch.randn(6, hkv, d, device="cuda")
    cos, sin = moe.rope_table(40, d)
    for table, starts, cu, nmax, bit, dead in (
            ([[0, 9]], [30], [0, 6], 40, moe.MOE_KV_BAD_PAGE, [2, 3, 4, 5]),
            ([[0, -1]], [30], [0, 6], 40, moe.MOE_KV_BAD_PAGE, [2, 3, 4, 5]),
            ([[0]], [30], [0, 6], 40, moe.MOE_KV_BAD_PAGE, [2, 3, 4, 5]),
            ([[0, 1]], [36], [0, 6], 40, moe.MOE_KV_BAD_POSITION, [4, 5]),
            ([[0, 1]], [-1], [0, 6], 40, moe.MOE_KV_BAD_LENGTH, range(6)),
            ([[0, 1]], [0], [0, 4], 40, moe.MOE_KV_BAD_LENGTH, [4, 5]),
            ([[0], [1]], [0, 0], [3, 1, 6], 40, moe.MOE_KV_BAD_LENGTH, [0, 1, 2])):
        pages = moe.kv_pages(2, hkv, d, ps)
        pages.fill_(0xEE)
        status = i32([0])
        q, k = moe.kv_append(pages, i32(table), i32(starts), i32(cu), x, x, page_size=ps, q=x, cos=cos, sin=sin,
                             status=status)
        assert int(status) == bit, (table, starts)
        assert moe.status_message(status) != ""
        gone = torch.zeros(6, dtype=torch.bool)
        gone[list(dead)] = True
        if bit != moe.MOE_KV_BAD_PAGE:     # no place in the rotation table
            assert torch.equal(torch.isnan(q.cpu()).all(-1).all(-1), gone)
            assert torch.equal(torch.isnan(k.cpu()).all(-1).all(-1), gone)
        status.zero_()
        kb, vb = moe.kv_read(pages, i32(table), i32(starts), i32(cu), 6, page_size=ps, n_kv_heads=hkv, head_dim=d,
                             dtype=torch.float32, status=status)
        if bit != moe.MOE_KV_BAD_POSITION:
            assert int(status) == bit
            assert torch.equal(torch.isnan(kb.cpu()).all(-1).all(-1), gone)
        touched = (pages != 0xEE).any(0)
        held = 6 - len(list(dead))
        assert bool(touched.any()) == (held > 0)


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,ps,lens,q_tokens,window", [
    (8, 8, 32, [1], 1, 0),
    (4, 1, 64, [0, 1, 2, 31, 32, 33, 64, 100], 1, 0),
    (7, 1, 96, [500, 3], 1, 0),
    (16, 1, 32, [257], 1, 0),
    (6, 2, 64, [65, 200], 5, 0),
    (2, 2, 32, [3, 0, 40], 8, 0),
    (8, 2, 64, [1, 7, 300, 129], 1, 1),
    (8, 2, 32, [300, 64], 3, 33),
    (3, 3, 128, [1000], 1, 100)])
def test_attention(d, dtype, hq, hkv, ps, lens, q_tokens, window):
    pages, table = filled(lens, ps, hkv, d, 7)
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(len(lens) * q_tokens, hq, d, generator=g, device="cuda").to(DT[dtype])
    check(q, pages, table, lens, ps, hkv, q_tokens, window)


@pytest.mark.parametrize("lens", [[20000], [1, 9000, 0, 513, 4096], [64] * 300])
def test_attention_split_over_ctas(lens):
    pages, table = filled(lens, 64, 2, 128, 11)
    q = torch.randn(len(lens), 8, 128, device="cuda").bfloat16()
    a, la = check(q, pages, table, lens, 64, 2)
    for _ in range(3):     # the same bits whenever it runs
        b, lb = moe.kv_attention(q, pages, table.cuda(), i32(lens), page_size=64, n_kv_heads=2, return_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("d,hq,hkv,q_tokens", [(64, 8, 8, 1), (128, 16, 8, 1), (256, 16, 8, 2), (128, 24, 2, 1)])
@pytest.mark.parametrize("n,longest", [(2, 9000), (9, 8000), (70, 5000), (200, 700)])
def test_attention_of_ragged_batches(d, hq, hkv, q_tokens, n, longest):
    # pairs that begin, end and go on anywhere in the warps' and CTAs' shares; every row, against 64 bits on the GPU
    g = torch.Generator().manual_seed(n + d)
    lens = [int(x) for x in torch.randint(0, longest, (n,), generator=g)]
    lens[n // 2] = longest
    pages, table = filled(lens, 64, hkv, d, n)
    td, q = table.cuda(), torch.randn(n * q_tokens, hq, d, device="cuda").half()
    out = moe.kv_attention(q, pages, td, i32(lens), page_size=64, n_kv_heads=hkv, q_tokens=q_tokens)
    for s, m in enumerate(lens):
        k, v = [x.double().repeat_interleave(hq // hkv, 1) for x in moe.kv_read(
            pages, td[s:s + 1], i32([0]), i32([0, m]), m, page_size=64, n_kv_heads=hkv, head_dim=d, dtype=torch.float32)]
        rows = slice(s * q_tokens, (s + 1) * q_tokens)
        z = torch.einsum("rhd,nhd->hrn", q[rows].double(), k) * d ** -0.5
        at = m - q_tokens + torch.arange(q_tokens, device="cuda")
        z.masked_fill_(torch.arange(m, device="cuda") > at[None, :, None], -float("inf"))
        w = torch.nan_to_num(torch.softmax(z, -1)) if m else z
        ref, mag = torch.einsum("hrn,nhd->rhd", w, v), torch.einsum("hrn,nhd->rhd", w, v.abs())
        size = (torch.einsum("rhd,nhd->hrn", q[rows].double().abs(), k.abs()) * d ** -0.5).amax(-1).T[..., None] if m else 0.0
        tol = mag * (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -17 * size) + R.EPS[q.dtype] * ref.abs() + 1e-30
        assert bool(((out[rows].double() - ref).abs() <= tol).all()), (s, m)


@pytest.mark.parametrize("v_size", [1e-5, 1e-3, 300.0, 3e5])
@pytest.mark.parametrize("q_size", [1e-6, 1.0, 1e4])
def test_attention_over_far_apart_sizes(v_size, q_size):
    lens = [700, 45]
    pages, table = filled(lens, 32, 2, 128, 5, v_size=v_size)
    q = (torch.randn(2, 4, 128, device="cuda") * q_size).bfloat16()
    check(q, pages, table, lens, 32, 2, scale=0.08 / max(1.0, q_size))


def test_value_scales_that_grow_along_the_sequence():
    lens, hkv, d = [640], 1, 64
    pages, table = filled(lens, 32, hkv, d, 5)
    size = 2.0 ** (torch.arange(640, device="cuda") // 32 - 8.0)
    v = torch.randn(640, hkv, d, device="cuda") * size[:, None, None]
    moe.kv_append(pages, table.cuda(), i32([0]), i32([0, 640]), torch.randn_like(v), v, page_size=32)
    check(torch.randn(1, 4, d, device="cuda").half(), pages, table, lens, 32, hkv)


def test_one_score_far_above_the_others():
    lens, hkv, d = [333], 1, 128
    pages, table = filled(lens, 32, hkv, d, 5)
    q = torch.randn(1, 2, d, device="cuda").bfloat16() * 40     # softmax is nearly one key's
    top = float(R.sequence(pages.cpu(), table[0], 333, 32, hkv, d)[1].abs().max()) / 7     # no scale is larger
    check(q, pages, table, lens, 32, hkv, scale=1.0, tiny=333 * 8 * 2.0 ** -25 * (1 + top) * max(2.0 ** -7, top / 16))


def test_what_a_row_does_not_see_does_not_reach_it():
    ps, hkv, d, n = 32, 1, 64, 70
    pages, table = filled([n], ps, hkv, d, 9)
    q = torch.randn(2, 4, d, device="cuda").half()
    clean = moe.kv_attention(q, pages, table.cuda(), i32([n]), page_size=ps, n_kv_heads=hkv, q_tokens=2, window=20)
    # NaN and infinities before the window, after the sequence, and, for the first row, in the last token
    k, v = [torch.full((45, hkv, d), float("nan"), device="cuda") for _ in range(2)]
    moe.kv_append(pages, table.cuda(), i32([0]), i32([0, 45]), k, v, page_size=ps)
    got = moe.kv_attention(q, pages, table.cuda(), i32([n]), page_size=ps, n_kv_heads=hkv, q_tokens=2, window=20)
    assert torch.equal(got, clean)
    moe.kv_append(pages, table.cuda(), i32([n - 1]), i32([0, 1]), k[:1], v[:1], page_size=ps)
    got = moe.kv_attention(q, pages, table.cuda(), i32([n]), page_size=ps, n_kv_heads=hkv, q_tokens=2, window=20)
    assert torch.equal(got[0], clean[0]) and bool(torch.isnan(got[1]).all())


def test_a_nan_query_stays_in_its_row():
    pages, table = filled([100], 32, 1, 128, 2)
    q = torch.randn(1, 4, 128, device="cuda").bfloat16()
    clean = moe.kv_attention(q, pages, table.cuda(), i32([100]), page_size=32, n_kv_heads=1)
    q[0, 2, 5] = float("nan")
    got = moe.kv_attention(q, pages, table.cuda(), i32([100]), page_size=32, n_kv_heads=1)
    assert bool(torch.isnan(got[0, 2]).all())
    assert torch.equal(got[0, [0, 1, 3]], clean[0, [0, 1, 3]])


def test_bad_pages_and_lengths_give_nan_and_a_status():
    ps, hkv, d = 32, 2, 64
    lens = [100, 80, 90]
    pages, table = filled(lens, ps, hkv, d, 4)
    q = torch.randn(3, 4, d, device="cuda").bfloat16()
    clean = moe.kv_attention(q, pages, table.cuda(), i32(lens), page_size=ps, n_kv_heads=hkv)
    for entry in (-1, pages.shape[0], 2147483647, -2147483648):
        t2, status = table.clone(), i32([0])
        t2[1, 1] = entry
        got, lse = moe.kv_attention(q, pages, t2.cuda(), i32(lens), page_size=ps, n_kv_heads=hkv, status=status,
                                    return_lse=True)
        assert int(status) == moe.MOE_KV_BAD_PAGE
        assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(lse[1]).all())
        assert torch.equal(got[[0, 2]], clean[[0, 2]])
    for n in (-1, 129, 2147483647, -2147483648):
        status = i32([0])
        got = moe.kv_attention(q, pages, table.cuda(), i32([100, n, 90]), page_size=ps, n_kv_heads=hkv, status=status)
        assert int(status) == moe.MOE_KV_BAD_LENGTH
        assert bool(torch.isnan(got[1]).all())
        assert torch.equal(got[[0, 2]], clean[[0, 2]])


def test_strided_queries_and_pages():
    lens, ps, hkv, d = [77, 130], 64, 2, 128
    pages, table = filled(lens, ps, hkv, d, 6)
    wide = torch.zeros(pages.shape[0], pages.shape[1] + 4096, dtype=torch.uint8, device="cuda")
    wide[:, :pages.shape[1]] = pages
    fused = torch.randn(2, 12, d, device="cuda").bfloat16()
    a = moe.kv_attention(fused[:, :8].contiguous(), pages, table.cuda(), i32(lens), page_size=ps, n_kv_heads=hkv)
    b = moe.kv_attention(fused[:, :8], wide, table.cuda(), i32(lens), page_size=ps, n_kv_heads=hkv)
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # the last pages of a cache of more than 4 GiB
    hkv, d, ps = 8, 128, 64
    n_pages = (5 << 30) // moe.kv_page_bytes(hkv, d, ps)
    pages = torch.empty(n_pages, moe.kv_page_bytes(hkv, d, ps), dtype=torch.uint8, device="cuda")
    table = i32([[n_pages - 1, n_pages - 2]])
    k, v = [torch.randn(100, hkv, d, device="cuda") for _ in range(2)]
    small, st = moe.kv_pages(2, hkv, d, ps), i32([[1, 0]])
    res = []
    for p, t in ((pages, table), (small, st)):
        moe.kv_append(p, t, i32([0]), i32([0, 100]), k, v, page_size=ps)
        q = torch.ones(1, 16, d, device="cuda").bfloat16()
        res.append((moe.kv_attention(q, p, t, i32([100]), page_size=ps, n_kv_heads=hkv),
                    moe.kv_read(p, t, i32([0]), i32([0, 100]), 100, page_size=ps, n_kv_heads=hkv, head_dim=d)[1]))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_other_streams_and_graphs():
    lens, ps, hkv, d = [5000, 40], 64, 2, 128
    pages, table = filled(lens, ps, hkv, d, 8)
    td, ln = table.cuda(), i32(lens)
    q = torch.randn(2, 8, d, device="cuda").bfloat16()
    want = moe.kv_attention(q, pages, td, ln, page_size=ps, n_kv_heads=hkv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.kv_attention(q, pages, td, ln, page_size=ps, n_kv_heads=hkv, stream=side)
    raw = moe.kv_attention(q, pages, td, ln, page_size=ps, n_kv_heads=hkv, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)
    # a whole step in one graph: append a token, then attend, replayed with new inputs
    starts, cu = i32([4999, 39]), i32([0, 1, 2])
    k, v = [torch.randn(2, hkv, d, device="cuda").bfloat16() for _ in range(2)]
    cos, sin = moe.rope_table(5000, d)

    def step():
        qr, _ = moe.kv_append(pages, td, starts, cu, k, v, page_size=ps, q=q, cos=cos, sin=sin)
        return moe.kv_attention(qr, pages, td, ln, page_size=ps, n_kv_heads=hkv)
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = step()
    for _ in range(3):
        q.normal_()
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, step())


def test_python_refusals():
    pages, table = filled([40], 32, 2, 64, 1)
    t, q = table.cuda(), torch.zeros(1, 4, 64, device="cuda").bfloat16()
    ok = dict(page_size=32, n_kv_heads=2)
    for bad in (lambda: moe.kv_attention(q.float(), pages, t, i32([40]), **ok),
                lambda: moe.kv_attention(q.cpu(), pages, t, i32([40]), **ok),
                lambda: moe.kv_attention(q, pages, t, i32([40, 1]), **ok),
                lambda: moe.kv_attention(q, pages, t, torch.tensor([40], device="cuda"), **ok),
                lambda: moe.kv_attention(q[:, :3], pages, t, i32([40]), **ok),
                lambda: moe.kv_attention(q, pages, t, i32([40]), q_tokens=2, **ok),
                lambda: moe.kv_attention(q.transpose(1, 2), pages, t, i32([40]), **ok),
                lambda: moe.kv_attention(q, pages[:, :-16], t, i32([40]), **ok),
                lambda: moe.kv_attention(q, pages, t, i32([40]), out=torch.zeros(1, 4, 64, device="cuda"), **ok),
                lambda: moe.kv_attention(q, pages, t, i32([40]), window=-1, **ok),
                lambda: moe.kv_append(pages, t, i32([0]), i32([0, 1]), q[:, :2], q[:, :3], page_size=32),
                lambda: moe.kv_append(pages, t, i32([0]), i32([0, 1]), q[:, :2], q[:, :2].half(), page_size=32),
                lambda: moe.kv_append(pages, t, i32([0]), i32([0]), q[:, :2], q[:, :2], page_size=32),
                lambda: moe.kv_append(pages, t, i32([0]), i32([0, 1]), q[:, :2], q[:, :2], page_size=32,
                                      cos=torch.zeros(4, 32, device="cuda")),
                lambda: moe.kv_read(pages, t, i32([0]), i32([0, 1]), 1, page_size=32, n_kv_heads=2, head_dim=96)):
        with pytest.raises(moe.MoeError):
            bad()
    e = moe.kv_attention(q[:0], pages, t[:0], i32([]), **ok)
    assert e.shape == (0, 4, 64)
