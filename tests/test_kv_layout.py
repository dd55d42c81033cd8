"""The paged cache's index arithmetic and every check of device-side numbers, on the
CPU: the header the kernels use, compiled with g++ (the kernels touch memory only
where these functions say so), and the entry points' refusals."""
import ctypes
import os
import subprocess

import pytest

import router_softmax_top_gb300 as moe
from router_softmax_top_gb300 import attention as A
from router_softmax_top_gb300 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER_DIR = os.path.join(ROOT, "router_softmax_top_gb300", "csrc")
WRAPPER = r'''
#include "kv_layout.h"
using namespace moe;
extern "C" {
int tile_bytes(int D) { return kv_tile_bytes(D); }
int code_off(int D, int v, int b, int t) { return kv_code_off(D, v, b, t); }
int scale_off(int D, int v, int b, int t) { return kv_scale_off(D, v, b, t); }
int64_t tile_off(int D, int ps, int h, int i) { return kv_tile_off(D, ps, h, i); }
int page(const int32_t *row, int w, int n, int ps, int64_t tile, int *in) { return kv_page(row, w, n, ps, tile, in); }
int64_t position(int64_t i, int64_t lo, int64_t hi, int64_t s) { return kv_position(i, lo, hi, s); }
void visible(int64_t len, int q, int j, int w, int64_t *lo, int64_t *hi) { kv_visible(len, q, j, w, lo, hi); }
int64_t tiles(int64_t len, int q, int w, int width, int ps, int64_t *f) { return kv_tiles(len, q, w, width, ps, f); }
}
'''


@pytest.fixture(scope="module")
def kv(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv")
    (d / "w.cpp").write_text(WRAPPER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", HEADER_DIR, "-o", str(d / "w.so"),
                    str(d / "w.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "w.so"))
    i64, pi64 = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    lib.tile_off.restype = lib.position.restype = lib.tiles.restype = i64
    lib.position.argtypes = [i64] * 4
    lib.page.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, ctypes.POINTER(ctypes.c_int)]
    lib.visible.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, pi64, pi64]
    lib.tiles.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, pi64]
    return lib


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_byte_of_a_tile_has_one_owner(kv, D):
    owner = [0] * kv.tile_bytes(D)
    for value in (0, 1):
        for tok in range(32):
            for b in range(D // 32):
                at, sc = kv.code_off(D, value, b, tok), kv.scale_off(D, value, b, tok)
                assert at % 16 == 0 and sc % 2 == 0
                for x in list(range(at, at + 16)) + [sc, sc + 1]:
                    owner[x] += 1
    assert owner == [1] * (36 * D)


@pytest.mark.parametrize("ps", [32, 96, 256])
def test_tiles_fill_a_page(kv, ps):
    offs = sorted(kv.tile_off(128, ps, h, i) for h in range(3) for i in range(ps // 32))
    assert offs == [x * 36 * 128 for x in range(3 * ps // 32)]
    # a tile of a far head stays exact past 2^31 bytes
    assert kv.tile_off(256, 65536, 1023, 2047) == (1023 * 2048 + 2047) * 36 * 256


def test_page_lookup_never_leaves_table_or_cache(kv):
    row = (ctypes.c_int32 * 6)(2, 0, -1, 5, 2147483647, -2147483648)
    n = ctypes.c_int()
    for ps in (32, 64, 96):
        per = ps // 32
        for tile in range(-3, 8 * per):
            p = kv.page(row, 4, 5, ps, tile, ctypes.byref(n))    # width 4: the last two entries are never read
            i = tile // per if tile >= 0 else -1
            want = row[i] if 0 <= i < 4 and 0 <= row[i] < 5 else -1
            assert p == want, (ps, tile)
            if p >= 0:
                assert n.value == tile % per
    assert kv.page(row, 6, 5, 32, 4, ctypes.byref(n)) == -1
    assert kv.page(row, 6, 5, 32, 5, ctypes.byref(n)) == -1
    assert kv.page(row, 0, 5, 32, 0, ctypes.byref(n)) == -1
    assert kv.page(row, 4, 5, 32, 1 << 40, ctypes.byref(n)) == -1


def test_positions(kv):
    assert kv.position(5, 3, 9, 100) == 102
    assert kv.position(2, 3, 9, 100) == -1       # before the sequence: offsets that decrease
    assert kv.position(9, 3, 9, 100) == -1
    assert kv.position(5, 3, 9, -1) == -1
    assert kv.position(0, 0, 1, 2147483647) == 2147483647


def test_visible_ranges_against_counting(kv):
    lo, hi, first = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    for length in (0, 1, 2, 31, 32, 33, 64, 97):
        for q in (1, 2, 5, 40):
            for w in (0, 1, 3, 32, 33, 1000):
                seen_any = set()
                for j in range(q):
                    p = length - q + j
                    seen = [k for k in range(length) if k <= p and (w == 0 or k > p - w)]
                    kv.visible(length, q, j, w, ctypes.byref(lo), ctypes.byref(hi))
                    assert list(range(lo.value, hi.value)) == seen, (length, q, w, j)
                    seen_any.update(seen)
                n = kv.tiles(length, q, w, 4, 32, ctypes.byref(first))
                if length > 128:
                    assert n == -1
                    continue
                assert n >= 0
                assert all(first.value <= k // 32 < first.value + n for k in seen_any)
                if seen_any:
                    assert first.value == min(seen_any) // 32
    assert kv.tiles(-1, 1, 0, 4, 32, ctypes.byref(first)) == -1
    assert kv.tiles(129, 1, 0, 4, 32, ctypes.byref(first)) == -1
    assert kv.tiles(1, 1, 0, 0, 32, ctypes.byref(first)) == -1
    assert kv.tiles(2147483647, 1, 0, 4, 32, ctypes.byref(first)) == -1


# ------------------------------------------------------------------- refusals (no GPU is touched)
@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return A._lib()


def _cache(**kw):
    c = dict(pages=1 << 20, page_stride=8 * 2 * 36 * 128, page_table=1 << 20, table_stride=4, status=0, n_pages=3,
             page_size=64, n_kv_heads=8, head_dim=128, n_seqs=2, table_width=4)
    c.update(kw)
    return A.MoeKvCache(*[c[f] for f, _ in A.MoeKvCache._fields_])


BAD_CACHES = [
    (dict(head_dim=96), moe.MOE_ERR_UNSUPPORTED), (dict(page_size=48), moe.MOE_ERR_UNSUPPORTED),
    (dict(page_size=0), moe.MOE_ERR_INVALID_ARG), (dict(n_kv_heads=0), moe.MOE_ERR_INVALID_ARG),
    (dict(pages=(1 << 20) + 8), moe.MOE_ERR_INVALID_ARG), (dict(pages=0), moe.MOE_ERR_INVALID_ARG),
    (dict(page_stride=8 * 2 * 36 * 128 - 16), moe.MOE_ERR_INVALID_ARG),
    (dict(page_stride=8 * 2 * 36 * 128 + 8), moe.MOE_ERR_INVALID_ARG),
    (dict(page_table=0), moe.MOE_ERR_INVALID_ARG), (dict(table_stride=3), moe.MOE_ERR_INVALID_ARG),
    (dict(n_seqs=-1), moe.MOE_ERR_INVALID_ARG), (dict(n_pages=-1), moe.MOE_ERR_INVALID_ARG),
]


def _calls(lib, c, **kw):
    a = dict(starts=1 << 20, cu=1 << 20, n=2, q=A.MoeTensor(1 << 20, 2048, 128), hq=16, k=A.MoeTensor(1 << 20, 1024, 128),
             v=A.MoeTensor(1 << 20, 1024, 128), cos=1 << 20, sin=1 << 20, rot=128, n_pos=10, q_out=1 << 20, k_out=1 << 20,
             dtype=1)
    a.update(kw)
    return lib.moe_kv_append(ctypes.byref(c), a["starts"], a["cu"], a["n"], ctypes.byref(a["q"]), a["hq"],
                             ctypes.byref(a["k"]), ctypes.byref(a["v"]), a["cos"], a["sin"], a["rot"], a["n_pos"], 0,
                             a["q_out"], a["k_out"], a["dtype"], None)


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, code):
    c = _cache(**change)
    assert _calls(lib, c) == code
    assert lib.moe_kv_read(ctypes.byref(c), 1 << 20, 1 << 20, 2, 1 << 20, 1 << 20, 1, None) == code
    q = A.MoeTensor(1 << 20, 2048, 128)
    assert lib.moe_kv_attention(ctypes.byref(c), 1 << 20, ctypes.byref(q), 16, 1, 1.0, 0, 1 << 20, None, 1, 1 << 20,
                                1 << 30, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(rot=24), moe.MOE_ERR_INVALID_ARG), (dict(rot=144), moe.MOE_ERR_INVALID_ARG), (dict(rot=-16), moe.MOE_ERR_INVALID_ARG),
    (dict(cos=0), moe.MOE_ERR_INVALID_ARG), (dict(sin=(1 << 20) + 4), moe.MOE_ERR_INVALID_ARG),
    (dict(n_pos=0), moe.MOE_ERR_INVALID_ARG), (dict(n=-1), moe.MOE_ERR_INVALID_ARG), (dict(starts=0), moe.MOE_ERR_INVALID_ARG),
    (dict(cu=0), moe.MOE_ERR_INVALID_ARG), (dict(dtype=3), moe.MOE_ERR_INVALID_ARG), (dict(hq=0), moe.MOE_ERR_INVALID_ARG),
    (dict(q_out=0), moe.MOE_ERR_INVALID_ARG), (dict(k_out=(1 << 20) + 2), moe.MOE_ERR_INVALID_ARG),
    (dict(k=A.MoeTensor(0, 1024, 128)), moe.MOE_ERR_INVALID_ARG),
    (dict(k=A.MoeTensor((1 << 20) + 2, 1024, 128)), moe.MOE_ERR_UNSUPPORTED),
    (dict(v=A.MoeTensor(1 << 20, 1025, 128)), moe.MOE_ERR_UNSUPPORTED),
    (dict(q=A.MoeTensor(1 << 20, 2048, 129)), moe.MOE_ERR_UNSUPPORTED)])
def test_bad_appends_are_refused(lib, change, code):
    assert _calls(lib, _cache(), **change) == code


def test_append_of_nothing_is_a_no_op(lib):
    assert _calls(lib, _cache(), n=0) == moe.MOE_OK


@pytest.mark.parametrize("change,code", [
    (dict(hq=12), moe.MOE_ERR_INVALID_ARG), (dict(hq=0), moe.MOE_ERR_INVALID_ARG), (dict(qt=0), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=0.0), moe.MOE_ERR_INVALID_ARG), (dict(scale=-0.1), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), moe.MOE_ERR_INVALID_ARG), (dict(scale=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(window=-1), moe.MOE_ERR_INVALID_ARG), (dict(dtype=0), moe.MOE_ERR_UNSUPPORTED), (dict(lens=0), moe.MOE_ERR_INVALID_ARG),
    (dict(out=0), moe.MOE_ERR_INVALID_ARG), (dict(ws=0), moe.MOE_ERR_INVALID_ARG), (dict(ws=(1 << 20) + 16), moe.MOE_ERR_INVALID_ARG),
    (dict(ws_bytes=4096), moe.MOE_ERR_INVALID_ARG), (dict(qt=1025), moe.MOE_ERR_UNSUPPORTED),
    (dict(q=A.MoeTensor((1 << 20) + 2, 2048, 128)), moe.MOE_ERR_UNSUPPORTED),
    (dict(q=A.MoeTensor(0, 2048, 128)), moe.MOE_ERR_INVALID_ARG)])
def test_bad_attention_calls_are_refused(lib, change, code):
    a = dict(lens=1 << 20, q=A.MoeTensor(1 << 20, 2048, 128), hq=16, qt=1, window=0, out=1 << 20, dtype=1, ws=1 << 20,
             ws_bytes=1 << 30, scale=1.0)
    a.update(change)
    rc = lib.moe_kv_attention(ctypes.byref(_cache()), a["lens"], ctypes.byref(a["q"]), a["hq"], a["qt"], a["scale"], a["window"],
                              a["out"], None, a["dtype"], a["ws"], a["ws_bytes"], None)
    assert rc == code


def _prompt(lib, **kw):
    a = dict(q=A.MoeTensor(1 << 20, 2048, 128), nq=5, hq=16, k=A.MoeTensor(1 << 20, 1024, 128),
             v=A.MoeTensor(1 << 20, 1024, 128), nk=5, hkv=8, d=128, cq=1 << 20, ck=1 << 20, n=2, scale=0.1, window=0,
             out=1 << 20, dtype=1)
    a.update(kw)
    return lib.moe_prompt_attention(ctypes.byref(a["q"]), a["nq"], a["hq"], ctypes.byref(a["k"]), ctypes.byref(a["v"]),
                                    a["nk"], a["hkv"], a["d"], a["cq"], a["ck"], a["n"], a["scale"], a["window"], a["out"],
                                    None, a["dtype"], None, None)


@pytest.mark.parametrize("change,code", [
    (dict(hq=12), moe.MOE_ERR_INVALID_ARG), (dict(hkv=0), moe.MOE_ERR_INVALID_ARG), (dict(d=96), moe.MOE_ERR_UNSUPPORTED),
    (dict(nq=-1), moe.MOE_ERR_INVALID_ARG), (dict(nk=-1), moe.MOE_ERR_INVALID_ARG), (dict(n=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(window=-1), moe.MOE_ERR_INVALID_ARG), (dict(dtype=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(scale=0.0), moe.MOE_ERR_INVALID_ARG), (dict(scale=-1.0), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), moe.MOE_ERR_INVALID_ARG), (dict(scale=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(cq=0), moe.MOE_ERR_INVALID_ARG), (dict(ck=0), moe.MOE_ERR_INVALID_ARG), (dict(out=0), moe.MOE_ERR_INVALID_ARG),
    (dict(out=(1 << 20) + 2), moe.MOE_ERR_INVALID_ARG), (dict(hq=65, hkv=1), moe.MOE_ERR_UNSUPPORTED),
    (dict(nq=1 << 30), moe.MOE_ERR_UNSUPPORTED), (dict(q=A.MoeTensor((1 << 20) + 2, 2048, 128)), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=A.MoeTensor(1 << 20, 1025, 128)), moe.MOE_ERR_UNSUPPORTED),
    (dict(v=A.MoeTensor(0, 1024, 128)), moe.MOE_ERR_INVALID_ARG)])
def test_bad_prompt_calls_are_refused(lib, change, code):
    assert _prompt(lib, **change) == code


def test_prompt_workspaces(lib):
    t = ctypes.byref(A.MoeTensor(1 << 20, 2048, 128))
    rc = lib.moe_prompt_attention_shared(t, 5, 16, t, t, 5000, 8, 128, 1 << 20, 1 << 20, 1, 0.1, 0, 1 << 20, None, 1, None,
                                         (1 << 20) + 64, 1 << 30, None)
    assert rc == moe.MOE_ERR_INVALID_ARG      # not 256-byte aligned
    for bad in ((0, 8, 5000, 8, 128, 1, 0), (5, 8, 5000, 0, 128, 1, 0), (5, 12, 5000, 8, 128, 1, 0), (5, 8, 5000, 8, 96, 1, 0),
                (5, 8, 5000, 8, 128, 0, 0), (5, 8, 5000, 8, 128, 1, -1), (5, 8, 0, 8, 128, 1, 0), (5, 65, 5000, 1, 128, 1, 0)):
        assert lib.moe_prompt_attention_workspace(*bad) == 0


def test_prompt_of_nothing_is_a_no_op(lib):
    assert _prompt(lib, nq=0) == moe.MOE_OK
    assert _prompt(lib, n=0) == moe.MOE_OK


def test_sizes(lib):
    assert moe.kv_page_bytes(8, 128, 64) == 8 * 64 * 128 * 36 // 32
    for bad in ((0, 128, 64), (8, 96, 64), (8, 128, 16), (8, 128, 0)):
        with pytest.raises(moe.MoeError) as e:
            moe.kv_page_bytes(*bad)
        assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_kv_attention_workspace(16, 8, 128, 1) > 0
    assert lib.moe_kv_attention_workspace(15, 8, 128, 1) == 0


def test_struct_layouts_match_header(tmp_path):
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include "moe_attention.h"\nint main(void) { printf("%zu %zu %zu %zu %zu\\n", '
                   'sizeof(moe_kv_cache), offsetof(moe_kv_cache, status), offsetof(moe_kv_cache, n_pages), '
                   'offsetof(moe_kv_cache, table_width), sizeof(moe_tensor)); return 0; }')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    c = A.MoeKvCache
    assert got == [ctypes.sizeof(c), c.status.offset, c.n_pages.offset, c.table_width.offset, ctypes.sizeof(A.MoeTensor)]
