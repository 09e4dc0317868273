"""Host-side checks of FP8, routing and the rows' way to experts (no GPU): pins of the oracle's functions
and every refusal of the C ABI before anything is launched."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import aaac_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_06_amd", "libaaac.so")

OK, INVALID, SHAPE, WS_SMALL = 0, 1, 2, 3
BF16, F16, F32, MXFP4, FP8 = 0, 1, 2, 3, 4
i64, vp = ctypes.c_int64, ctypes.c_void_p
FAKE = vp(1 << 20)                    # aligned; only ever passed to calls that must fail validation
OFF1, OFF2, OFF8 = vp((1 << 20) + 1), vp((1 << 20) + 2), vp((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libaaac.so is not built (python -m post_weight_quantization_06_amd.build)")
    L = ctypes.CDLL(LIB)
    L.aaac_last_error.restype = ctypes.c_char_p
    L.aaac_fp8_matmul_workspace_bytes.restype = ctypes.c_size_t
    L.aaac_fp8_matmul_workspace_bytes.argtypes = [i64] * 5 + [ctypes.c_int] * 2
    L.aaac_route_workspace_bytes.restype = ctypes.c_size_t
    L.aaac_route_workspace_bytes.argtypes = [i64, i64]
    return L


# ------------------------------------------------------------------ oracle pins

def test_e4m3_codes_are_torchs():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = ref.fp8_decode(np.arange(256, dtype=np.uint8)[None], np.ones((1, 2)))[0]
    assert np.array_equal(got, v, equal_nan=True)


@pytest.mark.parametrize("tile", [False, True])
def test_fp8_encode_is_torchs_rounding_of_the_quotient(tile):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(150, 300, generator=g) * torch.exp(3 * torch.randn(150, 1, generator=g))
    c, s = ref.fp8_encode(x.numpy(), tile)
    full = torch.from_numpy(ref._fp8_spread(s, 150, 300, tile))
    assert np.array_equal(c, (x / full).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # every block's largest element is its code 448, the scale its 448th part
    v = ref.fp8_decode(c, s, tile)
    assert abs(np.abs(v).max() - x.abs().max().item()) <= 2.0 ** -24 * x.abs().max().item()
    assert np.abs(v - x.double().numpy()).max() <= 2.0 ** -4 * x.abs().max().item()


def test_fp8_blocks_written_out():
    x = np.zeros((2, 130))
    x[0, :4] = [448, 17, 18.5, -0.001953125]     # 17: the tie of 16 and 18 goes to the even code
    x[0, 129], x[1, 0] = np.inf, 1e-45
    c, s = ref.fp8_encode(x)
    assert s[0, 0] == 1 and np.isnan(s[0, 1]) and s[1, 0] == np.float32(2.0 ** -126)
    assert ref.fp8_decode(c, s)[0, :5].tolist() == [448, 16, 18, -0.001953125, 0]
    assert (c[0, 128:] == 0x7f).all() and (c[1] == 0).all()


def test_route_written_out():
    l = np.log(np.array([[1, 2, 4, 1, 8, 0.5], [4, 4, 4, 4, 4, 4]]))
    e, w, off, rows, places = ref.route(l, 2)
    assert e.tolist() == [[4, 2], [0, 1]] and np.allclose(w, [[8 / 12, 4 / 12], [0.5, 0.5]])
    assert off.tolist() == [0, 1, 2, 3, 3, 4, 4] and rows.tolist() == [1, 1, 0, 0]
    assert places.tolist() == [[3, 2], [0, 1]]
    e, w = ref.route(l, 2, renormalize=False, scale=2.0)[:2]
    assert np.allclose(w[0], [16 / 16.5, 8 / 16.5]) and np.allclose(w[1], 2 / 6)
    # groups of two: sums 3, 5, 8.5; the best group alone, or the two best
    assert ref.route(l, 2, groups=3, top_groups=1, group_top=2)[0][0].tolist() == [4, 5]
    assert ref.route(l, 2, groups=3, top_groups=2, group_top=1)[0].tolist() == [[4, 2], [0, 1]]
    bias = np.array([9.0, 0, 0, 0, -np.inf, 0])
    e, w = ref.route(l, 3, score="sigmoid", bias=bias)[:2]
    s = 1 / (1 + np.exp(-l))
    assert e[0].tolist() == [0, 2, 1] and np.allclose(w[0], s[0, [0, 2, 1]] / s[0, [0, 2, 1]].sum())
    l[0], l[1, 1:] = -np.inf, -np.inf
    e, w, off, rows, places = ref.route(l, 2)
    assert e.tolist() == [[-1, -1], [0, -1]] and w.tolist() == [[0, 0], [1, 0]]
    assert off.tolist() == [0] + [1] * 6 and rows.tolist() == [1, -1, -1, -1]
    assert places.tolist() == [[-1, -1], [0, -1]]


# ------------------------------------------------------------------ refusals

def _quant(L, X=FAKE, xt=BF16, E=1, M=4, C=200, ldx=200, step=800, tile=0, codes=FAKE, ldq=208, s=FAKE):
    return L.aaac_fp8_quantize(X, xt, i64(E), i64(M), i64(C), i64(ldx), i64(step), tile, codes, i64(ldq),
                               s, None)


def test_quantize_refusals(lib):
    assert _quant(lib, M=0, X=None, codes=None, s=None) == OK
    for bad in (dict(E=0), dict(E=2), dict(M=-1), dict(C=0), dict(C=1 << 21, ldx=1 << 21, ldq=1 << 21),
                dict(ldx=199), dict(ldq=192), dict(ldq=201), dict(M=1 << 35), dict(ldx=1 << 59),
                dict(E=2, tile=1, step=799)):
        assert _quant(lib, **bad) == SHAPE, bad
    for bad in (dict(X=None), dict(X=OFF1), dict(codes=None), dict(codes=OFF8), dict(s=None), dict(s=OFF2),
                dict(xt=MXFP4), dict(xt=FP8), dict(tile=2), dict(xt=F32, X=OFF2)):
        assert _quant(lib, **bad) == INVALID, bad
    assert b"aaac_fp8_quantize" in lib.aaac_last_error()


def _dequant(L, codes=FAKE, ldq=200, s=FAKE, E=1, M=4, C=200, tile=0, Y=FAKE, yt=F32, ldy=200):
    return L.aaac_fp8_dequant(codes, i64(ldq), s, i64(E), i64(M), i64(C), tile, Y, yt, i64(ldy), None)


def test_dequant_refusals(lib):
    assert _dequant(lib, M=0, Y=None, codes=None, s=None) == OK
    for bad in (dict(ldq=199), dict(ldy=199), dict(M=-1), dict(E=2), dict(C=0)):
        assert _dequant(lib, **bad) == SHAPE, bad
    for bad in (dict(Y=None), dict(Y=OFF2), dict(codes=None), dict(s=OFF2), dict(yt=FP8), dict(tile=-1)):
        assert _dequant(lib, **bad) == INVALID, bad


def _mm(L, w=FAKE, ldw=208, ws_=FAKE, E=1, R=64, C=200, off=None, rows=None, x=FAKE, xt=FP8, xs=FAKE, Tx=4,
        ldx=208, T=4, y=FAKE, yt=F32, ldy=64, work=None, nwork=0):
    return L.aaac_fp8_matmul(w, i64(ldw), ws_, i64(E), i64(R), i64(C), off, rows, x, xt, xs, i64(Tx),
                             i64(ldx), i64(T), y, yt, i64(ldy), work, ctypes.c_size_t(nwork), None)


def test_product_refusals(lib):
    assert _mm(lib, T=0, Tx=0, x=None, y=None, xs=None) == OK
    assert _mm(lib, T=0, rows=FAKE, y=None) == OK
    for bad in (dict(E=0), dict(E=65536, off=FAKE), dict(R=0), dict(C=0), dict(C=1 << 21), dict(T=-1, Tx=-1),
                dict(Tx=5), dict(ldw=192), dict(ldw=200), dict(ldw=1 << 22), dict(ldx=192), dict(ldx=200),
                dict(ldx=1 << 22), dict(ldy=63), dict(R=1 << 31, ldy=1 << 31), dict(T=1 << 31, Tx=1 << 31),
                dict(R=1 << 30, ldy=1 << 30, T=1 << 30, Tx=1 << 30),
                dict(rows=FAKE, Tx=1 << 24), dict(rows=FAKE, Tx=-1)):
        assert _mm(lib, **bad) == SHAPE, bad
    for bad in (dict(E=2), dict(off=OFF2), dict(rows=OFF2), dict(w=None), dict(w=OFF8), dict(ws_=None),
                dict(ws_=OFF2), dict(x=None), dict(x=OFF8), dict(xs=None), dict(xs=OFF2), dict(y=None),
                dict(y=OFF2), dict(yt=FP8), dict(xt=MXFP4), dict(xt=7), dict(xt=BF16, ldx=200),
                dict(xt=BF16, xs=None, C=2200, ldw=2208, ldx=2200, T=40, Tx=40), dict(xt=F32, xs=None, ldx=200, x=OFF2)):
        assert _mm(lib, **bad) == INVALID, bad
    assert _mm(lib, xt=BF16, xs=None, ldx=199, work=FAKE, nwork=1 << 20) == SHAPE


def test_product_workspaces_and_plans(lib):
    need = lib.aaac_fp8_matmul_workspace_bytes
    for bad in ((0, 16, 64, 4, 4), (1, 0, 64, 4, 4), (1, 16, 0, 4, 4), (1, 16, 64, 0, 0), (1, 16, 64, 4, -1),
                (1, 16, 1 << 21, 4, 4), (65536, 16, 64, 4, 4)):
        assert need(*bad, 1, BF16) == 0
    assert need(1, 16, 64, 4, 4, 0, BF16) == need(1, 16, 64, 400, 400, 1, FP8) == 0
    assert need(1, 64, 200, 4, 4, 1, BF16) == 0        # few rows are quantized by the product itself
    n = need(1, 64, 2200, 40, 40, 1, BF16)
    assert n >= 40 * (2304 + 72)                 # codes of whole blocks and their scales
    assert need(1, 64, 2200, 40, 90, 1, BF16) > n      # of the rows of x
    args = dict(xt=BF16, xs=None, C=2200, ldw=2208, ldx=2200, T=40, Tx=40)
    assert _mm(lib, work=FAKE, nwork=n - 1, **args) == WS_SMALL
    assert _mm(lib, work=vp((1 << 20) + 128), nwork=n, **args) == INVALID
    split = need(1, 1024, 8192, 256, 256, 0, BF16)
    assert split >= 2 * 256 * 1024 * 4
    plan = (ctypes.c_int32 * 6)()
    f = lib.aaac_fp8_matmul_plan
    assert f(i64(1), i64(1024), i64(8192), i64(256), BF16, 1, plan) == OK and plan[2] > 1
    assert f(i64(1), i64(1024), i64(8192), i64(256), BF16, 0, plan) == OK and plan[2] == 1
    assert f(i64(1), i64(16), i64(64), i64(4), BF16, 1, plan) == OK and list(plan[:2]) == [0, 0]
    assert f(i64(1), i64(16), i64(64), i64(4), BF16, 1, None) == INVALID
    assert f(i64(1), i64(16), i64(64), i64(0), BF16, 1, plan) == SHAPE
    assert f(i64(1), i64(16), i64(64), i64(4), FP8, 1, plan) == INVALID


def test_queries_of_weights_past_2_to_40(lib):
    """The products refuse E * R * C of 2^40 and more, so the queries do: no bytes and no plan."""
    plan = (ctypes.c_int32 * 6)()
    for E, R, C in ((65535, (1 << 31) - 1, (1 << 21) - 1), (1, 1 << 30, 1024), (65535, (1 << 13) + 1, 1 << 11)):
        for T in (4, 40, 4000):
            for yt in (BF16, F32):
                assert lib.aaac_fp8_matmul_workspace_bytes(E, R, C, T, T, 1, yt) == 0
                assert lib.aaac_fp8_matmul_plan(i64(E), i64(R), i64(C), i64(T), yt, 1, plan) == SHAPE
        assert _mm(lib, E=E, R=R, C=C, ldw=1 << 21, ldx=1 << 21, ldy=R, off=FAKE) == SHAPE
    assert lib.aaac_fp8_matmul_plan(i64(1), i64(1 << 30), i64(896), i64(4), BF16, 1, plan) == OK


@pytest.mark.parametrize("E,R,C,T", [(1, 4096, 4096, 100), (1, 70, 2200, 33), (1, 1024, 8192, 256),
                                     (8, 1500, 1031, 500), (1, 4000, 896, 2000), (1, 16, 64, 4)])
def test_an_x_without_rows_needs_no_workspace(lib, E, R, C, T):
    """Such a product runs without parts and without quantized rows, also where one with rows is split or
    quantizes them first: the tiles, which take no empty x, are not chosen."""
    for yt in (BF16, F16, F32):
        for quantize in (0, 1):
            assert lib.aaac_fp8_matmul_workspace_bytes(E, R, C, T, 0, quantize, yt) == 0


def _route(L, x=FAKE, xt=F32, T=4, E=64, ldl=64, bias=None, score=0, k=4, groups=1, top=1, gt=1, e=FAKE,
           w=FAKE, off=FAKE, rows=FAKE, places=FAKE, work=None, nwork=0):
    return L.aaac_route(x, xt, i64(T), i64(E), i64(ldl), bias, score, i64(k), groups, top, gt, 1,
                        ctypes.c_float(1.0), e, w, off, rows, places, work, ctypes.c_size_t(nwork), None)


def test_route_refusals(lib):
    for bad in (dict(E=0), dict(E=513, ldl=513), dict(k=0), dict(k=65), dict(E=3, k=4), dict(groups=0),
                dict(groups=65), dict(groups=3), dict(groups=8, top=0), dict(groups=8, top=9),
                dict(groups=8, top=1, k=9), dict(gt=0), dict(gt=3), dict(T=-1), dict(T=1 << 30, k=2),
                dict(ldl=63)):
        assert _route(lib, **bad) == SHAPE, bad
    for bad in (dict(x=None), dict(x=OFF2), dict(xt=FP8), dict(score=2), dict(bias=OFF2), dict(e=None),
                dict(w=None), dict(off=None), dict(rows=None), dict(places=None), dict(e=OFF2),
                dict(w=OFF2), dict(off=OFF2), dict(rows=OFF2), dict(places=OFF2), dict(T=1000)):
        assert _route(lib, **bad) == INVALID, bad
    n = lib.aaac_route_workspace_bytes(1000, 64)
    assert n > 0 and _route(lib, T=1000, work=FAKE, nwork=n - 1) == WS_SMALL
    assert _route(lib, T=1000, work=OFF8, nwork=n) == INVALID
    assert lib.aaac_route_workspace_bytes(1, 64) == 0
    for bad in ((0, 64), (-1, 64), (5, 0), (5, 513), (1 << 31, 4)):
        assert lib.aaac_route_workspace_bytes(*bad) == 0


def _to(L, x=FAKE, el=2, T=4, C=64, ldx=64, places=FAKE, k=2, out=FAKE, N=8, ldo=64):
    return L.aaac_rows_to_experts(x, el, i64(T), i64(C), i64(ldx), places, i64(k), out, i64(N), i64(ldo), None)


def _from(L, y=FAKE, yt=BF16, N=8, C=64, ldy=64, places=FAKE, w=FAKE, T=4, k=2, out=FAKE, ot=BF16, ldo=64):
    return L.aaac_rows_from_experts(y, yt, i64(N), i64(C), i64(ldy), places, w, i64(T), i64(k), out, ot,
                                    i64(ldo), None)


def test_rows_refusals(lib):
    assert _to(lib, T=0, x=None, places=None, out=None) == OK and _to(lib, N=0, out=None) == OK
    assert _from(lib, T=0, y=None, places=None, w=None, out=None) == OK
    sizes = (dict(T=-1), dict(T=1 << 31), dict(N=-1), dict(N=1 << 31), dict(C=0), dict(k=0), dict(k=65),
             dict(ldo=63), dict(C=1 << 31))
    for bad in sizes + (dict(ldx=63),):
        assert _to(lib, **bad) == SHAPE, bad
    for bad in sizes + (dict(ldy=63),):
        assert _from(lib, **bad) == SHAPE, bad
    for bad in (dict(el=0), dict(el=8), dict(x=None), dict(x=OFF1), dict(out=None), dict(out=OFF1),
                dict(places=None), dict(places=OFF2)):
        assert _to(lib, **bad) == INVALID, bad
    for bad in (dict(y=None), dict(y=OFF1), dict(yt=FP8), dict(ot=FP8), dict(out=None), dict(out=OFF1),
                dict(places=None), dict(w=None), dict(w=OFF2), dict(ot=F32, out=OFF2)):
        assert _from(lib, **bad) == INVALID, bad
