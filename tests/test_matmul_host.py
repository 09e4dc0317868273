"""Host-side checks of MXFP4 and the products on 4-bit weights (no GPU): pins of the oracle's MXFP4
functions and every refusal of the C ABI and the binding before anything is launched."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import aaac_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_06_amd", "libaaac.so")

OK, INVALID, SHAPE, WS_SMALL = 0, 1, 2, 3
BF16, F16, F32, MXFP4 = 0, 1, 2, 3
PACKED, MX, MX_X, MX_QUANTIZE = 0, 1, 2, 3
i64 = ctypes.c_int64
FAKE = ctypes.c_void_p(1 << 20)       # aligned; only ever passed to calls that must fail validation
OFF2 = ctypes.c_void_p((1 << 20) + 2)
OFF8 = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libaaac.so is not built (python -m post_weight_quantization_06_amd.build)")
    L = ctypes.CDLL(LIB)
    L.aaac_last_error.restype = ctypes.c_char_p
    L.aaac_matmul_workspace_bytes.restype = ctypes.c_size_t
    L.aaac_matmul_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i64, i64]
    return L


# ------------------------------------------------------------------ oracle pins

def test_e2m1_codes_of_a_block_written_out():
    # top = 6 -> e = 0: every value is its own code; halves between neighbours go to the even code
    x = np.array([[0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6, -0.25, -0.75, -6, 1, 3]])
    codes, byte = ref.mxfp4_encode(np.concatenate([x, np.zeros((1, 16))], axis=1))
    want = [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 8, 10, 15, 2, 5]
    assert codes[0, :16].tolist() == want and byte.tolist() == [[127]]


@pytest.mark.parametrize("top,e", [(4.0, 0), (7.99, 0), (8.0, 1), (3.99, -1), (2.0 ** 127, 125),
                                   (2.0 ** -125, -127), (2.0 ** -140, -127), (0.0, -127)])
def test_scale_exponent(top, e):
    x = np.zeros((1, 32))
    x[0, 5] = top
    codes, byte = ref.mxfp4_encode(x)
    assert byte[0, 0] == e + 127
    v = ref.mxfp4_decode(codes, byte, 32)[0, 5]
    # magnitudes in (6, 8) times 2^e saturate at 6; below 2^-127 / 4 they vanish
    assert v == (6.0 * 2.0 ** e if top * 2.0 ** -e > 5 else
                 4.0 * 2.0 ** e if top * 2.0 ** -e >= 4 else v)


def test_blocks_with_infinities_and_nan_read_back_as_nan():
    x = np.ones((2, 70))
    x[0, 3], x[1, 69] = np.inf, np.nan
    codes, byte = ref.mxfp4_encode(x)
    assert byte.tolist() == [[255, 125, 125], [125, 125, 255]]
    v = ref.mxfp4_decode(codes, byte, 70)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all() and np.isnan(v[1, 64:]).all()


def test_encode_is_idempotent_and_within_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 100)) * np.exp(rng.standard_normal((5, 1)) * 4)
    c, s = ref.mxfp4_encode(x)
    v = ref.mxfp4_decode(c, s, 100)
    c2, s2 = ref.mxfp4_encode(v)
    assert np.array_equal(ref.mxfp4_decode(c2, s2, 100), v)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :100]
    a = np.abs(x) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    sat = a > 6
    assert np.all(np.abs(v - x)[~sat] <= (step * unit / 2)[~sat])
    assert np.all(np.abs(v)[sat] == (6 * unit)[sat])


def test_grouped_matmul_oracle_splits_the_rows():
    rng = np.random.default_rng(4)
    x, W = rng.standard_normal((6, 8)), rng.standard_normal((3, 5, 8))
    y = ref.grouped_matmul(x, W, [1, 3, 3, 5])
    assert np.isnan(y[[0, 5]]).all()
    assert np.allclose(y[1], W[0] @ x[1]) and np.allclose(y[4], W[2] @ x[4])


# ------------------------------------------------------------------ refusals of the C ABI

def _quant(lib, X=FAKE, t=BF16, M=4, C=64, ldx=64, codes=FAKE, scales=FAKE):
    return lib.aaac_mxfp4_quantize(X, t, i64(M), i64(C), i64(ldx), codes, scales, None)


def _deq(lib, codes=FAKE, scales=FAKE, M=4, C=64, Y=FAKE, t=BF16, ldy=64):
    return lib.aaac_mxfp4_dequant(codes, scales, i64(M), i64(C), Y, t, i64(ldy), None)


def _mx(lib, wc=FAKE, ws=FAKE, E=1, R=16, C=64, off=None, x=FAKE, t=BF16, xs=None, T=4, ldx=64,
        flags=0, y=FAKE, yt=BF16, ldy=16, work=None, nwork=0):
    return lib.aaac_mxfp4_matmul(wc, ws, i64(E), i64(R), i64(C), off, x, t, xs, i64(T), i64(ldx),
                                 flags, y, yt, i64(ldy), work, ctypes.c_size_t(nwork), None)


def _pk(lib, codes=FAKE, scales=FAKE, bitmap=None, tab=FAKE, E=1, R=16, C=128, g=128, S=128, n=16,
        off=None, x=FAKE, T=4, ldx=128, y=FAKE, yt=BF16, ldy=16, work=None, nwork=0):
    return lib.aaac_matmul(codes, scales, bitmap, tab, i64(E), i64(R), i64(C), g, S, n, off, x,
                           i64(T), i64(ldx), y, yt, i64(ldy), work, ctypes.c_size_t(nwork), None)


def test_mxfp4_quantize_and_dequant_refusals(lib):
    for f, ld in ((_quant, "ldx"), (_deq, "ldy")):
        assert f(lib, t=MXFP4) == INVALID and f(lib, t=-1) == INVALID
        assert f(lib, M=-1) == SHAPE and f(lib, C=0, **{ld: 0}) == SHAPE
        assert f(lib, **{ld: 63}) == SHAPE                        # rows would overlap
        assert f(lib, C=1 << 21, **{ld: 1 << 21}) == SHAPE
        assert f(lib, M=1 << 35) == SHAPE                         # M * Cp >= 2^40
        assert f(lib, codes=None) == INVALID and f(lib, scales=None) == INVALID
        assert f(lib, codes=OFF2) == INVALID
        assert len(lib.aaac_last_error()) > 0
    assert _quant(lib, X=None) == INVALID and _deq(lib, Y=None) == INVALID
    assert _quant(lib, X=OFF2, t=F32) == INVALID and _deq(lib, Y=OFF2, t=F32) == INVALID
    assert _quant(lib, codes=OFF8) == INVALID                     # 16-byte aligned codes
    assert _quant(lib, X=None, M=0) == OK and _deq(lib, Y=None, M=0) == OK   # nothing to do


def test_mxfp4_matmul_refusals(lib):
    assert _mx(lib, t=F32) == INVALID and _mx(lib, yt=MXFP4) == INVALID
    assert _mx(lib, E=0) == SHAPE and _mx(lib, E=65536, off=FAKE) == SHAPE
    assert _mx(lib, E=2) == INVALID                               # experts without offsets
    assert _mx(lib, off=OFF2) == INVALID
    assert _mx(lib, R=0) == SHAPE and _mx(lib, C=0) == SHAPE and _mx(lib, C=1 << 21) == SHAPE
    assert _mx(lib, C=-5) == SHAPE and _mx(lib, R=-1) == SHAPE
    assert _mx(lib, T=-1) == SHAPE and _mx(lib, T=1 << 31) == SHAPE
    assert _mx(lib, ldy=15) == SHAPE and _mx(lib, ldx=56) == SHAPE
    assert _mx(lib, C=60, ldx=64) == SHAPE                        # bf16 rows: C % 8
    assert _mx(lib, ldx=68) == SHAPE                              # bf16 rows: ldx % 8
    assert _mx(lib, C=60, t=MXFP4) == INVALID                     # any width, but x_scales missing
    assert _mx(lib, ldx=1 << 21) == SHAPE
    assert _mx(lib, xs=FAKE) == INVALID                           # bf16 x has no scales
    assert _mx(lib, x=OFF8) == INVALID and _mx(lib, x=None) == INVALID
    assert _mx(lib, y=None) == INVALID and _mx(lib, y=OFF2, yt=F32) == INVALID
    assert _mx(lib, wc=None) == INVALID and _mx(lib, wc=OFF8) == INVALID
    assert _mx(lib, ws=None) == INVALID
    assert _mx(lib, E=1, R=1 << 30, C=2048, ldx=2048, ldy=1 << 30) == SHAPE   # 2^40 weights and more
    assert _mx(lib, R=1 << 20, ldy=1 << 20, T=1 << 30) == SHAPE   # too many tiles
    assert b"tiles" in lib.aaac_last_error()
    assert _mx(lib, x=None, y=None, T=0) == OK


def test_packed_matmul_refusals(lib):
    assert _pk(lib, g=96) == SHAPE and _pk(lib, S=256) == SHAPE and _pk(lib, n=17) == SHAPE
    assert _pk(lib, C=72, g=8, S=8, ldx=72) == SHAPE              # C % 32
    assert _pk(lib, S=16) == INVALID and _pk(lib, bitmap=FAKE) == INVALID
    assert _pk(lib, tab=None) == INVALID and _pk(lib, scales=None) == INVALID
    assert _pk(lib, codes=OFF8) == INVALID and _pk(lib, x=OFF8) == INVALID
    assert _pk(lib, E=3) == INVALID and _pk(lib, E=0) == SHAPE
    assert _pk(lib, ldx=120) == SHAPE and _pk(lib, ldx=132) == SHAPE and _pk(lib, ldy=8) == SHAPE
    assert _pk(lib, T=-3) == SHAPE and _pk(lib, yt=7) == INVALID
    assert _pk(lib, x=None, y=None, T=0) == OK


def test_product_workspaces(lib):
    need = lib.aaac_matmul_workspace_bytes
    for kind in (PACKED, MX, MX_X, MX_QUANTIZE):
        for bad in ((0, 16, 64, 4), (1, 0, 64, 4), (1, 16, 0, 4), (1, 16, 64, 0), (1, 16, 1 << 21, 4),
                    (65536, 16, 64, 4), (1, 16, 64, -1), (1, 16, 64, 1 << 31)):
            assert need(kind, *bad) == 0
    assert need(4, 1, 16, 64, 4) == 0 and need(-1, 1, 16, 64, 4) == 0
    assert need(PACKED, 1, 16, 64, 4) == 0                        # a small product is not split
    # quantised x: codes and scale bytes of T rows
    assert need(MX_QUANTIZE, 1, 16, 65, 3) >= 3 * (48 + 3)
    # one 256-wide column of tiles cannot fill the GPU: its columns are split
    n = need(PACKED, 1, 1024, 8192, 256)
    assert n >= 2 * 256 * 1024 * 4
    args = dict(R=1024, C=8192, T=256, ldx=8192, ldy=1024)
    assert _pk(lib, work=FAKE, nwork=n - 1, **args) == WS_SMALL
    assert _pk(lib, work=ctypes.c_void_p((1 << 20) + 128), nwork=n, **args) == INVALID
    n = need(MX_QUANTIZE, 1, 16, 64, 4)
    assert _mx(lib, flags=1) == INVALID                           # quantising needs the workspace
    assert _mx(lib, flags=1, work=FAKE, nwork=n - 1) == WS_SMALL
    assert _mx(lib, flags=1, t=MXFP4, work=FAKE, nwork=n) == INVALID
    assert _mx(lib, flags=1, xs=FAKE, work=FAKE, nwork=n) == INVALID
    assert _mx(lib, flags=1, ldx=63, work=FAKE, nwork=n) == SHAPE
    assert _mx(lib, flags=1, t=F32, x=OFF2, work=FAKE, nwork=n) == INVALID
    assert _mx(lib, flags=2) == INVALID


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_cpu_tensors_and_unknown_modes():
    import post_weight_quantization_06_amd as P

    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    codes = torch.zeros(16, 32, dtype=torch.uint8)
    scales = torch.zeros(16, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        P.mxfp4_quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        P.mxfp4_matmul(codes, scales, x)
    with pytest.raises(ValueError, match="act"):
        P.mxfp4_matmul(codes, scales, x, act="int8")
    with pytest.raises(ValueError, match="GPU"):
        P.packed_matmul(codes, torch.zeros(16, 1, dtype=torch.int16), None,
                        torch.zeros(2, 16, dtype=torch.int16), x, 64, 64, 16)
    with pytest.raises(ValueError, match=r"\[R, C\]"):
        P.MXFP4Matrix.quantize(x[0])


def test_stacking_experts_of_different_shapes_is_refused():
    import types

    import post_weight_quantization_06_amd as P

    a = types.SimpleNamespace(R=4, C=64, g=32, S=32, n=16)
    b = types.SimpleNamespace(R=4, C=64, g=32, S=16, n=16)
    with pytest.raises(ValueError, match="expert 1"):
        P.PackedExperts.stack([a, b])


@pytest.mark.parametrize("K", [33, 39, 41, 64])
def test_mxfp4_matrix_refuses_other_columns_with_as_many_blocks(K):
    import post_weight_quantization_06_amd as P

    m = P.MXFP4Matrix(40, torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="x has %d columns, the weights 40" % K):
        m.matmul(torch.zeros(4, K, dtype=torch.bfloat16), act="mxfp4")


def test_forward_mode_tangents_are_refused():
    """A dual tensor does not require a gradient, and its tangent would be lost without a word."""
    import torch.autograd.forward_ad as fw

    import post_weight_quantization_06_amd as P

    x = torch.zeros(2, 32)
    P._lib._no_grad("call", x)
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        assert not d.requires_grad
        for v in (d, d[:1], d.reshape(-1)):
            with pytest.raises(ValueError, match="tangent"):
                P._lib._no_grad("call", v)
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            P._lib._no_grad("call", d)
        P._lib._no_grad("call", d.detach())
        P._lib._no_grad("call", x)


@pytest.mark.parametrize("K", [33, 39, 41, 64])
def test_mxfp4_matmul_refuses_other_columns_than_its_c(K):
    import post_weight_quantization_06_amd as P

    codes, scales = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    for act in ("bf16", "mxfp4"):
        with pytest.raises(ValueError, match="x has %d columns, the weights 40" % K):
            P.mxfp4_matmul(codes, scales, torch.zeros(4, K, dtype=torch.bfloat16), act=act, C=40)
    with pytest.raises(ValueError, match="GPU"):             # the right width goes on to the next check
        P.mxfp4_matmul(codes, scales, torch.zeros(4, 40, dtype=torch.bfloat16), C=40)


def test_results_of_another_last_axis_are_refused():
    """An out of as many elements whose rows are not the result's, or of another width than C."""
    import post_weight_quantization_06_amd as P

    codes, scales = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    ps, pt = torch.zeros(16, 1, dtype=torch.int16), torch.zeros(2, 16, dtype=torch.int16)
    for out in (torch.zeros(16, 6), torch.zeros(2, 3, 8), torch.zeros(96), torch.zeros(())):
        with pytest.raises(ValueError, match=r"out must be \[\.\.\., 16\]"):
            P.mxfp4_matmul(codes, scales, x, out=out)
        with pytest.raises(ValueError, match=r"out must be \[\.\.\., 16\]"):
            P.packed_matmul(codes, ps, None, pt, x, 64, 64, 16, out=out)
    for C in (33, 40, 64):                           # as many blocks, another width
        with pytest.raises(ValueError, match=r"out must be \[\.\.\., %d\] \(got \[16, 50\]\)" % C):
            P.mxfp4_dequant(codes, scales, C, out=torch.zeros(16, 50))
    for out in (torch.zeros(2, 3, 16), torch.zeros(6, 16)):  # the result's rows: on to the next check
        with pytest.raises(ValueError, match="GPU"):
            P.mxfp4_matmul(codes, scales, x, out=out)
    with pytest.raises(ValueError, match="GPU"):
        P.mxfp4_dequant(codes, scales, 50, out=torch.zeros(16, 50))


def test_plans_of_the_tested_forms(lib):
    """Every kernel and tile that a plan can pick is among the forms that the GPU tests run. Without a GPU
    the plan is that of 256 CUs."""
    from tests.test_gpu_matmul_forms import FORMS, MX, MXX, PK, form

    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("plans of another GPU")
    for kind, _, E, R, C, T, plan in FORMS:
        assert form(kind, E, R, C, T) == plan, (kind, E, R, C, T)
    few = {("few", 1, 1, 1), ("few", 1, 1, 4), ("few", 2, 1, 1)}
    for kind, tiles in ((PK, ((128, 32), (128, 64), (128, 128), (256, 256))),
                        (MX, ((128, 32), (128, 64), (128, 128), (256, 256))),
                        (MXX, ((64, 64), (128, 64), (128, 128), (256, 256)))):
        got = {f[-1] for f in FORMS if f[0] == kind}
        want = {("tile", bm, bn, split) for bm, bn in tiles for split in (False, True)}
        want |= few if kind != MXX else {("few", rt, nt, 1) for rt in (1, 2) for nt in (1, 2)}
        assert want <= got, want - got


def test_plan_query(lib):
    f = lib.aaac_matmul_plan
    plan = (ctypes.c_int32 * 6)(*[7] * 6)
    for bad in ((4, 1, 16, 64, 4), (0, 0, 16, 64, 4), (0, 1, 0, 64, 4), (0, 1, 16, 0, 4), (0, 1, 16, 64, 0)):
        assert f(bad[0], *[i64(v) for v in bad[1:]], 1, plan) == SHAPE and list(plan) == [7] * 6
    assert f(0, i64(1), i64(16), i64(64), i64(4), 1, None) == INVALID
    assert f(0, i64(1), i64(16), i64(64), i64(4), 1, plan) == OK and list(plan) == [0, 0, 1, 1, 1, 1]
    assert f(0, i64(1), i64(1024), i64(8192), i64(256), 1, plan) == OK and plan[2] > 1
    assert f(0, i64(1), i64(1024), i64(8192), i64(256), 0, plan) == OK and plan[2] == 1
