"""GPU parity of the products on 4-bit weights in the forms that sizes, addresses and callers can give
them, against the fp64 oracle or the framework's own dequantization. Small whole numbers throughout:
every partial sum is exact in fp32, so results have to be equal."""

import numpy as np
import pytest
import torch

from oracle import aaac_ref as ref
from tests.test_gpu_matmul import _dev, _mx, _packed, _say, _x

pytestmark = pytest.mark.gpu

P = pytest.importorskip("post_weight_quantization_06_amd")
L = P._lib

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    L.load()
    yield


def _moved(t, by):
    """t in memory that starts `by` elements past an aligned address."""
    room = torch.zeros(t.numel() + by + 64, dtype=t.dtype, device=t.device)
    v = room[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------ addresses of the weights

@pytest.mark.parametrize("g,S,n", [(8, 8, 16), (16, 16, 15), (16, 8, 16), (32, 32, 16), (32, 16, 16),
                                   (128, 128, 16), (128, 8, 13)])
@pytest.mark.parametrize("T", [3, 40, 300, 1030])
def test_packed_scales_and_bitmap_at_any_address(g, S, n, T):
    """The scales start on an odd element, the bitmap on an odd byte: as dequant reads them, in the
    few-row kernels and in tiles of every width."""
    rng = np.random.default_rng(g * 1009 + S + T)
    R, C = (72, 384) if T < 1000 else (4104, 128)
    codes, scales, bitmap, tables, _ = _packed(rng, 1, R, C, g, S, n, True)
    x, xd = _x(rng, T, C, True)
    bm = None if bitmap is None else bitmap[0]
    W = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
    L.aaac_dequant(codes.view(-1), scales.view(-1), None if bm is None else bm.view(-1),
                   tables.view(-1), R, C, g, S, n, W)
    want = torch.from_numpy(x).to(DEV) @ W.double().t()
    for by in (1, 2, 3):
        _say("packed addresses", g, S, n, T, by)
        sc = _moved(scales[0], by)
        assert sc.data_ptr() % 4 == 2 * (by % 2)
        y = P.packed_matmul(codes[0], sc, None if bm is None else _moved(bm, by),
                            _moved(tables[0], by), xd, g, S, n, dtype=torch.float32)
        assert torch.equal(y.double(), want)


def test_packed_experts_with_scales_on_an_odd_element():
    rng = np.random.default_rng(31)
    E, R, C, T = 4, 40, 160, 200
    for g, S in ((8, 8), (16, 16), (16, 8)):
        codes, scales, bitmap, tables, W = _packed(rng, E, R, C, g, S, 16, True)
        x, xd = _x(rng, T, C, True)
        off = np.array([0, 70, 70, 131, T], np.int32)
        _say("packed experts, odd scales", g, S)
        y = P.packed_matmul(codes, _moved(scales, 1), None if bitmap is None else _moved(bitmap, 1),
                            tables, xd, g, S, 16, _dev(off), dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), ref.grouped_matmul(x, W, off).astype(np.float32))


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_mxfp4_scales_at_any_address(act, T):
    rng = np.random.default_rng(T)
    R, C = 72, 768
    codes, scales, W = _mx(rng, 1, R, C, True)
    x, xd = _x(rng, T, C, True)
    xv = x if act == "bf16" else ref.mxfp4_decode(*ref.mxfp4_encode(x), C)
    for by in (1, 2, 3, 4):
        _say("mx addresses", act, T, by)
        y = P.mxfp4_matmul(codes[0], _moved(scales[0], by), xd, act=act, dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), (xv @ W[0].T).astype(np.float32))


# ------------------------------------------------------------------ launches of more than 2^32 threads

def _room(gib):
    free = torch.cuda.mem_get_info()[0] / 2 ** 30
    if free < gib:
        pytest.skip("needs %d GiB of free GPU memory (%.0f are)" % (gib, free))


def test_product_of_more_than_2_32_threads():
    """512 experts of 494000 x 32 with one row each: 8.4 million workgroups of 512 threads."""
    _room(16)
    _say("product, over 2^32 threads")
    E, R, C = 512, 494000, 32
    gen = torch.Generator(device=DEV).manual_seed(6)
    codes = torch.randint(0, 256, (E, R, C // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (E, R, 1), generator=gen, device=DEV, dtype=torch.uint8)
    x = torch.randint(-4, 5, (E, C), generator=gen, device=DEV).to(torch.bfloat16)
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32)
    for act in ("bf16", "mxfp4"):
        y = torch.full((E, R), 99.0, dtype=torch.float32, device=DEV)
        P.mxfp4_matmul(codes, scales, x, off, act=act, out=y)
        xv = x.double() if act == "bf16" else P.mxfp4_dequant(*P.mxfp4_quantize(x), C).double()
        for e in (0, 1, 100, 255, 256, 300, 400, 480, 509, 510, 511):
            W = P.mxfp4_dequant(codes[e], scales[e], C, dtype=torch.float32).double()
            assert torch.equal(y[e].double(), (W * xv[e]).sum(1)), e
    torch.cuda.empty_cache()


def test_tiles_of_more_than_2_32_threads():
    """4096 experts of 494000 x 32 with 17 rows each: 8.4 million workgroups of 512 threads."""
    _room(130)
    _say("tiles, over 2^32 threads")
    E, R, C, N = 4096, 494000, 32, 17
    gen = torch.Generator(device=DEV).manual_seed(8)
    codes = torch.randint(0, 256, (E, R, C // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (E, R, 1), generator=gen, device=DEV, dtype=torch.uint8)
    x = torch.randint(-4, 5, (E * N, C), generator=gen, device=DEV).to(torch.bfloat16)
    off = torch.arange(0, E * N + 1, N, device=DEV, dtype=torch.int32)
    y = torch.full((E * N, R), 99.0, dtype=torch.bfloat16, device=DEV)
    P.mxfp4_matmul(codes, scales, x, off, out=y)
    for e in (0, 1, 1000, 2047, 2048, 3000, 4000, 4080, 4094, 4095):
        W = P.mxfp4_dequant(codes[e], scales[e], C, dtype=torch.float32).double()
        want = x[e * N:e * N + N].double() @ W.t().contiguous()
        assert torch.equal(y[e * N:e * N + N], want.to(torch.bfloat16)), e
    del codes, scales, y
    torch.cuda.empty_cache()


def test_mxfp4_of_2_32_threads_and_more():
    """2^32 + 100 rows of one column: a thread a row, rows past 32 bits."""
    _room(100)
    _say("mxfp4, over 2^32 threads")
    M = 2 ** 32 + 100
    x = torch.empty(M, 1, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(7))
    codes, scales = P.mxfp4_quantize(x)
    back = torch.full((M, 1), 99.0, dtype=torch.bfloat16, device=DEV)
    P.mxfp4_dequant(codes, scales, 1, out=back)
    for r in (0, 2 ** 24, 2 ** 30 - 256, 2 ** 31 - 256, 2 ** 32 - 4096, 2 ** 32 - 256, M - 512):
        wc, ws = ref.mxfp4_encode(x[r:r + 512].double().cpu().numpy())
        assert np.array_equal(scales[r:r + 512].cpu().numpy(), ws), r
        assert np.array_equal(codes[r:r + 512, 0].cpu().numpy(), wc[:, 0]), r
        assert np.array_equal(back[r:r + 512].double().cpu().numpy(), ref.mxfp4_decode(wc, ws, 1)), r
    del x, codes, scales, back
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ tiles of one row

@pytest.mark.parametrize("R,T,C", [(129, 33, 64), (129, 65, 320), (257, 129, 96), (513, 97, 800),
                                   (2753, 1281, 64), (4097, 4097, 64), (4097, 4097, 200), (1, 257, 1280)])
def test_last_tiles_of_one_row(R, T, C):
    """One row of x and one weight row in the last tiles: the loads that run ahead of the last step
    then lie past the ends of the smallest buffers."""
    rng = np.random.default_rng(R + T + C)
    codes, scales, W = _mx(rng, 1, R, C, True)
    x, xd = _x(rng, T, C, True)
    xv = {"bf16": x, "mxfp4": ref.mxfp4_decode(*ref.mxfp4_encode(x), C)}
    for act, v in xv.items():
        _say("one row", act, R, T, C)
        y = P.mxfp4_matmul(codes[0], scales[0], xd, act=act, dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), (v @ W[0].T).astype(np.float32))
    if C % 32:
        return
    for g, S in ((32, 32), (16, 8)):
        _say("one row", g, S, R, T, C)
        pc, ps, pb, pt, pW = _packed(rng, 1, R, C, g, S, 16, True)
        y = P.packed_matmul(pc[0], ps[0], None if pb is None else pb[0], pt[0], xd, g, S, 16,
                            dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), (x @ pW[0].T).astype(np.float32))


# ------------------------------------------------------------------ refusals

def test_forward_mode_tangents_are_refused_by_every_call():
    import torch.autograd.forward_ad as fw

    rng = np.random.default_rng(14)
    mc, ms, _ = _mx(rng, 1, 16, 64, True)
    pc, ps, pb, pt, _ = _packed(rng, 1, 16, 64, 32, 16, 16, True)
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda v: P.mxfp4_quantize(v), lambda v: P.mxfp4_matmul(mc[0], ms[0], v),
                     lambda v: P.mxfp4_matmul(mc[0], ms[0], v, act="mxfp4"),
                     lambda v: P.packed_matmul(pc[0], ps[0], pb[0], pt[0], v, 32, 16, 16)):
            with pytest.raises(ValueError, match="tangent"):
                call(d)
            call(d.detach())


def test_mxfp4_matmul_with_the_width_given():
    rng = np.random.default_rng(15)
    codes, scales, W = _mx(rng, 1, 16, 40, True)
    x, xd = _x(rng, 6, 40, True)
    want = (x @ W[0].T).astype(np.float32)
    m = P.MXFP4Matrix(40, codes[0], scales[0])
    for y in (P.mxfp4_matmul(codes[0], scales[0], xd, dtype=torch.float32, C=40),
              P.mxfp4_matmul(codes[0], scales[0], xd, dtype=torch.float32),
              m.matmul(xd, dtype=torch.float32)):
        assert np.array_equal(y.cpu().numpy(), want)
    wide = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="64 columns, the weights 40"):
        P.mxfp4_matmul(codes[0], scales[0], wide, C=40)


def test_results_of_other_shapes_are_filled_row_by_row_or_refused():
    rng = np.random.default_rng(16)
    codes, scales, W = _mx(rng, 1, 24, 64, True)
    x, xd = _x(rng, 6, 64, True)
    want = torch.from_numpy((x @ W[0].T).astype(np.float32))
    for shape in ((2, 3, 24), (6, 24), (3, 2, 24)):
        y = torch.zeros(shape, device=DEV)
        P.mxfp4_matmul(codes[0], scales[0], xd.view(2, 3, 64), out=y)
        assert torch.equal(y.cpu().view(6, 24), want)
    with pytest.raises(ValueError, match="out must be"):
        P.mxfp4_matmul(codes[0], scales[0], xd.view(2, 3, 64), out=torch.zeros(24, 6, device=DEV))
    with pytest.raises(ValueError, match="out must be"):
        P.mxfp4_dequant(codes[0], scales[0], 64, out=torch.zeros(24, 60, device=DEV))


# ------------------------------------------------------------------ every kernel form, many steps

# (kind, (g, S, n) of packed weights, E, R, C, T, expected plan). Plans: ("few", rt, nt, chunks) or
# ("tile", weight rows, rows of x, split or not) on 256 CUs, by aaac_matmul_plan. R and T are cut by
# every tile; the columns make 6 steps and more, in MXFP4 x whole blocks of 256 or not.
PK, MX, MXX = L.MATMUL_PACKED, L.MATMUL_MXFP4, L.MATMUL_QUANTIZE_X
FORMS = [
    (PK, (128, 128, 16), 1, 1031, 640, 13, ("few", 1, 1, 1)),
    (PK, (128, 16, 16), 1, 1031, 1152, 13, ("few", 1, 1, 1)),
    (PK, (128, 128, 16), 1, 219, 8320, 3, ("few", 1, 1, 4)),        # x in LDS
    (PK, (64, 64, 15), 1, 219, 8320, 13, ("few", 1, 1, 4)),         # x read directly
    (PK, (128, 128, 16), 1, 8211, 640, 13, ("few", 2, 1, 1)),
    (PK, (16, 16, 15), 5, 1645, 608, 61, ("few", 2, 1, 1)),
    (PK, (128, 128, 16), 1, 8247, 8320, 5, ("few", 2, 1, 4)),
    (PK, (128, 128, 16), 1, 131, 640, 19, ("tile", 128, 32, True)),
    (PK, (16, 8, 16), 3, 300, 448, 99, ("tile", 128, 32, False)),
    (PK, (128, 16, 16), 1, 132, 640, 4110, ("tile", 128, 64, False)),
    (PK, (128, 128, 16), 1, 130, 4096, 513, ("tile", 128, 64, True)),
    (PK, (32, 32, 16), 1, 262, 544, 5501, ("tile", 128, 128, False)),
    (PK, (16, 16, 15), 5, 6231, 512, 97, ("tile", 128, 128, False)),
    (PK, (128, 128, 16), 1, 263, 2048, 2069, ("tile", 128, 128, True)),
    (PK, (128, 128, 16), 1, 7400, 640, 1031, ("tile", 256, 256, False)),
    (PK, (128, 16, 16), 1, 7400, 640, 1031, ("tile", 256, 256, False)),
    (PK, (16, 16, 15), 1, 7400, 640, 1031, ("tile", 256, 256, False)),
    (PK, (8, 8, 16), 10, 7615, 512, 1620, ("tile", 256, 256, False)),
    (PK, (128, 64, 16), 1, 258, 2176, 5674, ("tile", 256, 256, True)),
    (MX, None, 1, 1031, 648, 13, ("few", 1, 1, 1)),
    (MX, None, 1, 219, 8328, 3, ("few", 1, 1, 4)),
    (MX, None, 1, 219, 8320, 13, ("few", 1, 1, 4)),
    (MX, None, 1, 8211, 648, 13, ("few", 2, 1, 1)),
    (MX, None, 10, 1000, 512, 60, ("few", 2, 1, 1)),
    (MX, None, 1, 131, 648, 18, ("tile", 128, 32, True)),
    (MX, None, 3, 300, 456, 99, ("tile", 128, 32, False)),
    (MX, None, 1, 131, 552, 4171, ("tile", 128, 64, False)),
    (MX, None, 1, 130, 1032, 2059, ("tile", 128, 64, True)),
    (MX, None, 1, 260, 520, 5671, ("tile", 128, 128, False)),
    (MX, None, 1, 263, 2056, 2069, ("tile", 128, 128, True)),
    (MX, None, 1, 7400, 648, 1031, ("tile", 256, 256, False)),
    (MX, None, 10, 7366, 512, 1710, ("tile", 256, 256, False)),
    (MX, None, 1, 258, 2176, 5408, ("tile", 256, 256, True)),
    (MXX, None, 1, 1031, 2085, 13, ("few", 1, 1, 1)),
    (MXX, None, 1, 1031, 2304, 29, ("few", 1, 2, 1)),
    (MXX, None, 1, 8242, 2085, 13, ("few", 2, 1, 1)),
    (MXX, None, 1, 8391, 2080, 18, ("few", 2, 2, 1)),
    (MXX, None, 5, 1645, 2080, 61, ("few", 2, 1, 1)),
    (MXX, None, 1, 131, 2304, 70, ("tile", 64, 64, False)),
    (MXX, None, 1, 131, 4101, 70, ("tile", 64, 64, True)),
    (MXX, None, 1, 8249, 2304, 68, ("tile", 128, 64, False)),
    (MXX, None, 1, 8249, 2081, 68, ("tile", 128, 64, False)),
    (MXX, None, 1, 70, 4096, 2140, ("tile", 128, 64, True)),
    (MXX, None, 1, 260, 2304, 5775, ("tile", 128, 128, False)),
    (MXX, None, 1, 260, 2081, 5775, ("tile", 128, 128, False)),
    (MXX, None, 1, 300, 8192, 901, ("tile", 128, 128, True)),
    (MXX, None, 1, 7400, 2304, 1031, ("tile", 256, 256, False)),
    (MXX, None, 1, 7400, 2081, 1031, ("tile", 256, 256, False)),
    (MXX, None, 10, 7487, 2304, 1760, ("tile", 256, 256, False)),
    (MXX, None, 1, 8441, 8192, 403, ("tile", 256, 256, True)),
    (MXX, None, 1, 8441, 8160, 403, ("tile", 256, 256, True)),
]


def form(kind, E, R, C, T):
    bm, bn, split, rt, nt, chunks = L.matmul_plan(kind, E, R, C, T)
    return ("tile", bm, bn, split > 1) if bn else ("few", rt, nt, chunks)


def _mx_dev(gen, E, R, C):
    """MXFP4 weights of whole numbers up to 12, made on the GPU."""
    nb = -(-C // 32)
    whole = torch.tensor([0, 2, 4, 5, 6, 10, 12, 13], dtype=torch.uint8, device=DEV)
    q = whole[torch.randint(0, 8, (E, R, nb * 32), generator=gen, device=DEV)]
    q[..., C:] = 0
    s = torch.randint(127, 129, (E, R, nb), generator=gen, device=DEV, dtype=torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), s


def _packed_dev(gen, E, R, C, g, S, n):
    """Packed weights of whole numbers and halves, made on the GPU."""
    q = torch.randint(0, n, (E, R, C), generator=gen, device=DEV, dtype=torch.uint8)
    s = torch.tensor([0.5, 1.0, 2.0], device=DEV)[
        torch.randint(0, 3, (E, R, C // g), generator=gen, device=DEV)]
    words, bitmap = s.to(torch.bfloat16).view(torch.int16), None
    if S == g:
        words = words | (torch.randint(0, 2, words.shape, generator=gen, device=DEV) << 15).to(torch.int16)
    else:
        bitmap = torch.randint(0, 256, (E, (R * (C // S) + 7) // 8), generator=gen, device=DEV,
                               dtype=torch.uint8)
    T = torch.randint(-8, 8, (E, 2, n), generator=gen, device=DEV) * 2
    return q[..., 0::2] | (q[..., 1::2] << 4), words, bitmap, T.to(torch.bfloat16).view(torch.int16)


def _starts(gen, E, T):
    """Ascending offsets, one expert empty, on the CPU."""
    cuts = torch.randint(0, T + 1, (E - 1,), generator=gen).sort().values
    if E > 2:
        cuts[1] = cuts[0]
    return torch.nn.functional.pad(cuts, (1, 1), value=0).index_fill_(0, torch.tensor([E]), T).to(torch.int32)


@pytest.mark.parametrize("kind,fmt,E,R,C,T,plan", FORMS)
def test_every_kernel_form(kind, fmt, E, R, C, T, plan):
    """Each kernel and tile that a plan can pick, against the framework's own dequantized weights."""
    _say("form", kind, fmt, E, R, C, T, plan)
    assert form(kind, E, R, C, T) == plan
    gen = torch.Generator(device=DEV).manual_seed(R * 13 + C + T)
    x = torch.randint(-4, 5, (T, C), generator=gen, device=DEV).to(torch.bfloat16)
    at = [0, T] if E == 1 else _starts(torch.Generator().manual_seed(E + T), E, T).tolist()
    off = None if E == 1 else torch.tensor(at, dtype=torch.int32, device=DEV)
    if kind == PK:
        g, S, n = fmt
        w = _packed_dev(gen, E, R, C, g, S, n)
        one = [None if t is None else t[0] for t in w] if E == 1 else w
        y = P.packed_matmul(*one, x, g, S, n, off, dtype=torch.float32)
    else:
        w = _mx_dev(gen, E, R, C)
        one = [t[0] for t in w] if E == 1 else w
        y = P.mxfp4_matmul(*one, x, off, act="bf16" if kind == MX else "mxfp4", dtype=torch.float32, C=C)
        if kind == MXX:                              # whole numbers up to 4 are MXFP4 values
            assert torch.equal(P.mxfp4_dequant(*P.mxfp4_quantize(x), C), x)
    for e in range(E):
        if at[e] == at[e + 1]:
            continue
        if kind == PK:
            W = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
            L.aaac_dequant(w[0][e].reshape(-1), w[1][e].reshape(-1),
                           None if w[2] is None else w[2][e], w[3][e].reshape(-1), R, C, g, S, n, W)
        else:
            W = P.mxfp4_dequant(w[0][e], w[1][e], C, dtype=torch.float32)
        want = x[at[e]:at[e + 1]].double() @ W.double().t()
        assert float(want.abs().max()) < 2 ** 22
        assert torch.equal(y[at[e]:at[e + 1]].double(), want), e


# ------------------------------------------------------------------ x as codes, rows, split sums

SPREAD = [  # E, R, C, T: few rows, tiles, tiles with split columns, widths of no whole block
    (1, 200, 1000, 9), (1, 200, 1024, 29), (1, 131, 2304, 70), (1, 131, 4101, 70), (1, 700, 777, 900),
    (4, 300, 512, 40), (4, 300, 545, 500),
]


@pytest.mark.parametrize("E,R,C,T", SPREAD)
def test_x_given_as_codes_has_the_bits_of_x_quantized_in_the_call(E, R, C, T):
    _say("x as codes", E, R, C, T)
    rng = np.random.default_rng(R + C + T)
    codes, scales, W = _mx(rng, E, R, C, False)
    x, xd = _x(rng, T, C, False)
    off = _dev(np.linspace(0, T, E + 1).astype(np.int32))
    xc, xs = P.mxfp4_quantize(xd)
    ws = torch.full((L.matmul_workspace_bytes(L.MATMUL_MXFP4_X, E, R, C, T) or 256,), 0xFF, dtype=torch.uint8,
                    device=DEV)                      # NaN where a sum would read what it did not write
    for dtype in (torch.float32, torch.bfloat16):
        want = P.mxfp4_matmul(codes, scales, xd, off, act="mxfp4", dtype=dtype, C=C)
        y = torch.full((T, R), 99.0, dtype=dtype, device=DEV)
        P.aaac_mxfp4_matmul(codes, scales, C, xc, y, off, x_scales=xs)
        assert torch.equal(y, want)
        y.fill_(99.0)
        P.aaac_mxfp4_matmul(codes, scales, C, xc, y, off, x_scales=xs, ws=ws)
        assert torch.equal(y, want)
        y.fill_(99.0)
        P.aaac_mxfp4_matmul(codes, scales, C, xc, y, off, x_scales=_moved(xs, 1))
        assert torch.equal(y, want)
    # and near the exact product of the values: an fp32 sum of C terms
    xv = ref.mxfp4_decode(*ref.mxfp4_encode(x), C)
    full = ref.grouped_matmul(xv, W, off.cpu().numpy())
    mass = ref.grouped_matmul(np.abs(xv), np.abs(W), off.cpu().numpy())
    got = P.mxfp4_matmul(codes, scales, xd, off, act="mxfp4", dtype=torch.float32).double().cpu().numpy()
    assert np.all(np.abs(got - full) <= (C / 32 + 144) * 2.0 ** -23 * mass + 1e-30)
    y = torch.empty(0, R, device=DEV)
    P.aaac_mxfp4_matmul(codes, scales, C, xc[:0], y, off, x_scales=xs[:0])
    with pytest.raises(ValueError, match="x_scales"):
        P.aaac_mxfp4_matmul(codes, scales, C, xc, torch.empty(T, R, device=DEV), off, x_scales=xs[:-1])


def _three(E, R, C, seed):
    """(name, call(x, offsets, out)) of the three products on random weights."""
    rng = np.random.default_rng(seed)
    mc, ms, _ = _mx(rng, E, R, C, False)
    pc, ps, pb, pt, _ = _packed(rng, E, R, C, 32, 16, 16, False)
    return [("mx bf16", lambda x, o, y: P.mxfp4_matmul(mc, ms, x, o, out=y)),
            ("mx mxfp4", lambda x, o, y: P.mxfp4_matmul(mc, ms, x, o, act="mxfp4", out=y)),
            ("packed", lambda x, o, y: P.packed_matmul(pc, ps, pb, pt, x, 32, 16, 16, o, out=y))]


@pytest.mark.parametrize("E,R,C,T", [(3, 100, 512, 30), (1, 300, 608, 30), (3, 100, 512, 90),
                                     (2, 1000, 320, 700), (1, 131, 4096, 70), (3, 256, 4096, 200)])
def test_a_rows_result_depends_on_no_other_row(E, R, C, T):
    """Bitwise, in few-row kernels, tiles and split sums: other rows changed, made NaN or infinite, and
    the rows of an expert in another order."""
    at = np.linspace(0, T, E + 1).astype(np.int32)
    off = _dev(at)
    x, xd = _x(np.random.default_rng(T), T, C, False)
    keep = torch.zeros(T, dtype=torch.bool, device=DEV)
    keep[::3] = True
    order = torch.cat([torch.arange(int(a), int(b)).flip(0) for a, b in zip(at, at[1:])]).to(DEV)
    for name, call in _three(E, R, C, R + C):
        _say("row by row", name, E, R, C, T)
        want = torch.empty(T, R, dtype=torch.float32, device=DEV)
        call(xd, off, want)
        assert torch.isfinite(want).all()
        for other in (xd.flip(0) * 3, torch.full_like(xd, float("nan")),
                      torch.full_like(xd, float("inf")), torch.zeros_like(xd)):
            y = torch.empty_like(want)
            call(torch.where(keep[:, None], xd, other), off, y)
            assert torch.equal(y[keep], want[keep])
        y = torch.empty_like(want)
        call(xd[order], off, y)
        assert torch.equal(y, want[order])


def test_rows_of_no_expert_stay_as_they_were_with_split_columns():
    rng = np.random.default_rng(17)
    E, R, C, T = 2, 256, 4096, 64
    codes, scales, W = _mx(rng, E, R, C, True)
    x, xd = _x(rng, T, C, True)
    xd[:5], xd[50:] = float("nan"), float("inf")
    off = np.array([5, 20, 50], np.int32)
    want = ref.grouped_matmul(x, W, off)
    want[np.isnan(want)] = 55.0
    for act, kind in (("bf16", L.MATMUL_MXFP4), ("mxfp4", L.MATMUL_QUANTIZE_X)):
        _say("split, outside rows", act)
        assert form(kind, E, R, C, T)[-1] is True
        y = torch.full((T, R), 55.0, dtype=torch.float32, device=DEV)
        P.mxfp4_matmul(codes, scales, xd, _dev(off), act=act, out=y)
        assert np.array_equal(y.cpu().numpy(), want.astype(np.float32))


def test_x_of_more_than_2_32_elements():
    _room(40)
    E, R, C, T = 2, 40, 8192, 530000
    gen = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randint(-4, 5, (T, C), generator=gen, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    assert x.numel() > 2 ** 32
    at = [0, 400001, T]
    off = torch.tensor(at, dtype=torch.int32, device=DEV)
    mx, pk = _mx_dev(gen, E, R, C), _packed_dev(gen, E, R, C, 128, 16, 16)
    for name, call in (("mx bf16", lambda: P.mxfp4_matmul(*mx, x, off, dtype=torch.float32)),
                       ("mx mxfp4", lambda: P.mxfp4_matmul(*mx, x, off, act="mxfp4", dtype=torch.float32)),
                       ("packed", lambda: P.packed_matmul(*pk, x, 128, 16, 16, off, dtype=torch.float32))):
        _say("large x", name)
        y = call()
        for e in range(E):
            if name == "packed":
                W = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
                L.aaac_dequant(*[t[e].reshape(-1) for t in pk], R, C, 128, 16, 16, W)
            else:
                W = P.mxfp4_dequant(mx[0][e], mx[1][e], C, dtype=torch.float32)
            for r in (at[e], at[e] + 131071, 262143 if e == 0 else 524287, at[e + 1] - 300):
                assert torch.equal(y[r:r + 300].double(), x[r:r + 300].double() @ W.double().t()), (e, r)
    del x, y
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ calls at once

def test_calls_on_two_streams_at_once_and_two_graphs():
    """Products that use a workspace, in flight on two streams together, then captured into two graphs
    that replay in turn and together: each call has a workspace of its own."""
    E, R, C, T = 1, 256, 4096, 64
    for name, call in _three(E, R, C, 23):
        _say("at once", name)
        off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        xs = [_x(np.random.default_rng(s), T, C, False)[1] for s in (1, 2)]
        want = [torch.empty(T, R, dtype=torch.float32, device=DEV) for _ in xs]
        for x, w in zip(xs, want):
            call(x, off, w)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in xs]
        ys = [[torch.zeros_like(w) for _ in range(20)] for w in want]
        torch.cuda.synchronize()
        for k in range(20):
            for i, st in enumerate(streams):
                with torch.cuda.stream(st):
                    call(xs[i], off, ys[i][k])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i]) for i in (0, 1) for y in ys[i])
        graphs, outs = [], []
        for x in xs:
            y, g = torch.zeros_like(want[0]), torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(x, off, y)
            graphs.append(g)
            outs.append(y)
        for k in range(4):
            for y in outs:
                y.zero_()
            torch.mm(torch.ones(64, 64, device=DEV), torch.ones(64, 64, device=DEV))
            torch.cuda.synchronize()
            for i, st in enumerate(streams):
                with torch.cuda.stream(st):
                    graphs[i if k % 2 else 1 - i].replay()
                if k < 2:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            assert all(torch.equal(y, w) for y, w in zip(outs, want))
