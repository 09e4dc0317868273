"""GPU parity of FP8 in blocks of 128 (quantize, dequant, products) against the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import aaac_ref as ref

pytestmark = pytest.mark.gpu

P = pytest.importorskip("post_weight_quantization_06_amd")
L = P._lib

DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _say(*a):
    print("[case]", *a, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    L.load()
    yield


def _gen(*key):
    return torch.Generator().manual_seed(sum(int(k) * 7919 ** i for i, k in enumerate(key)) % (1 << 62))


def _bytes(codes):
    return codes.contiguous().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ quantize and dequant

def _check(x, tile):
    """Quantise x [M, C] on the GPU; codes and scales bit for bit against the oracle, and the values."""
    codes, scales = P.fp8_quantize(x, tile=tile)
    want_c, want_s = ref.fp8_encode(x.double().cpu().numpy(), tile)
    assert codes.shape == x.shape and codes.stride(0) % 16 == 0 and codes.data_ptr() % 16 == 0
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(_bytes(codes), want_c)
    # fp32 product of code and scale, rounded to the type
    value = torch.from_numpy(ref.fp8_decode(want_c, np.ones_like(want_s), tile)).float()
    value *= torch.from_numpy(ref._fp8_spread(want_s, *x.shape, tile))
    for dt in TYPES:
        got = P.fp8_dequant(codes, scales, dtype=dt).cpu()
        assert torch.equal(torch.nan_to_num(got.float(), 7e7, 8e7, 9e7),
                           torch.nan_to_num(value.to(dt).float(), 7e7, 8e7, 9e7))
    return codes, scales


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C", [(1, 1), (1, 15), (3, 16), (2, 127), (5, 129), (1, 4096), (129, 264),
                                 (257, 1000), (300, 515)])
def test_quantize_matches_the_oracle(dtype, M, C, tile):
    _say("fp8", dtype, M, C, tile)
    x = torch.randn(M, C, generator=_gen(M, C)) * torch.exp(2 * torch.randn(M, 1, generator=_gen(C, M)))
    _check(x.to(dtype).to(DEV), tile)


def test_every_bf16_value_beside_several_largest_ones():
    _say("fp8 all bf16")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for top in (0.0, 2.0 ** -126, 2.0 ** -90, 1.0, 448.0, 450.0, 3e38):
        x = bits.view(512, 128).clone()
        big = x.float().abs() > top              # the block's largest is top, where it is not 0
        if top:
            x[big] = torch.tensor(top).to(torch.bfloat16)
            x[:, 5] = top
        _check(x.to(DEV), False)


def test_fp32_ties_and_neighbours_of_ties():
    # scale 1 (the largest is 448) and powers of two: every midpoint of two codes, and its neighbours
    _say("fp8 ties")
    t = ref._e4m3_table()[:127]
    mid = ((t[1:] + t[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999))])
    v = np.concatenate([v, -v, [0.0, -0.0, 1e-30, -1e-30, 2.0 ** -10, 2.0 ** -10 * 1.0001]])
    v = np.resize(v, (7, 127)).astype(np.float32)
    rows = []
    for e in (-126, -100, -81, -80, -79, -3, 0, 5, 100, 119):
        with np.errstate(under="ignore"):
            rows.append(np.ldexp(np.concatenate([v, np.full((7, 1), 448, np.float32)], 1), e))
    _check(torch.from_numpy(np.concatenate(rows).astype(np.float32)).to(DEV), False)


@pytest.mark.parametrize("exp", [-140, -127, -110, -82, -60, 0, 100])
def test_quotients_by_scales_of_every_size(exp):
    # scales that are no powers of two, down to the least one: quotients are the rounded ones
    _say("fp8 scales", exp)
    x = torch.randn(300, 256, generator=_gen(exp + 200), dtype=torch.float64)
    x = torch.ldexp(x * (1 + torch.rand(300, 1, generator=_gen(exp + 201), dtype=torch.float64)),
                    torch.tensor(exp))
    _check(x.float().to(DEV), False)


def test_infinities_nan_and_zero_blocks():
    _say("fp8 inf nan")
    for dt in TYPES:
        for tile in (False, True):
            x = torch.randn(260, 300, generator=_gen(5)).to(dt)
            x[0, 0], x[1, 140], x[2, 299], x[3, 128:256] = float("inf"), float("-inf"), float("nan"), 0.0
            x[128:256, :128] = -0.0
            codes, scales = _check(x.to(DEV), tile)
            # the three bad elements lie in three rows' blocks, and in three tiles of the first row
            assert (~torch.isfinite(scales)).sum() == 3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C,ld,start", [(64, 96, 0), (64, 100, 3), (150, 177, 1), (256, 264, 8)])
def test_strided_rows_in_and_out(dtype, C, ld, start):
    _say("fp8 strides", dtype, C, ld, start)
    base = torch.randn(9 * ld + 16, generator=_gen(C)).to(dtype).to(DEV)
    x = base[start:start + 9 * ld].view(9, ld)[:, :C]
    for tile in (False, True):
        codes, scales = _check(x, tile)
        out = torch.full((9 * ld + 16,), 77.0, dtype=dtype, device=DEV)
        y = out[start:start + 9 * ld].view(9, ld)[:, :C]
        P.fp8_dequant(codes, scales, out=y)
        assert torch.equal(y, P.fp8_dequant(codes, scales, dtype=dtype))
        y.fill_(77.0)
        assert (out == 77.0).all()               # nothing between the rows was written
    # codes into wider rows: what follows the next 16 bytes stays
    wide = (C + 15) // 16 * 16
    buf = torch.full((9, wide + 32), 0x55, dtype=torch.uint8, device=DEV)
    codes = buf.view(torch.float8_e4m3fn)[:, :C]
    scales = torch.empty(9, (C + 127) // 128, device=DEV)
    L.aaac_fp8_quantize(x, codes, scales)
    assert np.array_equal(_bytes(codes), ref.fp8_encode(x.double().cpu().numpy())[0])
    assert (buf[:, C:wide] == 0).all() and (buf[:, wide:] == 0x55).all()


def test_codes_on_any_address_are_read_back():
    _say("fp8 dequant addresses")
    x = torch.randn(7, 203, generator=_gen(9)).to(DEV)
    codes, scales = P.fp8_quantize(x)
    flat = torch.empty(7 * 203 + 5, dtype=torch.uint8, device=DEV)
    for at in (0, 1, 5):
        v = flat[at:at + 7 * 203].view(7, 203)
        v.copy_(codes.view(torch.uint8))
        got = P.fp8_dequant(v.view(torch.float8_e4m3fn), scales, dtype=torch.float32)
        assert torch.equal(got, P.fp8_dequant(codes, scales, dtype=torch.float32))


def test_stack_of_experts_is_its_matrices():
    W = torch.randn(3, 150, 70, generator=_gen(1)).to(torch.bfloat16).to(DEV)
    m = P.FP8Matrix.quantize(W)
    assert m.codes.shape == (3, 150, 70) and m.scales.shape == (3, 2, 1)
    for e in range(3):
        c, s = P.fp8_quantize(W[e], tile=True)
        assert np.array_equal(_bytes(m.codes[e]), _bytes(c)) and torch.equal(m.scales[e], s)
    assert torch.equal(m.dequant()[1], P.fp8_dequant(m.codes[1], m.scales[1]))
    part = P.FP8Matrix.quantize(W[:, 10:140, 3:67])  # matrices further apart than their rows
    c, s = P.fp8_quantize(W[2, 10:140, 3:67].contiguous(), tile=True)
    assert np.array_equal(_bytes(part.codes[2]), _bytes(c)) and torch.equal(part.scales[2], s)


def test_leading_axes_and_no_rows():
    x = torch.randn(2, 3, 5, 130, generator=_gen(3)).to(DEV)
    c, s = P.fp8_quantize(x)
    assert c.shape == x.shape and s.shape == (2, 3, 5, 2)
    c1, s1 = P.fp8_quantize(x[1, 2])
    assert np.array_equal(_bytes(c[1, 2]), _bytes(c1)) and torch.equal(s[1, 2], s1)
    assert torch.equal(P.fp8_dequant(c, s)[1, 2], P.fp8_dequant(c1, s1))
    for tile in (False, True):
        c, s = P.fp8_quantize(torch.empty(0, 40, device=DEV), tile=tile)
        assert c.shape == (0, 40) and s.shape == (0, 1) and P.fp8_dequant(c, s).shape == (0, 40)


# ------------------------------------------------------------------ products

def _whole(shape, gen, top=2):
    """Whole numbers up to `top` as e4m3: every sum of their products is exact in fp32."""
    return torch.randint(-top, top + 1, shape, generator=gen).float().to(torch.float8_e4m3fn)


def _aligned(codes, junk=None):
    """The codes on the GPU in rows of whole 16 bytes; junk: what the bytes behind a row hold."""
    C = codes.shape[-1]
    wide = (C + 15) // 16 * 16 + (16 if junk is not None else 0)
    buf = torch.full((*codes.shape[:-1], wide), junk or 0, dtype=torch.uint8)
    buf[..., :C] = codes.view(torch.uint8)
    return buf.to(DEV).view(torch.float8_e4m3fn)[..., :C]


def _pow2(shape, gen):
    return torch.exp2(torch.randint(-2, 3, shape, generator=gen).float())


def _offsets(E, T, gen):
    cut = torch.randint(0, T + 1, (E - 1,), generator=gen).sort().values
    return torch.cat([torch.zeros(1), cut.float(), torch.full((1,), float(T))]).int()


def _exact_case(E, R, C, T, dtype=torch.float32, tokens=None, junk=0x7f, grouped=None):
    """A product whose every term and sum is exact, compared bit for bit. E = 0: one matrix, no offsets.
    tokens: rows of x, picked by an index with some outside x. junk 0x7f: NaN codes behind the rows."""
    g = _gen(E, R, C, T)
    n = max(E, 1)
    wc, ws = _whole((n, R, C), g), _pow2((n, -(-R // 128), -(-C // 128)), g)
    Tx = tokens or T
    xc, xs = _whole((Tx, C), g), _pow2((Tx, -(-C // 128)), g)
    off = _offsets(E, T, g) if E else None
    rows = torch.randint(-1, Tx + 1, (T,), generator=g).int() if tokens else None
    wv = torch.stack([torch.from_numpy(ref.fp8_decode(wc[e].view(torch.uint8).numpy(), ws[e].numpy(), True))
                      for e in range(n)])
    xv = torch.from_numpy(ref.fp8_decode(xc.view(torch.uint8).numpy(), xs.numpy()))
    if tokens:
        ok = (rows >= 0) & (rows < Tx)
        xv = torch.where(ok[:, None], xv[rows.long().clamp(0, Tx - 1)], torch.zeros(()).double())
    want = torch.full((T, R), 55.0, dtype=torch.float64)
    for e in range(n):
        a, b = (int(off[e]), int(off[e + 1])) if E else (0, T)
        want[a:b] = xv[a:b] @ wv[e].t()
    assert want.abs().max() < 2 ** 19            # and every partial sum: 24 bits hold steps of 2^-4
    codes = _aligned(wc if E else wc[0], junk)
    out = torch.full((T, R), 55.0, dtype=dtype, device=DEV)
    y = P.fp8_matmul(codes, (ws if E else ws[0]).to(DEV), _aligned(xc, junk),
                     None if off is None else off.to(DEV), None if rows is None else rows.to(DEV),
                     xs.to(DEV), out)
    assert torch.equal(y.cpu(), want.float().to(dtype))


# (E, R, C, T): the few-row kernels and every tile, whole and short in every direction
FORMS = [(0, 16, 128, 1), (0, 1, 1, 1), (0, 40, 16, 16), (0, 129, 200, 7), (0, 4096, 256, 3), (0, 6000, 300, 5),
         (0, 12000, 130, 9), (0, 300, 1030, 32), (0, 12000, 260, 20), (0, 64, 128, 33), (0, 200, 4096, 40),
         (0, 8192, 384, 64), (0, 1000, 640, 100), (0, 515, 2048, 129), (0, 2048, 1031, 500),
         (0, 4096, 520, 777), (0, 4000, 896, 2000), (0, 4000, 1030, 2100), (0, 500, 8200, 1000),
         (0, 1500, 8200, 700), (0, 3000, 8000, 600), (0, 250, 6000, 8000), (0, 3000, 8000, 1500),
         (1, 256, 256, 5), (7, 130, 300, 40), (40, 64, 129, 200), (5, 200, 256, 300), (3, 1030, 272, 900),
         (4, 1030, 8200, 300), (8, 1500, 1031, 500), (20, 130, 4100, 1000), (9, 2048, 384, 3000),
         (64, 256, 128, 64), (0, 70, 2200, 33), (0, 515, 2100, 129), (0, 1000, 2090, 100), (5, 200, 2080, 300),
         (40, 64, 2100, 200), (0, 300, 260, 600)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,R,C,T", FORMS)
def test_products_of_whole_numbers_are_exact(E, R, C, T, dtype):
    _say("fp8 product", E, R, C, T, dtype, L.fp8_matmul_plan(max(E, 1), R, C, T, dtype=dtype))
    _exact_case(E, R, C, T, dtype)


@pytest.mark.parametrize("E,R,C,T,tokens", [(0, 64, 128, 5, 3), (0, 130, 260, 50, 9), (6, 130, 260, 50, 9),
                                            (4, 1030, 272, 900, 301), (8, 2048, 1040, 2048, 600)])
def test_rows_of_x_by_an_index(E, R, C, T, tokens):
    _say("fp8 rows", E, R, C, T, tokens, L.fp8_matmul_plan(max(E, 1), R, C, T))
    _exact_case(E, R, C, T, tokens=tokens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,R,C,T", [(0, 130, 300, 3), (0, 131, 300, 200), (4, 1000, 256, 700)])
def test_result_types(dtype, E, R, C, T):
    _exact_case(E, R, C, T, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_tile_and_kernel_is_reached(dtype):
    got = set()
    for E, R, C, T in FORMS:
        bm, bn, split, rt, _, _ = L.fp8_matmul_plan(max(E, 1), R, C, T, dtype=dtype)
        got.add((bm, bn, split > 1, rt))
    want = {(0, 0, False, rt) for rt in (1, 2, 4)}
    want |= {(64, 64, False, 0), (64, 64, True, 0), (128, 128, False, 0), (128, 128, True, 0), (128, 64, False, 0),
             (128, 64, True, 0)}
    if dtype is not torch.float32:               # fp32 results have no larger tile
        want |= {(256, 256, False, 0), (256, 256, True, 0)}
    assert want <= got, want - got


def _bound(xv, wv, dtype, want):
    """Half a step of the result, and the sums: 128 exact products a block, each addition rounded or cut to
    24 bits (2^-23 of the sum of magnitudes), the block's factor and its addition round once each, blocks
    and the parts of waves and workgroups (up to 64) add up in fp32. Results of 16 bits may come from the
    FP8 instruction, which adds eight products aligned to the largest: each may lose what lies below 2^-13
    of it, seven beside the largest at most, so 8 * 2^-13 of the magnitudes' sum."""
    blocks = -(-xv.shape[1] // 128)
    mag = xv.abs() @ wv.abs().t()
    cut = 0.0 if dtype is torch.float32 else 8 * 2.0 ** -13
    return EPS[dtype] * want.abs() + mag * (128 * 2.0 ** -23 + (blocks + 66) * 2.0 ** -24 + cut)


@pytest.mark.parametrize("xtype", TYPES)
@pytest.mark.parametrize("R,C,T", [(200, 130, 1), (1000, 4096, 5), (515, 1000, 100), (2048, 2048, 700)])
def test_quantized_in_the_call(xtype, R, C, T):
    _say("fp8 quantize in the call", xtype, R, C, T)
    g = _gen(R, C, T)
    x = (torch.randn(T, C, generator=g) * torch.exp(torch.randn(C, generator=g))).to(xtype)
    W = torch.randn(R, C, generator=g).mul_(0.02).to(torch.bfloat16)
    m = P.FP8Matrix.quantize(W.to(DEV))
    xv = torch.from_numpy(ref.fp8_decode(*ref.fp8_encode(x.double().numpy())))
    wv = torch.from_numpy(ref.fp8_decode(*ref.fp8_encode(W.double().numpy(), True), True))
    want = xv @ wv.t()
    for dt in TYPES:
        y = m.matmul(x.to(DEV), dtype=dt)
        off = (y.double().cpu() - want).abs()
        assert bool((off <= _bound(xv, wv, dt, want)).all()), float((off / _bound(xv, wv, dt, want)).max())
        # as a whole: half steps, and at most 2^-15 beside them (1.4e-5 measured for normal values)
        assert off.norm() <= (EPS[dt] + (0 if dt is torch.float32 else 2.0 ** -15)) * want.norm() + \
            (1e-6 * want.norm() if dt is torch.float32 else 0)
    # the same bits as the two calls
    codes, scales = P.fp8_quantize(x.to(DEV))
    assert torch.equal(m.matmul(codes, x_scales=scales, dtype=torch.float32), m.matmul(x.to(DEV), dtype=torch.float32))


@pytest.mark.parametrize("xtype", TYPES)
@pytest.mark.parametrize("E,R,C,tokens,n", [(0, 300, 4096, 8, 0), (0, 300, 4000, 3, 16), (6, 70, 200, 11, 0),
                                            (8, 130, 4096, 16, 0), (8, 4096, 4096, 16, 0), (9, 130, 3900, 5, 17),
                                            (20, 200, 1031, 300, 0), (8, 130, 264, 60, 400)])
def test_quantized_in_the_call_by_experts(xtype, E, R, C, tokens, n):
    """The same bits as the two calls, quantised by the product's own workgroups or before it. n: slots that
    pick their row of x, some outside x."""
    _say("fp8 quantize in the call", xtype, E, R, C, tokens, n)
    g = _gen(E, R, C, n)
    x = (torch.randn(tokens, C, generator=g) * torch.exp(torch.randn(C, generator=g))).to(xtype).to(DEV)
    m = P.FP8Matrix.quantize(torch.randn(*([E] if E else []), R, C, generator=g).mul_(0.02).to(DEV))
    codes, scales = P.fp8_quantize(x)
    for off in [_offsets(E, n or tokens, g), torch.tensor([0] * E + [n or tokens]).int()] if E else [None]:
        off = None if off is None else off.to(DEV)
        rows = torch.randint(-1, tokens + 1, (n,), generator=g).int().to(DEV) if n else None
        for dt in TYPES:
            got = m.matmul(x, off, rows, dtype=dt)
            assert torch.equal(got, m.matmul(codes, off, rows, x_scales=scales, dtype=dt))


def test_rows_far_apart():
    """Rows and matrices whose offsets pass 2^31 and 2^32 bytes."""
    g = _gen(55)
    far, R, C = (1 << 22) - 16, 1100, 200
    wide = torch.empty(2 * R * far, dtype=torch.uint8, device=DEV)
    w = wide.view(torch.float8_e4m3fn).as_strided((R, C), (far, 1))
    x = wide.view(torch.float8_e4m3fn)[R * far:].as_strided((R, C), (far, 1))
    w.view(torch.uint8).copy_(_whole((R, C), g).view(torch.uint8))
    x.view(torch.uint8).copy_(_whole((R, C), g).view(torch.uint8))
    ws, xs = _pow2((-(-R // 128), 2), g).to(DEV), _pow2((R, 2), g).to(DEV)
    assert R * far > 1 << 32
    y = torch.empty(R * far, dtype=torch.bfloat16, device=DEV).as_strided((R, R), (far, 1))
    wc, xc = _aligned(w.cpu(), 0x7f), _aligned(x.cpu(), 0x7f)
    for T in (5, 300, R):
        _say("fp8 far", T)
        want = P.fp8_matmul(wc, ws, xc[R - T:], x_scales=xs[R - T:])
        got = P.fp8_matmul(w, ws, x[R - T:], x_scales=xs[R - T:], out=y[R - T:])
        assert torch.equal(got, want)
    codes = wide.view(torch.float8_e4m3fn).as_strided((R, R), (far, 1))
    scales = torch.empty(R, -(-R // 128), device=DEV)
    L.aaac_fp8_quantize(y, codes, scales)
    cc, sc = P.fp8_quantize(y.contiguous())
    assert torch.equal(codes.view(torch.uint8), cc.view(torch.uint8)) and torch.equal(scales, sc)
    P.fp8_dequant(codes, scales, out=y)
    assert torch.equal(y, P.fp8_dequant(cc, sc))


def test_two_streams_at_once():
    """Calls that overlap do not share what they write."""
    _say("fp8 streams")
    g = _gen(91)
    W = P.FP8Matrix.quantize(torch.randn(512, 8192, generator=g).to(DEV))
    xs = [torch.randn(T, 8192, generator=g).to(DEV) for T in (3, 40, 200, 200)]
    want = [W.matmul(x) for x in xs]
    sides = [torch.cuda.Stream() for _ in xs]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in xs]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(sides, xs)):
            with torch.cuda.stream(s):
                got[i].append(W.matmul(x))
    torch.cuda.synchronize()
    for w, ys in zip(want, got):
        for y in ys:
            assert torch.equal(y, w)


def test_nan_blocks_reach_only_their_products():
    _say("fp8 nan")
    g = _gen(77)
    for T in (4, 90):
        x = torch.randn(T, 300, generator=g).to(DEV)
        W = torch.randn(200, 300, generator=g).to(DEV)
        x[1, 200] = float("nan")
        W[150, 3] = float("inf")                 # its tile: rows 128 .. 199
        y = P.FP8Matrix.quantize(W).matmul(x, dtype=torch.float32)
        bad = torch.zeros(T, 200, dtype=torch.bool)
        bad[1], bad[:, 128:] = True, True
        assert torch.equal(torch.isnan(y).cpu(), bad)


def test_rows_of_no_expert_are_left_alone_and_bad_offsets_stay_inside():
    _say("fp8 offsets")
    g = _gen(8)
    for T, R in ((30, 130), (600, 300)):
        W = P.FP8Matrix.quantize(torch.randn(3, R, 256, generator=g).to(DEV))
        x = torch.randn(T, 256, generator=g).to(DEV)
        off = torch.tensor([2, 5, 5, T - 4], dtype=torch.int32, device=DEV)
        out = torch.full((T, R), 9.0, device=DEV)
        W.matmul(x, off, out=out)
        one = [P.FP8Matrix(W.codes[e], W.scales[e]).matmul(x, dtype=torch.float32) for e in range(3)]
        assert (out[:2] == 9).all() and (out[T - 4:] == 9).all()
        torch.testing.assert_close(out[2:5], one[0][2:5], rtol=1e-5, atol=1e-4)
        torch.testing.assert_close(out[5:T - 4], one[2][5:T - 4], rtol=1e-5, atol=1e-4)
        for bad in ([-7, 3, 1 << 30, -1], [5, 2, 1, 0], [T + 9, T + 9, T + 9, T + 9]):
            guard = torch.full((T + 2, R), 9.0, device=DEV)
            W.matmul(x, torch.tensor(bad, dtype=torch.int32, device=DEV), out=guard[1:T + 1])
            assert (guard[0] == 9).all() and (guard[T + 1] == 9).all()


def test_results_do_not_depend_on_the_workspace_or_other_rows():
    g = _gen(4)
    W = P.FP8Matrix.quantize(torch.randn(1024, 4096, generator=g).to(DEV))
    x, xs = P.fp8_quantize(torch.randn(256, 4096, generator=g).to(DEV))
    need = L.fp8_matmul_workspace_bytes(1, 1024, 4096, 256, 256, False, torch.float32)
    y = [torch.empty(256, 1024, device=DEV) for _ in range(2)]
    for i, fill in enumerate((0, 0xFF)):
        ws = torch.full((max(need, 256),), fill, dtype=torch.uint8, device=DEV)
        L.aaac_fp8_matmul(W.codes, W.scales, x, y[i], x_scales=xs, ws=ws)
    assert torch.equal(y[0], y[1])


def test_strided_results_and_leading_axes():
    g = _gen(6)
    W = P.FP8Matrix.quantize(torch.randn(70, 200, generator=g).to(DEV))
    for T in (3, 80):
        x = torch.randn(T, 200, generator=g).to(DEV)
        y = W.matmul(x)
        buf = torch.full((T, 91), 7.0, dtype=torch.bfloat16, device=DEV)
        W.matmul(x, out=buf[:, 3:73])
        assert torch.equal(buf[:, 3:73], y) and (buf[:, :3] == 7).all() and (buf[:, 73:] == 7).all()
        assert torch.equal(W.matmul(x.view(1, T, 200)), y.view(1, T, 70))
        assert W.matmul(x[:0]).shape == (0, 70)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C,T", [(33, 300, 40), (515, 2100, 129), (192, 2100, 70), (1031, 2100, 700), (2049, 300, 777),
                                   (4001, 1030, 2100), (4224, 1030, 2050), (515, 8200, 300)])
def test_results_on_any_address(dtype, R, C, T):
    """Rows of y that start anywhere hold the same, and nothing beside them is touched."""
    _say("fp8 addresses", dtype, R, C, T, L.fp8_matmul_plan(1, R, C, T, dtype=dtype))
    g = _gen(R, C, T)
    W = P.FP8Matrix.quantize(torch.randn(R, C, generator=g).to(DEV))
    x, xs = P.fp8_quantize(torch.randn(T, C, generator=g).to(DEV))
    want = None
    for start, ld in ((0, (R + 7) // 8 * 8 + 8), (0, R + 3), (1, R + 4 + R % 2), (2, R + 5), (3, R + 3 + (R + 1) % 2)):
        buf = torch.full((T + 1, ld), 7.0, dtype=dtype, device=DEV)
        y = buf.view(-1)[start:start + T * ld].view(T, ld)[:, :R]
        W.matmul(x, x_scales=xs, out=y)
        want = y.clone() if want is None else want
        assert torch.equal(y, want)
        y.fill_(7.0)
        assert (buf == 7).all()


def test_on_another_stream_and_captured():
    _say("fp8 graph")
    g = _gen(2)
    W = P.FP8Matrix.quantize(torch.randn(2, 300, 512, generator=g).to(DEV))
    x = torch.randn(90, 512, generator=g).to(DEV)
    off = torch.tensor([0, 40, 90], dtype=torch.int32, device=DEV)
    rows = torch.randperm(90, generator=g).int().to(DEV)
    want = W.matmul(x, off, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = W.matmul(x, off, rows)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    graphs, outs = [], []
    for _ in range(2):                           # two graphs: each has its own workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(W.matmul(x, off, rows))
        graphs.append(gr)
    for i in range(3):
        x.normal_()
        want = W.matmul(x, off, rows)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_refusals_of_the_calls():
    W = P.FP8Matrix.quantize(torch.randn(64, 200, device=DEV))
    x = torch.randn(4, 200, device=DEV)
    with pytest.raises(ValueError, match="gradient"):
        W.matmul(x.clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        P.fp8_quantize(x.clone().requires_grad_())
    with pytest.raises(ValueError, match="columns"):
        W.matmul(torch.randn(4, 201, device=DEV))
    with pytest.raises(TypeError):
        W.matmul(x.double())
    with pytest.raises(TypeError):
        P.fp8_quantize(x.double())
    with pytest.raises(ValueError):              # codes without scales are no numbers
        W.matmul(P.fp8_quantize(x)[0], x_scales=torch.ones(4, 1, device=DEV))
    with pytest.raises(TypeError):
        W.matmul(P.fp8_quantize(x)[0])
    with pytest.raises(ValueError, match="every tensor must be on the GPU"):
        W.matmul(x.cpu())
    with pytest.raises(L.AAACError):             # rows of codes off 16 bytes
        flat = torch.zeros(64 * 200, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        P.fp8_matmul(flat.view(64, 200), W.scales, x)
    with pytest.raises(ValueError):
        P.fp8_dequant(W.codes, torch.ones(3, 3, device=DEV))
    with pytest.raises(ValueError):
        W.matmul(x, rows=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(L.AAACError):             # every row the same memory
        P.fp8_quantize(torch.zeros(1, 64, device=DEV).expand(4, 64))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,R,C,T", [(0, 64, 128, 5), (0, 70, 2100, 33), (0, 4096, 4096, 100), (0, 1024, 8192, 256),
                                     (0, 4000, 896, 2000), (8, 1500, 1031, 500), (40, 64, 2100, 200)])
def test_an_x_without_rows_is_rows_of_zeros(E, R, C, T, dtype):
    """Every index lies outside an x without rows: zeros where the offsets reach, whatever kernel an x with
    rows would take, and rows of no expert stay."""
    _say("fp8 no rows of x", E, R, C, T, dtype)
    g = _gen(E, R, C, T)
    n = max(E, 1)
    codes, ws = _aligned(_whole((n, R, C), g), 0x7f), _pow2((n, -(-R // 128), -(-C // 128)), g).to(DEV)
    if not E:
        codes, ws = codes[0], ws[0]
    off = torch.cat([torch.tensor([2]), _offsets(E, T, g)[1:-1].clamp(2, T - 1), torch.tensor([T - 1])]).int() if E else None
    want = torch.full((T, R), 55.0, dtype=dtype)
    want[slice(2, T - 1) if E else slice(0, T)] = 0.0
    rows = torch.randint(-2, 3, (T,), generator=g).int().to(DEV)
    off = None if off is None else off.to(DEV)
    none = torch.empty(0, -(-C // 128), device=DEV)
    for xt in TYPES:
        out = torch.full((T, R), 55.0, dtype=dtype, device=DEV)
        P.fp8_matmul(codes, ws, torch.empty(0, C, dtype=xt, device=DEV), off, rows, out=out)
        assert torch.equal(out.cpu(), want)
    out = torch.full((T, R), 55.0, dtype=dtype, device=DEV)
    P.fp8_matmul(codes, ws, torch.empty(0, C, dtype=torch.float8_e4m3fn, device=DEV), off, rows, none, out)
    assert torch.equal(out.cpu(), want)


def test_rows_outside_x_times_infinite_scales():
    """A row of zeros times a weight of infinite value is NaN in the few-row kernels and in the tiles, for codes
    as for rows that the call quantizes."""
    g = _gen(41)
    codes = _aligned(torch.ones(300, 2200).to(torch.float8_e4m3fn))
    scales = torch.ones(3, 18, device=DEV)
    scales[1, 2] = float("inf")
    x = torch.randn(7, 2200, generator=g).to(DEV)
    xc, xs = P.fp8_quantize(x)
    for T in (5, 100):
        assert (L.fp8_matmul_plan(1, 300, 2200, T)[0] == 0) == (T == 5)
        _say("fp8 infinite scales", T)
        rows = torch.randint(0, 7, (T,), generator=g).int()
        rows[1], rows[3] = -1, 7
        want = torch.zeros(2, 300)
        want[:, 128:256] = float("nan")
        for dt in TYPES:
            for kw in (dict(x=x), dict(x=xc, x_scales=xs)):
                y = P.fp8_matmul(codes, scales, rows=rows.to(DEV), dtype=dt, **kw)[[1, 3]].float().cpu()
                assert torch.equal(torch.isnan(y), torch.isnan(want)) and (y.nan_to_num(0.0) == 0).all()


@pytest.mark.parametrize("R,C,T", [(515, 4096, 5), (515, 4096, 100), (4096, 8192, 300), (2048, 2048, 700)])
def test_fp16_results_are_rounded_fp32_sums(R, C, T):
    """Results of 11 bits come from the same sums as fp32 ones: those rounded once, bit for bit."""
    _say("fp8 fp16", R, C, T, L.fp8_matmul_plan(1, R, C, T, dtype=torch.float16))
    g = _gen(R, C, T)
    W = P.FP8Matrix.quantize(torch.randn(R, C, generator=g).mul_(0.02).to(DEV))
    x = torch.randn(T, C, generator=g).to(DEV)
    assert torch.equal(W.matmul(x, dtype=torch.float16), W.matmul(x, dtype=torch.float32).half())
    assert L.fp8_matmul_plan(1, R, C, T, dtype=torch.float16) == L.fp8_matmul_plan(1, R, C, T, dtype=torch.float32)


def test_scales_with_a_gradient_are_refused():
    W = P.FP8Matrix.quantize(torch.randn(64, 200, device=DEV))
    x, xs = P.fp8_quantize(torch.randn(4, 200, device=DEV))
    ws = W.scales.clone().requires_grad_()
    for call in (lambda: P.fp8_matmul(W.codes, ws, x, x_scales=xs), lambda: P.fp8_dequant(W.codes, ws),
                 lambda: W.matmul(x, x_scales=xs.clone().requires_grad_()),
                 lambda: P.fp8_matmul(W.codes, ws, torch.randn(4, 200, device=DEV)),
                 lambda: P.fp8_matmul(W.codes.detach().requires_grad_(), W.scales, torch.randn(4, 200, device=DEV)),
                 lambda: P.fp8_matmul(W.codes, W.scales, x.detach().requires_grad_(), x_scales=xs),
                 lambda: P.fp8_dequant(W.codes.detach().requires_grad_(), W.scales),
                 lambda: P.fp8_dequant(x, xs.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(W.scales, torch.ones_like(W.scales))
        with pytest.raises(ValueError, match="tangent"):
            P.fp8_matmul(W.codes, dual, x, x_scales=xs)
        with pytest.raises(ValueError, match="tangent"):
            P.fp8_dequant(W.codes, dual)


def test_one_row_of_codes_between_others():
    """A single row's codes are padded to 16 bytes inside their own row only; where they have no such room the
    call is refused."""
    x = torch.randn(1, 100, generator=_gen(23)).to(DEV)
    scales = torch.empty(1, 1, device=DEV)
    buf = torch.full((9, 100), 0x55, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="16"):
        L.aaac_fp8_quantize(x, buf.view(torch.float8_e4m3fn)[4:5], scales)       # starts on 16 bytes
    assert (buf == 0x55).all()
    with pytest.raises(ValueError, match="16"):              # the row's padding would lie behind the storage
        L.aaac_fp8_quantize(x, torch.empty(100, dtype=torch.float8_e4m3fn, device=DEV).as_strided((1, 100), (112, 1)), scales)
    wide = torch.full((3, 128), 0x55, dtype=torch.uint8, device=DEV)
    L.aaac_fp8_quantize(x, wide.view(torch.float8_e4m3fn)[1:2, :100], scales)
    assert np.array_equal(wide[1:2, :100].cpu().numpy(), ref.fp8_encode(x.double().cpu().numpy())[0])
    assert (wide[1, 100:112] == 0).all() and (wide[1, 112:] == 0x55).all() and (wide[[0, 2]] == 0x55).all()
    for n in (96, 112):                                      # whole 16 bytes need no room
        L.aaac_fp8_quantize(x[:, :n] if n < 100 else torch.randn(1, n, device=DEV),
                            torch.empty(1, n, dtype=torch.float8_e4m3fn, device=DEV), scales)


def test_grids_of_two_rows():
    """More workgroups than one row of a grid holds: every tile of the result is there."""
    g = _gen(61)
    R, C, T = 64 * 1024 + 64, 16, 16 * 2048
    W, x = _whole((R, C), g), _whole((T, C), g)
    ws, xs = torch.ones(-(-R // 128), 1, device=DEV), torch.ones(T, 1, device=DEV)
    y = torch.full((T, R), 55.0, dtype=torch.bfloat16, device=DEV)
    _say("fp8 grid", L.fp8_matmul_plan(1, R, C, T))
    P.fp8_matmul(W.to(DEV), ws, torch.empty(0, C, device=DEV), rows=torch.zeros(T, dtype=torch.int32, device=DEV), out=y)
    assert not y.any()                           # (R / 64) (T / 16) workgroups, 2^21 and some
    P.fp8_matmul(W.to(DEV), ws, x.to(DEV), x_scales=xs, out=y)
    wf, xf = W.float().to(DEV), x.float().to(DEV)
    for t in range(0, T, 1024):                  # whole numbers up to 64
        assert torch.equal(y[t:t + 1024], (xf[t:t + 1024] @ wf.t()).to(torch.bfloat16))


def test_rows_do_not_depend_on_other_rows():
    """A result's row is the same whatever the other rows of x hold, in every kernel that a plan picks."""
    for E, R, C, T, dt in ((0, 515, 4096, 5, torch.bfloat16), (0, 515, 4096, 5, torch.float32), (0, 300, 260, 600, torch.bfloat16),
                           (0, 1024, 4096, 256, torch.bfloat16), (0, 1024, 4096, 256, torch.float16),
                           (0, 8192, 384, 64, torch.bfloat16), (0, 4000, 896, 2000, torch.bfloat16),
                           (0, 4000, 896, 2000, torch.float32), (4, 1030, 8200, 300, torch.bfloat16)):
        _say("fp8 other rows", E, R, C, T, dt, L.fp8_matmul_plan(max(E, 1), R, C, T, dtype=dt))
        g = _gen(E, R, C, T)
        W = P.FP8Matrix.quantize(torch.randn(*([E] if E else []), R, C, generator=g).to(DEV))
        off = _offsets(E, T, g).to(DEV) if E else None
        x = torch.randn(T, C, generator=g).to(DEV)
        other = torch.randn(T, C, generator=g).to(DEV) * 1000
        other[::7] = float("nan")
        for same in ([0], [T - 1], list(range(1, T, 2))):
            mixed = other.clone()
            mixed[same] = x[same]
            assert torch.equal(W.matmul(x, off, dtype=dt)[same], W.matmul(mixed, off, dtype=dt)[same])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,R,C,T", [(0, 70, 300, 5), (0, 8192, 384, 64), (0, 200, 4096, 40), (0, 1024, 8192, 256),
                                     (0, 4000, 896, 2000), (7, 130, 300, 40), (4, 1030, 8200, 300), (9, 2048, 384, 3000)])
def test_rows_by_an_index_are_copied_rows(E, R, C, T, dtype):
    """One row of x for all, few and many, in the few-row kernels, tiles and split tiles: the bits that copied
    rows give, zeros for indices outside x."""
    _say("fp8 index", E, R, C, T, dtype, L.fp8_matmul_plan(max(E, 1), R, C, T, dtype=dtype))
    g = _gen(E, R, C, T)
    W = P.FP8Matrix.quantize(torch.randn(*([E] if E else []), R, C, generator=g).to(DEV))
    off = _offsets(E, T, g).to(DEV) if E else None
    for tokens in (1, 3, T, 2 * T + 1):
        xc, xs = P.fp8_quantize(torch.randn(tokens, C, generator=g).to(DEV))
        rows = torch.randint(-1, tokens + 1, (T,), generator=g).int().to(DEV)
        rows[T // 2] = tokens - 1
        ok = ((rows >= 0) & (rows < tokens))[:, None]
        at = rows.long().clamp(0, tokens - 1)
        copied = _aligned((xc.view(torch.uint8)[at] * ok).view(torch.float8_e4m3fn).cpu())
        want = W.matmul(copied, off, x_scales=(xs[at] * ok).contiguous(), dtype=dtype)
        assert torch.equal(W.matmul(xc, off, rows, x_scales=xs, dtype=dtype), want)


def test_indexed_rows_reach_every_kind_of_plan():
    got = {(bm > 0, split > 1) for bm, _, split, *_ in (
        L.fp8_matmul_plan(max(E, 1), R, C, T) for E, R, C, T in (
            (0, 70, 300, 5), (0, 8192, 384, 64), (0, 200, 4096, 40), (0, 1024, 8192, 256), (0, 4000, 896, 2000),
            (7, 130, 300, 40), (4, 1030, 8200, 300), (9, 2048, 384, 3000)))}
    assert got == {(False, False), (True, False), (True, True)}
