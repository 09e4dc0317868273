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
