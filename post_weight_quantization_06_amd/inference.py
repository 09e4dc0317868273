"""Products on 4-bit and 8-bit weights for any number of rows, dense and grouped by expert, the MXFP4
and FP8 formats, and the routing of rows to experts.

Three weight formats take part: the packed dual-codebook format of the quantizer (`QuantizedMatrix`,
`PackedExperts`), MXFP4 (`MXFP4Matrix`) and FP8 with a scale for each block of 128 (`FP8Matrix`), the last
two for one matrix or a stack of experts. Rows of x that belong to experts are sorted by expert and
described by `offsets`, int32 [E + 1] on the device: expert e has the rows offsets[e] <= t <
offsets[e + 1]. `route` makes them from a router's logits; its result moves rows to that order and back.
The weights are frozen: nothing here has a gradient.

Every call enqueues its kernels on the current stream of the tensors' device and returns.
"""

from __future__ import annotations

import dataclasses
from typing import Optional, Sequence, Tuple

import torch

from . import _lib as L


def mxfp4_quantize(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """MXFP4 codes u8 [..., Cp/2] and scale bytes u8 [..., Cp/32] of x [..., C] (bf16, fp16 or fp32),
    Cp = 32 ceil(C / 32): blocks of 32 along the last axis, two codes per byte."""
    lead, C = x.shape[:-1], x.shape[-1]
    x2 = x if x.dim() == 2 else x.reshape(-1, C)
    blocks = (C + 31) // 32
    codes = torch.empty(*lead, blocks * 16, dtype=torch.uint8, device=x.device)
    scales = torch.empty(*lead, blocks, dtype=torch.uint8, device=x.device)
    L.aaac_mxfp4_quantize(x2, codes, scales)
    return codes, scales


def _last_axis(out: torch.Tensor, n: int):
    """A result's rows are those of its last axis; one of another length would be filled out of order."""
    if out.dim() == 0 or out.shape[-1] != n:
        raise ValueError("out must be [..., %d] (got %s)" % (n, list(out.shape)))


def mxfp4_dequant(codes: torch.Tensor, scales: torch.Tensor, C: int,
                  dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values [..., C] of MXFP4 codes, in `out` (then of its type) or a new tensor of `dtype`."""
    if out is None:
        out = torch.empty(*codes.shape[:-1], C, dtype=dtype, device=codes.device)
    _last_axis(out, C)
    L.aaac_mxfp4_dequant(codes, scales, out if out.dim() == 2 else out.view(-1, C))
    return out


def _rows_of(x: torch.Tensor, R: int, out: Optional[torch.Tensor], dtype: torch.dtype):
    """(x as rows, output as rows, output) for x [..., C]."""
    if out is None:
        out = torch.empty(*x.shape[:-1], R, dtype=dtype, device=x.device)
    if x.dim() == 2:
        return x, out, out                       # the binding compares their shapes
    _last_axis(out, R)
    return x.reshape(-1, x.shape[-1]), out.view(-1, R), out


def mxfp4_matmul(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                 offsets: Optional[torch.Tensor] = None, act: str = "bf16",
                 out: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.bfloat16, C: Optional[int] = None) -> torch.Tensor:
    """[..., R] = x [..., C] times the transposed MXFP4 matrix (codes [R, Cp/2]), or with offsets
    each row times its expert's (codes [E, R, Cp/2]). act "bf16": x bf16 as it is; "mxfp4": x (bf16,
    fp16 or fp32) is quantized to MXFP4 first and the product is one of 4-bit values. Without `out`,
    rows outside the offsets hold nothing defined; with it they stay as they were.

    C: the width that the weights were quantized at, to refuse an x of another one. Codes hold whole
    blocks of 32 columns, so without C an x of any width with as many blocks is multiplied, its missing
    columns as zeros and those past the weights' width by zeros (MXFP4Matrix knows its C)."""
    K = x.shape[-1]
    if C is None:
        C = K
    elif C != K:
        raise ValueError("x has %d columns, the weights %d" % (K, C))
    x2, y2, out = _rows_of(x, codes.shape[-2], out, dtype)
    if act == "bf16":
        L.aaac_mxfp4_matmul(codes, scales, C, x2, y2, offsets)
    elif act == "mxfp4":
        L.aaac_mxfp4_matmul(codes, scales, C, x2, y2, offsets, None, L.QUANTIZE_X)
    else:
        raise ValueError("act must be 'bf16' or 'mxfp4' (got %r)" % (act,))
    return out


def packed_matmul(codes: torch.Tensor, scales: torch.Tensor, bitmap: Optional[torch.Tensor],
                  tables_bf16: torch.Tensor, x: torch.Tensor, g: int, S: int, n: int,
                  offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """[..., R] = x bf16 [..., C] times the transposed packed matrix, as aaac_dequant reads it; with
    offsets each row times its expert's (every weight tensor stacked along a first axis)."""
    x2, y2, out = _rows_of(x, codes.shape[-2], out, dtype)
    L.aaac_matmul(codes, scales, bitmap, tables_bf16, g, S, n, x2, y2, offsets)
    return out


@dataclasses.dataclass
class MXFP4Matrix:
    """One weight matrix in MXFP4, or a stack of experts."""
    C: int
    codes: torch.Tensor          # uint8 [R, Cp/2] or [E, R, Cp/2]
    scales: torch.Tensor         # uint8 [R, Cp/32] or [E, R, Cp/32]

    @classmethod
    def quantize(cls, W: torch.Tensor) -> "MXFP4Matrix":
        """W [R, C], or [E, R, C] for a stack of experts."""
        if W.dim() not in (2, 3):
            raise ValueError("W must be [R, C] or [E, R, C]")
        return cls(W.shape[-1], *mxfp4_quantize(W))

    def dequant(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return mxfp4_dequant(self.codes, self.scales, self.C, dtype)

    def matmul(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None, act: str = "bf16",
               out: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """x times the transposed matrix (see mxfp4_matmul)."""
        return mxfp4_matmul(self.codes, self.scales, x, offsets, act, out, dtype, self.C)


@dataclasses.dataclass
class PackedExperts:
    """The packed dual-codebook matrices of E experts, stacked."""
    g: int
    S: int
    n: int
    codes: torch.Tensor          # uint8 [E, R, C/2]
    scales: torch.Tensor         # int16 [E, R, C/g]
    bitmap: Optional[torch.Tensor]  # uint8 [E, ceil(R C / S / 8)] when S < g
    tables_bf16: torch.Tensor    # int16 [E, 2, n]

    @classmethod
    def stack(cls, experts: Sequence) -> "PackedExperts":
        """Stack QuantizedMatrix results of one shape and one (g, S, n)."""
        q0 = experts[0]
        key = (q0.R, q0.C, q0.g, q0.S, q0.n)
        for i, q in enumerate(experts):
            if (q.R, q.C, q.g, q.S, q.n) != key:
                raise ValueError("expert %d has (R, C, g, S, n) = %s, expert 0 %s" % (
                    i, (q.R, q.C, q.g, q.S, q.n), key))
        return cls(q0.g, q0.S, q0.n,
                   torch.stack([q.codes.view(q.R, q.C // 2) for q in experts]),
                   torch.stack([q.scales.view(q.R, q.C // q.g) for q in experts]),
                   None if q0.bitmap is None else torch.stack([q.bitmap for q in experts]),
                   torch.stack([q.tables_bf16.view(2, q.n) for q in experts]))

    def matmul(self, x: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """Each row of x times its expert's transposed matrix (see packed_matmul)."""
        return packed_matmul(self.codes, self.scales, self.bitmap, self.tables_bf16, x, self.g,
                             self.S, self.n, offsets, out, dtype)


def fp8_quantize(x: torch.Tensor, tile: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """FP8 codes (float8_e4m3fn, shaped as x) and fp32 scales of x (bf16, fp16 or fp32): a scale for each
    128 columns of a row, [..., ceil(C/128)]; with tile for each 128 x 128 of a matrix [R, C] or a stack
    [E, R, C], [..., ceil(R/128), ceil(C/128)]. Rows of codes start on 16 bytes, as the products need
    them: for a C that is no multiple of 16 the result is a view of wider rows."""
    dev = L._on_gpu("fp8_quantize", x)
    lead, C = x.shape[:-1], x.shape[-1]
    wide, blocks = (C + 15) // 16 * 16, (C + 127) // 128
    codes = torch.empty(*lead, wide, dtype=torch.float8_e4m3fn, device=x.device)
    if tile:
        if len(lead) not in (1, 2):
            raise ValueError("tile needs [R, C] or [E, R, C] (got %d-D)" % x.dim())
        scales = torch.empty(*lead[:-1], (lead[-1] + 127) // 128, blocks, dtype=torch.float32,
                             device=x.device)
        L._fp8_quantize(x, codes, wide, scales, True, dev)
    else:
        scales = torch.empty(*lead, blocks, dtype=torch.float32, device=x.device)
        L._fp8_quantize(x if len(lead) == 1 else x.reshape(-1, C), codes, wide, scales, False, dev)
    return (codes if wide == C else codes[..., :C]), scales


def fp8_dequant(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of FP8 codes, in `out` (then of its type) or a new tensor of `dtype`. The scales' shape
    says whether they are those of rows or of tiles (fp8_quantize)."""
    *lead, C = shape = codes.shape
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=codes.device)
    elif out.shape != shape:
        raise ValueError("out must be shaped as the codes (got %s and %s)" % (tuple(out.shape), tuple(shape)))
    blocks = (C + 127) // 128
    if scales.shape == (*lead, blocks):
        flat = len(lead) == 1
        L.aaac_fp8_dequant(codes if flat else codes.view(-1, C), scales, out if flat else out.view(-1, C))
    elif len(lead) in (1, 2) and scales.shape == (*lead[:-1], (lead[-1] + 127) // 128, blocks):
        L.aaac_fp8_dequant(codes, scales, out, True)
    else:
        raise ValueError("scales %s fit neither the rows nor the tiles of codes %s" % (
            tuple(scales.shape), tuple(codes.shape)))
    return out


def fp8_matmul(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
               x_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """[..., R] = x [..., C] times the transposed FP8 matrix (codes [R, C], scales of its tiles), or with
    offsets each row times its expert's (codes [E, R, C]). x is bf16, fp16 or fp32 and is quantized first,
    or codes with x_scales from fp8_quantize. rows: int32 [T], the result's row t multiplies row rows[t]
    of x [Tx, C] (a routing's `rows`: tokens need not be copied to their experts; rows outside x stand
    for zeros). Without `out`, rows outside the offsets hold nothing defined; with it they stay as they
    were. fp32 and fp16 results are fp32 sums; bf16 ones come faster from sums of fewer bits, off by a
    hundredth of what the rounding to bf16 is (aaac.h)."""
    if rows is not None:
        if x.dim() != 2:
            raise ValueError("with rows, x must be [Tx, C] (got %d-D)" % x.dim())
        if out is None:
            out = torch.empty(rows.shape[0], codes.shape[-2], dtype=dtype, device=x.device)
        x2, y2 = x, out
    else:
        x2, y2, out = _rows_of(x, codes.shape[-2], out, dtype)
    L.aaac_fp8_matmul(codes, scales, x2, y2, offsets, rows, x_scales)
    return out


@dataclasses.dataclass
class FP8Matrix:
    """One weight matrix in FP8 with a scale for each tile of 128 x 128, or a stack of experts."""
    codes: torch.Tensor          # float8_e4m3fn [R, C] or [E, R, C], rows on 16 bytes
    scales: torch.Tensor         # float32 [ceil(R/128), ceil(C/128)] or [E, .., ..]

    @classmethod
    def quantize(cls, W: torch.Tensor) -> "FP8Matrix":
        """W [R, C], or [E, R, C] for a stack of experts."""
        return cls(*fp8_quantize(W, tile=True))

    def dequant(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return fp8_dequant(self.codes, self.scales, dtype)

    def matmul(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
               rows: Optional[torch.Tensor] = None, x_scales: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """x times the transposed matrix (see fp8_matmul)."""
        return fp8_matmul(self.codes, self.scales, x, offsets, rows, x_scales, out, dtype)


@dataclasses.dataclass
class Routing:
    """Which experts T tokens go to, and the places of their rows in expert order. `route` makes experts, weights,
    rows and places as parts of one tensor: one that is kept holds the memory of all four, and one that is saved
    or has to outlive the others is cloned first."""
    experts: torch.Tensor        # int32 [T, k], best first, -1 where none is left
    weights: torch.Tensor        # float32 [T, k], 0 there
    offsets: torch.Tensor        # int32 [E + 1]: expert e has the places offsets[e] .. offsets[e + 1] - 1
    rows: torch.Tensor           # int32 [T k]: the token of each place, -1 behind the last expert's
    places: torch.Tensor         # int32 [T, k]: the place of each slot, -1 without an expert

    def to_experts(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """[T k, C]: the rows of x [T, C] in expert order (see rows_to_experts)."""
        return rows_to_experts(x, self.places, out)

    def from_experts(self, y: torch.Tensor, out: Optional[torch.Tensor] = None,
                     dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """[T, C]: each token's weighted sum of its experts' rows of y [T k, C]."""
        return rows_from_experts(y, self.places, self.weights, out, dtype)


def route(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          groups: int = 1, top_groups: Optional[int] = None, group_top: int = 1,
          renormalize: bool = True, scale: float = 1.0) -> Routing:
    """The k best of E experts for each token of logits [T, E] (bf16, fp16 or fp32).

    Scores are softmax(logits) over the experts or sigmoid(logits). Experts are chosen by score + bias
    (fp32 [E], for balance), weighted by the score alone: divided by its sum over the chosen ones with
    renormalize, times scale. With groups, the experts form that many groups of neighbours, and only the
    top_groups (default: all) with the largest best value (group_top 1) or sum of the two best (2) take
    part. Equals go to the lowest index. An expert whose logit or bias is -inf is left out, whatever the
    other is, so a row of -inf (a padded batch's) gets no expert; the type's lowest value is a number like
    any other."""
    if not isinstance(k, int) or k < 1:
        raise ValueError("k must be a positive whole number (got %r)" % (k,))
    inputs = L._route_inputs(logits, bias, score)
    T, E, dev = inputs[2], inputs[3], logits.device
    # one tensor's parts: 0.6 us of a call less than tensors of their own
    experts, places, rows, weights = torch.empty(4, T, k, dtype=torch.int32, device=dev).unbind(0)
    r = Routing(experts, weights.view(torch.float32), torch.empty(E + 1, dtype=torch.int32, device=dev),
                rows.view(-1), places)
    L._route(inputs, logits, k, experts, r.weights, r.offsets, rows, places, score, bias, groups,
             top_groups, group_top, renormalize, scale)
    return r


def rows_to_experts(x: torch.Tensor, places: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T k, C] with out[places[t, j]] = x[t], x [T, C] of any type of up to 4 bytes. Without `out`,
    rows that no place names hold nothing defined; with it they stay as they were."""
    if out is None:
        out = torch.empty(places.numel(), x.shape[-1], dtype=x.dtype, device=x.device)
    L.aaac_rows_to_experts(x, places, out)
    return out


def rows_from_experts(y: torch.Tensor, places: torch.Tensor, weights: torch.Tensor,
                      out: Optional[torch.Tensor] = None,
                      dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """[T, C] = the sum over j of weights[t, j] y[places[t, j]], in `out` or a new tensor of `dtype`
    (default: y's). Places of -1 add nothing."""
    if out is None:
        out = torch.empty(places.shape[0], y.shape[-1], dtype=dtype or y.dtype, device=y.device)
    L.aaac_rows_from_experts(y, places, weights, out)
    return out
