"""Products on 4-bit weights for any number of rows, dense and grouped by expert, and the MXFP4 format.

Two weight formats take part: the packed dual-codebook format of the quantizer (`QuantizedMatrix`,
`PackedExperts`) and MXFP4 (`MXFP4Matrix`, one matrix or a stack of experts). Rows of x that belong
to experts are sorted by expert and described by `offsets`, int32 [E + 1] on the device: expert e has
the rows offsets[e] <= t < offsets[e + 1]. The weights are frozen: nothing here has a gradient.

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
