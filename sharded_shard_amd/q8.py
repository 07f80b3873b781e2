"""Training in 8 bits: matrices with a power of two for each block of 128, their
products, and linear layers that keep their input in 8 bits for the backward
pass.

A ``Q8`` holds the codes (E4M3 or E5M2) and one E8M0 byte for each block of a
matrix; a code stands for code * 2^(byte - 127).  Blocks are 1 x 128 ("rows"),
128 x 1 ("cols") or 128 x 128 ("tiles"); a product's sum runs along its
operands' blocks.  Weights come gathered, from ``ShardedGroup.full_q8``;
``quantize`` makes the others.  torch only allocates memory; the arithmetic is
in the HIP kernels behind the C ABI.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import capi

FORMATS = {"e4m3": capi.FSDP_Q8_E4M3, "e5m2": capi.FSDP_Q8_E5M2}
BLOCKS = {"tensor": capi.FSDP_Q8_TENSOR, "rows": capi.FSDP_Q8_ROWS, "cols": capi.FSDP_Q8_COLS,
          "tiles": capi.FSDP_Q8_TILES}
_DTYPES = {torch.bfloat16: capi.FSDP_DTYPE_BF16, torch.float32: capi.FSDP_DTYPE_F32}
_HALF = (torch.bfloat16, torch.int16)      # the groups hold bf16 bits as int16
_BYTES = (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _known(table: dict, name: str, what: str) -> int:
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(map(repr, table))}, not {name!r}")
    return table[name]


def scale_lines(rows: int, cols: int, blocks: str):
    """(lines, bytes a line) of the scales of a [rows, cols] matrix."""
    if rows == 0 or cols == 0 or blocks == "tensor":
        return 0, 0
    down, across = _up(rows, 128) // 128, _up(cols, 128) // 128
    return {"rows": (across, rows), "cols": (down, cols), "tiles": (down, across)}[blocks]


def _rows_of(t: torch.Tensor, what: str, dtypes) -> int:
    """The leading dimension of a GPU matrix whose rows are contiguous."""
    if t.dim() != 2 or t.dtype not in dtypes:
        raise ValueError(f"{what}: a matrix of {' or '.join(str(d) for d in dtypes)} is needed, "
                         f"not {tuple(t.shape)} of {t.dtype}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what} is on {t.device}, not on the current GPU")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row must follow each other")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows overlap")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


class Q8:
    """A matrix in 8 bits.  ``codes`` [rows, cols] of uint8 (or a float8 dtype),
    rows contiguous; ``scales`` uint8, one line for each 128 of the matrix as
    ``scale_lines`` says, or None with blocks "tensor"; ``divisor``: one fp32 on
    the GPU by which values are divided (the FP8 copy-in's per-parameter scale).
    It is a view: it keeps the tensors, and reads them when it is used."""

    def __init__(self, codes: torch.Tensor, scales: Optional[torch.Tensor], blocks: str,
                 format: str = "e4m3", divisor: Optional[torch.Tensor] = None):
        kind, fmt = _known(BLOCKS, blocks, "blocks"), _known(FORMATS, format, "format")
        ld = _rows_of(codes, "codes", _BYTES)
        self.rows, self.cols = codes.shape
        lines, length = scale_lines(self.rows, self.cols, blocks)
        pitch = 0
        if lines:
            if scales is None:
                raise ValueError(f"blocks {blocks!r} have scales")
            pitch = _rows_of(scales, "scales", (torch.uint8,))
            if scales.shape[0] < lines or scales.shape[1] < length:
                raise ValueError(f"scales must hold {lines} lines of {length} bytes, "
                                 f"not {tuple(scales.shape)}")
        if divisor is not None:
            if divisor.dtype != torch.float32 or divisor.numel() != 1:
                raise ValueError("divisor: one fp32 is needed")
            capi._dev(divisor, 4, "divisor")
        self.codes, self.scales, self.divisor = codes, scales, divisor
        self.blocks, self.format = blocks, format
        self.device = codes.device
        self.c = capi.Q8Struct(codes.data_ptr(), scales.data_ptr() if lines else 0,
                               divisor.data_ptr() if divisor is not None else 0,
                               self.rows, self.cols, ld, pitch, fmt, kind)

    @classmethod
    def empty(cls, shape, blocks: str, format: str = "e4m3", device="cuda") -> "Q8":
        """Memory for a matrix of this shape, laid out so that products read it in
        place."""
        rows, cols = shape
        _known(BLOCKS, blocks, "blocks")
        if blocks == "tensor":
            raise ValueError("blocks must have scales")
        ld = _up(cols, 16)
        lines, length = scale_lines(rows, cols, blocks)
        pitch = _up(length, 16)
        # one piece of memory: the codes, then the scales
        both = torch.empty(rows * ld + lines * pitch, dtype=torch.uint8, device=device)
        codes = both[:rows * ld].view(rows, ld)[:, :cols]
        return cls(codes, both[rows * ld:].view(lines, pitch)[:, :length] if lines else both[:0].view(0, 0),
                   blocks, format)

    @property
    def shape(self):
        return self.rows, self.cols

    def codes_view(self) -> torch.Tensor:
        """The codes, uint8 [rows, cols]."""
        return self.codes.view(torch.uint8)

    def scales_view(self) -> torch.Tensor:
        """The scales' bytes: [columns / 128, rows], [rows / 128, columns] or, of
        tiles, [rows / 128, columns / 128], rounded up."""
        lines, length = scale_lines(self.rows, self.cols, self.blocks)
        return self.scales[:lines, :length]

    def nbytes(self) -> int:
        lines, length = scale_lines(self.rows, self.cols, self.blocks)
        return self.rows * self.cols + lines * length


def _here(*qs: Q8) -> None:
    for q in qs:
        if q.device.index != torch.cuda.current_device():
            raise ValueError(f"the 8-bit matrix is on {q.device}, not on the current device "
                             f"cuda:{torch.cuda.current_device()}")


def _on(stream):
    """The context in which memory is taken for work on `stream`: torch hands it out
    again in the order of the stream that it was taken on."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def quantize(x: torch.Tensor, blocks: str = "rows", format: str = "e4m3", out=None, stream=None):
    """``x`` [rows, cols] bf16 or fp32 in 8 bits.  blocks "both": a pair, along rows
    (what x W^T reads) and along columns (the checkpoint for the weight
    gradient), in one pass over x.  ``out``: a Q8 (or a pair) to write."""
    pair = blocks == "both"
    if not pair:
        _known(BLOCKS, blocks, "blocks")
    _known(FORMATS, format, "format")
    ldx = _rows_of(x, "x", _DTYPES)
    if out is None:
        kinds = ("rows", "cols") if pair else (blocks,)
        if stream is None:
            out = [Q8.empty(x.shape, k, format, x.device) for k in kinds]
        else:
            with _on(stream):
                out = [Q8.empty(x.shape, k, format, x.device) for k in kinds]
    else:
        out = list(out) if pair else [out]
        _here(*out)
        for q, k in zip(out, ("rows", "cols") if pair else (blocks,)):
            if q.shape != tuple(x.shape) or q.blocks != k or q.format != format:
                raise ValueError(f"out must be {tuple(x.shape)} in blocks {k!r} of {format}")
    capi.fsdp_q8_quantize(x.data_ptr(), _DTYPES[x.dtype], ldx, out[0].c,
                          out[1].c if pair else None, stream)
    return tuple(out) if pair else out[0]


def _result(shape, dtype, device, out, stream, dtypes):
    if out is None:
        if stream is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        else:
            with _on(stream):
                out = torch.empty(shape, dtype=dtype, device=device)
    elif tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {tuple(shape)}, not {tuple(out.shape)}")
    return out, _rows_of(out, "out", dtypes)


def dequantize(q: Q8, dtype: torch.dtype = torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """What ``q`` stands for, in bf16 or fp32."""
    _here(q)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    out, ldo = _result(q.shape, dtype, q.device, out, stream, (dtype,))
    capi.fsdp_q8_dequantize(q.c, out.data_ptr(), _DTYPES[dtype], ldo, stream)
    return out


def product(a: Q8, b: Q8, trans_a: bool = False, trans_b: bool = False, out=None, workspace=None,
            stream=None) -> torch.Tensor:
    """op(a) op(b) in bf16, with fp32 sums: x W^T (trans_b), dy W, dy^T x (trans_a).
    ``workspace``: a uint8 tensor for it, by default memory of the stream; calls
    that share one must follow each other."""
    _here(a, b)
    ta, tb = int(trans_a), int(trans_b)
    need = capi.fsdp_q8_product_workspace(a.c, ta, b.c, tb)
    shape = a.cols if trans_a else a.rows, b.rows if trans_b else b.cols
    out, ldo = _result(shape, torch.bfloat16, a.device, out, stream, _HALF)
    if need and workspace is None:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
        else:
            with _on(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
    capi.fsdp_q8_product(a.c, ta, b.c, tb, out.data_ptr(), ldo, workspace, 0, stream)
    return out


class Linear8:
    """A linear layer in 8 bits: y = x W^T of the gathered FP8 ``weight``, which keeps
    its input as 8-bit codes with a scale for each 128 tokens and channel (half
    the memory of bf16), and the gradients from those.

    ``forward`` keeps the checkpoint of its input; ``backward`` uses the oldest one
    and lets go of it, so microbatches run first in, first out.  ``grad_format``:
    "e4m3" or "e5m2" (more range, one bit less) for dy."""

    def __init__(self, weight: Q8, grad_format: str = "e4m3"):
        if weight.blocks not in ("tiles", "tensor"):
            raise ValueError("the weight must be in blocks of 128 x 128, or in none")
        if weight.format != "e4m3":
            raise ValueError("the weight must be E4M3")
        _known(FORMATS, grad_format, "grad_format")
        self.weight, self.grad_format = weight, grad_format
        self.saved = []

    def forward(self, x: torch.Tensor, out=None, save: bool = True, stream=None) -> torch.Tensor:
        """``x`` [tokens, in] bf16 or fp32 -> [tokens, out] bf16.  save: keep the 8-bit
        checkpoint (not for evaluation)."""
        if x.dim() != 2 or x.shape[1] != self.weight.cols:
            raise ValueError(f"x must be [tokens, {self.weight.cols}], not {tuple(x.shape)}")
        if save:
            rows, cols = quantize(x, "both", stream=stream)
        else:
            rows, cols = quantize(x, "rows", stream=stream), None
        y = product(rows, self.weight, trans_b=True, out=out, stream=stream)
        if save:
            self.saved.append(cols)
        return y

    def backward(self, dy: torch.Tensor, dweight: torch.Tensor, out=None,
                 stream=None) -> torch.Tensor:
        """``dy`` [tokens, out] -> dx [tokens, in] bf16; ``dweight`` [out, in] bf16 (the
        group's full gradient) is written."""
        if not self.saved:
            raise RuntimeError("backward without a saved forward")
        x = self.saved[0]
        if tuple(dy.shape) != (x.rows, self.weight.rows):
            raise ValueError(f"dy must be {(x.rows, self.weight.rows)}, not {tuple(dy.shape)}")
        rows, cols = quantize(dy, "both", self.grad_format, stream=stream)
        dx = product(rows, self.weight, out=out, stream=stream)
        product(cols, x, trans_a=True, out=dweight, stream=stream)
        self.saved.pop(0)
        return dx
