"""The norm between the blocks of a decoder layer (C ABI: ``include/kt_norm.h``).

``add_rms_norm`` adds the residual to the hidden states and norms them, in front
of the attention's projection and of the MoE layer, whose tokens it can write in
MXFP8.  The arithmetic runs in the library's CUDA kernel: this module checks
tensors, allocates outputs and passes pointers and the CUDA stream.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import attention as _a

_VP, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "kt_add_rms_norm": ([_VP, _VP, _VP, _I, _F, _I, _I, _I, _VP, _VP, _VP, _VP, _VP], _I),
}
MAX_HIDDEN = 32768   # KT_NORM_MAX_HIDDEN

TOKEN_ROWS = "Pq"    # kt_token_rows: ptr, token_stride
_ROWS_BYTES = struct.calcsize(TOKEN_ROWS)
_CALL = struct.Struct(4 * TOKEN_ROWS)
_NO_ROWS = (0, 0)


def _rows(t, name: str, dtype, device: int, shape):
    """(ptr, token stride) of a [tokens, hidden] tensor with contiguous rows on CUDA device `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{device}" if device >= 0 else "a CUDA device"))
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    by_token, by_element = t.stride()
    n, h = shape
    if by_element != 1 and h != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous, strides are {t.stride()}")
    return t.data_ptr(), (by_token if n > 1 else h)   # the stride of a dimension of one entry says nothing


def _bytes(t, name: str, device: int, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.uint8:
        raise TypeError(f"{name} must be torch.uint8, got {t.dtype}")
    if t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} on cuda:{device}")
    return t.data_ptr()


def _empty_mx(x, n: int, h: int, stream):
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty_mx(x, n, h, None)
    return (torch.empty((n, h), dtype=torch.uint8, device=x.device),
            torch.empty((n, h // 32), dtype=torch.uint8, device=x.device))


def _apart(outs, ins, n: int, h: int):
    """Refuse outputs that share memory with another output, or with an input whose rows are not their own.

    outs, ins: (name, ptr, row stride in bytes, row bytes); outputs may be the input of the same pointer and stride."""
    if n == 0 or h == 0:
        return

    def meet(a, b):
        (_, pa, sa, wa), (_, pb, sb, wb) = a, b
        if pa + (n - 1) * sa + wa <= pb or pb + (n - 1) * sb + wb <= pa:
            return False
        if sa == sb and sa > 0:                            # side by side in one buffer's rows
            between = (pb - pa) % sa
            return not wa <= between <= sa - wb
        return True

    for i, o in enumerate(outs):
        if n > 1 and o[2] < o[3]:
            raise ValueError(f"{o[0]}: its rows overlap")
        for x in outs[:i]:
            if meet(o, x):
                raise ValueError(f"{o[0]} shares memory with {x[0]}")
        for x in ins:
            if o[1:] != x[1:] and meet(o, x):
                raise ValueError(f"{o[0]} shares memory with {x[0]}")


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 plain: bool = True, mx: bool = False, out: torch.Tensor | None = None,
                 residual_out: torch.Tensor | None = None, mx_out: tuple | None = None, stream=None):
    """s = x + residual and y = s * weight / sqrt(mean(s^2) + eps) of each token, in one launch; returns
    (y, s, (codes, scales)).

    x, residual: bf16 or fp16 [tokens, hidden], rows by any stride that is a multiple of 8; weight [hidden] of their
    type or float32; all 16-byte aligned.  y is there with `plain` (x's type; None without), s with a residual (x's
    type), the pair with `mx`: y in MXFP8, codes uint8 e4m3 [tokens, hidden] and scales uint8 e8m0 [tokens,
    hidden / 32], as forward and MoeLayer take them in place of bf16 tokens (rounded once, from the fp32 y).  hidden: a
    multiple of 8 (of 32 with mx) up to 32768.  Squares are summed in fp32: where their sum passes 3.4e38, y is zeros
    (with eps 0, where it vanishes, not finite).  A token's bits do not depend on the call's other tokens.

    out and residual_out may be x or residual; they share no memory otherwise."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _a.DTYPE_CODES or x.dim() != 2:
        raise TypeError("x must be a bf16 or fp16 tensor [tokens, hidden]")
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    dev, dt, shape = x.get_device(), x.dtype, x.shape
    n, h = shape
    rx = _rows(x, "x", dt, dev, shape)
    w = _a._weight(weight, "weight", dt, h, dev)
    rr = ro = ry = _NO_ROWS
    codes = scales = None
    given = []                                             # outputs that the caller brings
    if residual is not None:
        rr = _rows(residual, "residual", dt, dev, shape)
        if residual_out is None:
            residual_out = _a._output(x, stream)
            ro = (residual_out.data_ptr(), h)
        else:
            ro = _rows(residual_out, "residual_out", dt, dev, shape)
            given.append(("residual_out", ro[0], 2 * ro[1], 2 * h))
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if plain:
        if out is None:
            out = _a._output(x, stream)
            ry = (out.data_ptr(), h)
        else:
            ry = _rows(out, "out", dt, dev, shape)
            given.append(("out", ry[0], 2 * ry[1], 2 * h))
    elif out is not None:
        raise ValueError("out needs plain=True")
    if mx:
        if h % 32:
            raise ValueError(f"hidden={h} must be a multiple of 32 for MXFP8")
        if mx_out is None:
            mx_out = _empty_mx(x, n, h, stream)
            codes, scales = mx_out[0].data_ptr(), mx_out[1].data_ptr()
        else:
            codes = _bytes(mx_out[0], "mx_out[0]", dev, (n, h))
            scales = _bytes(mx_out[1], "mx_out[1]", dev, (n, h // 32))
            given += [("mx_out[0]", codes, h, h), ("mx_out[1]", scales, h // 32, h // 32)]
    elif mx_out is not None:
        raise ValueError("mx_out needs mx=True")
    if given:
        ins = [("x", rx[0], 2 * rx[1], 2 * h), ("weight", w, 0, weight.element_size() * h)]
        if residual is not None:
            ins.append(("residual", rr[0], 2 * rr[1], 2 * h))
        _apart(given, ins, n, h)
    b = _a._buffer
    _CALL.pack_into(b.buf, 0, *rx, *rr, *ro, *ry)
    at = b.at
    _a._call(dev, stream, "kt_add_rms_norm", at, at + _ROWS_BYTES, w, _a.DTYPE_CODES.get(weight.dtype, _a.KT_DTYPE_F32),
             eps, n, h, _a.DTYPE_CODES[dt], at + 2 * _ROWS_BYTES, at + 3 * _ROWS_BYTES, codes, scales)
    return (out if plain else None), (residual_out if residual is not None else None), (tuple(mx_out) if mx else None)
