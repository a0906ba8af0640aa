"""64-bit statements of what the 8-bit operators store: MXFP8 rows, and e4m3 blocks of a key/value cache."""
import torch

import attn_oracle as R

BLOCK = 16
# Scale exponents of a cache whose values are numbers of the type: code * 2^X is exact in it.
LEAST, MOST = {torch.bfloat16: -117, torch.float16: -14}, {torch.bfloat16: 119, torch.float16: 7}


def e4m3(v):
    """The e4m3 number nearest to each of v (64 bits), ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def half_step(v):
    """Half the distance of e4m3 numbers around |v| (of the coarser side at a power of two)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6, max=448.0))) - 4)


def numbers(codes):
    return codes.view(torch.float8_e4m3fn).double()


def power(scales):
    return torch.exp2(scales.double() - 127)


def off_by_a_rounding(codes, scale, v, off):
    """How far |code * scale - v| is over what one rounding allows of a value that is off by at most `off`.

    A rounding to nearest is off by half a step of the numbers around (v + off) / scale; values beyond 448 saturate."""
    got = codes * scale
    edge = 448 * scale
    inside = torch.minimum(v.abs() + off, edge.expand_as(v))
    allowed = half_step(inside / scale) * scale + off + (v.abs() - edge).clamp(min=0)
    return (got - v).abs() - allowed


def rms_rows(x, residual, weight, eps):
    """(s, y) in 64 bits and the fp32 error of y before its rounding.

    fp32 steps: the residual's addition (1 rounding), a thread's at most 32 squares and sums, 5 shuffles and at most 32
    warps (their error halved by the root), the root (2 units) and three products: fewer than 64 roundings of y."""
    s = x.double().cpu()
    if residual is not None:
        s = s + residual.double().cpu()
    y = s / torch.sqrt(s.pow(2).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    return s, y, 64 * R.F32 * y.abs()


def floor_exponent(top):
    """OCP's shared exponent: floor(log2 top) - 8 (top > 0)."""
    return torch.floor(torch.log2(top)) - 8
