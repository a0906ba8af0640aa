"""Rows at the ends of the norm's range, every element of every output."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,small", [(torch.bfloat16, 2.0 ** -126), (torch.float16, 2.0 ** -24)])
@pytest.mark.parametrize("h", [256, 7168])
def test_rows_of_every_kind(dtype, small, h):
    """Zeros, the smallest numbers, large ones, NaN, infinity, and an ordinary row between them."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(7, h, generator=g).to(dtype)
    x[0] = 0
    x[1] = (small * (1 + torch.arange(h) % 5)).to(dtype)
    x[2] = (x[2].float() * (1e15 if dtype == torch.bfloat16 else 1e4)).to(dtype)
    x[3, 5] = float("nan")
    x[4, 7], x[4, h - 1] = float("inf"), -float("inf")
    x = x.to(DEV)
    w = 1 + torch.randn(h, generator=g).mul(0.1).to(DEV)
    y, s, mx = kt.add_rms_norm(x, w, torch.zeros_like(x), mx=True)
    torch.testing.assert_close(s, x, rtol=0, atol=0, equal_nan=True)
    assert not bool(y[0].any()) and not bool(mx[0][0].any()) and not bool(mx[1][0].any())
    rows = [1, 2, 5, 6]
    _, want, off = M.rms_rows(x[rows], None, w, 1e-6)
    assert bool(((y[rows].double().cpu() - want).abs()
                 <= R.ROUND[dtype] * (want.abs() + off) + off + R.TINY[dtype]).all())
    codes, scales = M.numbers(mx[0][rows].cpu()), mx[1][rows].cpu()
    top, slack = (t.reshape(len(rows), -1, 32).amax(-1) for t in (want.abs(), off))
    e = scales.double() - 127
    # exponents end at -127, and at 2^-118 the largest element has that one
    low, high = (M.floor_exponent(t.clamp(min=2.0 ** -119)).clamp(min=-127) for t in (top - slack, top + slack))
    assert bool(((e >= low) & (e <= high)).all())
    scale = torch.exp2(e).repeat_interleave(32, -1)
    assert float(M.off_by_a_rounding(codes, scale, want, off).max()) <= 0
    # a root of NaN, and one of infinity: x / infinity is 0, infinity / infinity is NaN
    assert bool(y[3].isnan().all()) and bool(((mx[0][3] & 0x7f) == 0x7f).all())
    odd = x[4].isinf()
    assert bool(y[4][odd].isnan().all()) and not bool(y[4][~odd].any())
    assert bool(((mx[0][4][odd] & 0x7f) == 0x7f).all()) and not bool((mx[0][4][~odd] & 0x7f).any())
