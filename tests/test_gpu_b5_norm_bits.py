"""A token's norm is the same bits whatever else is in the step: large steps against the same rows in small ones."""
import pytest
import torch

import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,h", [(4200, 1056), (2000, 2336), (1100, 4096), (700, 7168), (600, 8192), (40, 8224),
                                 (3000, 1024), (3000, 288)])
def test_rows_of_large_steps_and_small_ones(dtype, n, h):
    """Steps of more than 2^22 elements and parts of them below that (the last three: sizes with one form for all)."""
    g = torch.Generator(device=DEV).manual_seed(n)
    x, r = (torch.randn(n, h, generator=g, device=DEV).to(dtype) for _ in range(2))
    w = 1 + 0.1 * torch.randn(h, generator=g, device=DEV)
    y, s, mx = kt.add_rms_norm(x, w, r, mx=True)
    parts = [(0, n // 3), (n // 3, n // 2), (n // 2, n - 5), *((i, i + 1) for i in range(n - 5, n))]
    for lo, hi in parts:
        py, ps, pm = kt.add_rms_norm(x[lo:hi], w, r[lo:hi], mx=True)
        for whole, part in ((y, py), (s, ps), (mx[0], pm[0]), (mx[1], pm[1])):
            assert torch.equal(whole[lo:hi], part)
