"""Attention over an 8-bit cache whose values have the lowest powers: no key is left out beside larger ones."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hq,run", [(64, 4, 64), (128, 8, 32), (128, 16, 32), (64, 16, 64)])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("low", [7.0, 10.0, 14.0])
def test_many_keys_below_a_few(dtype, d, hq, run, new, low):
    """Keys whose values make the result weigh 2^-10, 2^-14 or 2^-20 of a few keys whose values are zero.

    One of those stands in every `run` of the first half of each 8 runs (a warp's block of keys, each warp's first and
    not its second).  bf16 results near its smallest normal number may be subnormals, rounded by half of 2^-133."""
    page, n = 64, 2048
    i = torch.arange(n)
    large = (i % (8 * run) < 4 * run) & (i % run == 5)

    def rows(b):
        k, v = torch.zeros(n, 1, d, dtype=torch.float64), torch.zeros(n, 1, d, dtype=torch.float64)
        k[:, 0, 0] = -low
        v[:, 0] = (1 + (i[:, None] + torch.arange(d)) % 8).double() * 2.0 ** (M.LEAST[dtype] + 5)
        k[large], v[large] = 0, 0
        return k, v

    kp, vp, ks, vs, table, k, v = M.paged8([n], page, 1, d, dtype, DEV, 1, rows=rows)
    assert bool((vs[table[0, :n // page].long()] == M.LEAST[dtype] + 127).all())
    q = torch.zeros(new, hq, d, dtype=dtype, device=DEV)
    q[:, :, 0] = 1
    out = kt.PagedKV8(kp, vp, ks, vs, dtype).attend(q, table, R.starts([new], DEV), torch.tensor(
        [n], dtype=torch.int32, device=DEV), new, scale=1.0)
    want, bound = R.attend(q, k, v, table, [new], [n], 1.0)
    off = (out.double().cpu() - want).abs()
    slack = 2.0 ** -134 if dtype == torch.bfloat16 else 0.0
    assert bool((off <= bound + slack).all()), f"{float((off / want.abs()).max()):.3e} of the result"
