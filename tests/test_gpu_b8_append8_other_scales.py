"""Appends to blocks whose scale another program wrote, below and above the powers that an append picks."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,byte", [(torch.float16, 127 + 8), (torch.float16, 127 + 13), (torch.float16, 254),
                                        (torch.float16, 127 - 20), (torch.float16, 0), (torch.bfloat16, 127 + 88),
                                        (torch.bfloat16, 253), (torch.bfloat16, 254), (torch.bfloat16, 127 - 118),
                                        (torch.bfloat16, 0)])
@pytest.mark.parametrize("older", [1, 5, 15])
def test_older_tokens_keep_their_numbers(dtype, byte, older):
    """A larger power than an append picks is kept, codes and all; a smaller one grows, and its codes are rescaled."""
    hk, d, page, new = 2, 64, 16, 20
    lens = [older + new]
    kp, vp, ks, vs, table, _, _ = M.paged8(lens, page, hk, d, dtype, DEV, 1)
    first = int(table[0, 0])
    ks[first], vs[first] = byte, byte
    before = [t.cpu().clone() for t in (kp, vp)]
    # some numbers that the larger powers hold; 16-bit types end below the largest of them
    size = min(2.0 ** (byte - 127), 2.0 ** 124 if dtype == torch.bfloat16 else 100.0) if byte > 127 else 1.0
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(new, hk, d, generator=g).mul(size).to(dtype).to(DEV) for _ in range(2))
    cache = kt.PagedKV8(kp, vp, ks, vs, dtype)
    cache.append(k, v, table, R.starts([new], DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert cache.read_error() == 0
    room = M.BLOCK - older
    for rows, codes, scales, had in ((k, kp, ks, before[0]), (v, vp, vs, before[1])):
        rows = rows[:room].double().cpu()
        top = rows.abs().amax(dim=(0, 2))
        x = torch.maximum(M.least_exponent(top, dtype), torch.full_like(top, byte - 127))
        assert torch.equal(scales[first, 0].double().cpu() - 127, x)
        got = M.numbers(codes[first].cpu())
        moved = M.e4m3(M.numbers(had[first, :older]) * torch.exp2(byte - 127 - x)[:, None])
        assert torch.equal(got[:older], moved), "older tokens"
        assert torch.equal(got[older:], M.e4m3(rows * torch.exp2(-x)[:, None])), "new tokens"
