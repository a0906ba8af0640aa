"""Norm and rotation of heads, and the append to a paged cache: what a refused token leaves as it was."""
import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d,rot", [(64, 64), (72, 8)])
def test_append_of_a_position_outside_the_table_writes_nothing(d, rot):
    """Neither key, value nor query of such a token is stored; its neighbours' are."""
    page = 16
    g = torch.Generator().manual_seed(1)
    kp, vp = (torch.randn(3, page, 2, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    k, v = (torch.randn(4, 2, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(4, 6, d, generator=g).to(torch.bfloat16).to(DEV)
    before_k, before_v = kp.clone(), vp.clone()
    q_out = torch.full_like(q, 3.0)
    cache = kt.PagedKV(kp, vp)
    # sequence 0 appends at 6 and 7 (the table's last), then 8; sequence 1 at 20
    cu, lens = R.starts([3, 1], DEV), torch.tensor([9, 21], dtype=torch.int32, device=DEV)
    bt = torch.tensor([[2, -1], [0, 1]], dtype=torch.int32, device=DEV)
    cache.append(k, v, bt, cu, lens, kt.rope_table(8, rot), q=q, q_out=q_out)
    assert cache.read_error() == A.KT_DEVERR_BAD_POSITION
    assert torch.equal(vp[2, 6:8], v[:2]) and not torch.equal(kp[2, 6:8], before_k[2, 6:8])
    assert bool((q_out[:2] != 3.0).any(-1).all()) and bool((q_out[2:] == 3.0).all())
    for now, before in ((kp, before_k), (vp, before_v)):
        now[2, 6:8] = before[2, 6:8]
        assert torch.equal(now, before)
