"""Attention whose bounded waits run out: told, over, and without consequence for the next call.

The test hook lets the first CTA withhold its first load of keys (nothing is loaded, nothing is signalled) and bounds
every wait by 50 ms.  No wait lasts longer, and no load is left in flight."""
import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
TIMEOUTS = kt.KT_DEVERR_TIMEOUT_LOAD | kt.KT_DEVERR_TIMEOUT_MMA | kt.KT_DEVERR_TIMEOUT_EPI


def _withheld_call_between_two(seqs, new, past, hq, hk, d, dtype):
    page, n = 64, new + past
    pages = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(1)
    kp, vp = (torch.randn(seqs * pages, page, hk, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    table = torch.randperm(seqs * pages, generator=g, device=DEV).to(torch.int32).view(seqs, pages)
    q = torch.randn(seqs * new, hq, d, generator=g, device=DEV).to(dtype)
    args = (q, table, R.starts([new] * seqs, DEV), torch.full((seqs,), n, dtype=torch.int32, device=DEV), new)
    cache = kt.PagedKV(kp, vp)
    ws = cache.workspace()
    want = cache.attend(*args, workspace=ws)
    assert cache.read_error() == 0
    kt.debug_configure(50_000, kt.KT_DEBUG_WITHHOLD_STAGE)
    try:
        cache.attend(*args, workspace=ws)
        code = cache.read_error()
    finally:
        kt.debug_configure()
    assert code & TIMEOUTS and not code & ~TIMEOUTS, hex(code)
    assert not bool(ws[:A.WORKSPACE_ZEROED].any()), "counters are left behind"
    for _ in range(2):
        assert torch.equal(cache.attend(*args, workspace=ws), want)
    assert cache.read_error() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float16, 128)])
@pytest.mark.parametrize("seqs,past", [(1, 20000), (1, 40), (400, 700)])
def test_few_rows(seqs, past, dtype, d):
    """One sequence cut over many CTAs, one that one CTA has, and more than there are CTAs, some cut."""
    _withheld_call_between_two(seqs, 1, past, 8, 1, d, dtype)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float16, 128)])
@pytest.mark.parametrize("seqs,new,past,hq", [(1, 40, 20000, 8), (1, 20, 40, 8), (3, 500, 300, 8), (20, 300, 0, 5)])
def test_chunks(seqs, new, past, hq, dtype, d):
    """Items that many CTAs share, that one has, and runs of several items, the last ones cut."""
    _withheld_call_between_two(seqs, new, past, hq, 1, d, dtype)
