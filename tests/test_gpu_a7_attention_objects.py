"""What a cache object keeps on the device, across streams: its error word, its workspaces."""
import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _busy(stream, products=300):
    """Some tens of milliseconds of work on the stream."""
    with torch.cuda.stream(stream):
        a = torch.zeros(4096, 4096, device=DEV, dtype=torch.bfloat16)
        for _ in range(products):
            a = a @ a


def test_error_word_is_clear_before_any_stream_uses_it():
    """A cache made on a stream with work ahead, and used at once on another: the bit that is set there stays."""
    kp, vp = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    bt, cu = torch.full((1, 1), 9, dtype=torch.int32, device=DEV), R.starts([1], DEV)
    lens = torch.ones(1, dtype=torch.int32, device=DEV)
    maker, user = torch.cuda.Stream(), torch.cuda.Stream()
    _busy(maker)                                             # (the library is loaded, the pool has grown)
    torch.cuda.synchronize()
    kt.PagedKV(kp, vp).append(k, k, bt, cu, lens, stream=user)
    torch.cuda.synchronize()
    _busy(maker)
    with torch.cuda.stream(maker):
        cache = kt.PagedKV(kp, vp)
    cache.append(k, k, bt, cu, lens, stream=user)            # page 9 of 2
    torch.cuda.synchronize()
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    assert cache.read_error() == 0
