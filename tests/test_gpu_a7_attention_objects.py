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


def test_outputs_that_share_memory_are_refused():
    """Before anything is launched: nothing is written."""
    n, hq, hk, d, page = 6, 4, 2, 64, 16
    qkv = torch.randn(n, hq + 2 * hk, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    q, k, v = qkv.split((hq, hk, hk), dim=1)
    before, w = qkv.clone(), torch.ones(d, device=DEV)
    kp, vp = (torch.zeros(2, page, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = kt.PagedKV(kp, vp)
    step = (torch.zeros(1, 1, dtype=torch.int32, device=DEV), R.starts([n], DEV),
            torch.full((1,), n, dtype=torch.int32, device=DEV))
    inside = kp.view(-1, hq, d)[:n]
    for out in (qkv[:, 1:1 + hq], qkv[:, hk:hk + hq], qkv.view(-1, hq, d)[:n]):
        with pytest.raises(ValueError, match="q_out"):
            kt.qk_norm_rope(q, k, q_weight=w, q_out=out)
        with pytest.raises(ValueError, match="q_out"):
            cache.append(k, v, *step, q=q, q_out=out)
        with pytest.raises(ValueError, match="out"):
            cache.attend(q, *step, n, out=out)
    with pytest.raises(ValueError, match="k_out"):
        kt.qk_norm_rope(q, k, q_weight=w, k_out=q[:, :hk])
    with pytest.raises(ValueError, match="q_out"):
        cache.append(k, v, *step, q=q, q_out=inside)
    with pytest.raises(ValueError, match="out"):
        cache.attend(q, *step, n, out=inside)
    torch.cuda.synchronize()
    assert torch.equal(qkv, before) and not bool(kp.any())


@pytest.mark.parametrize("new,past,seqs", [(1, 5000, 1), (1, 70, 400), (90, 3000, 1), (300, 0, 9)])
def test_attention_in_place_of_the_queries(new, past, seqs):
    """The same bits as into another tensor, pieces of sequences joined or not."""
    hq, hk, d, page, n = 8, 2, 64, 32, new + past
    pages = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(2)
    kp, vp = (torch.randn(seqs * pages, page, hk, d, generator=g, device=DEV).to(torch.float16) for _ in range(2))
    qkv = torch.randn(seqs * new, hq + 2 * hk, d, generator=g, device=DEV).to(torch.float16)
    q, rest = qkv[:, :hq], qkv[:, hq:].clone()
    args = (torch.arange(seqs * pages, dtype=torch.int32, device=DEV).view(seqs, pages), R.starts([new] * seqs, DEV),
            torch.full((seqs,), n, dtype=torch.int32, device=DEV), new)
    cache = kt.PagedKV(kp, vp)
    want = cache.attend(q, *args)
    assert cache.attend(q, *args, out=q) is q
    assert torch.equal(q, want) and torch.equal(qkv[:, hq:], rest) and cache.read_error() == 0


def test_caches_share_a_stream_s_workspace():
    """One for all the layers of a model; another stream has its own; the last cache takes it along."""
    d, page, n = 64, 16, 3000
    pages = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(3)
    made = [[torch.randn(pages, page, 1, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
            for _ in range(4)]
    q = torch.randn(70, 4, d, generator=g, device=DEV).to(torch.bfloat16)
    step = (torch.arange(pages, dtype=torch.int32, device=DEV)[None], R.starts([70], DEV),
            torch.full((1,), n, dtype=torch.int32, device=DEV), 70)
    ws = kt.PagedKV(*made[0]).workspace()
    want = [kt.PagedKV(*kv).attend(q, *step, workspace=ws) for kv in made]
    size = ws.numel()
    torch.cuda.synchronize()
    start = torch.cuda.memory_allocated()
    caches = [kt.PagedKV(*kv) for kv in made]
    out = torch.empty_like(q)
    for _ in range(2):
        for cache, w in zip(caches, want):
            assert torch.equal(cache.attend(q, *step, out=out), w)
    assert size <= torch.cuda.memory_allocated() - start < 2 * size
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    caches[0].attend(q, *step, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.cuda.memory_allocated() - start >= 2 * size
    del caches, cache
    assert torch.cuda.memory_allocated() - start < size
