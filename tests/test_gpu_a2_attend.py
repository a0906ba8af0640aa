"""Attention over a paged cache against the 64-bit statement: head layouts, lengths, masks, pages, streams."""
import math
import random

import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def _run(q_lens, past, hq, hk, d, dtype, page=16, layout="slots", window=0, sinks=None, scale=None, seed=0, qscale=2.0,
         max_q=None):
    lens = [a + b for a, b in zip(q_lens, past)]
    kp, vp, table = R.paged(lens, page, hk, d, dtype, DEV, seed, layout)
    n = sum(q_lens)
    q = _rand(n, hq, d, dtype=dtype, seed=seed + 1, scale=qscale)
    cache = kt.PagedKV(kp, vp)
    scale = R.softmax_scale(d) if scale is None else scale
    out = torch.full((n, hq, d), 9.0, dtype=dtype, device=DEV)
    cache.attend(q, table, R.starts(q_lens, DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                 max(q_lens + [0]) if max_q is None else max_q, scale=scale, window=window, sinks=sinks, out=out)
    assert cache.read_error() == 0
    want, bound = R.attend(q, kp, vp, table, q_lens, lens, scale, window, sinks)
    off = (out.double().cpu() - want).abs()
    assert bool(torch.isfinite(out).all()), "not finite"
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound, worst {float(off.max()):.3e}"
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 8), (4, 4, 64), (8, 1, 128), (12, 4, 96), (5, 1, 80), (40, 2, 64),
                                     (16, 1, 128), (34, 2, 72), (128, 1, 64)])
def test_single_tokens(dtype, hq, hk, d):
    _run([1, 1, 1, 1, 1], [0, 1, 15, 16, 130], hq, hk, d, dtype, page=16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,layout", [(16, "slots"), (48, "heads"), (64, "pairs"), (128, "heads"), (256, "slots")])
def test_pages(dtype, page, layout):
    _run([1, 3, 1, 2], [0, 61, 300, 126], 6, 2, 64, dtype, page=page, layout=layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,past,hq,hk,d,page", [
    ([64], [0], 8, 1, 128, 16),
    ([129, 0, 1, 33], [0, 5, 70, 100], 10, 2, 64, 32),
    ([70], [200], 6, 2, 96, 64),
    ([300, 1], [17, 400], 2, 2, 128, 16),
    ([31, 32, 33], [1, 0, 127], 16, 2, 80, 128),
    ([200], [60], 3, 1, 64, 48),
    ([9, 8], [0, 3], 128, 1, 128, 16),
])
def test_chunks(dtype, q_lens, past, hq, hk, d, page):
    _run(q_lens, past, hq, hk, d, dtype, page=page)


@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 72, 104, 120])
def test_chunks_of_other_head_sizes(d):
    _run([45, 3], [30, 100], 9, 3, d, torch.float16, page=16)


def test_expanded_queries():
    """Queries of stride zero (one head for all, one token for all)."""
    n, d = 40, 64
    kp, vp, table = R.paged([n + 9], 16, 1, d, torch.bfloat16, DEV, 5)
    one_head = _rand(n, 1, d, dtype=torch.bfloat16, seed=1).expand(n, 4, d)
    one_token = _rand(1, 4, d, dtype=torch.bfloat16, seed=2).expand(n, 4, d)
    for q in (one_head, one_token):
        out = kt.PagedKV(kp, vp).attend(q, table, R.starts([n], DEV),
                                        torch.tensor([n + 9], dtype=torch.int32, device=DEV), n)
        want, bound = R.attend(q, kp, vp, table, [n], [n + 9], R.softmax_scale(d))
        assert bool(((out.double().cpu() - want).abs() <= bound).all())


@pytest.mark.parametrize("seed", range(24))
def test_drawn_batches(seed):
    """Batches of mixed lengths, pages, heads, windows and sinks."""
    r = random.Random(seed)
    seqs = r.choice((1, 2, 5, 9))
    q_lens = [r.choice((0, 1, 1, r.randint(1, 20), r.randint(1, 90))) for _ in range(seqs)]
    q_lens[0] = max(q_lens[0], 1)
    past = [r.choice((0, r.randint(0, 40), r.randint(0, 300))) for _ in range(seqs)]
    hk = r.choice((1, 2, 3))
    hq = hk * r.choice((1, 2, 5, 8))
    sinks = torch.randn(hq, generator=torch.Generator().manual_seed(seed)).to(DEV) if r.random() < 0.5 else None
    _run(q_lens, past, hq, hk, r.choice((32, 64, 80, 128)), r.choice((torch.bfloat16, torch.float16)),
         page=r.choice((16, 32, 80, 128)), layout=r.choice(("slots", "heads", "pairs")),
         window=r.choice((0, 0, r.randint(1, 200))), sinks=sinks, seed=seed, max_q=r.choice((1, max(q_lens))))


def test_many_sequences_of_chunks():
    g = torch.Generator().manual_seed(2)
    b = 600
    past = torch.randint(0, 50, (b,), generator=g).tolist()
    q_lens = torch.randint(0, 4, (b,), generator=g).tolist()
    _run(q_lens, past, 2, 1, 32, torch.float16, max_q=100)


@pytest.mark.parametrize("new", [1, 70])
def test_calls_that_share_a_workspace(new):
    """Consecutive calls of different sizes on one workspace, each as if alone; a short workspace is refused."""
    d, page = 64, 16
    cases = []
    for length in (5000, 90, 2000):
        pages = -(-(length + new) // page)
        kp, vp = (_rand(pages, page, 1, d, dtype=torch.bfloat16, seed=length + i) for i in (0, 1))
        table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
        args = (_rand(new, 4, d, dtype=torch.bfloat16, seed=7), table, R.starts([new], DEV),
                torch.tensor([length + new], dtype=torch.int32, device=DEV), new)
        c = kt.PagedKV(kp, vp)
        cases.append((c, args, c.attend(*args)))
    ws = cases[0][0].workspace()
    outs = [c.attend(*args, workspace=ws) for c, args, _ in cases for _ in range(2)]
    for i, (_, _, want) in enumerate(cases):
        assert torch.equal(outs[2 * i], want) and torch.equal(outs[2 * i + 1], want)
    assert not bool(ws[:A.WORKSPACE_ZEROED].any())
    with pytest.raises(kt.KTError, match="workspace"):
        cases[0][0].attend(*cases[0][1], workspace=ws[:4096])
    with pytest.raises((TypeError, ValueError)):
        cases[0][0].attend(*cases[0][1], workspace=ws.view(torch.int32))


@pytest.mark.parametrize("window", [1, 2, 16, 60, 64, 129, 10_000])
@pytest.mark.parametrize("q_lens,past", [([1, 1], [200, 3]), ([150, 7], [100, 0])])
def test_windows(window, q_lens, past):
    _run(q_lens, past, 4, 1, 64, torch.bfloat16, page=32, window=window)


@pytest.mark.parametrize("q_lens,past", [([1, 1], [40, 300]), ([130], [10])])
def test_sinks(q_lens, past):
    sinks = torch.tensor([0.0, -math.inf, 30.0, -30.0, 3.0, 1.0], device=DEV)
    _run(q_lens, past, 6, 2, 128, torch.float16, sinks=sinks)
    _run(q_lens, past, 6, 2, 128, torch.bfloat16, sinks=sinks, window=5)


@pytest.mark.parametrize("scale,qscale", [(1.0, 3.0), (1e-3, 1.0), (0.125, 40.0)])
@pytest.mark.parametrize("q_lens,past", [([1], [700]), ([140], [60])])
def test_scales(scale, qscale, q_lens, past):
    """Peaked, flat, and very large logits."""
    _run(q_lens, past, 2, 1, 64, torch.bfloat16, scale=scale, qscale=qscale)


@pytest.mark.parametrize("max_q", [0, 1, 10_000])
def test_bound_on_new_tokens_is_a_hint(max_q):
    _run([3, 150, 1], [20, 30, 90], 4, 2, 64, torch.bfloat16, max_q=max_q)


@pytest.mark.parametrize("q_lens,lens", [([3, 1, 2], [1, 0, 2]), ([150, 2], [140, 0])])
def test_tokens_that_see_nothing(q_lens, lens):
    """Lengths shorter than the new tokens: those before position 0 see no key and get zeros."""
    d, page = 64, 16
    kp, vp, table = R.paged(lens, page, 1, d, torch.bfloat16, DEV, 1)
    q = _rand(sum(q_lens), 4, d, dtype=torch.bfloat16, seed=2)
    for sinks in (None, torch.zeros(4, device=DEV), torch.full((4,), -math.inf, device=DEV)):
        cache = kt.PagedKV(kp, vp)
        out = torch.full_like(q, 9.0)
        cache.attend(q, table, R.starts(q_lens, DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), max(q_lens),
                     sinks=sinks, out=out)
        want, bound = R.attend(q, kp, vp, table, q_lens, lens, R.softmax_scale(d), 0, sinks)
        assert bool(((out.double().cpu() - want).abs() <= bound).all())
        assert bool((out[0] == 0).all())


def test_keys_that_are_not_finite():
    """A NaN or infinite key past what a token sees does not reach it."""
    d, page = 64, 16
    lens = [100]
    for new in (4, 60):
        kp, vp, table = R.paged(lens, page, 1, d, torch.bfloat16, DEV, 1)
        last = int(table[0, 6])
        kp[last, 3] = float("nan")                            # position 99
        kp[last, 2] = float("inf")                            # position 98
        q = _rand(new, 2, d, dtype=torch.bfloat16, seed=2)
        out = kt.PagedKV(kp, vp).attend(q, table, R.starts([new], DEV),
                                        torch.tensor(lens, dtype=torch.int32, device=DEV), new)
        want, bound = R.attend(q, kp, vp, table, [new], lens, R.softmax_scale(d))
        ok = slice(0, new - 2)
        assert bool(((out[ok].double().cpu() - want[ok]).abs() <= bound[ok]).all())
        assert bool(out[new - 1].isnan().all())


@pytest.mark.parametrize("new", [1, 40])
def test_missing_pages_read_as_zeros(new):
    d, page = 64, 16
    lens = [100, 40]
    kp, vp, table = R.paged(lens, page, 2, d, torch.bfloat16, DEV, 3)
    q = _rand(2 * new, 4, d, dtype=torch.bfloat16, seed=2)
    whole = table.clone()
    table[0, 2] = kp.shape[0]
    table[0, 4] = -1
    cache = kt.PagedKV(kp, vp)
    out = cache.attend(q, table, R.starts([new, new], DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), new)
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    k0, v0 = kp.clone(), vp.clone()
    for i in (2, 4):
        k0[int(whole[0, i])] = 0
        v0[int(whole[0, i])] = 0
    want, bound = R.attend(q, k0, v0, whole, [new, new], lens, R.softmax_scale(d))
    assert bool(((out.double().cpu() - want).abs() <= bound).all())
    # a length past the table: the keys that it has
    short = torch.tensor([100, page * table.shape[1] + 5], dtype=torch.int32, device=DEV)
    full = torch.randint(0, kp.shape[0], tuple(table.shape), device=DEV, dtype=torch.int32)
    kp.nan_to_num_(0.25), vp.nan_to_num_(0.25)
    out = cache.attend(q, full, R.starts([new, new], DEV), short, new)
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    assert bool(torch.isfinite(out).all())


def test_strided_queries_and_outputs():
    """Queries sliced out of a packed projection, an output of another order, a transposed table."""
    n, hq, hk, d, page = 37, 6, 2, 64, 32
    lens = [n + 20]
    kp, vp, table = R.paged(lens, page, hk, d, torch.float16, DEV, 5)
    qkv = _rand(n, hq + 2 * hk, d, dtype=torch.float16, seed=6)
    q = qkv[:, :hq]
    wide = torch.zeros(1, table.shape[1] + 9, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    for max_q in (1, n):
        out = torch.zeros(hq, n, d, dtype=torch.float16, device=DEV).transpose(0, 1)
        kt.PagedKV(kp, vp).attend(q, wide[:, :table.shape[1]], R.starts([n], DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), max_q, out=out)
        want, bound = R.attend(q, kp, vp, table, [n], lens, R.softmax_scale(d))
        assert bool(((out.double().cpu() - want).abs() <= bound).all())


def test_tokens_of_no_sequence_are_left_alone():
    d = 64
    kp, vp, table = R.paged([5, 70], 16, 1, d, torch.bfloat16, DEV, 5)
    q = _rand(8, 4, d, dtype=torch.bfloat16, seed=6)
    for q_lens in ([1, 1], [1, 0], [2, 3]):
        out = torch.full_like(q, 9.0)
        kt.PagedKV(kp, vp).attend(q, table, R.starts(q_lens, DEV), torch.tensor([5, 70], dtype=torch.int32, device=DEV),
                                  3, out=out)
        want, bound = R.attend(q[:sum(q_lens)], kp, vp, table, q_lens, [5, 70], R.softmax_scale(d))
        assert bool(((out[:sum(q_lens)].double().cpu() - want).abs() <= bound).all())
        assert bool((out[sum(q_lens):] == 9.0).all())


def test_many_sequences():
    """More sequences than threads of a block, lengths of every kind."""
    g = torch.Generator().manual_seed(1)
    b = 700
    past = torch.randint(0, 90, (b,), generator=g).tolist()
    q_lens = torch.randint(0, 3, (b,), generator=g).tolist()
    _run(q_lens, past, 2, 1, 64, torch.bfloat16)


def _device_reference(q, k, v, last, scale):
    """64-bit attention of [n, hq, d] over contiguous [keys, hk, d] on the GPU; token t sees keys up to last[t]."""
    hk = k.shape[1]
    group = q.shape[1] // hk
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    weights = torch.empty_like(out)
    hidden = torch.arange(k.shape[0], device=q.device)[None] > last[:, None]
    for h in range(q.shape[1]):
        x = scale * (q[:, h].double() @ k[:, h // group].double().T)
        p = torch.softmax(x.masked_fill(hidden, -math.inf), dim=-1)
        out[:, h] = p @ v[:, h // group].double()
        weights[:, h] = p @ v[:, h // group].double().abs()
    return out, weights


@pytest.mark.parametrize("new,past,hq,hk,d", [(1, 30_000, 8, 1, 128), (3, 9000, 64, 8, 64), (257, 2000, 16, 2, 128),
                                             (1500, 0, 8, 1, 64), (600, 3333, 5, 1, 96)])
def test_long_sequences(new, past, hq, hk, d):
    """Sequences that many blocks share; bits do not change from call to call."""
    dt, page, n = torch.bfloat16, 64, new + past
    pages = -(-n // page)
    kp, vp = _rand(pages, page, hk, d, dtype=dt, seed=1), _rand(pages, page, hk, d, dtype=dt, seed=2)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)[None]
    q = _rand(new, hq, d, dtype=dt, seed=4, scale=2.0)
    cache = kt.PagedKV(kp, vp)
    args = (q, table, R.starts([new], DEV), torch.tensor([n], dtype=torch.int32, device=DEV), new)
    out = cache.attend(*args)
    k, v = (t[table[0].long()].reshape(-1, hk, d)[:n] for t in (kp, vp))
    scale = R.softmax_scale(d)
    want, weights = _device_reference(q, k, v, torch.arange(past, n, device=DEV), scale)
    # logits of at most ~2*6*sqrt(d)*sqrt(d)*scale: their fp32 error moves a weight by less than the 1e-3 allowed here
    bound = 1.01 * R.ROUND[dt] * (want.abs() + weights) + 1e-3 * weights
    assert bool(((out.double() - want).abs() <= bound).all())
    for _ in range(3):
        assert torch.equal(cache.attend(*args), out)
    # on another stream, and captured in a graph that is replayed twice
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = cache.attend(*args, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    got = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(*args, out=got)
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


@pytest.mark.parametrize("new", [1, 130])
def test_cache_past_32_bit_offsets(new):
    d, page, hk = 128, 64, 8
    pages = (1 << 31) // (page * hk * d) + 5
    kp = torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    need = -(-(new + 50) // page)
    table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV)[None]
    kp[-need:] = _rand(need, page, hk, d, dtype=torch.bfloat16, seed=1)
    vp[-need:] = _rand(need, page, hk, d, dtype=torch.bfloat16, seed=2)
    q = _rand(new, hk, d, dtype=torch.bfloat16, seed=3)
    lens = [new + 50]
    out = kt.PagedKV(kp, vp).attend(q, table, R.starts([new], DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                    new)
    small = torch.arange(need, dtype=torch.int32, device=DEV)[None]
    want, bound = R.attend(q, kp[-need:], vp[-need:], small, [new], lens, R.softmax_scale(d))
    assert bool(((out.double().cpu() - want).abs() <= bound).all())
