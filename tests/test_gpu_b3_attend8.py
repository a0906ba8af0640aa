"""Attention over a cache of 8 bits against the 64-bit statement over the numbers that the cache stands for.

Wherever no sequence has a key, codes and scales are any bytes, NaN among them."""
import math
import random

import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
TIMEOUTS = kt.KT_DEVERR_TIMEOUT_LOAD | kt.KT_DEVERR_TIMEOUT_MMA | kt.KT_DEVERR_TIMEOUT_EPI


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _near(out, want, bound):
    off = (out.double().cpu() - want).abs()
    assert bool(torch.isfinite(out).all()), "not finite"
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound, worst {float(off.max()):.3e}"


def _run(q_lens, past, hq, hk, d, dtype, page=16, layout="slots", window=0, sinks=None, scale=None, seed=0, qscale=0.5,
         max_q=None, codes=torch.uint8):
    lens = [a + b for a, b in zip(q_lens, past)]
    kp, vp, ks, vs, table, k, v = M.paged8(lens, page, hk, d, dtype, DEV, seed, layout)
    n = sum(q_lens)
    q = _rand(n, hq, d, dtype=dtype, seed=seed + 1, scale=qscale)
    cache = kt.PagedKV8(kp.view(codes), vp.view(codes), ks, vs, dtype)
    scale = R.softmax_scale(d) if scale is None else scale
    out = torch.full((n, hq, d), 9.0, dtype=dtype, device=DEV)
    cache.attend(q, table, R.starts(q_lens, DEV), _i32(lens), max(q_lens + [0]) if max_q is None else max_q, scale=scale,
                 window=window, sinks=sinks, out=out)
    assert cache.read_error() == 0
    _near(out, *R.attend(q, k, v, table, q_lens, lens, scale, window, sinks))
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 16), (4, 4, 64), (8, 1, 128), (12, 4, 96), (5, 1, 80), (40, 2, 64),
                                     (16, 1, 128), (34, 2, 112), (128, 1, 48)])
def test_single_tokens(dtype, hq, hk, d):
    _run([1, 1, 1, 1, 1], [0, 1, 15, 16, 130], hq, hk, d, dtype, page=16, codes=torch.float8_e4m3fn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,layout", [(16, "slots"), (48, "heads"), (64, "pairs"), (128, "heads"), (256, "slots")])
def test_pages(dtype, page, layout):
    _run([1, 3, 1, 2], [0, 61, 300, 126], 6, 2, 64, dtype, page=page, layout=layout)
    _run([40, 1], [61, 126], 6, 2, 128, dtype, page=page, layout=layout)


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


@pytest.mark.parametrize("d", [16, 32, 48, 112])
def test_chunks_of_other_head_sizes(d):
    _run([45, 3], [30, 100], 9, 3, d, torch.float16, page=16)


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


@pytest.mark.parametrize("window", [1, 2, 16, 60, 64, 129, 10_000])
@pytest.mark.parametrize("q_lens,past", [([1, 1], [200, 3]), ([150, 7], [100, 0])])
def test_windows(window, q_lens, past):
    _run(q_lens, past, 4, 1, 64, torch.bfloat16, page=32, window=window)


@pytest.mark.parametrize("q_lens,past", [([1, 1], [40, 300]), ([130], [10])])
def test_sinks(q_lens, past):
    sinks = torch.tensor([0.0, -math.inf, 30.0, -30.0, 3.0, 1.0], device=DEV)
    _run(q_lens, past, 6, 2, 128, torch.float16, sinks=sinks)
    _run(q_lens, past, 6, 2, 128, torch.bfloat16, sinks=sinks, window=5)


@pytest.mark.parametrize("scale,qscale", [(1.0, 1.0), (1e-3, 1.0), (0.125, 12.0)])
@pytest.mark.parametrize("q_lens,past", [([1], [700]), ([140], [60])])
def test_scales(scale, qscale, q_lens, past):
    """Peaked, flat, and very large logits."""
    _run(q_lens, past, 2, 1, 64, torch.bfloat16, scale=scale, qscale=qscale)


@pytest.mark.parametrize("q_lens,past", [([1, 1], [40, 90]), ([100], [30])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_code_and_power(dtype, q_lens, past):
    """Values of every finite code under the lowest, the highest and other exponents that an append writes.

    A sequence's values share an exponent, so that none vanishes beside another's; keys are of moderate size."""
    hk, d, page = 2, 64, 16
    lens = [a + b for a, b in zip(q_lens, past)]
    every = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    # |out| stays below the type's largest number: 448 * 2^X does
    for x in (M.LEAST[dtype], M.LEAST[dtype] + 7, -9, 0, 5, M.MOST[dtype] - 1, M.MOST[dtype]):
        kp, vp, ks, vs, table, k, v = M.paged8(lens, page, hk, d, dtype, DEV, 3)
        filled = v != 0
        codes = every[torch.arange(v.numel()) * 37 % len(every)].view(v.shape)
        own = vp.cpu()
        own[filled] = codes[filled]
        vp.copy_(own)
        vs.fill_(x + 127)
        v = torch.where(filled, M.numbers(own) * 2.0 ** x, v.double()).to(dtype)
        q = _rand(sum(q_lens), 4, d, dtype=dtype, seed=5, scale=0.1)
        cache = kt.PagedKV8(kp, vp, ks, vs, dtype)
        out = cache.attend(q, table, R.starts(q_lens, DEV), _i32(lens), max(q_lens))
        want, bound = R.attend(q, k, v, table, q_lens, lens, R.softmax_scale(d))
        # below bf16's normal numbers (2^-126) a result may be flushed or rounded to a subnormal
        _near(out, want, bound + 2.0 ** -126 * (dtype == torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [1, 20])
def test_weights_far_below_the_largest(dtype, new):
    """One key outweighs its neighbours by up to 2^190, and half its value's elements are zeros.

    A weight, relative to the largest of its block, is an fp16 number times 2^-10 (times 2^-24 of rounding below fp16's
    smallest normal one): off by at most 2^-35 of the largest, which is at most 1, times its value."""
    hk, d, page, n = 1, 64, 16, 60

    def rows(b):
        k, v = torch.zeros(n, hk, d, dtype=torch.float64), torch.ones(n, hk, d, dtype=torch.float64)
        k[:, 0, 0] = -torch.arange(n).double() / 4                # e4m3 keeps four bits of these
        k[0] = 0
        k[1:, 0, 0] -= 1.75
        v[0, 0, ::2] = 0
        return k, v

    kp, vp, ks, vs, table, k, v = M.paged8([n], page, hk, d, dtype, DEV, 1, rows=rows)
    q = torch.zeros(new, 4, d, dtype=dtype, device=DEV)
    q[:, :, 0] = torch.tensor([1.0, 2.0, 4.0, 8.0])
    out = kt.PagedKV8(kp, vp, ks, vs, dtype).attend(q, table, R.starts([new], DEV), _i32([n]), new, scale=1.0)
    want, bound = R.attend(q, k, v, table, [new], [n], 1.0)
    _near(out, want, bound + 2.0 ** -35 * n)


@pytest.mark.parametrize("q_lens,lens", [([3, 1, 2], [1, 0, 2]), ([150, 2], [140, 0])])
def test_tokens_that_see_nothing(q_lens, lens):
    d, page = 64, 16
    kp, vp, ks, vs, table, k, v = M.paged8(lens, page, 1, d, torch.bfloat16, DEV, 1)
    q = _rand(sum(q_lens), 4, d, dtype=torch.bfloat16, seed=2)
    for sinks in (None, torch.zeros(4, device=DEV), torch.full((4,), -math.inf, device=DEV)):
        out = torch.full_like(q, 9.0)
        kt.PagedKV8(kp, vp, ks, vs).attend(q, table, R.starts(q_lens, DEV), _i32(lens), max(q_lens), sinks=sinks, out=out)
        _near(out, *R.attend(q, k, v, table, q_lens, lens, R.softmax_scale(d), 0, sinks))
        assert bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [4, 60])
def test_blocks_of_nan(dtype, new):
    """A block of keys whose scale is NaN reaches the tokens that see one of them, and no token before it."""
    d, page, n = 64, 16, 100
    kp, vp, ks, vs, table, k, v = M.paged8([n], page, 1, d, dtype, DEV, 1)
    ks[table[0, 6].long(), 0] = 255                              # positions 96 to 99
    q = _rand(new, 2, d, dtype=dtype, seed=2, scale=0.5)
    out = kt.PagedKV8(kp, vp, ks, vs, dtype).attend(q, table, R.starts([new], DEV), _i32([n]), new)
    want, bound = R.attend(q, k, v, table, [new], [n], R.softmax_scale(d))
    ok = slice(0, new - 4)
    assert bool(((out[ok].double().cpu() - want[ok]).abs() <= bound[ok]).all())
    assert bool(out[new - 4:].isnan().all())
    # of values: every token that sees one
    vs[table[0, 0].long(), 0] = 255
    out = kt.PagedKV8(kp, vp, ks, vs, dtype).attend(q, table, R.starts([new], DEV), _i32([n]), new)
    assert bool(out.isnan().all())


@pytest.mark.parametrize("new", [1, 40])
def test_missing_pages_read_as_zeros(new):
    d, page = 64, 16
    lens = [100, 40]
    kp, vp, ks, vs, table, k, v = M.paged8(lens, page, 2, d, torch.bfloat16, DEV, 3)
    q = _rand(2 * new, 4, d, dtype=torch.bfloat16, seed=2)
    whole = table.clone()
    table[0, 2] = kp.shape[0]
    table[0, 4] = -1
    cache = kt.PagedKV8(kp, vp, ks, vs)
    out = cache.attend(q, table, R.starts([new, new], DEV), _i32(lens), new)
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    for i in (2, 4):
        k[int(whole[0, i])] = 0
        v[int(whole[0, i])] = 0
    _near(out, *R.attend(q, k, v, whole, [new, new], lens, R.softmax_scale(d)))
    short = _i32([100, page * table.shape[1] + 5])                # a length past the table: the keys that it has
    full = torch.randint(0, kp.shape[0], tuple(table.shape), device=DEV, dtype=torch.int32)
    kp.fill_(0x30), vp.fill_(0x30), ks.fill_(127), vs.fill_(127)
    out = cache.attend(q, full, R.starts([new, new], DEV), short, new)
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    assert bool((out == 0.5).all())


@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48])
def test_pages_behind_the_window_are_free(new, d, page):
    window, hq = 40, 8
    lens = [150 + i for i in range(33)]
    kp, vp, ks, vs, table, k, v = M.paged8(lens, page, 1, d, torch.bfloat16, DEV, 21)
    q = _rand(new * len(lens), hq, d, dtype=torch.bfloat16, seed=22, scale=0.5)
    want, bound = R.attend(q, k, v, table, [new] * len(lens), lens, R.softmax_scale(d), window)
    for b, n in enumerate(lens):
        behind = (n - new - window + 1) // page
        freed = table[b, :behind].long()
        kp[freed], vp[freed], ks[freed], vs[freed] = 0x7f, 0x7f, 255, 255
        table[b, :behind] = _i32([(-1, kp.shape[0], -2 ** 31)[i % 3] for i in range(behind)])
    cache = kt.PagedKV8(kp, vp, ks, vs)
    out = cache.attend(q, table, R.starts([new] * len(lens), DEV), _i32(lens), new, window=window)
    assert cache.read_error() == 0
    _near(out, want, bound)


def test_strided_queries_and_outputs():
    """Queries sliced out of a packed projection or expanded, an output of another order, in place."""
    n, hq, hk, d, page = 37, 6, 2, 64, 32
    lens = [n + 20]
    kp, vp, ks, vs, table, k, v = M.paged8(lens, page, hk, d, torch.float16, DEV, 5)
    qkv = _rand(n, hq + 2 * hk, d, dtype=torch.float16, seed=6, scale=0.5)
    q = qkv[:, :hq]
    cache = kt.PagedKV8(kp, vp, ks, vs, torch.float16)
    step = table, R.starts([n], DEV), _i32(lens)
    want, bound = R.attend(q, k, v, table, [n], lens, R.softmax_scale(d))
    for max_q in (1, n):
        out = torch.zeros(hq, n, d, dtype=torch.float16, device=DEV).transpose(0, 1)
        cache.attend(q, *step, max_q, out=out)
        _near(out, want, bound)
    one = q[:, :1].expand(n, hq, d)
    _near(cache.attend(one, *step, n), *R.attend(one, k, v, table, [n], lens, R.softmax_scale(d)))
    rest = qkv[:, hq:].clone()
    plain = cache.attend(q, *step, n)
    assert cache.attend(q, *step, n, out=q) is q and torch.equal(q, plain) and torch.equal(qkv[:, hq:], rest)
    inside = kp.view(torch.float16).flatten()[:hq * d].view(1, hq, d)
    with pytest.raises(ValueError, match="pages"):
        cache.attend(q[:1], table, R.starts([1], DEV), _i32(lens), 1, out=inside)


def test_tokens_of_no_sequence_are_left_alone():
    d = 64
    kp, vp, ks, vs, table, k, v = M.paged8([5, 70], 16, 1, d, torch.bfloat16, DEV, 5)
    q = _rand(8, 4, d, dtype=torch.bfloat16, seed=6)
    for q_lens in ([1, 1], [1, 0], [2, 3]):
        out = torch.full_like(q, 9.0)
        kt.PagedKV8(kp, vp, ks, vs).attend(q, table, R.starts(q_lens, DEV), _i32([5, 70]), 3, out=out)
        n = sum(q_lens)
        _near(out[:n], *R.attend(q[:n], k, v, table, q_lens, [5, 70], R.softmax_scale(d)))
        assert bool((out[n:] == 9.0).all())


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    past = torch.randint(0, 90, (700,), generator=g).tolist()
    q_lens = torch.randint(0, 3, (700,), generator=g).tolist()
    _run(q_lens, past, 2, 1, 64, torch.bfloat16)
    _run(q_lens, past, 2, 1, 32, torch.float16, max_q=100)


def _random_cache(pages, page, hk, d, seed):
    """Codes of every finite value, scales around 2^-8; and the numbers they stand for, on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    made = []
    for _ in range(2):
        c = torch.randn(pages, page, hk, d, generator=g, device=DEV).mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s = torch.randint(127 - 8, 127 - 5, (pages, page // M.BLOCK, hk), generator=g, device=DEV,
                          dtype=torch.int32).to(torch.uint8)
        made.append((c, s))
    return made


def _numbers(c, s):
    return c.double() * torch.exp2(s.double() - 127).repeat_interleave(M.BLOCK, 1)[..., None]


@pytest.mark.parametrize("new,past,hq,hk,d", [(1, 30_000, 8, 1, 128), (3, 9000, 64, 8, 64), (257, 2000, 16, 2, 128),
                                             (1500, 0, 8, 1, 64), (600, 3333, 5, 1, 96)])
def test_long_sequences(new, past, hq, hk, d):
    """Sequences that many blocks share; the same bits each time, on another stream and in a graph."""
    dt, page, n = torch.bfloat16, 64, new + past
    pages = -(-n // page)
    (kc, ks), (vc, vs) = _random_cache(pages, page, hk, d, 1)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)[None]
    q = _rand(new, hq, d, dtype=dt, seed=4)
    cache = kt.PagedKV8(kc, vc, ks, vs, dt)
    args = (q, table, R.starts([new], DEV), _i32([n]), new)
    out = cache.attend(*args)
    assert cache.read_error() == 0
    k, v = (_numbers(c, s)[table[0].long()].reshape(-1, hk, d)[:n] for c, s in ((kc, ks), (vc, vs)))
    scale, group = R.softmax_scale(d), hq // hk
    last = torch.arange(past, n, device=DEV)
    hidden = torch.arange(n, device=DEV)[None] > last[:, None]
    for h in range(hq):
        x = scale * (q[:, h].double() @ k[:, h // group].T)
        p = torch.softmax(x.masked_fill(hidden, -math.inf), dim=-1)
        want, weights = p @ v[:, h // group], p @ v[:, h // group].abs()
        # the fp32 error of logits of at most 64 moves a weight by less than the 1e-3 allowed here
        assert float(x.abs().max()) < 64
        bound = 1.01 * R.ROUND[dt] * (want.abs() + weights) + 1e-3 * weights
        assert bool(((out[:, h].double() - want).abs() <= bound).all())
    for _ in range(3):
        assert torch.equal(cache.attend(*args), out)
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
    pages = (1 << 32) // (page * hk * d) + 5
    need = -(-(new + 50) // page)
    kp, vp = (torch.zeros(pages, page, hk, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, page // M.BLOCK, hk), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    (kc, sk), (vc, sv) = _random_cache(need, page, hk, d, 1)
    kp[-need:], vp[-need:], ks[-need:], vs[-need:] = kc.view(torch.uint8), vc.view(torch.uint8), sk, sv
    table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV)[None]
    q = _rand(new, hk, d, dtype=torch.bfloat16, seed=3)
    lens = [new + 50]
    out = kt.PagedKV8(kp, vp, ks, vs).attend(q, table, R.starts([new], DEV), _i32(lens), new)
    k, v = (_numbers(c, s).to(torch.bfloat16) for c, s in ((kc, sk), (vc, sv)))
    _near(out, *R.attend(q, k, v, torch.arange(need)[None], [new], lens, R.softmax_scale(d)))


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float16, 128)])
@pytest.mark.parametrize("seqs,new,past,hq", [(1, 1, 20000, 8), (1, 1, 40, 8), (400, 1, 700, 8), (1, 40, 20000, 8),
                                              (3, 500, 300, 8), (20, 300, 0, 5)])
def test_waits_that_run_out(seqs, new, past, hq, dtype, d):
    """The test hook withholds a load, every wait ends after 50 ms: told, and without consequence for the next call."""
    page, n = 64, new + past
    pages = -(-n // page)
    (kc, ks), (vc, vs) = _random_cache(seqs * pages, page, 1, d, 1)
    table = torch.arange(seqs * pages, dtype=torch.int32, device=DEV).view(seqs, pages)
    q = _rand(seqs * new, hq, d, dtype=dtype, seed=2)
    args = (q, table, R.starts([new] * seqs, DEV), _i32([n] * seqs), new)
    cache = kt.PagedKV8(kc, vc, ks, vs, dtype)
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


def test_shares_its_workspace_with_16_bit_caches():
    """Caches of both kinds in turn on one stream and on one workspace, each as if alone."""
    d, page, n = 64, 16, 3000
    pages = -(-n // page)
    (kc, ks), (vc, vs) = _random_cache(pages, page, 1, d, 1)
    wide = [_numbers(c, s).to(torch.bfloat16) for c, s in ((kc, ks), (vc, vs))]
    for new in (1, 70):
        q = _rand(new, 4, d, dtype=torch.bfloat16, seed=3)
        step = (torch.arange(pages, dtype=torch.int32, device=DEV)[None], R.starts([new], DEV), _i32([n]), new)
        small, large = kt.PagedKV8(kc, vc, ks, vs), kt.PagedKV(*wide)
        ws = small.workspace()
        a, b = small.attend(q, *step, workspace=ws), large.attend(q, *step, workspace=ws)
        for _ in range(2):
            assert torch.equal(large.attend(q, *step), b) and torch.equal(small.attend(q, *step), a)
        assert small._workspaces.keys() == large._workspaces.keys()
        assert all(small._workspaces[i] is large._workspaces[i] for i in small._workspaces)
        off = (a.double() - b.double()).abs()
        assert bool((off <= 4 * R.ROUND[torch.bfloat16] * b.double().abs().max()).all())


def test_an_appended_step_is_attended():
    """Append and attend in turn, prompts and single tokens, as a serving program does, against the numbers stored."""
    d, hq, hk, page, dt = 96, 6, 2, 32, torch.bfloat16
    total = [75, 40]
    kp, vp, ks, vs, table, _, _ = M.paged8(total, page, hk, d, dt, DEV, 3)
    cache, rope = kt.PagedKV8(kp, vp, ks, vs, dt), kt.rope_table(128, d)
    w = torch.ones(d, dtype=dt, device=DEV)
    lens = [0, 0]
    for i, new in enumerate(([50, 3], [1, 1], [1, 20], [7, 0], [16, 16])):
        lens = [a + b for a, b in zip(lens, new)]
        qkv = _rand(sum(new), hq + 2 * hk, d, dtype=dt, seed=i)
        q, k, v = qkv.split((hq, hk, hk), dim=1)
        step = table, R.starts(new, DEV), _i32(lens)
        q = cache.append(k, v, *step, rope, q=q, q_weight=w, k_weight=w)
        out = cache.attend(q, *step, max(new))
        assert cache.read_error() == 0
        kn, vn = (_numbers(c.view(torch.float8_e4m3fn).cpu(), s.cpu()).to(dt) for c, s in ((kp, ks), (vp, vs)))
        _near(out, *R.attend(q, kn, vn, table, new, lens, R.softmax_scale(d)))
