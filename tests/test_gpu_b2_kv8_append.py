"""The append to a cache of 8 bits against the 64-bit statement: blocks begun, continued and rescaled."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = M.BLOCK


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _state(pages, scales):
    """(codes, scale bytes) on the CPU."""
    return pages.view(torch.uint8).cpu().clone(), scales.cpu().clone()


def _check_side(before, after, rows, off, table, q_lens, past, dtype):
    """Every byte of one side (keys or values) after an append of rows (64 bits, off by at most `off` before rounding)."""
    codes, scales = before[0].clone(), before[1].clone()
    page = codes.shape[1]
    at = 0
    table = table.cpu().long()
    for b, (a, h) in enumerate(zip(q_lens, past)):
        new, slack = rows[at:at + a], off[at:at + a]
        at += a
        lo = h
        while lo < h + a:
            base = lo // BLOCK * BLOCK
            hi = min(h + a, base + BLOCK)
            p, slot = int(table[b, base // page]), base % page
            where = p, slot // BLOCK
            v, o = new[lo - h:hi - h], slack[lo - h:hi - h]                       # [rows, heads, d]
            top, room = v.abs().amax(dim=(0, 2)), o.amax(dim=(0, 2))
            low, high = M.least_exponent((top - room).clamp(min=0), dtype), M.least_exponent(top + room, dtype)
            x = after[1][where].double() - 127
            if lo > base:
                old = scales[where].double() - 127
                low, high = torch.maximum(low, old), torch.maximum(high, old)
                had = M.numbers(codes[p, slot:slot + lo - base])
                moved = M.e4m3(had * torch.exp2(old - x)[:, None])
                got = M.numbers(after[0][p, slot:slot + lo - base])
                assert torch.equal(got, moved), "older tokens"
                codes[p, slot:slot + lo - base] = after[0][p, slot:slot + lo - base]
            assert bool(((x >= low) & (x <= high)).all()), f"exponents {x} outside {low} to {high}"
            span = slice(slot + lo - base, slot + hi - base)
            got = M.numbers(after[0][p, span])
            assert float(M.off_by_a_rounding(got, torch.exp2(x)[:, None], v, o).max()) <= 0, "new tokens"
            codes[p, span] = after[0][p, span]
            scales[where] = after[1][where]
            lo = hi
    assert torch.equal(codes, after[0]) and torch.equal(scales, after[1]), "bytes of no new token's block changed"


def _run(dtype, q_lens, past, hq, hk, d, rot, style, page, norm, layout="slots", extra=2, seed=4, grow=1.0):
    lens = [a + b for a, b in zip(q_lens, past)]
    n = sum(q_lens)
    # pages for all, blocks full up to `past`
    kp, vp, ks, vs, table, _, _ = M.paged8(lens, page, hk, d, dtype, DEV, 9, layout)
    qkv = _rand(n + extra, hq + 2 * hk, d, dtype=dtype, seed=seed, scale=grow)
    q = qkv[:, :hq] if hq else None
    k, v = qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    cs = kt.rope_table(max(lens + [1]), rot) if rot else None
    wq, wk = (_rand(d, dtype=dtype, seed=i) if norm else None for i in (1, 2))
    cache = kt.PagedKV8(kp, vp, ks, vs, dtype)
    before = _state(kp, ks), _state(vp, vs)
    pos = torch.cat([torch.arange(b, b + a) for a, b in zip(q_lens, past)])
    q_out = None if q is None else torch.full(q.shape, 3.0, dtype=dtype, device=DEV)
    kept = qkv.clone()
    got_q = cache.append(k, v, table, R.starts(q_lens, DEV), _i32(lens), cs, q=q, q_weight=wq, k_weight=wk, style=style,
                         q_out=q_out)
    assert cache.read_error() == 0 and torch.equal(qkv, kept)
    rows, bound = R.head_rows(k[:n], wk, 1e-6, cs, pos, style)
    off = bound - R.ROUND[dtype] * rows.abs()                 # the fp32 error alone, and a little more
    _check_side(before[0], _state(kp, ks), rows, off, table, q_lens, past, dtype)
    exact = v[:n].double().cpu()
    _check_side(before[1], _state(vp, vs), exact, torch.zeros_like(exact), table, q_lens, past, dtype)
    if q is None:
        assert got_q is None
    else:
        want, bound = R.head_rows(q[:n], wq, 1e-6, cs, pos, style)
        assert bool(((got_q[:n].double().cpu() - want).abs() <= bound).all())
        assert bool((got_q[n:] == 3.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["slots", "heads", "pairs"])
@pytest.mark.parametrize("q_lens,past,hq,hk,d,rot,style,page,norm", [
    ([1, 1, 1, 1], [0, 15, 16, 300], 8, 2, 128, 128, "halves", 16, False),
    ([1], [0], 0, 1, 16, 16, "interleaved", 16, False),
    ([5, 0, 1, 40], [11, 7, 0, 30], 12, 4, 96, 32, "interleaved", 48, True),
    ([130, 0, 0, 3], [1, 0, 5, 62], 5, 5, 80, 48, "halves", 64, True),
    ([16, 17, 15, 33], [16, 15, 1, 31], 3, 1, 112, 112, "interleaved", 32, True),
    ([2, 31], [13, 2], 4, 3, 64, 0, "halves", 128, False),
])
def test_append(dtype, layout, q_lens, past, hq, hk, d, rot, style, page, norm):
    _run(dtype, q_lens, past, hq, hk, d, rot, style, page, norm, layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("grow", [2.0 ** -9, 2.0 ** -3, 8.0, 300.0])
def test_blocks_that_grow_or_do_not(dtype, grow):
    """New tokens far smaller and far larger than the block's older ones."""
    _run(dtype, [3, 1, 14, 40], [5, 15, 1, 9], 2, 2, 64, 64, "halves", 32, False, grow=grow)


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    past = torch.randint(0, 70, (1100,), generator=g).tolist()
    q_lens = torch.randint(0, 4, (1100,), generator=g).tolist()
    q_lens[-1] = 1
    _run(torch.bfloat16, q_lens, past, 1, 1, 16, 16, "halves", 16, False)


def test_token_by_token():
    """A sequence written one token at a time: every step is checked, and what stands there at the end is near each."""
    d, hk, page, n, dt = 64, 2, 32, 50, torch.bfloat16
    kp, vp, ks, vs, table, _, _ = M.paged8([n], page, hk, d, dt, DEV, 3)
    cache = kt.PagedKV8(kp, vp, ks, vs, dt)
    rows = _rand(n, hk, d, dtype=dt, seed=5)
    rows *= torch.exp2((torch.arange(n, device=DEV) * 7 % 11 - 5).float())[:, None, None].to(dt)
    zero = torch.zeros(1, hk, d, dtype=torch.float64)
    for i in range(n):
        before = _state(kp, ks)
        cache.append(rows[i:i + 1], rows[i:i + 1], table, R.starts([1], DEV), _i32([i + 1]))
        _check_side(before, _state(kp, ks), rows[i:i + 1].double().cpu(), zero, table, [1], [i], dt)
    assert torch.equal(kp.cpu()[table[0, 0].item(), :page], vp.cpu()[table[0, 0].item(), :page])
    # a code that has been rescaled has been rounded twice at most a number: within a step of the value
    for i in range(n):
        p, slot = int(table[0, i // page]), i % page
        scale = M.power(ks[p, slot // BLOCK].cpu())[:, None]
        off = (M.numbers(kp[p, slot].cpu()) * scale - rows[i].double().cpu()).abs()
        assert bool((off <= 2 * M.half_step(rows[i].double().cpu() / scale) * scale).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_extreme_values(dtype):
    """Zeros, the largest and the smallest numbers; bf16 past 448 * 2^87 and fp16 past 448 * 2^7 saturate."""
    d, hk, page = 32, 1, 16
    most = torch.finfo(dtype).max
    for value in (0.0, most, most / 3, torch.finfo(dtype).tiny, torch.finfo(dtype).smallest_normal / 2, 1.0):
        kp, vp, ks, vs, table, _, _ = M.paged8([3], page, hk, d, dtype, DEV, 3)
        cache = kt.PagedKV8(kp, vp, ks, vs, dtype)
        rows = torch.full((3, hk, d), value, dtype=dtype, device=DEV)
        rows[1] *= -0.25
        before = _state(kp, ks)
        cache.append(rows, rows, table, R.starts([3], DEV), _i32([3]))
        exact = rows.double().cpu()
        _check_side(before, _state(kp, ks), exact, torch.zeros_like(exact), table, [3], [0], dtype)
    assert int(ks[table[0, 0], 0, 0]) == 127 - 8                # 1 <= 448 * 2^-8 = 1.75


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(what):
    """The block of that head is NaN until it is begun anew; other heads, blocks and the other side are not."""
    d, hk, page, dt = 64, 3, 32, torch.bfloat16
    kp, vp, ks, vs, table, _, _ = M.paged8([24], page, hk, d, dt, DEV, 3)
    cache = kt.PagedKV8(kp, vp, ks, vs, dt)
    rows = _rand(24, hk, d, dtype=dt, seed=2)
    bad = rows.clone()
    bad[5, 1, 7] = what
    step = table, R.starts([20], DEV), _i32([20])
    cache.append(bad[:20], rows[:20], *step)
    p = int(table[0, 0])
    assert ks[p, :, 1].tolist()[0] == 255 and int(ks[p, 1, 1]) != 255 and 255 not in ks[p, :, [0, 2]].flatten().tolist()
    assert 255 not in vs[p].flatten().tolist()
    cache.append(rows[12:14], rows[12:14], table, R.starts([2], DEV), _i32([14]))      # again, into the NaN block
    assert int(ks[p, 0, 1]) == 255
    cache.append(rows[:20], rows[:20], *step)                                           # anew
    assert torch.equal(ks[p], vs[p]) and torch.equal(kp[p, :20], vp[p, :20]) and 255 not in ks[p].flatten().tolist()


def test_bad_pages_and_positions():
    """A page outside the cache, a length outside the table, a position outside the rotation: told, not written."""
    d, page, dt = 64, 16, torch.bfloat16
    kp, vp = (torch.zeros(4, page, 1, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((4, 1, 1), 9, dtype=torch.uint8, device=DEV) for _ in range(2))
    cache = kt.PagedKV8(kp, vp, ks, vs, dt)
    k = torch.ones(4, 1, d, dtype=dt, device=DEV)
    cu = R.starts([1, 1, 1, 1], DEV)
    bt = _i32([[4, 0], [-1, 0], [1, 2], [3, 3]])
    cache.append(k, k, bt, cu, _i32([1, 1, 33, 0]))
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE and cache.read_error() == 0
    assert not bool(kp.any()) and not bool(vp.any()) and bool((ks == 9).all()) and bool((vs == 9).all())
    cache.append(k, k, bt, cu, _i32([17, 17, 1, 8]), kt.rope_table(8, d), q=k)
    assert cache.read_error() == A.KT_DEVERR_BAD_POSITION
    assert not bool(kp[0].any()) and int(ks[0, 0, 0]) == 9
    assert bool(kp[1, 0].any()) and bool(kp[3, 7].any())
    # the part of a block that the rotation reaches is written
    cache.append(k, k, _i32([[2]]), R.starts([4], DEV), _i32([10]), kt.rope_table(8, d))
    assert cache.read_error() == A.KT_DEVERR_BAD_POSITION
    assert bool(kp[2, 6:8].any(-1).all()) and not bool(kp[2, 8:].any()) and not bool(vp[2, 8:].any())
    # tokens before position 0
    kp.zero_()
    cache.append(k, k, _i32([[0]]), R.starts([4], DEV), _i32([2]))
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE
    assert bool(kp[0, :2].any(-1).all()) and not bool(kp[0, 2:].any())


def test_past_32_bit_offsets():
    d, page, hk, dt = 128, 64, 8, torch.bfloat16
    pages = (1 << 32) // (page * hk * d) + 3
    kp, vp = (torch.zeros(pages, page, hk, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pages, page // BLOCK, hk, dtype=torch.uint8, device=DEV) for _ in range(2))
    k = _rand(2, hk, d, dtype=dt, seed=1)
    bt = _i32([[0, pages - 1]])
    kt.PagedKV8(kp, vp, ks, vs, dt).append(k, k, bt, R.starts([2], DEV), _i32([page + 2]))
    assert not bool(kp[:2].any()) and not bool(kp[pages - 2].any()) and bool(ks[pages - 1, 0].all())
    x = M.power(ks[pages - 1, 0].cpu())[:, None]
    exact = k.double().cpu()
    assert float(M.off_by_a_rounding(M.numbers(kp[pages - 1, :2].cpu()), x, exact, 0 * exact).max()) <= 0
    assert torch.equal(kp[pages - 1], vp[pages - 1])


def test_streams_and_graph():
    """On a stream of the caller's, and captured and replayed: the same bytes each time."""
    d, hk, page, dt, n = 128, 2, 16, torch.float16, 45
    made = M.paged8([n + 7], page, hk, d, dt, DEV, 3)
    table = made[4]
    k, q, w, cs = (_rand(n, hk, d, dtype=dt, seed=1), _rand(n, 4, d, dtype=dt, seed=2), torch.ones(d, device=DEV),
                   kt.rope_table(n + 7, d))
    args = (k, k, table, R.starts([n], DEV), _i32([n + 7]), cs)
    first = [t.clone() for t in made[:4]]
    want_q = kt.PagedKV8(*first, dt).append(*args, q=q, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    side, second = torch.cuda.Stream(), [t.clone() for t in made[:4]]
    torch.cuda.synchronize()
    got_q = kt.PagedKV8(*second, dt).append(*args, q=q, q_weight=w, k_weight=w, stream=side)
    side.synchronize()
    third = [t.clone() for t in made[:4]]
    cache, out = kt.PagedKV8(*third, dt), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append(*args, q=q, q_weight=w, k_weight=w, q_out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(out, want_q)
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)
    # queries in place
    q_in = q.clone()
    assert cache.append(*args, q=q_in, q_weight=w, k_weight=w, q_out=q_in) is q_in and torch.equal(q_in, want_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_queries(dtype):
    _run(dtype, [150, 0, 181], [5, 3, 40], 40, 2, 96, 64, "interleaved", 48, True)
    _run(dtype, [320], [0], 64, 1, 48, 48, "halves", 16, False)


@pytest.mark.parametrize("norm", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,d", [(9, 8, 64), (400, 40, 80), (4200, 64, 128)])
def test_queries_beside_keys_and_values(norm, n, hq, d):
    """One launch for all writes what a launch for the queries and one for the rest do, at every number of queries."""
    hk, page, past, dt = 2, 16, 21, torch.bfloat16
    kp, vp, ks, vs, table, _, _ = M.paged8([n + past], page, hk, d, dt, DEV, 3)
    made = [kp, vp, ks, vs]
    twice = [t.clone() for t in made]
    q, k, v = _rand(n, hq + 2 * hk, d, dtype=dt, seed=1).split((hq, hk, hk), dim=1)
    wq, wk = (None if norm is None else _rand(d, dtype=norm, seed=i) for i in (2, 3))
    cs = kt.rope_table(n + past, d)
    step = table, R.starts([n], DEV), _i32([n + past]), cs
    got = kt.PagedKV8(*made, dt).append(k, v, *step, q=q, q_weight=wq, k_weight=wk)
    kt.PagedKV8(*twice, dt).append(k, v, *step, k_weight=wk)
    want, _ = kt.qk_norm_rope(q, None, torch.arange(past, past + n, dtype=torch.int32, device=DEV), cs, q_weight=wq)
    assert torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(made, twice))


def test_empty_step():
    kp, vp, ks, vs, table, _, _ = M.paged8([5], 16, 1, 32, torch.bfloat16, DEV, 3)
    before = _state(kp, ks)
    k = torch.empty(0, 1, 32, dtype=torch.bfloat16, device=DEV)
    kt.PagedKV8(kp, vp, ks, vs).append(k, k, table, R.starts([0], DEV), _i32([5]))
    after = _state(kp, ks)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
