"""Norm and rotation of heads, and the append to a paged cache, against the 64-bit statement."""
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


def _near(got, want, bound, what=""):
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), f"{what}: {float((off - bound).max()):.3e} over the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,hq,hk,d,rot,style", [
    (1, 32, 8, 128, 128, "halves"), (1, 1, 1, 8, 8, "halves"), (3, 5, 1, 64, 64, "interleaved"),
    (17, 12, 4, 96, 48, "halves"), (7, 3, 3, 80, 40, "halves"), (7, 3, 3, 80, 40, "interleaved"),
    (5, 2, 2, 256, 64, "interleaved"), (9, 4, 2, 200, 104, "halves"), (700, 20, 5, 128, 128, "halves"),
    (331, 64, 8, 64, 32, "interleaved"),
])
def test_norm_and_rotation(dtype, n, hq, hk, d, rot, style):
    qkv = _rand(n, hq + 2 * hk, d, dtype=dtype, seed=n + d)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 999, (n,), generator=g, dtype=torch.int32).to(DEV)
    pos[0] = 998
    table = kt.rope_table(999, rot, 5e5)
    wq, wk = _rand(d, dtype=dtype, seed=1), _rand(d, dtype=dtype, seed=2)
    kept = qkv.clone()
    qo, ko = kt.qk_norm_rope(q, k, pos, table, wq, wk, eps=1e-5, style=style)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        _near(got, *R.head_rows(x, w, 1e-5, table, pos, style), "norm and rotation")
    assert torch.equal(qkv, kept)
    qo, ko = kt.qk_norm_rope(q, k, pos, table, style=style)
    _near(qo, *R.head_rows(q, None, 0, table, pos, style), "rotation")
    qo, ko = kt.qk_norm_rope(q, k, q_weight=wq.float(), eps=0.0)
    _near(qo, *R.head_rows(q, wq.float(), 0.0, None, None, style), "norm")
    assert torch.equal(ko, k)
    # in place, q alone
    want, bound = R.head_rows(q, wq, 1e-6, table, pos, style)
    out, none = kt.qk_norm_rope(q, None, pos, table, wq, style=style, q_out=q)
    assert none is None and out is q
    _near(q, want, bound, "in place")
    assert torch.equal(qkv[:, hq:], kept[:, hq:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_large_steps_are_their_parts(dtype):
    """Steps beyond L2 take another path through it: the same bits as in parts that do not, dense and paged."""
    n, hq, hk, d, page = 6001, 40, 8, 128, 64
    qkv = torch.randn(n, hq + 2 * hk, d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    q, k, v = qkv.split((hq, hk, hk), dim=1)
    table, pos = kt.rope_table(n, d), torch.arange(n, dtype=torch.int32, device=DEV)
    w = _rand(d, dtype=dtype, seed=2)
    whole_q, whole_k = kt.qk_norm_rope(q, k, pos, table, w, w)
    pages = -(-n // page)
    bt = torch.arange(pages, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    whole = kt.PagedKV(*(torch.zeros(pages, page, hk, d, dtype=dtype, device=DEV) for _ in range(2)))
    parts = kt.PagedKV(*(torch.zeros(pages, page, hk, d, dtype=dtype, device=DEV) for _ in range(2)))
    got = whole.append(k, v, bt, R.starts([n], DEV), torch.tensor([n], dtype=torch.int32, device=DEV), table, q=q,
                       q_weight=w, k_weight=w)
    assert torch.equal(got, whole_q)
    for lo, hi in ((0, 2000), (2000, 4001), (4001, n)):
        pq, pk = kt.qk_norm_rope(q[lo:hi], k[lo:hi], pos[lo:hi], table, w, w)
        assert torch.equal(pq, whole_q[lo:hi]) and torch.equal(pk, whole_k[lo:hi])
        parts.append(k[lo:hi], v[lo:hi], bt, R.starts([hi - lo], DEV),
                     torch.tensor([hi], dtype=torch.int32, device=DEV), table, k_weight=w)
    assert torch.equal(whole.k_pages, parts.k_pages) and torch.equal(whole.v_pages, parts.v_pages)
    _near(whole_k[::500], *R.head_rows(k[::500], w, 1e-6, table, pos[::500], "halves"))


def test_unaligned_heads():
    """Heads that start 8 bytes into a 16-byte word, and outputs of another order of dimensions."""
    d, n, h = 64, 11, 4
    flat = _rand(n * h * d + 4, dtype=torch.bfloat16, seed=5)
    q = flat[4:].view(n, h, d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = kt.rope_table(n, d)
    out = torch.empty(h, n, d, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    kt.qk_norm_rope(q, None, pos, table, q_out=out)
    _near(out, *R.head_rows(q, None, 0, table, pos, "halves"))


def test_extreme_rows():
    """Zero rows under a norm stay zero, infinities and NaN stay in their head; positions outside the table are told."""
    d = 128
    q = _rand(6, 3, d, dtype=torch.float16, seed=6)
    q[0, 0] = 0
    q[1, 1, 7] = float("nan")
    q[2, 2, 9] = float("inf")
    q[3] *= 0
    q[3, :, 0] = 60000.0
    w = torch.ones(d, device=DEV)
    pos = torch.tensor([0, 1, 2, 3, -1, 10], dtype=torch.int32, device=DEV)
    table = kt.rope_table(10, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    kt.qk_norm_rope(q, None, pos, table, w, q_out=out, error=err)
    assert int(err) == A.KT_DEVERR_BAD_POSITION
    assert bool((out[4:] == 7.0).all())                        # not written
    assert bool((out[0, 0] == 0).all())
    assert bool(out[1, 1].isnan().all()) and not bool(out[1, 0].isnan().any()) and not bool(out[1, 2].isnan().any())
    assert not bool(out[2, :2].isnan().any())
    _near(out[3:4], *R.head_rows(q[3:4], w, 1e-6, table, pos[3:4], "halves"))


def test_empty_step():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, _ = kt.qk_norm_rope(q, None, q_weight=torch.ones(64, device=DEV))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["slots", "heads", "pairs"])
@pytest.mark.parametrize("q_lens,past,hq,hk,d,rot,style,page,norm", [
    ([1, 1, 1, 1], [0, 15, 16, 300], 8, 2, 128, 128, "halves", 16, False),
    ([1], [0], 0, 1, 8, 8, "interleaved", 16, False),
    ([5, 0, 1, 40], [11, 7, 0, 30], 12, 4, 96, 32, "interleaved", 48, True),
    ([130, 0, 0, 3], [1, 0, 5, 62], 5, 5, 80, 40, "halves", 64, True),
])
def test_append(dtype, layout, q_lens, past, hq, hk, d, rot, style, page, norm):
    lens = [a + b for a, b in zip(q_lens, past)]
    n, extra = sum(q_lens), 2                                  # two tokens of the step belong to no sequence
    kp, vp, table = R.paged(lens, page, hk, d, dtype, DEV, 9, layout, fill=0.5)
    qkv = _rand(n + extra, hq + 2 * hk, d, dtype=dtype, seed=4)
    q = qkv[:, :hq] if hq else None
    k, v = qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    cs = kt.rope_table(max(lens), rot)
    wq = _rand(d, dtype=dtype, seed=1) if norm else None
    wk = _rand(d, dtype=dtype, seed=2) if norm else None
    cache = kt.PagedKV(kp, vp)
    want_k, want_v = kp.double().cpu(), vp.double().cpu()
    bound = torch.zeros_like(want_k)
    pos = torch.cat([torch.arange(b, b + a) for a, b in zip(q_lens, past)]) if n else torch.zeros(0)
    rows, row_bound = R.head_rows(k[:n], wk, 1e-6, cs, pos, style)
    at = 0
    for b, a in enumerate(q_lens):
        for t in range(a):
            p = past[b] + t
            where = (int(table[b, p // page]), p % page)
            want_k[where], want_v[where], bound[where] = rows[at], v[at].double().cpu(), row_bound[at]
            at += 1
    q_out = None if q is None else torch.full(q.shape, 3.0, dtype=dtype, device=DEV)
    got_q = cache.append(k, v, table, R.starts(q_lens, DEV),
                         torch.tensor(lens, dtype=torch.int32, device=DEV), cs, q=q, q_weight=wq, k_weight=wk,
                         style=style, q_out=q_out)
    assert cache.read_error() == 0
    _near(kp, want_k, bound, "keys")
    assert torch.equal(vp.double().cpu(), want_v)
    if q is not None:
        _near(got_q[:n], *R.head_rows(q[:n], wq, 1e-6, cs, pos, style), "queries")
        assert bool((got_q[n:] == 3.0).all())
    else:
        assert got_q is None


def test_append_bad_pages_and_positions():
    """A page outside the cache, a length outside the table, a position outside the rotation: told, not written."""
    d, page = 64, 16
    kp = torch.zeros(4, page, 1, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    cache = kt.PagedKV(kp, vp)
    k = torch.ones(4, 1, d, dtype=torch.bfloat16, device=DEV)
    cu = R.starts([1, 1, 1, 1], DEV)
    bt = torch.tensor([[4, 0], [-1, 0], [1, 2], [3, 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1, 1, 33, 0], dtype=torch.int32, device=DEV)       # no page twice, past the table, before 0
    cache.append(k, k, bt, cu, lens)
    assert cache.read_error() == A.KT_DEVERR_BAD_PAGE and cache.read_error() == 0
    assert not bool(kp.any()) and not bool(vp.any())
    lens = torch.tensor([17, 17, 1, 8], dtype=torch.int32, device=DEV)
    cache.append(k, k, bt, cu, lens, kt.rope_table(8, d), q=k)
    assert cache.read_error() == A.KT_DEVERR_BAD_POSITION
    assert not bool(kp[0].any())
    assert bool(kp[1, 0].any()) and bool(kp[3, 7].any())


def test_append_past_32_bit_offsets():
    """Pages whose first element lies past 2^31 elements."""
    d, page, hk = 128, 64, 8
    pages = (1 << 31) // (page * hk * d) + 3
    kp = torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    k, v = _rand(2, hk, d, dtype=torch.bfloat16, seed=1), _rand(2, hk, d, dtype=torch.bfloat16, seed=2)
    bt = torch.tensor([[0, pages - 1]], dtype=torch.int32, device=DEV)
    kt.PagedKV(kp, vp).append(k, v, bt, R.starts([2], DEV), torch.tensor([page + 2], dtype=torch.int32, device=DEV))
    assert torch.equal(kp[pages - 1, :2], k) and torch.equal(vp[pages - 1, :2], v)
    assert not bool(kp[:2].any()) and not bool(kp[pages - 2].any())


def test_streams_and_graph():
    """On a stream of the caller's, and captured; the same bits each time."""
    n, h, d = 33, 4, 128
    q = _rand(n, h, d, dtype=torch.bfloat16, seed=8)
    w, table = torch.ones(d, device=DEV), kt.rope_table(64, d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    want, _ = kt.qk_norm_rope(q, None, pos, table, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = kt.qk_norm_rope(q, None, pos, table, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kt.qk_norm_rope(q, None, pos, table, w, q_out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
