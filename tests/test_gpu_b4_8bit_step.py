"""A decoder layer's step in 8 bits as a serving program runs it, and every key of an 8-bit cache counted once."""
import importlib.util
import os

import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


def _example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts,kw", [
    ((37, 150), {}),
    ((1, 15, 400), {"q_heads": 12, "kv_heads": 4, "head_dim": 64, "decode": 20}),
])
def test_decoding_matches_one_prefill(prompts, kw):
    """Tokens decoded one by one over an 8-bit cache against the same tokens in one prefill.

    A block's power of two may be smaller while it fills than at its end.  That changes an element's number only where
    the code is an e4m3 subnormal, by at most 2^-10 of the power, 2^-17.8 of the block's largest element.  What remains
    is as over a 16-bit cache: the attention kernels' roundings (2^-8) and the experts' activations that they move by a
    step (2^-4, a few percent of them): 1e-2 of a token's norm; 5e-2 is allowed.  Every expert is picked."""
    assert _example().run(prompts, experts=4, top_k=4, cache_bits=8, **kw) < 5e-2


def test_step_in_a_graph():
    """Norm, append, attention, norm and experts captured in one graph: the same bits as called one by one."""
    ex = _example()
    layer = ex.DecoderLayer(512, 8, 2, 64, experts=8, top_k=2, inter=256, num_pages=40, cache_bits=8)
    pages = ex.Pages(40, 16, DEV)
    for _ in range(3):
        pages.add_sequence()
    g = torch.Generator(device=DEV).manual_seed(1)
    xs = [torch.randn(n, 512, generator=g, device=DEV).to(torch.bfloat16) for n in (120, 3, 3)]
    layer(xs[0], *pages.step([100, 3, 17]))
    step = pages.step([1, 1, 1])
    saved = [t.clone() for t in (layer.cache.k_pages.view(torch.uint8), layer.cache.v_pages.view(torch.uint8),
                                 layer.cache.k_scales, layer.cache.v_scales)]

    def restore():
        for t, s in zip((layer.cache.k_pages.view(torch.uint8), layer.cache.v_pages.view(torch.uint8),
                         layer.cache.k_scales, layer.cache.v_scales), saved):
            t.copy_(s)

    want = layer(xs[1], *step).clone()
    after = [t.clone() for t in (layer.cache.k_pages.view(torch.uint8), layer.cache.k_scales)]
    restore()
    x = xs[1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                # warm-up of the matmuls
        layer(x, *step)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, *step)
    restore()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for a, b in zip(after, (layer.cache.k_pages.view(torch.uint8), layer.cache.k_scales)):
        assert torch.equal(a, b)
    x.copy_(xs[2])
    restore()
    graph.replay()
    got = out.clone()
    restore()
    assert torch.equal(got, layer(xs[2], *step)) and layer.cache.read_error() == 0


# Queries are zero, so that every weight is one and the sum is the number of keys n.  A value is one in a single
# element, which the key's position picks, and zero elsewhere: the output is that element's number of keys over n.
# Numbers, sums (of 700 at most, times 2^10 at most) and their powers of two are exact in fp32; the division and the
# rounding to fp16 leave a relative error of at most 2^-11 + 2^-22 (2^-25 where fp16 has no smaller step).  One key of
# 700 lost or taken twice changes the output by more than 2^-10 of itself.
BOUND, TINY = 2.0 ** -11 + 2.0 ** -22, 2.0 ** -25


def _count(q_lens, past, hq, hk, d, page, window, max_q, pick):
    lens = [a + b for a, b in zip(q_lens, past)]
    need = [-(-n // page) for n in lens]
    pages, n = sum(need), sum(q_lens)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32).to(DEV)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    kp = torch.randint(0, 0x7f, (pages, page, hk, d), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    vp = torch.full_like(kp, 0x44)                    # 3, past the sequences' ends: would count thrice
    # every block's own power of two, and values that are 1 under it: codes of 2^-3 to 2^3
    shift = torch.randint(-3, 4, (pages, page // 16, hk), generator=g, device=DEV, dtype=torch.int32)
    vs = (127 + shift).to(torch.uint8)
    ks = torch.full_like(vs, 120)
    one_of = ((7 - shift) << 3).to(torch.uint8).repeat_interleave(16, 1)[..., None]     # e4m3 of 2^-shift
    want = torch.zeros(n, d, dtype=torch.float64, device=DEV)
    at = row = 0
    for b, (ql, length) in enumerate(zip(q_lens, lens)):
        mine = order[at:at + need[b]]
        table[b, :need[b]] = mine
        key = torch.arange(length, device=DEV)
        one = torch.nn.functional.one_hot(pick(key) % d, d)
        rows = torch.full((need[b] * page, d), -1, device=DEV)
        rows[:length] = one
        rows = rows.view(need[b], page, 1, d)
        vp[mine.long()] = torch.where(rows < 0, vp[mine.long()], torch.where(rows == 1, one_of[mine.long()], 0))
        seen = torch.cat((torch.zeros(1, d, dtype=torch.int64, device=DEV), one.cumsum(0)))
        pos = torch.arange(length - ql, length, device=DEV)
        lo = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
        counts = seen[pos + 1] - seen[lo]
        assert ql == 0 or int(counts.max()) <= 700
        want[row:row + ql] = counts.double() / (pos + 1 - lo)[:, None]
        at, row = at + need[b], row + ql
    cache = kt.PagedKV8(kp, vp, ks, vs, torch.float16)
    out = cache.attend(torch.zeros(n, hq, d, dtype=torch.float16, device=DEV), table, R.starts(q_lens, DEV),
                       torch.tensor(lens, dtype=torch.int32, device=DEV), max_q, window=window)
    assert cache.read_error() == 0
    over = (out.double() - want[:, None]).abs() > (BOUND * want + TINY * (want > 0))[:, None]
    assert not bool(over.any()), f"{int(over.sum())} counts are off"


def _both_ways(q_lens, past, hq, hk, d, page, window=0, max_q=None):
    """By the position's last digits, so that an element's keys lie far apart, and by its first ones, together."""
    max_q = max(q_lens) if max_q is None else max_q
    most = max(a + b for a, b in zip(q_lens, past))
    _count(q_lens, past, hq, hk, d, page, window, max_q, lambda key: key)
    _count(q_lens, past, hq, hk, d, page, window, max_q, lambda key: key // -(-most // d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("past", [0, 1, 15, 16, 63, 64, 127, 500, 2047, 9001, 30000])
def test_one_token(d, past):
    _both_ways([1], [past], 8, 1, d, 64 if past % 2 else 16)


@pytest.mark.parametrize("hq,hk,page,window", [(4, 4, 16, 0), (64, 8, 64, 0), (10, 2, 48, 0), (8, 1, 16, 128),
                                               (8, 8, 128, 333), (24, 2, 32, 0), (80, 80, 16, 0)])
@pytest.mark.parametrize("d", [64, 96])
def test_single_tokens_of_many_sequences(d, hq, hk, page, window):
    g = torch.Generator().manual_seed(hq)
    past = torch.randint(0, 8000, (60,), generator=g).tolist() + [0, 1, 40_000]
    _both_ways([1] * len(past), past, hq, hk, d, page, window)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("new,past,group,window", [(2, 9000, 8, 0), (3, 700, 5, 0), (4, 3000, 8, 100), (20, 60, 1, 0),
                                                   (33, 30000, 8, 0), (257, 2000, 8, 0), (1500, 0, 3, 0),
                                                   (700, 900, 4, 128), (130, 20001, 16, 0), (300, 5000, 8, 1000)])
def test_a_chunk(new, past, group, window, d):
    _both_ways([new], [past], group, 1, d, 16 if new % 2 else 64, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q", [1, 2, None])
def test_mixed_batches(d, max_q):
    """Chunks and single tokens over every kernel (the bound on new tokens picks one)."""
    g = torch.Generator().manual_seed(7)
    q_lens = [1 if i % 3 else int(torch.randint(1, 300, (1,), generator=g)) for i in range(20)] + [0]
    past = torch.randint(0, 9000, (21,), generator=g).tolist()
    _both_ways(q_lens, past, 8, 1, d, 32, 0, max_q)
