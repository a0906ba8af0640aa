"""Every key that a token sees counts once: attention whose output is a count.

Queries are zero, so that every weight is one and the sum is the number of keys n.  A value is one in a single
element, which the key's position picks, and zero elsewhere: the output is that element's number of keys over n.  Both
numbers are whole and below 2^24, sums of them are exact in fp32, and the division and the rounding to fp16 leave a
relative error of at most 2^-11 + 2^-22 (2^-25 where fp16 has no smaller step).  An element counts at most 700 keys, so
that one key lost or taken twice changes it by more than 2^-10 of itself."""
import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOUND, TINY = 2.0 ** -11 + 2.0 ** -22, 2.0 ** -25


def _count(q_lens, past, hq, hk, d, page, window, max_q, pick):
    lens = [a + b for a, b in zip(q_lens, past)]
    need = [-(-n // page) for n in lens]
    pages, n = sum(need), sum(q_lens)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32).to(DEV)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    kp = torch.randn(pages, page, hk, d, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).half()
    vp = torch.full_like(kp, 3.0)                     # past the sequences' ends: would count thrice
    want = torch.zeros(n, d, dtype=torch.float64, device=DEV)
    at = row = 0
    for b, (ql, length) in enumerate(zip(q_lens, lens)):
        table[b, :need[b]] = order[at:at + need[b]]
        key = torch.arange(length, device=DEV)
        one = torch.nn.functional.one_hot(pick(key) % d, d)
        rows = torch.full((need[b] * page, d), 3.0, device=DEV)
        rows[:length] = one.float()
        vp[order[at:at + need[b]].long()] = rows.half().view(need[b], page, 1, d).expand(-1, -1, hk, -1)
        seen = torch.cat((torch.zeros(1, d, dtype=torch.int64, device=DEV), one.cumsum(0)))
        pos = torch.arange(length - ql, length, device=DEV)
        lo = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
        counts = seen[pos + 1] - seen[lo]
        assert ql == 0 or int(counts.max()) <= 700
        want[row:row + ql] = counts.double() / (pos + 1 - lo)[:, None]
        at, row = at + need[b], row + ql
    cache = kt.PagedKV(kp, vp)
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
                                               (8, 8, 128, 333)])
@pytest.mark.parametrize("d", [64, 96])
def test_single_tokens_of_many_sequences(d, hq, hk, page, window):
    g = torch.Generator().manual_seed(hq)
    past = torch.randint(0, 8000, (60,), generator=g).tolist() + [0, 1, 40_000]
    _both_ways([1] * len(past), past, hq, hk, d, page, window)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("new,past,group,window", [(20, 60, 1, 0), (33, 30000, 8, 0), (257, 2000, 8, 0),
                                                   (1500, 0, 3, 0), (600, 3333, 5, 0), (700, 900, 4, 128),
                                                   (130, 20001, 16, 0), (300, 5000, 8, 1000)])
def test_a_chunk(new, past, group, window, d):
    _both_ways([new], [past], group, 1, d, 16 if new % 2 else 64, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q", [1, None])
def test_mixed_batches(d, max_q):
    """Chunks and single tokens over both kernels (the bound on new tokens picks one)."""
    g = torch.Generator().manual_seed(7)
    q_lens = [1 if i % 3 else int(torch.randint(1, 300, (1,), generator=g)) for i in range(20)] + [0]
    past = torch.randint(0, 9000, (21,), generator=g).tolist()
    _both_ways(q_lens, past, 8, 2, d, 32, 0, max_q)
