"""Which outputs of the attention operators share memory with what the call reads (CPU tensors; nothing is launched)."""
import random

import pytest
import torch

from mxfp4_weight_moe_gb300 import attention as A


def _desc(t):
    n, h, d = t.shape
    by_token, by_head, _ = t.stride()
    return t.data_ptr(), (by_token if n > 1 else d), (by_head if h > 1 else d), h


def _elements(t):
    at = (t.data_ptr() - t.untyped_storage().data_ptr()) // 2
    (n, h, d), st = t.shape, t.stride()
    return {at + i * st[0] + j * st[1] + e for i in range(n) for j in range(h) for e in range(d)}


def _refused(out, own, others=(), spans=()):
    n, _, d = out.shape
    try:
        A._apart("out", _desc(out), n, d, _desc(own), [_desc(x) for x in others], spans)
    except ValueError:
        return True
    return False


def test_outputs_that_may_be():
    qkv = torch.zeros(5, 6, 8, dtype=torch.bfloat16)
    q, k, v = qkv.split((4, 1, 1), dim=1)
    assert not _refused(q, q, (k, v)) and not _refused(k, k, (q, v)) and not _refused(v, q, (k,))
    each = torch.zeros(5, 4, 3, 8, dtype=torch.bfloat16).unbind(2)      # q, k, v of a head side by side
    assert not _refused(each[0], each[0], each[1:]) and not _refused(each[2], each[0], each[1:2])
    assert not _refused(torch.zeros_like(q), q, (k, v))
    assert not _refused(qkv[:0, :4], qkv[:0, 1:5])
    assert not _refused(qkv[:1, :4], qkv[1:2, :4])


def test_outputs_that_may_not_be():
    qkv = torch.zeros(5, 6, 8, dtype=torch.bfloat16)
    q, k, v = qkv.split((4, 1, 1), dim=1)
    assert _refused(qkv[:, 1:5], q) and _refused(qkv[:, 2:], q, (k,))   # a head further on
    assert _refused(q, torch.zeros_like(q), (q,))                        # another's input
    assert _refused(k, q, (k,)) and _refused(q, q, (k, qkv[:, 3:4]))
    flat = torch.zeros(200, dtype=torch.bfloat16)
    assert _refused(flat[8:168].view(5, 4, 8), flat[:160].view(5, 4, 8))            # a row further on
    assert _refused(flat[4:164].view(5, 4, 8), flat[:160].view(5, 4, 8))            # half a row
    assert _refused(flat[:160].view(4, 5, 8).transpose(0, 1), flat[:160].view(5, 4, 8))   # the same memory, turned
    one = flat[:32].view(1, 4, 8)
    assert _refused(flat[:160].view(5, 4, 8), one.expand(5, 4, 8))
    pages = torch.zeros(3, 16, 2, 8, dtype=torch.bfloat16)
    span = (pages.data_ptr(), pages.data_ptr() + pages.numel() * 2)
    assert _refused(pages[1, :5], q, (), (span,)) and not _refused(q, q, (), (span,))


@pytest.mark.parametrize("seed", range(40))
def test_drawn_layouts_against_their_elements(seed):
    r = random.Random(seed)
    store = torch.zeros(4096, dtype=torch.bfloat16)
    for _ in range(50):
        n, d = r.randint(1, 5), r.choice((4, 8, 12))
        made = []
        for _ in range(2):
            h = r.randint(1, 4)
            strides = r.choice(((h * d + r.choice((0, 4, 24)), d), (d, n * d), (72, 24), (96, 16),
                                (4 * r.randint(0, 30), 4 * r.randint(0, 30))))
            made.append(store.as_strided((n, h, d), (*strides, 1), 4 * r.randint(0, 60)))
        out, x = made
        if n > 1 and out.stride(0) < 4 or out.shape[1] > 1 and out.stride(1) < 4:
            continue                                                     # (such an output is refused before)
        same = _desc(out) == _desc(x)
        assert _refused(out, x) == (not same and bool(_elements(out) & _elements(x)))
        other = torch.zeros(n, 1, d, dtype=torch.bfloat16)
        assert _refused(out, other, (x,)) == bool(_elements(out) & _elements(x))
