"""Host-side checks of the 8-bit cache's C ABI and binding, and of its 64-bit statement (no GPU needed).

Every argument check returns its documented status before anything touches the GPU; pointers are fake addresses."""
import ctypes
import math
import struct

import pytest
import torch

import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A
from test_attn_host import ALIGN, HEADER, INVALID, KT_OK, SHAPE, WS, P, _ref, batch, heads, transform


class PagedKV8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")] + [
        (n, ctypes.c_int64) for n in ("k_page_stride", "k_slot_stride", "k_head_stride", "v_page_stride",
                                      "v_slot_stride", "v_head_stride")] + [
        (n, ctypes.c_int) for n in ("num_pages", "page_size", "heads", "head_dim", "dtype")]


def cache(**kw):
    d = dict(k=P, v=P, k_scales=P, v_scales=P, k_page_stride=16 * 2 * 128, k_slot_stride=2 * 128, k_head_stride=128,
             v_page_stride=16 * 2 * 128, v_slot_stride=2 * 128, v_head_stride=128, num_pages=4, page_size=16, heads=2,
             head_dim=128, dtype=0)
    d.update(kw)
    return PagedKV8(**d)


def test_packed_descriptor_is_the_header_s_struct():
    assert struct.calcsize(A.PAGED_KV8) == ctypes.sizeof(PagedKV8)
    values = [i + 1 for i in range(len(PagedKV8._fields_))]
    made = PagedKV8.from_buffer_copy(struct.pack(A.PAGED_KV8, *values))
    assert [getattr(made, n) for n, _ in PagedKV8._fields_] == values
    assert f"#define KT_KV8_BLOCK {kt.PagedKV8.BLOCK}\n" in open(HEADER).read() and kt.PagedKV8.BLOCK == M.BLOCK


def _bad_caches(call):
    assert call(c=None) == INVALID and call(c=cache(dtype=2)) == INVALID
    assert call(c=cache(page_size=24)) == SHAPE and call(c=cache(head_dim=144)) == SHAPE
    assert call(c=cache(head_dim=120)) == SHAPE and call(c=cache(num_pages=0)) == INVALID
    for name in ("k", "v", "k_scales", "v_scales"):
        assert call(c=cache(**{name: None})) == INVALID
    assert call(c=cache(v_slot_stride=0)) == INVALID and call(c=cache(v_slot_stride=264)) == ALIGN
    assert call(c=cache(k=P + 8)) == ALIGN and call(c=cache(k_page_stride=1 << 40)) == SHAPE


def _append(c=cache(), b=batch(), k=heads(n=2), v=heads(n=2), q=None, qo=None, tf=transform(), err=None):
    return kt.lib().kt_kv8_append(_ref(c), _ref(b), _ref(k), _ref(v), _ref(q), _ref(qo), _ref(tf), err, None)


def test_append_checks():
    _bad_caches(_append)
    assert _append(b=None) == INVALID and _append(k=None) == INVALID and _append(v=None) == INVALID
    assert _append(b=batch(tokens=0), k=heads(ptr=None)) == KT_OK and _append(b=batch(seqs=0)) == KT_OK
    assert _append(b=batch(seqs=-1)) == INVALID and _append(b=batch(cu_q=None)) == INVALID
    assert _append(k=heads(n=3)) == INVALID and _append(q=heads()) == INVALID
    assert _append(k=heads(ptr=P + 8, n=2)) == ALIGN and _append(v=heads(token=1028, n=2)) == ALIGN
    assert _append(q=heads(), qo=heads(n=4)) == INVALID and _append(err=P + 1) == ALIGN
    assert _append(tf=transform(rotary_dim=40)) == SHAPE and _append(tf=transform(rotary_dim=144)) == SHAPE
    assert _append(tf=transform(k_weight=P, eps=math.nan)) == INVALID


def _attend(c=cache(), b=batch(), q=heads(), out=heads(), max_q=3, scale=0.1, window=0, sinks=None, ws=P,
            ws_bytes=1 << 40):
    return kt.lib().kt_paged_attention8(_ref(c), _ref(b), _ref(q), _ref(out), max_q, scale, window, sinks, None, ws,
                                        ws_bytes, None)


def test_attention_checks():
    _bad_caches(_attend)
    need = kt.lib().kt_paged_attention_workspace_bytes()
    assert _attend(q=None) == INVALID and _attend(out=None) == INVALID and _attend(max_q=-1) == INVALID
    assert _attend(window=-1) == INVALID and _attend(scale=math.inf) == INVALID
    assert _attend(b=batch(tokens=0), q=heads(ptr=None), ws=None) == KT_OK
    assert _attend(q=heads(ptr=P + 8)) == ALIGN and _attend(q=heads(n=7), out=heads(n=7)) == INVALID
    assert _attend(c=cache(heads=1), q=heads(n=129), out=heads(n=129)) == SHAPE
    assert _attend(ws=None) == INVALID and _attend(ws=P + 64) == WS and _attend(ws_bytes=need - 1) == WS


def test_binding_refusals():
    pages, scales = torch.zeros(2, 32, 1, 64, dtype=torch.uint8), torch.zeros(2, 2, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kt.PagedKV8(pages, pages, scales, scales)
    with pytest.raises(TypeError):
        kt.PagedKV8(pages.half(), pages.half(), scales, scales)
    with pytest.raises(TypeError):
        kt.PagedKV8(pages, pages, scales, scales, torch.float32)


def test_the_statement_of_the_exponent():
    for dt in (torch.bfloat16, torch.float16):
        lo, hi = M.LEAST[dt], M.MOST[dt]
        x = torch.arange(lo, hi + 1, dtype=torch.float64)
        edge = 448 * torch.exp2(x)
        assert torch.equal(M.least_exponent(edge, dt), x)
        assert torch.equal(M.least_exponent(edge[:-1] * (1 + 1e-9), dt), x[1:])
        assert torch.equal(M.least_exponent(edge[1:] / 2 * (1 + 1e-9), dt), x[1:])
        assert float(M.least_exponent(torch.tensor(0.0, dtype=torch.float64), dt)) == lo
        # every number of such a block is one of the type
        codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
        v = M.numbers(codes)[:, None] * torch.exp2(x)
        assert torch.equal(v.to(dt).double(), v) and bool(v.to(dt).isfinite().all())


def test_rounding_statement():
    """What off_by_a_rounding allows: the nearest number, and nothing two steps further on (1.3 is more than 1.5 steps)."""
    v = torch.linspace(-500, 500, 4001, dtype=torch.float64)
    one = torch.ones(1, dtype=torch.float64)
    got = M.e4m3(v)
    assert float(M.off_by_a_rounding(got, one, v, 0 * v).max()) <= 0
    inside = (v.abs() > 1) & (v.abs() < 300)
    wrong = M.e4m3(got[inside] * 1.3)
    assert bool((M.off_by_a_rounding(wrong, one, v[inside], 0 * v[inside]) > 0).all())
