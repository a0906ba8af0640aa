"""Host-side checks of the attention operators' C ABI and binding (no GPU needed).

Every argument check returns its documented status before anything touches the
GPU; pointers are fake addresses that are never dereferenced.
"""
import ctypes
import math
import os
import re
import struct

import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import attention as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kt_attn.h")
KT_OK, INVALID, SHAPE, WS, ALIGN = 0, -1, -2, -3, -7
P = 0x7F0000000000


class Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int)]


class PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("k_page_stride", "k_slot_stride", "k_head_stride", "v_page_stride",
                                      "v_slot_stride", "v_head_stride")] + [
        (n, ctypes.c_int) for n in ("num_pages", "page_size", "heads", "head_dim", "dtype")]


class Batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("cu_q", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("seqs", ctypes.c_int),
                ("tokens", ctypes.c_int)]


class Transform(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("style", ctypes.c_int), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("weight_dtype", ctypes.c_int), ("eps", ctypes.c_float)]


def heads(ptr=P, token=1024, head=128, n=8):
    return Heads(ptr, token, head, n)


def cache(**kw):
    d = dict(k=P, v=P, k_page_stride=16 * 2 * 128, k_slot_stride=2 * 128, k_head_stride=128,
             v_page_stride=16 * 2 * 128, v_slot_stride=2 * 128, v_head_stride=128, num_pages=4, page_size=16, heads=2,
             head_dim=128, dtype=0)
    d.update(kw)
    return PagedKV(**d)


def batch(**kw):
    d = dict(block_table=P, table_stride=8, max_pages=8, cu_q=P, seq_lens=P, seqs=2, tokens=5)
    d.update(kw)
    return Batch(**d)


def transform(**kw):
    d = dict(table=P, positions=64, rotary_dim=128, style=0, q_weight=None, k_weight=None, weight_dtype=0, eps=1e-6)
    d.update(kw)
    return Transform(**d)


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(kt_[a-z0-9_]+)\s*\(", src))
    assert declared == set(A.SIGNATURES)
    assert not [n for n in declared if not hasattr(kt.lib(), n)]


def test_packed_descriptors_are_the_header_s_structs():
    for fmt, s in ((A.HEADS, Heads), (A.PAGED_KV, PagedKV), (A.PAGED_BATCH, Batch), (A.HEAD_TRANSFORM, Transform)):
        assert struct.calcsize(fmt) == ctypes.sizeof(s)
        values = [i + 1 for i in range(len(s._fields_))]
        made = s.from_buffer_copy(struct.pack(fmt, *values))
        assert [getattr(made, n) for n, _ in s._fields_] == values
    assert A._buffer.buf._length_ >= max(x.size for x in (A._NORM_CALL, A._APPEND_CALL, A._ATTEND_CALL))
    src = open(HEADER).read()
    assert f"#define KT_PAGED_ATTENTION_ZEROED {A.WORKSPACE_ZEROED}\n" in src
    for name in ("KT_DEVERR_BAD_PAGE", "KT_DEVERR_BAD_POSITION"):
        assert f"#define {name} 0x{getattr(A, name):x} " in src


def _norm(q=heads(), k=heads(n=2), qo=heads(), ko=heads(n=2), positions=P, tokens=3, dim=128, dtype=0,
          tf=transform(), err=None):
    return kt.lib().kt_qk_norm_rope(_ref(q), _ref(k), _ref(qo), _ref(ko), positions, tokens, dim, dtype, _ref(tf), err,
                                    None)


def test_norm_rope_checks():
    assert _norm(q=None) == INVALID and _norm(qo=None) == INVALID and _norm(ko=None) == INVALID
    assert _norm(tf=None) == INVALID
    assert _norm(dtype=2) == INVALID
    assert _norm(tokens=-1) == INVALID
    assert _norm(dim=100) == SHAPE and _norm(dim=264) == SHAPE
    assert _norm(tokens=0, q=heads(ptr=None)) == KT_OK
    assert _norm(q=heads(ptr=None)) == INVALID
    assert _norm(q=heads(ptr=P + 4)) == ALIGN
    assert _norm(q=heads(token=1026)) == ALIGN
    assert _norm(q=heads(n=0)) == INVALID
    assert _norm(qo=heads(n=4)) == INVALID
    assert _norm(positions=None) == INVALID
    assert _norm(positions=P + 2) == ALIGN
    assert _norm(tf=transform(style=2)) == INVALID
    assert _norm(tf=transform(rotary_dim=136)) == SHAPE and _norm(tf=transform(rotary_dim=12)) == SHAPE
    assert _norm(tf=transform(positions=0)) == INVALID
    assert _norm(tf=transform(table=P + 4)) == ALIGN
    assert _norm(tf=transform(q_weight=P, weight_dtype=1)) == INVALID
    assert _norm(tf=transform(q_weight=P, eps=math.nan)) == INVALID
    assert _norm(tf=transform(q_weight=P + 1)) == ALIGN
    assert _norm(tokens=1 << 30, q=heads(n=64), qo=heads(n=64)) == SHAPE


def _append(c=cache(), b=batch(), k=heads(n=2), v=heads(n=2), q=None, qo=None, tf=transform(), err=None):
    return kt.lib().kt_kv_append(_ref(c), _ref(b), _ref(k), _ref(v), _ref(q), _ref(qo), _ref(tf), err, None)


def test_append_checks():
    assert _append(c=None) == INVALID and _append(b=None) == INVALID and _append(k=None) == INVALID
    assert _append(b=batch(tokens=0), k=heads(ptr=None)) == KT_OK and _append(b=batch(seqs=0)) == KT_OK
    assert _append(c=cache(dtype=2)) == INVALID
    assert _append(c=cache(page_size=24)) == SHAPE and _append(c=cache(head_dim=136)) == SHAPE
    assert _append(c=cache(head_dim=100)) == SHAPE
    assert _append(c=cache(num_pages=0)) == INVALID and _append(c=cache(k=None)) == INVALID
    assert _append(c=cache(v_slot_stride=0)) == INVALID and _append(c=cache(v_slot_stride=260)) == ALIGN
    assert _append(c=cache(k=P + 8)) == ALIGN
    assert _append(b=batch(seqs=-1)) == INVALID and _append(b=batch(seqs=1 << 17)) == SHAPE
    assert _append(b=batch(cu_q=None)) == INVALID and _append(b=batch(block_table=None)) == INVALID
    assert _append(b=batch(seq_lens=P + 2)) == ALIGN
    assert _append(k=heads(n=3)) == INVALID
    assert _append(q=heads()) == INVALID
    assert _append(q=heads(), qo=heads(n=4)) == INVALID
    assert _append(err=P + 1) == ALIGN


def _attend(c=cache(), b=batch(), q=heads(), out=heads(), max_q=3, scale=0.1, window=0, sinks=None, ws=P,
            ws_bytes=1 << 40):
    return kt.lib().kt_paged_attention(_ref(c), _ref(b), _ref(q), _ref(out), max_q, scale, window, sinks, None, ws,
                                       ws_bytes, None)


def test_attention_checks():
    need = kt.lib().kt_paged_attention_workspace_bytes()
    assert need > A.WORKSPACE_ZEROED
    assert _attend(c=None) == INVALID and _attend(q=None) == INVALID and _attend(out=None) == INVALID
    assert _attend(max_q=-1) == INVALID and _attend(window=-1) == INVALID
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert _attend(scale=scale) == INVALID
    assert _attend(b=batch(tokens=0), q=heads(ptr=None), ws=None) == KT_OK
    assert _attend(q=heads(ptr=P + 8)) == ALIGN and _attend(out=heads(token=1028)) == ALIGN
    assert _attend(q=heads(n=7), out=heads(n=7)) == INVALID and _attend(out=heads(n=4)) == INVALID
    assert _attend(c=cache(heads=1), q=heads(n=129), out=heads(n=129)) == SHAPE
    assert _attend(b=batch(tokens=1 << 28)) == SHAPE
    assert _attend(sinks=P + 2) == ALIGN
    assert _attend(ws=None) == INVALID and _attend(ws=P + 64) == WS and _attend(ws_bytes=need - 1) == WS
    assert "workspace" in kt.lib().kt_last_error().decode()


def test_binding_refusals():
    """What the binding checks before the library is called."""
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kt.qk_norm_rope(q, None, q_weight=torch.ones(64))
    with pytest.raises(TypeError):
        kt.qk_norm_rope(q.float(), None)
    with pytest.raises(TypeError):
        kt.qk_norm_rope(None, None)
    with pytest.raises(TypeError):
        kt.PagedKV(torch.zeros(2, 16, 1, 64), torch.zeros(2, 16, 1, 64))
    with pytest.raises(ValueError):
        kt.PagedKV(torch.zeros(2, 16, 1, 64, dtype=torch.float16), torch.zeros(2, 16, 1, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        kt.rope_table(16, 12, device="cpu")
    with pytest.raises(ValueError):
        A._written(torch.zeros(3, 1, 8).expand(3, 4, 8), "out")
    with pytest.raises(ValueError):
        A._written(torch.zeros(64).as_strided((3, 2, 8), (12, 8, 1)), "out")
    A._written(torch.zeros(2, 3, 8).transpose(0, 1), "out")
    A._written(torch.zeros(3, 6, 8)[:, :4], "out")


def test_rope_table():
    t = kt.rope_table(50, 16, 100.0, device="cpu")
    assert t.shape == (50, 16) and t.dtype == torch.float32
    for p in (0, 1, 49):
        for i in range(8):
            a = p * 100.0 ** (-2 * i / 16)
            assert abs(float(t[p, i]) - math.cos(a)) < 1e-6 and abs(float(t[p, 8 + i]) - math.sin(a)) < 1e-6


def test_oracle_against_a_dense_softmax():
    """The 64-bit statement of the paged attention, against torch's dense softmax on one sequence."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, h, 16, generator=g, dtype=torch.float64) for n, h in ((5, 4), (12, 2), (12, 2)))
    kp = torch.zeros(3, 16, 2, 16, dtype=torch.float64)
    vp = torch.zeros_like(kp)
    kp[2, :12], vp[2, :12] = k, v
    # (its bound needs a 16-bit type: the values are 16-bit ones)
    q, kp, vp = q.half(), kp.half(), vp.half()
    out, bound = R.attend(q, kp, vp, torch.tensor([[2]]), [5], [12], 0.25)
    for h in range(4):
        x = 0.25 * q[:, h].double() @ kp[2, :12, h // 2].double().T
        x.masked_fill_(torch.ones(5, 12, dtype=torch.bool).triu(8), -math.inf)
        want = torch.softmax(x, -1) @ vp[2, :12, h // 2].double()
        assert torch.allclose(out[:, h], want, rtol=0, atol=1e-12)
    assert bool((bound > 0).all()) and float(bound.max()) < 1e-2
