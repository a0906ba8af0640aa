"""Host-side checks of the residual norm's C ABI and binding, and of its 64-bit statement (no GPU needed).

Every argument check returns its documented status before anything touches the GPU; pointers are fake addresses."""
import ctypes
import math
import os
import re

import pytest
import torch

import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import norm as N

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kt_norm.h")
KT_OK, INVALID, SHAPE, WS, ALIGN = 0, -1, -2, -3, -7
P = 0x7F0000000000


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64)]


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def rows(ptr=P, stride=256):
    return Rows(ptr, stride)


def _norm(x=rows(), r=rows(), w=P, wt=0, eps=1e-6, tokens=3, hidden=256, dtype=0, ro=rows(), out=rows(), codes=P,
          scales=P):
    return kt.lib().kt_add_rms_norm(_ref(x), _ref(r), w, wt, eps, tokens, hidden, dtype, _ref(ro), _ref(out), codes,
                                    scales, None)


def test_header_and_binding_agree():
    src = open(HEADER).read()
    declared = set(re.findall(r"\b(kt_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert declared == set(N.SIGNATURES) and all(hasattr(kt.lib(), n) for n in declared)
    assert f"#define KT_NORM_MAX_HIDDEN {N.MAX_HIDDEN}\n" in src
    assert N._ROWS_BYTES == ctypes.sizeof(Rows)


def test_argument_checks():
    assert _norm(dtype=2) == INVALID and _norm(wt=1) == INVALID and _norm(tokens=-1) == INVALID
    assert _norm(hidden=0) == INVALID and _norm(hidden=252) == SHAPE and _norm(hidden=248) == SHAPE
    assert _norm(hidden=N.MAX_HIDDEN + 32) == SHAPE
    for eps in (math.nan, math.inf, -1e-6):
        assert _norm(eps=eps) == INVALID
    assert _norm(codes=None) == INVALID and _norm(scales=None) == INVALID
    assert _norm(tokens=0, x=None) == KT_OK
    assert _norm(ro=None, out=None, codes=None, scales=None) == INVALID
    assert _norm(r=None) == INVALID and _norm(r=rows(ptr=None)) == INVALID       # residual_out without a residual
    assert _norm(x=None) == INVALID and _norm(x=rows(ptr=None)) == INVALID and _norm(w=None) == INVALID
    assert _norm(x=rows(ptr=P + 8)) == ALIGN and _norm(out=rows(stride=252)) == ALIGN
    assert _norm(r=rows(stride=-8)) == INVALID and _norm(ro=rows(ptr=P + 2)) == ALIGN
    assert _norm(w=P + 4) == ALIGN and _norm(codes=P + 8) == ALIGN


def _forward(codes=P, scales=P, routing=(None, None, None), T=2, H=256):
    return kt.lib().kt_mxfp4_moe_forward_mx(codes, scales, T, H, P, P, 2, *routing, P, P, P, P, 4, 128, P, P, 0, None,
                                            None)


def test_forward_of_mx_tokens_checks():
    assert _forward(codes=None) == INVALID and _forward(scales=None) == INVALID
    assert _forward(codes=P + 8) == ALIGN and _forward(scales=P + 2) == ALIGN
    assert _forward(routing=(P, None, P)) == INVALID and _forward(routing=(P, P, P + 4)) == ALIGN
    assert _forward(H=200) == SHAPE and _forward(T=0, codes=None) == KT_OK
    assert _forward() == WS                                  # the last check before a launch: a workspace of no bytes


def test_binding_refusals():
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        kt.add_rms_norm(x, w)
    for wrong in (x.float(), x[0], None):
        with pytest.raises(TypeError):
            kt.add_rms_norm(wrong, w)
    with pytest.raises(TypeError):
        kt.add_rms_norm(x, None)


def _row(t):
    return ("t", t.data_ptr(), 2 * t.stride(0), 2 * t.shape[1])


def test_outputs_that_share_memory():
    wide = torch.zeros(5, 96, dtype=torch.bfloat16)
    a, b, c = wide[:, :32], wide[:, 32:64], wide[:, 64:]

    def refused(outs, ins):
        try:
            N._apart([_row(o) for o in outs], [_row(i) for i in ins], 5, 32)
        except ValueError:
            return True
        return False

    assert not refused([a], [a, b]) and not refused([c, b], [a, b]) and not refused([a, b], [a, b])
    assert refused([wide[:, 8:40]], [a, b]) and refused([a, a], [b]) and refused([wide[:, 24:56]], [c, b])
    assert refused([a.as_strided((5, 32), (16, 1))], [c])                    # rows that overlap
    flat = torch.zeros(400, dtype=torch.bfloat16)
    assert refused([flat[32:192].view(5, 32)], [flat[:160].view(5, 32)])    # a row further on
    assert not refused([flat[160:320].view(5, 32)], [flat[:160].view(5, 32)])


def test_e4m3_statement_against_torch():
    """The 64-bit rounding, on every number of the format, the points between them and past the ends."""
    codes = torch.arange(256, dtype=torch.uint8)
    v = M.numbers(codes)
    v = v[v.isfinite()].sort().values
    assert torch.equal(M.e4m3(v), v)
    mid = (v[1:] + v[:-1]) / 2
    for x in (mid, mid * (1 + 1e-6), mid * (1 - 1e-6)):
        assert torch.equal(M.e4m3(x), x.float().to(torch.float8_e4m3fn).double())
    assert float(M.e4m3(torch.tensor(1e9, dtype=torch.float64))) == 448
    assert bool(((v[1:] - v[:-1]) / 2 <= M.half_step(torch.maximum(v[1:].abs(), v[:-1].abs()))).all())
