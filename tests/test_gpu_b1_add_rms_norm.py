"""The residual's addition and the RMS norm, in 16 bits and in MXFP8, and the MoE layer on MXFP8 tokens."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt
from mxfp4_weight_moe_gb300 import synthetic as syn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def _within(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), f"{what}: {float((off - bound).max()):.3e} over the bound"


def _check_mx(mx, y, off):
    codes, scales = M.numbers(mx[0].cpu()), mx[1].cpu()
    n, h = y.shape
    top, slack = (t.reshape(n, -1, 32).amax(-1) for t in (y.abs(), off))
    x = scales.double() - 127
    low, high = M.floor_exponent((top - slack).clamp(min=2.0 ** -118)), M.floor_exponent(top + slack)
    assert bool(((x >= low) & (x <= high)).all()), "exponents"
    scale = torch.exp2(x).repeat_interleave(32, -1)
    assert float(M.off_by_a_rounding(codes, scale, y, off).max()) <= 0, "codes"


def _check(x, r, w, eps, y, s, mx):
    want_s, want_y, off = M.rms_rows(x, r, w, eps)
    dt = x.dtype
    tiny = R.TINY[dt]
    if s is not None:
        _within(s, want_s, R.ROUND[dt] * (1 + 2.0 ** -10) * want_s.abs() + tiny, "residual")
    if y is not None:
        _within(y, want_y, R.ROUND[dt] * (want_y.abs() + off) + off + tiny, "norm")
    if mx is not None:
        _check_mx(mx, want_y, off)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,h", [(1, 32), (3, 64), (5, 256), (9, 288), (2, 1024), (7, 1056), (1, 2048), (4, 2080),
                                 (3, 4096), (2, 7168), (1, 8192), (3, 8224), (2, 16416), (1, 32768)])
def test_sizes(dtype, n, h):
    x, r = _rand(n, h, dtype=dtype, seed=n + h), _rand(n, h, dtype=dtype, seed=h, scale=4.0)
    w = 1 + 0.1 * _rand(h, dtype=dtype, seed=2)
    kept = x.clone(), r.clone()
    y, s, mx = kt.add_rms_norm(x, w, r, mx=True)
    _check(x, r, w, 1e-6, y, s, mx)
    assert torch.equal(x, kept[0]) and torch.equal(r, kept[1])
    y2, s2, none = kt.add_rms_norm(x, w, r)
    assert none is None and torch.equal(y2, y) and torch.equal(s2, s)
    none, s2, mx2 = kt.add_rms_norm(x, w, r, plain=False, mx=True)
    assert none is None and torch.equal(s2, s) and all(torch.equal(a, b) for a, b in zip(mx, mx2))
    y, s, mx = kt.add_rms_norm(x, w.float(), eps=0.5, mx=True)
    assert s is None
    _check(x, None, w.float(), 0.5, y, s, mx)


@pytest.mark.parametrize("h", [8, 40, 264, 7160])
def test_sizes_of_no_whole_scale(h):
    x, r, w = (_rand(*s, dtype=torch.bfloat16, seed=h) for s in ((5, h), (5, h), (h,)))
    y, s, _ = kt.add_rms_norm(x, w, r)
    _check(x, r, w, 1e-6, y, s, None)
    with pytest.raises(ValueError, match="32"):
        kt.add_rms_norm(x, w, r, mx=True)


def test_many_rows_are_their_parts():
    """Steps beyond L2: the same bits as in parts."""
    n, h = 9001, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r = (torch.randn(n, h, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(h, device=DEV)
    y, s, mx = kt.add_rms_norm(x, w, r, mx=True)
    for lo in range(0, n, 1500):
        py, ps, pm = kt.add_rms_norm(x[lo:lo + 1500], w, r[lo:lo + 1500], mx=True)
        for whole, part in ((y, py), (s, ps), (mx[0], pm[0]), (mx[1], pm[1])):
            assert torch.equal(whole[lo:lo + 1500], part)
    _check(x[::3000], r[::3000], w, 1e-6, y[::3000], s[::3000], (mx[0][::3000], mx[1][::3000]))


def test_strides_and_places():
    """Rows of wider buffers, one row for all tokens, and outputs in place of the inputs."""
    n, h = 11, 320
    wide = _rand(n, 3 * h + 8, dtype=torch.float16, seed=1)
    x, r = wide[:, :h], wide[:, h:2 * h]
    w = torch.ones(h, dtype=torch.float16, device=DEV)
    y, s, mx = kt.add_rms_norm(x, w, r, mx=True)
    _check(x, r, w, 1e-6, y, s, mx)
    one = x[:1].expand(n, h)
    y1, _, _ = kt.add_rms_norm(one, w)
    assert torch.equal(y1, kt.add_rms_norm(one.contiguous(), w)[0])
    rest = wide[:, 2 * h:].clone()
    got = kt.add_rms_norm(x, w, r, out=x, residual_out=r)
    assert got[0] is x and got[1] is r and torch.equal(x, y) and torch.equal(r, s)
    assert torch.equal(wide[:, 2 * h:], rest)
    with pytest.raises(ValueError, match="shares"):
        kt.add_rms_norm(x, w, r, out=wide[:, 8:h + 8])
    with pytest.raises(ValueError, match="shares"):
        kt.add_rms_norm(x, w, r, out=x, residual_out=x)
    with pytest.raises(ValueError, match="needs"):
        kt.add_rms_norm(x, w, residual_out=r)
    with pytest.raises(ValueError, match="needs"):
        kt.add_rms_norm(x, w, plain=False, mx=True, out=x)


def test_extreme_rows():
    """Zeros, the smallest and largest numbers, and rows that are not finite, which stay among themselves."""
    h = 256
    x = _rand(6, h, dtype=torch.bfloat16, seed=6)
    x[0] = 0
    x[1] *= 1e-38
    x[2] *= 1e18
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    w = torch.ones(h, device=DEV)
    y, s, mx = kt.add_rms_norm(x, w, torch.zeros_like(x), mx=True)
    assert not bool(y[0].any()) and not bool(mx[0][0].any()) and not bool(mx[1][0].any())
    for i in (2, 5):
        _check(x[i:i + 1], None, w, 1e-6, y[i:i + 1], None, (mx[0][i:i + 1], mx[1][i:i + 1]))
    assert bool(y[3].isnan().all()) and bool(torch.isfinite(y[[0, 1, 2, 5]]).all())
    assert torch.equal(s, x + 0) or bool(s[3, 5].isnan())


def test_empty_stream_and_graph():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    y, s, mx = kt.add_rms_norm(x, w, x, mx=True)
    assert y.shape == s.shape == mx[0].shape == (0, 64) and mx[1].shape == (0, 2)
    x, r = _rand(33, 64, dtype=torch.bfloat16, seed=1), _rand(33, 64, dtype=torch.bfloat16, seed=2)
    want = kt.add_rms_norm(x, w, r, mx=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kt.add_rms_norm(x, w, r, mx=True, stream=side)
    side.synchronize()
    out, res = torch.zeros_like(x), torch.zeros_like(x)
    pair = tuple(torch.zeros_like(t) for t in want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kt.add_rms_norm(x, w, r, mx=True, out=out, residual_out=res, mx_out=pair)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip((*want[:2], *want[2]), (*got[:2], *got[2]), (out, res, *pair)):
        assert torch.equal(a, b) and torch.equal(a, c)


def _quantised(x):
    """(codes, scales) of the MoE layer's rule for bf16 rows, by torch."""
    b = x.float().unflatten(-1, (-1, 32))
    e = torch.where(b.abs().amax(-1) > 0, torch.frexp(b.abs().amax(-1))[1] - 9, -127).clamp(min=-127)
    codes = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(torch.uint8).contiguous(), (e + 127).to(torch.uint8)


@pytest.mark.parametrize("T,H,E,k,I", [(1, 128, 2, 2, 128), (7, 1152, 16, 4, 256), (300, 1024, 16, 4, 512),
                                       (70, 7168, 8, 2, 128)])
def test_moe_layer_on_mx_tokens(T, H, E, k, I):
    """The same bits as on the bf16 tokens whose quantisation they are."""
    W = [torch.stack(t).contiguous() for t in zip(*[syn.make_expert(e, H, I, 3, DEV) for e in range(E)])]
    hidden = _rand(T, H, dtype=torch.bfloat16, seed=4)
    hidden[0, :64] = 0
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(5)).to(DEV)
    mx = _quantised(hidden)
    ids, w, offs, perm, inv = kt.route_permute(logits, k)
    for options in ({}, {"gate_up": "interleaved", "activation": "swiglu_clamped"}):
        want = kt.forward(hidden, ids, w, *W, **options)
        assert torch.equal(kt.forward(mx, ids, w, *W, **options), want)
        assert torch.equal(kt.forward(mx, ids, w, *W, routing=(offs, perm, inv), **options), want)
        layer = kt.MoeLayer(*W, k, **options)
        want = layer(hidden, logits)[0].clone()
        assert torch.equal(layer(mx, logits)[0], want)
    with pytest.raises(ValueError, match="single launch"):
        kt.MoeLayer(*W, k, single_launch=True)(mx, logits)
    with pytest.raises(ValueError):
        kt.forward((mx[0], mx[1][:, :1].contiguous()), ids, w, *W)
    with pytest.raises(TypeError):
        kt.forward((mx[0].float(), mx[1]), ids, w, *W)


def test_norm_into_the_moe_layer():
    """The norm's MXFP8 tokens are what the layer quantises its 16-bit ones to, but for their second rounding.

    The layer's tokens are y rounded to bf16, then to e4m3: at most an e4m3 step from y rounded once."""
    T, H, E, k, I = 65, 1024, 16, 4, 512
    x, r = _rand(T, H, dtype=torch.bfloat16, seed=1), _rand(T, H, dtype=torch.bfloat16, seed=2, scale=3.0)
    y, _, mx = kt.add_rms_norm(x, torch.ones(H, device=DEV), r, mx=True)
    codes, scales = _quantised(y)
    same = (mx[1] == scales).repeat_interleave(32, -1)
    a, b = (M.numbers(t.cpu()) for t in (mx[0], codes))
    step = 2 * M.half_step(torch.maximum(a.abs(), b.abs()))
    assert bool(((a - b).abs() <= step)[same.cpu()].all()) and float(same.float().mean()) > 0.98
