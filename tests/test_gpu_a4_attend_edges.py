"""Attention over a paged cache where it can go wrong in small ways: the weights' own error, pages behind a window."""
import pytest
import torch

import attn_oracle as R
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _weights_total(q, k_pages, v_pages, table, lens, scale):
    """(out, sum of weight |value|, sum of |value|, fp32 error of a weight) of single tokens, in 64 bits."""
    n, hq, d = q.shape
    hk = k_pages.shape[2]
    out, by_weight, plain, off = (torch.zeros(n, hq, d, dtype=torch.float64) for _ in range(4))
    for b, length in enumerate(lens):
        used = table[b, :-(-length // k_pages.shape[1])].long().cpu()
        kk, vv = (t.double().cpu()[used].flatten(0, 1)[:length] for t in (k_pages, v_pages))
        for h in range(hq):
            x = scale * (kk[:, h * hk // hq] @ q[b, h].double().cpu())
            size = scale * (kk[:, h * hk // hq].abs() @ q[b, h].double().cpu().abs())
            p = torch.softmax(x, 0)
            v = vv[:, h * hk // hq]
            out[b, h], by_weight[b, h], plain[b, h] = p @ v, p @ v.abs(), v.abs().sum(0)
            off[b, h] = (d + 4) * R.F32 * (size.max() + 2 * x.abs().max()) + (2 * length + 64) * R.F32
    return out, by_weight, plain, off


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_weights_of_few_rows_keep_two_parts(dtype, d):
    """The kernel for few rows multiplies the values with each softmax weight in two 16-bit parts.

    Bound: the result's one rounding, the weights' error of a 16-bit rounding of what a 16-bit rounding left (fp16: or
    half its smallest step, to each of two parts), and fp32 arithmetic as in the 64-bit statement.  Few keys and small
    logits, so that the arithmetic's part is far below a 16-bit rounding of the weights."""
    lens, hq, hk, page = [2, 3, 4, 5, 6, 9, 14, 31], 16, 2, 16
    kp, vp, table = R.paged(lens, page, hk, d, dtype, DEV, 11)
    q = _rand(len(lens), hq, d, dtype=dtype, seed=12, scale=0.5)
    scale = R.softmax_scale(d)
    cache = kt.PagedKV(kp, vp)
    out = cache.attend(q, table, R.starts([1] * len(lens), DEV), _i32(lens), 1)
    assert cache.read_error() == 0
    want, by_weight, plain, off = _weights_total(q, kp, vp, table, lens, scale)
    bound = 1.01 * (R.ROUND[dtype] * want.abs() + (R.ROUND[dtype] ** 2 + 2 * off) * by_weight
                    + 2 * R.TINY[dtype] * plain) + R.TINY[dtype]
    over = (out.double().cpu() - want).abs() - bound
    assert float(over.max()) <= 0, f"{int((over > 0).sum())} of {over.numel()} over the bound, {float(over.max()):.2e}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [1, 40])
def test_infinite_values_that_a_token_sees(dtype, new):
    """An infinite element of a value that every token sees makes that element of their outputs infinite, no other.

    Position 0 holds it, with a key that is zero: no logit is far above it, so that its weight is no zero."""
    d, page, n = 64, 16, new + 20
    kp, vp, table = R.paged([n], page, 1, d, dtype, DEV, 31)
    q = _rand(new, 2, d, dtype=dtype, seed=32, scale=0.25)
    first = int(table[0, 0])
    kp[first, 0] = 0
    vp[first, 0, 0, 5], vp[first, 0, 0, 50] = float("inf"), float("-inf")
    out = kt.PagedKV(kp, vp).attend(q, table, R.starts([new], DEV), _i32([n]), new)
    want, bound = R.attend(q, kp, vp, table, [new], [n], R.softmax_scale(d))
    assert bool((out[..., 5] == float("inf")).all()) and bool((out[..., 50] == float("-inf")).all())
    rest = [i for i in range(d) if i not in (5, 50)]
    assert bool(((out.double().cpu() - want)[..., rest].abs() <= bound[..., rest]).all())


@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48])
def test_pages_behind_the_window_are_free(new, d, page):
    """A page that no token's window reaches need not be one: its entry says nothing, what it holds reaches nothing.

    33 lengths, so that windows start at every place of a block of keys; single tokens and chunks of three take the
    kernels for few rows and for many."""
    window, hq, hk = 40, 8, 1
    lens = [150 + i for i in range(33)]
    kp, vp, table = R.paged(lens, page, hk, d, torch.bfloat16, DEV, 21)
    q = _rand(new * len(lens), hq, d, dtype=torch.bfloat16, seed=22)
    want, bound = R.attend(q, kp, vp, table, [new] * len(lens), lens, R.softmax_scale(d), window)
    for b, n in enumerate(lens):
        behind = (n - new - window + 1) // page              # pages before the first token's first key
        freed = table[b, :behind].long()
        kp[freed], vp[freed] = float("nan"), float("nan")
        table[b, :behind] = _i32([(-1, kp.shape[0], -2 ** 31)[i % 3] for i in range(behind)])
    cache = kt.PagedKV(kp, vp)
    out = cache.attend(q, table, R.starts([new] * len(lens), DEV), _i32(lens), new, window=window)
    assert cache.read_error() == 0
    assert bool(((out.double().cpu() - want).abs() <= bound).all())


@pytest.mark.parametrize("q_lens,lens", [([8, 2], [3, 9]), ([60, 40], [30, 90])])
def test_the_widest_window_is_none(q_lens, lens):
    """Windows as large as an int allows, also for tokens before position 0, which see nothing."""
    d, page = 64, 16
    kp, vp, table = R.paged(lens, page, 1, d, torch.bfloat16, DEV, 41)
    q = _rand(sum(q_lens), 4, d, dtype=torch.bfloat16, seed=42)
    args = (q, table, R.starts(q_lens, DEV), _i32(lens), max(q_lens))
    cache = kt.PagedKV(kp, vp)
    want, bound = R.attend(q, kp, vp, table, q_lens, lens, R.softmax_scale(d))
    for window in (2 ** 31 - 1, 2 ** 31 - 2):
        out = cache.attend(*args, window=window)
        assert bool(((out.double().cpu() - want).abs() <= bound).all())


@pytest.mark.parametrize("new", [1, 40])
def test_numbers_beyond_an_int(new):
    """A window or a bound on new tokens that no int holds means what it says; negative ones are refused."""
    d, page, n = 64, 16, 200
    kp, vp, table = R.paged([n], page, 1, d, torch.bfloat16, DEV, 51)
    q = _rand(new, 4, d, dtype=torch.bfloat16, seed=52)
    args = (q, table, R.starts([new], DEV), _i32([n]))
    cache = kt.PagedKV(kp, vp)
    want = cache.attend(*args, new)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 63):
        assert torch.equal(cache.attend(*args, new, window=window), want)
    chunk = cache.attend(*args, 2 ** 31 - 1)
    for most in (2 ** 31, 2 ** 32 + 1, 2 ** 63):
        assert torch.equal(cache.attend(*args, most), chunk)
    for wrong in (-1, -2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(kt.KTError):
            cache.attend(*args, new, window=wrong)
        with pytest.raises(kt.KTError):
            cache.attend(*args, wrong)
