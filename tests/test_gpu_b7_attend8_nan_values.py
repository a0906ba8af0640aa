"""Values that are not finite in an 8-bit cache, in calls of up to 32 query rows a cache head: tokens that see none of
their block's keys are as without them."""
import pytest
import torch

import attn_oracle as R
import mx8_oracle as M
import mxfp4_weight_moe_gb300 as kt

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hq", [(64, 2), (128, 2), (96, 1), (64, 4)])
@pytest.mark.parametrize("new,n,first,last,window", [
    (8, 100, 96, 99, 0),      # the sequence's end: the step's last four tokens see them
    (3, 98, 96, 97, 0),       # the last two
    (8, 100, 80, 95, 3),      # a window that has passed them for the last two tokens
    (4, 100, 16, 31, 40),     # behind every token's window
])
def test_a_block_that_some_tokens_see(dtype, d, hq, new, n, first, last, window):
    page = 32
    kp, vp, ks, vs, table, k, v = M.paged8([n], page, 1, d, dtype, DEV, 1)
    at = int(table[0, first // page])
    vs[at, first % page // M.BLOCK] = 255
    vp[at, first % page:last % page + 1, 0, ::3] = 0x7f          # NaN codes in it as well
    q = torch.randn(new, hq, d, generator=torch.Generator().manual_seed(2)).mul(0.5).to(dtype).to(DEV)
    pos = torch.arange(n - new, n)
    sees = (pos >= first) & ((pos - window < last) if window else True)
    assert bool(sees.any()) == (first != 16) and not bool(sees.all())
    out = kt.PagedKV8(kp, vp, ks, vs, dtype).attend(q, table, R.starts([new], DEV), _i32([n]), new, window=window)
    want, bound = R.attend(q, k, v, table, [new], [n], R.softmax_scale(d), window)
    assert bool(((out.double().cpu() - want).abs() <= bound)[~sees].all())
    assert bool(out[sees.to(DEV)].isnan().all())


def test_as_appended():
    """The third of eight new tokens has a value that is not finite, in one of two heads."""
    d, hk, page, past, new, dt = 64, 2, 16, 94, 8, torch.bfloat16
    lens = [past + new]
    kp, vp, ks, vs, table, _, _ = M.paged8(lens, page, hk, d, dt, DEV, 3)
    cache = kt.PagedKV8(kp, vp, ks, vs, dt)
    g = torch.Generator().manual_seed(4)
    k, v, q = (torch.randn(new, heads, d, generator=g).mul(0.5).to(dt).to(DEV) for heads in (hk, hk, 2 * hk))
    v[2, 1, 7] = float("inf")                                    # position 96: the first of a block
    step = table, R.starts([new], DEV), _i32(lens)
    cache.append(k, v, *step)
    out = cache.attend(q, *step, new)
    kn, vn = ((M.numbers(c.cpu()) * M.power(s.cpu()).repeat_interleave(M.BLOCK, 1)[..., None])
              for c, s in ((kp, ks), (vp, vs)))
    want, bound = R.attend(q, kn.to(dt), vn.to(dt).nan_to_num(0.0), table, [new], lens, R.softmax_scale(d))
    ok = torch.ones(new, 2 * hk, dtype=torch.bool)
    ok[2:, 2:] = False                                           # tokens from position 96 on, heads of cache head 1
    assert bool(((out.double().cpu() - want).abs() <= bound)[ok].all())
    assert bool(out[~ok.to(DEV)].isnan().all()) and cache.read_error() == 0
