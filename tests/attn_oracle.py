"""64-bit CPU statements of the attention operators, and error bounds that follow from the element types."""
import math

import torch

# Unit roundoff of the element types: half a unit in the last place, relative.
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# Absolute rounding step of the smallest numbers (fp16 has subnormals within reach of softmax weights).
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
F32 = 2.0 ** -24


def head_rows(x, weight, eps, table, positions, style):
    """(norm + rotation in 64 bits, bound on the kernel's error before its one rounding to x's type).

    fp32 steps: the sum of squares over D elements, rsqrt (2 units), two products, then two products and a sum for
    the rotation: fewer than D/2 + 16 roundings of values no larger than |a| + |b| of the pair."""
    dt, d = x.dtype, x.shape[-1]
    y = x.double().cpu()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    size = y.abs()
    if table is not None:
        cs = table.double().cpu()[positions.long().cpu()]
        rot = cs.shape[1]
        i = torch.arange(rot // 2)
        a, b = (i, i + rot // 2) if style == "halves" else (2 * i, 2 * i + 1)
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        z = y.clone()
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        size = size.clone()
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
        y = z
    pre = (d / 2 + 16) * F32 * size if weight is not None else 16 * F32 * size
    return y, ROUND[dt] * (y.abs() + pre) + pre + 2.0 ** -25 * (dt == torch.float16)


def attend(q, k_pages, v_pages, block_table, q_lens, seq_lens, scale, window=0, sinks=None):
    """(output in 64 bits, bound on the kernel's error), token by token over the keys that it sees.

    The bound: the result's rounding to its type, each softmax weight's rounding to it (relative, and absolute where
    fp16 weights underflow), and fp32 arithmetic: a logit x is off by at most (D + 4) roundings of sum |q k| scale and
    of |x|, which moves each weight by that much relative; sums of n weights and products add 2 n roundings at most,
    the running maximum's rescaling one per tile."""
    dt = q.dtype
    n, hq, d = q.shape
    hk = k_pages.shape[2]
    group = hq // hk
    q64, k64, v64 = q.double().cpu(), k_pages.double().cpu(), v_pages.double().cpu()
    table = block_table.cpu()
    page = k_pages.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    bound = torch.zeros(n, hq, d, dtype=torch.float64)
    at = 0
    for b, ql in enumerate(q_lens):
        length = seq_lens[b]
        need = -(-max(length, 0) // page)
        used = table[b, :need].long()
        kk = k64[used].reshape(-1, hk, d)[:max(length, 0)]
        vv = v64[used].reshape(-1, hk, d)[:max(length, 0)]
        for t in range(ql):
            pos = length - ql + t
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                at += 1
                continue
            for h in range(hq):
                c = h // group
                ks, vs = kk[lo:pos + 1, c], vv[lo:pos + 1, c]
                x = scale * (ks @ q64[at, h])
                size = scale * (ks.abs() @ q64[at, h].abs())
                top = x.max() if sinks is None else max(x.max(), sinks[h].double().cpu())
                p = torch.exp(x - top)
                total = p.sum() + (0.0 if sinks is None else torch.exp(sinks[h].double().cpu() - top))
                p = p / total
                out[at, h] = p @ vs
                off = (d + 4) * F32 * (size.max() + x.abs().max() + top.abs()) + (2 * len(p) + 64) * F32
                weights = p @ vs.abs()
                bound[at, h] = (ROUND[dt] * (out[at, h].abs() + weights) + 2 * off * weights
                                + TINY[dt] / total * vs.abs().sum(0)) * 1.01 + TINY[dt]
            at += 1
    return out, bound


def paged(seq_lens, page, hk, d, dtype, device, seed, layout="slots", spare=3, fill=float("nan")):
    """(k_pages, v_pages, block_table): random keys and values in shuffled pages of a cache that is `fill` wherever no
    sequence has a key; table entries past a sequence's pages are no pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in seq_lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    if layout == "slots":                                  # [pages, slots, heads, d]
        k, v = (torch.full((pages, page, hk, d), fill, dtype=dtype) for _ in range(2))
        k, v = k.to(device), v.to(device)
    elif layout == "heads":                                # [pages, heads, slots, d] in memory
        k, v = (torch.full((pages, hk, page, d), fill, dtype=dtype).to(device).transpose(1, 2) for _ in range(2))
    else:                                                  # keys and values of a page side by side
        kv = torch.full((pages, 2, page, hk, d), fill, dtype=dtype).to(device)
        k, v = kv[:, 0], kv[:, 1]
    width = max(need + [1]) + 1
    table = torch.full((len(seq_lens), width), -7, dtype=torch.int32)
    table[:, -1] = 2 ** 31 - 1
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m].to(torch.int32)
        at += m
        for i in range(m):
            fillable = min(page, seq_lens[b] - i * page)
            for t in (k, v):
                t[int(table[b, i]), :fillable] = torch.randn(fillable, hk, d, generator=g).to(dtype).to(device)
    return k, v, table.to(device)


def starts(q_lens, device):
    c = [0]
    for x in q_lens:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device=device)


def softmax_scale(d):
    return 1.0 / math.sqrt(d)
