"""64-bit statements of what the 8-bit operators store: MXFP8 rows, and e4m3 blocks of a key/value cache."""
import torch

import attn_oracle as R

BLOCK = 16
# Scale exponents of a cache: code * 2^X is a number of the type, and fp32 sums of 2^24 of them, 2^8 times, are finite.
LEAST, MOST = {torch.bfloat16: -117, torch.float16: -14}, {torch.bfloat16: 87, torch.float16: 7}


def e4m3(v):
    """The e4m3 number nearest to each of v (64 bits), ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def half_step(v):
    """Half the distance of e4m3 numbers around |v| (of the coarser side at a power of two)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6, max=448.0))) - 4)


def numbers(codes):
    return codes.view(torch.float8_e4m3fn).double()


def power(scales):
    return torch.exp2(scales.double() - 127)


def off_by_a_rounding(codes, scale, v, off):
    """How far |code * scale - v| is over what one rounding allows of a value that is off by at most `off`.

    A rounding to nearest is off by half a step of the numbers around (v + off) / scale; values beyond 448 saturate."""
    got = codes * scale
    edge = 448 * scale
    inside = torch.minimum(v.abs() + off, edge.expand_as(v))
    allowed = half_step(inside / scale) * scale + off + (v.abs() - edge).clamp(min=0)
    return (got - v).abs() - allowed


def rms_rows(x, residual, weight, eps):
    """(s, y) in 64 bits and the fp32 error of y before its rounding.

    fp32 steps: the residual's addition (1 rounding), a thread's at most 32 squares and sums, 5 shuffles and at most 32
    warps (their error halved by the root), the root (2 units) and three products: fewer than 64 roundings of y."""
    s = x.double().cpu()
    if residual is not None:
        s = s + residual.double().cpu()
    y = s / torch.sqrt(s.pow(2).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    return s, y, 64 * R.F32 * y.abs()


def floor_exponent(top):
    """OCP's shared exponent: floor(log2 top) - 8 (top > 0)."""
    return torch.floor(torch.log2(top)) - 8


def least_exponent(top, dtype):
    """The least X with top <= 448 * 2^X that a cache of dtype holds (top = 0: the lowest)."""
    x = torch.ceil(torch.log2(top / 448)).clamp(LEAST[dtype], MOST[dtype])
    # log2 may be off by a rounding next to a power of two
    x = torch.where(448 * torch.exp2(x - 1) >= top, x - 1, x)
    x = torch.where(448 * torch.exp2(x) < top, x + 1, x)
    return x.clamp(LEAST[dtype], MOST[dtype])


def paged8(seq_lens, page, hk, d, dtype, device, seed, layout="slots", spare=3, sizes=True, rows=None):
    """A cache of 8 bits: (k_pages, v_pages, k_scales, v_scales, block_table, k, v) with shuffled pages.

    Wherever no sequence has a key the codes and the scales are any bytes, NaN among them.  k, v: the numbers that the
    codes stand for, of dtype (which holds them exactly).  sizes: blocks and heads of unlike magnitude.  rows(b): the
    keys and values of sequence b (both [len, hk, d], 64 bits); default: random ones."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in seq_lens]
    pages, blocks = sum(need) + spare, page // BLOCK
    order = torch.randperm(pages, generator=g)

    def empty(last, what):
        if layout == "slots":
            return torch.zeros(pages, page, hk, last, dtype=what)
        if layout == "heads":
            return torch.zeros(pages, hk, page, last, dtype=what).transpose(1, 2)
        return torch.zeros(pages, 2, page, hk, last, dtype=what)[:, 0]

    out = []
    codes = [empty(d, torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 256, (pages, blocks, hk), generator=g, dtype=torch.int32).to(torch.uint8)
              for _ in range(2)]
    for s in scales:
        s[torch.rand(s.shape, generator=g) < 0.3] = 255
    numbers_of = [torch.zeros(pages, page, hk, d, dtype=torch.float64) for _ in range(2)]
    for t in codes:
        t.copy_(torch.randint(0, 256, (pages, page, hk, d), generator=g, dtype=torch.int32).to(torch.uint8))
        t[torch.rand(t.shape, generator=g) < 0.2] = 0x7f
    table = torch.full((len(seq_lens), max(need + [1]) + 1), -7, dtype=torch.int32)
    table[:, -1] = 2 ** 31 - 1
    at = 0
    for b, (m, n) in enumerate(zip(need, seq_lens)):
        table[b, :m] = order[at:at + m].to(torch.int32)
        at += m
        if n <= 0:
            continue
        whole = -(-n // BLOCK) * BLOCK
        given = rows(b) if rows is not None else None
        p = torch.arange(whole)
        where = table[b].long()[p // page], p % page
        for side in range(2):
            v = torch.zeros(whole, hk, d, dtype=torch.float64)
            if given is None:
                v[:n] = torch.randn(n, hk, d, generator=g, dtype=torch.float64)
                if sizes:
                    v *= torch.exp2(torch.randint(-3, 3, (whole // BLOCK, hk), generator=g).double()) \
                        .repeat_interleave(BLOCK, 0)[..., None]
            else:
                v[:n] = given[side]
            x = least_exponent(v.unflatten(0, (-1, BLOCK)).abs().amax(dim=(1, 3)), dtype)
            power_of = torch.exp2(x).repeat_interleave(BLOCK, 0)[..., None]
            c = e4m3(v / power_of)
            filled = tuple(i[:n] for i in where)
            codes[side][filled] = c[:n].to(torch.float8_e4m3fn).view(torch.uint8)
            numbers_of[side][filled] = (c * power_of)[:n]
            scales[side][where[0][::BLOCK], where[1][::BLOCK] // BLOCK] = (x + 127).to(torch.uint8)
    for t in codes:
        if layout == "pairs":
            wide = torch.zeros(pages, 2, page, hk, d, dtype=torch.uint8, device=device)
            wide[:, 0] = t.to(device)
            out.append(wide[:, 0])
        elif layout == "heads":
            out.append(t.transpose(1, 2).contiguous().to(device).transpose(1, 2))
        else:
            out.append(t.to(device))
    numbers_of = [t.to(dtype) for t in numbers_of]
    return (*out, *(s.to(device) for s in scales), table.to(device), *numbers_of)
