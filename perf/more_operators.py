"""Measured cases of the operators that carry a decoder layer's step in 8 bits.

Three operators of one serving step, each reached through the package's public calls:

* ``norm``: the residual's addition and the RMS norm of the hidden states, its result in 16 bits (the router's input),
  in MXFP8 (the experts' input), or both (``add_rms_norm``);
* ``append``: new keys and values to a paged cache of e4m3 numbers with one power of two for each block of 16 positions
  and head, keys normed and rotated on the way, the step's queries with them (``PagedKV8.append``);
* ``attend``: attention of every sequence's new tokens over such pages (``PagedKV8.attend``).

``run`` computes the plain form with elementary torch operations in 32 bits (``own`` false) or makes the package's
calls (``own`` true).  ``exact`` states the same outputs in 64 bits from the definitions.  What is held in 8 bits is
returned as e4m3 and e8m0 numbers, the values that the bytes stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16                                                   # positions that share a scale in the cache
LEAST, MOST = {"bf16": -117, "fp16": -14}, {"bf16": 119, "fp16": 7}   # scale exponents: code * 2^X is a number of the type


def listed():
    """The smallest calls, ordinary ones and the largest of each operator."""
    return [
        # between attention and experts in the decode step of one conversation: all latency
        {"name": "norm 1 token", "op": "norm", "dtype": "bf16", "tokens": 1, "hidden": 7168, "residual": True,
         "plain": True, "mx": True},
        # the same in the largest MoE prefill
        {"name": "norm 8192 tokens", "op": "norm", "dtype": "bf16", "tokens": 8192, "hidden": 7168, "residual": True,
         "plain": True, "mx": True},
        # a model's first norm, of a batch of no round size: no residual yet, and nobody reads 16 bits
        {"name": "norm 1001 tokens 8 bits", "op": "norm", "dtype": "fp16", "tokens": 1001, "hidden": 4096,
         "residual": False, "plain": False, "mx": True},
        # a decode step of 48 conversations: one token each, most of them into a block that has older ones
        {"name": "append 48 single tokens", "op": "append", "dtype": "bf16", "seqs": 48, "new": 1, "past": 8191,
         "hq": 64, "hk": 8, "d": 128, "rot": 128, "style": "halves", "page": 16, "norm": False},
        # a prefill step of three prompts, keys and queries normed as well
        {"name": "append 3 prompts", "op": "append", "dtype": "bf16", "seqs": 3, "new": 3500, "past": 2000,
         "hq": 64, "hk": 8, "d": 128, "rot": 128, "style": "halves", "page": 64, "norm": True},
        # odd heads, a rotation of part of the head with pairs interleaved, keys and values alone
        {"name": "append odd heads", "op": "append", "dtype": "fp16", "seqs": 7, "new": 333, "past": 1001, "hq": 0,
         "hk": 5, "d": 96, "rot": 32, "style": "interleaved", "page": 32, "norm": False},
        # the decode step of one short conversation: all latency
        {"name": "attend 1 token short", "op": "attend", "dtype": "bf16", "seqs": 1, "new": 1, "past": 700, "hq": 32,
         "hk": 8, "d": 128, "page": 16, "window": 0, "sinks": False},
        # a decode step of 64 conversations of very different lengths: all bandwidth
        {"name": "attend 64 single tokens", "op": "attend", "dtype": "bf16", "seqs": 64, "new": 1, "past": 16383,
         "hq": 64, "hk": 8, "d": 128, "page": 64, "window": 0, "sinks": False},
        # a decode step of a few very long conversations: one sequence has to spread over the GPU
        {"name": "attend 4 tokens long", "op": "attend", "dtype": "fp16", "seqs": 4, "new": 1, "past": 131071,
         "hq": 64, "hk": 8, "d": 64, "page": 128, "window": 0, "sinks": True},
        # a step in which some conversations decode and others prefill; heads and groups of no power of two
        {"name": "attend mixed batch", "op": "attend", "dtype": "bf16", "seqs": 24, "new": 500, "past": 3001,
         "hq": 40, "hk": 8, "d": 96, "page": 32, "window": 0, "sinks": False},
        # prompts of a model with sinks whose layer looks back 128 tokens
        {"name": "attend window 128", "op": "attend", "dtype": "bf16", "seqs": 4, "new": 4096, "past": 2048,
         "hq": 64, "hk": 8, "d": 64, "page": 16, "window": 128, "sinks": True},
        # a whole prompt, as large as the largest MoE prefill
        {"name": "attend prompt 8192", "op": "attend", "dtype": "bf16", "seqs": 1, "new": 8192, "past": 0,
         "hq": 64, "hk": 8, "d": 128, "page": 64, "window": 0, "sinks": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(("norm", "append", "attend", "attend"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "norm":
        mx = rng.choice((True, True, False))
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 8192), "hidden": 32 * _log(rng, 4, 224),
                "residual": rng.choice((True, True, False)), "plain": not mx or rng.choice((True, False)), "mx": mx}
    d = rng.choice((64, 80, 96, 128, 128))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        hk, seqs = rng.choice((1, 2, 4, 5, 8)), _log(rng, 1, 64)
        return {"op": op, "dtype": dtype, "seqs": seqs, "new": _log(rng, 1, 8192 // seqs), "past": _log(rng, 1, 4096),
                "hq": hk * rng.choice((0, 1, 3, 4, 8)), "hk": hk, "d": d, "rot": d if d % 32 else rng.choice((d, d // 2)),
                "style": rng.choice(("halves", "interleaved")), "page": page, "norm": rng.choice((True, False))}
    hk, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 5, 8))
    while True:
        seqs, new, past = _log(rng, 1, 64), rng.choice((1, 1, _log(rng, 2, 8192))), _log(rng, 1, 131071)
        total = new + past
        if seqs * new * total * hk * group <= 2 << 30 and seqs * total * hk * d <= 300 << 20 and seqs * new <= 16384:
            break
    return {"op": op, "dtype": dtype, "seqs": seqs, "new": new, "past": past, "hq": hk * group, "hk": hk, "d": d,
            "page": page, "window": rng.choice((0, 0, 0, _log(rng, 16, 4096))), "sinks": rng.choice((True, False))}


def _lengths(case):
    """(new tokens, tokens before them) of each sequence: the first has the most of both, the others up to that.

    In a batch of chunks every third sequence decodes a single token, and in one of more than four a sequence
    has no new token in this step."""
    r = random.Random("%(seqs)d %(new)d %(past)d" % case)
    seqs, new, past = case["seqs"], case["new"], case["past"]
    q, h = [new], [past]
    for b in range(1, seqs):
        n = 1 if new == 1 or b % 3 == 2 else r.randint(max(1, new // 4), new)
        q.append(0 if seqs > 4 and b == 4 and new > 1 else n)
        h.append(r.randint(max(min(past, 1), past // 4), past))
    return q, h


def _table(positions, rot, device):
    """cos | sin of every position, f32 [positions, rot]: the table that a model keeps."""
    inv = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv[None]
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def _exponent(top, dtype):
    """The least integer X with top <= 448 * 2^X that the type's caches hold."""
    m, e = torch.frexp(top)                                    # top = m * 2^e, m in [1/2, 1)
    x = e - torch.where(m > 0.875, 8, 9)
    return torch.where(top == 0, LEAST[dtype], x.clamp(LEAST[dtype], MOST[dtype])).to(torch.int32)


def _codes(v, x):
    """The e4m3 numbers nearest to v * 2^-x."""
    return torch.ldexp(v, -x).clamp(-448, 448).to(torch.float8_e4m3fn)


def _full_pages(pages, page, heads, d, dtype, randn):
    """(codes, scale bytes) of a cache whose every block is full, its heads of unlike sizes."""
    size = torch.exp2(torch.arange(heads, device="cuda", dtype=torch.float32) % 5 - 2)
    codes, scales = [], []
    for n in range(0, pages, 4096):                            # (a part at a time: the values are four times their codes)
        v = randn(min(4096, pages - n), page // BLOCK, BLOCK, heads, d, dtype=torch.float32)
        v *= size[:, None]
        x = _exponent(v.abs().amax(dim=(2, 4)), dtype)
        codes.append(_codes(v, x[:, :, None, :, None]).flatten(1, 2))
        scales.append((x + 127).to(torch.uint8))
    return torch.cat(codes), torch.cat(scales)


def _inputs(case, seed):
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case)
    if case["op"] == "norm":
        n, h = case["tokens"], case["hidden"]
        s["x"], s["weight"] = randn(n, h), (1 + 0.1 * randn(h)).to(dt)
        s["residual_of"] = 4 * randn(n, h) if case["residual"] else None     # grows with the layers
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    q_lens, past = _lengths(case)
    lens = [a + b for a, b in zip(q_lens, past)]
    n, page = sum(q_lens), case["page"]
    need = [-(-x // page) for x in lens]
    pages = sum(need)
    # pages of the sequences in random order; the entries that a sequence does not need say nothing
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((case["seqs"], max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    s["block_table"] = table.to(dev)
    s["cu_q"] = torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_q"] = max(q_lens)
    s["k_pages"], s["k_scales"] = _full_pages(pages, page, hk, d, case["dtype"], randn)
    s["v_pages"], s["v_scales"] = _full_pages(pages, page, hk, d, case["dtype"], randn)
    if case["op"] == "append":
        qkv = randn(n, hq + 2 * hk, d)
        s["q"] = qkv[:, :hq] if hq else None
        s["k"], s["v"] = qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["table"] = _table(max(lens), case["rot"], dev)
        s["q_weight"] = (1 + 0.1 * randn(d)).to(dt) if case["norm"] and hq else None
        s["k_weight"] = (1 + 0.1 * randn(d)).to(dt) if case["norm"] else None
    else:
        s["q"] = randn(n, hq, d)
        s["sinks_of"] = randn(hq, dtype=torch.float32) if case["sinks"] else None
    return s


def prepare(case, seed):
    """The inputs of one step, and the handle of the cache that a serving program keeps."""
    s = _inputs(case, seed)
    if own and "k_pages" in s:
        import mxfp4_weight_moe_gb300 as kt

        s["cache"] = kt.PagedKV8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], DTYPES[case["dtype"]])
    return s


def _power(scale_bytes):
    return torch.exp2(scale_bytes.float() - 127)


def _plain_norm(s):
    x = s["x"].float()
    out = {}
    if s["residual_of"] is not None:
        x = x + s["residual_of"].float()
        out["residual"] = x.to(s["x"].dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    if s["plain"]:
        out["y"] = y.to(s["x"].dtype)
    if s["mx"]:                                                # OCP: exponent floor(log2 amax) - 8, saturating
        b = y.unflatten(-1, (-1, 32))
        e = torch.frexp(b.abs().amax(-1))[1] - 1 - 8
        out["codes"] = _codes(b, e[..., None]).flatten(1)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm(x, weight, eps=1e-6):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def _rotate(x, cos_sin, style):
    """x [N, heads, d] turned by cos_sin [N, rot] (cos | sin), the first rot elements of each head."""
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    if style == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _sequence_of(s, n):
    """(sequence, position) of every new token."""
    t = torch.arange(n, device=s["cu_q"].device)
    b = torch.searchsorted(s["cu_q"], t.to(torch.int32), right=True) - 1
    return b, (s["seq_lens"][b] - s["cu_q"][b + 1] + t).long()


def _plain_write(s, pages, scales, rows, seq, pos):
    """rows (new tokens, 32 bits) into their blocks of the pages."""
    cu, page = s["cu_q"].long(), s["page"]
    seqs, heads, d = s["seqs"], rows.shape[1], rows.shape[2]
    start = s["seq_lens"].long() - (cu[1:] - cu[:-1])          # tokens before the step
    # a sequence touches at most tokens / 16 + 2 blocks; block 0 of its own is the one its tokens start in
    first = cu[:-1] // BLOCK + 2 * torch.arange(seqs, device=cu.device)
    block = first[seq] + pos // BLOCK - start[seq] // BLOCK
    top = torch.zeros(rows.shape[0] // BLOCK + 2 * seqs, heads, device=rows.device)
    top.index_reduce_(0, block, rows.abs().amax(-1), "amax")
    x = _exponent(top, s["dtype"])
    # blocks that have older tokens keep at least their exponent; those tokens are rescaled
    behind = (start - 1).clamp(min=0) // BLOCK * BLOCK         # a block that is this sequence's alone
    where = s["block_table"][torch.arange(seqs, device=cu.device), behind // page].long()
    slot = behind % page
    older = (start % BLOCK > 0) & (cu[1:] > cu[:-1])
    old = scales[where, slot // BLOCK].int() - 127
    grown = torch.where(older[:, None], torch.maximum(old, x[first]), old)
    x[first] = torch.where(older[:, None], grown, x[first])
    slots = slot[:, None] + torch.arange(BLOCK, device=cu.device)
    had = pages[where[:, None], slots]
    moved = _codes(had.float(), (grown - old)[:, None, :, None])
    keep = (torch.arange(BLOCK, device=cu.device) < (start % BLOCK)[:, None]) & older[:, None]
    pages[where[:, None], slots] = torch.where(keep[..., None, None], moved.float(), had.float()).to(pages.dtype)
    at = s["block_table"][seq, pos // page].long()
    pages[at, pos % page] = _codes(rows, x[block][..., None])
    scales[at, pos % page // BLOCK] = (x[block] + 127).to(torch.uint8)


def _plain_append(s):
    seq, pos = _sequence_of(s, s["k"].shape[0])
    cs = s["table"][pos]
    _plain_write(s, s["k_pages"], s["k_scales"], _rotate(_norm(s["k"].float(), s["k_weight"]), cs, s["style"]), seq, pos)
    _plain_write(s, s["v_pages"], s["v_scales"], s["v"].float(), seq, pos)
    if s["q"] is not None:
        return _rotate(_norm(s["q"].float(), s["q_weight"]), cs, s["style"]).to(s["q"].dtype)
    return None


def _plain_attend(s):
    """All sequences at once, padded to the longest."""
    q, hk = s["q"], s["hk"]
    n, hq, d = q.shape
    seq, pos = _sequence_of(s, n)
    row = torch.arange(n, device=q.device) - s["cu_q"][seq]
    pages = s["block_table"].clamp(min=0).long()

    def values(codes, scales):                                 # [B, keys, hk, d]
        v = codes[pages].float().unflatten(2, (-1, BLOCK)) * _power(scales[pages])[:, :, :, None, :, None]
        return v.flatten(1, 3)

    k, v = values(s["k_pages"], s["k_scales"]), values(s["v_pages"], s["v_scales"])
    seqs, keys = k.shape[:2]
    qp = torch.zeros(seqs, s["max_q"], hk, hq // hk, d, device=q.device)
    qp[seq, row] = q.float().reshape(n, hk, hq // hk, d)
    last = torch.full((seqs, s["max_q"]), -1, device=q.device, dtype=torch.long)
    last[seq, row] = pos
    qp = qp.permute(0, 2, 3, 1, 4).reshape(seqs, hk, -1, d)
    x = torch.matmul(qp, k.permute(0, 2, 3, 1)).mul_(d ** -0.5).reshape(seqs, hk, hq // hk, s["max_q"], keys)
    key = torch.arange(keys, device=q.device)
    seen = key <= last[..., None]
    if s["window"]:
        seen &= key > last[..., None] - s["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if s["sinks_of"] is not None:
        sink = s["sinks_of"].reshape(1, hk, hq // hk, 1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    if s["sinks_of"] is not None:
        total = total + torch.exp(sink - top)
    y = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).reshape(seqs, hk, hq // hk, s["max_q"], d)
    y = (y / torch.where(total == 0, torch.ones_like(total), total)).permute(0, 3, 1, 2, 4)
    return y[seq, row].reshape(n, hq, d).to(q.dtype)


def _cache_of(s, q):
    out = {"k": s["k_pages"], "v": s["v_pages"], "k_scales": s["k_scales"].view(torch.float8_e8m0fnu),
           "v_scales": s["v_scales"].view(torch.float8_e8m0fnu)}
    if q is not None:
        out["q"] = q
    return out


def run(s):
    """One call of the operator: its outputs, the whole cache among those of an append."""
    if not own:
        if s["op"] == "norm":
            return _plain_norm(s)
        return _plain_attend(s) if s["op"] == "attend" else _cache_of(s, _plain_append(s))
    if s["op"] == "norm":
        import mxfp4_weight_moe_gb300 as kt

        y, residual, mx = kt.add_rms_norm(s["x"], s["weight"], s["residual_of"], plain=s["plain"], mx=s["mx"])
        out = {}
        if residual is not None:
            out["residual"] = residual
        if y is not None:
            out["y"] = y
        if mx is not None:
            out["codes"], out["scales"] = mx[0].view(torch.float8_e4m3fn), mx[1].view(torch.float8_e8m0fnu)
        return out
    if s["op"] == "attend":
        return s["cache"].attend(s["q"], s["block_table"], s["cu_q"], s["seq_lens"], s["max_q"], window=s["window"],
                                 sinks=s["sinks_of"])
    return _cache_of(s, s["cache"].append(s["k"], s["v"], s["block_table"], s["cu_q"], s["seq_lens"], s["table"],
                                          q=s["q"], q_weight=s["q_weight"], k_weight=s["k_weight"], style=s["style"]))


def work(case):
    """Inputs read once, outputs written once; two multiply-adds per visible pair, head and element."""
    if case["op"] == "norm":
        n, h = case["tokens"], case["hidden"]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["plain"] else 0) + (1 + 1 / 32 if case["mx"] else 0)
        return {"bytes": n * h * each + 2 * h, "flops": 6 * n * h}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    q, past = _lengths(case)
    n = sum(q)
    if case["op"] == "append":
        return {"bytes": n * (4 * hq * d + 6 * hk * d + 4 * case["rot"]),
                "flops": n * (hq + 2 * hk) * d * (10 if case["norm"] else 6)}
    pairs = keys = 0
    for a, b in zip(q, past):
        w = case["window"] or a + b
        pairs += sum(min(b + t + 1, w) for t in range(a))
        keys += min(a + b, a + w - 1) if a else 0
    return {"bytes": 4 * n * hq * d + 2 * keys * hk * (d + 1 / BLOCK), "flops": 4 * pairs * hq * d}


def _nearest(v):
    """The e4m3 number nearest to each of v (64 bits), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_norm(s, case):
    x = s["x"].double()
    out = {}
    if s["residual_of"] is not None:
        x = x + s["residual_of"].double()
        out["residual"] = x
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[1] + 1e-6) * s["weight"].double()
    if case["plain"]:
        out["y"] = y
    if case["mx"]:
        blocks = y.reshape(-1, 32)
        scale = torch.exp2(torch.floor(torch.log2(blocks.abs().max(dim=1, keepdim=True).values)) - 8)
        out["codes"] = _nearest(blocks / scale).reshape(y.shape)
        out["scales"] = scale.reshape(y.shape[0], -1)
    return out


def _exact_rows(x, weight, cs, style):
    """RMS norm and rotation in 64 bits, each pair of elements as a complex number."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()
    half = cs.shape[1] // 2
    turn = torch.complex(cs[:, :half].double(), cs[:, half:].double())[:, None]
    first = torch.arange(half, device=x.device) * (2 if style == "interleaved" else 1)
    second = first + (1 if style == "interleaved" else half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_write(codes, scales, rows, table, before, page, dtype):
    """One sequence's new rows (64 bits) into its blocks; codes and scales in 64 bits."""
    end = before + rows.shape[0]
    low = before // BLOCK * BLOCK
    p = torch.arange(low, -(-end // BLOCK) * BLOCK, device=rows.device)
    at = (table[p // page], p % page)
    fresh = torch.zeros(len(p), *rows.shape[1:], dtype=torch.float64, device=rows.device)
    fresh[before - low:end - low] = rows
    top = fresh.reshape(-1, BLOCK, *rows.shape[1:]).abs().amax(dim=(1, 3))
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(LEAST[dtype], MOST[dtype]))      # [blocks, heads]
    had = scales[at[0][::BLOCK], at[1][::BLOCK] // BLOCK]
    if before > low:
        scale[0] = torch.maximum(scale[0], had[0])
        fresh[:before - low] = (codes[at] * had.repeat_interleave(BLOCK, 0)[..., None])[:before - low]
    stored = _nearest(fresh / scale.repeat_interleave(BLOCK, 0)[..., None])
    at = (at[0][:end - low], at[1][:end - low])
    codes[at] = stored[:end - low]
    scales[at[0][::BLOCK], at[1][::BLOCK] // BLOCK] = scale


def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits, sequence by sequence."""
    s = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    q_lens, past = _lengths(case)
    page, hk, d = case["page"], case["hk"], case["d"]
    if case["op"] == "append":
        out = {n: s[n + "_pages"].double() for n in ("k", "v")}
        out |= {n: s[n].view(torch.float8_e8m0fnu).double() for n in ("k_scales", "v_scales")}
        qs, at = [], 0
        for b, (a, h) in enumerate(zip(q_lens, past)):
            if a == 0:
                continue
            new = slice(at, at + a)
            at += a
            cs = s["table"][h:h + a]
            table = s["block_table"][b].long()
            _exact_write(out["k"], out["k_scales"], _exact_rows(s["k"][new], s["k_weight"], cs, case["style"]), table, h,
                         page, case["dtype"])
            _exact_write(out["v"], out["v_scales"], s["v"][new].double(), table, h, page, case["dtype"])
            if s["q"] is not None:
                qs.append(_exact_rows(s["q"][new], s["q_weight"], cs, case["style"]))
        if s["q"] is not None:
            out["q"] = torch.cat(qs)
        return out
    group = case["hq"] // hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (a, h) in enumerate(zip(q_lens, past)):
        used = s["block_table"][b, :-(-(a + h) // page)].long()
        for c in range(hk):
            kc, vc = (torch.ldexp(s[n + "_pages"][used, :, c].double().reshape(-1, BLOCK, d),
                                  s[n + "_scales"][used, :, c].reshape(-1, 1, 1).int() - 127).reshape(-1, d)[:a + h]
                      for n in ("k", "v"))
            for head in range(c * group, (c + 1) * group) if a else ():
                z = s["q"][at:at + a, head].double() @ kc.T / math.sqrt(d)
                hidden = torch.ones_like(z, dtype=torch.bool).triu(h + 1)
                if case["window"]:
                    hidden |= torch.ones_like(z, dtype=torch.bool).tril(h - case["window"])
                z[hidden] = -math.inf
                if s["sinks_of"] is not None:
                    z = torch.cat((z, s["sinks_of"][head].double().expand(a, 1)), dim=1)
                y[at:at + a, head] = torch.softmax(z, dim=-1)[:, :a + h] @ vc
        at += a
    return y
