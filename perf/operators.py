"""Measured cases of the attention operators that stand in front of the MoE layer.

Three operators of one decoder layer's serving path, each reached through the package's public calls:

* ``norm_rope``: RMS norm of each query and key head and the rotation by position, in one pass
  (``qk_norm_rope``);
* ``append``: new keys and values written to a paged cache, keys normed and rotated on the way, the step's
  queries with them (``PagedKV.append``);
* ``attend``: attention of every sequence's new tokens over its pages (``PagedKV.attend``).

``run`` computes the plain form with elementary torch operations in 32 bits (``own`` false) or makes the
package's calls (``own`` true).  ``exact`` states the same outputs in 64 bits from the definitions.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    """The smallest calls, ordinary ones and the largest of each operator."""
    return [
        # the decode step of one conversation: all latency
        {"name": "norm_rope 1 token", "op": "norm_rope", "dtype": "bf16", "tokens": 1, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "style": "halves", "positions": 8192},
        # a prefill step as large as the largest MoE prefill, heads sliced out of one packed projection
        {"name": "norm_rope 8192 tokens", "op": "norm_rope", "dtype": "bf16", "tokens": 8192, "hq": 64, "hk": 8,
         "d": 128, "rot": 128, "style": "halves", "positions": 32768},
        # a decode step of 32 conversations: one token each, queries rotated by the same call
        {"name": "append 32 single tokens", "op": "append", "dtype": "bf16", "seqs": 32, "new": 1, "past": 8191,
         "hq": 64, "hk": 8, "d": 128, "rot": 128, "style": "halves", "page": 16, "norm": False},
        # a prefill step of three prompts, keys and queries normed as well
        {"name": "append 3 prompts", "op": "append", "dtype": "bf16", "seqs": 3, "new": 3500, "past": 2000,
         "hq": 64, "hk": 8, "d": 128, "rot": 128, "style": "halves", "page": 64, "norm": True},
        # a model with odd heads and a rotation of part of the head, pairs interleaved, keys and values alone
        {"name": "append odd heads", "op": "append", "dtype": "fp16", "seqs": 7, "new": 333, "past": 1001, "hq": 0,
         "hk": 5, "d": 96, "rot": 32, "style": "interleaved", "page": 32, "norm": False},
        # the decode step of one short conversation: all latency
        {"name": "attend 1 token short", "op": "attend", "dtype": "bf16", "seqs": 1, "new": 1, "past": 500, "hq": 32,
         "hk": 8, "d": 128, "page": 16, "window": 0, "sinks": False},
        # a decode step of 64 conversations of very different lengths: all bandwidth
        {"name": "attend 64 single tokens", "op": "attend", "dtype": "bf16", "seqs": 64, "new": 1, "past": 8191,
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
        # a chunk of a long prompt
        {"name": "attend chunk 2048 long", "op": "attend", "dtype": "fp16", "seqs": 1, "new": 2048, "past": 30001,
         "hq": 32, "hk": 8, "d": 128, "page": 16, "window": 0, "sinks": False},
        # a whole prompt, as large as the largest MoE prefill
        {"name": "attend prompt 8192", "op": "attend", "dtype": "bf16", "seqs": 1, "new": 8192, "past": 0,
         "hq": 64, "hk": 8, "d": 128, "page": 64, "window": 0, "sinks": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(("norm_rope", "append", "attend", "attend"))
    dtype = rng.choice(("bf16", "fp16"))
    d = rng.choice((64, 80, 96, 128, 128))
    rot = rng.choice((d, d, d // 2))
    style = rng.choice(("halves", "interleaved"))
    if op == "norm_rope":
        hk = rng.choice((1, 2, 4, 5, 8))
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 8192), "hq": hk * rng.choice((1, 3, 4, 8)), "hk": hk,
                "d": d, "rot": rot, "style": style, "positions": _log(rng, 64, 32768)}
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        hk, seqs = rng.choice((1, 2, 4, 5, 8)), _log(rng, 1, 64)
        return {"op": op, "dtype": dtype, "seqs": seqs, "new": _log(rng, 1, 8192 // seqs), "past": _log(rng, 1, 4096),
                "hq": hk * rng.choice((0, 1, 3, 4, 8)), "hk": hk, "d": d, "rot": rot, "style": style, "page": page,
                "norm": rng.choice((True, False))}
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
        h.append(r.randint(past // 4, past))
    return q, h


def _table(positions, rot, device):
    """cos | sin of every position, f32 [positions, rot]: the table that a model keeps."""
    inv = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv[None]
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def _inputs(case, seed):
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "norm_rope":
        n = case["tokens"]
        qkv = randn(n, hq + 2 * hk, d)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]          # slices of the packed projection
        s["positions_of"] = torch.randint(0, case["positions"], (n,), generator=g, device=dev, dtype=torch.int32)
        s["table"] = _table(case["positions"], case["rot"], dev)
        s["q_weight"], s["k_weight"] = (1 + 0.1 * randn(d)).to(dt), (1 + 0.1 * randn(d)).to(dt)
        return s
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
    s["k_pages"], s["v_pages"] = randn(pages, page, hk, d), randn(pages, page, hk, d)
    if case["op"] == "append":
        qkv = randn(n, hq + 2 * hk, d)
        s["q"] = qkv[:, :hq] if hq else None
        s["k"], s["v"] = qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["table"] = _table(max(lens), case["rot"], dev)
        s["q_weight"] = (1 + 0.1 * randn(d)).to(dt) if case["norm"] and hq else None
        s["k_weight"] = (1 + 0.1 * randn(d)).to(dt) if case["norm"] else None
    else:
        s["q"] = 2 * randn(n, hq, d)                                # logits of standard deviation two
        s["sinks_of"] = randn(hq, dtype=torch.float32) if case["sinks"] else None
    return s


def prepare(case, seed):
    """The inputs of one step, and the handle of the cache that a serving program keeps."""
    s = _inputs(case, seed)
    if own and "k_pages" in s:
        import mxfp4_weight_moe_gb300 as kt

        s["cache"] = kt.PagedKV(s["k_pages"], s["v_pages"])
    return s


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


def _sequence_of(s):
    """(sequence, position) of every new token."""
    n = s["k"].shape[0] if s["op"] == "append" else s["q"].shape[0]
    t = torch.arange(n, device=s["cu_q"].device)
    b = torch.searchsorted(s["cu_q"], t.to(torch.int32), right=True) - 1
    return b, s["seq_lens"][b] - s["cu_q"][b + 1] + t


def _plain_attend(s):
    """All sequences at once, padded to the longest."""
    q, page, hk = s["q"], s["page"], s["hk"]
    n, hq, d = q.shape
    seq, pos = _sequence_of(s)
    pos = pos.long()
    row = torch.arange(n, device=q.device) - s["cu_q"][seq]
    pages = s["block_table"].clamp(min=0).long()
    k = s["k_pages"][pages].flatten(1, 2).float()                   # [B, keys, hk, d]
    v = s["v_pages"][pages].flatten(1, 2).float()
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


def _plain(s):
    if s["op"] == "norm_rope":
        cs = s["table"][s["positions_of"].long()]
        return {n: _rotate(_norm(s[n].float(), s[n + "_weight"]), cs, s["style"]).to(s[n].dtype) for n in ("q", "k")}
    if s["op"] == "attend":
        return _plain_attend(s)
    seq, pos = _sequence_of(s)
    pos = pos.long()
    page = s["block_table"][seq, pos // s["page"]].long()
    cs = s["table"][pos]
    s["k_pages"][page, pos % s["page"]] = _rotate(_norm(s["k"].float(), s["k_weight"]), cs, s["style"]).to(s["k"].dtype)
    s["v_pages"][page, pos % s["page"]] = s["v"]
    out = {"k": s["k_pages"], "v": s["v_pages"]}
    if s["q"] is not None:
        out["q"] = _rotate(_norm(s["q"].float(), s["q_weight"]), cs, s["style"]).to(s["q"].dtype)
    return out


def run(s):
    """One call of the operator: its outputs, the cache's pages among those of an append."""
    if not own:
        return _plain(s)
    import mxfp4_weight_moe_gb300 as kt

    if s["op"] == "norm_rope":
        q, k = kt.qk_norm_rope(s["q"], s["k"], s["positions_of"], s["table"], s["q_weight"], s["k_weight"],
                               style=s["style"])
        return {"q": q, "k": k}
    if s["op"] == "attend":
        return s["cache"].attend(s["q"], s["block_table"], s["cu_q"], s["seq_lens"], s["max_q"], window=s["window"],
                                 sinks=s["sinks_of"])
    q = s["cache"].append(s["k"], s["v"], s["block_table"], s["cu_q"], s["seq_lens"], s["table"], q=s["q"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], style=s["style"])
    out = {"k": s["k_pages"], "v": s["v_pages"]}
    if q is not None:
        out["q"] = q
    return out


def work(case):
    """Inputs read once, outputs written once; two multiply-adds per visible pair, head and element."""
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "norm_rope":
        n = case["tokens"]
        return {"bytes": n * (4 * (hq + hk) * d + 4 * case["rot"] + 4), "flops": n * (hq + hk) * d * 8}
    q, past = _lengths(case)
    n = sum(q)
    if case["op"] == "append":
        heads = hq + 2 * hk
        return {"bytes": n * (4 * heads * d + 4 * case["rot"]), "flops": n * (hq + hk) * d * (8 if case["norm"] else 4)}
    pairs = keys = 0
    for a, b in zip(q, past):
        w = case["window"] or a + b
        pairs += sum(min(b + t + 1, w) for t in range(a))
        keys += min(a + b, a + w - 1) if a else 0
    return {"bytes": 4 * n * hq * d + 4 * keys * hk * d, "flops": 4 * pairs * hq * d}


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


def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits, sequence by sequence."""
    s = _inputs(case, seed)
    if case["op"] == "norm_rope":
        cs = s["table"][s["positions_of"].long()]
        return {n: _exact_rows(s[n], s[n + "_weight"], cs, case["style"]) for n in ("q", "k")}
    q_lens, past = _lengths(case)
    page, hk, d = case["page"], case["hk"], case["d"]
    if case["op"] == "append":
        out = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
        qs, at = [], 0
        for b, (a, h) in enumerate(zip(q_lens, past)):
            if a == 0:
                continue
            new = slice(at, at + a)
            at += a
            p = torch.arange(h, h + a, device=s["k"].device)
            where = s["block_table"][b].long()[p // page], p % page
            out["k"][where] = _exact_rows(s["k"][new], s["k_weight"], s["table"][p], case["style"])
            out["v"][where] = s["v"][new].double()
            if s["q"] is not None:
                qs.append(_exact_rows(s["q"][new], s["q_weight"], s["table"][p], case["style"]))
        if s["q"] is not None:
            out["q"] = torch.cat(qs)
        return out
    group = case["hq"] // hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (a, h) in enumerate(zip(q_lens, past)):
        used = s["block_table"][b, :-(-(a + h) // page)].long()
        for c in range(hk):
            kc = s["k_pages"][used, :, c].reshape(-1, d)[:a + h].double()
            vc = s["v_pages"][used, :, c].reshape(-1, d)[:a + h].double()
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
