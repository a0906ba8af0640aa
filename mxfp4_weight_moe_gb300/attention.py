"""Attention operators in front of the MoE layer (C ABI: ``include/kt_attn.h``).

``qk_norm_rope`` norms and rotates query and key heads; ``PagedKV`` is a cache
in pages, whose ``append`` writes a step's keys (normed and rotated on the way)
and values and whose ``attend`` computes the attention of the step's tokens
over it.  As everywhere in the package, the arithmetic runs in the library's
CUDA kernels: this module checks tensors, allocates outputs and passes pointers
and the CUDA stream.

A step's batch is three int32 tensors: ``block_table`` [B, max_pages] (the pages
of each sequence in order), ``cu_q`` [B + 1] (sequence b has the step's tokens
cu_q[b] .. cu_q[b+1]) and ``seq_lens`` [B] (its keys in all, the step's own
included, so that its last new token has position seq_lens[b] - 1).
"""
from __future__ import annotations

import ctypes

import torch

import mxfp4_weight_moe_gb300 as kt

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}   # KT_DTYPE_*
KT_DTYPE_F32 = 2
ROPE_STYLES = {"halves": 0, "interleaved": 1}

KT_DEVERR_BAD_PAGE = 0x20
KT_DEVERR_BAD_POSITION = 0x40

_VP, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class Heads(ctypes.Structure):
    _fields_ = [("ptr", _VP), ("token_stride", _I64), ("head_stride", _I64), ("heads", _I)]


class PagedKVDesc(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP),
                ("k_page_stride", _I64), ("k_slot_stride", _I64), ("k_head_stride", _I64),
                ("v_page_stride", _I64), ("v_slot_stride", _I64), ("v_head_stride", _I64),
                ("num_pages", _I), ("page_size", _I), ("heads", _I), ("head_dim", _I), ("dtype", _I)]


class PagedBatch(ctypes.Structure):
    _fields_ = [("block_table", _VP), ("table_stride", _I64), ("max_pages", _I), ("cu_q", _VP), ("seq_lens", _VP),
                ("seqs", _I), ("tokens", _I)]


class HeadTransform(ctypes.Structure):
    _fields_ = [("table", _VP), ("positions", _I), ("rotary_dim", _I), ("style", _I), ("q_weight", _VP),
                ("k_weight", _VP), ("weight_dtype", _I), ("eps", _F)]


_P = ctypes.POINTER
SIGNATURES = {
    "kt_qk_norm_rope": ([_P(Heads), _P(Heads), _P(Heads), _P(Heads), _VP, _I, _I, _I, _P(HeadTransform), _VP, _VP], _I),
    "kt_kv_append": ([_P(PagedKVDesc), _P(PagedBatch), _P(Heads), _P(Heads), _P(Heads), _P(Heads), _P(HeadTransform),
                      _VP, _VP], _I),
    "kt_paged_attention_workspace_bytes": ([], ctypes.c_size_t),
    "kt_paged_attention": ([_P(PagedKVDesc), _P(PagedBatch), _P(Heads), _P(Heads), _I, _F, _I, _VP, _VP, _VP,
                            ctypes.c_size_t, _VP], _I),
}


def _heads(t, name: str, dtype, dim: int, device, tokens: int | None = None, heads: int | None = None) -> Heads:
    """Descriptor of a [tokens, heads, dim] tensor with contiguous heads."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (tokens is not None and shape[0] != tokens) or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {dim}], got {tuple(shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected {device if device.type == 'cuda' else 'a CUDA device'}")
    st = t.stride()
    if st[2] != 1 and dim != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous, strides are {st}")
    # the stride of a dimension of one entry says nothing
    return Heads(t.data_ptr(), st[0] if shape[0] > 1 else dim, st[1] if shape[1] > 1 else dim, shape[1])


def _written(t, name: str):
    """An output whose elements overlap would be written by several threads at once."""
    shape, st = t.shape, t.stride()
    if t.numel() and ((shape[1] > 1 and st[1] < shape[2]) or (shape[0] > 1 and st[0] < shape[2])
                      or (shape[0] > 1 and shape[1] > 1
                          and st[0] < (shape[1] - 1) * st[1] + shape[2] and st[1] < (shape[0] - 1) * st[0] + shape[2])):
        raise ValueError(f"{name}: its rows overlap, strides are {st}")


def _ints(t, name: str, ndim: int, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != ndim or t.device != device:
        raise ValueError(f"{name} must have {ndim} dims on {device}, got {tuple(t.shape)} on {t.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous")


def _batch(block_table, cu_q, seq_lens, tokens: int, device) -> PagedBatch:
    _ints(block_table, "block_table", 2, device)
    _ints(cu_q, "cu_q", 1, device)
    _ints(seq_lens, "seq_lens", 1, device)
    seqs, max_pages = block_table.shape
    if seq_lens.shape[0] != seqs or cu_q.shape[0] != seqs + 1:
        raise ValueError(f"block_table {tuple(block_table.shape)}, cu_q {tuple(cu_q.shape)} and seq_lens "
                         f"{tuple(seq_lens.shape)} must be [B, max_pages], [B + 1] and [B]")
    return PagedBatch(block_table.data_ptr(), block_table.stride(0) if seqs > 1 else max_pages, max_pages,
                      cu_q.data_ptr(), seq_lens.data_ptr(), seqs, tokens)


def _transform(table, q_weight, k_weight, eps: float, style: str, dtype, dim: int, device) -> HeadTransform:
    t = HeadTransform()
    t.eps = eps
    if table is not None:
        if table.dtype is not torch.float32:
            raise TypeError(f"table must be torch.float32, got {table.dtype}")
        if table.dim() != 2 or table.device != device or not table.is_contiguous():
            raise ValueError(f"table must be contiguous [positions, rotary_dim] on {device}")
        if style not in ROPE_STYLES:
            raise ValueError(f"style must be one of {tuple(ROPE_STYLES)}")
        t.table = table.data_ptr()
        t.positions, t.rotary_dim = table.shape
        t.style = ROPE_STYLES[style]
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if w.dtype is not dtype and w.dtype is not torch.float32:
            raise TypeError(f"{name} must be {dtype} or torch.float32, got {w.dtype}")
        if w.shape != (dim,) or w.device != device or not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous [{dim}] on {device}")
        setattr(t, name, w.data_ptr())
        t.weight_dtype = DTYPE_CODES.get(w.dtype, KT_DTYPE_F32)
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    return t


class _allocating_on:
    """Tensors made inside belong to `stream` (None: the current one), whose pointer is `.ptr`."""
    __slots__ = ("ctx", "ptr")

    def __init__(self, stream, device):
        self.ctx = None if stream is None else torch.cuda.stream(stream)
        self.ptr = kt._stream_ptr(stream, device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def rope_table(positions: int, rotary_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos | sin of every position: f32 [positions, rotary_dim], angles p * theta^(-2i / rotary_dim)."""
    if positions <= 0 or rotary_dim <= 0 or rotary_dim % 8:
        raise ValueError("positions must be positive and rotary_dim a positive multiple of 8")
    inv = float(theta) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv[None, :]
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 table: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, style: str = "halves",
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 error: torch.Tensor | None = None, stream=None):
    """RMS norm of each head (where its weight is given) and rotation by position (where a table is given) of
    q [tokens, q heads, head_dim] and k [tokens, k heads, head_dim] (or None) in one launch; returns (q_out, k_out).

    bf16 or fp16; heads may be slices of a packed projection, outputs may be the inputs.  positions: int32 [tokens];
    table: rope_table's; style "halves" (pairs i, i + rotary_dim/2) or "interleaved" (2i, 2i+1).  error: an int32
    [1] tensor that gets KT_DEVERR_BAD_POSITION for a position outside the table (that token is not written)."""
    if not isinstance(q, torch.Tensor) or q.dtype not in DTYPE_CODES or q.dim() != 3:
        raise TypeError("q must be a bf16 or fp16 tensor [tokens, heads, head_dim]")
    dev, dt = q.device, q.dtype
    n, _, dim = q.shape
    hq = _heads(q, "q", dt, dim, dev)
    hk = None if k is None else _heads(k, "k", dt, dim, dev, n)
    if table is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        _ints(positions, "positions", 1, dev)
        if positions.shape[0] != n:
            raise ValueError(f"positions must be [{n}]")
    tf = _transform(table, q_weight, k_weight, eps, style, dt, dim, dev)
    if error is not None:
        _ints(error, "error", 1, dev)
    with _allocating_on(stream, dev) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dt, device=dev)
        else:
            _written(q_out, "q_out")
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=dt, device=dev)
        elif k_out is not None:
            _written(k_out, "k_out")
    hqo = _heads(q_out, "q_out", dt, dim, dev, n, q.shape[1])
    hko = None if k is None else _heads(k_out, "k_out", dt, dim, dev, n, k.shape[1])
    with kt._on_device(dev):
        kt._check(kt.lib().kt_qk_norm_rope(hq, hk, hqo, hko, kt._ptr(positions) if table is not None else None, n, dim,
                                           DTYPE_CODES[dt], tf, kt._ptr(error), s.ptr), "kt_qk_norm_rope")
    return q_out, (k_out if k is not None else None)


class PagedKV:
    """A key/value cache in pages: k_pages and v_pages are [num_pages, page_size, heads, head_dim] (bf16 or fp16) by
    any strides with contiguous heads, page_size a multiple of 16, head_dim a multiple of 8 up to 128.

    The tensors are checked once and stay the caller's.  `append` and `attend` report device-side conditions in an
    error word (`read_error`): KT_DEVERR_BAD_PAGE, KT_DEVERR_BAD_POSITION.  `attend` keeps one workspace per stream
    that it is called on (while a CUDA graph is captured, one of the graph's own)."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or t.dtype not in DTYPE_CODES:
                raise TypeError(f"{name} must be a bf16 or fp16 tensor")
            if t.dim() != 4 or not t.is_cuda or (t.stride(3) != 1 and t.shape[3] != 1):
                raise ValueError(f"{name} must be a CUDA tensor [num_pages, page_size, heads, head_dim] with "
                                 f"contiguous heads, got {tuple(t.shape)} on {t.device}")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must have one shape, dtype and device")
        self.num_pages, self.page_size, self.heads, self.head_dim = k_pages.shape
        if self.page_size % 16 or self.head_dim % 8 or self.head_dim > 128 or k_pages.numel() == 0:
            raise ValueError(f"page_size={self.page_size} must be a multiple of 16 and head_dim={self.head_dim} a "
                             "multiple of 8 up to 128")
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self.k_pages, self.v_pages = k_pages, v_pages   # keep them alive
        dense = (self.page_size * self.heads * self.head_dim, self.heads * self.head_dim, self.head_dim)
        strides = [st if size > 1 else d for t in (k_pages, v_pages)
                   for st, size, d in zip(t.stride(), t.shape[:3], dense)]
        self._desc = PagedKVDesc(k_pages.data_ptr(), v_pages.data_ptr(), *strides, self.num_pages, self.page_size,
                                 self.heads, self.head_dim, DTYPE_CODES[self.dtype])
        self._error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._err = self._error.data_ptr()
        self._workspaces = {}

    def read_error(self, clear: bool = True) -> int:
        """The error bits since the last clearing (waits for the current stream)."""
        code = int(self._error.item())
        if clear and code:
            self._error.zero_()
        return code

    def workspace(self) -> torch.Tensor:
        """A zeroed workspace for `attend`; calls that share one must not overlap."""
        with kt._on_device(self.device):
            n = int(kt.lib().kt_paged_attention_workspace_bytes())
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def _workspace(self, stream_ptr) -> torch.Tensor:
        if torch.cuda.is_current_stream_capturing():
            return self.workspace()   # lives in the graph's memory, zeroed by the graph
        ws = self._workspaces.get(stream_ptr)
        if ws is None:
            ws = self._workspaces[stream_ptr] = self.workspace()
        return ws

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
               seq_lens: torch.Tensor, table: torch.Tensor | None = None, q: torch.Tensor | None = None,
               q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
               style: str = "halves", q_out: torch.Tensor | None = None, stream=None):
        """Write the step's keys k and values v [tokens, heads, head_dim] to their pages, the keys normed (k_weight)
        and rotated (table) on the way; with q [tokens, q heads, head_dim], also return it normed (q_weight) and
        rotated.  One launch.  Tokens past cu_q[B] are left alone; options as qk_norm_rope's."""
        dt, dev, dim = self.dtype, self.device, self.head_dim
        n = k.shape[0]
        hk = _heads(k, "k", dt, dim, dev, None, self.heads)
        hv = _heads(v, "v", dt, dim, dev, n, self.heads)
        hq = None if q is None else _heads(q, "q", dt, dim, dev, n)
        batch = _batch(block_table, cu_q, seq_lens, n, dev)
        tf = _transform(table, q_weight, k_weight, eps, style, dt, dim, dev)
        with _allocating_on(stream, dev) as s:
            if q is not None and q_out is None:
                q_out = torch.empty(q.shape, dtype=dt, device=dev)
            elif q_out is not None:
                _written(q_out, "q_out")
        hqo = None if q is None else _heads(q_out, "q_out", dt, dim, dev, n, q.shape[1])
        with kt._on_device(dev):
            kt._check(kt.lib().kt_kv_append(self._desc, batch, hk, hv, hq, hqo, tf, self._err, s.ptr), "kt_kv_append")
        return q_out if q is not None else None

    def attend(self, q: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
               max_q_len: int, scale: float | None = None, window: int = 0, sinks: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the step's queries q [tokens, q heads, head_dim] over their sequences' pages, causal (the
        step's own keys are appended before); returns out of q's shape.

        max_q_len: an upper bound of the sequences' new tokens (it picks the kernel, not the result).  scale: default
        head_dim ** -0.5.  window > 0: each token sees its last `window` positions, its own among them.  sinks: f32
        [q heads], logits added to each softmax's sum.  A token that sees no key gets zeros.

        A non-finite value row reaches, besides the tokens that see it, others of the sequence that share a tile with
        those; rows past a sequence's keys reach nothing."""
        dt, dev, dim = self.dtype, self.device, self.head_dim
        hq = _heads(q, "q", dt, dim, dev)
        n, heads = q.shape[:2]
        batch = _batch(block_table, cu_q, seq_lens, n, dev)
        if sinks is not None and (sinks.dtype is not torch.float32 or sinks.shape != (heads,) or sinks.device != dev
                                  or not sinks.is_contiguous()):
            raise ValueError(f"sinks must be contiguous float32 [{heads}] on {dev}")
        with _allocating_on(stream, dev) as s:
            if out is None:
                out = torch.empty(q.shape, dtype=dt, device=dev)
            else:
                _written(out, "out")
            if workspace is None:
                workspace = self._workspace(s.ptr)
        ho = _heads(out, "out", dt, dim, dev, n, heads)
        with kt._on_device(dev):
            kt._check(kt.lib().kt_paged_attention(self._desc, batch, hq, ho, int(max_q_len),
                                                  dim ** -0.5 if scale is None else float(scale), int(window),
                                                  kt._ptr(sinks), self._err, workspace.data_ptr(), workspace.numel(),
                                                  s.ptr), "kt_paged_attention")
        return out
