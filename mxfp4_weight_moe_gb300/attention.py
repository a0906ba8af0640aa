"""Attention operators in front of the MoE layer (C ABI: ``include/kt_attn.h``).

``qk_norm_rope`` norms and rotates query and key heads; ``PagedKV`` is a cache
in pages, whose ``append`` writes a step's keys (normed and rotated on the way)
and values and whose ``attend`` computes the attention of the step's tokens
over it; ``PagedKV8`` is one that holds 8 bits an element.  As everywhere in the
package, the arithmetic runs in the library's CUDA kernels: this module checks
tensors, allocates outputs and passes pointers and the CUDA stream.

A step's batch is three int32 tensors: ``block_table`` [B, max_pages] (the pages
of each sequence in order), ``cu_q`` [B + 1] (sequence b has the step's tokens
cu_q[b] .. cu_q[b+1]) and ``seq_lens`` [B] (its keys in all, the step's own
included, so that its last new token has position seq_lens[b] - 1).
"""
from __future__ import annotations

import ctypes
import struct
import threading
import weakref

import torch

import mxfp4_weight_moe_gb300 as kt

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}   # KT_DTYPE_*
KT_DTYPE_F32 = 2
ROPE_STYLES = {"halves": 0, "interleaved": 1}

KT_DEVERR_BAD_PAGE = 0x20
KT_DEVERR_BAD_POSITION = 0x40

# The descriptors of kt_attn.h as packed fields (64-bit hosts).  A decode step's calls take a few microseconds on the
# GPU, so a call packs its descriptors into one buffer of the thread's and passes addresses in it.
HEADS = "Pqqixxxx"                    # kt_heads: ptr, token_stride, head_stride, heads
PAGED_KV = "PPqqqqqqiiiiixxxx"        # kt_paged_kv: k, v, strides, num_pages, page_size, heads, head_dim, dtype
PAGED_KV8 = "PPPPqqqqqqiiiiixxxx"     # kt_paged_kv8: k, v, their scales, strides, sizes, dtype
PAGED_BATCH = "PqixxxxPPii"           # kt_paged_batch: block_table, table_stride, max_pages, cu_q, seq_lens, sizes
HEAD_TRANSFORM = "PiiixxxxPPif"       # kt_head_transform: table, positions, rotary_dim, style, weights, dtype, eps
_HEADS_BYTES, _BATCH_BYTES = struct.calcsize(HEADS), struct.calcsize(PAGED_BATCH)
_NORM_CALL = struct.Struct(HEAD_TRANSFORM + 4 * HEADS)
_APPEND_CALL = struct.Struct(HEAD_TRANSFORM + PAGED_BATCH + 4 * HEADS)
_ATTEND_CALL = struct.Struct(PAGED_BATCH + 2 * HEADS)
_TRANSFORM_BYTES = struct.calcsize(HEAD_TRANSFORM)
_NO_HEADS = (0, 0, 0, 0)

WORKSPACE_ZEROED = 4096   # KT_PAGED_ATTENTION_ZEROED


class _Buffer(threading.local):
    def __init__(self):
        self.buf = ctypes.create_string_buffer(512)
        self.at = ctypes.addressof(self.buf)


_buffer = _Buffer()

_VP, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "kt_qk_norm_rope": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP], _I),
    "kt_kv_append": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP], _I),
    "kt_paged_attention_workspace_bytes": ([], ctypes.c_size_t),
    "kt_kv8_append": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP], _I),
    "kt_paged_attention8": ([_VP, _VP, _VP, _VP, _I, _F, _I, _VP, _VP, _VP, ctypes.c_size_t, _VP], _I),
    "kt_paged_attention": ([_VP, _VP, _VP, _VP, _I, _F, _I, _VP, _VP, _VP, ctypes.c_size_t, _VP], _I),
}


def _heads(t, name: str, dtype, dim: int, device: int, tokens: int, heads: int):
    """(ptr, token stride, head stride, heads) of a [tokens, heads, dim] tensor with contiguous heads on CUDA device
    `device` (tokens, heads: -1 for any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{device}" if device >= 0 else "a CUDA device"))
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (tokens >= 0 and shape[0] != tokens) or (heads >= 0 and shape[1] != heads):
        raise ValueError(f"{name} must be [{tokens if tokens >= 0 else 'tokens'}, {heads if heads >= 0 else 'heads'}, "
                         f"{dim}], got {tuple(shape)}")
    by_token, by_head, by_element = t.stride()
    if by_element != 1 and dim != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous, strides are {t.stride()}")
    # the stride of a dimension of one entry says nothing
    n, h, _ = shape
    return t.data_ptr(), (by_token if n > 1 else dim), (by_head if h > 1 else dim), h


def _written(t, name: str):
    """An output whose elements overlap would be written by several threads at once."""
    if t.is_contiguous():
        return
    (n, h, d), st = t.shape, t.stride()
    if t.numel() and ((h > 1 and st[1] < d) or (n > 1 and st[0] < d)
                      or (n > 1 and h > 1 and st[0] < (h - 1) * st[1] + d and st[1] < (n - 1) * st[0] + d)):
        raise ValueError(f"{name}: its rows overlap, strides are {st}")


def _rows_meet(a, b, n: int, dim: int) -> bool:
    """Whether a row of a and one of b (n tokens each, as _heads describes them) share an element."""
    between = (b[0] - a[0]) // 2
    (_, ta, ha, na), (_, tb, hb, nb) = a, b
    if ta == tb and (na - 1) * ha + dim <= between % ta <= ta - (nb - 1) * hb - dim:
        return False                                     # side by side in every token: slices of one projection
    if ta == tb and ha == hb and ta % ha == 0 and dim <= between % ha <= ha - dim:
        return False                                     # side by side in every head
    first = (torch.arange(n)[:, None] * ta + torch.arange(na) * ha).flatten().sort().values
    other = (torch.arange(n)[:, None] * tb + torch.arange(nb) * hb).flatten() + between
    after = torch.searchsorted(first, other, right=True)     # the first row that starts after each of the others
    return bool(((after > 0) & (first[(after - 1).clamp(min=0)] + dim > other)).any()
                or ((after < len(first)) & (first[after.clamp(max=len(first) - 1)] < other + dim)).any())


def _span(a, n: int, dim: int):
    return a[0], a[0] + 2 * ((n - 1) * a[1] + (a[3] - 1) * a[2] + dim)


def _apart(name: str, out, n: int, dim: int, own, others=(), spans=()):
    """Refuse an output that shares memory with an input or another output, where threads would write what others read.

    out, own and the `others` are as _heads describes them; out may be `own`, the input of the same rows.  spans: from
    one end to the other of a cache's pages; out lies outside them."""
    if n == 0 or dim == 0 or out[3] == 0:
        return
    lo, hi = _span(out, n, dim)
    for x in (own, *others) if out != own else others:
        a, b = _span(x, n, dim)
        if a < hi and lo < b and _rows_meet(out, x, n, dim):
            raise ValueError(f"{name} shares memory with another tensor of the call")
    for a, b in spans:
        if a < hi and lo < b:
            raise ValueError(f"{name} lies among the cache's pages")


def _ints(t, name: str, ndim: int, device: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != ndim or t.get_device() != device:
        raise ValueError(f"{name} must have {ndim} dims on cuda:{device}, got {tuple(t.shape)} on {t.device}")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous")


def _batch(block_table, cu_q, seq_lens, tokens: int, device: int):
    _ints(block_table, "block_table", 2, device)
    _ints(cu_q, "cu_q", 1, device)
    _ints(seq_lens, "seq_lens", 1, device)
    seqs, max_pages = block_table.shape
    if seq_lens.shape[0] != seqs or cu_q.shape[0] != seqs + 1:
        raise ValueError(f"block_table {tuple(block_table.shape)}, cu_q {tuple(cu_q.shape)} and seq_lens "
                         f"{tuple(seq_lens.shape)} must be [B, max_pages], [B + 1] and [B]")
    return (block_table.data_ptr(), block_table.stride(0) if seqs > 1 else max_pages, max_pages, cu_q.data_ptr(),
            seq_lens.data_ptr(), seqs, tokens)


def _weight(w, name: str, dtype, dim: int, device: int):
    if w.dtype is not dtype and w.dtype is not torch.float32:
        raise TypeError(f"{name} must be {dtype} or torch.float32, got {w.dtype}")
    if w.shape != (dim,) or w.get_device() != device or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{dim}] on cuda:{device}")
    return w.data_ptr()


def _transform(table, q_weight, k_weight, eps: float, style: str, dtype, dim: int, device: int):
    t = positions = rot = code = qw = kw = weight_dtype = 0
    if table is not None:
        if table.dtype is not torch.float32:
            raise TypeError(f"table must be torch.float32, got {table.dtype}")
        if table.dim() != 2 or table.get_device() != device or not table.is_contiguous():
            raise ValueError(f"table must be contiguous [positions, rotary_dim] on cuda:{device}")
        if style not in ROPE_STYLES:
            raise ValueError(f"style must be one of {tuple(ROPE_STYLES)}")
        t, (positions, rot), code = table.data_ptr(), table.shape, ROPE_STYLES[style]
    if q_weight is not None:
        qw = _weight(q_weight, "q_weight", dtype, dim, device)
        weight_dtype = DTYPE_CODES.get(q_weight.dtype, KT_DTYPE_F32)
    if k_weight is not None:
        kw = _weight(k_weight, "k_weight", dtype, dim, device)
        weight_dtype = DTYPE_CODES.get(k_weight.dtype, KT_DTYPE_F32)
        if q_weight is not None and q_weight.dtype is not k_weight.dtype:
            raise TypeError("q_weight and k_weight must have one dtype")
    return t, positions, rot, code, qw, kw, weight_dtype, eps


def _int(x) -> int:
    """A count as the library's int, which wraps: the largest one for larger counts, -1 (which is refused) below 0."""
    return min(max(int(x), -1), 0x7FFFFFFF)


def _output(like, stream):
    """A contiguous output of like's shape that belongs to `stream` (None: the current one)."""
    if stream is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(like, memory_format=torch.contiguous_format)


_functions = {}


def _call(device: int, stream, name: str, *args):
    """The library's `name` on the device, with args and the stream's pointer."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(kt.lib(), name)
    ptr = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, ptr)
    else:
        with torch.cuda.device(device):
            status = fn(*args, ptr)
    if status:
        kt._check(status, name)


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

    bf16 or fp16; heads may be slices of a packed projection.  q_out may be q and k_out k; they share no memory
    otherwise.  positions: int32 [tokens];
    table: rope_table's; style "halves" (pairs i, i + rotary_dim/2) or "interleaved" (2i, 2i+1).  error: an int32
    [1] tensor that gets KT_DEVERR_BAD_POSITION for a position outside the table (that token is not written)."""
    if not isinstance(q, torch.Tensor) or q.dtype not in DTYPE_CODES or q.dim() != 3:
        raise TypeError("q must be a bf16 or fp16 tensor [tokens, heads, head_dim]")
    dev, dt = q.get_device(), q.dtype
    n, heads, dim = q.shape
    hq = _heads(q, "q", dt, dim, dev, -1, -1)
    hk = _NO_HEADS if k is None else _heads(k, "k", dt, dim, dev, n, -1)
    pos = 0
    if table is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        _ints(positions, "positions", 1, dev)
        if positions.shape[0] != n:
            raise ValueError(f"positions must be [{n}]")
        pos = positions.data_ptr()
    tf = _transform(table, q_weight, k_weight, eps, style, dt, dim, dev)
    if error is not None:
        _ints(error, "error", 1, dev)
    q_given, k_given = q_out is not None, k is not None and k_out is not None
    if q_given:
        _written(q_out, "q_out")
    else:
        q_out = _output(q, stream)
    hqo, hko = _heads(q_out, "q_out", dt, dim, dev, n, heads), _NO_HEADS
    if k is not None:
        if k_given:
            _written(k_out, "k_out")
        else:
            k_out = _output(k, stream)
        hko = _heads(k_out, "k_out", dt, dim, dev, n, hk[3])
    if q_given:
        _apart("q_out", hqo, n, dim, hq, () if k is None else (hk, hko))
    if k_given:
        _apart("k_out", hko, n, dim, hk, (hq, hqo))
    b = _buffer
    _NORM_CALL.pack_into(b.buf, 0, *tf, *hq, *hk, *hqo, *hko)
    at = b.at + _TRANSFORM_BYTES
    _call(dev, stream, "kt_qk_norm_rope", at, at + _HEADS_BYTES if k is not None else None, at + 2 * _HEADS_BYTES,
          at + 3 * _HEADS_BYTES if k is not None else None, pos, n, dim, DTYPE_CODES[dt], b.at,
          None if error is None else error.data_ptr())
    return q_out, (k_out if k is not None else None)


class PagedKV:
    """A key/value cache in pages: k_pages and v_pages are [num_pages, page_size, heads, head_dim] (bf16 or fp16) by
    any strides with contiguous heads, page_size a multiple of 16, head_dim a multiple of 8 up to 128.

    The tensors are checked once and stay the caller's.  `append` and `attend` report device-side conditions in an
    error word (`read_error`): KT_DEVERR_BAD_PAGE, KT_DEVERR_BAD_POSITION, of `attend` also KT_DEVERR_TIMEOUT_*; making
    the object waits for the current stream, so that the word is clear for calls on any.  `attend` needs a workspace
    (`workspace`): it keeps one for each stream that it is called on, which all cache objects share there.  While a CUDA
    graph is captured, each call takes one of the graph's own and clears its counters; passing one `workspace()` to all
    of a graph's calls leaves that out."""

    _shared = weakref.WeakValueDictionary()   # (device, stream) -> workspace, kept by the objects that use it
    _append, _attend = "kt_kv_append", "kt_paged_attention"

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
        self._spans = self._spans_of(k_pages, v_pages)
        self._describe(struct.pack(PAGED_KV, k_pages.data_ptr(), v_pages.data_ptr(), *self._strides_of(k_pages, v_pages),
                                   self.num_pages, self.page_size, self.heads, self.head_dim, DTYPE_CODES[self.dtype]))

    @staticmethod
    def _strides_of(*pages):
        """Page, slot and head strides of each (the stride of a dimension of one entry says nothing: a dense one)."""
        _, page_size, heads, dim = pages[0].shape
        return [st if size > 1 else d for t in pages
                for st, size, d in zip(t.stride(), t.shape[:3], (page_size * heads * dim, heads * dim, dim))]

    @staticmethod
    def _spans_of(*tensors):
        """From one end to the other of each tensor's memory."""
        return tuple((t.data_ptr(), t.data_ptr() + t.element_size() * (1 + sum((size - 1) * st for size, st in
                                                                              zip(t.shape, t.stride()))))
                     for t in tensors)

    def _describe(self, desc: bytes):
        self._index = self.device.index
        self._desc = ctypes.create_string_buffer(desc)
        self._desc_at = ctypes.addressof(self._desc)
        with torch.cuda.device(self.device):
            self._error = torch.zeros(1, dtype=torch.int32, device=self.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()   # calls may come on any stream: it is zero before the first
        self._err = self._error.data_ptr()
        self._workspaces = {}

    def read_error(self, clear: bool = True, stream=None) -> int:
        """The error bits since the last clearing; waits for `stream` (default: the current one), on which the calls in
        question were made, and clears the bits that it returns."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.read_error(clear)
        code = int(self._error.item())
        if clear and code:
            self._error.bitwise_and_(~code)
            torch.cuda.current_stream(self.device).synchronize()   # before calls on other streams set them again
        return code

    def workspace(self) -> torch.Tensor:
        """A workspace for `attend` (some 40 MB: partial results of two pieces of 256 query rows for each SM, whatever
        the cache's size); calls that share one must not overlap."""
        with torch.cuda.device(self.device):
            n = int(kt.lib().kt_paged_attention_workspace_bytes())
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
            ws[:WORKSPACE_ZEROED].zero_()
        return ws

    def _workspace(self, stream) -> torch.Tensor:
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._workspace(None)
        if torch.cuda.is_current_stream_capturing():
            return self.workspace()   # lives in the graph's memory, cleared by the graph
        ptr = torch._C._cuda_getCurrentRawStream(self._index)
        ws = self._workspaces.get(ptr)
        if ws is None:
            ws = self._shared.get((self._index, ptr))   # calls on one stream do not overlap
            if ws is None:
                ws = self._shared[self._index, ptr] = self.workspace()
            self._workspaces[ptr] = ws
        return ws

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
               seq_lens: torch.Tensor, table: torch.Tensor | None = None, q: torch.Tensor | None = None,
               q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
               style: str = "halves", q_out: torch.Tensor | None = None, stream=None):
        """Write the step's keys k and values v [tokens, heads, head_dim] to their pages, the keys normed (k_weight)
        and rotated (table) on the way; with q [tokens, q heads, head_dim], also return it normed (q_weight) and
        rotated (q_out may be q).  One launch.  Tokens past cu_q[B] are left alone; options as qk_norm_rope's."""
        dt, dev, dim = self.dtype, self._index, self.head_dim
        hk = _heads(k, "k", dt, dim, dev, -1, self.heads)
        n = k.shape[0]
        hv = _heads(v, "v", dt, dim, dev, n, self.heads)
        hq, hqo = _NO_HEADS, _NO_HEADS
        if q is not None:
            hq = _heads(q, "q", dt, dim, dev, n, -1)
            if q_out is None:
                q_out = _output(q, stream)
                hqo = _heads(q_out, "q_out", dt, dim, dev, n, hq[3])
            else:
                _written(q_out, "q_out")
                hqo = _heads(q_out, "q_out", dt, dim, dev, n, hq[3])
                _apart("q_out", hqo, n, dim, hq, (hk, hv), self._spans)
        tf = _transform(table, q_weight, k_weight, eps, style, dt, dim, dev)
        b = _buffer
        _APPEND_CALL.pack_into(b.buf, 0, *tf, *_batch(block_table, cu_q, seq_lens, n, dev), *hk, *hv, *hq, *hqo)
        at = b.at + _TRANSFORM_BYTES
        heads = at + _BATCH_BYTES
        _call(dev, stream, self._append, self._desc_at, at, heads, heads + _HEADS_BYTES,
              heads + 2 * _HEADS_BYTES if q is not None else None, heads + 3 * _HEADS_BYTES if q is not None else None,
              b.at, self._err)
        return q_out if q is not None else None

    def attend(self, q: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
               max_q_len: int, scale: float | None = None, window: int = 0, sinks: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the step's queries q [tokens, q heads, head_dim] over their sequences' pages, causal (the
        step's own keys are appended before); returns out, of q's shape and possibly q itself.

        max_q_len: an upper bound of the sequences' new tokens (it picks the kernel, not the result).  scale: default
        head_dim ** -0.5.  window > 0: each token sees its last `window` positions, its own among them.  sinks: f32
        [q heads], logits added to each softmax's sum.  A token that sees no key gets zeros.  Pages that lie before
        every token's window are not read, whatever their entries say.

        A non-finite value row reaches, besides the tokens that see it, others of the sequence that share a tile with
        those; rows past a sequence's keys reach nothing."""
        dt, dev, dim = self.dtype, self._index, self.head_dim
        hq = _heads(q, "q", dt, dim, dev, -1, -1)
        n, heads = q.shape[0], hq[3]
        batch = _batch(block_table, cu_q, seq_lens, n, dev)
        sink = None
        if sinks is not None:
            if (sinks.dtype is not torch.float32 or sinks.shape != (heads,) or sinks.get_device() != dev
                    or not sinks.is_contiguous()):
                raise ValueError(f"sinks must be contiguous float32 [{heads}] on {self.device}")
            sink = sinks.data_ptr()
        if out is None:
            out = _output(q, stream)
            ho = _heads(out, "out", dt, dim, dev, n, heads)
        else:
            _written(out, "out")
            ho = _heads(out, "out", dt, dim, dev, n, heads)
            _apart("out", ho, n, dim, hq, (), self._spans)
        if workspace is None:
            workspace = self._workspace(stream)
        elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous uint8 on {self.device}")
        b = _buffer
        _ATTEND_CALL.pack_into(b.buf, 0, *batch, *hq, *ho)
        at = b.at + _BATCH_BYTES
        _call(dev, stream, self._attend, self._desc_at, b.at, at, at + _HEADS_BYTES, _int(max_q_len),
              dim ** -0.5 if scale is None else float(scale), _int(window), sink, self._err, workspace.data_ptr(),
              workspace.numel())
        return out


class PagedKV8(PagedKV):
    """A key/value cache in pages of 8 bits an element: k_pages and v_pages are [num_pages, page_size, heads, head_dim]
    (float8_e4m3fn or uint8 codes) by any strides that are multiples of 16 with contiguous heads, page_size and head_dim
    multiples of 16, head_dim up to 128; k_scales and v_scales are contiguous uint8 (e8m0) [num_pages, page_size / 16,
    heads].  An element stands for e4m3(code) * 2^(scale - 127): a power of two for each 16 positions and head.

    dtype: of the keys, values and queries that come in and of the attention's output (bf16 or fp16).  `append` and
    `attend` are PagedKV's: `append` picks the powers (the least that hold the 16 positions' values, from 2^-117 to
    2^87 for bf16 and from 2^-14 to 2^7 for fp16, past which values saturate at 448 times that; a block that has older
    tokens keeps its power or rescales their codes to a larger one), and `attend` computes with the numbers that the
    cache stands for.  A rotation table's width is a multiple of 16, k and v are 16-byte aligned with strides that are
    multiples of 8 (queries that are not so have a launch of their own).  A key or value element that is not finite
    makes its 16 positions of that head NaN, until the first of them is appended anew (taking the token back does not
    bring the older ones back): what sees one of them is NaN.  Values that are NaN reach other tokens of the sequence
    (attend) only in calls of more than 32 query rows, max_q_len times the query heads of a cache head."""

    BLOCK = 16   # KT_KV8_BLOCK
    _append, _attend = "kt_kv8_append", "kt_paged_attention8"

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                 dtype: torch.dtype = torch.bfloat16):
        if dtype not in DTYPE_CODES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or t.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"{name} must be a float8_e4m3fn or uint8 tensor")
            if t.dim() != 4 or not t.is_cuda or (t.stride(3) != 1 and t.shape[3] != 1):
                raise ValueError(f"{name} must be a CUDA tensor [num_pages, page_size, heads, head_dim] with "
                                 f"contiguous heads, got {tuple(t.shape)} on {t.device}")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must have one shape, dtype and device")
        self.num_pages, self.page_size, self.heads, self.head_dim = k_pages.shape
        if self.page_size % self.BLOCK or self.head_dim % 16 or self.head_dim > 128 or k_pages.numel() == 0:
            raise ValueError(f"page_size={self.page_size} must be a multiple of {self.BLOCK} and head_dim="
                             f"{self.head_dim} a multiple of 16 up to 128")
        shape = (self.num_pages, self.page_size // self.BLOCK, self.heads)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8:
                raise TypeError(f"{name} must be a uint8 tensor")
            if t.shape != shape or t.device != k_pages.device or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {list(shape)} on {k_pages.device}")
        self.dtype, self.device = dtype, k_pages.device
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self._spans = self._spans_of(k_pages, v_pages, k_scales, v_scales)
        self._describe(struct.pack(PAGED_KV8, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                                   v_scales.data_ptr(), *self._strides_of(k_pages, v_pages), *k_pages.shape,
                                   DTYPE_CODES[dtype]))
