"""Binding of libvqv's operators around the projections in a verify round
(include/vqv_round.h): rotary positions and the append to a paged cache,
attention over it, its pages, and edits of logits.

The classes hold a call's tensors and the struct that the library reads, made
once; the functions carry the C names and only marshal arguments. The library
sees pointers, so every tensor's device, type, size and layout is checked
here. Calls go to the current stream unless `stream` names another (its
handle, or a torch stream); what a call allocates, outputs or a workspace, then
belongs to that stream.
"""

from __future__ import annotations

import ctypes

import torch

from .vqv import VQV_BF16, VQV_FP16, VQV_FP32, VqvError
from .vqv import _on_device
from .vqv import lib as _load
from .vqv import vqv_status_string, vqv_verify_workspace_bytes

ROUND_EXPORTS = ("vqv_rope_plan", "vqv_rope_append", "vqv_paged_attn_workspace_bytes",
                 "vqv_paged_attn", "vqv_cache_workspace_bytes", "vqv_cache_copy",
                 "vqv_cache_trim", "vqv_cache_reserve", "vqv_cache_fork", "vqv_cache_compact",
                 "vqv_logits_edit", "vqv_logits_verify")
ROPE_SCALINGS = ("none", "linear", "ntk", "yarn", "smooth")

_DTYPES = {torch.bfloat16: VQV_BF16, torch.float16: VQV_FP16, torch.float32: VQV_FP32}
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("layers", _i), ("pages", _i), ("page_size", _i),
                ("kv_heads", _i), ("dim", _i), ("dtype", _i), ("layer_stride", _i64),
                ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64)]


class _Seqs(ctypes.Structure):
    _fields_ = [("row_start", _vp), ("kv_len", _vp), ("table", _vp), ("table_stride", _i64),
                ("n_seqs", _i), ("table_width", _i), ("n_rows", _i), ("max_rows", _i),
                ("max_kv", _i)]


class _Rope(ctypes.Structure):
    _fields_ = [("rot", _i), ("interleaved", _i), ("mscale", ctypes.c_float), ("reserved", _i),
                ("turns", ctypes.c_double * 128)]


class _Pages(ctypes.Structure):
    _fields_ = [("ref", _vp), ("table", _vp), ("held", _vp), ("length", _vp), ("pages", _i),
                ("rows", _i), ("width", _i), ("page_size", _i)]


class _Edits(ctypes.Structure):
    _fields_ = [("n_seqs", _i), ("n", _i), ("counts", _vp), ("seen", _vp), ("repetition", _vp),
                ("frequency", _vp), ("presence", _vp), ("bias_start", _vp), ("bias_token", _vp),
                ("bias_value", _vp), ("n_bias", _i), ("reserved", _i)]


_lib = None


def _round_lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _load()
        p = ctypes.POINTER
        cache, seqs, rope, pages, edits = p(_Cache), p(_Seqs), p(_Rope), p(_Pages), p(_Edits)
        f32, f64 = ctypes.c_float, ctypes.c_double
        for name, res, args in (
                ("vqv_rope_plan", _i, [rope, _i, f64, _i, _i, f64, _i]),
                ("vqv_rope_append", _i, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i, _i,
                                         cache, _i, seqs, rope, _vp, _vp]),
                ("vqv_paged_attn_workspace_bytes", _sz, [cache, seqs, _i, _i, _i]),
                ("vqv_paged_attn", _i, [_vp, cache, _i, seqs, _i, f32, _i, _i, _vp, _vp, _sz,
                                        _vp]),
                ("vqv_cache_workspace_bytes", _sz, [pages]),
                ("vqv_cache_copy", _i, [cache, _vp, _vp, _i, _vp]),
                ("vqv_cache_trim", _i, [pages, _vp, _vp, _i, _vp]),
                ("vqv_cache_reserve", _i, [pages, _vp, _i, _vp, _vp, _sz, _vp]),
                ("vqv_cache_fork", _i, [cache, pages, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
                ("vqv_cache_compact", _i, [cache, seqs, _vp, _vp, _vp]),
                ("vqv_logits_edit", _i, [_vp, edits, _vp, _i, _vp, _vp, _vp]),
                ("vqv_logits_verify", _i, [_vp, edits, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _sz,
                                           _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status:
        raise VqvError(status, vqv_status_string(status))


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _stream(stream, device: torch.device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _take(t: torch.Tensor | None, name: str, shape: tuple, dtype: torch.dtype,
          device: torch.device) -> int | None:
    """Pointer of a dense tensor that holds exactly `shape`."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense {dtype} tensor of shape {list(shape)} on "
                         f"{device}, got {t.dtype} {list(t.shape)} on {t.device}"
                         + ("" if t.is_contiguous() else ", not dense"))
    return t.data_ptr()


def _new(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """An empty tensor that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(workspace: torch.Tensor | None, need: int, device: torch.device, stream) -> tuple:
    """(tensor, pointer, bytes) of the caller's workspace, or of one made here."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _new(need, torch.uint8, device, stream)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a dense tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


class PagedCache:
    """Keys and values [layers, pages, page size, kv heads, dim] (bf16 or fp16,
    views of any order with a dense last dimension, the same strides)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be [layers, pages, page size, kv heads, dim] with the "
                             "same shape, type and strides")
        if k.stride(4) != 1 and k.shape[4] > 1:
            raise ValueError("k and v must be dense in their last dimension")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"unsupported cache type {k.dtype}")
        self.device = _device(k, "k")
        if v.device != self.device:
            raise ValueError(f"v is on {v.device}, k on {self.device}")
        self.k, self.v, self.dtype = k, v, k.dtype
        self.layers, self.pages, self.page_size, self.kv_heads, self.dim = k.shape
        # A dimension of one has no stride to speak of.
        st = [s if n > 1 else 0 for s, n in zip(k.stride(), k.shape)]
        self.c = _Cache(k.data_ptr(), v.data_ptr(), *k.shape, _DTYPES[k.dtype], *st[:4])


class Sequences:
    """The new rows of a call, sequence after sequence: row_start [n + 1],
    kv_len [n] (the new rows among them) and table [n, width], all int32.
    n_rows is row_start's last value; max_rows and max_kv bound what the device
    holds (counts of rows, kv_len)."""

    def __init__(self, row_start: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor,
                 n_rows: int, max_rows: int, max_kv: int):
        dev = self.device = _device(row_start, "row_start")
        n = kv_len.numel()
        if table.dim() != 2 or table.shape[0] < n or table.dtype != torch.int32 \
                or table.device != dev or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError(f"table must be int32 [n_seqs or more, width] on {dev}, its rows dense")
        self.row_start, self.kv_len, self.table = row_start, kv_len, table
        self.n_seqs, self.n_rows, self.max_rows, self.max_kv = n, n_rows, max_rows, max_kv
        self.c = _Seqs(_take(row_start, "row_start", (n + 1,), torch.int32, dev),
                       _take(kv_len, "kv_len", (n,), torch.int32, dev), table.data_ptr(),
                       max(table.stride(0), table.shape[1]) if table.shape[0] == 1
                       else table.stride(0),
                       n, table.shape[1], n_rows, max_rows, max_kv)


class Rope:
    """Rotary positions of the first `rot` values of each head, as pairs (2i,
    2i+1) (interleaved) or (i, i + rot/2); scaling is one of ROPE_SCALINGS,
    over `factor`, for a model trained on `original_len` positions."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: int = 0):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {ROPE_SCALINGS}")
        self.rot, self.interleaved = rot, interleaved
        self.c = _Rope()
        _check(_round_lib().vqv_rope_plan(ctypes.byref(self.c), rot, base, int(interleaved),
                                          ROPE_SCALINGS.index(scaling), factor, original_len))


class Pages:
    """Which table row holds which page: ref [pages], table [rows, width],
    held [rows] and length [rows], all int32; page ids of -1 where none."""

    def __init__(self, ref: torch.Tensor, table: torch.Tensor, held: torch.Tensor,
                 length: torch.Tensor, page_size: int):
        dev = self.device = _device(ref, "ref")
        if table.dim() != 2:
            raise ValueError("table must be [rows, width]")
        rows, width = table.shape
        self.ref, self.table, self.held, self.length = ref, table, held, length
        self.rows, self.page_size = rows, page_size
        self.c = _Pages(_take(ref, "ref", (ref.numel(),), torch.int32, dev),
                        _take(table, "table", (rows, width), torch.int32, dev),
                        _take(held, "held", (rows,), torch.int32, dev),
                        _take(length, "length", (rows,), torch.int32, dev),
                        ref.numel(), rows, width, page_size)


class Edits:
    """What is done to the logits of n_seqs sequences over `vocab` tokens, see
    include/vqv_round.h: counts [n_seqs, vocab] int32, seen [n_seqs,
    ceil(vocab/32)] int32 bits; repetition, frequency, presence [n_seqs] fp32;
    biases as bias_start [n_seqs + 1], bias_token int32 and bias_value fp32."""

    def __init__(self, n_seqs: int, vocab: int, counts=None, seen=None, repetition=None,
                 frequency=None, presence=None, bias_start=None, bias_token=None,
                 bias_value=None):
        given = [t for t in (counts, seen, repetition, frequency, presence, bias_start)
                 if t is not None]
        dev = self.device = _device(given[0], "edits") if given else None
        self.n_seqs, self.vocab, self.words = n_seqs, vocab, -(-vocab // 32)
        n_bias = 0
        if bias_start is not None:
            if bias_token is None or bias_value is None:
                raise ValueError("bias_start needs bias_token and bias_value")
            n_bias = bias_token.numel()
        else:
            bias_token = bias_value = None
        i32, f32 = torch.int32, torch.float32
        self.tensors = (counts, seen, repetition, frequency, presence, bias_start, bias_token,
                        bias_value)
        self.c = _Edits(n_seqs, vocab, _take(counts, "counts", (n_seqs, vocab), i32, dev),
                        _take(seen, "seen", (n_seqs, self.words), i32, dev),
                        _take(repetition, "repetition", (n_seqs,), f32, dev),
                        _take(frequency, "frequency", (n_seqs,), f32, dev),
                        _take(presence, "presence", (n_seqs,), f32, dev),
                        _take(bias_start, "bias_start", (n_seqs + 1,), i32, dev),
                        _take(bias_token, "bias_token", (n_bias,), i32, dev),
                        _take(bias_value, "bias_value", (n_bias,), f32, dev), n_bias, 0)


def _rows(t: torch.Tensor, name: str, shape: tuple, dtype, device) -> tuple:
    if t.shape != shape or t.dtype != dtype or t.device != device or t.stride(2) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)} on {device} with "
                         f"a dense last dimension, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else 0, t.stride(1) if shape[1] > 1 else 0


def _same(device: torch.device, **others) -> None:
    for name, x in others.items():
        if x.device != device:
            raise ValueError(f"{name} is on {x.device}, the cache on {device}")


def vqv_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedCache,
                    seqs: Sequences, rope: Rope, layer: int = 0,
                    q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotated q [n_rows, heads, dim] in the cache's type; rotated k and v
    [n_rows, kv heads, dim] are written to the sequences' pages. q, k and v may
    be slices of one stacked projection, in bf16, fp16 or fp32."""
    dev, n = cache.device, seqs.n_rows
    _same(dev, seqs=seqs)
    if q.dim() != 3 or q.dtype not in _DTYPES:
        raise ValueError("q must be [n_rows, heads, dim] in bf16, fp16 or fp32")
    heads = q.shape[1]
    ins = (*_rows(q, "q", (n, heads, cache.dim), q.dtype, dev),
           *_rows(k, "k", (n, cache.kv_heads, cache.dim), q.dtype, dev),
           *_rows(v, "v", (n, cache.kv_heads, cache.dim), q.dtype, dev))
    if q_out is None:
        q_out = _new((n, heads, cache.dim), cache.dtype, dev, stream)
    out = _take(q_out, "q_out", (n, heads, cache.dim), cache.dtype, dev)
    _check(_on_device(
        dev, _round_lib().vqv_rope_append, *ins, _DTYPES[q.dtype], heads, cache.c, layer, seqs.c,
        rope.c, out, _stream(stream, dev)))
    return q_out


def vqv_paged_attn_workspace_bytes(cache: PagedCache, seqs: Sequences, heads: int,
                                   window: int = 0, sinks: int = 0) -> int:
    return _round_lib().vqv_paged_attn_workspace_bytes(cache.c, seqs.c, heads, window, sinks)


def vqv_paged_attn(q: torch.Tensor, cache: PagedCache, seqs: Sequences, scale: float,
                   window: int = 0, sinks: int = 0, layer: int = 0,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Causal attention of q [n_rows, heads, dim] over the sequences' pages;
    with a window, over the last `window` tokens and the first `sinks`."""
    dev = cache.device
    _same(dev, seqs=seqs)
    if q.dim() != 3:
        raise ValueError("q must be [n_rows, heads, dim]")
    heads = q.shape[1]
    shape = (seqs.n_rows, heads, cache.dim)
    qp = _take(q, "q", shape, cache.dtype, dev)
    if out is None:
        out = _new(shape, cache.dtype, dev, stream)
    op = _take(out, "out", shape, cache.dtype, dev)
    need = 0 if workspace is not None else vqv_paged_attn_workspace_bytes(cache, seqs, heads,
                                                                          window, sinks)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _round_lib().vqv_paged_attn, qp, cache.c, layer, seqs.c, heads, scale, window, sinks,
        op, wp, wn, _stream(stream, dev)))
    return out


def vqv_cache_workspace_bytes(pages: Pages) -> int:
    return _round_lib().vqv_cache_workspace_bytes(pages.c)


def _list(t: torch.Tensor, name: str, n: int, device) -> int:
    return _take(t, name, (n,), torch.int32, device)


def vqv_cache_copy(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Pages src[i] to dst[i] (int32), on all layers."""
    n = src.numel()
    _check(_on_device(
        cache.device, _round_lib().vqv_cache_copy, cache.c, _list(src, "src", n, cache.device),
        _list(dst, "dst", n, cache.device), n, _stream(stream, cache.device)))


def vqv_cache_trim(pages: Pages, keep_len: torch.Tensor, rows: torch.Tensor | None = None,
                   stream=None) -> None:
    """Gives back the pages of table rows (`rows`, or the first ones) past
    keep_len tokens. A row that is cut inside pages that others hold too gets
    no room from vqv_cache_reserve: go on with a fork of it."""
    n, dev = keep_len.numel(), pages.device
    _check(_on_device(
        dev, _round_lib().vqv_cache_trim, pages.c, _list(keep_len, "keep_len", n, dev),
        _list(rows, "rows", n, dev), n, _stream(stream, dev)))


def vqv_cache_reserve(pages: Pages, goal_len: torch.Tensor, ok: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Takes free pages until the first rows hold goal_len tokens' worth;
    returns ok [rows] int32, 0 where there are too few or the row's next token
    would be written to a page that other rows hold too."""
    n, dev = goal_len.numel(), pages.device
    if ok is None:
        ok = _new(n, torch.int32, dev, stream)
    need = 0 if workspace is not None else vqv_cache_workspace_bytes(pages)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _round_lib().vqv_cache_reserve, pages.c, _list(goal_len, "goal_len", n, dev), n,
        _list(ok, "ok", n, dev), wp, wn, _stream(stream, dev)))
    return ok


def vqv_cache_fork(cache: PagedCache, pages: Pages, parent: torch.Tensor, child: torch.Tensor,
                   ok: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Table rows child[i] become branches of rows parent[i]; returns ok [n]
    int32."""
    n, dev = parent.numel(), pages.device
    _same(cache.device, pages=pages)
    if ok is None:
        ok = _new(n, torch.int32, dev, stream)
    need = 0 if workspace is not None else vqv_cache_workspace_bytes(pages)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _round_lib().vqv_cache_fork, cache.c, pages.c, _list(parent, "parent", n, dev),
        _list(child, "child", n, dev), n, _list(ok, "ok", n, dev), wp, wn, _stream(stream, dev)))
    return ok


def vqv_cache_compact(cache: PagedCache, seqs: Sequences, keep: torch.Tensor,
                      new_len: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Moves each sequence's kept rows (keep [n_rows] int32, not 0) together,
    on all layers; returns its new lengths [n_seqs] int32. The bytes move as
    they are: a prefix of the rows stays where it is, a row kept behind a
    dropped one keeps a key that was turned for its old place."""
    dev = cache.device
    _same(dev, seqs=seqs)
    if new_len is None:
        new_len = _new(seqs.n_seqs, torch.int32, dev, stream)
    _check(_on_device(
        dev, _round_lib().vqv_cache_compact, cache.c, seqs.c, _list(keep, "keep", seqs.n_rows, dev),
        _list(new_len, "new_len", seqs.n_seqs, dev), _stream(stream, dev)))
    return new_len


def _logits_in(logits, edits: Edits, draft, B: int, T: int, mask) -> tuple:
    dev = _device(logits, "logits")
    if edits.n_seqs != B:
        raise ValueError(f"the edits are of {edits.n_seqs} sequences, the call of {B}")
    if edits.device is not None and edits.device != dev:
        raise ValueError(f"the edits are on {edits.device}, logits on {dev}")
    lp = _take(logits, "logits", (B * T, edits.vocab), torch.float32, dev)
    dp = None
    if draft is not None and T > 1:
        dp = _take(draft, "draft", (B, T - 1), torch.int32, dev)
    return dev, lp, dp, _take(mask, "mask", (B * T, edits.words), torch.int32, dev)


def vqv_logits_edit(logits: torch.Tensor, edits: Edits, draft: torch.Tensor | None, B: int, T: int,
                    mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Edited logits [B*T, vocab] fp32 (out may be logits itself); the drafts
    [B, T-1] int32 count as fed at rows 1..T-1; mask [B*T, ceil(vocab/32)]
    int32 bits of the allowed tokens."""
    dev, lp, dp, mp = _logits_in(logits, edits, draft, B, T, mask)
    if out is None:
        out = _new(logits.shape, torch.float32, dev, stream)
    op = _take(out, "out", (B * T, edits.vocab), torch.float32, dev)
    _check(_on_device(
        dev, _round_lib().vqv_logits_edit, lp, edits.c, dp, T, mp, op, _stream(stream, dev)))
    return out


def vqv_logits_verify(logits: torch.Tensor, edits: Edits, draft: torch.Tensor | None, B: int,
                      T: int, mask: torch.Tensor | None = None,
                      draft_len: torch.Tensor | None = None,
                      argmax: torch.Tensor | None = None, accept_len: torch.Tensor | None = None,
                      margin: torch.Tensor | None = None, want_margin: bool = True,
                      workspace: torch.Tensor | None = None, stream=None):
    """(argmax [B*T] int32, accept_len [B] int32, margin [B*T] fp32 or None) of
    the edited logits, which are not written."""
    dev, lp, dp, mp = _logits_in(logits, edits, draft, B, T, mask)
    if argmax is None:
        argmax = _new(B * T, torch.int32, dev, stream)
    if accept_len is None:
        accept_len = _new(B, torch.int32, dev, stream)
    if margin is None and want_margin:
        margin = _new(B * T, torch.float32, dev, stream)
    need = 0 if workspace is not None else vqv_verify_workspace_bytes(B, T, edits.vocab)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _round_lib().vqv_logits_verify, lp, edits.c, dp,
        _take(draft_len, "draft_len", (B,), torch.int32, dev), T, mp,
        _take(argmax, "argmax", (B * T,), torch.int32, dev),
        _take(accept_len, "accept_len", (B,), torch.int32, dev),
        _take(margin, "margin", (B * T,), torch.float32, dev), wp, wn, _stream(stream, dev)))
    return argmax, accept_len, margin
