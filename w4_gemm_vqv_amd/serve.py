"""Binding of libvqv's operators for batches of many requests
(include/vqv_serve.h): a paged cache held in 4 bits with the append and the
attention that read it, verification by sampling, and low-rank adapters.

As in round.py, classes hold a call's tensors and the struct that the library
reads, and functions carry the C names and only marshal arguments; every
tensor's device, type, size and layout is checked here. Calls go to the current
stream unless `stream` names another.
"""

from __future__ import annotations

import ctypes

import torch

from .round import (_DTYPES, PagedCache, Rope, Sequences, _check, _device, _new, _Rope, _rows,
                    _same, _scratch, _Seqs, _stream, _take)
from .vqv import _on_device
from .vqv import lib as _load

SERVE_EXPORTS = ("vqv_q4_record_bytes", "vqv_rope_append_q4", "vqv_cache_q4_read",
                 "vqv_paged_attn_q4_workspace_bytes", "vqv_paged_attn_q4_type_workspace_bytes",
                 "vqv_paged_attn_q4", "vqv_verify_sampled_workspace_bytes", "vqv_verify_sampled",
                 "vqv_lora_add_workspace_bytes", "vqv_lora_add")

_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


class _CacheQ4(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("layers", _i), ("pages", _i), ("page_size", _i),
                ("kv_heads", _i), ("dim", _i), ("reserved", _i), ("layer_stride", _i64),
                ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64)]


class _Adapters(ctypes.Structure):
    _fields_ = [("a", _vp), ("b", _vp), ("scale", _vp), ("ranks", _vp), ("n", _i), ("rank", _i),
                ("K", _i), ("N", _i), ("dtype", _i), ("reserved", _i)]


_lib = None


def _serve_lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _load()
        p = ctypes.POINTER
        cache, seqs, rope, ad = p(_CacheQ4), p(_Seqs), p(_Rope), p(_Adapters)
        f32 = ctypes.c_float
        for name, res, args in (
                ("vqv_q4_record_bytes", _sz, [_i]),
                ("vqv_rope_append_q4", _i, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i,
                                            _i, cache, _i, seqs, rope, _vp, _i, _vp]),
                ("vqv_cache_q4_read", _i, [cache, _i, seqs, _vp, _vp, _i, _vp]),
                ("vqv_paged_attn_q4_workspace_bytes", _sz, [cache, seqs, _i, _i, _i]),
                ("vqv_paged_attn_q4_type_workspace_bytes", _sz, [cache, seqs, _i, _i, _i, _i]),
                ("vqv_paged_attn_q4", _i, [_vp, _i, cache, _i, seqs, _i, f32, _i, _i, _vp, _vp,
                                           _sz, _vp]),
                ("vqv_verify_sampled_workspace_bytes", _sz, [_i, _i, _i]),
                ("vqv_verify_sampled", _i, [_vp] * 6 + [_i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
                ("vqv_lora_add_workspace_bytes", _sz, [ad, _i]),
                ("vqv_lora_add", _i, [_vp, _i, ad, _vp, _i, _vp, _i64, _vp, _i64, _vp, _sz,
                                      _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def vqv_q4_record_bytes(dim: int) -> int:
    """Bytes of a token's record for one key head, 0 for a dim that is not supported."""
    return _serve_lib().vqv_q4_record_bytes(dim)


class PagedCacheQ4:
    """Keys and values of heads of `dim` values in 4 bits: uint8 records
    [layers, pages, page size, kv heads, vqv_q4_record_bytes(dim)] (views of any
    order with a dense last dimension, the same strides). `records` is a
    PagedCache over the same memory, for the calls that move pages and rows
    (vqv_cache_copy, vqv_cache_fork, vqv_cache_compact)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, dim: int):
        size = vqv_q4_record_bytes(dim)
        if not size:
            raise ValueError(f"unsupported dim {dim}")
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.shape[4] != size:
            raise ValueError(f"k and v must be [layers, pages, page size, kv heads, {size}] with "
                             "the same strides")
        if k.dtype != torch.uint8 or v.dtype != torch.uint8:
            raise ValueError("k and v must be uint8")
        if k.stride(4) != 1:
            raise ValueError("k and v must be dense in their last dimension")
        self.device = _device(k, "k")
        if v.device != self.device:
            raise ValueError(f"v is on {v.device}, k on {self.device}")
        self.k, self.v, self.dim = k, v, dim
        self.layers, self.pages, self.page_size, self.kv_heads, _ = k.shape
        # A dimension of one has no stride to speak of.
        st = [s if n > 1 else 0 for s, n in zip(k.stride(), k.shape)]
        self.c = _CacheQ4(k.data_ptr(), v.data_ptr(), *k.shape[:4], dim, 0, *st[:4])
        self._records = None

    @property
    def records(self) -> PagedCache:
        if self._records is None:
            if any(n > 1 and s % 2 for s, n in zip(self.k.stride()[:4], self.k.shape)):
                raise ValueError("the records' strides must be multiples of 16 bytes")
            self._records = PagedCache(self.k.view(torch.bfloat16), self.v.view(torch.bfloat16))
        return self._records


def vqv_rope_append_q4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedCacheQ4,
                       seqs: Sequences, rope: Rope, layer: int = 0,
                       q_out: torch.Tensor | None = None, q_dtype: torch.dtype = torch.bfloat16,
                       stream=None) -> torch.Tensor:
    """vqv_rope_append into a 4-bit cache. The rotated queries are of q_out's
    type, or of q_dtype (bf16 or fp16) where it is made here."""
    dev, n = cache.device, seqs.n_rows
    _same(dev, seqs=seqs)
    if q.dim() != 3 or q.dtype not in _DTYPES:
        raise ValueError("q must be [n_rows, heads, dim] in bf16, fp16 or fp32")
    heads = q.shape[1]
    ins = (*_rows(q, "q", (n, heads, cache.dim), q.dtype, dev),
           *_rows(k, "k", (n, cache.kv_heads, cache.dim), q.dtype, dev),
           *_rows(v, "v", (n, cache.kv_heads, cache.dim), q.dtype, dev))
    q_dtype = q_dtype if q_out is None else q_out.dtype
    if q_dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q_out must be bf16 or fp16, not {q_dtype}")
    if q_out is None:
        q_out = _new((n, heads, cache.dim), q_dtype, dev, stream)
    out = _take(q_out, "q_out", (n, heads, cache.dim), q_dtype, dev)
    _check(_on_device(
        dev, _serve_lib().vqv_rope_append_q4, *ins, _DTYPES[q.dtype], heads, cache.c, layer, seqs.c,
        rope.c, out, _DTYPES[q_dtype], _stream(stream, dev)))
    return q_out


def vqv_cache_q4_read(cache: PagedCacheQ4, seqs: Sequences, layer: int = 0,
                      k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                      dtype: torch.dtype = torch.float32, stream=None, *, want_k: bool = True,
                      want_v: bool = True):
    """(k, v) [n_rows, kv heads, dim]: the sequences' new rows as the cache
    holds them, in the outputs' type or `dtype`; None for one that is neither given
    nor wanted. Rows that no sequence holds are left as they were."""
    dev = cache.device
    _same(dev, seqs=seqs)
    given = [t for t in (k_out, v_out) if t is not None]
    dtype = given[0].dtype if given else dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported type {dtype}")
    shape = (seqs.n_rows, cache.kv_heads, cache.dim)

    def made(t, want):
        return _new(shape, dtype, dev, stream) if t is None and want else t

    k_out, v_out = made(k_out, want_k), made(v_out, want_v)
    kp, vp = _take(k_out, "k_out", shape, dtype, dev), _take(v_out, "v_out", shape, dtype, dev)
    _check(_on_device(
        dev, _serve_lib().vqv_cache_q4_read, cache.c, layer, seqs.c, kp, vp, _DTYPES[dtype],
        _stream(stream, dev)))
    return k_out, v_out


def vqv_paged_attn_q4_workspace_bytes(cache: PagedCacheQ4, seqs: Sequences, heads: int,
                                      window: int = 0, sinks: int = 0,
                                      dtype: torch.dtype | None = None) -> int:
    """Bytes that a call needs, of queries of `dtype` or (None) of either type."""
    if dtype is not None:
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"queries are bf16 or fp16, not {dtype}")
        return _serve_lib().vqv_paged_attn_q4_type_workspace_bytes(
            cache.c, seqs.c, _DTYPES[dtype], heads, window, sinks)
    return _serve_lib().vqv_paged_attn_q4_workspace_bytes(cache.c, seqs.c, heads, window, sinks)


def vqv_paged_attn_q4(q: torch.Tensor, cache: PagedCacheQ4, seqs: Sequences, scale: float,
                      window: int = 0, sinks: int = 0, layer: int = 0,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """vqv_paged_attn over a 4-bit cache: q [n_rows, heads, dim] in bf16 or
    fp16, and the output in its type."""
    dev = cache.device
    _same(dev, seqs=seqs)
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q must be [n_rows, heads, dim] in bf16 or fp16")
    heads = q.shape[1]
    shape = (seqs.n_rows, heads, cache.dim)
    qp = _take(q, "q", shape, q.dtype, dev)
    if out is None:
        out = _new(shape, q.dtype, dev, stream)
    op = _take(out, "out", shape, q.dtype, dev)
    need = 0 if workspace is not None else vqv_paged_attn_q4_workspace_bytes(
        cache, seqs, heads, window, sinks, q.dtype)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _serve_lib().vqv_paged_attn_q4, qp, _DTYPES[q.dtype], cache.c, layer, seqs.c, heads,
        scale, window, sinks, op, wp, wn, _stream(stream, dev)))
    return out


def vqv_verify_sampled_workspace_bytes(B: int, T: int, N: int) -> int:
    return _serve_lib().vqv_verify_sampled_workspace_bytes(B, T, N)


def vqv_verify_sampled(logits: torch.Tensor, draft: torch.Tensor | None, uniform: torch.Tensor,
                       B: int, T: int, draft_probs: torch.Tensor | None = None,
                       temperature: torch.Tensor | None = None,
                       draft_len: torch.Tensor | None = None, token: torch.Tensor | None = None,
                       accept_len: torch.Tensor | None = None,
                       logprob: torch.Tensor | None = None, want_logprob: bool = True,
                       workspace: torch.Tensor | None = None, stream=None):
    """(token [B] int32, accept_len [B] int32, logprob [B, T] fp32 or None) of
    fp32 logits [B*T, N], drafts [B, T-1] int32 with the drafter's
    probabilities [B, T-1, N] fp32 (None: the drafts were not drawn) and random
    numbers [B, T] fp32 in [0, 1): the drafts that are accepted, and the token
    drawn behind them. temperature [B] fp32 (None: 1; 0: greedy)."""
    dev, f32, i32 = _device(logits, "logits"), torch.float32, torch.int32
    N = logits.shape[-1]
    lp = _take(logits, "logits", (B * T, N), f32, dev)
    dp = qp = None
    if T > 1:
        if draft is None:
            raise ValueError("draft is needed when T > 1")
        dp = _take(draft, "draft", (B, T - 1), i32, dev)
        qp = _take(draft_probs, "draft_probs", (B, T - 1, N), f32, dev)
    if token is None:
        token = _new(B, i32, dev, stream)
    if accept_len is None:
        accept_len = _new(B, i32, dev, stream)
    if logprob is None and want_logprob:
        logprob = _new((B, T), f32, dev, stream)
    need = 0 if workspace is not None else vqv_verify_sampled_workspace_bytes(B, T, N)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _serve_lib().vqv_verify_sampled, lp, dp, qp,
        _take(draft_len, "draft_len", (B,), i32, dev),
        _take(temperature, "temperature", (B,), f32, dev),
        _take(uniform, "uniform", (B, T), f32, dev), B, T, N, _take(token, "token", (B,), i32, dev),
        _take(accept_len, "accept_len", (B,), i32, dev),
        _take(logprob, "logprob", (B, T), f32, dev), wp, wn, _stream(stream, dev)))
    return token, accept_len, logprob


class Adapters:
    """Low-rank adapters of one projection: a [n, rank, K] and b [n, N, rank]
    in bf16 or fp16, scale [n] fp32, and ranks [n] int32 where adapters use
    fewer than `rank` of their ranks."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor,
                 ranks: torch.Tensor | None = None):
        dev = self.device = _device(a, "a")
        if a.dim() != 3 or b.dim() != 3 or a.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("a must be [n, rank, K] and b [n, N, rank], in bf16 or fp16")
        self.n, self.rank, self.K = a.shape
        self.N, self.dtype = b.shape[1], a.dtype
        self.tensors = (a, b, scale, ranks)
        self.c = _Adapters(_take(a, "a", (self.n, self.rank, self.K), self.dtype, dev),
                           _take(b, "b", (self.n, self.N, self.rank), self.dtype, dev),
                           _take(scale, "scale", (self.n,), torch.float32, dev),
                           _take(ranks, "ranks", (self.n,), torch.int32, dev),
                           self.n, self.rank, self.K, self.N, _DTYPES[self.dtype], 0)


def vqv_lora_add_workspace_bytes(adapters: Adapters, M: int) -> int:
    return _serve_lib().vqv_lora_add_workspace_bytes(adapters.c, M)


def _columns(t: torch.Tensor, name: str, shape: tuple, device) -> tuple:
    """Pointer and row stride of fp32 rows, dense in themselves."""
    if t.shape != shape or t.dtype != torch.float32 or t.device != device \
            or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a torch.float32 tensor of shape {list(shape)} on {device} "
                         f"with dense rows, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def vqv_lora_add(x: torch.Tensor, adapters: Adapters, which: torch.Tensor, y: torch.Tensor,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y [M, N] fp32 plus each row's adapter (which [M] int32; none where it is
    outside [0, n)) applied to x [M, K]; out may be y itself. y and out may be
    columns of a wider tensor."""
    dev, M = adapters.device, which.numel()
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported activation dtype {x.dtype}")
    xp = _take(x, "x", (M, adapters.K), x.dtype, dev)
    shape = (M, adapters.N)
    if out is None:
        out = _new(shape, torch.float32, dev, stream)
    need = 0 if workspace is not None else vqv_lora_add_workspace_bytes(adapters, M)
    workspace, wp, wn = _scratch(workspace, need, dev, stream)
    _check(_on_device(
        dev, _serve_lib().vqv_lora_add, xp, _DTYPES[x.dtype], adapters.c,
        _take(which, "which", (M,), torch.int32, dev), M, *_columns(y, "y", shape, dev),
        *_columns(out, "out", shape, dev), wp, wn, _stream(stream, dev)))
    return out
