"""Batched speculative-decoding verify step on GB300 (sm_103a).

Python binding of the C ABI in ``include/specv.h``: the functions below keep
the C names and only marshal arguments (torch tensors for device memory and
the current CUDA stream); every step of the verify path runs in the
library's CUDA kernels.  There is no CPU fallback: if ``libspecv.so`` cannot
be loaded, or no sm_103 device is present, the calls raise.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (ST_ACCEPTED, ST_BLOCK, ST_ERROR_MASK, ST_FILTER, ST_LENGTH, ST_NO_ROOM, ST_NONFINITE, ST_PARENT, ST_PATH,
                   ST_Q_INVALID, ST_TEMPERATURE, ST_TIMEOUT, ST_TOKEN_RANGE, ST_UNIFORM_RANGE, ST_ZERO_RESIDUAL,
                   SPECV_BF16, SPECV_F32)

__all__ = [
    "SpecvError",
    "Handle",
    "specv_create",
    "specv_destroy",
    "specv_verify_sample",
    "specv_verify_greedy",
    "specv_verify_sample_host",
    "specv_cache_append",
    "specv_tree_attention",
    "specv_tree_attention_workspace",
    "specv_cache_compact",
    "specv_prefix_attention",
    "specv_prefix_attention_workspace",
    "specv_cache_append_norm",
    "specv_attention_mass",
    "specv_cache_evict",
    "specv_plan_cluster",
    "specv_test_withhold_stage",
    "specv_launch_count",
    "ST_ERROR_MASK",
    "ST_NONFINITE",
    "ST_TOKEN_RANGE",
    "ST_UNIFORM_RANGE",
    "ST_TEMPERATURE",
    "ST_ZERO_RESIDUAL",
    "ST_Q_INVALID",
    "ST_TIMEOUT",
    "ST_ACCEPTED",
    "ST_NO_ROOM",
    "ST_PARENT",
    "ST_FILTER",
    "ST_LENGTH",
    "ST_BLOCK",
    "ST_PATH",
]


class SpecvError(RuntimeError):
    def __init__(self, status, what=""):
        lib = _lib.load()
        msg = lib.specv_status_string(status).decode()
        if status == _lib.SPECV_ERR_CUDA or status == _lib.SPECV_ERR_UNSUPPORTED:
            msg += ": " + lib.specv_last_cuda_error().decode()
        super().__init__(f"{what}: {msg}" if what else msg)
        self.status = status


def _check(status, what):
    if status != _lib.SPECV_OK:
        raise SpecvError(status, what)


class Handle:
    """An open ``specv_handle`` (closed by ``specv_destroy`` or on garbage
    collection)."""

    def __init__(self, ptr, device, max_batch, max_k, vocab):
        self.ptr = ptr
        self.device = device
        self.max_batch = max_batch
        self.max_k = max_k
        self.vocab = vocab
        self._workspace = {}  # bytes of workspace by the sizes of a call

    def __del__(self):
        try:
            specv_destroy(self)
        except Exception:
            pass


def specv_create(device=0, max_batch=1 << 20, max_k=31, vocab=262144) -> Handle:
    lib = _lib.load()
    h = ctypes.c_void_p()
    _check(lib.specv_create(ctypes.byref(h), int(device), int(max_batch), int(max_k), int(vocab)), "specv_create")
    return Handle(h.value, device, max_batch, max_k, vocab)


def specv_destroy(h: Handle) -> None:
    if h is not None and h.ptr:
        _lib.load().specv_destroy(h.ptr)
        h.ptr = None


def _torch():
    import torch

    return torch


def _dev(t, dtype, name, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _logits_dtype(logits):
    torch = _torch()
    if logits.dtype == torch.bfloat16:
        return SPECV_BF16
    if logits.dtype == torch.float32:
        return SPECV_F32
    raise TypeError("target logits must be bfloat16 or float32")


def _stream_ptr(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def specv_verify_sample(h: Handle, logits, q, x, u, T, *, debug=False, out=None, stream=None):
    """Verify a batch (asynchronous on ``stream``, default: torch's current
    stream).  logits [B,k+1,V] bf16/fp32, q [B,k,V] fp32 or None (one-hot
    drafts: q is the point mass at each draft token), x [B,k] int32,
    u [B,k+1,2] fp32, T [B] fp32 (0 = greedy row), all CUDA tensors.
    Returns a dict of CUDA tensors: num_accepted [B], out_tokens [B,k+1],
    row_status [B] and, with ``debug``, p_at_draft, q_at_draft, row_max,
    row_sumexp, residual_mass.  ``out`` may supply preallocated outputs."""
    torch = _torch()
    B, k1, V = logits.shape
    k = k1 - 1
    dt = _logits_dtype(logits)
    _dev(logits, logits.dtype, "logits")
    pq = None if q is None else _dev(q, torch.float32, "q", (B, k, V))
    px = _dev(x, torch.int32, "x", (B, k))
    pu = _dev(u, torch.float32, "u", (B, k + 1, 2))
    pt = _dev(T, torch.float32, "T", (B,))
    dev = logits.device
    if out is None:
        out = {
            "num_accepted": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, k + 1), dtype=torch.int32, device=dev),
            "row_status": torch.empty(B, dtype=torch.int32, device=dev),
        }
    dbg_struct = None
    if debug:
        for name, shape in (("p_at_draft", (B, k)), ("q_at_draft", (B, k)), ("row_max", (B, k + 1)),
                            ("row_sumexp", (B, k + 1)), ("residual_mass", (B,))):
            if name not in out:
                out[name] = torch.empty(shape, dtype=torch.float32, device=dev)
        dbg_struct = _lib.SpecvDebug(out["p_at_draft"].data_ptr(), out["q_at_draft"].data_ptr(),
                                     out["row_max"].data_ptr(), out["row_sumexp"].data_ptr(),
                                     out["residual_mass"].data_ptr())
    lib = _lib.load()
    st = lib.specv_verify_sample(
        h.ptr, dt, ctypes.c_void_p(logits.data_ptr()), ctypes.c_void_p(pq), ctypes.c_void_p(px),
        ctypes.c_void_p(pu), ctypes.c_void_p(pt), B, k, V, ctypes.c_void_p(out["num_accepted"].data_ptr()),
        ctypes.c_void_p(out["out_tokens"].data_ptr()), ctypes.c_void_p(out["row_status"].data_ptr()),
        ctypes.byref(dbg_struct) if dbg_struct is not None else None, _stream_ptr(stream))
    _check(st, "specv_verify_sample")
    return out


def specv_verify_greedy(h: Handle, logits, x, *, out=None, stream=None):
    """Greedy verification of every row: logits [B,k+1,V], x [B,k] int32."""
    torch = _torch()
    B, k1, V = logits.shape
    k = k1 - 1
    dt = _logits_dtype(logits)
    _dev(logits, logits.dtype, "logits")
    px = _dev(x, torch.int32, "x", (B, k))
    dev = logits.device
    if out is None:
        out = {
            "num_accepted": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, k + 1), dtype=torch.int32, device=dev),
            "row_status": torch.empty(B, dtype=torch.int32, device=dev),
        }
    st = _lib.load().specv_verify_greedy(
        h.ptr, dt, ctypes.c_void_p(logits.data_ptr()), ctypes.c_void_p(px), B, k, V,
        ctypes.c_void_p(out["num_accepted"].data_ptr()), ctypes.c_void_p(out["out_tokens"].data_ptr()),
        ctypes.c_void_p(out["row_status"].data_ptr()), _stream_ptr(stream))
    _check(st, "specv_verify_greedy")
    return out


def specv_verify_sample_filtered(h: Handle, logits, q, x, u, T, top_k, top_p, *, out=None, stream=None):
    """Sampled verification with top-k / top-p applied to the target rows:
    as specv_verify_sample (q may be None: one-hot drafts, or a pinned CPU
    tensor, read in place), plus top_k [B] int32 in 1..4096 and top_p [B]
    fp32 in (0, 1], CUDA tensors."""
    torch = _torch()
    B, k1, V = logits.shape
    k = k1 - 1
    dt = _logits_dtype(logits)
    _dev(logits, logits.dtype, "logits")
    if q is not None and not q.is_cuda:
        if not q.is_pinned() or q.dtype != torch.float32 or not q.is_contiguous() or tuple(q.shape) != (B, k, V):
            raise ValueError("a CPU q must be a pinned, contiguous float32 tensor of shape [B, k, V]")
        pq = q.data_ptr()
    else:
        pq = None if q is None else _dev(q, torch.float32, "q", (B, k, V))
    px = _dev(x, torch.int32, "x", (B, k))
    pu = _dev(u, torch.float32, "u", (B, k + 1, 2))
    pt = _dev(T, torch.float32, "T", (B,))
    pk = _dev(top_k, torch.int32, "top_k", (B,))
    pp = _dev(top_p, torch.float32, "top_p", (B,))
    dev = logits.device
    if out is None:
        out = {
            "num_accepted": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, k + 1), dtype=torch.int32, device=dev),
            "row_status": torch.empty(B, dtype=torch.int32, device=dev),
        }
    st = _lib.load().specv_verify_sample_filtered(
        h.ptr, dt, ctypes.c_void_p(logits.data_ptr()), ctypes.c_void_p(pq), ctypes.c_void_p(px), ctypes.c_void_p(pu),
        ctypes.c_void_p(pt), ctypes.c_void_p(pk), ctypes.c_void_p(pp), B, k, V,
        ctypes.c_void_p(out["num_accepted"].data_ptr()), ctypes.c_void_p(out["out_tokens"].data_ptr()),
        ctypes.c_void_p(out["row_status"].data_ptr()), _stream_ptr(stream))
    _check(st, "specv_verify_sample_filtered")
    return out


def specv_verify_tree_greedy(h: Handle, logits, tokens, parents, *, out=None, stream=None):
    """Greedy verification of draft trees: logits [B, M+1, V] (row 0 after
    the prefix, row 1+i after node i), tokens and parents [B, M] int32
    (parent -1: a child of the prefix).  Returns num_accepted [B],
    out_tokens [B, M+1], path [B, M], row_status [B]."""
    torch = _torch()
    B, m1, V = logits.shape
    M = m1 - 1
    dt = _logits_dtype(logits)
    _dev(logits, logits.dtype, "logits")
    pt = _dev(tokens, torch.int32, "tokens", (B, M))
    pp = _dev(parents, torch.int32, "parents", (B, M))
    dev = logits.device
    if out is None:
        out = {
            "num_accepted": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, M + 1), dtype=torch.int32, device=dev),
            "path": torch.empty((B, M), dtype=torch.int32, device=dev),
            "row_status": torch.empty(B, dtype=torch.int32, device=dev),
        }
    st = _lib.load().specv_verify_tree_greedy(
        h.ptr, dt, ctypes.c_void_p(logits.data_ptr()), ctypes.c_void_p(pt), ctypes.c_void_p(pp), B, M, V,
        ctypes.c_void_p(out["num_accepted"].data_ptr()), ctypes.c_void_p(out["out_tokens"].data_ptr()),
        ctypes.c_void_p(out["path"].data_ptr()), ctypes.c_void_p(out["row_status"].data_ptr()), _stream_ptr(stream))
    _check(st, "specv_verify_tree_greedy")
    return out


def specv_verify_sample_host(h: Handle, logits, q, x, u, T, *, out=None, stream=None):
    """Host-buffer verification: CPU tensors in (pinned memory copies
    fastest), CPU tensors out; the call copies, verifies and synchronises.
    ``logits`` is a bfloat16 or float32 CPU tensor."""
    torch = _torch()
    B, k1, V = logits.shape
    k = k1 - 1
    dt = _logits_dtype(logits)
    for t, name in ((logits, "logits"), (q, "q"), (x, "x"), (u, "u"), (T, "T")):
        if t is None and name == "q":
            continue  # one-hot drafts
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    if out is None:
        pin = logits.is_pinned()
        out = {
            "num_accepted": torch.empty(B, dtype=torch.int32, pin_memory=pin),
            "out_tokens": torch.empty((B, k + 1), dtype=torch.int32, pin_memory=pin),
            "row_status": torch.empty(B, dtype=torch.int32, pin_memory=pin),
        }
    st = _lib.load().specv_verify_sample_host(
        h.ptr, dt, ctypes.c_void_p(logits.data_ptr()), ctypes.c_void_p(None if q is None else q.data_ptr()),
        ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(u.data_ptr()), ctypes.c_void_p(T.data_ptr()), B, k, V,
        ctypes.c_void_p(out["num_accepted"].data_ptr()), ctypes.c_void_p(out["out_tokens"].data_ptr()),
        ctypes.c_void_p(out["row_status"].data_ptr()), _stream_ptr(stream))
    _check(st, "specv_verify_sample_host")
    return out


def specv_rollback(h: Handle, num_accepted, k, seq_lens, block_tables, num_blocks, block_size, free_list,
                   free_count, *, row_status=None, stream=None):
    """Paged KV-cache rollback after verification, in place on CUDA int32
    tensors: num_accepted [B], seq_lens [B], block_tables [B, max_blocks],
    num_blocks [B], free_list [capacity], free_count [1]; row_status [B]
    (optional) receives 0 / 128 (invalid row) / 256 (no room)."""
    torch = _torch()
    B = num_accepted.shape[0]
    mb = block_tables.shape[1] if block_tables.dim() == 2 else 0
    ptrs = []
    for t, name, shape in ((num_accepted, "num_accepted", (B,)), (seq_lens, "seq_lens", (B,)),
                           (block_tables, "block_tables", (B, mb)), (num_blocks, "num_blocks", (B,)),
                           (free_list, "free_list", None), (free_count, "free_count", (1,))):
        ptrs.append(_dev(t, torch.int32, name, shape))
    prs = None if row_status is None else _dev(row_status, torch.int32, "row_status", (B,))
    st = _lib.load().specv_rollback(
        h.ptr, ctypes.c_void_p(ptrs[0]), B, int(k), ctypes.c_void_p(ptrs[1]), ctypes.c_void_p(ptrs[2]), mb,
        ctypes.c_void_p(ptrs[3]), int(block_size), ctypes.c_void_p(ptrs[4]), free_list.numel(),
        ctypes.c_void_p(ptrs[5]), ctypes.c_void_p(prs), _stream_ptr(stream))
    _check(st, "specv_rollback")


# ------------------------------------------------------------------ paged KV cache
# A serving loop makes these calls once a layer: what a call checks is a few
# attribute reads a tensor, and what is wrong is found out only if they fail.
_cache_dtypes = None


def _cache_setup():
    """torch's names that every call needs, looked up once."""
    global _cache_dtypes, _i32, _f32, _raw_stream
    import torch

    _i32, _f32 = torch.int32, torch.float32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _cache_dtypes = {torch.bfloat16: SPECV_BF16, torch.float32: SPECV_F32}


def _on(h, t, dtype, name, shape=None):
    """Pointer of a contiguous CUDA tensor on the handle's device."""
    try:
        if (t.dtype is dtype and t.get_device() == h.device and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}, the handle on cuda:{h.device}")


def _inner(t, n):
    """Whether the last n dimensions of ``t`` lie behind one another without
    gaps (dimensions of size one may have any stride); their size."""
    want = 1
    for size, stride in zip(reversed(t.shape[-n:]), reversed(t.stride()[-n:])):
        if size != 1 and stride != want:
            return None
        want *= size
    return want


def _strides_match(a, b):
    return all(x == y for x, y, n in zip(a.stride(), b.stride(), a.shape) if n > 1)


def _kv_cache(h, k_cache, v_cache, block_tables, seq_lens, layered=False):
    """The descriptor of a cache; with ``layered`` the pools may have a
    leading dimension of layers.  Returns (descriptor, layers, layer_stride)."""
    if _cache_dtypes is None:
        _cache_setup()
    try:
        dt = _cache_dtypes[k_cache.dtype]
    except (AttributeError, KeyError):
        raise TypeError("the cache pools must be bfloat16 or float32 tensors") from None
    if k_cache.get_device() != h.device or v_cache.get_device() != h.device:
        raise ValueError(f"k_cache and v_cache must be on the handle's device, cuda:{h.device}")
    if v_cache.dtype is not k_cache.dtype:
        raise TypeError(f"v_cache must be {k_cache.dtype}, got {v_cache.dtype}")
    shape = k_cache.shape
    if len(shape) != 4 and not (layered and len(shape) == 5):
        raise ValueError("the cache pools have the shape "
                         + ("[layers, blocks, heads, block_size, head_dim] or " if layered else "")
                         + "[blocks, heads, block_size, head_dim]")
    if v_cache.shape != shape:
        raise ValueError(f"v_cache has shape {tuple(v_cache.shape)}, expected {tuple(shape)}")
    blocks, heads, block_size, head_dim = shape[-4:]
    inner = heads * block_size * head_dim
    layers = shape[0] if len(shape) == 5 else 1
    block_stride, layer_stride = inner, blocks * inner
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        if _inner(k_cache, 3) is None or _inner(v_cache, 3) is None:
            raise ValueError("the cache pools must be contiguous inside a block")
        if not _strides_match(k_cache, v_cache):
            raise ValueError("k_cache and v_cache must have the same strides")
        block_stride = k_cache.stride(-4) if blocks > 1 else inner
        layer_stride = k_cache.stride(0) if layers > 1 else 0
    tables = _on(h, block_tables, _i32, "block_tables")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must have the shape [B, max_blocks]")
    batch, max_blocks = block_tables.shape
    lens = _on(h, seq_lens, _i32, "seq_lens", (batch,))
    c = _lib.SpecvKvCache(dt, heads, head_dim, block_size, max_blocks, k_cache.data_ptr(), v_cache.data_ptr(), blocks,
                          block_stride, tables, lens)
    return c, layers, layer_stride


def _token_rows(h, t, name, like, shape):
    """Pointer and row stride of a [B, rows, heads, head_dim] tensor whose
    rows are evenly spaced (a slice of a fused projection will do)."""
    if t.get_device() != h.device:
        raise ValueError(f"{name} must be on the handle's device, cuda:{h.device}")
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    B, rows, heads, dim = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * dim
    s = t.stride()
    stride = s[1] if rows > 1 else s[0] if B > 1 else heads * dim
    if not (s[3] == 1 and (s[2] == dim or heads == 1)) or (B > 1 and rows > 1 and s[0] != rows * stride):
        raise ValueError(f"{name} must have contiguous heads and evenly spaced rows")
    return t.data_ptr(), stride


def _stream_of(h, stream):
    return _raw_stream(h.device) if stream is None else stream.cuda_stream


def _empty(h, shape, dtype, stream, zero=False):
    """A tensor for a call on ``stream``: allocated there, so that its memory
    is not handed on before the call has run."""
    torch = _torch()
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=torch.device("cuda", h.device))
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=torch.device("cuda", h.device))


def _append_args(h, k_cache, v_cache, block_tables, seq_lens, k, v, q, inv_freq, parents, row_counts, out, stream):
    """What the two appends have in common: the arguments up to v's stride, the
    rotation's, those from parents to rows, and the outputs'."""
    c, _, _ = _kv_cache(h, k_cache, v_cache, block_tables, seq_lens)
    if k.dim() != 4:
        raise ValueError("k must have the shape [B, rows, kv_heads, head_dim]")
    B, rows = k.shape[:2]
    if B != block_tables.shape[0]:
        raise ValueError(f"k holds {B} sequences, block_tables {block_tables.shape[0]}")
    pk, k_stride = _token_rows(h, k, "k", k_cache, (B, rows, c.kv_heads, c.head_dim))
    pv, v_stride = _token_rows(h, v, "v", k_cache, (B, rows, c.kv_heads, c.head_dim))
    pf, rot = None, 0
    if inv_freq is not None:
        pf = _on(h, inv_freq, _f32, "inv_freq")
        rot = 2 * inv_freq.numel()
    pp = None if parents is None else _on(h, parents, _i32, "parents", (B, rows - 1))
    pc = None if row_counts is None else _on(h, row_counts, _i32, "row_counts", (B,))
    out = {} if out is None else out
    pq, q_stride, q_heads, po = None, 0, 0, None
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must have the shape [B, rows, q_heads, head_dim]")
        q_heads = q.shape[2]
        pq, q_stride = _token_rows(h, q, "q", k_cache, (B, rows, q_heads, c.head_dim))
        if "q_out" not in out:
            out["q_out"] = _empty(h, (B, rows, q_heads, c.head_dim), k_cache.dtype, stream)
        po = _on(h, out["q_out"], k_cache.dtype, "q_out", (B, rows, q_heads, c.head_dim))
    if "row_status" not in out:
        out["row_status"] = _empty(h, (B,), _i32, stream)
    ps = _on(h, out["row_status"], _i32, "row_status", (B,))
    return (h.ptr, c, pq, q_stride, q_heads, pk, k_stride, pv, v_stride), (pf, rot), (pp, pc, B, rows), (po, ps), out


def specv_cache_append(h: Handle, k_cache, v_cache, block_tables, seq_lens, k, v, *, q=None, inv_freq=None,
                       interleaved=False, parents=None, row_counts=None, out=None, stream=None):
    """Append the keys and values of a pass to a paged cache, in place, and
    rotate queries and keys by their positions on the way.  k_cache, v_cache
    [blocks, kv_heads, block_size, head_dim] bf16 or fp32; block_tables
    [B, max_blocks], seq_lens [B] int32, the lengths with the pass's rows;
    k, v [B, rows, kv_heads, head_dim] and q [B, rows, q_heads, head_dim]
    (optional) of the caches' type, rows evenly spaced; inv_freq
    [rot_dim / 2] fp32 (None: no rotation); parents [B, rows - 1] int32
    (None: chains, or prompts); row_counts [B] int32 (None: all rows are
    tokens; counts below ``rows`` are for prompts, as specv_tree_attention and
    specv_cache_compact know none).  Returns a dict: q_out (with q) and row_status [B]; ``out`` may
    supply them."""
    head, turn, rows, to, out = _append_args(h, k_cache, v_cache, block_tables, seq_lens, k, v, q, inv_freq, parents,
                                             row_counts, out, stream)
    st = _lib.load().specv_cache_append(*head, *turn, 1 if interleaved else 0, *rows, *to, _stream_of(h, stream))
    _check(st, "specv_cache_append")
    return out


def specv_cache_append_norm(h: Handle, k_cache, v_cache, block_tables, seq_lens, k, v, *, q=None, q_norm=None,
                            k_norm=None, eps=1e-6, weight_add=0.0, inv_freq=None, interleaved=False, positions=None,
                            pair_axis=None, offsets=None, parents=None, row_counts=None, out=None, stream=None):
    """specv_cache_append for models that norm the heads of queries and keys,
    and for positions on several axes.  q_norm, k_norm [head_dim] of the
    caches' type (None: not normed): a head x becomes x * rsqrt(mean(x^2) +
    eps) * (weight + weight_add) before it turns.  positions [B, rows, axes]
    int32: each row's position on each axis, with pair_axis, bytes (or a
    sequence) of rot_dim / 2 numbers, the axis that turns each pair (None with
    one axis); or offsets [B] int32, added to base + depth.  The rest, and the
    result, as for specv_cache_append."""
    head, turn, rows, to, out = _append_args(h, k_cache, v_cache, block_tables, seq_lens, k, v, q, inv_freq, parents,
                                             row_counts, out, stream)
    norm = places = None
    if q_norm is not None or k_norm is not None:
        shape = k_cache.shape[-1:]
        norm = _lib.SpecvHeadNorm(None if q_norm is None else _on(h, q_norm, k_cache.dtype, "q_norm", shape),
                                  None if k_norm is None else _on(h, k_norm, k_cache.dtype, "k_norm", shape), eps,
                                  weight_add)
    if positions is not None:
        if positions.dim() != 3:
            raise ValueError("positions must have the shape [B, rows, axes]")
        axes = positions.shape[2]
        if axes < 1:
            raise ValueError("positions need an axis")
        pa = None if pair_axis is None else bytes(pair_axis)
        if pa is not None and len(pa) != turn[1] // 2:
            raise ValueError(f"pair_axis has {len(pa)} entries, expected {turn[1] // 2}")
        if offsets is not None or parents is not None:
            raise ValueError("positions go with neither offsets nor parents")
        places = _lib.SpecvPositions(axes, _on(h, positions, _i32, "positions", (*k.shape[:2], axes)), pa, None)
    elif pair_axis is not None:
        raise ValueError("pair_axis needs positions")
    elif offsets is not None:
        places = _lib.SpecvPositions(1, None, None, _on(h, offsets, _i32, "offsets", (k.shape[0],)))
    st = _lib.load().specv_cache_append_norm(*head, norm, *turn, 1 if interleaved else 0, places, *rows, *to,
                                             _stream_of(h, stream))
    _check(st, "specv_cache_append_norm")
    return out


def _attention_args(h, q, k_cache, v_cache, block_tables, seq_lens, parents, scale, lse, out, stream):
    """What the two attentions have in common: the cache's descriptor, the
    sizes that the workspace depends on, the arguments from q to the row
    status, and the outputs."""
    c, _, _ = _kv_cache(h, k_cache, v_cache, block_tables, seq_lens)
    if q.dim() != 4:
        raise ValueError("q must have the shape [B, rows, q_heads, head_dim]")
    B, rows, q_heads = q.shape[:3]
    if B != block_tables.shape[0]:
        raise ValueError(f"q holds {B} sequences, block_tables {block_tables.shape[0]}")
    pq, q_stride = _token_rows(h, q, "q", k_cache, (B, rows, q_heads, c.head_dim))
    pp = None if parents is None else _on(h, parents, _i32, "parents", (B, rows - 1))
    out = {} if out is None else out
    if "out" not in out:
        out["out"] = _empty(h, (B, rows, q_heads, c.head_dim), k_cache.dtype, stream)
    po = _on(h, out["out"], k_cache.dtype, "out", (B, rows, q_heads, c.head_dim))
    if "row_status" not in out:
        out["row_status"] = _empty(h, (B,), _i32, stream)
    ps = _on(h, out["row_status"], _i32, "row_status", (B,))
    pl = None
    if lse:
        if "lse" not in out:
            out["lse"] = _empty(h, (B, rows, q_heads), _f32, stream)
        pl = _on(h, out["lse"], _f32, "lse", (B, rows, q_heads))
    sizes = (c.dtype, c.kv_heads, c.head_dim, q_heads, B, rows)
    return c, sizes, (pq, q_stride, q_heads, pp, B, rows, c.head_dim ** -0.5 if scale is None else scale, po, pl, ps), out


def _workspace_of(h, workspace, need, key, sizes, stream):
    """Pointer and bytes of a call's workspace; without one, new memory of
    as many bytes as ``need`` says for the sizes, asked once."""
    if workspace is None:
        n = h._workspace.get((key, sizes))
        if n is None:
            n = h._workspace[key, sizes] = need(h.ptr, *sizes)
        workspace = _empty(h, (n,), _torch().uint8, stream) if n else None
    if workspace is None:
        return None, 0
    return _on(h, workspace, _torch().uint8, "workspace"), workspace.numel()


def specv_tree_attention(h: Handle, q, k_cache, v_cache, block_tables, seq_lens, *, parents=None, scale=None,
                         lse=False, out=None, workspace=None, stream=None):
    """Attention of a pass's rows over the paged cache they were appended to:
    q [B, rows, q_heads, head_dim], rows evenly spaced, rows <= max_k + 1;
    the caches, block_tables and seq_lens as for specv_cache_append; parents
    [B, rows - 1] int32 (None: chains); scale defaults to head_dim ** -0.5.
    The pass's rows are the last ``rows`` positions of every sequence.  Weights
    of a bf16 cache are rounded to bf16 for the product with the values.
    Returns a dict: out [B, rows, q_heads, head_dim], row_status [B] and,
    with ``lse``, lse [B, rows, q_heads] fp32; ``out`` may supply them.
    ``workspace`` may supply a CUDA uint8 tensor of at least
    specv_tree_attention_workspace bytes that no other call uses meanwhile."""
    c, sizes, args, out = _attention_args(h, q, k_cache, v_cache, block_tables, seq_lens, parents, scale, lse, out, stream)
    lib = _lib.load()
    work = _workspace_of(h, workspace, lib.specv_tree_attention_workspace, "tree", sizes, stream)
    _check(lib.specv_tree_attention(h.ptr, c, *args, *work, _stream_of(h, stream)), "specv_tree_attention")
    return out


def specv_prefix_attention(h: Handle, q, k_cache, v_cache, block_tables, seq_lens, prefix_table, prefix_len, *,
                           parents=None, scale=None, lse=False, out=None, workspace=None, stream=None):
    """specv_tree_attention for a batch whose sequences share a prefix, read
    once for all of them: the first prefix_len positions ([1] int32 on the
    device, a multiple of the block size) are those of prefix_table
    [prefix_blocks] int32, the others each sequence's own, by block_tables
    (whose entries for the prefix are not looked at); seq_lens counts both.
    The rest, and the result, as for specv_tree_attention; ``workspace`` of at
    least specv_prefix_attention_workspace bytes."""
    c, sizes, args, out = _attention_args(h, q, k_cache, v_cache, block_tables, seq_lens, parents, scale, lse, out, stream)
    pt = _on(h, prefix_table, _i32, "prefix_table")
    if prefix_table.dim() != 1:
        raise ValueError("prefix_table must have the shape [prefix_blocks]")
    pn = _on(h, prefix_len, _i32, "prefix_len", (1,))
    lib = _lib.load()
    work = _workspace_of(h, workspace, lib.specv_prefix_attention_workspace, "prefix", sizes, stream)
    _check(lib.specv_prefix_attention(h.ptr, c, pt, prefix_table.shape[0], pn, *args, *work, _stream_of(h, stream)),
           "specv_prefix_attention")
    return out


def specv_prefix_attention_workspace(h: Handle, dtype, kv_heads, head_dim, q_heads, batch, rows) -> int:
    """Bytes of workspace a specv_prefix_attention call of these sizes needs
    (dtype SPECV_BF16 or SPECV_F32)."""
    return int(_lib.load().specv_prefix_attention_workspace(h.ptr, dtype, kv_heads, head_dim, q_heads, batch, rows))


def specv_tree_attention_workspace(h: Handle, dtype, kv_heads, head_dim, q_heads, batch, rows) -> int:
    """Bytes of workspace a specv_tree_attention call of these sizes needs
    (dtype SPECV_BF16 or SPECV_F32)."""
    return int(_lib.load().specv_tree_attention_workspace(h.ptr, dtype, kv_heads, head_dim, q_heads, batch, rows))


def specv_cache_compact(h: Handle, k_cache, v_cache, block_tables, seq_lens, path, num_accepted, *, row_status=None,
                        stream=None):
    """Move the kept path of a verified tree together in the caches, in place,
    before specv_rollback: path [B, M] and num_accepted [B] int32 as
    specv_verify_tree_greedy returns them, the caches [blocks, kv_heads,
    block_size, head_dim] or [layers, blocks, ...] for all layers at once,
    seq_lens [B] with the tree's nodes the last M.  row_status [B] (optional)
    receives 0 or the bits of a refused sequence."""
    c, layers, layer_stride = _kv_cache(h, k_cache, v_cache, block_tables, seq_lens, layered=True)
    B = block_tables.shape[0]
    if path.dim() != 2:
        raise ValueError("path must have the shape [B, M]")
    M = path.shape[1]
    pp = _on(h, path, _i32, "path", (B, M))
    pn = _on(h, num_accepted, _i32, "num_accepted", (B,))
    ps = None if row_status is None else _on(h, row_status, _i32, "row_status", (B,))
    st = _lib.load().specv_cache_compact(h.ptr, c, layers, layer_stride, pp, pn, B, M, ps,
                                         _stream_of(h, stream))
    _check(st, "specv_cache_compact")


def specv_attention_mass(h: Handle, q, k_cache, v_cache, block_tables, seq_lens, lse, *, mass=None, first=0,
                         parents=None, path=None, num_accepted=None, scale=None, out=None, stream=None):
    """The attention weight that the cache's positions gather from a pass:
    mass[b, h, t] plus the sum of exp(scale * q . k_t - lse) over the pass's
    rows that see position t and the query heads of kv head h.  q, the cache,
    parents and scale as for specv_tree_attention, lse [B, rows, q_heads] fp32
    as it left it (rows of an infinite lse take no part); mass [B, kv_heads,
    width] fp32 (None: zeros; the pass's own positions start from zero);
    positions before ``first`` are left alone.  path [B, rows - 1] (None:
    chains) and num_accepted [B] int32 as a verify call gives them: rejected
    drafts take no part, and kept nodes' masses go where specv_cache_compact,
    behind this call, moves their keys.  Returns a dict: mass [B,
    kv_heads, width] and row_status [B]; ``out`` may supply them (mass itself
    among them).  Without it mass is new, zero where nothing is written, and
    as wide as ``mass`` or the table."""
    c, _, _ = _kv_cache(h, k_cache, v_cache, block_tables, seq_lens)
    if q.dim() != 4:
        raise ValueError("q must have the shape [B, rows, q_heads, head_dim]")
    B, rows, q_heads = q.shape[:3]
    if B != block_tables.shape[0]:
        raise ValueError(f"q holds {B} sequences, block_tables {block_tables.shape[0]}")
    pq, q_stride = _token_rows(h, q, "q", k_cache, (B, rows, q_heads, c.head_dim))
    pp = None if parents is None else _on(h, parents, _i32, "parents", (B, rows - 1))
    pl = _on(h, lse, _f32, "lse", (B, rows, q_heads))
    if path is not None and num_accepted is None:
        raise ValueError("path needs num_accepted")
    pt = None if path is None else _on(h, path, _i32, "path", (B, rows - 1))
    pa = None if num_accepted is None else _on(h, num_accepted, _i32, "num_accepted", (B,))
    out = {} if out is None else out
    if "mass" not in out:
        width = c.max_blocks * c.block_size if mass is None else mass.shape[-1]
        out["mass"] = _empty(h, (B, c.kv_heads, width), _f32, stream, zero=True)
    width = out["mass"].shape[-1]
    po = _on(h, out["mass"], _f32, "out['mass']", (B, c.kv_heads, width))
    pm = None if mass is None else _on(h, mass, _f32, "mass", (B, c.kv_heads, width))
    if "row_status" not in out:
        out["row_status"] = _empty(h, (B,), _i32, stream)
    ps = _on(h, out["row_status"], _i32, "row_status", (B,))
    st = _lib.load().specv_attention_mass(
        h.ptr, c, pq, q_stride, q_heads, pp, B, rows, c.head_dim ** -0.5 if scale is None else scale, pl, pt, pa, pm, po,
        width, int(first), ps, _stream_of(h, stream))
    _check(st, "specv_attention_mass")
    return out


def specv_cache_evict(h: Handle, k_cache, v_cache, block_tables, seq_lens, mass, budget, *, recent=0, first=0, out=None,
                      stream=None):
    """Bring sequences longer than ``budget`` back to it, in place in the
    caches [blocks, kv_heads, block_size, head_dim] or [layers, blocks, ...]:
    of each layer and kv head the first ``first`` and the last ``recent``
    positions stay, and of those between the ones of the largest mass; kept
    ones above budget - recent fill the holes below it in order, the recent
    ones follow.  mass [B, kv_heads, width] or [layers, B, kv_heads, width]
    fp32.  Returns a dict: mass (new memory: the remaining positions' masses, zero
    behind them), seq_lens [B] (the new lengths), evicted [B] and row_status
    [B]; ``out`` may supply them, none of them the inputs' memory.  Rotary
    positions go on with offsets raised by ``evicted``; specv_rollback with the
    new lengths and num_accepted = k frees the blocks behind them."""
    c, layers, layer_stride = _kv_cache(h, k_cache, v_cache, block_tables, seq_lens, layered=True)
    B = block_tables.shape[0]
    shape = (B, c.kv_heads) if k_cache.dim() == 4 else (layers, B, c.kv_heads)
    pm = _on(h, mass, _f32, "mass", (*shape, mass.shape[-1]) if mass.dim() else None)
    if mass.dim() == 0:
        raise ValueError("mass must have the shape [B, kv_heads, width] or [layers, B, kv_heads, width]")
    width = mass.shape[-1]
    out = {} if out is None else out
    if "mass" not in out:
        out["mass"] = _empty(h, mass.shape, _f32, stream, zero=True)
    for name in ("seq_lens", "evicted", "row_status"):
        if name not in out:
            out[name] = _empty(h, (B,), _i32, stream)
    po = _on(h, out["mass"], _f32, "out['mass']", mass.shape)
    pn, pe, ps = (_on(h, out[name], _i32, name, (B,)) for name in ("seq_lens", "evicted", "row_status"))
    st = _lib.load().specv_cache_evict(h.ptr, c, layers, layer_stride, pm, po, width, B, int(budget), int(recent),
                                       int(first), pn, pe, ps, _stream_of(h, stream))
    _check(st, "specv_cache_evict")
    return out


def specv_plan_cluster(h: Handle, logits_dtype, B, k, V) -> int:
    return int(_lib.load().specv_plan_cluster(h.ptr, logits_dtype, B, k, V))


def specv_test_withhold_stage(h: Handle, stage_use: int, polls: int) -> None:
    """Test hook: the next split-vocabulary launch (or that of a tcgen05 kernel of
    the cache calls) on ``h`` never fills stage use ``stage_use`` of CTA 0 and its waits give up after
    ``polls`` polls (see include/specv.h)."""
    _check(_lib.load().specv_test_withhold_stage(h.ptr, int(stage_use), int(polls)), "specv_test_withhold_stage")


def specv_launch_count(h: Handle) -> int:
    return int(_lib.load().specv_launch_count(h.ptr))
