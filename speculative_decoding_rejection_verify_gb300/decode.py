"""The operators of a decode step around the verify step (``include/spec_decode.h``), on device tensors.

One round of speculative decoding with a target model:

* in every layer ``kv_append`` rotates the new tokens' queries and keys and puts the keys and values
  into the paged cache, and ``paged_attention`` lets the new tokens attend over it;
* on the logits ``process_logits`` applies penalties, biases and grammar masks at every drafted
  position; then ``verify`` or ``verify_multi``;
* after a tree of drafts ``kv_keep`` moves the accepted branch's entries up behind the context.

Two ways to keep a long context small:

* a float8_e4m3fn cache with a scale per page and head instead of one per head: pass ``k_scale`` and ``v_scale`` as
  ``[num_pages, heads]`` to every one of these calls; ``kv_append``, ``kv_keep`` and ``kv_move`` set them;
* eviction: ``kv_weigh`` adds up the weight that the accepted tokens' attention gave every entry (``paged_attention`` leaves the rows' sums in ``lse``),
  ``kv_select`` picks the entries of every head that stay within a budget, ``kv_move`` brings them together.  Weights
  (float32) and positions (int32) of the entries are tensors ``[num_pages, heads, page_size]``.

The cache is a pair of tensors ``[num_pages, page_size, heads, head_dim]`` (bfloat16, or float8_e4m3fn
with a scale per head); any memory order with ``head_dim`` innermost does, so a pool laid out
``[num_pages, heads, page_size, head_dim]`` is passed as its ``transpose(1, 2)``.  ``pages [B, max_pages]``
says which page holds each stretch of a request's slots; the new tokens of a step take the slots from
``ctx_len[b]`` on.  Argument marshalling only; every call is asynchronous on its stream.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import speculative_decoding_rejection_verify_gb300 as sv

DTYPE_E4M3 = 2
FLAG_BAD_SLOT = 64
FLAG_BAD_POSITION = 128

MAX_BATCH = 65535
MAX_NEW = 64
MAX_GROUP = 128
MAX_PAGE = 4096
MAX_SLOTS = 1 << 30
MAX_HISTORY = 1048448
MAX_BIAS = 2046

DECODE_EXPORTS = ("spec_kv_append", "spec_kv_append_ex", "spec_paged_attention_workspace_bytes", "spec_paged_attention",
                  "spec_paged_attention_ex", "spec_kv_keep", "spec_kv_keep_ex", "spec_kv_weigh", "spec_kv_select",
                  "spec_kv_move", "spec_process_logits")

_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class HeadsStruct(ctypes.Structure):
    _fields_ = [("data", _P), ("row_stride", _L), ("token_stride", _L), ("head_stride", _L)]


class CacheStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("layer_stride", _L), ("page_stride", _L), ("slot_stride", _L),
                ("head_stride", _L), ("layers", _I), ("num_pages", _I), ("page_size", _I), ("heads", _I),
                ("head_dim", _I), ("dtype", _I), ("k_scale", _P), ("v_scale", _P)]


class PageScalesStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("layer_stride", _L)]


class RecordStruct(ctypes.Structure):
    _fields_ = [("weight", _P), ("position", _P), ("layer_stride", _L), ("layers", _I), ("num_pages", _I),
                ("page_size", _I), ("heads", _I)]


class BatchStruct(ctypes.Structure):
    _fields_ = [("pages", _P), ("ctx_len", _P), ("t_per_row", _P), ("B", _I), ("T", _I), ("max_pages", _I)]


class RotaryStruct(ctypes.Structure):
    _fields_ = [("cos_table", _P), ("sin_table", _P), ("positions", _P), ("rot_dim", _I), ("max_positions", _I),
                ("interleaved", _I)]


class RulesStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("history", "history_len", "prompt_len", "draft", "t_per_row", "repetition",
                                  "presence", "frequency", "bias_ids", "bias", "mask")] + \
        [("history_stride", _I), ("bias_n", _I)]


def declare(lib) -> None:
    """The entry points' argument types.  Structs go as packed bytes (or ctypes.byref of the classes above)."""
    lib.spec_kv_append.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P]
    lib.spec_kv_append.restype = _I
    lib.spec_paged_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
    lib.spec_paged_attention_workspace_bytes.restype = _Z
    lib.spec_paged_attention.argtypes = [_P, _P, _I, _P, _P, _P, _F, _P, _Z, _P]
    lib.spec_paged_attention.restype = _I
    lib.spec_kv_keep.argtypes = [_P, _P, _P, _P, _I, _P]
    lib.spec_kv_keep.restype = _I
    lib.spec_kv_append_ex.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P]
    lib.spec_kv_append_ex.restype = _I
    lib.spec_paged_attention_ex.argtypes = [_P, _P, _I, _P, _P, _P, _P, _F, _P, _P, _Z, _P]
    lib.spec_paged_attention_ex.restype = _I
    lib.spec_kv_keep_ex.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P]
    lib.spec_kv_keep_ex.restype = _I
    lib.spec_kv_weigh.argtypes = [_P, _I, _P, _P, _P, _P, _F, _P, _P, _P, _P]
    lib.spec_kv_weigh.restype = _I
    lib.spec_kv_select.argtypes = [_P, _P, _P, _P, _I, _I, _P, _P, _I, _P, _P, _P]
    lib.spec_kv_select.restype = _I
    lib.spec_kv_move.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _P]
    lib.spec_kv_move.restype = _I
    lib.spec_process_logits.argtypes = [_P, _P, _P, _I, _I, _I, _I, _P]
    lib.spec_process_logits.restype = _I


# The structs as bytes, field by field as in the classes above (NULL is 0).
_pack_heads = struct.Struct("Pqqq").pack
_pack_cache = struct.Struct("PPqqqqiiiiiiPP").pack
_pack_scales = struct.Struct("PPq").pack
_pack_record = struct.Struct("PPqiiii").pack
_pack_batch = struct.Struct("PPPiiixxxx").pack
_pack_rotary = struct.Struct("PPPiiixxxx").pack
_pack_rules = struct.Struct("11Pii").pack


# A small call's time is mostly this module's: the checks below look at a tensor once and say what is wrong
# with it only when something is.
_torch = None
_raw_stream = None
_current_device = None


def _load():
    """(torch, the library), and this module's shortcuts to them."""
    global _torch, _raw_stream, _current_device
    lib = sv.load()
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch = torch
    return _torch, lib


def _fits(t, name, shape, dtype, index) -> int:
    """The address of a contiguous tensor of this shape and dtype on CUDA device ``index``."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        sv._check(t, name, shape, dtype, _torch.device("cuda", index))
    return t.data_ptr()


def _maybe(t, name, shape, dtype, index) -> int:
    return 0 if t is None else _fits(t, name, shape, dtype, index)


def _heads(x, name, shape, index):
    """A [B, T, heads, head_dim] bfloat16 tensor of any strides with head_dim innermost."""
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)} != {tuple(shape)}")
    if x.dtype is not _torch.bfloat16:
        raise TypeError(f"{name}: dtype {x.dtype} != {_torch.bfloat16}")
    if x.get_device() != index:
        raise ValueError(f"{name}: on {x.device}, expected cuda:{index}")
    row, token, head, one = x.stride()
    if one != 1:
        raise ValueError(f"{name}: head_dim must be innermost")
    return _pack_heads(x.data_ptr(), row, token, head)


def _cache(k_cache, v_cache, k_scale, v_scale, layered):
    """(the struct, heads, head_dim, the device's index)"""
    shape, st, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    index = k_cache.get_device()
    if index < 0:
        raise ValueError("k_cache must be a CUDA tensor")
    if index != _current_device():
        sv._launches_on(index)
    if len(shape) != 4 and not (layered and len(shape) == 5):
        raise ValueError("k_cache must be [num_pages, page_size, heads, head_dim]" +
                         (", or with layers in front of it" if layered else ""))
    if v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("v_cache must have k_cache's shape and strides")
    if v_cache.dtype is not dtype or v_cache.get_device() != index:
        raise ValueError("v_cache must have k_cache's dtype and device")
    if st[-1] != 1:
        raise ValueError("k_cache: head_dim must be innermost")
    if dtype is _torch.bfloat16:
        dt = sv.DTYPE_BF16
    elif dtype is _torch.float8_e4m3fn:
        dt = DTYPE_E4M3
    else:
        raise TypeError(f"k_cache must be bfloat16 or float8_e4m3fn, got {dtype}")
    layers, layer = (1, 0) if len(shape) == 4 else (shape[0], st[0])
    num_pages, page, heads, D = shape[-4:]
    scales, ks, vs = None, 0, 0
    if k_scale is not None or v_scale is not None:
        f32 = _torch.float32
        if (v_scale if k_scale is None else k_scale).dim() > 1:
            if k_scale is None or v_scale is None:
                raise ValueError("k_scale and v_scale must both have a scale per page, or neither")
            at = (num_pages, heads) if len(shape) == 4 else (layers, num_pages, heads)
            scales = _pack_scales(_fits(k_scale, "k_scale", at, f32, index), _fits(v_scale, "v_scale", at, f32, index), num_pages * heads)
        else:
            ks, vs = _maybe(k_scale, "k_scale", (heads,), f32, index), _maybe(v_scale, "v_scale", (heads,), f32, index)
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), layer, st[-4], st[-3], st[-2], layers, num_pages, page,
                       heads, D, dt, ks, vs), heads, D, index, scales


def _record(weight, position, shape, index):
    """The struct of weights and positions [num_pages, heads, page_size] (with layers in front), either of which may be None."""
    if weight is None and position is None:
        return None
    num_pages, heads, page = shape[-3:]
    return _pack_record(_maybe(weight, "weight", shape, _torch.float32, index), _maybe(position, "position", shape, _torch.int32, index),
                        num_pages * heads * page, 1 if len(shape) == 3 else shape[0], num_pages, page, heads)


def _record_shape(cache):
    """The shape of what is recorded of a cache's entries."""
    s = tuple(cache.shape)
    return (s[0], s[2], s[1]) if len(s) == 4 else (s[0], s[1], s[3], s[2])


def _batch(pages, ctx_len, t_per_row, B, T, index):
    i32 = _torch.int32
    if pages.dim() != 2:
        raise ValueError("pages must be [B, max_pages]")
    max_pages = pages.shape[1]
    return _pack_batch(_fits(pages, "pages", (B, max_pages), i32, index), _fits(ctx_len, "ctx_len", (B,), i32, index),
                       _maybe(t_per_row, "t_per_row", (B,), i32, index), B, T, max_pages)


def _like(x, stream):
    """A new output of x's shape, allocated on the stream that writes it."""
    if stream is None:
        return _torch.empty_like(x)
    with _torch.cuda.stream(stream):
        return _torch.empty_like(x)


@functools.lru_cache(maxsize=None)
def _attention_bytes(T: int, q_heads: int, heads: int, D: int) -> int:
    """The workspace does not depend on the number of requests.  0: the call itself says what is wrong."""
    return sv.load().spec_paged_attention_workspace_bytes(1, T, q_heads, heads, D)


def kv_append(q, k, v, k_cache, v_cache, pages, ctx_len, cos=None, sin=None, t_per_row=None, positions=None,
              interleaved: bool = False, k_scale=None, v_scale=None, out=None, flags=None, stream=None):
    """Rotate the new tokens' ``q [B, T, q_heads, head_dim]`` and ``k [B, T, heads, head_dim]`` and put k and
    ``v`` into the cache at slots ``ctx_len[b] + t`` (spec_kv_append); returns the rotated q (``out``, which may
    be q itself).  ``k_scale``/``v_scale [heads]``, or ``[num_pages, heads]``: set by what goes into each page
    (spec_kv_append_ex).  ``q`` may be None.  ``cos``/``sin [max_positions, rot_dim / 2]``: None = no rotation;
    ``positions [B, T]``: None = ``ctx_len[b] + t``.  ``t_per_row [B]``: each request's valid tokens (the
    others' rotated q is 0).  ``flags [B]`` int32, cleared by the caller: FLAG_* bits are ORed into it."""
    torch, lib = _load()
    c, heads, D, index, scales = _cache(k_cache, v_cache, k_scale, v_scale, False)
    if k.dim() != 4:
        raise ValueError("k must be [B, T, heads, head_dim]")
    B, T = k.shape[:2]
    b = _batch(pages, ctx_len, t_per_row, B, T, index)
    shape = (B, T, heads, D)
    hk, hv = _heads(k, "k", shape, index), _heads(v, "v", shape, index)
    hq = ho = None
    n = 0
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, q_heads, head_dim]")
        n = q.shape[2]
        shape = (B, T, n, D)
        hq = _heads(q, "q", shape, index)
        if out is None:
            out = _like(q, stream)
        ho = _heads(out, "out", shape, index)
    r = None
    if cos is not None:
        if sin is None or cos.dim() != 2:
            raise ValueError("cos and sin must both be [max_positions, rot_dim / 2]")
        table = tuple(cos.shape)
        r = _pack_rotary(_fits(cos, "cos", table, torch.float32, index), _fits(sin, "sin", table, torch.float32, index),
                         _maybe(positions, "positions", (B, T), torch.int32, index), 2 * table[1], table[0],
                         1 if interleaved else 0)
    elif sin is not None:
        raise ValueError("sin without cos: both are [max_positions, rot_dim / 2]")
    f = _maybe(flags, "flags", (B,), torch.int32, index)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if scales is None:
        rc = lib.spec_kv_append(hq, hk, hv, ho, n, c, b, r, f, handle)
    else:
        rc = lib.spec_kv_append_ex(hq, hk, hv, ho, n, c, scales, b, r, f, handle)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_append")
    return out


def paged_attention(q, k_cache, v_cache, pages, ctx_len, t_per_row=None, mask=None, scale: Optional[float] = None,
                    k_scale=None, v_scale=None, out=None, workspace_tensor=None, stream=None, lse=None):
    """Attention of the new tokens' ``q [B, T, q_heads, head_dim]`` over the cache, their own entries included
    (spec_paged_attention, after ``kv_append``); returns ``out`` of q's shape.  ``mask [B, T]`` int64: bit i of
    ``mask[b, t]`` says whether new token t attends to new token i (None: causal); every token attends to the
    whole context.  ``scale``: None = head_dim ** -0.5.  ``k_scale``/``v_scale [heads]``, or ``[num_pages, heads]``.
    ``lse [B, T, q_heads]`` float32: takes the log of every row's sum of exponentials (spec_paged_attention_ex).  ``workspace_tensor``: None = the binding's own scratch, which is
    the graph's own while one is being captured."""
    torch, lib = _load()
    c, heads, D, index, scales = _cache(k_cache, v_cache, k_scale, v_scale, False)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    B, T, n, _ = shape = q.shape
    b = _batch(pages, ctx_len, t_per_row, B, T, index)
    hq = _heads(q, "q", (B, T, n, D), index)
    if out is None:
        out = _like(q, stream)
    ho = _heads(out, "out", shape, index)
    m = _maybe(mask, "mask", (B, T), torch.int64, index)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    ws = workspace_tensor
    if ws is None:
        nbytes = _attention_bytes(T, n, heads, D)
        ws = sv._scratch.buffers.get((index, handle))
        if ws is None or ws.numel() < nbytes or (torch.cuda.is_current_stream_capturing() if stream is None else sv._capturing(stream)):
            ws = sv.workspace(nbytes, k_cache.device, stream if stream is not None else torch.cuda.current_stream(index))
    else:
        sv._given_workspace(ws, k_cache.device)
    scale = max(D, 1) ** -0.5 if scale is None else scale
    if scales is None and lse is None:
        rc = lib.spec_paged_attention(hq, ho, n, c, b, m, scale, ws.data_ptr(), ws.numel(), handle)
    else:
        rc = lib.spec_paged_attention_ex(hq, ho, n, c, scales, b, m, scale, _maybe(lse, "lse", (B, T, n), torch.float32, index),
                                         ws.data_ptr(), ws.numel(), handle)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_paged_attention")
    return out


def kv_keep(k_cache, v_cache, pages, ctx_len, path, n_keep, stream=None, k_scale=None, v_scale=None, weight=None,
            position=None) -> None:
    """Move the accepted branch's entries up behind the context (spec_kv_keep): in every layer slot
    ``ctx_len[b] + i`` takes slot ``ctx_len[b] + path[b, i]`` for ``i < n_keep[b]``.  The cache may have a leading
    layer dimension; ``path [B, max_keep]`` holds strictly increasing indices of new tokens.  With page scales
    ``k_scale``/``v_scale [num_pages, heads]`` (layers in front as the cache has them) an entry takes its new page's, which grows where it has
    to; ``weight`` and ``position`` move with the entries (spec_kv_keep_ex)."""
    torch, lib = _load()
    c, heads, _, index, scales = _cache(k_cache, v_cache, k_scale, v_scale, True)
    if path.dim() != 2:
        raise ValueError("path must be [B, max_keep]")
    B, most = path.shape
    b = _batch(pages, ctx_len, None, B, 0, index)
    p, n = _fits(path, "path", (B, most), torch.int32, index), _fits(n_keep, "n_keep", (B,), torch.int32, index)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if k_scale is None and v_scale is None and weight is None and position is None:
        rc = lib.spec_kv_keep(c, b, p, n, most, handle)
    else:
        if scales is None and (k_scale is not None or v_scale is not None):
            raise ValueError("k_scale and v_scale of kv_keep are scales per page: a scale per head moves with nothing")
        rc = lib.spec_kv_keep_ex(c, scales, _record(weight, position, _record_shape(k_cache), index), b, p, n, most, handle)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_keep")


def kv_weigh(q, k_cache, pages, ctx_len, lse, weight, position=None, t_per_row=None, mask=None, positions=None,
             scale: Optional[float] = None, k_scale=None, stream=None) -> None:
    """Add up what the new tokens' attention gives every entry (spec_kv_weigh): ``weight [num_pages, heads, page_size]``
    float32 gains the weights that the rows of ``q`` (with the ``lse`` that ``paged_attention`` left, and its arguments) give the
    context's entries, and takes those that they give one another; ``position`` (int32, of weight's shape) takes the new tokens'
    ``positions [B, T]`` (None: ``ctx_len[b] + t``).  A row whose ``lse`` is infinite has no part.  Called after the verdict, with the
    accepted tokens as ``t_per_row`` (a chain) or an infinite ``lse`` for the other rows (a tree, before ``kv_keep``), it leaves out rejected drafts."""
    torch, lib = _load()
    paged = k_scale is not None and k_scale.dim() > 1
    c, heads, D, index, scales = _cache(k_cache, k_cache, k_scale, k_scale if paged else None, False)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    if weight is None:
        raise ValueError("weight must be [num_pages, heads, page_size]")
    B, T, n, _ = q.shape
    b = _batch(pages, ctx_len, t_per_row, B, T, index)
    rc = lib.spec_kv_weigh(_heads(q, "q", (B, T, n, D), index), n, c, scales, b, _maybe(mask, "mask", (B, T), torch.int64, index),
                           max(D, 1) ** -0.5 if scale is None else scale, _fits(lse, "lse", (B, T, n), torch.float32, index),
                           _record(weight, position, _record_shape(k_cache), index),
                           _maybe(positions, "positions", (B, T), torch.int32, index),
                           _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_weigh")


def kv_select(weight, position, pages, ctx_len, budget, seen=None, first: int = 0, recent: int = 0, out=None, stream=None):
    """Pick the ``min(ctx_len[b], budget[b])`` entries of largest weight that stay, of every head by itself (spec_kv_select):
    ``weight`` and ``position [num_pages, heads, page_size]``, or with layers in front.  Entries at positions ``< first`` or
    ``>= seen[b] - recent`` (``seen [B]``: tokens so far, None: ``ctx_len``) go before all others; ``position`` may be None without
    them.  Returns ``(source, target, moves, new_len)`` for ``kv_move``: lists ``[(layers,) B, heads, slots // 2]`` of which
    the first ``moves [(layers,) B, heads]`` count, and the context's new lengths ``[B]`` (``out``: such tensors to write to, the
    lengths' may be ``ctx_len`` itself)."""
    torch, lib = _load()
    if not (0 <= first < 1 << 31 and 0 <= recent < 1 << 31):
        raise ValueError("first and recent must lie in [0, 2^31)")
    if weight.dim() not in (3, 4):
        raise ValueError("weight must be [num_pages, heads, page_size], or with layers in front of it")
    index = weight.get_device()
    if index < 0:
        raise ValueError("weight must be a CUDA tensor")
    if index != _current_device():
        sv._launches_on(index)
    shape = tuple(weight.shape)
    r = _record(weight, position, shape, index)
    if pages.dim() != 2:
        raise ValueError("pages must be [B, max_pages]")
    B = pages.shape[0]
    b = _batch(pages, ctx_len, None, B, 0, index)
    lists = (B, shape[1]) if len(shape) == 3 else (shape[0], B, shape[2])
    if out is None:
        most = pages.shape[1] * shape[-1] // 2
        new = lambda size: torch.empty(size, dtype=torch.int32, device=weight.device)  # noqa: E731
        if stream is None:
            out = new(lists + (most,)), new(lists + (most,)), new(lists), new((B,))
        else:
            with torch.cuda.stream(stream):
                out = new(lists + (most,)), new(lists + (most,)), new(lists), new((B,))
    source, target, moves, new_len = out
    most = source.shape[-1] if source.dim() else 0
    i32, full = torch.int32, lists + (most,)
    rc = lib.spec_kv_select(r, b, _fits(budget, "budget", (B,), i32, index), _maybe(seen, "seen", (B,), i32, index), first, recent,
                            _fits(source, "source", full, i32, index), _fits(target, "target", full, i32, index),
                            most, _fits(moves, "moves", lists, i32, index), _fits(new_len, "new_len", (B,), i32, index),
                            _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_select")
    return source, target, moves, new_len


def kv_move(k_cache, v_cache, pages, new_len, source, target, moves, k_scale=None, v_scale=None, weight=None, position=None,
            stream=None) -> None:
    """Move the entries that ``kv_select`` picked to the front (spec_kv_move): in every layer and head slot
    ``target[..., i]`` takes slot ``source[..., i]`` for ``i < moves``, keys, values, page scales, ``weight`` and ``position``.
    The context has ``new_len`` entries from then on; they keep their rotation, so the next tokens' positions have to be given."""
    torch, lib = _load()
    c, heads, _, index, scales = _cache(k_cache, v_cache, k_scale, v_scale, True)
    if scales is None and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale and v_scale of kv_move are scales per page: a scale per head moves with nothing")
    if pages.dim() != 2 or source.dim() < 1:
        raise ValueError("pages must be [B, max_pages], and source [B, heads, n]")
    B, most = pages.shape[0], source.shape[-1]
    b = _batch(pages, new_len, None, B, 0, index)
    lists, i32 = (B, heads) if k_cache.dim() == 4 else (k_cache.shape[0], B, heads), torch.int32
    full = lists + (most,)
    r = None if weight is None and position is None else _record(weight, position, _record_shape(k_cache), index)
    rc = lib.spec_kv_move(c, scales, r, b, _fits(source, "source", full, i32, index), _fits(target, "target", full, i32, index),
                          _fits(moves, "moves", lists, i32, index), most, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_move")


def process_logits(logits, history=None, history_len=None, prompt_len=None, draft=None, t_per_row=None,
                   repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, mask=None, out=None,
                   stream=None):
    """Penalties, biases and grammar masks on ``logits [B, T, V]`` (spec_process_logits); returns ``out``, which may
    be logits itself.  ``history [B, n]`` int32 with ``history_len [B]`` valid ids, the first ``prompt_len[b]`` of them
    the prompt; ``draft [B, T-1]``: the drafts, which count at the positions behind them; ``repetition``,
    ``presence``, ``frequency [B]``; ``bias_ids``/``bias [B, n]``; ``mask [B, T, ceil(V / 32)]`` int32 words of allowed
    tokens.  Rows past ``t_per_row[b]`` are neither read nor written."""
    torch, lib = _load()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, T, V]")
    B, T, V = shape = logits.shape
    index = logits.get_device()
    if index < 0:
        raise ValueError("logits must be a CUDA tensor")
    if index != _current_device():
        sv._launches_on(index)
    dt = sv._dtype_code(logits)
    i32, f32 = torch.int32, torch.float32
    z = _fits(logits, "logits", shape, logits.dtype, index)
    if out is None:
        out = _like(logits, stream)
    o = _fits(out, "out", shape, logits.dtype, index)
    stride = nb = 0
    hist = ids = bias_at = 0
    if history is not None:
        if history.dim() != 2 or history_len is None:
            raise ValueError("history must be [B, n], with history_len")
        stride = history.shape[1]
        hist = _fits(history, "history", (B, stride), i32, index)
    if bias_ids is not None:
        if bias_ids.dim() != 2 or bias is None:
            raise ValueError("bias_ids must be [B, n], with bias")
        nb = bias_ids.shape[1]
        ids = _fits(bias_ids, "bias_ids", (B, nb), i32, index)
        bias_at = _fits(bias, "bias", (B, nb), f32, index)
    elif bias is not None:
        raise ValueError("bias needs the bias_ids [B, n] that it is for")
    row = (B,)
    r = _pack_rules(hist, _maybe(history_len, "history_len", row, i32, index),
                    _maybe(prompt_len, "prompt_len", row, i32, index),
                    _maybe(draft, "draft", (B, max(T - 1, 0)), i32, index), _maybe(t_per_row, "t_per_row", row, i32, index),
                    _maybe(repetition, "repetition", row, f32, index), _maybe(presence, "presence", row, f32, index),
                    _maybe(frequency, "frequency", row, f32, index), ids, bias_at,
                    _maybe(mask, "mask", (B, T, (V + 31) // 32), i32, index), stride, nb)
    rc = lib.spec_process_logits(z, o, r, B, T, V, dt, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_process_logits")
    return out
