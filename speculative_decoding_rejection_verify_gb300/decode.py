"""The operators of a decode step around the verify step (``include/spec_decode.h``), on device tensors.

One round of speculative decoding with a target model:

* in every layer ``kv_append`` rotates the new tokens' queries and keys and puts the keys and values
  into the paged cache, and ``paged_attention`` lets the new tokens attend over it;
* on the logits ``process_logits`` applies penalties, biases and grammar masks at every drafted
  position; then ``verify`` or ``verify_multi``;
* after a tree of drafts ``kv_keep`` moves the accepted branch's entries up behind the context.

The cache is a pair of tensors ``[num_pages, page_size, heads, head_dim]`` (bfloat16, or float8_e4m3fn
with a scale per head); any memory order with ``head_dim`` innermost does, so a pool laid out
``[num_pages, heads, page_size, head_dim]`` is passed as its ``transpose(1, 2)``.  ``pages [B, max_pages]``
says which page holds each stretch of a request's slots; the new tokens of a step take the slots from
``ctx_len[b]`` on.  Argument marshalling only; every call is asynchronous on its stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import speculative_decoding_rejection_verify_gb300 as sv

DTYPE_E4M3 = 2
FLAG_BAD_SLOT = 64
FLAG_BAD_POSITION = 128

MAX_NEW = 64
MAX_GROUP = 128
MAX_PAGE = 4096
MAX_SLOTS = 1 << 30
MAX_HISTORY = 1048448
MAX_BIAS = 2046

DECODE_EXPORTS = ("spec_kv_append", "spec_paged_attention_workspace_bytes", "spec_paged_attention", "spec_kv_keep",
                  "spec_process_logits")

_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class HeadsStruct(ctypes.Structure):
    _fields_ = [("data", _P), ("row_stride", _L), ("token_stride", _L), ("head_stride", _L)]


class CacheStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("layer_stride", _L), ("page_stride", _L), ("slot_stride", _L),
                ("head_stride", _L), ("layers", _I), ("num_pages", _I), ("page_size", _I), ("heads", _I),
                ("head_dim", _I), ("dtype", _I), ("k_scale", _P), ("v_scale", _P)]


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
    """The entry points' argument types."""
    H, C, B = ctypes.POINTER(HeadsStruct), ctypes.POINTER(CacheStruct), ctypes.POINTER(BatchStruct)
    lib.spec_kv_append.argtypes = [H, H, H, H, _I, C, B, ctypes.POINTER(RotaryStruct), _P, _P]
    lib.spec_kv_append.restype = _I
    lib.spec_paged_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
    lib.spec_paged_attention_workspace_bytes.restype = _Z
    lib.spec_paged_attention.argtypes = [H, H, _I, C, B, _P, _F, _P, _Z, _P]
    lib.spec_paged_attention.restype = _I
    lib.spec_kv_keep.argtypes = [C, B, _P, _P, _I, _P]
    lib.spec_kv_keep.restype = _I
    lib.spec_process_logits.argtypes = [_P, _P, ctypes.POINTER(RulesStruct), _I, _I, _I, _I, _P]
    lib.spec_process_logits.restype = _I


def _heads(x, name, shape, device):
    """A [B, T, heads, head_dim] bfloat16 tensor of any strides with head_dim innermost."""
    torch = sv._torch()
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)} != {tuple(shape)}")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name}: dtype {x.dtype} != {torch.bfloat16}")
    if x.device != device:
        raise ValueError(f"{name}: on {x.device}, expected {device}")
    s = x.stride()
    if s[3] != 1:
        raise ValueError(f"{name}: head_dim must be innermost")
    return HeadsStruct(x.data_ptr(), s[0], s[1], s[2])


def _cache(k_cache, v_cache, k_scale, v_scale):
    torch = sv._torch()
    shape, st = k_cache.shape, k_cache.stride()
    dev = k_cache.device
    if dev.type != "cuda":
        raise ValueError("k_cache must be a CUDA tensor")
    if len(shape) != 4 and len(shape) != 5:
        raise ValueError("k_cache must be [num_pages, page_size, heads, head_dim], or with layers in front of it")
    if v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("v_cache must have k_cache's shape and strides")
    if v_cache.dtype != k_cache.dtype or v_cache.device != dev:
        raise ValueError("v_cache must have k_cache's dtype and device")
    if st[-1] != 1:
        raise ValueError("k_cache: head_dim must be innermost")
    if k_cache.dtype == torch.bfloat16:
        dt = sv.DTYPE_BF16
    elif k_cache.dtype == torch.float8_e4m3fn:
        dt = DTYPE_E4M3
    else:
        raise TypeError(f"k_cache must be bfloat16 or float8_e4m3fn, got {k_cache.dtype}")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None:
            sv._check(t, name, (shape[-2],), torch.float32, dev)
    layers, lst = (1, 0) if len(shape) == 4 else (shape[0], st[0])
    return CacheStruct(k_cache.data_ptr(), v_cache.data_ptr(), lst, st[-4], st[-3], st[-2], layers, shape[-4],
                       shape[-3], shape[-2], shape[-1], dt, sv._ptr(k_scale), sv._ptr(v_scale))


def _batch(pages, ctx_len, t_per_row, T, device):
    i32 = sv._torch().int32
    if pages.dim() != 2:
        raise ValueError("pages must be [B, max_pages]")
    B, max_pages = pages.shape
    sv._check(pages, "pages", (B, max_pages), i32, device)
    sv._check(ctx_len, "ctx_len", (B,), i32, device)
    if t_per_row is not None:
        sv._check(t_per_row, "t_per_row", (B,), i32, device)
    return BatchStruct(pages.data_ptr(), ctx_len.data_ptr(), sv._ptr(t_per_row), B, T, max_pages)


def _empty(shape, dtype, device, stream):
    """A new output, allocated on the stream that writes it."""
    torch = sv._torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kv_append(q, k, v, k_cache, v_cache, pages, ctx_len, cos=None, sin=None, t_per_row=None, positions=None,
              interleaved: bool = False, k_scale=None, v_scale=None, out=None, flags=None, stream=None):
    """Rotate the new tokens' ``q [B, T, q_heads, head_dim]`` and ``k [B, T, heads, head_dim]`` and put k and
    ``v`` into the cache at slots ``ctx_len[b] + t`` (spec_kv_append); returns the rotated q (``out``, which may
    be q itself).  ``q`` may be None.  ``cos``/``sin [max_positions, rot_dim / 2]``: None = no rotation;
    ``positions [B, T]``: None = ``ctx_len[b] + t``.  ``t_per_row [B]``: each request's valid tokens (the
    others' rotated q is 0).  ``flags [B]`` int32, cleared by the caller: FLAG_* bits are ORed into it."""
    torch = sv._torch()
    lib = sv.load()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    if k_cache.dim() != 4:
        raise ValueError("k_cache: one layer, [num_pages, page_size, heads, head_dim]")
    if k.dim() != 4:
        raise ValueError("k must be [B, T, heads, head_dim]")
    B, T = k.shape[0], k.shape[1]
    b = _batch(pages, ctx_len, t_per_row, T, dev)
    if b.B != B:
        raise ValueError(f"pages: {b.B} rows for {B} requests")
    shape = (B, T, c.heads, c.head_dim)
    hk, hv = _heads(k, "k", shape, dev), _heads(v, "v", shape, dev)
    hq = ho = None
    n = 0
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, q_heads, head_dim]")
        n = q.shape[2]
        qs = (B, T, n, c.head_dim)
        hq = _heads(q, "q", qs, dev)
        if out is None:
            out = _empty(qs, q.dtype, dev, stream)
        ho = _heads(out, "out", qs, dev)
    r = None
    if cos is not None:
        if sin is None or cos.dim() != 2:
            raise ValueError("cos and sin must both be [max_positions, rot_dim / 2]")
        sv._check(cos, "cos", cos.shape, torch.float32, dev)
        sv._check(sin, "sin", cos.shape, torch.float32, dev)
        if positions is not None:
            sv._check(positions, "positions", (B, T), torch.int32, dev)
        r = ctypes.byref(RotaryStruct(cos.data_ptr(), sin.data_ptr(), sv._ptr(positions), 2 * cos.shape[1],
                                      cos.shape[0], int(interleaved)))
    if flags is not None:
        sv._check(flags, "flags", (B,), torch.int32, dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    rc = lib.spec_kv_append(hq, hk, hv, ho, n, c, b, r, sv._ptr(flags), st.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_append")
    return out


def paged_attention(q, k_cache, v_cache, pages, ctx_len, t_per_row=None, mask=None, scale: Optional[float] = None,
                    k_scale=None, v_scale=None, out=None, workspace_tensor=None, stream=None):
    """Attention of the new tokens' ``q [B, T, q_heads, head_dim]`` over the cache, their own entries included
    (spec_paged_attention, after ``kv_append``); returns ``out`` of q's shape.  ``mask [B, T]`` int64: bit i of
    ``mask[b, t]`` says whether new token t attends to new token i (None: causal); every token attends to the
    whole context.  ``scale``: None = head_dim ** -0.5."""
    torch = sv._torch()
    lib = sv.load()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    if k_cache.dim() != 4:
        raise ValueError("k_cache: one layer, [num_pages, page_size, heads, head_dim]")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    B, T, n, D = q.shape
    b = _batch(pages, ctx_len, t_per_row, T, dev)
    if b.B != B:
        raise ValueError(f"pages: {b.B} rows for {B} requests")
    hq = _heads(q, "q", (B, T, n, c.head_dim), dev)
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    ho = _heads(out, "out", q.shape, dev)
    if mask is not None:
        sv._check(mask, "mask", (B, T), torch.int64, dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = workspace_tensor
    if ws is None:
        nbytes = lib.spec_paged_attention_workspace_bytes(B, T, n, c.heads, D)
        if nbytes == 0:
            raise sv.SpecVerifyError(1, "spec_paged_attention_workspace_bytes")
        ws = sv.workspace(nbytes, dev, st)
    rc = lib.spec_paged_attention(hq, ho, n, c, b, sv._ptr(mask), D ** -0.5 if scale is None else scale,
                                  ws.data_ptr(), ws.numel(), st.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_paged_attention")
    return out


def kv_keep(k_cache, v_cache, pages, ctx_len, path, n_keep, stream=None) -> None:
    """Move the accepted branch's entries up behind the context (spec_kv_keep): in every layer slot
    ``ctx_len[b] + i`` takes slot ``ctx_len[b] + path[b, i]`` for ``i < n_keep[b]``.  The cache may have a leading
    layer dimension; ``path [B, max_keep]`` holds strictly increasing indices of new tokens."""
    torch = sv._torch()
    lib = sv.load()
    c = _cache(k_cache, v_cache, None, None)
    dev = k_cache.device
    b = _batch(pages, ctx_len, None, 0, dev)
    if path.dim() != 2:
        raise ValueError("path must be [B, max_keep]")
    sv._check(path, "path", (b.B, path.shape[1]), torch.int32, dev)
    sv._check(n_keep, "n_keep", (b.B,), torch.int32, dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    rc = lib.spec_kv_keep(c, b, path.data_ptr(), n_keep.data_ptr(), path.shape[1], st.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_kv_keep")


def process_logits(logits, history=None, history_len=None, prompt_len=None, draft=None, t_per_row=None,
                   repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, mask=None, out=None,
                   stream=None):
    """Penalties, biases and grammar masks on ``logits [B, T, V]`` (spec_process_logits); returns ``out``, which may
    be logits itself.  ``history [B, n]`` int32 with ``history_len [B]`` valid ids, the first ``prompt_len[b]`` of them
    the prompt; ``draft [B, T-1]``: the drafts, which count at the positions behind them; ``repetition``,
    ``presence``, ``frequency [B]``; ``bias_ids``/``bias [B, n]``; ``mask [B, T, ceil(V / 32)]`` int32 words of allowed
    tokens.  Rows past ``t_per_row[b]`` are neither read nor written."""
    torch = sv._torch()
    lib = sv.load()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, T, V]")
    B, T, V = logits.shape
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("logits must be a CUDA tensor")
    dt = sv._dtype_code(logits)
    i32, f32 = torch.int32, torch.float32
    sv._check(logits, "logits", (B, T, V), logits.dtype, dev)
    if out is None:
        out = _empty(logits.shape, logits.dtype, dev, stream)
    else:
        sv._check(out, "out", (B, T, V), logits.dtype, dev)
    stride = nb = 0
    if history is not None:
        if history.dim() != 2 or history_len is None:
            raise ValueError("history must be [B, n], with history_len")
        stride = history.shape[1]
        sv._check(history, "history", (B, stride), i32, dev)
    if bias_ids is not None:
        if bias_ids.dim() != 2 or bias is None:
            raise ValueError("bias_ids must be [B, n], with bias")
        nb = bias_ids.shape[1]
        sv._check(bias_ids, "bias_ids", (B, nb), i32, dev)
        sv._check(bias, "bias", (B, nb), f32, dev)
    for t, name in ((history_len, "history_len"), (prompt_len, "prompt_len"), (t_per_row, "t_per_row")):
        if t is not None:
            sv._check(t, name, (B,), i32, dev)
    for t, name in ((repetition, "repetition"), (presence, "presence"), (frequency, "frequency")):
        if t is not None:
            sv._check(t, name, (B,), f32, dev)
    if draft is not None:
        sv._check(draft, "draft", (B, T - 1), i32, dev)
    if mask is not None:
        sv._check(mask, "mask", (B, T, (V + 31) // 32), i32, dev)
    p = sv._ptr
    r = RulesStruct(p(history), p(history_len), p(prompt_len), p(draft), p(t_per_row), p(repetition), p(presence),
                    p(frequency), p(bias_ids), p(bias), p(mask), stride, nb)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    rc = lib.spec_process_logits(logits.data_ptr(), out.data_ptr(), r, B, T, V, dt, st.cuda_stream)
    if rc != sv.SPEC_OK:
        raise sv.SpecVerifyError(rc, "spec_process_logits")
    return out
