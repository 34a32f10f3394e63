"""Operators of a decoding step: 4-bit linear layers, rotary positions,
attention of drafted tokens over a cache, logit penalties.

    table = rotary_table(positions, dim)                       # once
    qkv = w4_linear(x, codes, scales, zeros)                   # [tokens, n] -> [tokens, m]
    q = rotary_append(q, k, v, table, positions, k_cache, v_cache, slots)
    o = tree_attention(q, k_cache, v_cache, kv_lens, tree, page_table=pages)
    l = penalize_logits(logits, history=ids, repetition=r)

Arguments are CUDA tensors; every step runs in the library's kernels, and this
module only checks and marshals them.  An argument that does not fit raises
DbsError (DBS_ERR_INVALID_ARG).  Calls are asynchronous on `stream` (default:
the current stream); what they return is allocated on that stream, and the
caller orders its own use of tensors on other streams.
"""
from __future__ import annotations

import math
import struct

import torch

from . import _lib

F32, F16, BF16 = 0, 1, 2
_DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_I32 = torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _bad(fn, why):
    raise _lib.DbsError(fn, 1, why)


def _device(fn, t, **others):
    """The CUDA device index that every given tensor is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad(fn, "CUDA tensors are needed")
    dev = t.get_device()
    for name, o in others.items():
        if o is not None and (not isinstance(o, torch.Tensor) or not o.is_cuda or o.get_device() != dev):
            _bad(fn, f"{name} has to be a tensor on the same CUDA device")
    return dev


def _stream(dev, stream):
    """(handle, whether tensors made now belong to that stream)."""
    current = _raw_stream(dev)
    if stream is None:
        return current, True
    h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return h, h == current


def _empty(shape, dtype, dev, handle, here):
    if here:
        return torch.empty(shape, dtype=dtype, device=dev)
    s = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=dev)


def _rows(fn, name, t, shape, dtype):
    """Row stride of a 2-d tensor of that shape and type, rows contiguous."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        _bad(fn, f"{name} has to be {dtype} of shape {shape}")
    if shape[1] > 1 and t.stride(1) != 1:
        _bad(fn, f"{name}: the last dimension has to be contiguous")
    return t.stride(0)


def _vector(fn, name, t, n, dtype):
    if t is None:
        return 0
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _bad(fn, f"{name} has to be a contiguous {dtype} tensor of {n} values")
    return t.data_ptr()


def dbs_w4_linear(x, q, scales, zeros=None, *, group: int = 128, y=None, stream=None):
    """dbs_w4_linear: y[t, i] = sum_j x[t, j] (q[i, j] - z[i, j // group]) s[i, j // group].

    x [tokens, n] or [n], float32, float16 or bfloat16; q uint8 [m, ceil(n/2)]
    (column 2c in the low half of byte c); scales [m, ceil(n/group)] in any of
    those types; zeros uint8 of the same shape, or None for 8.  Rows of q that
    start on 16-byte boundaries are the fast case.  Returns y [tokens, m] (or
    [m]) in x's type."""
    fn = "dbs_w4_linear"
    dev = _device(fn, x, q=q, scales=scales, zeros=zeros, y=y)
    one = x.dim() == 1
    if one:
        x = x[None]
    if x.dim() != 2 or q.dim() != 2 or scales.dim() != 2:
        _bad(fn, "x is [tokens, n] or [n], q and scales have two dimensions")
    tokens, n = x.shape
    m = q.shape[0]
    dt, sd = _DTYPES.get(x.dtype), _DTYPES.get(scales.dtype)
    if dt is None or sd is None:
        _bad(fn, "x and scales have to be float32, float16 or bfloat16")
    if group not in (32, 64, 128, 256):
        _bad(fn, "group has to be 32, 64, 128 or 256")
    xs = _rows(fn, "x", x, (tokens, n), x.dtype)
    qs = _rows(fn, "q", q, (m, (n + 1) // 2), torch.uint8)
    groups = -(-n // group)
    ss = _rows(fn, "scales", scales, (m, groups), scales.dtype)
    zs = 0 if zeros is None else _rows(fn, "zeros", zeros, (m, groups), torch.uint8)
    handle, here = _stream(dev, stream)
    if y is None:
        y = _empty((tokens, m), x.dtype, dev, handle, here)
        ys, out = m, y[0] if one else y
    else:
        out, y = y, y[None] if one and y.dim() == 1 else y
        ys = _rows(fn, "y", y, (tokens, m), x.dtype)
    _lib.check(fn, _lib.load().dbs_w4_linear(
        x.data_ptr(), dt, tokens, xs, q.data_ptr(), qs, scales.data_ptr(), sd, ss,
        0 if zeros is None else zeros.data_ptr(), zs, m, n, group, y.data_ptr(), ys, handle))
    return out


def dbs_rotary_table(positions: int, dim: int, *, base: float = 10000.0, scaling=None, factor: float = 1.0,
                     trained: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None, stream=None):
    """dbs_rotary_table: float32 [positions, dim], cosines then sines.
    scaling: None, "linear", "ntk" or "yarn" (with `trained` positions)."""
    fn = "dbs_rotary_table"
    if scaling not in _SCALINGS:
        _bad(fn, "scaling is None, 'linear', 'ntk' or 'yarn'")
    positions, dim = int(positions), int(dim)
    if positions < 0 or dim < 2 or dim > 512 or dim % 2:
        _bad(fn, "positions >= 0, dim even and in 2..512")
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        _bad(fn, "a CUDA device is needed")
    dev = torch.cuda.current_device() if dev.index is None else dev.index
    handle, here = _stream(dev, stream)
    table = _empty((positions, dim), torch.float32, dev, handle, here)
    _lib.check(fn, _lib.load().dbs_rotary_table(positions, dim, float(base), _SCALINGS[scaling], float(factor),
                                                float(trained), float(beta_fast), float(beta_slow), table.data_ptr(),
                                                handle))
    return table


def _tokens(fn, name, t, like, dtype):
    """[batch, tokens, heads, head_dim], or [tokens, heads, head_dim], as four sizes and the three outer strides."""
    if t.dtype != dtype or t.dim() not in (3, 4):
        _bad(fn, f"{name} has to be a {dtype} tensor [batch, tokens, heads, head_dim] or [tokens, heads, head_dim]")
    if t.dim() == 4:
        (b, n, h, d), (sb, sn, sh, sd) = t.shape, t.stride()
    else:
        (n, h, d), (sn, sh, sd) = t.shape, t.stride()
        b, sb = 1, 0
    if like is not None and (b, n, d) != like:
        _bad(fn, f"{name} has to have {like[0]} x {like[1]} tokens and heads of {like[2]}")
    if d > 1 and sd != 1:
        _bad(fn, f"{name}: the last dimension has to be contiguous")
    return (b, n, h, d), (sb, sn, sh)


def _turning(fn, q, table, positions, slots):
    dev = _device(fn, q, table=table, positions=positions, slots=slots)
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        _bad(fn, "q has to be float32, float16 or bfloat16")
    (b, n, h, d), st = _tokens(fn, "q", q, None, q.dtype)
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous() or table.shape[1] > d:
        _bad(fn, "table has to be contiguous float32 [positions, dim], dim at most head_dim")
    for name, t in (("positions", positions), ("slots", slots)):
        if t is not None and (t.dtype != _I32 or t.numel() != b * n or not t.is_contiguous()):
            _bad(fn, f"{name} has to be contiguous int32, one for each token")
    return dev, dt, (b, n, h, d), st


def _turned(fn, t, out, size, strides, dev, handle, here):
    """(out, its strides) for the rotated t."""
    if out is None:
        out = _empty(t.shape, t.dtype, dev, handle, here)
    elif out is t:
        return out, strides
    else:
        _device(fn, t, out=out)
        if out.shape != t.shape:
            _bad(fn, "outputs have their input's shape")
    return out, _tokens(fn, "output", out, None, t.dtype)[1]


def dbs_rotary(q, k, table, positions, *, interleaved: bool = False, transposed: bool = False, q_out=None, k_out=None,
               stream=None):
    """dbs_rotary: q and k (or None) [batch, tokens, heads, head_dim] or
    [tokens, heads, head_dim], turned by their tokens' positions (int32).  The
    first table.shape[1] entries of a head are turned, in pairs (i, i + dim/2)
    or, interleaved, (2i, 2i + 1); the rest is copied.  transposed turns the
    other way: the gradient.  Returns (q, k), new tensors unless q_out and
    k_out are given (the inputs themselves: in place)."""
    fn = "dbs_rotary"
    dev, dt, (b, n, h, d), st = _turning(fn, q, table, positions, None)
    handle, here = _stream(dev, stream)
    q_out, so = _turned(fn, q, q_out, (b, n, h, d), st, dev, handle, here)
    args = [q.data_ptr(), q_out.data_ptr(), *st, *so, h, 1, 0]
    parts = 1
    if k is not None:
        _device(fn, q, k=k)
        (_, _, hk, _), sk = _tokens(fn, "k", k, (b, n, d), q.dtype)
        k_out, so = _turned(fn, k, k_out, (b, n, hk, d), sk, dev, handle, here)
        args += [k.data_ptr(), k_out.data_ptr(), *sk, *so, hk, 1, 0]
        parts = 2
    _lib.check(fn, _lib.load().dbs_rotary(
        struct.pack("@" + _lib.ROTARY_HEADS * parts, *args), parts, dt, b, n, d, table.shape[1], table.data_ptr(),
        table.shape[0], positions.data_ptr(), 0, 0, 1, interleaved, transposed, handle))
    return q_out, (k_out if k is not None else None)


def dbs_rotary_append(q, k, v, table, positions, k_cache, v_cache, slots, *, interleaved: bool = False, q_out=None,
                      stream=None):
    """dbs_rotary with a cache: q is turned and returned; k, turned, and v go to
    entry slots[token] (int32; outside the cache: not written) of k_cache and
    v_cache [pages, page_size, kv_heads, head_dim], in the same launch."""
    fn = "dbs_rotary_append"
    dev, dt, (b, n, h, d), st = _turning(fn, q, table, positions, slots)
    _device(fn, q, k=k, v=v, k_cache=k_cache, v_cache=v_cache)
    (_, _, hk, _), sk = _tokens(fn, "k", k, (b, n, d), q.dtype)
    (_, _, hv, _), sv = _tokens(fn, "v", v, (b, n, d), q.dtype)
    if k_cache.dim() != 4 or k_cache.shape[2:] != (hk, d) or hv != hk or v_cache.shape != k_cache.shape:
        _bad(fn, "caches have to be [pages, page_size, kv_heads, head_dim]")
    (pages, page, _, _), ck = _tokens(fn, "k_cache", k_cache, None, q.dtype)
    cv = _tokens(fn, "v_cache", v_cache, None, q.dtype)[1]
    handle, here = _stream(dev, stream)
    q_out, so = _turned(fn, q, q_out, (b, n, h, d), st, dev, handle, here)
    heads = struct.pack("@" + _lib.ROTARY_HEADS * 3, q.data_ptr(), q_out.data_ptr(), *st, *so, h, 1, 0,
                        k.data_ptr(), k_cache.data_ptr(), *sk, *ck, hk, 1, 1,
                        v.data_ptr(), v_cache.data_ptr(), *sv, *cv, hk, 0, 1)
    _lib.check(fn, _lib.load().dbs_rotary(
        heads, 3, dt, b, n, d, table.shape[1], table.data_ptr(), table.shape[0], positions.data_ptr(),
        slots.data_ptr(), pages, max(page, 1), interleaved, 0, handle))
    return q_out


def dbs_tree_attention(q, k_cache, v_cache, kv_lens, tree=None, *, tree_lens=None, page_table=None, scale=None, out=None,
                       return_lse: bool = False, stream=None):
    """dbs_tree_attention: drafted tokens q [batch, tokens, q_heads, head_dim]
    (float16 or bfloat16) against caches [pages, page_size, kv_heads, head_dim]
    with page_table int32 [batch, max_pages], or, without one, [batch, entries,
    kv_heads, head_dim].  kv_lens int32 [batch] counts a sequence's entries, its
    drafted tokens last among them; tree_lens int32 [batch] counts those (None:
    all of q's tokens).  tree int64 [batch, tokens, ceil(tokens / 64)]: bit i of
    token t's words is set if it sees drafted token i (None: i <= t).  Returns
    out like q, and with return_lse the float32 [batch, tokens, q_heads]
    logarithm of each row's sum."""
    fn = "dbs_tree_attention"
    dev = _device(fn, q, k_cache=k_cache, v_cache=v_cache, kv_lens=kv_lens, tree=tree, tree_lens=tree_lens,
                  page_table=page_table)
    dt = _DTYPES.get(q.dtype)
    if dt is None or dt == F32 or q.dim() != 4:
        _bad(fn, "q has to be float16 or bfloat16 [batch, tokens, q_heads, head_dim]")
    (b, t, h, d), sq = _tokens(fn, "q", q, None, q.dtype)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[3] != d or d > 256 or d < 1:
        _bad(fn, "caches have to be [pages, page_size, kv_heads, head_dim], heads like q's and of at most 256")
    (pages, page, hk, _), sk = _tokens(fn, "k_cache", k_cache, None, q.dtype)
    sv = _tokens(fn, "v_cache", v_cache, None, q.dtype)[1]
    if hk == 0 or h == 0 or h % hk or t > 1024:
        _bad(fn, "q_heads has to be a multiple of kv_heads, tokens at most 1024")
    if page_table is None:
        if pages < b:
            _bad(fn, "without a page_table the caches are [batch, entries, kv_heads, head_dim]")
        max_pages, page_row, pt = 1, 0, 0
    else:
        if page_table.dim() != 2 or page_table.shape[0] != b:
            _bad(fn, "page_table has to be int32 [batch, max_pages]")
        max_pages = page_table.shape[1]
        page_row = _rows(fn, "page_table", page_table, (b, max_pages), _I32)
        pt = page_table.data_ptr()
    lens = _vector(fn, "kv_lens", kv_lens, b, _I32)
    tlens = _vector(fn, "tree_lens", tree_lens, b, _I32)
    if tree is not None and (tree.dtype != torch.int64 or tree.shape != (b, t, (t + 63) // 64) or not tree.is_contiguous()):
        _bad(fn, "tree has to be contiguous int64 [batch, tokens, ceil(tokens / 64)]")
    handle, here = _stream(dev, stream)
    if out is None:
        out = _empty((b, t, h, d), q.dtype, dev, handle, here)
        so = (t * h * d, h * d, d)
    else:
        _device(fn, q, out=out)
        if out.shape != q.shape:
            _bad(fn, "out has to have q's shape")
        so = _tokens(fn, "out", out, None, q.dtype)[1]
    lse = _empty((b, t, h), torch.float32, dev, handle, here) if return_lse else None
    lib = _lib.load()
    args = [dt, d, h, hk, b, t, q.data_ptr(), *sq, k_cache.data_ptr(), v_cache.data_ptr(), *sk, *sv, pages, page, pt,
            max_pages, page_row, lens, tlens, 0 if tree is None else tree.data_ptr(),
            1.0 / math.sqrt(d) if scale is None else float(scale), out.data_ptr(), *so,
            0 if lse is None else lse.data_ptr(), 0, 0]
    need = _lib.I64()
    _lib.check(fn, lib.dbs_tree_attention_scratch(_lib.ATTENTION_ARGS.pack(*args), _lib.ctypes.byref(need)))
    if need.value:
        scratch = _empty((need.value,), torch.uint8, dev, handle, here)
        args[-2:] = scratch.data_ptr(), need.value
    _lib.check(fn, lib.dbs_tree_attention(_lib.ATTENTION_ARGS.pack(*args), handle))
    return (out, lse) if return_lse else out


def dbs_penalize_logits(logits, *, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
                        frequency=None, bias_ids=None, bias_vals=None, allowed=None, out=None, stream=None):
    """dbs_penalize_logits: logits [batch, vocab] (float32, float16, bfloat16)
    with the penalties of the tokens in history int32 [batch, history_max]
    (history_lens int32 [batch] of them; the first prompt_lens[b] count for
    repetition alone), biases float32 bias_vals at int32 bias_ids [batch, n],
    and -inf where bit v % 32 of allowed int32 [batch, ceil(vocab / 32)] is
    clear.  repetition, presence and frequency: float32 [batch].  Returns
    float32, or `out` (which may be logits: in place)."""
    fn = "dbs_penalize_logits"
    dev = _device(fn, logits, history=history, history_lens=history_lens, prompt_lens=prompt_lens,
                  repetition=repetition, presence=presence, frequency=frequency, bias_ids=bias_ids, bias_vals=bias_vals,
                  allowed=allowed, out=out)
    dt = _DTYPES.get(logits.dtype)
    if dt is None or logits.dim() != 2:
        _bad(fn, "logits have to be float32, float16 or bfloat16 [batch, vocab]")
    b, vocab = logits.shape
    ls = _rows(fn, "logits", logits, (b, vocab), logits.dtype)
    if history is None:
        if history_lens is not None or prompt_lens is not None or repetition is not None or presence is not None \
                or frequency is not None:
            _bad(fn, "penalties and lengths need a history")
        hist, hmax, hs = 0, 0, 0
    else:
        if history.dim() != 2 or history.shape[0] != b:
            _bad(fn, "history has to be int32 [batch, history_max]")
        hmax = history.shape[1]
        hs, hist = _rows(fn, "history", history, (b, hmax), _I32), history.data_ptr()
    nb = bs = ids = vals = 0
    if bias_ids is not None or bias_vals is not None:
        if bias_ids is None or bias_vals is None or bias_ids.dim() != 2 or bias_ids.shape[0] != b:
            _bad(fn, "bias_ids int32 and bias_vals float32 [batch, n] come together")
        nb = bias_ids.shape[1]
        bs = _rows(fn, "bias_ids", bias_ids, (b, nb), _I32)
        if _rows(fn, "bias_vals", bias_vals, (b, nb), torch.float32) != bs and b > 1:
            _bad(fn, "bias_ids and bias_vals have to have the same strides")
        ids, vals = bias_ids.data_ptr(), bias_vals.data_ptr()
    aw = 0 if allowed is None else _rows(fn, "allowed", allowed, (b, (vocab + 31) // 32), _I32)
    handle, here = _stream(dev, stream)
    if out is None:
        out, os = _empty((b, vocab), torch.float32, dev, handle, here), vocab
    else:
        if out.dtype not in _DTYPES:
            _bad(fn, "out has to be float32, float16 or bfloat16")
        os = _rows(fn, "out", out, (b, vocab), out.dtype)
    _lib.check(fn, _lib.load().dbs_penalize_logits(_lib.LOGITS_ARGS.pack(
        logits.data_ptr(), dt, ls, out.data_ptr(), _DTYPES[out.dtype], os, b, vocab, hist, hmax, hs,
        _vector(fn, "history_lens", history_lens, b, _I32), _vector(fn, "prompt_lens", prompt_lens, b, _I32),
        _vector(fn, "repetition", repetition, b, torch.float32), _vector(fn, "presence", presence, b, torch.float32),
        _vector(fn, "frequency", frequency, b, torch.float32), ids, vals, nb, bs,
        0 if allowed is None else allowed.data_ptr(), aw), handle))
    return out


# short names
w4_linear = dbs_w4_linear
rotary_table = dbs_rotary_table
rotary = dbs_rotary
rotary_append = dbs_rotary_append
tree_attention = dbs_tree_attention
penalize_logits = dbs_penalize_logits
