"""Operators of a decoding step: 4-bit linear layers, rotary positions,
attention of drafted tokens over a cache, logit penalties.

    table = rotary_table(positions, dim)                       # once
    qkv = w4_linear(x, codes, scales, zeros)                   # [tokens, n] -> [tokens, m]
    q = rotary_append(q, k, v, table, positions, k_cache, v_cache, slots)
    o = tree_attention(q, k_cache, v_cache, kv_lens, tree, page_table=pages)
    l = penalize_logits(logits, history=ids, repetition=r)

Arguments are CUDA tensors on the current device; every step runs in the
library's kernels, and the binding (csrc/binding.cpp) only checks and marshals
them.  An argument that does not fit raises DbsError (DBS_ERR_INVALID_ARG).
Calls are asynchronous on `stream` (a torch stream or a cudaStream_t; default:
the current stream); what they return is allocated on that stream, and the
caller orders its own use of tensors on other streams.  A kernel whose wait runs
out (after two seconds) leaves NaN, and operators_check reports it.  Nothing is
recorded for autograd: a tensor that requires a gradient is refused where
gradients are recorded, and tensors written in place count as changed.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch  # noqa: F401  (the binding uses its libraries)

from . import _build, _lib


def _load():
    _lib.load()
    if not os.path.exists(_build.OPS):
        raise RuntimeError(f"{_build.OPS} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("_dbsops", _build.OPS)
    ops = importlib.util.module_from_spec(importlib.util.spec_from_loader("_dbsops", loader))
    ops._set_error(_lib.DbsError)
    return ops


_ops = _load()

w4_linear = dbs_w4_linear = _ops.w4_linear
rotary_table = dbs_rotary_table = _ops.rotary_table
rotary = dbs_rotary = _ops.rotary
rotary_append = dbs_rotary_append = _ops.rotary_append
tree_attention = dbs_tree_attention = _ops.tree_attention
penalize_logits = dbs_penalize_logits = _ops.penalize_logits
