"""Refusals of the decoding step's operators: through the C ABI, whose checks
run on the host before anything is launched, with addresses that are never
read; and through the Python binding, without a GPU."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
import dynamic_sparsity_spmspv_gb300 as dbs  # noqa: E402
from dynamic_sparsity_spmspv_gb300 import _lib  # noqa: E402

A = 4096                                     # an address; nothing behind it is touched
OK, BAD = 0, 1


def w4(**kw):
    a = dict(x=A, dtype=0, tokens=2, xs=64, q=A, qs=32, s=A, sd=0, ss=1, z=0, zs=0, m=8, n=64, group=64, y=A, ys=8)
    a.update(kw)
    return _lib.load().dbs_w4_linear(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(x=0), dict(q=0), dict(s=0), dict(y=0), dict(dtype=3), dict(dtype=-1), dict(sd=7),
                                dict(tokens=-1), dict(m=-1), dict(n=-2), dict(m=1 << 31), dict(n=1 << 31), dict(group=0),
                                dict(group=48), dict(group=16), dict(group=512), dict(xs=-1), dict(qs=-1), dict(ss=-1),
                                dict(z=A, zs=-1), dict(ys=7)])
def test_w4_refusals(kw):
    assert w4(**kw) == BAD


def test_w4_nothing_to_do():
    assert w4(tokens=0, x=0, y=0) == OK and w4(m=0, q=0, y=0) == OK


def rotary(parts=None, n=1, **kw):
    a = dict(nparts=n, dtype=2, batch=1, tokens=4, d=64, dim=64, table=A, rows=10, pos=A, slots=0, pages=0, page=1, il=0, tr=0)
    a.update(kw)
    heads = parts if parts is not None else head() * n
    return _lib.load().dbs_rotary(heads, *a.values(), None)


def head(inp=A, out=A, heads=2, rotate=1, slots=0):
    import struct
    return struct.pack("@" + _lib.ROTARY_HEADS, inp, out, *[64] * 6, heads, rotate, slots)


@pytest.mark.parametrize("kw", [dict(n=0), dict(n=4), dict(dtype=9), dict(batch=-1), dict(tokens=-1), dict(d=0), dict(d=1025),
                                dict(dim=65), dict(dim=66), dict(dim=-2), dict(table=0), dict(pos=0), dict(rows=-1),
                                dict(batch=1 << 20, tokens=1 << 20), dict(parts=head(inp=0)), dict(parts=head(out=0)),
                                dict(parts=head(heads=-1)), dict(parts=head(slots=1)),
                                dict(parts=head(slots=1), slots=A, pages=-1), dict(parts=head(slots=1), slots=A, pages=4, page=0),
                                dict(parts=head(slots=1), slots=A, pages=1 << 30, page=64)])
def test_rotary_refusals(kw):
    assert rotary(**kw) == BAD


def test_rotary_nothing_to_do():
    assert rotary(tokens=0) == OK and rotary(batch=0, parts=head(inp=0)) == OK and rotary(parts=head(heads=0, inp=0)) == OK
    assert _lib.load().dbs_rotary(None, 1, 2, 1, 4, 64, 64, A, 10, A, 0, 0, 1, 0, 0, None) == BAD


@pytest.mark.parametrize("a", [(-1, 64, 1e4, 0, 1, 0, 0, 0), (8, 63, 1e4, 0, 1, 0, 0, 0), (8, 0, 1e4, 0, 1, 0, 0, 0),
                               (8, 514, 1e4, 0, 1, 0, 0, 0), (8, 64, 1.0, 0, 1, 0, 0, 0), (8, 64, float("nan"), 0, 1, 0, 0, 0),
                               (8, 64, float("inf"), 0, 1, 0, 0, 0), (8, 64, 1e4, 4, 1, 0, 0, 0), (8, 64, 1e4, 1, 0.5, 0, 0, 0),
                               (8, 2, 1e4, 2, 2, 0, 0, 0), (8, 64, 1e4, 3, 4, 0, 32, 1), (8, 64, 1e4, 3, 4, 4096, 1, 32),
                               (8, 64, 1e4, 3, 4, 4096, 32, 0)])
def test_rotary_table_refusals(a):
    assert _lib.load().dbs_rotary_table(*a, A, None) == BAD


def test_rotary_table_null():
    assert _lib.load().dbs_rotary_table(8, 64, 1e4, 0, 1, 0, 0, 0, None, None) == BAD
    assert _lib.load().dbs_rotary_table(0, 64, 1e4, 0, 1, 0, 0, 0, None, None) == OK


ATT = dict(dtype=2, d=64, hq=8, hk=2, batch=2, tokens=3, q=A, q0=512, q1=512, q2=64, k=A, v=A, k0=64, k1=64, k2=64, v0=64,
           v1=64, v2=64, pages=9, page=16, pt=A, maxp=4, prow=4, kv=A, tl=0, tree=0, scale=0.125, out=A, o0=512, o1=512, o2=64,
           lse=0, scratch=A, bytes=1 << 40)


def attention(**kw):
    a = dict(ATT)
    a.update(kw)
    p = _lib.ATTENTION_ARGS.pack(*a.values())
    need = ctypes.c_int64(-1)
    return _lib.load().dbs_tree_attention(p, None), _lib.load().dbs_tree_attention_scratch(p, ctypes.byref(need)), need.value


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=5), dict(d=0), dict(d=257), dict(hk=0), dict(hq=7), dict(hq=1),
                                dict(batch=-1), dict(tokens=-1), dict(tokens=1025), dict(q=0), dict(k=0), dict(v=0), dict(kv=0),
                                dict(out=0), dict(pages=0), dict(pages=-1), dict(page=-1), dict(maxp=-1), dict(pt=0),
                                dict(pt=0, maxp=1, pages=1), dict(page=1 << 20, maxp=1 << 12), dict(scale=float("nan")),
                                dict(scale=float("inf"))])
def test_attention_refusals(kw):
    st, st2, _ = attention(**kw)
    assert st == BAD and st2 == BAD


def test_attention_nothing_to_do_and_nulls():
    assert attention(batch=0, q=0)[0] == OK and attention(tokens=0, out=0)[0] == OK
    lib = _lib.load()
    assert lib.dbs_tree_attention(None, None) == BAD and lib.dbs_tree_attention_scratch(None, None) == BAD
    assert lib.dbs_tree_attention_scratch(_lib.ATTENTION_ARGS.pack(*ATT.values()), None) == BAD


LOG = dict(x=A, dtype=0, xs=100, out=2 * A, od=0, os=100, batch=2, vocab=100, hist=A, hmax=5, hs=5, hl=0, pl=0, rep=0, pres=0,
           freq=0, ids=A, vals=A, nb=3, bs=3, allowed=A, aw=4)


def logits(**kw):
    a = dict(LOG)
    a.update(kw)
    return _lib.load().dbs_penalize_logits(_lib.LOGITS_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw", [dict(x=0), dict(out=0), dict(dtype=3), dict(od=-1), dict(batch=-1), dict(vocab=-1),
                                dict(vocab=1 << 31), dict(hmax=-1), dict(nb=-1), dict(ids=0), dict(vals=0), dict(xs=-1),
                                dict(os=99), dict(hs=-1), dict(bs=-1), dict(aw=-1), dict(out=A, od=1), dict(out=A, os=101)])
def test_logits_refusals(kw):
    assert logits(**kw) == BAD


def test_logits_nothing_to_do():
    assert logits(batch=0, x=0) == OK and logits(vocab=0, out=0) == OK
    assert _lib.load().dbs_penalize_logits(None, None) == BAD


def test_python_refuses_host_tensors():
    x, q, s = torch.zeros(2, 64), torch.zeros((8, 32), dtype=torch.uint8), torch.zeros(8, 1)
    h = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: dbs.w4_linear(x, q, s, group=64), lambda: dbs.rotary(h, h, torch.zeros(9, 64), i),
                 lambda: dbs.rotary_append(h, h, h, torch.zeros(9, 64), i, c, c, i),
                 lambda: dbs.tree_attention(h[None], c, c, i[:1]), lambda: dbs.penalize_logits(x),
                 lambda: dbs.rotary_table(8, 63), lambda: dbs.rotary_table(8, 64, scaling="other"),
                 lambda: dbs.w4_linear(np.zeros((2, 64)), q, s)):
        with pytest.raises(dbs.DbsError) as e:
            call()
        assert e.value.status == BAD


def test_argument_structs_have_the_header_s_size():
    import struct
    import subprocess
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = ('#include "include/dbspmspv.h"\n_Static_assert(sizeof(dbs_rotary_heads) == %d && sizeof(dbs_attention_args) == %d && '
           "sizeof(dbs_logits_args) == %d && offsetof(dbs_attention_args, out) == 200 && offsetof(dbs_logits_args, history) == 64, "
           '"sizes");\n' % (struct.calcsize("@" + _lib.ROTARY_HEADS), _lib.ATTENTION_ARGS.size, _lib.LOGITS_ARGS.size))
    assert subprocess.run(["gcc", "-x", "c", "-fsyntax-only", "-I", root, "-"], input=src.encode(), cwd=root).returncode == 0
