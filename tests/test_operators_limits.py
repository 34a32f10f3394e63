"""What the decoding step's operators refuse at the ends of their ranges: through
the C ABI, whose checks run on the host before anything is launched."""
import ctypes

import pytest

pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
from dynamic_sparsity_spmspv_gb300 import _lib  # noqa: E402

OK, BAD = 0, 1


def test_limits_of_the_waits():
    lib = _lib.load()
    for limit, block in ((0, -1), (-5, 0), (2_000_000_001, -1), (1000, -3)):
        assert lib.dbs_debug_operator_waits(limit, block) == BAD
    assert lib.dbs_debug_operator_waits(2_000_000_000, -1) == OK


A = 4096                                     # an address; nothing behind it is touched
ATT = dict(dtype=2, d=64, hq=8, hk=2, batch=0, tokens=3, q=A, q0=512, q1=512, q2=64, k=A, v=A, k0=64, k1=64, k2=64, v0=64,
           v1=64, v2=64, pages=9, page=16, pt=A, maxp=4, prow=4, kv=A, tl=0, tree=0, scale=0.125, out=A, o0=1536, o1=512, o2=64,
           lse=0, scratch=A, bytes=1 << 40)


def attention(**kw):
    """Status of asking for a call's scratch: its checks, then (without a GPU) the device that is not there."""
    a = dict(ATT)
    a.update(kw)
    need = ctypes.c_int64(-1)
    return _lib.load().dbs_tree_attention_scratch(_lib.ATTENTION_ARGS.pack(*a.values()), ctypes.byref(need))


def test_attention_entries_that_an_int_cannot_number():
    """A tile may end up to 127 entries behind the last one: that number has to be an int too."""
    for page, maxp in ((64, (1 << 25) - 1), (1, (1 << 31) - 1), (1 << 30, 2), ((1 << 31) - 1, 1), (1, (1 << 31) - 1023)):
        assert attention(batch=2, page=page, maxp=maxp, prow=maxp) == BAD
    assert attention(batch=2, page=1, maxp=(1 << 31) - 1024, prow=1 << 31) != BAD
