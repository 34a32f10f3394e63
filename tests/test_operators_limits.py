"""What the decoding step's operators refuse at the ends of their ranges: through
the C ABI, whose checks run on the host before anything is launched."""
import ctypes
import struct

import pytest

torch = pytest.importorskip("torch")

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


@pytest.mark.parametrize("kw", [dict(o2=0), dict(o2=63), dict(o1=0), dict(o0=0), dict(o0=-64), dict(o1=-64), dict(o2=-64), dict(q0=-1), dict(q1=-1),
                                dict(q2=-1), dict(k0=-1), dict(k1=-1), dict(k2=-1), dict(v0=-1), dict(v1=-1), dict(v2=-1), dict(prow=-1)])
def test_attention_refuses_outputs_that_share_memory_and_negative_strides(kw):
    assert attention(**{"batch": 2, **kw}) == BAD
    one = dict(batch=1, tokens=1, hq=1, hk=1)
    if min(kw.values()) >= 0:
        assert attention(**one, **kw) != BAD                               # (of one head, any)


def rotary(heads=2, tokens=4, batch=2, slots=0, pages=3, page=8, inp=A, out=2 * A, strides=(512, 128, 64) * 2):
    part = struct.pack("@" + _lib.ROTARY_HEADS, inp, out, *strides, heads, 1, slots)
    return _lib.load().dbs_rotary(part, 1, 2, batch, tokens, 64, 64, A, 10, A, A, pages, page, 0, 0, None)


@pytest.mark.parametrize("kw", [dict(strides=(512, 128, 64, 512, 128, 0)), dict(strides=(512, 128, 64, 512, 128, 63)), dict(strides=(512, 128, 64, 512, 0, 64)),
                                dict(strides=(512, 128, 64, 0, 128, 64)), dict(strides=(512, 128, 64, 512, 128, -64)),
                                dict(strides=(-512, 128, 64) + (512, 128, 64)), dict(strides=(512, -128, 64) + (512, 128, 64)),
                                dict(strides=(512, 128, -64) + (512, 128, 64)), dict(slots=1, strides=(512, 128, 64, 0, 128, 64)),
                                dict(slots=1, strides=(512, 128, 64, 1024, 0, 64)), dict(out=A, strides=(512, 128, 64, 512, 64, 256)),
                                dict(out=A, slots=1)])
def test_rotary_refuses_outputs_that_share_memory_and_negative_strides(kw):
    assert rotary(**kw) == BAD


def test_rotary_takes_any_stride_of_a_single_head():
    for kw in (dict(), dict(out=A), dict(heads=1, tokens=1, batch=1, strides=(0, 0, 0) * 2), dict(slots=1, pages=1, strides=(512, 128, 64, 0, 128, 64)),
               dict(out=A, heads=1, tokens=1, batch=1, strides=(1, 2, 3, 4, 5, 6))):
        assert torch.cuda.is_available() or rotary(**kw) != BAD             # (where there is no GPU that would run it)


def test_w4_does_not_write_over_its_input():
    lib = _lib.load()
    assert lib.dbs_w4_linear(A, 2, 2, 64, 2 * A, 32, 3 * A, 0, 1, 0, 0, 64, 64, 64, A, 64, None) == BAD
