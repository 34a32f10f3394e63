"""Refusals of the operators around a paged cache: through the C ABI, whose checks
run on the host before anything is launched, with addresses that are never
read; and through the Python binding, without a GPU."""
import ctypes
import struct

import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
import dynamic_sparsity_spmspv_gb300 as dbs  # noqa: E402
from dynamic_sparsity_spmspv_gb300 import _lib  # noqa: E402

A = 4096                                     # an address; nothing behind it is touched
OK, BAD = 0, 1
NO_GPU = not torch.cuda.is_available()


def part(inp=A, out=2 * A, strides=(512, 128, 64) * 2, heads=2, rotate=1, slots=0, weight=A, wtype=0):
    return struct.pack("@" + _lib.NORM_HEADS, inp, out, *strides, heads, rotate, slots, weight, wtype)


def norm(parts=None, n=1, **kw):
    a = dict(dtype=2, batch=1, tokens=4, d=64, dim=64, eps=1e-6, table=A, rows=10, pos=A, slots=0, pages=0, page=1, il=0)
    a.update(kw)
    return _lib.load().dbs_norm_rotary(parts if parts is not None else part() * n, n, *a.values(), None)


@pytest.mark.parametrize("kw", [dict(n=0), dict(n=4), dict(dtype=9), dict(batch=-1), dict(tokens=-1), dict(d=0), dict(d=1025), dict(dim=65),
                                dict(dim=66), dict(dim=-2), dict(table=0), dict(pos=0), dict(rows=-1), dict(eps=-1e-9), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(batch=1 << 20, tokens=1 << 20), dict(batch=1 << 12, tokens=1 << 14),
                                dict(parts=part(inp=0)), dict(parts=part(out=0)), dict(parts=part(heads=-1)), dict(parts=part(heads=16385)),
                                dict(parts=part(wtype=3)), dict(parts=part(slots=1)), dict(parts=part(slots=1), slots=A, pages=-1),
                                dict(parts=part(slots=1), slots=A, pages=4, page=0), dict(parts=part(slots=1), slots=A, pages=1 << 30, page=64),
                                dict(parts=part(strides=(512, 128, 64, 512, 128, 63))), dict(parts=part(strides=(512, 128, 64, 512, 0, 64))),
                                dict(parts=part(strides=(512, -128, 64, 512, 128, 64))), dict(parts=part(out=A, strides=(512, 64, 256, 512, 128, 64))),
                                dict(parts=part(out=A, slots=1), slots=A, pages=4, page=16)])
def test_norm_refusals(kw):
    assert norm(**kw) == BAD


def test_norm_nothing_to_do():
    assert norm(tokens=0) == OK and norm(batch=0, parts=part(inp=0)) == OK and norm(parts=part(heads=0, inp=0)) == OK
    assert norm(parts=part(slots=1, out=0), slots=A, pages=0) == OK
    assert _lib.load().dbs_norm_rotary(None, 1, 2, 1, 4, 64, 64, 1e-6, A, 10, A, 0, 0, 1, 0, None) == BAD


GRAD = dict(grad=A, inp=2 * A, out=3 * A, strides=(512, 128, 64) * 3, heads=2, wtype=0, weight=A, dw=A)


def gpart(**kw):
    a = dict(GRAD)
    a.update(kw)
    return struct.pack("@" + _lib.NORM_GRADIENT_HEADS, a["grad"], a["inp"], a["out"], *a["strides"], a["heads"], a["wtype"], a["weight"], a["dw"])


def gradient(parts=None, n=1, **kw):
    a = dict(dtype=2, batch=1, tokens=4, d=64, dim=64, eps=1e-6, table=A, rows=10, pos=A, il=0, scratch=0, bytes=0)
    a.update(kw)
    return _lib.load().dbs_norm_rotary_gradient(parts if parts is not None else gpart() * n, n, *a.values(), None)


@pytest.mark.parametrize("kw", [dict(n=0), dict(n=3), dict(dtype=9), dict(batch=-1), dict(tokens=-1), dict(d=0), dict(d=1025), dict(dim=65),
                                dict(dim=-2), dict(table=0), dict(pos=0), dict(rows=-1), dict(eps=-1.0), dict(parts=gpart(grad=0)),
                                dict(parts=gpart(inp=0)), dict(parts=gpart(out=0)), dict(parts=gpart(heads=-1)), dict(parts=gpart(wtype=5)),
                                dict(parts=gpart(strides=(512, 128, 64, 512, 128, 64, 512, 128, 63))),
                                dict(parts=gpart(strides=(-512, 128, 64, 512, 128, 64, 512, 128, 64))),
                                dict(parts=gpart(strides=(512, 128, 64, 512, -128, 64, 512, 128, 64))),
                                dict(parts=gpart(out=A, strides=(512, 64, 256, 512, 128, 64, 512, 128, 64))),
                                dict(parts=gpart(out=2 * A, strides=(512, 128, 64, 512, 64, 256, 512, 128, 64)))])
def test_norm_gradient_refusals(kw):
    assert gradient(**kw) == BAD


def test_norm_gradient_nothing_to_do_and_scratch():
    assert gradient(parts=gpart(dw=0), tokens=0) == OK and gradient(parts=gpart(dw=0, heads=0, grad=0)) == OK
    need = ctypes.c_int64(-1)
    size = _lib.load().dbs_norm_rotary_gradient_scratch
    assert size(0, 64, ctypes.byref(need)) == BAD and size(3, 64, ctypes.byref(need)) == BAD and size(1, 0, ctypes.byref(need)) == BAD
    assert size(1, 1025, ctypes.byref(need)) == BAD and size(1, 64, None) == BAD
    if not NO_GPU:
        assert size(2, 64, ctypes.byref(need)) == OK and need.value > 0
        assert gradient(scratch=0, bytes=1 << 30) == BAD and gradient(scratch=A, bytes=need.value // 4) == BAD and gradient(scratch=A + 8, bytes=1 << 30) == BAD


WIN = dict(dtype=2, d=64, hq=8, hk=2, batch=2, tokens=3, q=A, q0=1536, q1=512, q2=64, k=A, v=A, k0=64, k1=64, k2=64, v0=64, v1=64, v2=64, pages=9,
           page=16, pt=A, maxp=4, prow=4, kv=A, ql=0, window=5, sinks=0, scale=0.125, out=2 * A, o0=1536, o1=512, o2=64, lse=0,
           scratch=A, bytes=1 << 40)


def window(**kw):
    a = dict(WIN)
    a.update(kw)
    return _lib.load().dbs_window_attention(_lib.WINDOW_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=4), dict(d=0), dict(d=257), dict(hk=0), dict(hk=3), dict(hq=0), dict(hq=1), dict(hq=65538),
                                dict(batch=-1), dict(tokens=-1), dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(kv=0), dict(pages=-1), dict(pages=0),
                                dict(page=-1), dict(maxp=-1), dict(window=0), dict(window=-3), dict(sinks=-1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(q0=-1), dict(q1=-1), dict(q2=-1), dict(k0=-1), dict(k1=-1), dict(k2=-1), dict(v0=-1),
                                dict(v1=-1), dict(v2=-1), dict(prow=-1), dict(o2=63), dict(o1=0), dict(o0=0), dict(pt=0), dict(pt=0, maxp=1, pages=1),
                                dict(batch=1 << 31), dict(tokens=1 << 31), dict(batch=1 << 16, tokens=1 << 15), dict(batch=1 << 14, tokens=1 << 14),
                                dict(page=64, maxp=(1 << 25) - 1), dict(page=1 << 30, maxp=2), dict(page=(1 << 31) - 1, maxp=1), dict(pages=1 << 31),
                                dict(out=A)])
def test_window_refusals(kw):
    a = dict(WIN)
    a.update(kw)
    need = ctypes.c_int64(-1)
    assert window(**kw) == BAD and _lib.load().dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*a.values()), ctypes.byref(need)) == BAD


def test_window_nothing_to_do():
    assert window(batch=0, q=0, out=0, kv=0) == OK and window(tokens=0, q=0, out=0) == OK
    assert _lib.load().dbs_window_attention(None, None) == BAD and _lib.load().dbs_window_attention_scratch(None, None) == BAD
    assert _lib.load().dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*WIN.values()), None) == BAD


STATE = dict(table=A, batch=3, maxp=4, prow=4, kv=A, refs=A, pages=9, page=16)


def state(**kw):
    a = dict(STATE)
    a.update(kw)
    return _lib.PAGE_STATE.pack(*a.values())


BAD_STATES = [dict(batch=-1), dict(batch=1 << 24), dict(maxp=-1), dict(prow=3), dict(kv=0), dict(pages=-1), dict(page=0), dict(page=-4),
              dict(pages=1 << 28), dict(maxp=1 << 28, prow=1 << 28), dict(pages=0x7fffffff, page=1), dict(page=1 << 31, pages=0, maxp=0), dict(table=0)]


@pytest.mark.parametrize("kw", BAD_STATES)
def test_page_state_refusals(kw):
    lib, big = _lib.load(), 1 << 40
    assert lib.dbs_cache_resize(state(**kw), 2 * A, A, 0, 0, A, big, None) == BAD
    assert lib.dbs_cache_fork(data(), state(**kw), A, A, 2, A, A, big, None) == BAD


def data(k=A, v=A, layers=2, heads=2, d=64, e=2, strides=(18432, 2048, 128, 64) * 2):
    return _lib.CACHE_DATA.pack(k, v, layers, heads, d, e, *strides)


def test_resize_refusals():
    lib, big = _lib.load(), 1 << 40

    def resize(s=state(), lens=2 * A, status=3 * A, slots=0, columns=0, scratch=A, size=big):
        return lib.dbs_cache_resize(s, lens, status, slots, columns, scratch, size, None)

    large = state(batch=2000)                                              # (few sequences need no scratch)
    for kw in (dict(s=None), dict(lens=0), dict(status=0), dict(columns=-1), dict(columns=1 << 31), dict(s=large, scratch=0),
               dict(s=large, scratch=A + 4), dict(s=large, size=16), dict(s=state(refs=0)), dict(lens=A), dict(status=A), dict(status=2 * A)):
        assert resize(**kw) == BAD, kw
    assert resize(s=state(batch=0, kv=0, table=0), lens=0, status=0, scratch=0) == OK
    need = ctypes.c_int64(-1)
    assert lib.dbs_cache_resize_scratch(large, 0, ctypes.byref(need)) == OK and need.value >= 4 * (3 * 2000 + 9)
    assert lib.dbs_cache_resize_scratch(state(), 5, ctypes.byref(need)) == OK and need.value == 0
    for bad in ((state(), 0, None), (None, 0, ctypes.byref(need)), (state(), -1, ctypes.byref(need)), (state(), 1 << 31, ctypes.byref(need))):
        assert lib.dbs_cache_resize_scratch(*bad) == BAD


def test_fork_refusals():
    lib, big = _lib.load(), 1 << 40

    def fork(d=data(), s=state(), parents=A, children=A, n=2, status=A, scratch=A, size=big):
        return lib.dbs_cache_fork(d, s, parents, children, n, status, scratch, size, None)

    cases = [dict(d=None), dict(s=None), dict(parents=0), dict(children=0), dict(n=-1), dict(n=65536), dict(status=0), dict(scratch=0),
             dict(scratch=A + 8), dict(size=8), dict(s=state(refs=0))]
    cases += [dict(d=data(**kw)) for kw in BAD_DATA]
    for kw in cases:
        assert fork(**kw) == BAD, kw
    assert fork(n=0, parents=0, children=0, status=0, scratch=0) == OK
    need = ctypes.c_int64(-1)
    assert lib.dbs_cache_fork_scratch(state(), 3, ctypes.byref(need)) == OK and need.value > 0
    assert lib.dbs_cache_fork_scratch(state(), -1, ctypes.byref(need)) == BAD and lib.dbs_cache_fork_scratch(state(), 3, None) == BAD


BAD_DATA = [dict(k=0), dict(v=0), dict(layers=-1), dict(layers=32768), dict(heads=-1), dict(heads=1 << 31), dict(d=-1), dict(d=1 << 31),
            dict(heads=1 << 16, d=1 << 16), dict(e=3), dict(e=0), dict(e=16), dict(strides=(18432, 2048, 128, 63) + (18432, 2048, 128, 64)),
            dict(strides=(18432, 2048, 128, 64) + (18432, 2048, 0, 64)), dict(strides=(18432, 0, 128, 64) + (18432, 2048, 128, 64)),
            dict(strides=(0, 2048, 128, 64) * 2), dict(strides=(-18432, 2048, 128, 64) * 2)]


def test_compact_refusals():
    lib = _lib.load()

    def compact(d=data(), s=state(), tree=A, acc=A, most=4, stride=4, lens=0, new=2 * A):
        return lib.dbs_cache_compact(d, s, tree, acc, most, stride, lens, new, None)

    cases = [dict(d=None), dict(s=None), dict(tree=0), dict(acc=0), dict(most=-1), dict(most=1 << 31), dict(stride=-1), dict(new=0), dict(new=A), dict(tree=2 * A), dict(lens=2 * A),
             dict(s=state(batch=65536)), dict(s=state(table=0)), dict(s=state(table=0, maxp=1, pages=2)), dict(s=state(pages=0))]
    cases += [dict(d=data(**kw)) for kw in BAD_DATA]
    for kw in cases:
        assert compact(**kw) == BAD, kw
    assert compact(s=state(batch=0, kv=0, table=0), tree=0, acc=0, new=0) == OK


@pytest.mark.skipif(not NO_GPU, reason="host tensors are refused before anything else")
def test_binding_refuses_host_tensors_and_wrong_arguments():
    t, i = torch.zeros(2, 3, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    calls = [lambda: dbs.norm_rotary(t, None, None, None, t, i), lambda: dbs.norm_rotary_append(t, t, t, None, None, t, i, t, t, i),
             lambda: dbs.norm_rotary_gradient(t, None, t, None, None, None, t, i), lambda: dbs.window_attention(t, t, t, i, 4),
             lambda: dbs.cache_resize(i, i, i, i, 16), lambda: dbs.cache_fork(t, t, i, i, i, i, i), lambda: dbs.cache_compact(t, t, i, i, i)]
    for call in calls:
        with pytest.raises(dbs.DbsError):
            call()
    for name in ("norm_rotary", "norm_rotary_append", "norm_rotary_gradient", "window_attention", "cache_resize", "cache_fork", "cache_compact"):
        with pytest.raises(TypeError):
            getattr(dbs, name)(t)
        assert getattr(dbs, "dbs_" + name) is getattr(dbs, name) and getattr(dbs, name).__doc__
    with pytest.raises(TypeError):
        dbs.window_attention(t, t, t, i, 4, windows=3)


def test_argument_structs_have_the_header_s_size():
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sizes = {"dbs_norm_heads": struct.calcsize("@" + _lib.NORM_HEADS), "dbs_norm_gradient_heads": struct.calcsize("@" + _lib.NORM_GRADIENT_HEADS),
             "dbs_window_args": _lib.WINDOW_ARGS.size, "dbs_page_state": _lib.PAGE_STATE.size, "dbs_cache_data": _lib.CACHE_DATA.size}
    src = '#include <stddef.h>\n#include "include/dbspmspv.h"\n' + "".join(f'_Static_assert(sizeof({k}) == {v}, "size");\n' for k, v in sizes.items())
    src += '_Static_assert(offsetof(dbs_window_args, scale) == 200 && offsetof(dbs_cache_data, k_layer) == 48, "places");\n'
    assert subprocess.run(["gcc", "-x", "c", "-fsyntax-only", "-I", root, "-"], input=src.encode(), cwd=root).returncode == 0


# (heads, tokens, batch of 2, 4, 2 or pages of 16 entries) strides that are each a head's size, of places that meet all the same
TANGLED = [(512, 64, 64), (64, 128, 64), (512, 128, 128), (512, 128, 65), (320, 128, 64), (256, 128, 100)]


@pytest.mark.parametrize("by", TANGLED)
def test_outputs_whose_strides_do_not_step_over_one_another_are_refused(by):
    lib = _lib.load()
    assert norm(batch=2, parts=part(strides=(512, 128, 64) + by)) == BAD
    assert norm(batch=2, parts=part(slots=1, strides=(512, 128, 64) + (4 * by[0], *by[1:])), slots=A, pages=2, page=16) == BAD
    assert gradient(batch=2, parts=gpart(strides=(512, 128, 64) * 2 + by)) == BAD
    need = ctypes.c_int64(-1)
    a = dict(WIN, hq=2, hk=1, tokens=4, out=1 << 20, o0=by[0], o1=by[1], o2=by[2])
    assert lib.dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*a.values()), ctypes.byref(need)) == BAD
    heads = struct.pack("@" + _lib.ROTARY_HEADS, A, 1 << 20, 512, 128, 64, *by, 2, 1, 0)
    assert lib.dbs_rotary(heads, 1, 2, 2, 4, 64, 64, A, 10, A, 0, 0, 1, 0, 0, None) == BAD
    tree = _lib.ATTENTION_ARGS.pack(2, 64, 2, 1, 2, 4, A, 512, 128, 64, A, A, *[64] * 6, 9, 16, A, 4, 4, A, 0, 0, 0.125, 1 << 20, *by, 0, A, 1 << 40)
    assert lib.dbs_tree_attention_scratch(tree, ctypes.byref(need)) == BAD


@pytest.mark.parametrize("by", [(18432, 2048, 64, 64), (18432, 2048, 128, 65), (18432, 1984, 128, 64), (18431, 2048, 128, 64), (2048, 2048, 128, 64),
                                (64, 128, 2304, 64), (18432, 2048, 64, 1000)])
def test_caches_whose_places_meet_are_refused(by):
    lib, big, plain, far = _lib.load(), 1 << 40, (18432, 2048, 128, 64), 1 << 30
    for strides in (by + plain, plain + by):
        d = data(k=A, v=far, strides=strides)
        assert lib.dbs_cache_fork(d, state(), A, A, 2, A, A, big, None) == BAD
        assert lib.dbs_cache_compact(d, state(), A, A, 4, 4, 0, 2 * A, None) == BAD


def test_permuted_and_sliced_outputs_are_taken():
    need = ctypes.c_int64(-1)
    for by in ((1536, 512, 64), (1536, 64, 192), (64, 128, 384), (4096, 1024, 128), (192, 64, 384), (64, 1 << 40, 1 << 50), (1 << 60, 512, 64)):
        a = dict(WIN, out=1 << 40, o0=by[0], o1=by[1], o2=by[2])
        assert _lib.load().dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*a.values()), ctypes.byref(need)) != BAD, by


FAR = 1 << 30


def test_outputs_that_lie_on_inputs_in_part_are_refused():
    """Shifted views, other strides of the same memory, an output on another group's input or output; places in between, and the very
    same place where a call works in place, are not."""
    need = ctypes.c_int64(-1)

    def win(**kw):
        return _lib.load().dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*{**WIN, "q": FAR, "k": 2 * FAR, "v": 3 * FAR, "out": 4 * FAR, **kw}.values()), ctypes.byref(need))

    size = 2 * 3 * 8 * 64 * 2                                              # of q
    for shift in (-size + 2, -128, 128, 1024, size - 2):
        assert win(out=FAR + shift) == BAD
    assert win(out=FAR + size) != BAD and win(out=FAR - size) != BAD
    k = dict(k0=2048, k1=128, k2=64, v0=2048, v1=128, v2=64)               # nine pages
    assert win(out=2 * FAR + 9 * 4096 - 2, **k) == BAD and win(out=2 * FAR + 9 * 4096, **k) != BAD
    assert win(out=3 * FAR + 4096 - size, **k) == BAD
    fused = dict(q0=3 * 1024, q1=1024, q2=64, o0=3 * 1024, o1=1024, o2=64)  # q and another tensor of eight heads, side by side
    assert win(out=FAR + 1024, **fused) != BAD and win(out=FAR + 1022, **fused) == BAD and win(out=FAR - 128, **fused) == BAD
    q, k = part(inp=FAR, out=2 * FAR), part(inp=3 * FAR, out=4 * FAR)
    for bad in (part(inp=3 * FAR, out=2 * FAR), part(inp=3 * FAR, out=2 * FAR + 1022), part(inp=3 * FAR, out=FAR), part(inp=3 * FAR, out=FAR + 512),
                part(inp=3 * FAR, out=3 * FAR + 128), part(inp=2 * FAR, out=4 * FAR), part(inp=3 * FAR, out=3 * FAR - 1022)):
        assert norm(parts=q + bad, n=2) == BAD and norm(parts=bad + q, n=2) == BAD
        turn = q[:_rotary] + bad[:_rotary]
        assert _lib.load().dbs_rotary(turn, 2, 2, 1, 4, 64, 64, A, 10, A, 0, 0, 1, 0, 0, None) == BAD
    assert norm(parts=part(inp=FAR, out=2 * FAR, slots=1) + part(inp=3 * FAR, out=3 * FAR, slots=1), n=2, slots=A, pages=4, page=16) == BAD
    g = dict(grad=FAR, inp=2 * FAR, out=3 * FAR, dw=4 * FAR)
    other = dict(grad=5 * FAR, inp=6 * FAR, out=7 * FAR, dw=8 * FAR)
    for kw in (dict(out=3 * FAR), dict(out=3 * FAR + 128), dict(out=FAR), dict(out=2 * FAR + 1022), dict(out=5 * FAR - 128), dict(out=6 * FAR + 128), dict(dw=4 * FAR),
               dict(dw=4 * FAR - 252), dict(dw=3 * FAR), dict(inp=3 * FAR), dict(grad=3 * FAR + 256)):
        assert gradient(parts=gpart(**g) + gpart(**{**other, **kw}), n=2) == BAD, kw


_rotary = struct.calcsize("@" + _lib.ROTARY_HEADS)


def test_arrays_of_a_cache_s_pages_that_overlap_are_refused():
    lib, big = _lib.load(), 1 << 40
    apart = dict(table=FAR, kv=2 * FAR, refs=3 * FAR)

    def resize(lens=4 * FAR, status=5 * FAR, slots=6 * FAR, **kw):
        return lib.dbs_cache_resize(state(**dict(apart, **kw)), lens, status, slots, 2, A, big, None)

    for kw in (dict(lens=2 * FAR + 8), dict(status=4 * FAR - 8), dict(slots=4 * FAR - 20), dict(slots=2 * FAR + 4), dict(status=6 * FAR + 20), dict(refs=2 * FAR + 8),
               dict(kv=FAR + 4), dict(lens=3 * FAR + 32), dict(status=FAR + 44), dict(refs=FAR - 32), dict(lens=FAR + 40)):
        assert resize(**kw) == BAD, kw

    def fork(parents=4 * FAR, children=5 * FAR, status=6 * FAR, d=data(k=7 * FAR, v=8 * FAR), **kw):
        return lib.dbs_cache_fork(d, state(**dict(apart, **kw)), parents, children, 2, status, A, big, None)

    for kw in (dict(status=4 * FAR + 4), dict(children=6 * FAR - 4), dict(parents=2 * FAR + 8), dict(children=3 * FAR), dict(refs=2 * FAR), dict(status=FAR),
               dict(d=data(k=7 * FAR, v=7 * FAR + 128))):
        assert fork(**kw) == BAD, kw

    def compact(tree=4 * FAR, acc=5 * FAR, lens=6 * FAR, new=9 * FAR, d=data(k=7 * FAR, v=8 * FAR), **kw):
        return lib.dbs_cache_compact(d, state(**dict(apart, **kw)), tree, acc, 4, 4, lens, new, None)

    for kw in (dict(new=4 * FAR + 8), dict(new=5 * FAR + 44), dict(new=6 * FAR - 8), dict(new=2 * FAR - 8), dict(new=FAR + 12), dict(d=data(k=7 * FAR, v=7 * FAR)),
               dict(d=data(k=7 * FAR, v=7 * FAR + 2 * 18432 * 2 - 2))):
        assert compact(**kw) == BAD, kw


@pytest.mark.parametrize("tokens,heads", [(4, 2), (300, 40), (2000, 128)])
def test_outputs_at_an_input_s_address_with_other_strides_are_refused(tokens, heads):
    """Heads before tokens and tokens before heads, with room between heads: places that meet in many ways or few, the first of them for certain."""
    step = 72
    plain, turned = (0, heads * step, step), (0, step, tokens * step)
    for a, b in ((plain, turned), (turned, plain)):
        assert norm(tokens=tokens, parts=part(inp=FAR, out=FAR, heads=heads, strides=a + b)) == BAD
        assert gradient(tokens=tokens, parts=gpart(grad=FAR, inp=2 * FAR, out=FAR, dw=0, heads=heads, strides=a + a + b)) == BAD
        need = ctypes.c_int64(-1)
        w = {**WIN, "batch": 1, "tokens": tokens, "hq": heads, "hk": 2, "q": FAR, "out": FAR, "q1": a[1], "q2": a[2], "o1": b[1], "o2": b[2]}
        assert _lib.load().dbs_window_attention_scratch(_lib.WINDOW_ARGS.pack(*w.values()), ctypes.byref(need)) == BAD
        turn = struct.pack("@" + _lib.ROTARY_HEADS, FAR, FAR, *a, *b, heads, 1, 0)
        assert _lib.load().dbs_rotary(turn, 1, 2, 1, tokens, 64, 64, A, 10, A, 0, 0, 1, 0, 0, None) == BAD
