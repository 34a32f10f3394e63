"""GPU parity of the operators around a paged cache against plain 64-bit forms:
norms with rotation and their gradient, attention with a window and sinks, pages.

Tolerances, from the formulas (u = unit roundoff of the type that a result is
rounded to: 2^-24 fp32, 2^-11 fp16, 2^-8 bf16; e = 2^-24):
  norm       a head's sum of squares: at most 32 terms a lane and 5 exchanges, each
             rounded once, and the squares, so 38 e relative; its root halves that; with the division,
             root, two products and a turn (3 e of |a cos| + |b sin|) at most 28 e:
             32 e (|a cos| + |b sin|) + u |y|, and half the spacing of fp16's subnormals
  gradient   x': the same root, a dot product of the same shape (38 e of the sum of its
             magnitudes), products: 64 e r (|w g| + |n| mean |w g n|) + u |x'|, |g| taken as
             |a cos| + |b sin|; w': chains of at most 64 + 64 terms here:
             192 e sum |g n| + u |w'|
  attention  (u + 3e-4) * sum p |v| + u |out|: probabilities rounded once to the
             caches' type, and fp32 scores, whose error is at most
             head_dim * 2^-23 * scale * sum |q k| (1.1e-4 at head_dim 128,
             1.6e-4 at 256 for N(0,1) inputs), twice (numerator and sum)
  pages      whole numbers and copies: equal
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
import dynamic_sparsity_spmspv_gb300 as dbs  # noqa: E402

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
ETA = {"f32": 2.0**-140, "f16": 2.0**-25, "bf16": 2.0**-133}
E = 2.0**-24
NAN, INF = float("nan"), float("inf")


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - ref) <= tol)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} off, worst {np.nanmax(np.abs(got - ref)[~ok] / np.broadcast_to(tol, ok.shape)[~ok])} x tolerance"


def rnd(rng, dt, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dt]).to(DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- norms with rotation ----


def turned(x, table, pos, il, back=False):
    """Turned heads and |a cos| + |b sin|; x [..., tokens, heads, D], pos [..., tokens]."""
    dim = table.shape[1]
    c, s = table[pos][..., None, : dim // 2], table[pos][..., None, dim // 2:] * (-1 if back else 1)
    y, mag = x.copy(), np.abs(x)
    lo, hi = (slice(0, dim, 2), slice(1, dim, 2)) if il else (slice(0, dim // 2), slice(dim // 2, dim))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mag[..., lo], mag[..., hi] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return y, mag


def norm_ref(x, w, table, pos, il, eps):
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return turned(n if w is None else n * w, table, pos, il)


def grad_ref(g, x, w, table, pos, il, eps):
    w = np.ones(x.shape[-1]) if w is None else w
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    g, mag = turned(g, table, pos, il, back=True)
    dx = r * (w * g - n * (w * g * n).mean(-1, keepdims=True))
    dx_mag = r * (np.abs(w) * mag + np.abs(n) * (np.abs(w * n) * mag).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, dx_mag, (g * n).sum(axes), (mag * np.abs(n)).sum(axes)


def heads_of(rng, dt, lead, heads, D, layout, size=1.0):
    """[*lead, heads, D] in one of several layouts."""
    t = (size * torch.from_numpy(rng.standard_normal((*lead, heads, D)).astype(np.float32))).to(DT[dt]).to(DEV)
    if layout == "first" and len(lead) == 2:
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd":
        wide = torch.full((*lead, heads, D + 5), NAN, dtype=DT[dt], device=DEV)
        wide[..., 3:3 + D] = t
        return wide[..., 3:3 + D]
    return t


NORM_CASES = [
    # tokens, heads, head_dim, dim, interleaved, layout
    ((1,), 1, 2, 2, False, "plain"), ((1,), 1, 1, 0, False, "plain"), ((3,), 2, 7, 4, True, "plain"), ((5,), 40, 128, 128, False, "plain"),
    ((2, 9), 4, 64, 64, True, "plain"), ((2, 9), 4, 128, 64, False, "first"), ((1, 33), 3, 96, 96, True, "first"),
    ((1, 33), 3, 96, 48, False, "plain"), ((2, 5), 2, 80, 80, False, "plain"), ((2, 5), 2, 80, 40, True, "plain"), ((7,), 3, 256, 256, False, "plain"),
    ((4,), 2, 256, 24, True, "odd"), ((3,), 1, 1024, 512, False, "plain"), ((3,), 2, 1024, 512, True, "odd"), ((2, 3), 1, 1000, 510, False, "plain"),
    ((17,), 9, 72, 8, True, "plain"), ((0,), 2, 64, 64, False, "plain"), ((2, 0), 2, 64, 64, False, "plain"), ((6,), 5, 520, 512, False, "plain"),
    ((400,), 12, 128, 128, False, "plain")]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lead,heads,D,dim,il,layout", NORM_CASES)
def test_norm_rotary(dt, lead, heads, D, dim, il, layout):
    rng = np.random.default_rng(len(lead) * 7 + heads * 1000 + D + dim)
    q, k = heads_of(rng, dt, lead, heads, D, layout, 2.0), heads_of(rng, dt, lead, max(1, heads // 3), D, layout, 0.5)
    qw, kw = rnd(rng, dt, D), rnd(rng, "f32", D)
    table = dbs.rotary_table(50, dim) if dim else torch.zeros((50, 0), device=DEV)
    pos = torch.from_numpy(rng.integers(0, 50, lead).astype(np.int32)).to(DEV)
    qo, ko = dbs.norm_rotary(q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    assert qo.dtype == q.dtype and ko.shape == k.shape
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        ref, mag = norm_ref(f64(x), f64(w), f64(table), pos.cpu().numpy(), il, np.float64(np.float32(1e-5)))
        close(got, ref, 32 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
    again = dbs.norm_rotary(q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    assert torch.equal(again[0], qo) and torch.equal(again[1], ko)
    # in place, and without weights and keys
    x = q.clone()
    r = dbs.norm_rotary(x, None, qw, None, table, pos, eps=1e-5, interleaved=il, q_out=x)
    assert r[0].data_ptr() == x.data_ptr() and r[1] is None
    if layout == "odd":                                                    # (the copy lies on other boundaries: sums in another order)
        ref, mag = norm_ref(f64(q), f64(qw), f64(table), pos.cpu().numpy(), il, np.float64(np.float32(1e-5)))
        close(x, ref, 32 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
    else:
        assert torch.equal(x, qo)
    bare = dbs.norm_rotary(q, None, None, None, table, pos, eps=1e-5, interleaved=il)[0]
    ref, mag = norm_ref(f64(q), None, f64(table), pos.cpu().numpy(), il, np.float64(np.float32(1e-5)))
    close(bare, ref, 32 * E * mag + U[dt] * np.abs(ref) + ETA[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lead,heads,D,dim,il,layout", NORM_CASES)
def test_norm_rotary_gradient(dt, lead, heads, D, dim, il, layout):
    rng = np.random.default_rng(len(lead) * 11 + heads * 1000 + D + dim)
    kv = max(1, heads // 3)
    q, k = heads_of(rng, dt, lead, heads, D, layout, 2.0), heads_of(rng, dt, lead, kv, D, layout, 0.5)
    qg, kg = heads_of(rng, dt, lead, heads, D, layout), heads_of(rng, dt, lead, kv, D, "plain")
    qw, kw = rnd(rng, "f32", D), rnd(rng, dt, D)
    table = dbs.rotary_table(50, dim) if dim else torch.zeros((50, 0), device=DEV)
    pos = torch.from_numpy(rng.integers(0, 50, lead).astype(np.int32)).to(DEV)
    got = dbs.norm_rotary_gradient(qg, kg, q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    eps, t, p = np.float64(np.float32(1e-5)), f64(table), pos.cpu().numpy()
    for dx, dw, g, x, w in ((got[0], got[2], qg, q, qw), (got[1], got[3], kg, k, kw)):
        assert dx.dtype == x.dtype and dw.dtype == torch.float32
        ref, mag, wref, wmag = grad_ref(f64(g), f64(x), f64(w), t, p, il, eps)
        close(dx, ref, 64 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
        close(dw, wref, 192 * E * wmag + E * np.abs(wref) + 1e-30)
    again = dbs.norm_rotary_gradient(qg, kg, q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    alone = dbs.norm_rotary_gradient(qg, None, q, None, None, None, table, pos, eps=1e-5, interleaved=il)
    assert alone[1] is None and alone[3] is None
    ref, mag, wref, wmag = grad_ref(f64(qg), f64(q), None, t, p, il, eps)
    close(alone[0], ref, 64 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
    close(alone[2], wref, 192 * E * wmag + E * np.abs(wref) + 1e-30)


MANY_TOKENS = [((2, 6000), 16, 8, 64, 64, False, "plain"), ((1, 12000), 8, 4, 128, 64, False, "first"), ((12001,), 8, 4, 96, 96, True, "plain"),
               ((2, 5000), 17, 16, 128, 128, True, "plain"), ((10000,), 9, 5, 256, 0, False, "plain")]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lead,hq,hk,D,dim,il,layout", MANY_TOKENS)
def test_norm_rotary_of_many_tokens(dt, lead, hq, hk, D, dim, il, layout):
    """Several turns of every warp; a few positions outside the table, a few slots outside the cache."""
    rng = np.random.default_rng(hq + D)
    n = int(np.prod(lead))
    q, k, v = heads_of(rng, dt, lead, hq, D, layout, 2.0), heads_of(rng, dt, lead, hk, D, layout), heads_of(rng, dt, lead, hk, D, layout)
    qw, kw = rnd(rng, dt, D), rnd(rng, "f32", D)
    table = dbs.rotary_table(60, dim) if dim else torch.zeros((60, 0), device=DEV)
    p = rng.integers(0, 60, lead).astype(np.int32)
    p.reshape(-1)[::997] = [-1, 60, 5][n % 3]
    pos = torch.from_numpy(p).to(DEV)
    out = dbs.norm_rotary(q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    good = (p >= 0) & (p < 60)
    eps, t, pc = np.float64(np.float32(1e-5)), f64(table), np.where(good, p, 0)
    for got, x, w in ((out[0], q, qw), (out[1], k, kw)):
        ref, mag = norm_ref(f64(x), f64(w), t, pc, il, eps)
        ref[~good, :, :dim] = NAN
        close(got, ref, 32 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
    x = q.clone()
    assert torch.equal(dbs.norm_rotary(x, None, qw, None, table, pos, eps=1e-5, interleaved=il, q_out=x)[0].nan_to_num(7), out[0].nan_to_num(7))
    # into a cache
    page, slots = 16, rng.permutation(n + 40)[:n].astype(np.int32)
    slots[::501] = -1
    kc = torch.zeros((n // page + 4, page, hk, D), dtype=DT[dt], device=DEV)
    vc = torch.ones_like(kc)
    rk, rv = kc.flatten(0, 1).clone(), vc.flatten(0, 1).clone()
    qo = dbs.norm_rotary_append(q, k, v, qw, kw, table, pos, kc, vc, ints(slots), eps=1e-5, interleaved=il)
    assert torch.equal(qo.nan_to_num(7), out[0].nan_to_num(7))
    take = torch.from_numpy(slots >= 0).to(DEV)
    at = ints(slots).long()[take]
    rk[at], rv[at] = out[1].reshape(-1, hk, D)[take], v.reshape(-1, hk, D)[take]
    assert torch.equal(kc.flatten(0, 1).nan_to_num(7), rk.nan_to_num(7)) and torch.equal(vc.flatten(0, 1), rv)
    # the gradient (its chains are no longer here: 17 heads of 10,000 tokens are 56 turns of 3040 groups of lanes)
    qg, kg = heads_of(rng, dt, lead, hq, D, "plain"), heads_of(rng, dt, lead, hk, D, layout)
    pos = torch.from_numpy(pc).to(DEV)
    got = dbs.norm_rotary_gradient(qg, kg, q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    for dx, dw, g, y, w in ((got[0], got[2], qg, q, qw), (got[1], got[3], kg, k, kw)):
        ref, mag, wref, wmag = grad_ref(f64(g), f64(y), f64(w), t, pc, il, eps)
        close(dx, ref, 64 * E * mag + U[dt] * np.abs(ref) + ETA[dt])
        close(dw, wref, 192 * E * wmag + E * np.abs(wref) + 1e-30)
    again = dbs.norm_rotary_gradient(qg, kg, q, k, qw, kw, table, pos, eps=1e-5, interleaved=il)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_norm_rotary_gradient_against_differences():
    """d/ds of sum(G * norm_rotary(x + s d)) at 0 by central differences in 64 bits (the forward reference, checked
    above); their own error is h^2 / 6 times a third derivative of about 40 here, and rounding 2^-52 / h of sums of
    about 100: with h = 1e-4 below 1e-6."""
    rng = np.random.default_rng(5)
    x, G, d = rng.standard_normal((3, 2, 16)).astype(np.float32), rng.standard_normal((3, 2, 16)).astype(np.float32), rng.standard_normal((3, 2, 16))
    w, dw = rng.standard_normal(16).astype(np.float32), rng.standard_normal(16)
    table, pos = dbs.rotary_table(20, 16), ints([4, 0, 19])
    eps, t, p, h = np.float64(np.float32(1e-5)), f64(table), pos.cpu().numpy(), 1e-4

    def value(s, u):
        return (G.astype(np.float64) * norm_ref(x + s * d, w + u * dw, t, p, False, eps)[0]).sum()

    dx, _, dwt, _ = dbs.norm_rotary_gradient(*(torch.from_numpy(a).to(DEV) if a is not None else None for a in (G, None, x, None, w, None)),
                                             table, pos, eps=1e-5)
    for got, want in (((f64(dx) * d).sum(), (value(h, 0) - value(-h, 0)) / (2 * h)), ((f64(dwt) * dw).sum(), (value(0, h) - value(0, -h)) / (2 * h))):
        assert abs(got - want) < 1e-4                                         # 96 and 16 products of fp32 results of magnitude below 10


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page,D,odd", [(1, 64, False), (16, 128, False), (24, 80, False), (5, 33, True)])
def test_norm_rotary_append(dt, page, D, odd):
    rng = np.random.default_rng(page * 100 + D)
    n, hq, hkv, pages = 11, 6, 2, -(-20 // page)
    q, k, v = (heads_of(rng, dt, (n,), h, D, "odd" if odd else "plain") for h in (hq, hkv, hkv))
    kc, vc = rnd(rng, dt, pages, page, hkv, D), rnd(rng, dt, pages, page, hkv, D)
    before = kc.clone(), vc.clone()
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    slots[3], slots[7] = -1, pages * page
    table, pos = dbs.rotary_table(64, D // 2 * 2), torch.from_numpy(rng.integers(0, 64, n).astype(np.int32)).to(DEV)
    qw, kw = rnd(rng, dt, D), rnd(rng, dt, D)
    out = dbs.norm_rotary_append(q, k, v, qw, kw, table, pos, kc, vc, ints(slots), eps=1e-6)
    qo, ko = dbs.norm_rotary(q, k, qw, kw, table, pos, eps=1e-6)
    assert torch.equal(out, qo)
    for got, base, new in ((kc, before[0], ko), (vc, before[1], v)):
        ref = base.clone().flatten(0, 1)
        for i, s in enumerate(slots):
            if 0 <= s < pages * page:
                ref[s] = new[i]
        assert torch.equal(got.flatten(0, 1), ref)


def test_norm_rotary_outside_the_table_and_what_is_not_finite():
    rng = np.random.default_rng(8)
    q, w, table = rnd(rng, "f32", 6, 2, 32), rnd(rng, "f32", 32), dbs.rotary_table(10, 16)
    ok = dbs.norm_rotary(q, None, w, None, table, ints([0, 1, 2, 3, 4, 5]))[0]
    out = dbs.norm_rotary(q, None, w, None, table, ints([0, 10, -1, 3, 4, 5]))[0]
    assert torch.isnan(out[1:3, :, :16]).all() and torch.equal(out[1:3, :, 16:], ok[1:3, :, 16:])
    assert torch.equal(out[[0, 3, 4, 5]], ok[[0, 3, 4, 5]])
    q[2, 1, 5], q[4, 0, 31] = NAN, INF
    out = dbs.norm_rotary(q, None, w, None, table, ints([0, 1, 2, 3, 4, 5]))[0]
    assert torch.isnan(out[2, 1]).all() and torch.isnan(out[4, 0, 31])
    rest = torch.ones(6, 2, dtype=torch.bool, device=DEV)
    rest[2, 1] = rest[4, 0] = False
    assert torch.equal(out[rest], ok[rest])
    zero = dbs.norm_rotary(torch.zeros_like(q), None, w, None, table, ints([0, 1, 2, 3, 4, 5]))[0]
    assert (zero == 0).all()
    g = dbs.norm_rotary_gradient(ok, None, torch.zeros_like(q), None, w, None, table, ints([0, 1, 2, 3, 4, 5]))
    assert torch.isfinite(g[0]).all() and (g[2] == 0).all()


# ---- attention with a window and sinks ----


def window_ref(q, k, v, kv, tl, window, sinks, scale, table=None, page=0):
    """out, the sum of p |v|, and lse, in 64 bits."""
    B, T, H, D = q.shape
    G = H // k.shape[2]
    o, mag, lse = np.zeros((B, T, H, D)), np.zeros((B, T, H, D)), np.full((B, T, H), -INF)
    for b in range(B):
        n, first = kv[b], kv[b] - tl[b]
        if table is None:
            kb, vb = k[b, :n], v[b, :n]
        else:
            at = np.clip(table[b], 0, k.shape[0] - 1)
            kb, vb = k[at].reshape(-1, *k.shape[2:])[:n], v[at].reshape(-1, *v.shape[2:])[:n]
        for t in range(tl[b]):
            p = first + t
            if p < 0:
                continue
            j = np.arange(p + 1)
            j = j[(p - j < window) | (j < sinks)]
            for h in range(H):
                x = kb[j, h // G] @ q[b, t, h] * scale
                top = x.max()
                e = np.exp(x - top)
                o[b, t, h], mag[b, t, h] = e @ vb[j, h // G] / e.sum(), e @ np.abs(vb[j, h // G]) / e.sum()
                lse[b, t, h] = top + np.log(e.sum())
    return o, mag, lse


def window_inputs(rng, dt, B, T, hq, hkv, D, S, page, extra=2):
    q = rnd(rng, dt, B, T, hq, D)
    if not page:
        return q, rnd(rng, dt, B, S, hkv, D), rnd(rng, dt, B, S, hkv, D), None
    per = -(-S // page)
    pages = B * per + extra
    table = rng.permutation(pages)[:B * per].astype(np.int32).reshape(B, per)
    return q, rnd(rng, dt, pages, page, hkv, D), rnd(rng, dt, pages, page, hkv, D), table


def check_window(dt, q, k, v, table, kv, tl, window, sinks, scale=None, **kw):
    out, lse = dbs.window_attention(q, k, v, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table),
                                    scale=scale, return_lse=True, **kw)
    s = 1 / np.sqrt(q.shape[-1]) if scale is None else scale
    ref, mag, rl = window_ref(f64(q), f64(k), f64(v), kv, tl, window, sinks, s, table)
    close(out, ref, (U[dt] + 3e-4) * mag + U[dt] * np.abs(ref) + ETA[dt])
    close(lse, rl, 4e-4)
    again = dbs.window_attention(q, k, v, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table),
                                 scale=scale)
    assert torch.equal(again, out)
    return out, lse


WINDOW_CASES = [
    # B, T, hq, hkv, D, S, page, window, sinks
    (1, 1, 1, 1, 64, 1, 0, 1, 0), (1, 1, 4, 1, 128, 300, 0, 64, 4), (2, 1, 8, 2, 128, 513, 16, 100, 0), (3, 1, 5, 1, 96, 200, 24, 64, 70),
    (2, 1, 16, 1, 64, 400, 8, 399, 3), (1, 1, 32, 2, 256, 150, 16, 33, 1), (2, 2, 8, 1, 128, 260, 16, 130, 5), (2, 3, 10, 2, 80, 77, 16, 20, 2),
    (3, 4, 4, 4, 64, 300, 64, 128, 16), (2, 5, 12, 2, 128, 700, 16, 257, 4), (1, 17, 2, 2, 128, 333, 16, 50, 0), (2, 33, 6, 1, 128, 200, 32, 40, 9),
    (1, 64, 8, 1, 64, 500, 16, 200, 4), (2, 130, 4, 2, 128, 130, 16, 1000, 0), (1, 300, 1, 1, 128, 300, 0, 64, 4), (1, 257, 3, 1, 64, 400, 128, 128, 130),
    (2, 100, 7, 1, 128, 150, 16, 31, 1), (1, 200, 5, 1, 256, 200, 16, 90, 4), (2, 65, 2, 1, 256, 300, 0, 100, 20), (1, 140, 4, 4, 40, 140, 8, 17, 2),
    (1, 9, 130, 1, 64, 40, 16, 16, 1), (2, 70, 4, 2, 128, 100, 5, 33, 3), (1, 50, 4, 2, 64, 100, 1, 33, 3), (1, 6, 3, 1, 33, 60, 16, 20, 2),
    (2, 40, 2, 2, 7, 60, 3, 20, 2), (1, 600, 2, 1, 128, 700, 256, 1, 0), (1, 520, 8, 2, 128, 520, 16, 128, 0),
    (1, 40, 4, 1, 64, 2000, 16, 1500, 4), (2, 30, 4, 2, 128, 2100, 24, 2100, 0), (1, 20, 2, 2, 256, 1500, 0, 1000, 30), (3, 8, 8, 1, 128, 1300, 64, 1200, 64)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,hq,hkv,D,S,page,window,sinks", WINDOW_CASES)
def test_window_attention(dt, B, T, hq, hkv, D, S, page, window, sinks):
    rng = np.random.default_rng(B * 7 + T * 31 + hq + D + S)
    q, k, v, table = window_inputs(rng, dt, B, T, hq, hkv, D, S, page)
    check_window(dt, q, k, v, table, [S] * B, [min(T, S)] * B, window, sinks)
    tl = [int(rng.integers(0, T + 1)) for _ in range(B)]
    kv = [int(rng.integers(0, S + 1)) for _ in range(B)]
    check_window(dt, q, k, v, table, kv, tl, window, sinks, scale=0.2)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,page", [(1, 4, 16), (3, 2, 0), (40, 4, 16), (200, 2, 16), (150, 2, 5)])
def test_window_what_is_not_seen_takes_no_part(dt, T, hq, page):
    """NaN and infinities before the windows, behind the entries, in other tokens' places: rows that do not see them."""
    rng = np.random.default_rng(T + hq)
    B, D, S, window, sinks = 2, 128, 420, 60, 3
    q, k, v, table = window_inputs(rng, dt, B, T, hq, 1, D, S, page)
    kv, tl = [390, 300], [T, T - T // 3]
    ref = check_window(dt, q, k, v, table, kv, tl, window, sinks)

    def spoil(c, b, j, value):
        if table is None:
            c[b, j] = value
        else:
            c[int(table[b, j // page]), j % page] = value

    k2, v2 = k.clone(), v.clone()
    for b in range(B):
        lo = max(0, kv[b] - tl[b] - window + 1)
        for i, j in enumerate([*range(sinks, lo), *range(kv[b], S)]):          # seen by no token
            for c in (k2, v2):
                spoil(c, b, j, (NAN, INF, -INF)[(i + b) % 3])
    out, lse = dbs.window_attention(q, k2, v2, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table),
                                    return_lse=True)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    # the entry of one token (of sequence 0) is spoiled: rows before it, and rows whose window is past it, stay
    t = T // 2
    j = kv[0] - tl[0] + t
    for value in (NAN, INF):
        k3, v3 = k.clone(), v.clone()
        spoil(v3, 0, j, value)
        got = dbs.window_attention(q, k3, v3, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table))
        sees = torch.arange(T, device=DEV)
        sees = (sees >= t) & (sees < t + window)
        clean = torch.ones((B, T), dtype=torch.bool, device=DEV)
        clean[0] = ~sees
        o, mag, _ = window_ref(f64(q), f64(k), f64(v), kv, tl, window, sinks, D**-0.5, table)
        at = clean.cpu().numpy()
        close(got[clean], o[at], (U[dt] + 3e-4) * mag[at] + U[dt] * np.abs(o[at]))
        hit = got[0][sees]
        assert torch.isnan(hit).all() if value != value else (torch.isinf(hit) & (hit > 0)).all()
        spoil(k3, 0, j, NAN)
        got = dbs.window_attention(q, k3, v3, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table))
        close(got[clean], o[at], (U[dt] + 3e-4) * mag[at] + U[dt] * np.abs(o[at]))
        assert torch.isnan(got[0][sees]).all()


@pytest.mark.parametrize("T", [1, 5, 60, 300])
def test_window_layouts_and_given_outputs(T):
    """Strides other than the usual, an output among others, rows behind the last token, scales of any sign."""
    rng = np.random.default_rng(T)
    B, hq, hkv, D, S, page = 2, 4, 2, 64, 330, 16
    q, k, v, table = window_inputs(rng, "bf16", B, T, hq, hkv, D, S, page)
    kv, tl = [S, 321], [T, (T + 1) // 2]
    ref = check_window("bf16", q, k, v, table, kv, tl, 50, 4)[0]
    q2 = q.transpose(1, 2).contiguous().transpose(1, 2)
    both = torch.empty((k.shape[0], hkv, 2, page, D), dtype=q.dtype, device=DEV)          # heads before entries, K and V side by side
    both[:, :, 0], both[:, :, 1] = k.transpose(1, 2), v.transpose(1, 2)
    k2, v2 = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    wide = torch.full((B, T, hq, D + 8), 7.0, dtype=q.dtype, device=DEV)
    out = dbs.window_attention(q2, k2, v2, ints(kv), 50, sinks=4, q_lens=ints(tl), page_table=ints(table), out=wide[..., :D])
    assert torch.equal(out, ref) and (wide[..., D:] == 7.0).all() and (out[1, tl[1]:] == 0).all()
    odd = torch.full((B, T, hq, D + 3), 7.0, dtype=q.dtype, device=DEV)
    out = dbs.window_attention(q2, k2, v2, ints(kv), 50, sinks=4, q_lens=ints(tl), page_table=ints(table), out=odd[..., 1:D + 1])
    assert torch.equal(out, ref) and (odd[..., D + 1:] == 7.0).all() and (odd[..., 0] == 7.0).all()
    check_window("bf16", q, k, v, table, kv, tl, 50, 4, scale=-0.1)
    check_window("bf16", q, k, v, table, kv, tl, 50, 4, scale=0.0)
    # the page table's other numbers are clamped, and those that no token needs are not looked at
    t2 = table.copy()
    lo = min(kv[0] - T, kv[1] - tl[1]) - 50
    t2[:, 1:max(1, lo // page)] = -5
    out = dbs.window_attention(q, k, v, ints(kv), 50, sinks=4, q_lens=ints(tl), page_table=ints(t2))
    assert torch.equal(out, ref)


class waits_run_out:
    """Waits of that block of each kernel (-2: of all) run out, after a millisecond."""

    def __init__(self, block):
        self.block = block

    def __enter__(self):
        assert dbs._lib.load().dbs_debug_operator_waits(1_000_000, self.block) == 0

    def __exit__(self, *_):
        torch.cuda.synchronize()
        assert dbs._lib.load().dbs_debug_operator_waits(2_000_000_000, -1) == 0


@pytest.mark.parametrize("B,T,hq,hk,D,S,window", [(2, 1, 8, 2, 128, 900, 400), (40, 1, 4, 4, 64, 200, 100), (1, 3, 4, 2, 256, 300, 200),
                                                  (2, 90, 8, 2, 128, 700, 150), (1, 300, 4, 1, 64, 300, 100), (2, 100, 2, 2, 256, 200, 90),
                                                  (3, 1500, 2, 2, 128, 1500, 200)])
def test_window_that_gives_up_leaves_nan(B, T, hq, hk, D, S, window):
    """All rows that a block whose wait ran out had in hand or still ahead are NaN, the others as ever, and so is the
    next call."""
    rng = np.random.default_rng(B + T)
    q, k, v, table = window_inputs(rng, "f16", B, T, hq, hk, D, S, 16)
    dbs.operators_check()

    def call():
        return dbs.window_attention(q, k, v, ints([S] * B), window, sinks=3, page_table=ints(table), out=torch.full_like(q, 5.0), return_lse=True)

    clean, lse = call()
    assert dbs.operators_check() == 0
    for block in (-2, 0, 1):
        with waits_run_out(block):
            got, gl = call()
        assert dbs.operators_check() == 4 and dbs.operators_check() == 0
        nan = torch.isnan(got)
        assert (nan.all(3) == nan.any(3)).all() and (nan.any(3) == torch.isnan(gl)).all()
        nan = nan.any(3)
        assert nan.all() if block == -2 else nan.any()
        assert torch.equal(got[~nan], clean[~nan]) and torch.equal(gl[~nan], lse[~nan])
        again, al = call()
        assert torch.equal(again, clean) and torch.equal(al, lse)


def test_window_of_everything_is_plain_attention():
    rng = np.random.default_rng(12)
    q, k, v, table = window_inputs(rng, "f16", 2, 24, 8, 2, 64, 300, 16)
    a = dbs.window_attention(q, k, v, ints([300, 211]), 1 << 40, sinks=1 << 40, page_table=ints(table))
    b = dbs.tree_attention(q, k, v, ints([300, 211]), page_table=ints(table))
    o, mag, _ = window_ref(f64(q), f64(k), f64(v), [300, 211], [24, 24], 1 << 40, 0, 0.125, table)
    for got in (a, b):
        close(got, o, (U["f16"] + 3e-4) * mag + U["f16"] * np.abs(o))


# ---- pages ----


class Pool:
    """The page table by the book, one sequence after another."""

    def __init__(self, batch, per, pages, page):
        self.table, self.kv, self.refs, self.page = np.full((batch, per), -7, np.int32), np.zeros(batch, np.int32), np.zeros(pages, np.int32), page

    def device(self):
        return [ints(self.table), ints(self.kv), ints(self.refs)]

    def resize(self, lens, columns=0):
        B, per = self.table.shape
        page, old = self.page, self.kv.copy()
        status, slots = np.zeros(B, np.int32), np.full((B, columns), -1, np.int32)
        for b in range(B):
            if 0 <= lens[b] < self.kv[b]:
                for c in range(-(-lens[b] // page), -(-self.kv[b] // page)):
                    self.refs[self.table[b, c]] -= 1
                self.kv[b] = lens[b]
        free, asked, cut = np.flatnonzero(self.refs == 0), 0, self.refs.copy()
        for b in range(B):
            n, had = lens[b], self.kv[b]
            if n <= had:
                continue
            if n > per * page:
                status[b] = 3
                continue
            if had % page and cut[self.table[b, had // page]] > 1:
                status[b] = 2
                continue
            new = range(-(-had // page), -(-n // page))
            asked += len(new)
            if len(new) and asked > len(free):
                status[b] = 1
                continue
            for c, p in zip(new, free[asked - len(new):asked]):
                self.table[b, c], self.refs[p] = p, 1
            self.kv[b] = n
            for i in range(min(columns, n - old[b])):
                j = old[b] + i
                slots[b, i] = self.table[b, j // page] * page + j % page
        return status, slots

    def fork(self, parents, children, *caches):
        lens, taken, asked, status = self.kv.copy(), set(), 0, []
        free, page = np.flatnonzero(self.refs == 0), self.page
        for p, c in zip(parents, children):
            if not (0 <= p < len(lens) and 0 <= c < len(lens)) or lens[c] > 0 or c in taken:
                status.append(2)
                continue
            taken.add(c)
            n, rest = int(lens[p]) // page, int(lens[p]) % page
            if rest:
                asked += 1
                if asked > len(free):
                    status.append(1)
                    continue
            for i in range(n):
                self.table[c, i] = self.table[p, i]
                self.refs[self.table[p, i]] += 1
            if rest:
                f = int(free[asked - 1])
                self.table[c, n], self.refs[f] = f, 1
                for x in caches:
                    x[:, f, :rest] = x[:, int(self.table[p, n]), :rest]
            self.kv[c] = lens[p]
            status.append(0)
        return np.array(status, np.int32)

    def same(self, state):
        for got, want in zip(state, (self.table, self.kv, self.refs)):
            assert np.array_equal(got.cpu().numpy(), want)

    def consistent(self):
        count = np.zeros(len(self.refs), np.int32)
        for b, n in enumerate(self.kv):
            for c in range(-(-int(n) // self.page)):
                count[self.table[b, c]] += 1
        assert np.array_equal(count, self.refs)


@pytest.mark.parametrize("batch,per,pages,page", [(1, 4, 3, 1), (5, 9, 30, 16), (40, 12, 200, 7), (1500, 3, 3000, 4), (30, 64, 70000, 16), (6, 3, 4, 24)])
def test_cache_resize_walk(batch, per, pages, page):
    """Random growth, cuts and releases, short of pages now and then."""
    rng = np.random.default_rng(batch + pages)
    pool = Pool(batch, per, pages, page)
    if pages > 60000:                                                      # pages far back: the first are taken by others
        pool.refs[:50000] = 9
    state = pool.device()
    for turn in range(10):
        kind = rng.integers(0, 5, batch)
        lens = np.where(kind == 0, -1, np.where(kind == 1, 0, np.where(kind == 2, pool.kv + rng.integers(0, page + 2, batch),
                                                                       rng.integers(0, per * page + 2, batch)))).astype(np.int32)
        columns = [0, 1, 5, 300][turn % 4]
        status, slots = dbs.cache_resize(*state, ints(lens), page, columns=columns)
        want, where = pool.resize(lens, columns)
        assert np.array_equal(status.cpu().numpy(), want) and np.array_equal(slots.cpu().numpy(), where)
        pool.same(state)
        if pages <= 60000:
            pool.consistent()
    assert dbs.cache_resize(*state, ints([0] * batch), page)[1] is None
    pool.resize([0] * batch)
    pool.same(state)


CACHES = [(1, 2, 8, "bf16", 4), (3, 2, 64, "f16", 5), (2, 1, 33, "bf16", 5), (2, 3, 5, "u8", 5), (2, 2, 40, "f32", 5)]


def make_caches(rng, layers, heads, D, dt, dims, pages, page):
    shape = (layers, pages, page, heads, D)
    if dt == "u8":
        k, v = (torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).to(DEV) for _ in range(2))
    else:
        k, v = rnd(rng, dt, *shape), rnd(rng, dt, *shape)
    return (k[0], v[0]) if dims == 4 else (k, v)


def plain(c):
    """[layers, pages, page, heads, D] on the host."""
    return (c if c.dim() == 5 else c[None]).cpu().clone()


@pytest.mark.parametrize("layers,heads,D,dt,dims", CACHES)
@pytest.mark.parametrize("page,pages", [(1, 40), (16, 40), (24, 40), (5, 25)])
def test_cache_fork(layers, heads, D, dt, dims, page, pages):
    rng = np.random.default_rng(layers + D + page)
    pool = Pool(12, 9, pages, page)
    pool.resize(np.array([3 * page, 2 * page + page // 2, 1, 0, 5 * page + max(page - 1, 0), 0, 0, 0, 0, 0, 0, 0]))
    k, v = make_caches(rng, layers, heads, D, dt, dims, pages, page)
    state, hk, hv = pool.device(), plain(k), plain(v)
    for parents, children in (([1], [5]), ([0, 1, 1, 4, 2, 3], [6, 7, 8, 9, 10, 11]), ([1, 4], [1, 3])):
        status = dbs.cache_fork(k, v, *state, ints(parents), ints(children))
        assert np.array_equal(status.cpu().numpy(), pool.fork(parents, children, hk, hv))
        pool.same(state)
        pool.consistent()
        assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)
    # the same child twice, numbers outside, a child of an empty parent
    lens = np.full(12, -1, np.int32)
    lens[[5, 6, 7, 8]] = 0
    dbs.cache_resize(*state, ints(lens), page)
    pool.resize(lens)
    for parents, children in (([1, 4, 0], [5, 5, 5]), ([-1, 12, 0, 1, 2, 3], [6, 6, -1, 12, 2**31 - 1, 7]), ([6, 1, 6], [6, 8, 7])):
        status = dbs.cache_fork(k, v, *state, ints(parents), ints(children))
        assert np.array_equal(status.cpu().numpy(), pool.fork(parents, children, hk, hv))
        pool.same(state)
        pool.consistent()
        assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)
    assert dbs.cache_fork(k, v, *state, ints([]), ints([])).shape == (0,)
    pool.same(state)


@pytest.mark.parametrize("n,first", [(1023, 0), (1024, 0), (1025, 0), (1500, 0), (5, 17000), (700, 40000)])
def test_cache_fork_of_many_and_far_pages(n, first):
    """As many as one block has threads, and more; free pages behind those of `first` that others own; too few of them in the end."""
    rng = np.random.default_rng(n)
    pool = Pool(n + 60, 3, first + n // 2 + 90, 4)
    pool.refs[:first] = 3
    pool.resize(np.concatenate([rng.integers(1, 12, 40), np.zeros(n + 20, int)]))
    k, v = make_caches(rng, 1, 1, 8, "f16", 5, len(pool.refs), 4)
    state, hk, hv = pool.device(), plain(k), plain(v)
    parents, children = rng.integers(0, 42, n), 40 + rng.permutation(n + 20)[:n]
    children[rng.integers(0, n, 5)] = children[0]
    status = dbs.cache_fork(k, v, *state, ints(parents.tolist()), ints(children.tolist()))
    want = pool.fork(parents.tolist(), children.tolist(), hk, hv)
    assert np.array_equal(status.cpu().numpy(), want) and (n < 100 or set(want.tolist()) == {0, 1, 2})
    pool.same(state)
    assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)
    lens = np.where(rng.random(n + 60) < 0.3, 0, -1).astype(np.int32)
    lens[40:50] = 11
    status, slots = dbs.cache_resize(*state, ints(lens.tolist()), 4, columns=12)
    s, w = pool.resize(lens, 12)
    assert np.array_equal(status.cpu().numpy(), s) and np.array_equal(slots.cpu().numpy(), w)
    pool.same(state)


def test_cache_resize_of_long_sequences():
    """Thousands of pages cut, and taken, by a few sequences; refs that start at an odd address."""
    pages, page = 30000, 8
    pool = Pool(5, 9000, pages, page)
    base = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
    state = [ints(pool.table), ints(pool.kv), base[1:]]
    for lens in ([60000, 3, 0, 50001, -1], [100, 72000, 9, 0, 0], [0, 71999, 72001, 5, 72000], [0, 0, 0, 0, 0]):
        status, slots = dbs.cache_resize(*state, ints(lens), page, columns=3000)
        s, w = pool.resize(lens, 3000)
        assert np.array_equal(status.cpu().numpy(), s) and np.array_equal(slots.cpu().numpy(), w)
        pool.same(state)
        pool.consistent()


def test_cache_fork_short_of_pages_and_growth_into_a_shared_page():
    pool = Pool(6, 4, 5, 8)
    pool.resize([8, 13, 5, 0, 0, 0])
    rng = np.random.default_rng(2)
    k, v = make_caches(rng, 2, 1, 16, "f16", 5, 5, 8)
    state, hk, hv = pool.device(), plain(k), plain(v)
    status = dbs.cache_fork(k, v, *state, ints([1, 2, 0]), ints([3, 4, 5]))          # one free page: for the first of the two
    want = pool.fork([1, 2, 0], [3, 4, 5], hk, hv)
    assert want.tolist() == [0, 1, 0] and np.array_equal(status.cpu().numpy(), want)
    pool.same(state)
    assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)
    # cut inside a shared full page, then grown: refused; once the other has gone it may grow
    for lens, want in (([4, -1, -1, -1, -1, -1], [0] * 6), ([6, -1, -1, -1, -1, -1], [2, 0, 0, 0, 0, 0]), ([6, -1, -1, -1, -1, 0], [0] * 6)):
        status, slots = dbs.cache_resize(*state, ints(lens), 8, columns=3)
        s, w = pool.resize(lens, 3)
        assert s.tolist() == want and np.array_equal(status.cpu().numpy(), s) and np.array_equal(slots.cpu().numpy(), w)
        pool.same(state)


@pytest.mark.parametrize("layers,heads,D,dt,dims", CACHES)
@pytest.mark.parametrize("T,page", [(1, 16), (6, 16), (40, 5), (700, 24), (3, 0)])
def test_cache_compact(layers, heads, D, dt, dims, T, page):
    rng = np.random.default_rng(T + D + page)
    B, S = 4, T + 50
    per = -(-S // page) if page else 1
    pages, size = (B * per + 1, page) if page else (B, S)
    k, v = make_caches(rng, layers, heads, D, dt, dims, pages, size)
    table = rng.permutation(pages)[:B * per].astype(np.int32).reshape(B, per) if page else np.arange(B, dtype=np.int32)[:, None]
    kv, tree = [S, S - 7, min(20, T), 0], [T, max(T // 2, 1), T, T]
    acc = np.full((B, T), -1, np.int32)
    for b in range(B):
        take = np.flatnonzero(rng.random(T) < [0.5, 0.9, 0.3, 1.0][b])
        acc[b, :len(take)] = take
    if T == 6:
        acc[0], acc[1], acc[2] = [0, 2, 2, 3, 4, 5], [1, 0, 2, 3, 4, 5], [0, 3, 6, 7, 8, 9]      # ends where it does not ascend, or leaves the tree
    lens = np.array([T if T == 40 else min(int((acc[b] >= 0).sum()), [T, T, 4, T][b]) for b in range(B)], np.int32)
    hk, hv, want = plain(k), plain(v), []
    for b in range(B):
        tr = min(tree[b], kv[b])
        first, n = kv[b] - tr, 0
        for i in range(lens[b]):
            a = acc[b, i]
            if not 0 <= a < tr or (i and a <= acc[b, i - 1]):
                break
            for x in (hk, hv):
                x[:, table[b, (first + i) // size], (first + i) % size] = x[:, table[b, (first + a) // size], (first + a) % size]
            n += 1
        want.append(first + n)
    lens_in = ints(kv)
    got = dbs.cache_compact(k, v, lens_in, ints(tree), ints(acc), ints(lens) if T != 40 else None, page_table=ints(table) if page else None)
    assert got.tolist() == want and lens_in.tolist() == kv
    assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)


def test_caches_of_other_layouts():
    """Heads before entries, layers between: forked and compacted as the plain layout is."""
    rng = np.random.default_rng(9)
    layers, pages, page, heads, D = 3, 20, 8, 2, 24
    base = [make_caches(rng, layers, heads, D, "bf16", 5, pages, page) for _ in range(1)][0]
    other = [torch.full((pages, heads, layers, page, D + 8), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    views = [o[..., :D].permute(2, 0, 3, 1, 4) for o in other]
    for a, b in zip(views, base):
        a.copy_(b)
    pools = [Pool(5, 4, pages, page) for _ in range(2)]
    states = []
    for p, c in zip(pools, (base, views)):
        p.resize([11, 30, 5, 0, 0])
        states.append(p.device())
        dbs.cache_fork(*c, *states[-1], ints([1, 0]), ints([3, 4]))
        dbs.cache_compact(*c, states[-1][1], ints([3, 6, 2, 6, 3]), ints([[0, 2, -1], [1, 3, 5], [1, -1, -1], [0, 1, 4], [1, 2, -1]]), page_table=states[-1][0])
    assert all(torch.equal(a, b) for a, b in zip(*states)) and all(torch.equal(a, b) for a, b in zip(base, views))
    assert all((o[..., D:] == 3.0).all() for o in other)


# ---- a run of them together ----


def test_a_step_of_drafted_tokens_forked_and_cut_back():
    """Grow, append, attend, keep what was accepted, fork and go on: against a dense cache of each sequence's own."""
    rng = np.random.default_rng(21)
    B, hq, hkv, D, page, pages, window, sinks, dt = 4, 4, 2, 64, 8, 64, 20, 2, "bf16"
    state = [torch.full((B, 12), -1, dtype=torch.int32, device=DEV), ints([0] * B), ints([0] * pages)]
    kc, vc = (torch.full((pages, page, hkv, D), NAN, dtype=DT[dt], device=DEV) for _ in range(2))
    table, w = dbs.rotary_table(128, D), rnd(rng, "f32", D)
    kept = {b: [] for b in range(B)}                                       # (k, v) of every entry
    live = [0, 1]

    def step(counts, accepted):
        T = max(counts)
        lens = state[1].cpu().numpy()
        want = np.array([lens[b] + counts[b] if b in live else -1 for b in range(B)], np.int32)
        status, slots = dbs.cache_resize(*state, ints(want), page, columns=T)
        assert (status == 0).all()
        q, k, v = rnd(rng, dt, B, T, hq, D), rnd(rng, dt, B, T, hkv, D), rnd(rng, dt, B, T, hkv, D)
        pos = ints(lens[:, None] + np.arange(T, dtype=np.int32))
        qt = dbs.norm_rotary_append(q, k, v, w, w, table, pos, kc, vc, slots)
        kt = dbs.norm_rotary(k, None, w, None, table, pos)[0]
        tl = np.array([counts[b] if b in live else 0 for b in range(B)], np.int32)
        out = dbs.window_attention(qt, kc, vc, state[1], window, sinks=sinks, q_lens=ints(tl), page_table=state[0])
        for b in live:
            kept[b] += [(f64(kt[b, i]), f64(v[b, i])) for i in range(counts[b])]
            dense = [np.stack([e[i] for e in kept[b]])[None] for i in range(2)]
            ref, mag, _ = window_ref(f64(qt[b:b + 1]), *dense, [len(kept[b])], [counts[b]], window, sinks, D**-0.5)
            close(out[b], ref[0], (U[dt] + 3e-4) * mag[0] + U[dt] * np.abs(ref[0]))
        acc = np.full((B, T), -1, np.int32)
        for b in live:
            acc[b, :len(accepted[b])] = accepted[b]
            first = len(kept[b]) - counts[b]
            kept[b] = kept[b][:first] + [kept[b][first + a] for a in accepted[b]]
        new = dbs.cache_compact(kc, vc, state[1], ints(tl), ints(acc), page_table=state[0])
        assert (dbs.cache_resize(*state, new, page)[0] == 0).all()
        assert state[1].tolist() == [len(kept[b]) for b in range(B)]

    step([37, 21, 0, 0], {0: range(37), 1: range(21)})
    step([6, 4, 0, 0], {0: [0, 2, 5], 1: [0]})
    assert dbs.cache_fork(kc, vc, *state, ints([0, 1]), ints([2, 3])).tolist() == [0, 0]
    kept[2], kept[3], live = list(kept[0]), list(kept[1]), [0, 1, 2, 3]
    step([5, 9, 7, 3], {0: [0, 1, 4], 1: [0, 3, 8], 2: [0, 6], 3: [0, 1, 2]})
    step([1, 1, 1, 1], {b: [0] for b in range(4)})
    assert dbs.cache_resize(*state, ints([0] * B), page)[0].tolist() == [0] * B and (state[2] == 0).all() and dbs.operators_check() == 0


def test_captured_and_replayed_on_another_stream():
    """One step captured in a graph and replayed gives what calls on a stream give."""
    rng = np.random.default_rng(31)
    B, T, hq, hkv, D, page = 3, 2, 8, 2, 128, 16
    q, k, v = rnd(rng, "f16", B, T, hq, D), rnd(rng, "f16", B, T, hkv, D), rnd(rng, "f16", B, T, hkv, D)
    w, table, pos = rnd(rng, "f16", D), dbs.rotary_table(200, D), ints(np.array([[50, 51], [9, 10], [120, 121]]))
    pool = Pool(B + 1, 10, 40, page)
    pool.resize([50, 9, 120, 0])
    kc0, vc0 = make_caches(rng, 1, hkv, D, "f16", 4, 40, page)

    def run(state, kc, vc):
        grown, slots = dbs.cache_resize(*state, ints_grow, page, columns=T)
        qt = dbs.norm_rotary_append(q, k, v, w, w, table, pos, kc, vc, slots[:B].contiguous())
        out = dbs.window_attention(qt, kc, vc, state[1][:B], 40, sinks=4, page_table=state[0][:B])
        forked = dbs.cache_fork(kc, vc, *state, one, three)
        lens = dbs.cache_compact(kc, vc, state[1], trees, accepted, page_table=state[0])
        cut, _ = dbs.cache_resize(*state, lens, page)
        grads = dbs.norm_rotary_gradient(qt, k, q, k, w, w, table, pos)
        return [grown, slots, qt, out, forked, lens, cut, *grads]

    ints_grow, one, three = ints([52, 11, 122, -1]), ints([1]), ints([3])
    trees, accepted = ints([2, 2, 2, 0]), ints([[1, -1], [0, 1], [0, -1], [-1, -1]])
    state = pool.device()
    kc, vc = kc0.clone(), vc0.clone()
    want = [t.clone() for t in (*run(state, kc, vc), *state, kc, vc)]
    side = torch.cuda.Stream()
    state2, kc2, vc2 = pool.device(), kc0.clone(), vc0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(state2, kc2, vc2)
    for _ in range(3):
        for t, f in zip((*state2, kc2, vc2), (*pool.device(), kc0, vc0)):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, *state2, kc2, vc2), want):
            assert torch.equal(a, b)


# ---- what is not finite and seen, calls at once, far and many places ----


@pytest.mark.parametrize("T,hq,hk,D,S,page", [(1, 8, 2, 128, 4000, 16), (1, 4, 4, 64, 300, 5), (7, 4, 2, 256, 900, 0), (40, 4, 1, 64, 2000, 16),
                                              (600, 8, 2, 128, 1500, 16), (900, 2, 1, 256, 960, 64), (20, 3, 1, 40, 500, 3)])
def test_window_not_finite_values_that_all_rows_see(T, hq, hk, D, S, page):
    """Values are taken column by column, and sums (lse) do not take them at all."""
    rng = np.random.default_rng(T + D)
    q, k, v, table = window_inputs(rng, "bf16", 1, T, hq, hk, D, S, page)
    kw = dict(sinks=2, page_table=None if table is None else ints(table), return_lse=True)
    out, lse = dbs.window_attention(q, k, v, ints([S]), S, **kw)
    at = (0, 1) if table is None else (int(table[0, 0]), 1) if page > 1 else (int(table[0, 1]), 0)     # entry 1, a sink
    for column, value in ((3, NAN), (D - 1, INF)):
        v2 = v.clone()
        v2[at][..., column] = value
        got, gl = dbs.window_attention(q, k, v2, ints([S]), S, **kw)
        rest = [c for c in range(D) if c != column]
        assert torch.equal(gl, lse) and torch.equal(got[..., rest], out[..., rest])
        assert not torch.isfinite(got[..., column]).any()
    got, gl = dbs.window_attention(q, k, torch.full_like(v, NAN), ints([S]), S, **kw)
    assert torch.equal(gl, lse) and torch.isnan(got).all()
    # from the middle on: rows before it stay, the others have NaN
    v2, p = v.clone(), S - (T + 1) // 2
    flat = v2 if table is None else v2[torch.from_numpy(table[0]).long().to(DEV)].reshape(1, -1, hk, D)
    flat[:, p:] = NAN
    if table is not None:
        v2[torch.from_numpy(table[0]).long().to(DEV)] = flat.reshape(-1, page, hk, D)
    got, gl = dbs.window_attention(q, k, v2, ints([S]), S, **kw)
    before = p - (S - T)
    o, mag, _ = window_ref(f64(q), f64(k), f64(v), [S], [T], S, 2, D**-0.5, table)
    close(got[:, :before], o[:, :before], (U["bf16"] + 3e-4) * mag[:, :before] + U["bf16"] * np.abs(o[:, :before]))
    assert torch.isnan(got[:, before:]).all() and torch.equal(gl, lse)


def test_calls_at_once_on_two_streams_and_in_two_graphs():
    """Two sets of tensors, their calls on two streams and as two graphs replayed at once, give what each gives alone."""
    rng = np.random.default_rng(41)
    page, D = 16, 128
    sets = []
    for B, T, hq, hkv, S in ((2, 90, 8, 2, 700), (5, 1, 8, 1, 1500)):
        q, k, v, table = window_inputs(rng, "f16", B, T, hq, hkv, D, S, page)
        x = rnd(rng, "f16", B, T, hkv, D)
        pool = Pool(B + 1, k.shape[0] // B, 3 * k.shape[0], page)
        pool.resize([100 + 7 * b for b in range(B)] + [0])
        sets.append(dict(q=q, k=k, v=v, table=ints(table), kv=ints([S - 3 * b for b in range(B)]), x=x, w=rnd(rng, "f16", D),
                         rot=dbs.rotary_table(256, D), pos=ints(rng.integers(0, 256, (B, T))), state=pool.device(), start=pool.device(),
                         lens=ints([100 + 20 * b for b in range(B)] + [-1]), caches=make_caches(rng, 1, hkv, D, "f16", 4, 3 * k.shape[0], page),
                         parents=ints([B - 1]), children=ints([B])))

    def run(s, **kw):
        for a, b in zip(s["state"], s["start"]):
            a.copy_(b)
        out = dbs.window_attention(s["q"], s["k"], s["v"], s["kv"], 600, sinks=4, page_table=s["table"], return_lse=True, **kw)
        grads = dbs.norm_rotary_gradient(s["q"], s["x"], s["q"], s["x"], s["w"], s["w"], s["rot"], s["pos"], **kw)
        turned_ = dbs.norm_rotary(s["q"], s["x"], s["w"], s["w"], s["rot"], s["pos"], **kw)
        grown = dbs.cache_resize(*s["state"], s["lens"], page, columns=40, **kw)
        forked = dbs.cache_fork(*s["caches"], *s["state"], s["parents"], s["children"], **kw)
        return [*out, *grads, *turned_, *grown, forked, *s["state"]]

    want = [[t.clone() for t in run(s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append([t.clone() for t in run(s)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    # a stream given by hand
    out = dbs.window_attention(sets[0]["q"], sets[0]["k"], sets[0]["v"], sets[0]["kv"], 600, sinks=4, page_table=sets[0]["table"], stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(out, want[0][0])
    graphs, got = [], []
    for s, stream in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got.append(run(s))
        graphs.append(g)
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert dbs.operators_check() == 0


def test_caches_past_32_bits():
    """Entries behind 2^32 elements: appended, seen, forked and compacted as those of a small cache are."""
    rng = np.random.default_rng(51)
    page, heads, D, hq, dt = 16, 8, 128, 16, "bf16"
    per, far = 4, (1 << 32) // (16 * 8 * 128) + 5                          # the numbers of the pages in use begin there
    big = [torch.empty((far + 12, page, heads, D), dtype=DT[dt], device=DEV) for _ in range(2)]
    small = [torch.zeros((12, page, heads, D), dtype=DT[dt], device=DEV) for _ in range(2)]
    for c in big:
        c[far:] = 0
    B, T, w, table = 2, 40, rnd(rng, "f32", D), dbs.rotary_table(64, D)
    q, k, v = rnd(rng, dt, B, T, hq, D), rnd(rng, dt, B, T, heads, D), rnd(rng, dt, B, T, heads, D)
    pos = ints(np.tile(np.arange(T), (B, 1)))
    results = []
    for caches, first in ((small, 0), (big, far)):
        refs = torch.zeros(first + 12, dtype=torch.int32, device=DEV)
        refs[:first] = 1                                                   # (taken by others)
        state = [torch.full((B + 1, per), -1, dtype=torch.int32, device=DEV), ints([0] * (B + 1)), refs]
        status, slots = dbs.cache_resize(*state, ints([T, T, -1]), page, columns=T)
        qt = dbs.norm_rotary_append(q, k, v, w, w, table, pos, *caches, slots[:B])
        outs = [dbs.window_attention(qt, *caches, state[1][:B], 25, sinks=2, page_table=state[0][:B]),
                dbs.window_attention(qt[:, -1:], *caches, state[1][:B], 25, sinks=2, page_table=state[0][:B])]
        forked = dbs.cache_fork(*caches, *state, ints([1]), ints([2]))
        lens = dbs.cache_compact(*caches, state[1], ints([7, 8, 0]), ints([[0, 2, 5], [3, 4, 7], [-1, -1, -1]]), page_table=state[0])
        results.append([status, torch.where(slots < 0, -1, slots - first * page), torch.where(state[0] < 0, -1, state[0] - first), state[1], refs[first:],
                        qt, *outs, forked, lens, *(c[first:] for c in caches)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    del big, caches, results
    torch.cuda.empty_cache()


def test_many_sequences():
    """More sequences than a grid's second and third dimension have blocks, or one less where that is the limit."""
    rng = np.random.default_rng(61)
    B, D = 70000, 64
    q, k, v, _ = window_inputs(rng, "f16", B, 1, 2, 1, D, 3, 0)
    kv = rng.integers(0, 4, B)
    out = dbs.window_attention(q, k, v, ints(kv), 2, sinks=1)
    some = np.r_[0:20, 32760:32780, 65530:65545, B - 20:B]
    at = torch.from_numpy(some).to(DEV)
    o, mag, _ = window_ref(f64(q[at]), f64(k[at]), f64(v[at]), kv[some], [1] * len(some), 2, 1, D**-0.5)
    close(out[at], o, (U["f16"] + 3e-4) * mag + U["f16"] * np.abs(o) + ETA["f16"])
    n, page = 65535, 2
    pool = Pool(2 * n + 1, 1, n + 5, page)
    pool.resize([1] + [0] * (2 * n))
    state = pool.device()
    caches = make_caches(rng, 1, 1, 8, "f16", 4, n + 5, page)
    host = [plain(c).clone() for c in caches]
    parents, children = np.zeros(n, np.int32), np.arange(1, n + 1, dtype=np.int32)
    assert np.array_equal(dbs.cache_fork(*caches, *state, ints(parents), ints(children)).cpu().numpy(), pool.fork(parents, children, *host))
    pool.same(state)
    assert all(torch.equal(plain(c), h) for c, h in zip(caches, host))
    lens = np.where(np.arange(2 * n + 1) < 3, 2, -1).astype(np.int32)
    lens[n:] = 1
    want = pool.resize(lens)
    assert np.array_equal(dbs.cache_resize(*state, ints(lens), page)[0].cpu().numpy(), want[0])
    pool.same(state)


def test_inputs_that_require_a_gradient_are_refused():
    q = torch.zeros((1, 2, 2, 64), dtype=torch.float16, device=DEV, requires_grad=True)
    x, w, table, i = q.detach(), torch.ones(64, device=DEV, requires_grad=True), dbs.rotary_table(4, 64), ints([0, 1])
    one = ints([2])
    for call in (lambda: dbs.norm_rotary(q, None, None, None, table, i), lambda: dbs.norm_rotary(x, None, w, None, table, i),
                 lambda: dbs.norm_rotary_gradient(x, None, x, None, w, None, table, i), lambda: dbs.window_attention(q, x, x, one, 4),
                 lambda: dbs.window_attention(x, x, q, one, 4), lambda: dbs.cache_compact(q, x, one, one, ints([[0]]))):
        with pytest.raises(dbs.DbsError, match="requires a gradient"):
            call()
    with torch.no_grad():
        assert torch.equal(dbs.norm_rotary(q, None, w, None, table, i)[0], torch.zeros_like(x))
    with pytest.raises(dbs.DbsError):
        dbs.window_attention(x, x, x, one, 4, out=x)


@pytest.mark.parametrize("outside", [-1, -7, 11, 2**31 - 1])
def test_cache_compact_passes_over_pages_that_are_none(outside):
    """Pages of a drafted tree that are none: nothing is read from or written to another page for them, and the lengths are as ever."""
    rng = np.random.default_rng(31)
    B, per, page, pages, T = 3, 3, 4, 11, 12
    k, v = make_caches(rng, 2, 2, 24, "f16", 5, pages, page)
    table = (1 + rng.permutation(9)).astype(np.int32).reshape(B, per)      # the first and the last page belong to others
    table[0, 1] = table[1, 0] = table[2, 2] = outside
    acc = np.array([[1, 2, 4, 5, 7, 8, 9, 11, -1, -1, -1, -1], [0, 2, 3, 5, 6, 9, 10, 11, -1, -1, -1, -1], [3, 4, 8, 9, 10, 11, -1, -1, -1, -1, -1, -1]], np.int32)
    hk, hv, want = plain(k), plain(v), []
    for b in range(B):
        path = [a for a in acc[b] if a >= 0]
        for i, a in enumerate(path):
            src, dst = table[b, a // page], table[b, i // page]
            if 0 <= src < pages and 0 <= dst < pages:
                for x in (hk, hv):
                    x[:, dst, i % page] = x[:, src, a % page]
        want.append(len(path))
    got = dbs.cache_compact(k, v, ints([T] * B), ints([T] * B), ints(acc), page_table=ints(table))
    assert got.tolist() == want
    assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)


@pytest.mark.parametrize("page,T", [(1, 2), (16, 5), (4, 256), (1, 300)])
def test_cache_compact_of_lists_with_anything_behind_their_end(page, T):
    """Sequences that fill their rows of the table, lists far longer than the tree that ascend again behind their end: what stands
    there asks for no entry (places behind the tree's lie behind the row, and of the last sequence behind the table)."""
    rng = np.random.default_rng(page + T)
    B, most = 3, 1000
    per = -(-(T + 30) // page)
    S, pages = per * page, 3 * per
    k, v = make_caches(rng, 2, 1, 16, "bf16", 5, pages, page)
    table = rng.permutation(pages).astype(np.int32).reshape(B, per)
    acc = np.tile(np.arange(T, dtype=np.int32), (B, -(-most // T)))[:, :most]          # 0 .. T - 1, again and again
    acc[1, min(1, T - 1)] = T - 1                                                      # 0, T - 1, then it no longer ascends
    acc[2, 0] = 1
    acc[2, 1:T] = np.arange(1, T)                                                      # 1, and that again
    hk, hv = plain(k), plain(v)
    kept = [T, 2, 1]
    for b in range(B):
        for i in range(kept[b]):
            for x in (hk, hv):
                x[:, table[b, (S - T + i) // page], (S - T + i) % page] = x[:, table[b, (S - T + acc[b, i]) // page], (S - T + acc[b, i]) % page]
    got = dbs.cache_compact(k, v, ints([S] * B), ints([T] * B), ints(acc), page_table=ints(table))
    assert got.tolist() == [S - T + n for n in kept]
    assert torch.equal(plain(k), hk) and torch.equal(plain(v), hv)


@pytest.mark.parametrize("T,hq,hk,D,S,page", [(1, 8, 2, 128, 4000, 16), (1, 4, 1, 64, 9000, 0), (1, 2, 1, 256, 3000, 16), (2, 4, 2, 64, 2500, 5), (1, 4, 2, 33, 600, 16),
                                              (7, 4, 2, 128, 900, 16), (40, 4, 1, 64, 3000, 16), (100, 2, 2, 128, 2000, 24), (30, 4, 1, 256, 1500, 64)])
@pytest.mark.parametrize("loud,odd", [(5, 2), (2, 5)])
def test_what_a_row_sees_counts_however_little_it_weighs(T, hq, hk, D, S, page, loud, odd):
    """One entry's score is some 300 above all others (320 or more in base e, so that their weights are 0 in fp32), another entry in
    another part of the line has a NaN key, or a value that is not finite: the rows are NaN, and lse where the key is."""
    q, one = torch.ones((1, T, hq, D), dtype=torch.bfloat16, device=DEV), dict(dtype=torch.bfloat16, device=DEV)
    shape = (-(-S // page), page, hk, D) if page else (1, S, hk, D)
    table = torch.arange(shape[0], dtype=torch.int32, device=DEV)[None] if page else None
    loud, odd = loud * (S - T) // 6, odd * (S - T) // 6
    k, v = torch.zeros(shape, **one), torch.ones(shape, **one)
    k.view(-1, hk, D)[loud] = 64
    kw = dict(page_table=table, return_lse=True)
    attend = [lambda: dbs.window_attention(q, k, v, ints([S]), S, **kw), lambda: dbs.tree_attention(q, k, v, ints([S]), **kw)]
    for f in attend:
        out, lse = f()
        assert (out == 1).all() and torch.isfinite(lse).all()
    flat = v.view(-1, hk, D)
    for value in (NAN, INF):
        flat[odd, :, 1] = value
        out, lse = attend[0]()
        assert not torch.isfinite(out[..., 1]).any() and torch.isfinite(lse).all()
        assert (out[..., [c for c in range(D) if c != 1]] == 1).all()
    flat[odd] = 1
    k.view(-1, hk, D)[odd] = NAN
    for f in attend:
        out, lse = f()
        assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_outputs_within_the_inputs_buffers():
    """Heads of q, k and v side by side in one buffer: turned in place and attended into v's place, bit for bit as with tensors of their own; views
    that lie on an input in part are refused."""
    rng = np.random.default_rng(8)
    B, T, hq, hk, D = 2, 40, 4, 4, 64
    fused = rnd(rng, "bf16", B, T, hq + 2 * hk, D)
    q, k, v = fused.split([hq, hk, hk], 2)
    w, table, pos = rnd(rng, "bf16", D), dbs.rotary_table(64, D), ints([list(range(T))] * B)
    own = dbs.norm_rotary(q.clone(), k.clone(), w, w, table, pos)
    kc, vc = own[1].contiguous(), v.clone()
    want = dbs.window_attention(own[0], kc, vc, ints([T] * B), 17)
    dbs.norm_rotary(q, k, w, w, table, pos, q_out=q, k_out=k)
    assert torch.equal(q, own[0]) and torch.equal(k, own[1])
    assert dbs.window_attention(q, kc, vc, ints([T] * B), 17, out=v) is v and torch.equal(v, want)
    one, heads = fused.flatten(), (B, T, hq, D)
    for bad in (fused[:, :, 1:1 + hq], fused[:, :, 2:2 + hq], one[64:].as_strided(heads, q.stride()), one.as_strided(heads, (T * hq * D, hq * D, D, 1))):
        with pytest.raises(dbs.DbsError):
            dbs.window_attention(q, kc, vc, ints([T] * B), 17, out=bad)
        with pytest.raises(dbs.DbsError):
            dbs.norm_rotary(q, None, w, None, table, pos, q_out=bad)
        with pytest.raises(dbs.DbsError):
            dbs.rotary(q, None, table, pos, q_out=bad)
    with pytest.raises(dbs.DbsError):
        dbs.norm_rotary(q, k, w, w, table, pos, q_out=k)
    with pytest.raises(dbs.DbsError):
        dbs.window_attention(q, kc, vc, ints([T] * B), 17, out=vc)
    lens = ints([5, 6, 7, 8])
    with pytest.raises(dbs.DbsError):
        dbs.cache_resize(ints([[-1, -1]] * 3), lens[:3], ints([0] * 8), lens[1:], 4)
    with pytest.raises(dbs.DbsError):
        dbs.cache_compact(kc, kc, ints([T] * B), ints([2] * B), ints([[1]] * B))


def test_cache_resize_of_many_long_sequences():
    """More sequences than a block has threads, cut by numbers of pages that keep a warp's lanes busy for different times."""
    rng = np.random.default_rng(12)
    batch, per, page = 1100, 70, 1
    pool = Pool(batch, per, 60000, page)
    state = pool.device()
    for turn in range(6):
        lens = rng.integers(0, per + 2, batch) if turn % 2 == 0 else np.where(rng.random(batch) < 0.2, -1, rng.integers(0, 4, batch) * pool.kv // 4)
        status, slots = dbs.cache_resize(*state, ints(lens.tolist()), page, columns=3)
        want, where = pool.resize(lens, 3)
        assert np.array_equal(status.cpu().numpy(), want) and np.array_equal(slots.cpu().numpy(), where)
        pool.same(state)
        pool.consistent()


# ---- more units than blocks, longer lines ----


def window_ref_gpu(q, k, v, kv, tl, window, sinks, table):
    """window_ref of all rows in 64 bits on the GPU, a kv head of a sequence and 512 tokens at a time."""
    B, T, H, D = q.shape
    hk = k.shape[2]
    o, mag = (torch.zeros((B, T, H, D), dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((B, T, H), -INF, dtype=torch.float64, device=DEV)
    for b in range(B):
        n, first = int(kv[b]), int(kv[b] - tl[b])
        kb, vb = (x[b] if table is None else x[torch.from_numpy(table[b]).long().to(DEV)].flatten(0, 1) for x in (k, v))
        for t0 in range(max(0, -first), int(tl[b]), 512):
            t1 = min(int(tl[b]), t0 + 512)
            p, j = torch.arange(first + t0, first + t1, device=DEV)[:, None], torch.arange(n, device=DEV)
            hide = (j > p) | ((p - j >= window) & (j >= sinks))
            for h in range(hk):
                G = slice(h * (H // hk), (h + 1) * (H // hk))
                x = torch.einsum("tgd,jd->gtj", q[b, t0:t1, G].double(), kb[:n, h].double()) * D**-0.5
                x.masked_fill_(hide, -INF)
                lse[b, t0:t1, G] = torch.logsumexp(x, -1).T
                e = torch.softmax(x, -1)
                o[b, t0:t1, G] = torch.einsum("gtj,jd->tgd", e, vb[:n, h].double())
                mag[b, t0:t1, G] = torch.einsum("gtj,jd->tgd", e, vb[:n, h].double().abs())
    return o, mag, lse


def check_window_gpu(dt, q, k, v, table, kv, tl, window, sinks):
    out, lse = dbs.window_attention(q, k, v, ints(kv), window, sinks=sinks, q_lens=ints(tl), page_table=None if table is None else ints(table), return_lse=True)
    o, mag, rl = window_ref_gpu(q, k, v, kv, tl, window, sinks, table)
    assert ((out.double() - o).abs() <= (U[dt] + 3e-4) * mag + U[dt] * o.abs() + ETA[dt]).all()
    assert ((lse == rl) | ((lse.double() - rl).abs() <= 4e-4)).all()


MANY_UNITS = [
    # B, T, hq, hkv, D, S, page, window, sinks: three units of rows and more for a multiprocessor
    (64, 70, 32, 8, 64, 200, 16, 50, 3), (64, 70, 32, 8, 128, 230, 16, 90, 0), (40, 70, 32, 8, 256, 150, 64, 60, 5), (96, 40, 8, 8, 128, 300, 0, 1000, 0),
    (1, 4100, 32, 8, 128, 4100, 16, 700, 4), (1, 4100, 32, 8, 64, 4200, 0, 1500, 70), (1, 2050, 16, 8, 256, 2050, 32, 300, 4), (1, 4100, 16, 8, 256, 4100, 16, 300, 4), (2, 3000, 40, 8, 128, 3300, 24, 64, 0)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,hq,hkv,D,S,page,window,sinks", MANY_UNITS)
def test_window_of_more_units_than_blocks(dt, B, T, hq, hkv, D, S, page, window, sinks):
    """Blocks go from unit to unit, some of them without tokens, without entries, or with fewer entries than tokens."""
    rng = np.random.default_rng(B + T + D)
    q, k, v, table = window_inputs(rng, dt, B, T, hq, hkv, D, S, page)
    if B <= 2:
        kv, tl = np.array([S, S - 100][:B]), np.array([T, T - 77][:B])
    else:
        kv, tl = rng.integers(0, S + 1, B), np.where(rng.random(B) < 0.2, 0, rng.integers(0, T + 1, B))
        kv[:4], tl[:4] = [0, T // 2, S, 1], [T, T, T, 1]
    check_window_gpu(dt, q, k, v, table, kv.tolist(), tl.tolist(), window, sinks)


@pytest.mark.parametrize("B,T,hq,hk,D,S,window,least", [(1, 4100, 32, 8, 128, 4100, 200, 500), (64, 70, 32, 8, 64, 100, 60, 500), (1, 2050, 16, 8, 256, 2050, 100, 4),
                                                        (1, 4100, 16, 8, 256, 4100, 100, 250)])
def test_window_that_gives_up_among_its_units_leaves_nan(B, T, hq, hk, D, S, window, least):
    """A block whose wait ran out leaves NaN in all units that it had ahead, the others have theirs.  Units are 256 rows, of heads of 256
    128; the first of a call have the last tokens, which may be few.  With 152 blocks: 520 units, three and more a block, two of them
    full; 1024 units, half of them of 6 tokens; 264 units, of which block 0 has the first alone, of 2050 - 32 * 64 tokens of 2 heads; 520."""
    rng = np.random.default_rng(B + T)
    q, k, v, table = window_inputs(rng, "bf16", B, T, hq, hk, D, S, 16)
    dbs.operators_check()

    def call():
        return dbs.window_attention(q, k, v, ints([S] * B), window, sinks=3, page_table=ints(table), out=torch.full_like(q, 5.0), return_lse=True)

    clean, lse = call()
    assert dbs.operators_check() == 0
    for block in (-2, 0, 70):
        with waits_run_out(block):
            got, gl = call()
        assert dbs.operators_check() == 4 and dbs.operators_check() == 0
        nan = torch.isnan(got)
        assert (nan.all(3) == nan.any(3)).all() and (nan.any(3) == torch.isnan(gl)).all()
        nan = nan.any(3)
        assert nan.all() if block == -2 else least <= nan.sum().item() <= nan.numel() // 20
        assert torch.equal(got[~nan], clean[~nan]) and torch.equal(gl[~nan], lse[~nan])
        again, al = call()
        assert torch.equal(again, clean) and torch.equal(al, lse)


def test_window_values_that_are_not_finite_among_many_units():
    """NaN in entries that only some rows see, in a prompt of more units than blocks: the rows that see them are NaN, the others as without."""
    rng = np.random.default_rng(77)
    T, hq, hk, D, window = 4100, 32, 8, 128, 300
    q, k, v, _ = window_inputs(rng, "bf16", 1, T, hq, hk, D, T, 0)
    clean, lse = dbs.window_attention(q, k, v, ints([T]), window, sinks=2, return_lse=True)
    sees = torch.zeros(T, dtype=torch.bool, device=DEV)
    for j in (700, 701, 2303, 4000):
        v[:, j] = NAN
        sees[j:j + window] = True
    got, gl = dbs.window_attention(q, k, v, ints([T]), window, sinks=2, return_lse=True)
    assert torch.equal(gl, lse) and torch.isnan(got[0, sees]).all()
    # rows near them are made anew, without the rounding of probabilities (2^-8 of sum p |v|, which is below 2 here; both results are rounded)
    assert ((got[0, ~sees].float() - clean[0, ~sees].float()).abs() <= 2**-7 * clean[0, ~sees].float().abs() + 2**-7).all()
    far = ~sees
    for j in (700, 701, 2303, 4000):
        far[max(0, j - 300):j + window + 300] = False
    assert torch.equal(got[0, far], clean[0, far])


LONG_LINES = [
    # B, T, hq, hkv, D, S, page, window, sinks: few rows, up to sixteen blocks to a line
    (1, 1, 8, 1, 128, 2000, 16, 5000, 0), (1, 1, 8, 2, 128, 4001, 16, 3900, 4), (1, 1, 32, 8, 128, 9001, 0, 8192, 4), (1, 1, 16, 1, 64, 9001, 8, 9000, 0),
    (1, 2, 8, 8, 64, 6000, 16, 5000, 100), (1, 1, 8, 1, 256, 5003, 16, 5003, 0), (2, 1, 16, 8, 256, 3001, 0, 2500, 7), (1, 3, 5, 1, 96, 7777, 5, 7000, 3),
    (1, 1, 8, 2, 128, 4000, 1, 3000, 0), (3, 4, 4, 4, 128, 4500, 64, 4000, 1), (1, 16, 1, 1, 64, 8000, 24, 100000, 0)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,hq,hkv,D,S,page,window,sinks", LONG_LINES)
def test_window_of_few_rows_over_long_lines(dt, B, T, hq, hkv, D, S, page, window, sinks):
    rng = np.random.default_rng(T + D + S)
    q, k, v, table = window_inputs(rng, dt, B, T, hq, hkv, D, S, page)
    check_window_gpu(dt, q, k, v, table, [S] + [S - 1000 * b - 13 for b in range(1, B)], [T] * B, window, sinks)


@pytest.mark.parametrize("T", [2, 7])
def test_window_long_line_with_values_that_are_not_finite(T):
    """Few rows over sixteen blocks: rows before the first entry that is not finite are as without it, the others NaN."""
    rng = np.random.default_rng(T)
    S, hq, hk, D = 4000, 8, 4, 128
    q, k, v, table = window_inputs(rng, "bf16", 1, T, hq, hk, D, S, 16)
    before = T // 2
    v2, p = v.clone(), S - T + before
    assert before > 0
    flat = v2[torch.from_numpy(table[0]).long().to(DEV)].reshape(1, -1, hk, D)
    flat[:, p:] = NAN
    v2[torch.from_numpy(table[0]).long().to(DEV)] = flat.reshape(-1, 16, hk, D)
    got, gl = dbs.window_attention(q, k, v2, ints([S]), S, sinks=2, page_table=ints(table), return_lse=True)
    o, mag, lse = window_ref_gpu(q, k, v, [S], [T], S, 2, table)
    assert torch.isnan(got[:, before:]).all() and ((gl - lse).abs() <= 4e-4).all()
    assert ((got[:, :before].double() - o[:, :before]).abs() <= (U["bf16"] + 3e-4) * mag[:, :before] + U["bf16"] * o[:, :before].abs()).all()


@pytest.mark.parametrize("B,T,hq,hk,D,S,page", [(1, 1, 8, 2, 128, 4000, 16), (1, 1, 4, 1, 64, 40000, 0), (1, 2, 4, 2, 64, 2500, 5), (1, 1, 4, 2, 33, 600, 16), (1, 40, 4, 1, 64, 3000, 16),
                                                (2, 100, 2, 2, 128, 2000, 24), (1, 30, 4, 1, 256, 1500, 64), (3, 7, 2, 2, 128, 5000, 16)])
@pytest.mark.parametrize("loud,odd", [(5, 2), (2, 5)])
def test_tree_values_count_however_little_they_weigh(B, T, hq, hk, D, S, page, loud, odd):
    """As above for drafted tokens: one value that is not finite, in the part that all see, in an entry whose weight is 0 in fp32."""
    q, one = torch.ones((B, T, hq, D), dtype=torch.bfloat16, device=DEV), dict(dtype=torch.bfloat16, device=DEV)
    per = -(-S // page) if page else 1
    shape = (B * per, page, hk, D) if page else (B, S, hk, D)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per) if page else None
    k, v = torch.zeros(shape, **one), torch.ones(shape, **one)
    kb, vb = k.view(B, -1, hk, D), v.view(B, -1, hk, D)
    kb[:, loud * (S - T) // 6] = 64
    out, lse = dbs.tree_attention(q, k, v, ints([S] * B), page_table=table, return_lse=True)
    assert (out == 1).all() and torch.isfinite(lse).all()
    for value in (NAN, INF):
        vb[:, odd * (S - T) // 6, :, 1] = value
        got, gl = dbs.tree_attention(q, k, v, ints([S] * B), page_table=table, return_lse=True)
        assert not torch.isfinite(got[..., 1]).any() and torch.equal(gl, lse)
        assert (got[..., [c for c in range(D) if c != 1]] == 1).all()
