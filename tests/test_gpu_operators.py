"""GPU parity of the decoding step's operators against plain 64-bit forms.

Tolerances, from the formulas (u = unit roundoff of the type that a result is
rounded to: 2^-24 fp32, 2^-11 fp16, 2^-8 bf16):
  w4         1e-5 * sum |x (q - z) s| + u |y|: exact products, fp32 sums of at
             most 256 terms a group (8 accumulation steps of 16 in a tensor
             core, each within 2^-22 of the magnitudes) and of the groups
  rotary     3 * 2^-24 (|a cos| + |b sin|) + u |y| + 2^-25 for fp16 (half the
             spacing of its subnormals)
  attention  (u + 3e-4) * sum p |v| + u |out|: probabilities rounded once to the
             caches' type, and fp32 scores, whose error is at most
             head_dim * 2^-23 * scale * sum |q k| (1.1e-4 at head_dim 128,
             1.6e-4 at 256 for N(0,1) inputs), twice (numerator and sum)
  logits     8 * 2^-24 times the sum of the magnitudes that meet, + u |y|
"""
import importlib.util
import math
import os

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
ETA = {"f32": 0.0, "f16": 2.0**-25, "bf16": 0.0}
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


# ---- 4-bit linear layers ----


def w4_inputs(rng, T, m, n, dt, sd, group, zeros, pad=16):
    cols, groups = (n + 1) // 2, -(-n // group)
    q = torch.from_numpy(rng.integers(0, 256, (m, -(-cols // pad) * pad), dtype=np.uint8)).to(DEV)[:, :cols]
    s = torch.from_numpy(rng.uniform(0.001, 0.02, (m, groups)).astype(np.float32)).to(DT[sd]).to(DEV)
    z = torch.from_numpy(rng.integers(0, 16, (m, groups), dtype=np.uint8)).to(DEV) if zeros else None
    return rnd(rng, dt, T, n), q, s, z


def w4_ref(x, q, s, z, group):
    n = x.shape[1]
    qn = q.cpu().numpy()
    w = np.stack([qn & 15, qn >> 4], 2).reshape(qn.shape[0], -1)[:, :n].astype(np.float64)
    zn = np.full(s.shape, 8.0) if z is None else z.cpu().numpy().astype(np.float64)
    w = (w - np.repeat(zn, group, 1)[:, :n]) * np.repeat(f64(s), group, 1)[:, :n]
    xn = f64(x)
    return xn @ w.T, np.abs(xn) @ np.abs(w).T


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,m,n,group,zeros,pad", [
    (1, 1, 1, 32, False, 16), (1, 16, 32, 32, True, 16), (1, 1000, 2051, 64, True, 16), (2, 17, 129, 128, True, 16),
    (3, 130, 4096, 256, False, 16), (7, 33, 1000, 32, True, 1), (8, 64, 512, 64, True, 16), (9, 300, 777, 128, False, 16),
    (24, 515, 1024, 128, True, 16), (33, 48, 640, 64, False, 16), (70, 129, 300, 32, True, 16), (1, 4096, 11008, 128, False, 16),
    (64, 257, 2050, 256, True, 16), (1, 5, 12000, 32, True, 1)])
def test_w4(dt, T, m, n, group, zeros, pad):
    rng = np.random.default_rng(T * 1000 + m + n)
    x, q, s, z = w4_inputs(rng, T, m, n, dt, dt, group, zeros, pad)
    y = dbs.w4_linear(x, q, s, z, group=group)
    assert y.dtype == x.dtype
    ref, mag = w4_ref(x, q, s, z, group)
    close(y, ref, 1e-5 * mag + U[dt] * np.abs(ref) + 1e-30)
    assert torch.equal(y, dbs.w4_linear(x, q, s, z, group=group))           # the same bits again


@pytest.mark.parametrize("sd", ["f32", "f16", "bf16"])
def test_w4_scale_types_strides_and_one_vector(sd):
    rng = np.random.default_rng(3)
    T, m, n, group = 5, 200, 1111, 64
    x, q, s, z = w4_inputs(rng, T, m, n, "f32", sd, group, True)
    wide = torch.full((T, n + 13), NAN, device=DEV)
    wide[:, 3:3 + n] = x
    zw = torch.zeros((m, z.shape[1] + 3), dtype=torch.uint8, device=DEV)
    zw[:, :z.shape[1]] = z
    sw = torch.full((m, s.shape[1] + 1), NAN, dtype=s.dtype, device=DEV)
    sw[:, :s.shape[1]] = s
    out = torch.full((T, m + 7), 5.0, device=DEV)
    y = dbs.w4_linear(wide[:, 3:3 + n], q, sw[:, :s.shape[1]], zw[:, :z.shape[1]], group=group, y=out[:, :m])
    ref, mag = w4_ref(x, q, s, z, group)
    close(y, ref, 1e-5 * mag + U["f32"] * np.abs(ref))
    assert (out[:, m:] == 5.0).all()
    one = dbs.w4_linear(x[2], q, s, z, group=group)
    assert one.shape == (m,)
    close(one, ref[2], 1e-5 * mag[2] + U["f32"] * np.abs(ref[2]))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_w4_what_lies_behind_the_columns_takes_no_part(dt):
    """Codes behind column n (the padding of a row) and scales of no group."""
    rng = np.random.default_rng(4)
    T, m, n, group = 3, 40, 70, 32
    x, q, s, z = w4_inputs(rng, T, m, n, dt, "f32", group, True)
    base = torch.full((m, 64), 255, dtype=torch.uint8, device=DEV)
    base[:, :35] = q
    y = dbs.w4_linear(x, base[:, :35], s, z, group=group)
    ref, mag = w4_ref(x, q, s, z, group)
    close(y, ref, 1e-5 * mag + U[dt] * np.abs(ref))


def test_w4_infinities_stay_with_their_token():
    rng = np.random.default_rng(5)
    x, q, s, z = w4_inputs(rng, 4, 64, 512, "f32", "f32", 128, False)
    q |= 0x88                                                              # every code at least 8
    q |= 0x11                                                              # and none equal to the zero point
    ref, mag = w4_ref(x, q, s, z, 128)
    x[1, 100] = INF
    x[2, 7] = NAN
    x[3, 9] = 3e38
    y = dbs.w4_linear(x, q, s, z, group=128)
    close(y[0], ref[0], 1e-5 * mag[0] + U["f32"] * np.abs(ref[0]))
    assert torch.isinf(y[1]).all() and (y[1] > 0).all() and torch.isnan(y[2]).all()
    big, bm = w4_ref(x[3:4], q, s, z, 128)
    close(y[3:4], big, 1e-5 * bm)


@pytest.mark.parametrize("dt,sd", [("f16", "f32"), ("bf16", "bf16"), ("bf16", "f16"), ("f16", "f16")])
@pytest.mark.parametrize("T,m,n,group,zeros", [
    (13, 128, 256, 128, True), (17, 129, 2051, 64, True), (32, 1, 4096, 256, False), (33, 640, 1000, 32, True), (64, 130, 3001, 128, True),
    (65, 257, 513, 32, False), (24, 19461, 300, 64, True), (200, 1000, 777, 256, True), (31, 2500, 5000, 32, True), (40, 300, 1, 64, True)])
def test_w4_of_several_tokens(dt, sd, T, m, n, group, zeros):
    """Rows and tokens in tiles, columns shared out among blocks or not; x's rows on and off 16-byte boundaries."""
    rng = np.random.default_rng(T + m + n + group)
    x, q, s, z = w4_inputs(rng, T, m, n, dt, sd, group, zeros)
    ref, mag = w4_ref(x, q, s, z, group)
    bound = 1e-5 * mag + U[dt] * np.abs(ref) + ETA[dt] + 1e-30
    for pad, at in ((-n % 8 + 8, 0), (-n % 8 + 9, 1)):
        wide = torch.full((T, n + pad), NAN, dtype=x.dtype, device=DEV)
        wide[:, at:at + n] = x
        out = torch.full((T, m + 3), 7.0, dtype=x.dtype, device=DEV)
        y = dbs.w4_linear(wide[:, at:at + n], q, s, z, group=group, y=out[:, :m])
        close(y, ref, bound)
        assert (out[:, m:] == 7).all()
        assert torch.equal(y, dbs.w4_linear(wide[:, at:at + n], q, s, z, group=group))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_w4_infinities_stay_with_their_token_among_several(dt):
    rng = np.random.default_rng(7)
    x, q, s, z = w4_inputs(rng, 20, 200, 600, dt, "f32", 64, True)
    ref, mag = w4_ref(x, q, s, z, 64)
    x[3, 100], x[11, 599] = INF, NAN
    y = dbs.w4_linear(x, q, s, z, group=64)
    rest = [t for t in range(20) if t not in (3, 11)]
    close(y[rest], ref[rest], 1e-5 * mag[rest] + U[dt] * np.abs(ref[rest]) + ETA[dt])
    w = np.stack([f64(q) % 16, f64(q) // 16], -1).reshape(200, -1)[:, 100] - (f64(z)[:, 100 // 64] % 128)
    assert torch.isnan(y[11]).all()
    got = f64(y[3])
    assert (np.isnan(got) == (w == 0)).all() and (got[w > 0] == INF).all() and (got[w < 0] == -INF).all()


def test_w4_exact_on_whole_numbers():
    """Small whole x and power-of-two scales: every sum is exact in fp32."""
    rng = np.random.default_rng(6)
    x, q, s, z = w4_inputs(rng, 6, 100, 1000, "f32", "f32", 64, True)
    x = torch.from_numpy(rng.integers(-8, 9, (6, 1000)).astype(np.float32)).to(DEV)
    s.fill_(0.5)
    ref, _ = w4_ref(x, q, s, z, 64)
    assert np.array_equal(f64(dbs.w4_linear(x, q, s, z, group=64)), ref)


# ---- rotary positions ----


def table_ref(P, R, base=10000.0, scaling=None, factor=1.0, trained=0.0):
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    f = base ** (-np.arange(0, R, 2) / R)
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        at = lambda beta: R * math.log(trained / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32))), min(R // 2 - 1, math.ceil(at(1)))
        hi = hi if hi > lo else lo + 0.001
        r = np.clip((np.arange(R // 2) - lo) / (hi - lo), 0, 1)
        f = f * (1 - r) + f / factor * r
        amp = 0.1 * math.log(factor) + 1
    a = np.arange(P)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1) * amp


@pytest.mark.parametrize("P,R,kw", [
    (1, 2, {}), (70000, 128, {}), (5000, 64, dict(base=500000.0)), (9000, 128, dict(scaling="linear", factor=4.0)),
    (9000, 96, dict(scaling="ntk", factor=8.0)), (20000, 128, dict(scaling="yarn", factor=16.0, trained=4096)),
    (300, 32, dict(scaling="yarn", factor=2.0, trained=64))])
def test_rotary_table(P, R, kw):
    t = dbs.rotary_table(P, R, **kw)
    # angles in fp64 (one rounding of the frequency and one of the product:
    # 2^-52 of the angle), then rounded to fp32
    close(t, table_ref(P, R, **kw), 2.0**-24 * 1.5 + P * 2.0**-50)


def rot_ref(x, table, pos, R, interleaved, transposed):
    """[b, t, h, d] -> values, magnitudes."""
    y = f64(x).copy()
    mag = np.zeros_like(y)
    tb = f64(table)[pos]                                                   # [b, t, R]
    c, s = tb[:, :, None, :R // 2], tb[:, :, None, R // 2:]
    s = -s if transposed else s
    i = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    j = i + 1 if interleaved else i + R // 2
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    mag[..., i], mag[..., j] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return y, mag


ROT = [(1, 1, 1, 1, 2, 2), (1, 5, 32, 8, 128, 128), (2, 37, 6, 1, 80, 40), (3, 4, 5, 5, 96, 96), (1, 300, 4, 2, 256, 128),
       (2, 9, 3, 1, 33, 22), (1, 17, 2, 2, 64, 24), (4, 64, 8, 2, 64, 64), (1, 3, 2, 1, 16, 0), (1, 1030, 12, 4, 128, 64)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,hq,hk,D,R", ROT)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(dt, B, T, hq, hk, D, R, interleaved):
    rng = np.random.default_rng(B * 100 + T + D)
    table = torch.from_numpy(table_ref(500, max(R, 2)).astype(np.float32)).to(DEV)[:, :R].contiguous()
    pos = rng.integers(0, 500, (B, T)).astype(np.int32)
    pt = torch.from_numpy(pos).to(DEV)
    q, k = rnd(rng, dt, B, T, hq, D), rnd(rng, dt, B, hk, T, D).transpose(1, 2)      # k: heads before tokens
    for transposed in (False, True):
        qo, ko = dbs.rotary(q, k, table, pt, interleaved=interleaved, transposed=transposed)
        for x, y in ((q, qo), (k, ko)):
            ref, mag = rot_ref(x, table, pos, R, interleaved, transposed)
            close(y, ref, 3 * 2.0**-24 * mag + U[dt] * np.abs(ref) + ETA[dt])
            assert torch.equal(y[..., R:], x[..., R:])
    q2 = q.clone()
    again, none = dbs.rotary(q2, None, table, pt, interleaved=interleaved, q_out=q2)  # in place
    assert again is q2 and none is None
    assert torch.equal(q2, dbs.rotary(q, k, table, pt, interleaved=interleaved)[0])


def test_rotary_views_and_positions_outside_the_table():
    """q and k as views of one fused projection; unaligned heads; a position
    outside the table gives NaN in the rotated entries of its token alone."""
    rng = np.random.default_rng(8)
    T, hq, hk, D, R = 6, 4, 2, 20, 12
    table = torch.from_numpy(table_ref(50, R).astype(np.float32)).to(DEV)
    fused = rnd(rng, "bf16", T, (hq + 2 * hk) * D + 1)
    q = fused[:, 1:1 + hq * D].unflatten(1, (hq, D))
    k = fused[:, 1 + hq * D:1 + (hq + hk) * D].unflatten(1, (hk, D))
    pos = np.array([0, 49, 50, 7, -1, 3], np.int32)
    qo, ko = dbs.rotary(q, k, table, torch.from_numpy(pos).to(DEV))
    bad = (pos < 0) | (pos >= 50)
    for x, y in ((q, qo), (k, ko)):
        ref, mag = rot_ref(x[None], table, np.where(bad, 0, pos)[None], R, False, False)
        ref, mag = ref[0], mag[0]
        ref[bad, :, :R] = NAN
        close(y, ref, 3 * 2.0**-24 * mag + U["bf16"] * np.abs(np.nan_to_num(ref)))


def test_rotary_gradient_against_differences():
    """loss = sum w * rotary(x), linear in x: the central difference along v
    with step 1 is the derivative, up to the rounding of 2 n products."""
    rng = np.random.default_rng(9)
    B, T, h, D, R = 2, 11, 3, 48, 32
    table = torch.from_numpy(table_ref(64, R).astype(np.float32) * 1.25).to(DEV)
    pos = torch.from_numpy(rng.integers(0, 64, (B, T)).astype(np.int32)).to(DEV)
    for interleaved in (False, True):
        x, w, v = (rnd(rng, "f32", B, T, h, D) for _ in range(3))
        grad, _ = dbs.rotary(w, None, table, pos, interleaved=interleaved, transposed=True)
        hi, lo = (dbs.rotary(x + e * v, None, table, pos, interleaved=interleaved)[0] for e in (1, -1))
        diff = ((f64(hi) - f64(lo)) / 2 * f64(w)).sum()
        exact = (f64(grad) * f64(v)).sum()
        size = ((np.abs(f64(hi)) + np.abs(f64(lo)) + np.abs(f64(grad)) + 4) * (np.abs(f64(w)) + np.abs(f64(v)))).sum()
        assert abs(diff - exact) <= 4 * 2.0**-24 * size


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,hq,hk,D,R,page", [(1, 4, 1, 64, 64, 16), (5, 32, 8, 128, 128, 16), (77, 6, 2, 80, 40, 24),
                                              (40, 3, 3, 33, 10, 1), (700, 8, 4, 128, 128, 64)])
def test_rotary_append(dt, N, hq, hk, D, R, page):
    rng = np.random.default_rng(N)
    pages = -(-(2 * N + 5) // page)
    table = torch.from_numpy(table_ref(900, R).astype(np.float32)).to(DEV)
    q, k, v = rnd(rng, dt, N, hq, D), rnd(rng, dt, N, hk, D), rnd(rng, dt, N, hk, D)
    kc, vc = rnd(rng, dt, pages, page, hk, D), rnd(rng, dt, pages, hk, page, D).transpose(1, 2)
    pos = rng.integers(0, 900, N).astype(np.int32)
    slots = rng.permutation(pages * page)[:N].astype(np.int32)
    if N > 4:
        slots[1], slots[3] = -1, pages * page                              # padding tokens: nothing is written
    k0, v0 = kc.clone(), vc.clone()
    qo = dbs.rotary_append(q, k, v, table, torch.from_numpy(pos).to(DEV), kc, vc, torch.from_numpy(slots).to(DEV),
                           interleaved=N % 2 == 0)
    ref, mag = rot_ref(q[None], table, pos[None], R, N % 2 == 0, False)
    close(qo, ref[0], 3 * 2.0**-24 * mag[0] + U[dt] * np.abs(ref[0]) + ETA[dt])
    ref, mag = rot_ref(k[None], table, pos[None], R, N % 2 == 0, False)
    left = np.ones(pages * page, bool)
    for i, s in enumerate(slots):
        if 0 <= s < pages * page:
            left[s] = False
            close(kc[s // page, s % page], ref[0, i], 3 * 2.0**-24 * mag[0, i] + U[dt] * np.abs(ref[0, i]) + ETA[dt])
            assert torch.equal(vc[s // page, s % page], v[i])
    keep = torch.from_numpy(left.reshape(pages, page)).to(DEV)
    assert torch.equal(kc[keep], k0[keep]) and torch.equal(vc[keep], v0[keep])


# ---- attention of drafted tokens over a cache ----


def tree_bits(rng, B, T):
    bits = np.zeros((B, T, -(-T // 64)), np.uint64)
    for b in range(B):
        for i in range(T):
            if i:
                bits[b, i] = bits[b, rng.integers(max(0, i - 5), i)]
            bits[b, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return bits


def attn_ref(q, k, v, kv, tl, bits, pages, scale):
    """k, v [pages, page, hk, d] (fp64), pages [B, n]; returns out, sum p|v|, lse.
    Entries that are not seen are never touched."""
    B, T, hq, D = q.shape
    hk = k.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, T, hq), -INF)
    page = k.shape[1]
    for b in range(B):
        j = np.arange(kv[b])
        kb, vb = k[pages[b][j // page], j % page], v[pages[b][j // page], j % page]
        for t in range(tl[b]):
            node = j - (kv[b] - tl[b])
            see = node < 0
            inside = np.clip(node, 0, None)
            see |= (node <= t if bits is None else
                    ((bits[b, t][inside // 64] >> (inside % 64).astype(np.uint64)) & np.uint64(1)).astype(bool))
            if not see.any():
                continue
            for h in range(hq):
                a = kb[see, h // (hq // hk)] @ q[b, t, h] * scale
                top = a.max()
                p = np.exp(a - top)
                lse[b, t, h] = top + np.log(p.sum())
                p /= p.sum()
                out[b, t, h] = p @ vb[see, h // (hq // hk)]
                mag[b, t, h] = p @ np.abs(vb[see, h // (hq // hk)])
    return out, mag, lse


def attn_case(rng, dt, B, T, hq, hk, D, S, page, ragged=True):
    q = rnd(rng, dt, B, T, hq, D)
    if page:
        per = max(1, -(-S // page))
        pages = rng.permutation(B * per).reshape(B, per)
        k, v = rnd(rng, dt, B * per, page, hk, D), rnd(rng, dt, B * per, page, hk, D)
    else:
        pages = np.arange(B)[:, None]
        k, v = rnd(rng, dt, B, S, hk, D), rnd(rng, dt, B, S, hk, D)
    tl = rng.integers(1, T + 1, B) if ragged else np.full(B, T)
    kv = np.array([rng.integers(min(t, S), S + 1) for t in tl]) if ragged else np.full(B, S)
    return q, k, v, pages, kv.astype(np.int32), tl.astype(np.int32)


def dev(a, t=None):
    return torch.from_numpy(np.ascontiguousarray(a) if t is None else np.ascontiguousarray(a).astype(t)).to(DEV)


def attn_check(dt, q, k, v, pages, kv, tl, bits, page, scale=None, **kw):
    out, lse = dbs.tree_attention(q, k, v, dev(kv), None if bits is None else dev(bits.view(np.int64)), tree_lens=dev(tl),
                                  page_table=dev(pages, np.int32) if page else None, scale=scale, return_lse=True, **kw)
    kk, vv = f64(k), f64(v)
    ref, mag, rl = attn_ref(f64(q), kk, vv, kv, tl, bits, pages, q.shape[3]**-0.5 if scale is None else scale)
    close(out, ref, (U[dt] + 3e-4) * mag + U[dt] * np.abs(ref) + 1e-7)
    with np.errstate(invalid="ignore"):
        close(lse, rl, 3e-4 + 1e-6 * np.abs(np.where(np.isinf(rl), 0, rl)))
    assert (f64(out)[np.isinf(rl)] == 0).all()
    return out


ATTN = [(1, 1, 1, 1, 64, 1, 0), (1, 1, 8, 8, 128, 5, 0), (1, 1, 32, 8, 128, 2001, 0), (2, 5, 8, 2, 128, 300, 16),
        (3, 16, 8, 1, 64, 130, 24), (2, 33, 4, 4, 96, 513, 64), (5, 3, 10, 2, 256, 77, 7), (4, 64, 8, 1, 128, 700, 256),
        (1, 64, 16, 2, 256, 190, 16), (7, 12, 12, 4, 128, 1000, 1), (2, 100, 2, 2, 64, 400, 16), (2, 7, 6, 3, 80, 129, 0),
        (2, 9, 4, 2, 36, 150, 5), (3, 4, 2, 1, 33, 65, 0), (1, 1, 5, 5, 1, 9, 0), (40, 1, 16, 4, 128, 260, 16),
        (1, 200, 8, 2, 128, 333, 16), (1, 3, 71, 1, 128, 128, 64), (60, 2, 8, 4, 64, 300, 16), (170, 1, 8, 4, 64, 100, 16),
        (24, 2, 16, 8, 128, 500, 64), (9, 3, 4, 4, 256, 500, 32), (40, 1, 8, 4, 256, 200, 16)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,hq,hk,D,S,page", ATTN)
def test_tree_attention(dt, B, T, hq, hk, D, S, page):
    rng = np.random.default_rng(B * 31 + T * 7 + S)
    q, k, v, pages, kv, tl = attn_case(rng, dt, B, T, hq, hk, D, S, page)
    bits = tree_bits(rng, B, T)
    out = attn_check(dt, q, k, v, pages, kv, tl, bits, page)
    again = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), tree_lens=dev(tl),
                               page_table=dev(pages, np.int32) if page else None)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_tree_attention_chain_scale_and_long(dt):
    rng = np.random.default_rng(11)
    q, k, v, pages, kv, tl = attn_case(rng, dt, 2, 20, 8, 2, 128, 9000, 48)
    attn_check(dt, q, k, v, pages, kv, tl, None, 48, scale=0.05)
    q, k, v, pages, kv, tl = attn_case(rng, dt, 3, 1, 8, 2, 128, 20000, 0)
    attn_check(dt, q, k, v, pages, kv, tl, None, 0)


@pytest.mark.parametrize("T,hq", [(6, 4), (40, 8)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_tree_attention_empty_rows_and_lengths(dt, T, hq):
    """Sequences without entries, without drafted tokens, with fewer entries
    than drafted tokens, with lengths out of range (clamped), and tokens whose
    mask leaves nothing."""
    rng = np.random.default_rng(12)
    B, S, page = 8, 96, 16
    q, k, v, pages, _, _ = attn_case(rng, dt, B, T, hq, 2, 64, S, page)
    kv = np.array([0, 50, 3, S, T, 1, S, 64], np.int32)
    tl = np.array([T, 0, T, 1, T, 1, T, T // 2], np.int32)
    bits = tree_bits(rng, B, T)
    bits[4, T // 2] = 0                       # nothing before the drafted tokens, and none of them
    bits[2, 2] = 0
    attn_check(dt, q, k, v, pages, kv, tl, bits, page)
    over = dbs.tree_attention(q, k, v, dev(kv + np.where(kv == S, 1000, 0).astype(np.int32)), dev(bits.view(np.int64)),
                              tree_lens=dev(tl + np.where(tl == T, 99, 0).astype(np.int32)), page_table=dev(pages, np.int32))
    base = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), tree_lens=dev(tl), page_table=dev(pages, np.int32))
    assert torch.equal(over, base)
    none = dbs.tree_attention(q, k, v, dev(np.minimum(kv, 0) - 3), dev(bits.view(np.int64)), page_table=dev(pages, np.int32))
    assert (none == 0).all()


@pytest.mark.parametrize("T,hq,hk,D", [(5, 4, 2, 128), (48, 8, 1, 128), (9, 8, 4, 64), (20, 4, 1, 256), (3, 2, 1, 40)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_tree_attention_what_is_not_seen_takes_no_part(dt, T, hq, hk, D):
    """NaN and infinities in drafted entries that a token does not see, behind
    the last entry and on unused pages change nothing; for the tokens that see
    such a value they count."""
    rng = np.random.default_rng(13)
    B, S, page = 3, 200, 16
    q, k, v, pages, kv, tl = attn_case(rng, dt, B, T, hq, hk, D, S, page)
    tl[:] = T
    kv[:] = [T, 100 + T, S - 20]
    bits = tree_bits(rng, B, T)
    last = T - 1                                # seen by itself alone
    clean = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), page_table=dev(pages, np.int32))
    for b in range(B):
        j = np.arange(kv[b], pages.shape[1] * page)
        for c in (k, v):
            c[dev(pages[b][j // page]), dev(j % page)] = NAN
        e = kv[b] - 1
        v[int(pages[b][e // page]), e % page, :, 0] = NAN
        v[int(pages[b][e // page]), e % page, :, 1] = INF
        k[int(pages[b][e // page]), e % page, 0, 3] = [NAN, INF, -INF][b]
    got = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), page_table=dev(pages, np.int32))
    assert torch.equal(got[:, :last], clean[:, :last])
    assert torch.isnan(got[:, last, :, 0]).all()
    if hk > 1:
        head = got[:, last, hq // hk:, 1]       # the second kv head's k is finite
        assert torch.isinf(head).all() and torch.equal(got[:, last, hq // hk:, 2:], clean[:, last, hq // hk:, 2:])


@pytest.mark.parametrize("T,hq,hk,D", [(1, 8, 2, 128), (5, 4, 2, 128), (9, 8, 4, 64), (3, 2, 1, 256)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_tree_attention_of_few_rows_with_room_for_a_long_text(dt, T, hq, hk, D):
    """A page table for many more entries than there are: the work is shared out by the lengths."""
    rng = np.random.default_rng(15)
    B, S, page = 6, 900, 16
    q, k, v, pages, kv, tl = attn_case(rng, dt, B, T, hq, hk, D, S, page)
    pages = np.concatenate([pages, np.full((B, 4200), -5)], 1)
    kv[:] = [0, 50, T, S, 1, 700]
    tl[:] = [T, 0, T, T, T, 1]
    bits = tree_bits(rng, B, T)
    bits[2, T // 2] = 0
    attn_check(dt, q, k, v, pages, kv, tl, bits, page)
    table = dev(pages, np.int32)
    clean = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), tree_lens=dev(tl), page_table=table)
    e = S - 1                                   # seen by the last token alone
    v[int(pages[3][e // page]), e % page, :, 0] = NAN
    v[int(pages[3][e // page]), e % page, :, 1] = INF
    got = dbs.tree_attention(q, k, v, dev(kv), dev(bits.view(np.int64)), tree_lens=dev(tl), page_table=table)
    rest = [b for b in range(B) if b != 3]
    assert torch.equal(got[rest], clean[rest]) and torch.equal(got[3, :T - 1], clean[3, :T - 1])
    assert torch.isnan(got[3, T - 1, :, 0]).all() and torch.isinf(got[3, T - 1, :, 1]).all()
    assert torch.equal(got[3, T - 1, :, 2:], clean[3, T - 1, :, 2:])


def test_tree_attention_large_scores_and_views():
    """Scores that grow along the cache (the running maximum moves at every
    entry) and fall; q, caches and out as views with other strides."""
    rng = np.random.default_rng(14)
    for dt, slope in (("f16", 0.02), ("bf16", -0.02), ("f16", 0.2)):
        B, T, hq, hk, D, S = 2, 20, 8, 2, 128, 777
        base = torch.zeros((B, hk, S, 2 * D), dtype=DT[dt], device=DEV)
        k, v = base[..., :D].transpose(1, 2), base[..., D:].transpose(1, 2)
        q0 = rnd(rng, dt, B, T, hq + 3, D)
        q0[..., 0] = 4.0
        k.copy_(rnd(rng, dt, B, S, hk, D))
        k[..., 0] = (torch.arange(S, device=DEV) * slope).to(DT[dt])[None, :, None]
        v.copy_(rnd(rng, dt, B, S, hk, D))
        out = torch.full((B, hq, T, D), 9.0, dtype=DT[dt], device=DEV).transpose(1, 2)
        q = q0[:, :, 2:2 + hq]
        tl, kv = np.array([T, 11], np.int32), np.array([S, 500], np.int32)
        got = attn_check(dt, q, k, v, np.arange(B)[:, None], kv, tl, tree_bits(rng, B, T), 0, out=out)
        assert got is out


def test_tree_attention_page_numbers_out_of_range_are_clamped():
    rng = np.random.default_rng(15)
    q, k, v, pages, kv, tl = attn_case(rng, "bf16", 2, 3, 4, 2, 64, 100, 16, ragged=False)
    bad, good = pages.copy(), pages.copy()
    bad[0, 2], good[0, 2] = 10**6, k.shape[0] - 1
    bad[1, 1], good[1, 1] = -5, 0
    a, b = (dbs.tree_attention(q, k, v, dev(kv), page_table=dev(p, np.int32)) for p in (bad, good))
    assert torch.equal(a, b)


def test_tree_attention_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: pages at its end."""
    rng = np.random.default_rng(16)
    pages, page, hk, D = 34000, 64, 8, 128                                 # 4.5 GB each
    k = torch.empty((pages, page, hk, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    use = np.array([[pages - 1, pages - 3, 5, pages - 2]])
    for c in (k, v):
        c[dev(use[0])] = rnd(rng, "bf16", 4, page, hk, D)
    q = rnd(rng, "bf16", 1, 4, 16, D)
    small_k, small_v = k[dev(use[0])].contiguous(), v[dev(use[0])].contiguous()
    kv = dev(np.array([250], np.int32))
    a = dbs.tree_attention(q, k, v, kv, page_table=dev(use, np.int32))
    b = dbs.tree_attention(q, small_k, small_v, kv, page_table=dev(np.arange(4)[None], np.int32))
    assert torch.equal(a, b)
    slots = dev(np.array([pages * page - 1, 7], np.int32))
    kt, vt = rnd(rng, "bf16", 2, hk, D), rnd(rng, "bf16", 2, hk, D)
    dbs.rotary_append(q[0, :2], kt, vt, dbs.rotary_table(8, D), dev(np.zeros(2, np.int32)), k, v, slots)
    assert torch.equal(v[-1, -1], vt[0]) and torch.equal(k[-1, -1], kt[0])


# ---- logits ----


def logits_ref(x, hist, hl, pl, rep, pres, freq, ids, vals, allowed):
    y = f64(x).copy()
    B, V = y.shape
    mag = np.zeros_like(y)
    for b in range(B):
        mag[b] = np.abs(y[b])
        h = hist[b, :max(0, hl[b])]
        ok = (h >= 0) & (h < V)
        u = np.unique(h[ok])
        y[b, u] = np.where(y[b, u] > 0, y[b, u] / rep[b], y[b, u] * rep[b])
        mag[b, u] += np.abs(y[b, u])
        o = h[max(0, pl[b]):]
        u, c = np.unique(o[(o >= 0) & (o < V)], return_counts=True)
        y[b, u] -= c * freq[b] + pres[b]
        mag[b, u] += c * np.abs(freq[b]) + np.abs(pres[b])
        if ids is not None:
            fine = (ids[b] >= 0) & (ids[b] < V)
            np.add.at(y[b], ids[b][fine], vals[b][fine].astype(np.float64))
            np.add.at(mag[b], ids[b][fine], np.abs(vals[b][fine]))
        if allowed is not None:
            y[b, np.unpackbits(allowed[b].view(np.uint8), bitorder="little")[:V] == 0] = -INF
    return y, mag


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,V,L,NB,mask", [(1, 1, 1, 0, False), (1, 32000, 700, 16, True), (3, 4097, 33, 5, True), (2, 1000, 0, 3, False),
                                           (5, 50021, 9000, 300, True), (17, 333, 100, 0, True), (2, 12288, 2000, 64, False),
                                           (1, 100003, 20011, 0, False), (70, 5000, 64, 7, True),
                                           # more rows than run at once: slices of other widths, ranks instead of words
                                           (310, 5001, 200, 9, True), (311, 7, 30, 3, False), (64, 40003, 3001, 40, True),
                                           (30, 90007, 20011, 0, True), (31, 90001, 9000, 300, False), (320, 1031, 0, 0, True)])
def test_penalize_logits(dt, B, V, L, NB, mask):
    rng = np.random.default_rng(V + L)
    x = rnd(rng, dt, B, V) * 4
    x[:, V // 2] = 0
    hist = (rng.random((B, L))**3 * V).astype(np.int32)
    if L > 10:
        hist[:, 3], hist[:, 7] = -1, V                                     # skipped
    hl = rng.integers(0, L + 1, B).astype(np.int32)
    pl = (rng.random(B) * (hl + 3)).astype(np.int32)
    rep, pres, freq = (rng.uniform(a, b, B).astype(np.float32) for a, b in ((0.8, 1.5), (-1, 1), (-0.2, 0.5)))
    ids = rng.integers(-1, V + 1, (B, NB)).astype(np.int32) if NB else None           # some listed again, some outside
    vals = rng.normal(0, 5, (B, NB)).astype(np.float32) if NB else None
    allowed = rng.integers(-2**31, 2**31, (B, (V + 31) // 32)).astype(np.int32) if mask else None
    if mask and B > 2:
        allowed[1] = 0                                                      # nothing allowed
        allowed[2] = -1
    kw = dict(history=dev(hist), history_lens=dev(hl), prompt_lens=dev(pl), repetition=dev(rep), presence=dev(pres),
              frequency=dev(freq), bias_ids=None if ids is None else dev(ids), bias_vals=None if vals is None else dev(vals),
              allowed=None if allowed is None else dev(allowed))
    ref, mag = logits_ref(x, hist, hl, pl, rep, pres, freq, ids, vals, allowed)
    y = dbs.penalize_logits(x, **kw)
    assert y.dtype == torch.float32
    size = np.abs(np.where(np.isinf(ref), 0, ref))
    close(y, ref, 8 * 2.0**-24 * mag + U["f32"] * size)
    for od in ("f16", "bf16"):
        z = dbs.penalize_logits(x, out=torch.empty_like(x, dtype=DT[od]), **kw)
        close(z, ref, 8 * 2.0**-24 * mag + U[od] * size + (6e-8 if od == "f16" else 0))
    x2 = x.clone()
    assert dbs.penalize_logits(x2, out=x2, **kw) is x2                      # in place
    assert torch.equal(x2, dbs.penalize_logits(x, out=torch.empty_like(x), **kw))


def test_penalize_logits_parts_and_odd_values():
    rng = np.random.default_rng(20)
    B, V, L = 3, 777, 50
    x = rnd(rng, "f32", B, V + 5)[:, 2:2 + V]
    assert torch.equal(dbs.penalize_logits(x), x)
    hist = rng.integers(0, V, (B, L)).astype(np.int32)
    zero, one = np.zeros(B, np.float32), np.ones(B, np.float32)
    full, none = np.full(B, L), np.zeros(B, int)
    for kw, args in ((dict(repetition=dev(one * 1.3)), (one * np.float32(1.3), zero, zero)),
                     (dict(presence=dev(one * 0.5)), (one, one * 0.5, zero)),
                     (dict(frequency=dev(one * 0.25)), (one, zero, one * 0.25)), ({}, (one, zero, zero))):
        ref, mag = logits_ref(x, hist, full, none, *args, None, None, None)
        close(dbs.penalize_logits(x, history=dev(hist), **kw), ref, 8 * 2.0**-24 * mag)
    y = x.clone()
    y[0, 5], y[0, 6], y[1, 7], y[2, 8] = NAN, INF, -INF, 3.0
    h = dev(np.array([[5, 6], [7, 7], [8, 8]], np.int32))
    bits = np.full((B, (V + 31) // 32), -1, np.int32)
    bits[0, 0] &= ~(1 << 5)                                                 # a NaN in a masked place
    z = dbs.penalize_logits(y, history=h, repetition=dev(one * 2), frequency=dev(one), allowed=dev(bits))
    assert z[0, 5] == -INF and z[0, 6] == INF and z[1, 7] == -INF and z[2, 8] == 3.0 / 2 - 2
    # the same id several times: added in the list's order
    ids, vals = dev(np.array([[9, 9, 4, 9]] * B, np.int32)), dev(np.array([[1e8, 1.0, 2.0, -1e8]] * B, np.float32))
    z = dbs.penalize_logits(torch.zeros((B, V), device=DEV), bias_ids=ids, bias_vals=vals)
    assert (z[:, 9] == np.float32(np.float32(np.float32(1e8) + np.float32(1)) - np.float32(1e8))).all() and (z[:, 4] == 2).all()


# ---- streams and graphs ----


def step_inputs(rng):
    T, hq, hk, D, S, n = 6, 8, 2, 64, 300, 512
    x, w, s, _ = w4_inputs(rng, T, hq * D, n, "bf16", "f32", 64, False)
    return dict(x=x, w=w, s=s, k=rnd(rng, "bf16", T, hk, D), v=rnd(rng, "bf16", T, hk, D), table=dbs.rotary_table(400, D),
                pos=torch.arange(290, 296, dtype=torch.int32, device=DEV), kc=rnd(rng, "bf16", 20, 16, hk, D),
                vc=rnd(rng, "bf16", 20, 16, hk, D), slots=torch.arange(294, 300, dtype=torch.int32, device=DEV),
                kv=dev(np.array([S], np.int32)), tree=dev(tree_bits(rng, 1, T).view(np.int64)),
                pages=torch.arange(20, dtype=torch.int32, device=DEV)[None], hist=dev(rng.integers(0, 512, (T, 40)).astype(np.int32)),
                rep=torch.full((T,), 1.2, device=DEV))


def step(a, **kw):
    q = dbs.w4_linear(a["x"], a["w"], a["s"], group=64, **kw).unflatten(1, (8, 64))
    q = dbs.rotary_append(q, a["k"], a["v"], a["table"], a["pos"], a["kc"], a["vc"], a["slots"], **kw)
    o = dbs.tree_attention(q[None], a["kc"], a["vc"], a["kv"], a["tree"], page_table=a["pages"], **kw)
    return dbs.penalize_logits(o[0].flatten(1), history=a["hist"], repetition=a["rep"], **kw)


def test_operators_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(30)
    a = step_inputs(rng)
    ref = step(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kw in (dict(stream=side), dict(stream=side.cuda_stream)):
        got = step(a, **kw)
        side.synchronize()
        assert torch.equal(got, ref)
    with torch.cuda.stream(side):
        got = step(a)
    side.synchronize()
    assert torch.equal(got, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(a)
    x2 = torch.randn_like(a["x"])
    a["x"].copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, step(a)) and not torch.equal(out, ref)


def test_nothing_to_do():
    z = dict(device=DEV)
    assert dbs.w4_linear(torch.zeros((0, 64), **z), torch.zeros((8, 32), dtype=torch.uint8, **z), torch.zeros((8, 1), **z), group=64).shape == (0, 8)
    assert (dbs.w4_linear(torch.zeros((2, 0), **z), torch.zeros((8, 0), dtype=torch.uint8, **z), torch.zeros((8, 0), **z)) == 0).all()
    e = torch.zeros((0, 4, 64), dtype=torch.bfloat16, **z)
    q, k = dbs.rotary(e, e, dbs.rotary_table(0, 64), torch.zeros(0, dtype=torch.int32, **z))
    assert q.shape == k.shape == (0, 4, 64)
    c = torch.zeros((0, 16, 2, 64), dtype=torch.bfloat16, **z)
    o = dbs.tree_attention(torch.ones((2, 3, 4, 64), dtype=torch.bfloat16, **z), c, c, torch.zeros(2, dtype=torch.int32, **z),
                           page_table=torch.zeros((2, 0), dtype=torch.int32, **z))
    assert (o == 0).all()
    assert dbs.tree_attention(torch.ones((0, 3, 4, 64), dtype=torch.bfloat16, **z), c, c, torch.zeros(0, dtype=torch.int32, **z),
                              page_table=torch.zeros((0, 4), dtype=torch.int32, **z)).shape == (0, 3, 4, 64)
    assert dbs.penalize_logits(torch.zeros((0, 10), **z)).shape == (0, 10)
    assert dbs.penalize_logits(torch.zeros((3, 0), **z)).shape == (3, 0)


@pytest.mark.parametrize("call", [
    lambda: dbs.w4_linear(torch.zeros((2, 64), device=DEV), torch.zeros((8, 31), dtype=torch.uint8, device=DEV), torch.zeros((8, 1), device=DEV), group=64),
    lambda: dbs.w4_linear(torch.zeros((2, 64), device=DEV).double(), torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.zeros((8, 1), device=DEV), group=64),
    lambda: dbs.w4_linear(torch.zeros((64, 2), device=DEV).t(), torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.zeros((8, 1), device=DEV), group=64),
    lambda: dbs.w4_linear(torch.zeros((2, 64), device=DEV), torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.zeros((8, 1)), group=64),
    lambda: dbs.w4_linear(torch.zeros((2, 64), device=DEV), torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.zeros((8, 2), device=DEV), group=64),
    lambda: dbs.rotary(torch.zeros((4, 2, 64), device=DEV), None, torch.zeros((9, 66), device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)),
    lambda: dbs.rotary(torch.zeros((4, 2, 64), device=DEV), None, torch.zeros((9, 64), device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)),
    lambda: dbs.rotary(torch.zeros((4, 2, 64), device=DEV), torch.zeros((3, 2, 64), device=DEV), torch.zeros((9, 64), device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)),
    lambda: dbs.tree_attention(torch.zeros((1, 2, 4, 64), device=DEV), torch.zeros((1, 8, 2, 64), device=DEV), torch.zeros((1, 8, 2, 64), device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)),
    lambda: dbs.tree_attention(torch.zeros((2, 2, 4, 64), device=DEV).half(), torch.zeros((1, 8, 2, 64), device=DEV).half(), torch.zeros((1, 8, 2, 64), device=DEV).half(), torch.zeros(2, dtype=torch.int32, device=DEV)),
    lambda: dbs.tree_attention(torch.zeros((1, 2, 4, 64), device=DEV).half(), torch.zeros((1, 8, 2, 64), device=DEV).half(), torch.zeros((1, 8, 2, 64), device=DEV).half(), torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros((1, 2, 2), dtype=torch.int64, device=DEV)),
    lambda: dbs.penalize_logits(torch.zeros((2, 9), device=DEV), repetition=torch.ones(2, device=DEV)),
    lambda: dbs.penalize_logits(torch.zeros((2, 9), device=DEV), history=torch.zeros((3, 4), dtype=torch.int32, device=DEV)),
    lambda: dbs.penalize_logits(torch.zeros((2, 9), device=DEV), allowed=torch.zeros((2, 2), dtype=torch.int32, device=DEV)),
    lambda: dbs.penalize_logits(torch.zeros((2, 9), device=DEV), bias_ids=torch.zeros((2, 2), dtype=torch.int32, device=DEV))])
def test_refusals_of_shapes_and_types(call):
    with pytest.raises(dbs.DbsError) as e:
        call()
    assert e.value.status == 1


def test_example_of_drafted_steps():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    text, got, steps, logits, got_logits = example.main(24)
    assert steps < 24
    # logits of order 1 from some ten roundings to 2^-11 of them, each by its own order of sums; where two of them are as
    # near as that, the texts may part
    same = next((i for i, (a, b) in enumerate(zip(text, got)) if a != b), 24)
    assert (logits - got_logits)[:same + 1].abs().max() < 0.05
    assert same == 24 or (logits[same, text[same]] - logits[same, got[same]]).abs() < 0.1
