"""The decoding step's operators at the ends of their ranges, against plain 64-bit forms."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
import dynamic_sparsity_spmspv_gb300 as dbs  # noqa: E402

DEV = "cuda"


def yarn_table(P, R, base, factor, trained, fast=32.0, slow=1.0):
    """The published formula: between the pairs that turn `fast` and `slow` times within the trained positions, rounded
    outwards and kept within 0 and R - 1, the share of the divided frequency grows linearly with the pair's index."""
    def pair(turns):
        return R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)
    share = np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
    f = share * f / factor + (1 - share) * f
    a = np.arange(P)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1) * (0.1 * math.log(factor) + 1), f


@pytest.mark.parametrize("R,base,factor,trained", [
    (128, 1e4, 4.0, 131072), (128, 1e4, 8.0, 65536), (64, 1e4, 2.0, 1 << 20), (96, 500.0, 16.0, 8192), (8, 1e4, 4.0, 1 << 24),
    (128, 1e4, 16.0, 4096), (2, 1e4, 4.0, 4096), (128, 1e6, 4.0, 100.0)])
def test_yarn_table_of_any_trained_length(R, base, factor, trained):
    """Trained lengths at which the slowest pairs still turn more than once, and others."""
    P = 3000
    ref, f = yarn_table(P, R, base, factor, trained)
    t = dbs.rotary_table(P, R, base=base, scaling="yarn", factor=factor, trained=trained).double().cpu().numpy()
    # angles in 64 bits (roundings of the frequency and of the product, 2^-50 of the angle), then one to 32
    assert (np.abs(t - ref) <= 2.0**-24 * 1.5 + P * 2.0**-50).all()
    # a pair that turns more than once within the trained positions is never divided by the whole factor
    i = np.arange(R // 2)
    plain = base ** (-2.0 * i / R)
    turns = trained * plain / (2 * math.pi)
    assert (f[turns > 1.001] > plain[turns > 1.001] / factor).all()


@pytest.mark.parametrize("T,hq", [(1, 4), (3, 4), (40, 4), (300, 4)])
def test_attention_over_caches_without_entries(T, hq):
    """Pages of no entry, no pages at all, a table of no pages: nothing is seen."""
    f = dict(device=DEV, dtype=torch.bfloat16)
    q = torch.ones((2, T, hq, 64), **f)
    lens = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    for pages, size, table in ((5, 0, 4), (0, 0, 4), (5, 16, 0), (5, 0, 0), (0, 16, 0)):
        c = torch.zeros((pages, size, 2, 64), **f)
        o, lse = dbs.tree_attention(q, c, c, lens, page_table=torch.zeros((2, table), dtype=torch.int32, device=DEV), return_lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()
    c = torch.zeros((2, 0, 2, 64), **f)
    assert (dbs.tree_attention(q, c, c, lens) == 0).all()


def test_appending_to_caches_without_entries():
    """Every slot is outside of them: only q is turned."""
    f = dict(device=DEV, dtype=torch.bfloat16)
    q = torch.ones((5, 4, 64), **f)
    n = q[:, :2]
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    table = dbs.rotary_table(3, 64)
    for pages, size in ((5, 0), (0, 16), (0, 0)):
        c = torch.zeros((pages, size, 2, 64), **f)
        assert torch.equal(dbs.rotary_append(q, n, n, table, pos, c, c.clone(), pos), dbs.rotary(q, None, table, pos)[0])


class waits_run_out:
    """Waits of one block of each launch (-2: of all blocks) run out, after a millisecond."""

    def __init__(self, block):
        self.block = block

    def __enter__(self):
        assert dbs._lib.load().dbs_debug_operator_waits(1_000_000, self.block) == 0

    def __exit__(self, *_):
        torch.cuda.synchronize()
        assert dbs._lib.load().dbs_debug_operator_waits(2_000_000_000, -1) == 0


@pytest.mark.parametrize("page", [16, 1])                                  # tiled copies, and others
@pytest.mark.parametrize("B,T,hq,hk,D,S", [
    (3, 12, 16, 2, 128, 700), (2, 96, 12, 2, 64, 1500), (5, 40, 8, 1, 128, 900), (2, 80, 2, 1, 256, 300), (190, 20, 8, 4, 64, 60)])
def test_attention_that_gives_up_leaves_nan(B, T, hq, hk, D, S, page):
    """All rows of the units that a block whose wait ran out had in hand or still ahead are NaN, the others as ever, and so
    is the next call."""
    g = torch.Generator(device=DEV).manual_seed(B + T)
    per = -(-S // page)
    q = torch.randn((B, T, hq, D), generator=g, device=DEV).half()
    k, v = (torch.randn((B * per, page, hk, D), generator=g, device=DEV).half() for _ in range(2))
    pages = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
    lens = torch.randint(S // 2, S + 1, (B,), generator=g, device=DEV).to(torch.int32)

    def call():
        # (memory that the scratch is likely to be given holds numbers that nobody may use)
        junk = torch.full((1 << 24,), 0x7f7f7f7f, dtype=torch.int32, device=DEV)
        del junk
        out = torch.full_like(q, 5.0)
        return dbs.tree_attention(q, k, v, lens, page_table=pages, out=out, return_lse=True)

    clean, lse = call()
    rows = min(256 if D <= 128 and T * hq // hk > 128 else 128, T * hq // hk)     # of a unit
    for block in (-2, 0, 7):
        with waits_run_out(block):
            got, gl = call()
        nan = torch.isnan(got)
        assert (nan.all(3) == nan.any(3)).all() and (nan.any(3) == torch.isnan(gl)).all()
        nan = nan.any(3)
        if block == -2:
            assert nan.all()
        else:
            assert nan.any()
            keep = ~nan
            assert torch.equal(got[keep], clean[keep]) and torch.equal(gl[keep], lse[keep])
            # whole units: rows are tokens times the heads of a kv head
            by_unit = nan.view(B, T, hk, hq // hk).transpose(1, 2).reshape(B, hk, -1)
            for u in by_unit.split(rows, 2):
                assert (u.all(2) == u.any(2)).all()
        again, al = call()
        assert torch.equal(again, clean) and torch.equal(al, lse)


@pytest.mark.parametrize("T,m,n,dt,group", [
    (1, 4096, 1024, torch.float32, 128), (1, 9000, 700, torch.bfloat16, 32), (7, 3000, 2050, torch.float16, 64), (9, 500, 20000, torch.float32, 256),
    (25, 700, 3000, torch.float32, 128), (20, 4096, 4096, torch.bfloat16, 128), (24, 40000, 600, torch.float16, 64),
    (70, 1000, 8192, torch.float16, 128), (150, 9000, 304, torch.bfloat16, 32)])
def test_w4_that_gives_up_leaves_nan(T, m, n, dt, group):
    """Rows of one matrix instruction's tiles, rows of clusters that share columns, rows of blocks with several units."""
    g = torch.Generator(device=DEV).manual_seed(T + m)
    x = torch.randn((T, n), generator=g, device=DEV).to(dt)
    q = torch.randint(0, 256, (m, -(-n // 32) * 16), generator=g, device=DEV, dtype=torch.uint8)[:, :(n + 1) // 2]
    s = torch.rand((m, -(-n // group)), generator=g, device=DEV)

    def call():
        return dbs.w4_linear(x, q, s, group=group, y=torch.full((T, m), 5.0, dtype=dt, device=DEV))

    clean = call()
    for block in (-2, 0, 3):
        with waits_run_out(block):
            y = call()
        nan = torch.isnan(y)
        if block == -2:
            assert nan.all()
        else:
            assert nan.any() and not nan.all() and torch.equal(y[~nan], clean[~nan])
        assert torch.equal(call(), clean)


def test_attention_whose_queries_wait_too_long():
    """A limit that only the warps which load queries reach, as they wait for all scores of the unit before: what comes out is
    right or NaN."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, T, hq, D, S, page = 400, 30, 4, 64, 1 << 19, 4
    q = torch.randn((B, T, hq, D), generator=g, device=DEV).half()
    k, v = (torch.randn((S // page, page, 1, D), generator=g, device=DEV).half() for _ in range(2))
    pages = torch.arange(S // page, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    clean = dbs.tree_attention(q, k, v, lens, page_table=pages)
    lib = dbs._lib.load()
    assert lib.dbs_debug_operator_waits(20_000, -1) == 0
    try:
        got = dbs.tree_attention(q, k, v, lens, page_table=pages)
        torch.cuda.synchronize()
    finally:
        lib.dbs_debug_operator_waits(2_000_000_000, -1)
    nan = torch.isnan(got)
    assert (nan | (got == clean)).all()


def test_waits_that_run_out_are_reported_once():
    f = dict(device=DEV)
    codes = torch.zeros((4096, 512), dtype=torch.uint8, **f)
    scales, q = torch.ones((4096, 8), **f), torch.ones((2, 40, 8, 64), dtype=torch.float16, **f)
    cache, lens = torch.ones((2, 300, 2, 64), dtype=torch.float16, **f), torch.full((2,), 300, dtype=torch.int32, **f)
    calls = [lambda: dbs.w4_linear(torch.ones((1, 1024), **f), codes, scales), lambda: dbs.w4_linear(torch.ones((20, 1024), **f).half(), codes, scales),
             lambda: dbs.w4_linear(torch.ones((50, 1024), **f).half(), codes, scales), lambda: dbs.tree_attention(q, cache, cache, lens)]
    side = torch.cuda.Stream()
    dbs.operators_check()                                                  # (what earlier tests left)
    for call in calls:
        call()
        assert dbs.operators_check() == 0
        with waits_run_out(0):
            call()
        assert dbs.operators_check() == 4 and dbs.operators_check(side) == 0
        with waits_run_out(-2), torch.cuda.stream(side):
            call()
        assert dbs.operators_check(side) == 4 and dbs.operators_check() == 0
        call()
        assert dbs.operators_check() == 0


@pytest.mark.parametrize("tokens,D,R", [(1, 64, 32), (3, 4, 2), (1, 8, 8)])
def test_rotary_of_as_many_heads_as_there_may_be(tokens, D, R):
    """16384 heads in each group, of which parts are turned and parts copied."""
    rng = np.random.default_rng(D)
    H = 16384
    table = torch.from_numpy(rng.standard_normal((9, R)).astype(np.float32)).to(DEV)
    q, k, v = (torch.from_numpy(rng.standard_normal((tokens, H, D)).astype(np.float32)).to(DEV) for _ in range(3))
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    kc, vc = torch.zeros((tokens, 2, H, D), device=DEV), torch.zeros((tokens, 2, H, D), device=DEV)
    qo = dbs.rotary_append(q, k, v, table, pos, kc, vc, 2 * pos + 1)
    c, s = (t.double()[pos.long()][:, None] for t in table.split(R // 2, 1))

    def turned(x):
        a, b, rest = x.double().split([R // 2, R // 2, D - R], 2)
        return torch.cat([a * c - b * s, a * s + b * c, rest], 2), torch.cat([(a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs(), rest * 0], 2)

    for got, x in ((qo, q), (kc[:, 1], k)):
        ref, size = turned(x)
        # two products and a sum, rounded to 32 bits
        assert ((got.double() - ref).abs() <= 3 * 2.0**-24 * size).all()
    assert torch.equal(vc[:, 1], v) and (kc[:, 0] == 0).all() and (vc[:, 0] == 0).all()


@pytest.mark.parametrize("B", [2, 200])
def test_penalize_logits_of_any_repetition(B):
    """Penalties whose reciprocal is no normal number, or none at all; a quotient is rounded once.  B: slices of both kinds."""
    V, L = 40001, 64
    rng = np.random.default_rng(B)
    x = (rng.standard_normal((B, V)) * 4).astype(np.float32)
    hist = np.stack([rng.choice(V, L, replace=False) for _ in range(B)]).astype(np.int32)
    rep = np.resize(np.array([1e-39, 3e38, 1.1, 3.0, 1.3, 7e-42, 2.0**127], np.float32), B)
    x[rep < 1e-30] *= np.float32(1e-12)
    y = dbs.penalize_logits(torch.from_numpy(x).to(DEV), history=torch.from_numpy(hist).to(DEV), repetition=torch.from_numpy(rep).to(DEV))
    ref = x.copy()
    for b in range(B):
        l = x[b, hist[b]]
        with np.errstate(over="ignore", under="ignore"):
            ref[b, hist[b]] = np.where(l > 0, (l.astype(np.float64) / np.float64(rep[b])).astype(np.float32),
                                       (l.astype(np.float64) * np.float64(rep[b])).astype(np.float32))
    assert np.array_equal(y.cpu().numpy(), ref)


def test_outputs_that_share_memory_are_refused():
    f = dict(dtype=torch.float16, device=DEV)
    h, cache, ids = torch.ones((4, 2, 64), **f), torch.ones((4, 2, 2, 64), **f), torch.zeros(4, dtype=torch.int32, device=DEV)
    table, same = torch.zeros((9, 64), device=DEV), torch.zeros((1, 1, 64), **f)
    for call in (lambda: dbs.rotary(h, h, table, ids, q_out=same.expand(4, 2, 64)), lambda: dbs.rotary(h, h, table, ids, k_out=same.expand(4, 2, 64)),
                 lambda: dbs.rotary_append(h, h, h, table, ids, same.expand(4, 2, 2, 64), cache, ids),
                 lambda: dbs.tree_attention(h[None], cache[:1], cache[:1], ids[:1], out=same.expand(1, 4, 2, 64)),
                 lambda: dbs.penalize_logits(h[0], out=same[0].expand(2, 64)),
                 lambda: dbs.w4_linear(h[:, 0], torch.zeros((8, 32), dtype=torch.uint8, device=DEV), torch.ones((8, 1), device=DEV), group=64,
                                       y=same[0, :, :8].expand(4, 8))):
        with pytest.raises(dbs.DbsError) as e:
            call()
        assert e.value.status == 1


def test_gradients_are_never_lost_in_silence():
    """What would need a gradient is refused where autograd records, and what is written in place counts as changed."""
    f = dict(device=DEV)
    x, codes, scales = torch.ones((2, 64), **f), torch.zeros((8, 32), dtype=torch.uint8, **f), torch.ones((8, 1), **f)
    h, cache = torch.ones((4, 2, 64), dtype=torch.float16, **f), torch.zeros((2, 16, 2, 64), dtype=torch.float16, **f)
    ids, table = torch.zeros(4, dtype=torch.int32, **f), torch.zeros((9, 64), **f)
    slots = torch.arange(4, dtype=torch.int32, **f)
    one = torch.ones(2, **f)
    calls = [lambda g: dbs.w4_linear(g(x), codes, scales, group=64), lambda g: dbs.w4_linear(x, codes, g(scales), group=64),
             lambda g: dbs.rotary(g(h), None, table, ids), lambda g: dbs.rotary(h, g(h), table, ids), lambda g: dbs.rotary(h, h, g(table), ids),
             lambda g: dbs.rotary_append(h, h, g(h), table, ids, cache, cache.clone(), slots),
             lambda g: dbs.tree_attention(g(h[None]), cache[:1], cache[:1], ids[:1]),
             lambda g: dbs.tree_attention(h[None], cache[:1], g(cache[:1]), ids[:1]),
             lambda g: dbs.penalize_logits(g(x)), lambda g: dbs.penalize_logits(x, history=codes[:2, :3].int(), repetition=g(one))]
    for call in calls:
        with pytest.raises(dbs.DbsError) as e:
            call(lambda t: t.clone().requires_grad_())
        assert e.value.status == 1
        call(lambda t: t)
        with torch.no_grad():
            call(lambda t: t.clone().requires_grad_())
    with torch.inference_mode():
        t, y = torch.ones((2, 64), **f), torch.empty((2, 8), **f)
        dbs.w4_linear(t, codes, scales, group=64, y=y)
    assert torch.equal(dbs.w4_linear(t, codes, scales, group=64), dbs.w4_linear(x, codes, scales, group=64))

    def changed(t, call):
        before = t._version
        call()
        assert t._version > before

    y, kc, vc, q = torch.empty((2, 8), **f), cache.clone(), cache.clone(), h.clone()
    changed(y, lambda: dbs.w4_linear(x, codes, scales, group=64, y=y))
    for t in (q, kc, vc):
        changed(t, lambda: dbs.rotary_append(q, h, h, table, ids, kc, vc, slots, q_out=q))
    changed(q, lambda: dbs.rotary(h, h, table, ids, q_out=q))
    k2 = h.clone()
    changed(k2, lambda: dbs.rotary(h, h, table, ids, k_out=k2))
    o = h[None].clone()
    changed(o, lambda: dbs.tree_attention(h[None], cache[:1], cache[:1], ids[:1], out=o))
    l = x.clone()
    changed(l, lambda: dbs.penalize_logits(l, out=l))
    # a saved tensor that was overwritten
    w = torch.ones((2, 64), requires_grad=True, **f)
    s = x.clone()
    z = (w * s).sum()
    dbs.penalize_logits(s, out=s)
    with pytest.raises(RuntimeError):
        z.backward()


def attention64(q, k, v, lens, tree_lens, bits, table):
    """Attention in 64 bits, with the sums of p |v|; bits: a bool [B, T, T] of what a drafted token sees, or None."""
    B, T, hq, D = q.shape
    out, size = torch.zeros((2, *q.shape), dtype=torch.float64, device=DEV)
    for b in range(B):
        n, t = int(lens[b]), int(tree_lens[b])
        kb, vb = ((c[table[b].long()].flatten(0, 1)[:n] if table is not None else c[b, :n]).double().repeat_interleave(hq // c.shape[2], 1) for c in (k, v))
        node = torch.arange(n, device=DEV) - (n - t)
        see = (node < 0) | (node[None] <= torch.arange(t, device=DEV)[:, None]) if bits is None else (node < 0) | bits[b, :t][:, node.clamp(min=0)]
        for h in range(hq):
            p = torch.softmax((q[b, :t, h].double() @ kb[:, h].t() * D**-0.5).masked_fill(~see, -math.inf), 1).nan_to_num(0.0)
            seen = torch.where(torch.isfinite(vb[:, h]), vb[:, h], 0.0)    # (those that are not: see the callers)
            out[b, :t, h], size[b, :t, h] = p @ seen, p @ seen.abs()
    return out, size


# head sizes of each kernel; up to 128 rows of a kv head, and more; pages that eight does not divide, and others
@pytest.mark.parametrize("page", [12, 5, 32, 0])
@pytest.mark.parametrize("D", [40, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("B,T,hq,hk,S", [(5, 23, 10, 2, 900), (3, 70, 6, 1, 1500), (150, 20, 2, 2, 90)])
def test_attention_of_many_rows_over_caches_of_any_page(B, T, hq, hk, S, D, page):
    g = torch.Generator(device=DEV).manual_seed(B + D + page)
    dt, u = (torch.float16, 2.0**-11) if D in (40, 128, 200) else (torch.bfloat16, 2.0**-8)
    size = page or S
    per = -(-S // size)
    q = torch.randn((B, T, hq, D), generator=g, device=DEV).to(dt)
    k, v = (torch.randn((B * per, size, hk, D), generator=g, device=DEV).to(dt) for _ in range(2))
    if not page:
        k = k[:, :, :1].expand(-1, -1, hk, -1)                             # (heads that share keys: no tiled copies)
    table = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per) if page else None
    tl = torch.randint(1, T + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens = torch.maximum(torch.randint(1, S + 1, (B,), generator=g, device=DEV), tl).clamp(max=S).to(torch.int32)
    lens[0], tl[0] = S, T
    bits = torch.rand((B, T, T), generator=g, device=DEV) < 0.3
    bits |= torch.eye(T, dtype=torch.bool, device=DEV)
    bits[:, :-1, T - 1] = False                                            # the last drafted token: seen by itself alone
    tree = torch.zeros((B, T, -(-T // 64)), dtype=torch.int64, device=DEV)
    for i in range(T):
        tree[:, :, i // 64] |= bits[:, :, i].long() << (i % 64)
    for mask, words in ((bits, tree), (None, None)):
        def call():
            return dbs.tree_attention(q, k, v, lens, words, tree_lens=tl, page_table=table)

        got = call()
        ref, mag = attention64(q, k, v, lens, tl, mask, table)
        # probabilities rounded once to the caches' type, scores in 32 bits (3e-4 for head sizes to 256), the result rounded
        assert ((got.double() - ref).abs() <= (u + 3e-4) * mag + u * ref.abs() + 1e-7).all()
        assert torch.equal(got, call())
    # a NaN in the last drafted token's value reaches that token alone
    e = int(lens[0]) - 1
    at = (int(table[0, e // page]), e % page) if page else (0, e)
    clean = dbs.tree_attention(q, k, v, lens, tree, tree_lens=tl, page_table=table)
    v[at[0], at[1], :, 0] = math.nan
    got = dbs.tree_attention(q, k, v, lens, tree, tree_lens=tl, page_table=table)
    assert torch.isnan(got[0, T - 1, :, 0]).all()
    got[0, T - 1, :, 0] = clean[0, T - 1, :, 0]
    assert torch.equal(got, clean)
