"""Cases of the operators around a paged cache: norms of queries and keys with
their rotation, attention with a sliding window and sinks, and the cache's pages
(reserving, forking, compacting, freeing).

`run` computes one pass: with `own` through the package's entry points, without
it from elementary torch operations in 32 bits."""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NEG_INF = float("-inf")
EPS = 1e-6


def listed():
    return [
        # one sequence, one token over a contiguous cache: latency counts
        dict(name="window token", op="window", B=1, T=1, Hq=32, Hkv=8, D=128, S=9001, window=1024, sinks=4, page=0, ragged=False,
             dtype="bf16"),
        # a serving batch, one token each, every sequence with a length of its own
        dict(name="window batch", op="window", B=64, T=1, Hq=32, Hkv=8, D=128, S=16384, window=4096, sinks=4, page=16, ragged=True,
             dtype="bf16"),
        # a few drafted tokens of each of a few sequences, an odd window
        dict(name="window drafted", op="window", B=8, T=8, Hq=32, Hkv=4, D=128, S=8192, window=2047, sinks=64, page=64, ragged=False,
             dtype="f16"),
        # a whole prompt
        dict(name="window prompt", op="window", B=1, T=8192, Hq=32, Hkv=8, D=128, S=8192, window=4096, sinks=4, page=16, ragged=False,
             dtype="bf16"),
        # one step of a few drafted tokens: norm and turn q and k, put k and v into the paged cache
        dict(name="norm append step", op="norm_append", N=5, Hq=32, Hkv=8, D=128, R=128, page=16, interleaved=False, dtype="bf16"),
        # a long prompt, half of each head turned
        dict(name="norm prompt", op="norm", B=2, T=8191, Hq=32, Hkv=8, D=128, R=64, interleaved=False, heads_first=False, dtype="bf16"),
        # the gradient of a training batch, interleaved pairs, heads before tokens
        dict(name="norm gradient", op="norm_grad", B=4, T=2048, Hq=16, Hkv=16, D=96, R=96, interleaved=True, heads_first=True,
             dtype="f32"),
        # the gradient of a small batch in 16 bits
        dict(name="norm gradient small", op="norm_grad", B=1, T=301, Hq=8, Hkv=2, D=128, R=128, interleaved=False, heads_first=False,
             dtype="bf16"),
        # a drafted tree of one sequence: what was accepted moves up, in the caches of two layers
        dict(name="compact one", op="compact", layers=2, B=1, T=12, Hkv=8, D=128, S=500, page=16, dtype="bf16"),
        # the trees of a serving batch, all layers in one call
        dict(name="compact batch", op="compact", layers=16, B=32, T=48, Hkv=8, D=128, S=256, page=16, dtype="bf16"),
        # a step of a few sequences: entries for drafted tokens, one fork, everything cut back
        dict(name="pages small", op="pages", layers=2, B=6, forks=1, T=5, Hkv=2, D=64, S=200, page=16, dtype="f16"),
        # a step of a serving batch with a fork of each sequence, all layers in one call
        dict(name="pages batch", op="pages", layers=16, B=96, forks=32, T=8, Hkv=8, D=128, S=255, page=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "norm_append", "norm", "norm_grad", "compact", "pages"])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "window":
        while True:
            T = rng.choice([1, _log(rng, 1, 16), _log(rng, 16, 8192)])
            S = max(T, _log(rng, 64, 16384))
            c = dict(op=op, B=_log(rng, 1, 64), T=T, Hq=hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=hkv, D=rng.choice([64, 96, 128, 128, 256]),
                     S=S, window=_log(rng, 16, 8192), sinks=rng.choice([0, 4, _log(rng, 1, 200)]), page=rng.choice([0, 16, 24, 64, 256]),
                     ragged=rng.random() < 0.7, dtype=rng.choice(["f16", "bf16"]))
            w = work(c)
            if w["bytes"] <= 6e8 and w["flops"] <= 3e11 and c["B"] * T * c["Hq"] * S <= 2.5e9 and c["B"] * S * hkv * c["D"] <= 5e8:
                return c
    if op in ("norm_append", "norm", "norm_grad"):
        D = rng.choice([64, 80, 96, 128, 256])
        c = dict(op=op, Hq=hkv * rng.choice([1, 2, 4, 6]), Hkv=hkv, D=D, R=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.5,
                 dtype=rng.choice(["f32", "f16", "bf16"]))
        if op == "norm_append":
            return dict(c, N=_log(rng, 1, 2048), page=rng.choice([1, 16, 24, 64]))
        return dict(c, B=_log(rng, 1, 8), T=_log(rng, 1, 1024), heads_first=rng.random() < 0.5)
    c = dict(op=op, layers=_log(rng, 1, 16), B=_log(rng, 2, 64), T=_log(rng, 1, 64), Hkv=hkv, D=rng.choice([64, 80, 128, 256]), S=_log(rng, 64, 512),
             page=rng.choice([1, 16, 24, 64]), dtype=rng.choice(["f16", "bf16", "f32"]))
    while c["layers"] * c["B"] * c["S"] * hkv * c["D"] > 6e7:
        c["layers"], c["B"] = (c["layers"] + 1) // 2, max(2, c["B"] // 2)
    return dict(c, forks=rng.randint(1, c["B"] // 2)) if op == "pages" else c


def _lengths(case):
    """Entries of every sequence (the call's tokens among them) and its tokens: fixed by the case."""
    B, T, S = case["B"], case["T"], case["S"]
    if not case.get("ragged", True):
        return [S] * B, [T] * B
    r = random.Random(B * 1000003 + T * 1009 + S)
    tl = [r.randint((T + 1) // 2, T) for _ in range(B)]
    return [r.randint(max(S // 4, tl[b]), max(S, T)) for b in range(B)], tl


def _accepted(case):
    """The accepted nodes of every sequence's tree, node 0 (the last token of the text) among them: a path of the tree."""
    r = random.Random(case["B"] * 10007 + case["T"])
    paths = []
    for tl in _lengths(case)[1]:
        path = [0]
        while path[-1] + 1 < tl and r.random() < 0.85:
            path.append(r.randint(path[-1] + 1, min(tl - 1, path[-1] + 4)))
        paths.append(path)
    return paths


def _plan(case):
    """Of a pages case: lengths before the step (the children empty), in it, and after it; parents and children."""
    r = random.Random(case["B"] * 131 + case["S"])
    B, F, T, S = case["B"], case["forks"], case["T"], case["S"]
    live = B - F
    before = [r.randint(max(1, S // 4), S) for _ in range(live)] + [0] * F
    grown = [n + r.randint(1, T) for n in before[:live]] + [-1] * F
    after = [n + r.randint(0, g - n) for n, g in zip(before[:live], grown)]
    return before, grown, after, [r.randrange(live) for _ in range(F)], list(range(live, B))


def _max_pages(case):
    return -(-(case["S"] + case["T"]) // case["page"])


def work(case):
    e, op = _SIZE[case["dtype"]], case["op"]
    if op == "window":
        kv, tl = _lengths(case)
        W, s, pairs, seen = case["window"], case["sinks"], 0, 0
        for n, t in zip(kv, tl):
            first = n - t
            for p in range(first, n):
                lo = max(0, p - W + 1)
                pairs += p + 1 - lo + min(s, lo)
            lo = max(0, first - W + 1)
            seen += n - lo + min(s, lo)
        rows = case["B"] * case["T"] * case["Hq"]
        return {"bytes": 2 * seen * case["Hkv"] * case["D"] * e + 2 * rows * case["D"] * e + 8 * case["B"],
                "flops": 4.0 * case["D"] * case["Hq"] * pairs}
    if op in ("norm_append", "norm", "norm_grad"):
        n = case["N"] if op == "norm_append" else case["B"] * case["T"]
        heads = case["Hq"] + case["Hkv"]
        moved = 2 * (heads + case["Hkv"]) if op == "norm_append" else 2 * heads if op == "norm" else 3 * heads
        angles = (n if op == "norm_append" else case["T"]) * case["R"] * 4
        return {"bytes": n * moved * case["D"] * e + angles + n * (8 if op == "norm_append" else 4) + 2 * case["D"] * e,
                "flops": (12.0 if op == "norm_grad" else 6.0) * n * heads * case["D"]}
    entry = case["layers"] * 2 * case["Hkv"] * case["D"] * e
    if op == "compact":
        paths = _accepted(case)
        moved = sum(t != i for p in paths for i, t in enumerate(p))
        return {"bytes": 2 * moved * entry + 4 * sum(map(len, paths)) + 16 * case["B"], "flops": float(moved)}
    before, grown, _, parents, _ = _plan(case)
    page = case["page"]
    copied = sum(max(grown[p], 0) % page for p in parents)
    names = sum(-(-grown[p] // page) for p in parents)
    pages = case["B"] * (_max_pages(case) + 1)
    return {"bytes": 2 * copied * entry + 12 * names + 4 * pages + 40 * case["B"] + 4 * case["B"] * case["T"], "flops": float(copied + names)}


def _table(positions, R, base=10000.0):
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    a = np.arange(positions, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    dt, op, D, hkv = _DT[case["dtype"]], case["op"], case["D"], case["Hkv"]
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if op == "window":
        B, T, S, page = (case[k] for k in ("B", "T", "S", "page"))
        kv, tl = _lengths(case)
        s["q"] = normal(B, T, case["Hq"], D)
        if page:
            per = -(-S // page)
            s["k_cache"], s["v_cache"] = normal(B * per, page, hkv, D), normal(B * per, page, hkv, D)
            s["page_table"] = torch.from_numpy(r.permutation(B * per).astype(np.int32).reshape(B, per)).cuda()
        else:
            s["k_cache"], s["v_cache"], s["page_table"] = normal(B, S, hkv, D), normal(B, S, hkv, D), None
        s["kv_lens"], s["q_lens"] = _ints(kv), _ints(tl)
    elif op in ("norm_append", "norm", "norm_grad"):
        for k in ("q_weight", "k_weight"):
            s[k] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        if op == "norm_append":
            N, page = case["N"], case["page"]
            pages = -(-(N + N // 2 + 3) // page)
            s["q"], s["k"], s["v"] = 3 * normal(N, case["Hq"], D), 3 * normal(N, hkv, D), normal(N, hkv, D)
            s["k_cache"], s["v_cache"] = normal(pages, page, hkv, D), normal(pages, page, hkv, D)
            s["slots"] = torch.from_numpy(r.permutation(pages * page)[:N].astype(np.int32)).cuda()
            s["positions"] = torch.from_numpy(r.integers(0, 4096, N).astype(np.int32)).cuda()
            s["table"] = _table(4096, case["R"])
        else:
            B, T = case["B"], case["T"]

            def heads(h, size=3):
                return size * (normal(B, h, T, D).transpose(1, 2) if case["heads_first"] else normal(B, T, h, D))

            s["q"], s["k"] = heads(case["Hq"]), heads(hkv)
            if op == "norm_grad":
                s["q_grad"], s["k_grad"] = heads(case["Hq"], 1), heads(hkv, 1)
            first = torch.from_numpy(r.integers(0, 64, (B, 1)).astype(np.int32)).cuda()
            s["positions"] = (torch.arange(T, device="cuda", dtype=torch.int32)[None, :] + first).contiguous()
            s["table"] = _table(T + 64, case["R"])
    else:
        B, page, per = case["B"], case["page"], _max_pages(case)
        pages = B * per
        shape = (case["layers"], pages, page, hkv, D)
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
        table = r.permutation(pages).astype(np.int32).reshape(B, per)
        s["page_table"] = torch.from_numpy(table).cuda()
        if op == "compact":
            kv, tl = _lengths(case)
            paths = _accepted(case)
            acc = np.full((B, case["T"]), -1, np.int32)
            for b, p in enumerate(paths):
                acc[b, : len(p)] = p
            s["accepted"], s["accepted_lens"] = torch.from_numpy(acc).cuda(), _ints([len(p) for p in paths])
            s["kv_lens"], s["tree_lens"] = _ints(kv), _ints(tl)
        else:
            before, grown, after, parents, children = _plan(case)
            refs = np.zeros(pages, np.int32)
            for b, n in enumerate(before):
                refs[table[b, : -(-n // page)]] += 1
            s["kv_lens"], s["refs"] = _ints(before), torch.from_numpy(refs).cuda()
            s["parents"], s["children"] = _ints(parents), _ints(children)
            # the step reserves entries, forks, keeps some of the entries and drops the children; then it is undone
            s["grown"], s["after"], s["before"] = _ints(grown), _ints(after + [0] * len(children)), _ints(before)
    return s


def run(s):
    if own:
        return _own(s)
    return {"window": _window, "norm_append": _norm_append, "norm": _norm, "norm_grad": _norm_grad, "compact": _compact,
            "pages": _pages}[s["op"]](s)


def _own(s):
    import dynamic_sparsity_spmspv_gb300 as dbs

    op = s["op"]
    if op == "window":
        return dbs.window_attention(s["q"], s["k_cache"], s["v_cache"], s["kv_lens"], s["window"], sinks=s["sinks"], q_lens=s["q_lens"],
                                    page_table=s["page_table"])
    if op == "norm_append":
        q = dbs.norm_rotary_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["table"], s["positions"], s["k_cache"],
                                   s["v_cache"], s["slots"], eps=EPS, interleaved=s["interleaved"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "norm":
        return dbs.norm_rotary(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"], eps=EPS,
                               interleaved=s["interleaved"])
    if op == "norm_grad":
        return dbs.norm_rotary_gradient(s["q_grad"], s["k_grad"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"],
                                        eps=EPS, interleaved=s["interleaved"])
    if op == "compact":
        lens = dbs.cache_compact(s["k_cache"], s["v_cache"], s["kv_lens"], s["tree_lens"], s["accepted"], s["accepted_lens"],
                                 page_table=s["page_table"])
        return [lens, s["k_cache"], s["v_cache"]]
    state = (s["page_table"], s["kv_lens"], s["refs"])
    grown, slots = dbs.cache_resize(*state, s["grown"], s["page"], columns=s["T"])
    forked = dbs.cache_fork(s["k_cache"], s["v_cache"], *state, s["parents"], s["children"])
    table, lens, refs = (t.clone() for t in state)
    cut, _ = dbs.cache_resize(*state, s["after"], s["page"])
    dbs.cache_resize(*state, s["before"], s["page"])
    return [grown, slots, forked, table, lens, refs, cut, *state, s["k_cache"], s["v_cache"]]


# ---- plain forms ----


def _window(s):
    B, T, hq, hkv, D, S = (s[k] for k in ("B", "T", "Hq", "Hkv", "D", "S"))
    k, v = s["k_cache"], s["v_cache"]
    if s["page_table"] is not None:
        at = s["page_table"].long()
        k, v = k[at].flatten(1, 2)[:, :S], v[at].flatten(1, 2)[:, :S]
    k, v = k.float().permute(0, 2, 3, 1), v.float().permute(0, 2, 1, 3)
    j, parts = torch.arange(S, device=k.device), []
    step = max(1, min(T, int(4e8) // (B * hq * S)))
    for t0 in range(0, T, step):
        n = min(step, T - t0)
        q = s["q"][:, t0 : t0 + n].float().reshape(B, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
        p = (q @ k).mul_(1 / math.sqrt(D)).view(B, hkv, hq // hkv, n, S)
        t = torch.arange(t0, t0 + n, device=k.device)
        pos = ((s["kv_lens"] - s["q_lens"])[:, None] + t)[:, :, None]
        seen = (j <= pos) & ((j > pos - s["window"]) | (j < s["sinks"])) & (t < s["q_lens"][:, None])[:, :, None]
        p.masked_fill_(~seen[:, None, None], NEG_INF)
        p.sub_(p.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
        total = p.sum(-1, keepdim=True).clamp_(min=1e-30)
        o = (p.view(B, hkv, -1, S) @ v).view(B, hkv, hq // hkv, n, D) / total
        parts.append(o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, D).to(s["q"].dtype))
    return torch.cat(parts, 1) if len(parts) > 1 else parts[0]


def _angles(s):
    row = s["table"][s["positions"].long()][..., None, :]
    return row[..., : s["R"] // 2], row[..., s["R"] // 2 :]


def _turn(y, cos, sin, R, interleaved):
    """y [..., heads, D] in 32 bits, cos and sin [..., 1, R/2]."""
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., : R // 2], y[..., R // 2 : R])
    u, v = a * cos - b * sin, a * sin + b * cos
    t = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([t, y[..., R:]], -1)


def _normed(x, w, cos, sin, s):
    y = x.float()
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
    return _turn(y, cos, sin, s["R"], s["interleaved"]).to(x.dtype)


def _norm(s):
    cos, sin = _angles(s)
    return tuple(_normed(s[k], s[k + "_weight"], cos, sin, s) for k in ("q", "k"))


def _norm_append(s):
    q, k = _norm(s)
    at = s["slots"].long()
    s["k_cache"].flatten(0, 1)[at] = k
    s["v_cache"].flatten(0, 1)[at] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _norm_grad(s):
    cos, sin = _angles(s)
    dx, dw = [], []
    for k in ("q", "k"):
        x = s[k].float()
        g = _turn(s[k + "_grad"].float(), cos, -sin, s["R"], s["interleaved"])
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n = x * r
        dw.append((g * n).sum((0, 1, 2)))
        g = g * s[k + "_weight"].float()
        dx.append((r * (g - n * (g * n).mean(-1, keepdim=True))).to(s[k].dtype))
    return [*dx, *dw]


def _compact(s):
    page, T = s["page"], s["T"]
    i = torch.arange(T, device=s["kv_lens"].device)
    first = (s["kv_lens"] - s["tree_lens"])[:, None]
    take = (i < s["accepted_lens"][:, None]).flatten()

    def slots(j):
        return (s["page_table"].gather(1, (j // page).clamp(0, s["page_table"].shape[1] - 1).long()) * page + j % page).flatten()[take].long()

    src, dst = slots(first + s["accepted"].clamp(min=0)), slots(first + i)
    for c in ("k_cache", "v_cache"):
        flat = s[c].flatten(1, 2)
        flat[:, dst] = flat[:, src]
    return [(first[:, 0] + s["accepted_lens"]).to(torch.int32), s["k_cache"], s["v_cache"]]


def _resize(table, kv, refs, lens, page, columns=0):
    B, M = table.shape
    col = torch.arange(M, device=kv.device)[None, :]
    want = torch.where(lens < 0, kv, lens)
    long = want > M * page
    want = torch.where(long, kv, want)
    had, have = (kv + page - 1) // page, (want + page - 1) // page
    gone = (col >= have[:, None]) & (col < had[:, None])
    refs.scatter_add_(0, table.long().flatten(), -gone.int().flatten())
    last = table.gather(1, (had - 1).clamp(min=0)[:, None].long())[:, 0]
    shared = (want > kv) & (kv % page != 0) & (refs[last.long()] > 1)
    need = torch.where(shared, 0, (have - had).clamp(min=0))
    end = need.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0]
    short = (need > 0) & (end > free.shape[0])
    status = torch.where(long, 3, torch.where(shared, 2, torch.where(short, 1, 0))).int()
    want, have = torch.where(shared | short, kv, want), torch.where(shared | short, had, have)
    new = (col >= had[:, None]) & (col < have[:, None])
    names = free[((end - need - had)[:, None] + col)[new]].int()
    table[new] = names
    refs[names.long()] = 1
    i = torch.arange(columns, device=kv.device)[None, :]
    j = (kv[:, None] + i).clamp(max=M * page - 1)
    slots = table.gather(1, (j // page).long()) * page + j % page
    slots = torch.where(i < (want - kv)[:, None], slots, -1).int()
    kv.copy_(want)
    return status, slots


def _fork(s):
    table, kv, refs, page = s["page_table"], s["kv_lens"], s["refs"], s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    col = torch.arange(table.shape[1], device=kv.device)[None, :]
    n, i = kv[parents], torch.arange(len(parents), device=kv.device)
    bad = (kv[children] != 0) | ((children[:, None] == children[None, :]) & (i[None, :] < i[:, None])).any(1)
    need = ((n % page != 0) & ~bad).long()
    end = need.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0]
    short = (need > 0) & (end > free.shape[0])
    good = ~(bad | short)
    rows = table[parents]
    keep = good[:, None] & (col < (n // page)[:, None])
    refs.scatter_add_(0, rows.long().flatten(), keep.int().flatten())
    part = good & (need > 0)
    to = free[(end - 1)[part]]
    src = rows.gather(1, (n // page).long()[:, None].clamp(max=table.shape[1] - 1))[:, 0].long()[part]
    rows = torch.where(keep, rows, table[children])
    rows[part] = rows[part].scatter(1, (n // page).long()[part][:, None], to.int()[:, None])
    refs[to] = 1
    table[children[good]] = rows[good]
    kv[children[good]] = n[good]
    off = torch.arange(page, device=kv.device)[None, :]
    m = off < (n % page)[part][:, None]
    a, b = (src[:, None] * page + off)[m], (to[:, None] * page + off)[m]
    for c in ("k_cache", "v_cache"):
        flat = s[c].flatten(1, 2)
        flat[:, b] = flat[:, a]
    return torch.where(bad, 2, torch.where(short, 1, 0)).int()


def _pages(s):
    state = (s["page_table"], s["kv_lens"], s["refs"])
    grown, slots = _resize(*state, s["grown"], s["page"], s["T"])
    forked = _fork(s)
    table, lens, refs = (t.clone() for t in state)
    cut, _ = _resize(*state, s["after"], s["page"])
    _resize(*state, s["before"], s["page"])
    return [grown, slots, forked, table, lens, refs, cut, *state, s["k_cache"], s["v_cache"]]


# ---- from the definitions, in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case.get("page", 0)
    if op == "window":
        if work(case)["flops"] > 3e12:
            return None
        kv, tl = _lengths(case)
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        G = case["Hq"] // case["Hkv"]
        for b in range(case["B"]):
            k, v = (s[c][b] if s["page_table"] is None else s[c][s["page_table"][b].long()].flatten(0, 1) for c in ("k_cache", "v_cache"))
            for t0 in range(0, tl[b], 512):
                t1 = min(tl[b], t0 + 512)
                p0, p1 = kv[b] - tl[b] + t0, kv[b] - tl[b] + t1
                lo = max(0, p0 - case["window"] + 1)
                at = torch.arange(p1, device="cuda")
                at = at[(at >= lo) | (at < case["sinks"])]
                p = torch.arange(p0, p1, device="cuda")[:, None]
                hide = (at > p) | ((p - at >= case["window"]) & (at >= case["sinks"]))
                for h in range(case["Hkv"]):
                    ks, vs = k[at, h].double(), v[at, h].double()
                    a = torch.einsum("tgd,jd->gtj", s["q"][b, t0:t1, h * G : h * G + G].double(), ks) * case["D"] ** -0.5
                    o[b, t0:t1, h * G : h * G + G] = torch.einsum("gtj,jd->tgd", torch.softmax(a.masked_fill(hide, NEG_INF), -1), vs)
        return o
    if op in ("norm_append", "norm", "norm_grad"):
        R, D = case["R"], case["D"]
        row = s["table"].double()[s["positions"].long()]
        z = torch.complex(row[..., : R // 2], row[..., R // 2 :])[..., None, :]
        lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, R // 2), slice(R // 2, R))

        def turned(x, z):
            y = x.clone()
            c = torch.complex(y[..., lo], y[..., hi]) * z
            y[..., lo], y[..., hi] = c.real, c.imag
            return y

        def size(x):
            return torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)

        if op == "norm_grad":
            dx, dw = [], []
            for c in ("q", "k"):
                x, g = s[c].double(), turned(s[c + "_grad"].double(), z.conj())
                r, w = size(x), s[c + "_weight"].double()
                dw.append(torch.einsum("bthd,bthd->d", g, x / r))
                # the derivative of x / r along each coordinate: (1 - x x' / (D r^2)) / r
                gw = g * w
                dx.append(gw / r - x * torch.einsum("bthd,bthd->bth", gw, x)[..., None] / (D * r**3))
            return [*dx, *dw]
        q, k = (turned(s[c].double() / size(s[c].double()) * s[c + "_weight"].double(), z) for c in ("q", "k"))
        if op == "norm":
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at, off = s["slots"].long() // page, s["slots"].long() % page
        kc[at, off], vc[at, off] = k, s["v"].double()
        return [q, kc, vc]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    table, kv = s["page_table"].cpu().numpy().copy(), s["kv_lens"].cpu().numpy().copy()

    def ints(x):
        return torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()

    if op == "compact":
        tl = s["tree_lens"].cpu().numpy()
        lens = []
        src, dst = [], []
        for b, path in enumerate(_accepted(case)):
            for i, t in enumerate(path):
                j0, j1 = kv[b] - tl[b] + t, kv[b] - tl[b] + i
                src.append((int(table[b, j0 // page]), j0 % page))
                dst.append((int(table[b, j1 // page]), j1 % page))
            lens.append(kv[b] - tl[b] + len(path))
        (sp, so), (dp, do) = (torch.tensor(x, device="cuda").t() for x in (src, dst))
        for c in (kc, vc):
            c[:, dp, do] = c[:, sp, so]
        return [ints(lens), kc, vc]
    refs = s["refs"].cpu().numpy().copy()

    def resize(lens, columns=0):
        status, slots, old = np.zeros(case["B"], np.int32), np.full((case["B"], columns), -1, np.int32), kv.copy()
        for b, n in enumerate(lens):
            if 0 <= n < kv[b]:
                for c in range(-(-n // page), -(-kv[b] // page)):
                    refs[table[b, c]] -= 1
                kv[b] = n
        free, taken = np.flatnonzero(refs == 0), 0
        want = refs.copy()
        for b, n in enumerate(lens):
            if n <= kv[b]:
                continue
            if kv[b] % page and want[table[b, kv[b] // page]] > 1:
                status[b] = 2
                continue
            names = range(-(-kv[b] // page), -(-n // page))
            taken += len(names)
            if len(names) and taken > len(free):
                status[b] = 1
                continue
            for c, f in zip(names, free[taken - len(names) : taken]):
                table[b, c], refs[f] = f, 1
            kv[b] = n
            for i in range(min(columns, n - old[b])):
                slots[b, i] = table[b, (old[b] + i) // page] * page + (old[b] + i) % page
        return status, slots

    _, grow, after, parents, children = _plan(case)
    grown, slots = resize(grow, case["T"])
    forked, free, taken = [], np.flatnonzero(refs == 0), 0
    for p, c in zip(parents, children):
        n, rest = kv[p] // page, kv[p] % page
        taken += int(rest > 0)
        if rest and taken > len(free):
            forked.append(1)
            continue
        table[c, :n] = table[p, :n]
        np.add.at(refs, table[p, :n], 1)
        if rest:
            f = int(free[taken - 1])
            table[c, n], refs[f] = f, 1
            for x in (kc, vc):
                x[:, f, :rest] = x[:, int(table[p, n]), :rest]
        kv[c] = kv[p]
        forked.append(0)
    mid = [ints(table), ints(kv), ints(refs)]
    cut, _ = resize(after + [0] * len(children))
    resize(s["before"].cpu().numpy())
    return [ints(grown), ints(slots), ints(forked), *mid, ints(cut), ints(table), ints(kv), ints(refs), kc, vc]
