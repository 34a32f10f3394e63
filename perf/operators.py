"""Cases of the decoding step's operators: 4-bit linear layers, rotary positions,
attention for a tree of drafted tokens over a cache, and logit penalties.

`run` computes one pass of one operator: with `own` through the package's entry
points, without it from elementary torch operations in 32 bits."""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NEG_INF = float("-inf")


def listed():
    return [
        # a small projection of one token, odd sizes: latency counts
        dict(name="w4 token small", op="w4", T=1, m=1000, n=2051, dtype="f16", group=64, zeros=True),
        # the decoding layer's shape for one token, in the decoding layer's type
        dict(name="w4 token layer", op="w4", T=1, m=4096, n=11008, dtype="f32", group=128, zeros=False),
        # the last product of a step with a drafted tree: every token against the whole vocabulary
        dict(name="w4 tree vocabulary", op="w4", T=24, m=128000, n=4096, dtype="bf16", group=128, zeros=True),
        # one step of a few drafted tokens: rotate q and k, put k and v into the paged cache
        dict(name="rotary append step", op="append", N=5, Hq=32, Hkv=8, D=128, R=128, page=16, interleaved=False, dtype="bf16"),
        # a long prompt, half of each head rotated
        dict(name="rotary prompt", op="rotary", B=2, T=8191, Hq=32, Hkv=8, D=128, R=64, interleaved=False, grad=False,
             heads_first=False, dtype="bf16"),
        # the gradient through the rotation of a training batch, heads before tokens
        dict(name="rotary gradient", op="rotary", B=4, T=2048, Hq=16, Hkv=16, D=96, R=96, interleaved=True, grad=True,
             heads_first=True, dtype="f32"),
        # one sequence, one token: plain decoding over a contiguous cache
        dict(name="attention token", op="tree", B=1, T=1, Hq=32, Hkv=8, D=128, S=2001, page=0, ragged=False, dtype="bf16"),
        # a serving batch of small trees, every sequence with a length of its own, paged
        dict(name="attention tree batch", op="tree", B=16, T=12, Hq=32, Hkv=8, D=128, S=4096, page=16, ragged=True, dtype="bf16"),
        # a few long contexts with wide trees
        dict(name="attention tree long", op="tree", B=4, T=48, Hq=32, Hkv=4, D=128, S=32768, page=64, ragged=False, dtype="f16"),
        # one sequence's logits
        dict(name="logits token", op="logits", B=1, V=32000, L=700, NB=16, mask=True, dtype="f32"),
        # a batch with long histories over an odd vocabulary
        dict(name="logits long history", op="logits", B=12, V=100003, L=20000, NB=0, mask=False, dtype="f16"),
        # a large batch with everything on
        dict(name="logits batch", op="logits", B=96, V=128000, L=4096, NB=64, mask=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w4", "append", "rotary", "tree", "tree", "logits"])
    if op == "w4":
        return dict(op=op, T=_log(rng, 1, 32), m=_log(rng, 256, 32768), n=_log(rng, 256, 12000), dtype=rng.choice(["f32", "f16", "bf16"]),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    if op in ("append", "rotary"):
        D = rng.choice([64, 80, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, Hq=hkv * rng.choice([1, 2, 4, 6]), Hkv=hkv, D=D, R=rng.choice([D, D, D // 2]),
                 interleaved=rng.random() < 0.5, dtype=rng.choice(["f32", "f16", "bf16"]))
        if op == "append":
            return dict(c, N=_log(rng, 1, 2048), page=rng.choice([1, 16, 24, 64]))
        return dict(c, B=_log(rng, 1, 8), T=_log(rng, 1, 1024), grad=rng.random() < 0.5, heads_first=rng.random() < 0.5)
    if op == "tree":
        while True:
            hkv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, B=_log(rng, 1, 64), T=rng.choice([1, _log(rng, 1, 64)]), Hq=hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=hkv,
                     D=rng.choice([64, 96, 128, 128, 256]), S=_log(rng, 64, 32768), page=rng.choice([0, 16, 24, 64, 256]),
                     ragged=rng.random() < 0.7, dtype=rng.choice(["f16", "bf16"]))
            w = work(c)
            if w["bytes"] <= 2.5e8 and w["flops"] <= 5e10:
                return c
    return dict(op=op, B=_log(rng, 1, 64), V=_log(rng, 1000, 160000), L=_log(rng, 1, 20000), NB=rng.choice([0, _log(rng, 1, 300)]),
                mask=rng.random() < 0.6, dtype=rng.choice(["f32", "f16", "bf16"]))


def _lengths(case):
    """Entries in the cache (drafted ones among them) and drafted tokens of every sequence: fixed by the case."""
    B, T, S = case["B"], case["T"], case["S"]
    if not case["ragged"]:
        return [S] * B, [T] * B
    r = random.Random(B * 1000003 + T * 1009 + S)
    tl = [r.randint(1, T) for _ in range(B)]
    return [r.randint(max(S // 8, tl[b]), S) for b in range(B)], tl


def work(case):
    e, op = _SIZE[case["dtype"]], case["op"]
    if op == "w4":
        T, m, n = case["T"], case["m"], case["n"]
        groups = -(-n // case["group"])
        return {"bytes": m * -(-n // 2) + m * groups * (2 if case["zeros"] else 1) + m * groups * (e - 1) + T * (n + m) * e,
                "flops": 2.0 * T * m * n}
    if op in ("append", "rotary"):
        n = case["N"] if op == "append" else case["B"] * case["T"]
        heads = case["Hq"] + case["Hkv"] * (2 if op == "append" else 1)
        tokens = n if op == "append" else case["T"]
        return {"bytes": 2 * n * heads * case["D"] * e + tokens * case["R"] * 4 + n * (12 if op == "append" else 4),
                "flops": 3.0 * n * (case["Hq"] + case["Hkv"]) * case["R"]}
    if op == "tree":
        kv, tl = _lengths(case)
        rows = case["B"] * case["T"] * case["Hq"]
        pairs = sum(k * t for k, t in zip(kv, tl)) * case["Hq"]
        return {"bytes": 2 * sum(kv) * case["Hkv"] * case["D"] * e + 2 * rows * case["D"] * e + 8 * case["B"] * case["T"],
                "flops": 4.0 * case["D"] * pairs}
    B, V = case["B"], case["V"]
    return {"bytes": B * V * (e + 4) + 4 * B * case["L"] + (4 * B * -(-V // 32) if case["mask"] else 0) + 8 * B * case["NB"] + 20 * B,
            "flops": 6.0 * B * V}


def _table(positions, R, base=10000.0):
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    a = np.arange(positions, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    dt, op = _DT[case["dtype"]], case["op"]
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    if op == "w4":
        m, n = case["m"], case["n"]
        groups, cols = -(-n // case["group"]), -(-n // 2)
        # rows start on 16-byte boundaries
        q = torch.randint(0, 256, (m, -(-cols // 16) * 16), generator=g, device="cuda", dtype=torch.uint8)
        s["q"] = q[:, :cols]
        s["scales"] = (torch.rand((m, groups), generator=g, device="cuda") * 0.004 + 0.001).to(dt)
        s["zero"] = torch.randint(4, 12, (m, groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["x"] = normal(case["T"], n)
    elif op == "append":
        N, hkv, D, page = case["N"], case["Hkv"], case["D"], case["page"]
        pages = -(-(N + N // 2 + 3) // page)
        s["q"], s["k"], s["v"] = normal(N, case["Hq"], D), normal(N, hkv, D), normal(N, hkv, D)
        s["k_cache"], s["v_cache"] = normal(pages, page, hkv, D), normal(pages, page, hkv, D)
        s["slots"] = torch.from_numpy(r.permutation(pages * page)[:N].astype(np.int32)).cuda()
        s["positions"] = torch.from_numpy(r.integers(0, 4096, N).astype(np.int32)).cuda()
        s["table"] = _table(4096, case["R"])
    elif op == "rotary":
        B, T, D = case["B"], case["T"], case["D"]

        def heads(h):
            return normal(B, h, T, D).transpose(1, 2) if case["heads_first"] else normal(B, T, h, D)

        s["q"], s["k"] = heads(case["Hq"]), heads(case["Hkv"])
        first = torch.from_numpy(r.integers(0, 64, (B, 1)).astype(np.int32)).cuda()
        s["positions"] = (torch.arange(T, device="cuda", dtype=torch.int32)[None, :] + first).contiguous()
        s["table"] = _table(T + 64, case["R"])
    elif op == "tree":
        B, T, hkv, D, S, page = (case[k] for k in ("B", "T", "Hkv", "D", "S", "page"))
        kv, tl = _lengths(case)
        s["q"] = normal(B, T, case["Hq"], D)
        if page:
            per = -(-S // page)
            s["k_cache"], s["v_cache"] = normal(B * per, page, hkv, D), normal(B * per, page, hkv, D)
            s["page_table"] = torch.from_numpy(r.permutation(B * per).astype(np.int32).reshape(B, per)).cuda()
        else:
            s["k_cache"], s["v_cache"] = normal(B, S, hkv, D), normal(B, S, hkv, D)
            s["page_table"] = None
        bits = np.zeros((B, T), np.uint64)  # node i sees itself and its ancestors; node 0 is the last accepted token
        for b in range(B):
            for i in range(T):
                bits[b, i] = np.uint64(1 << i) | (bits[b, r.integers(max(0, i - 6), i)] if i else np.uint64(0))
        s["tree"] = torch.from_numpy(bits.view(np.int64)[:, :, None].copy()).cuda()
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["tree_lens"] = torch.tensor(tl, dtype=torch.int32, device="cuda")
    else:
        B, V, L, NB = case["B"], case["V"], case["L"], case["NB"]
        s["logits"] = (torch.randn((B, V), generator=g, device="cuda") * 4).to(dt)
        ids = torch.rand((B, L), generator=g, device="cuda") ** 3  # few tokens are frequent, many are rare
        s["history"] = (ids * V).to(torch.int32).clamp_(max=V - 1)
        lens = r.integers((L + 1) // 2, L + 1, B)
        s["history_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["prompt_lens"] = torch.from_numpy((lens * r.random(B)).astype(np.int32)).cuda()
        for k, lo, hi in (("repetition", 1.0, 1.4), ("presence", 0.0, 1.0), ("frequency", 0.0, 0.5)):
            s[k] = torch.from_numpy(r.uniform(lo, hi, B).astype(np.float32)).cuda()
        s["bias_ids"] = s["bias_vals"] = s["allowed"] = None
        if NB:
            s["bias_ids"] = torch.from_numpy(np.stack([r.choice(V, NB, replace=False) for _ in range(B)]).astype(np.int32)).cuda()
            s["bias_vals"] = torch.from_numpy(r.normal(0, 5, (B, NB)).astype(np.float32)).cuda()
        if case["mask"]:
            s["allowed"] = torch.randint(-2**31, 2**31, (B, -(-V // 32)), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    return s


def run(s):
    if own:
        return _own(s)
    return {"w4": _w4, "append": _append, "rotary": _rotary, "tree": _tree, "logits": _logits}[s["op"]](s)


def _own(s):
    import dynamic_sparsity_spmspv_gb300 as dbs

    op = s["op"]
    if op == "w4":
        return dbs.w4_linear(s["x"], s["q"], s["scales"], s["zero"], group=s["group"])
    if op == "append":
        q = dbs.rotary_append(s["q"], s["k"], s["v"], s["table"], s["positions"], s["k_cache"], s["v_cache"], s["slots"],
                              interleaved=s["interleaved"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "rotary":
        return dbs.rotary(s["q"], s["k"], s["table"], s["positions"], interleaved=s["interleaved"], transposed=s["grad"])
    if op == "tree":
        return dbs.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["kv_lens"], s["tree"], tree_lens=s["tree_lens"],
                                  page_table=s["page_table"])
    return dbs.penalize_logits(s["logits"], history=s["history"], history_lens=s["history_lens"], prompt_lens=s["prompt_lens"],
                               repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"],
                               bias_vals=s["bias_vals"], allowed=s["allowed"])


# ---- plain forms ----


def _w4(s):
    n, group = s["n"], s["group"]
    w = torch.stack([s["q"] & 15, s["q"] >> 4], 2).flatten(1)[:, :n].float()
    z = 8.0 if s["zero"] is None else s["zero"].float().repeat_interleave(group, 1)[:, :n]
    w = (w - z) * s["scales"].float().repeat_interleave(group, 1)[:, :n]
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def _turn(x, cos, sin, R, interleaved):
    """x [..., heads, D], cos and sin [..., 1, R/2]."""
    y = x.float()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., : R // 2], y[..., R // 2 : R])
    u, v = a * cos - b * sin, a * sin + b * cos
    t = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([t, y[..., R:]], -1).to(x.dtype)


def _append(s):
    R = s["R"]
    row = s["table"][s["positions"].long()][:, None, :]
    cos, sin = row[..., : R // 2], row[..., R // 2 :]
    q = _turn(s["q"], cos, sin, R, s["interleaved"])
    k = _turn(s["k"], cos, sin, R, s["interleaved"])
    at = s["slots"].long()
    s["k_cache"].flatten(0, 1)[at] = k
    s["v_cache"].flatten(0, 1)[at] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _rotary(s):
    R = s["R"]
    row = s["table"][s["positions"].long()][:, :, None, :]
    cos, sin = row[..., : R // 2], row[..., R // 2 :]
    if s["grad"]:
        sin = -sin
    return tuple(_turn(s[k], cos, sin, R, s["interleaved"]) for k in ("q", "k"))


def _tree(s):
    B, T, hq, hkv, D, S = (s[k] for k in ("B", "T", "Hq", "Hkv", "D", "S"))
    k, v = s["k_cache"], s["v_cache"]
    if s["page_table"] is not None:
        at = s["page_table"].long()
        k, v = k[at].flatten(1, 2)[:, :S], v[at].flatten(1, 2)[:, :S]
    k, v = k.float().permute(0, 2, 3, 1), v.float().permute(0, 2, 1, 3)
    q = s["q"].float().reshape(B, T, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D)
    p = (q @ k) / math.sqrt(D)
    node = torch.arange(S, device=q.device)[None, :] - (s["kv_lens"] - s["tree_lens"])[:, None]
    seen = (s["tree"] >> node.clamp(0, 63)[:, None, :]) & 1
    seen = (node[:, None, :] < 0) | (seen.bool() & (node < s["tree_lens"][:, None])[:, None, :])
    seen = seen & (torch.arange(T, device=q.device)[None, :] < s["tree_lens"][:, None])[:, :, None]
    seen = seen[:, None, :, None, :].expand(B, 1, T, hq // hkv, S).reshape(B, 1, -1, S)
    p = p.masked_fill_(~seen, NEG_INF)
    top = p.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = (p - top).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_(min=1e-30)
    return o.reshape(B, hkv, T, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, hq, D).to(s["q"].dtype)


def _logits(s):
    B, V, L = s["B"], s["V"], s["L"]
    at, j = s["history"].long(), torch.arange(L, device=s["logits"].device)[None, :]
    used, out = j < s["history_lens"][:, None], j >= s["prompt_lens"][:, None]
    seen = torch.zeros((B, V), device=at.device).scatter_add_(1, at, used.float())
    count = torch.zeros((B, V), device=at.device).scatter_add_(1, at, (used & out).float())
    x = s["logits"].float()
    rep = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - count * s["frequency"][:, None] - (count > 0) * s["presence"][:, None]
    if s["bias_ids"] is not None:
        x.scatter_add_(1, s["bias_ids"].long(), s["bias_vals"])
    if s["allowed"] is not None:
        v = torch.arange(V, device=at.device)
        x = x.masked_fill_((s["allowed"][:, v // 32] >> (v % 32)) & 1 == 0, NEG_INF)
    return x


# ---- from the definitions, in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "w4":
        x, parts = s["x"].double(), []
        group = torch.arange(case["n"], device="cuda") // case["group"]
        for i in range(0, case["m"], 8192):
            q = s["q"][i : i + 8192].to(torch.int16)
            w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = q % 16, q // 16
            w = w[:, : case["n"]]
            w -= 8 if s["zero"] is None else s["zero"][i : i + 8192].double()[:, group]
            w *= s["scales"][i : i + 8192].double()[:, group]
            parts.append(torch.einsum("tj,ij->ti", x, w))
        return torch.cat(parts, 1)
    if op in ("append", "rotary"):
        R, grad = case["R"], case.get("grad", False)
        row = s["table"].double()[s["positions"].long()]
        z = torch.complex(row[..., : R // 2], row[..., R // 2 :])[..., None, :]
        z = z.conj() if grad else z

        def turned(x):
            y = x.double().clone()
            lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
            c = torch.complex(y[..., lo], y[..., hi]) * z
            y[..., lo], y[..., hi] = c.real, c.imag
            return y

        if op == "rotary":
            return turned(s["q"]), turned(s["k"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        page, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        kc[page, off], vc[page, off] = turned(s["k"]), s["v"].double()
        return [turned(s["q"]), kc, vc]
    if op == "tree":
        if work(case)["flops"] > 2e11:
            return None
        kv, tl = _lengths(case)
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        tree = s["tree"][:, :, 0].cpu().numpy().view(np.uint64)
        per = case["Hq"] // case["Hkv"]
        for b in range(case["B"]):
            k, v = (s[c] if s["page_table"] is None else s[c][s["page_table"][b].long()].flatten(0, 1)[None] for c in ("k_cache", "v_cache"))
            k, v = (c[b if s["page_table"] is None else 0, : kv[b]].double() for c in (k, v))
            see = np.ones((tl[b], kv[b]), bool)
            for t in range(tl[b]):
                see[t, kv[b] - tl[b] :] = [(int(tree[b, t]) >> i) & 1 for i in range(tl[b])]
            hide = torch.from_numpy(~see).cuda()
            for h in range(case["Hq"]):
                a = (s["q"][b, : tl[b], h].double() @ k[:, h // per].t()) * case["D"] ** -0.5
                o[b, : tl[b], h] = torch.softmax(a.masked_fill(hide, NEG_INF), 1) @ v[:, h // per]
        return o
    x = s["logits"].double().cpu().numpy()
    hist, hl, pl = (s[k].cpu().numpy() for k in ("history", "history_lens", "prompt_lens"))
    rep, pres, freq = (s[k].double().cpu().numpy() for k in ("repetition", "presence", "frequency"))
    for b in range(case["B"]):
        ids = np.unique(hist[b, : hl[b]])
        x[b, ids] = np.where(x[b, ids] > 0, x[b, ids] / rep[b], x[b, ids] * rep[b])
        ids, c = np.unique(hist[b, pl[b] : hl[b]], return_counts=True)
        x[b, ids] -= c * freq[b] + pres[b]
        if s["bias_ids"] is not None:
            np.add.at(x[b], s["bias_ids"][b].cpu().numpy(), s["bias_vals"][b].double().cpu().numpy())
        if s["allowed"] is not None:
            words = s["allowed"][b].cpu().numpy().view(np.uint8)
            x[b, np.unpackbits(words, bitorder="little")[: case["V"]] == 0] = NEG_INF
    return torch.from_numpy(x).cuda()
