"""Timing cases of the paged-cache and log-probability operators.

Four operators of one verification round are covered: the write of a window's
keys and values into a paged cache (with the per-head norms and the rotation),
the attention of the window's rows over that cache, the commit of an accepted
tree path inside it, and the log probabilities of given tokens.  With ``own``
false ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it calls the library.  ``exact`` computes the same values in 64
bits.
"""

import math

import numpy as np
import torch

own = False


# ---- cases ---------------------------------------------------------------------------

def _attend(name, B, N, H, Hkv, D, page, longest, ragged, cache, tree, short):
    return dict(name=name, op="attend", B=B, N=N, H=H, Hkv=Hkv, D=D, page=page, longest=longest,
                ragged=ragged, cache=cache, tree=tree, short=short)


def _append(name, B, N, H, Hkv, D, rot, interleaved, page, cache, before, short):
    return dict(name=name, op="append", B=B, N=N, H=H, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved,
                page=page, cache=cache, before=before, short=short)


def _commit(name, G, B, N, Hkv, D, page, pages, cache, deepest):
    return dict(name=name, op="commit", G=G, B=B, N=N, Hkv=Hkv, D=D, page=page, pages=pages, cache=cache,
                deepest=deepest)


def _logprob(name, R, V, dtype, T, k, pad):
    return dict(name=name, op="logprob", R=R, V=V, dtype=dtype, T=T, k=k, pad=pad)


def listed():
    return [
        # one request decoding one token after a short conversation: latency
        _attend("attend_one_1k", 1, 1, 32, 8, 128, 16, 1000, False, "bf16", False, False),
        # a serving batch decoding one token each, lengths from a few tokens to 8k
        _attend("attend_one_b64_8k", 64, 1, 32, 8, 128, 16, 8192, True, "bf16", False, False),
        # draft chains of up to 7 tokens (a window of 8 rows) over an 8-bit cache
        _attend("attend_chain_b32_e4m3", 32, 8, 32, 8, 128, 32, 4096, True, "e4m3", False, True),
        # the draft trees of 33 nodes that the tree verification takes, 64 requests
        _attend("attend_tree_b64_n33", 64, 33, 32, 8, 128, 16, 2048, True, "bf16", True, False),
        # one request with a long document behind it, a draft chain of 4
        _attend("attend_chain_b1_128k", 1, 5, 32, 8, 128, 64, 131000, False, "bf16", False, False),
        # one decoded token written to the cache: latency
        _append("append_one", 1, 1, 32, 8, 128, 128, False, 16, "bf16", 1000, False),
        # a batch of draft trees written to an 8-bit cache
        _append("append_tree_b64_e4m3", 64, 33, 32, 8, 128, 128, False, 16, "e4m3", 700, True),
        # a prompt chunk written to the cache
        _append("append_prompt_8k", 1, 8191, 32, 8, 128, 128, False, 64, "bf16", 37, False),
        # one request's accepted path, 36 layers of keys and values
        _commit("commit_b1", 72, 1, 33, 8, 128, 16, 4, "bf16", 5),
        # a batch's accepted paths, 36 layers of keys and values
        _commit("commit_b64", 72, 64, 33, 8, 128, 16, 4, "bf16", 7),
        # the emitted tokens of 8 rows with 5 alternatives each, fp32 logits: latency
        _logprob("logprob_8_f32", 8, 151936, "f32", 1.0, 5, False),
        # every row of a verification batch (B=256, K=7), 20 alternatives each
        _logprob("logprob_2048_bf16", 2048, 151936, "bf16", 0.7, 20, False),
    ]


def _is8(c):
    return c["cache"] == "e4m3"


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "commit", "logprob"])
    H, Hkv, D = rng.choice([(32, 8, 128), (12, 12, 64), (28, 4, 128), (40, 8, 128), (8, 1, 256), (25, 5, 64)])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "attend":
        B, N = _log(rng, 1, 96), rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 9, 64)])
        longest = _log(rng, 1, max(2, min(40000, 16000000 // (B * N * H), 400000000 // (B * Hkv * D))))
        return {k: v for k, v in _attend("", B, N, H, Hkv, D, page, longest, rng.random() < 0.7, cache,
                                         N > 2 and rng.random() < 0.5, rng.random() < 0.5).items() if k != "name"}
    if op == "append":
        B, N = _log(rng, 1, 128), _log(rng, 1, 4000)
        N = max(1, min(N, 8000 // B))
        rot = rng.choice([D, D, D // 2])
        return {k: v for k, v in _append("", B, N, H, Hkv, D, rot, rng.random() < 0.3, page, cache,
                                         _log(rng, 1, 3000), rng.random() < 0.5).items() if k != "name"}
    if op == "commit":
        B, N = _log(rng, 1, 64), _log(rng, 2, 64)
        return {k: v for k, v in _commit("", 2 * _log(rng, 1, 32), B, N, Hkv, D, page, -(-160 // page), cache,
                                         rng.randint(1, min(N - 1, 12))).items() if k != "name"}
    dtype = rng.choice(["bf16", "f32"])
    V = _log(rng, 100, 150000)
    R = _log(rng, 1, max(2, min(2000, 150000000 // V)))
    return {k: v for k, v in _logprob("", R, V, dtype, round(rng.uniform(0.4, 1.6), 2), rng.randint(0, 20),
                                      rng.random() < 0.5).items() if k != "name"}


# ---- what a case fixes apart from the seed: lengths -------------------------------------

def _spread(n, salt):
    """n numbers in [0, 1), the same for every seed."""
    i = np.arange(n, dtype=np.float64) + 1
    return np.modf(i * 0.6180339887498949 + salt * 0.7548776662466927)[0]


def _lengths(c):
    """(base, counts): cached tokens before the window and rows in the window, per request."""
    B, N = c["B"], c["N"]
    base = np.full(B, c["longest"] - min(N, c["longest"] - 1) if c["longest"] > 1 else 0)
    if c["ragged"]:
        # a few long requests and many shorter ones; the first has the longest
        base = np.floor(base * np.where(_spread(B, 1) < 0.5, _spread(B, 2), 0.1 + 0.9 * _spread(B, 3)))
        base[0] = c["longest"] - min(N, c["longest"] - 1)
    counts = np.full(B, N)
    if c["short"]:
        counts = 1 + np.floor(_spread(B, 4) * N)
        counts[0] = N
    return base.astype(np.int64), counts.astype(np.int64)


def _accepted(c):
    d = np.floor(_spread(c["B"], 5) * (c["deepest"] + 1)).astype(np.int64)
    d[0] = c["deepest"]
    return d


def work(case):
    c = case
    if c["op"] == "attend":
        base, counts = _lengths(c)
        row = 2 * c["Hkv"] * (c["D"] + 4 if _is8(c) else c["D"] * 2)
        rows = float(counts.sum()) * c["H"] * c["D"] * 2 * 2
        return {"bytes": float((base + counts).sum()) * row + rows,
                "flops": 4.0 * c["H"] * c["D"] * float(((base + counts / 2) * counts).sum())}
    if c["op"] == "append":
        T = float(_append_counts(c).sum())
        es = c["D"] + 4 if _is8(c) else c["D"] * 2
        return {"bytes": T * ((c["H"] + 2 * c["Hkv"]) * c["D"] * 2 + c["H"] * c["D"] * 2 + 2 * c["Hkv"] * es),
                "flops": T * (c["H"] + c["Hkv"]) * c["D"] * 7.0}
    if c["op"] == "commit":
        es = c["D"] + 4 if _is8(c) else c["D"] * 2
        return {"bytes": 2.0 * float(_accepted(c).sum()) * c["G"] * c["Hkv"] * es + 4.0 * c["B"] * (c["N"] + 4), "flops": 0}
    R = c["R"] - (_padded(c).sum() if c["pad"] else 0)
    return {"bytes": float(R) * c["V"] * (2 if c["dtype"] == "bf16" else 4) + c["R"] * (16 + 8.0 * c["k"]),
            "flops": 5.0 * float(R) * c["V"]}


def _append_counts(c):
    counts = np.full(c["B"], c["N"])
    if c["short"]:
        counts = 1 + np.floor(_spread(c["B"], 6) * c["N"])
        counts[0] = c["N"]
    return counts.astype(np.int64)


def _padded(c):
    return _spread(c["R"], 7) < 0.4 if c["R"] > 1 else np.zeros(1, bool)


# ---- inputs ----------------------------------------------------------------------------

def _dev():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _int(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).to(_dev())


def _trees(rng, B, N):
    """A main path of a third of the nodes with branches hanging off earlier nodes."""
    par = np.full((B, N), -1)
    for j in range(1, N):
        par[:, j] = j - 1 if j <= N // 3 else rng.integers(0, j, B)
    return par


def _quantise(x):
    """e4m3 values and one scale for each row of the last dimension."""
    s = (x.float().abs().amax(-1) / 448).clamp_min(1e-30)
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn), s


def _table(rng, B, P):
    return rng.permutation(B * P).reshape(B, P)


def prepare(case, seed):
    c, dev, g = case, _dev(), _gen(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32)

    s = dict(case)
    if c["op"] == "attend":
        B, N, H, Hkv, D, page = (c[k] for k in ("B", "N", "H", "Hkv", "D", "page"))
        base, counts = _lengths(c)
        P = int(-(-(base + N).max() // page))
        k, v = normal(B * P, Hkv, page, D), normal(B * P, Hkv, page, D)
        s["k_scales"] = s["v_scales"] = None
        if _is8(c):
            (k, s["k_scales"]), (v, s["v_scales"]) = _quantise(k), _quantise(v)
        s.update(q=normal(B, N, H, D) * 2.5, k=k, v=v, table=_int(_table(rng, B, P)), base=_int(base),
                 counts=_int(counts) if c["short"] else None,
                 parents=_int(_trees(rng, B, N)) if c["tree"] else None, scale=1 / math.sqrt(D),
                 out=torch.zeros(B, N, H, D, dtype=torch.bfloat16, device=dev),
                 lse=torch.zeros(B, N, H, device=dev))
    elif c["op"] == "append":
        B, N, H, Hkv, D, page, rot = (c[k] for k in ("B", "N", "H", "Hkv", "D", "page", "rot"))
        qkv = normal(B, N, (H + 2 * Hkv) * D) * 1.7  # the projection's output: q, k and v side by side
        base = np.floor(c["before"] * _spread(B, 8)).astype(np.int64)
        P = int(-(-(base + N).max() // page))
        most = int((base + N).max())
        angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * 1e6 ** (
            -torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        dt = torch.float8_e4m3fn if _is8(c) else torch.bfloat16
        pages = [torch.zeros(B * P, Hkv, page, D, dtype=torch.bfloat16, device=dev).to(dt) for _ in range(2)]
        scales = [torch.zeros(B * P, Hkv, page, device=dev) if _is8(c) else None for _ in range(2)]
        s.update(q=qkv[..., :H * D].unflatten(-1, (H, D)), k=qkv[..., H * D:(H + Hkv) * D].unflatten(-1, (Hkv, D)),
                 v=qkv[..., (H + Hkv) * D:].unflatten(-1, (Hkv, D)), wq=1 + 0.2 * normal(D), wk=1 + 0.2 * normal(D),
                 rope=torch.cat([angle.cos(), angle.sin()], 1).float(), k_pages=pages[0], v_pages=pages[1],
                 k_scales=scales[0], v_scales=scales[1], table=_int(_table(rng, B, P)), base=_int(base),
                 positions=_int(base[:, None] + np.arange(N)[None, :]),
                 counts=_int(_append_counts(c)) if c["short"] else None,
                 q_out=torch.zeros(B, N, H, D, dtype=torch.bfloat16, device=dev))
    elif c["op"] == "commit":
        G, B, N, Hkv, D, page, P = (c[k] for k in ("G", "B", "N", "Hkv", "D", "page", "pages"))
        kv = normal(G, B * P, Hkv, page, D)
        s["scales"] = None
        if _is8(c):
            kv, s["scales"] = _quantise(kv)
        d = _accepted(c)
        path = np.full((B, N), -1)
        for b in range(B):
            path[b, :d[b]] = np.sort(rng.choice(np.arange(1, N), d[b], replace=False))
        tree = rng.integers(0, page * P - N, B)
        s.update(kv=kv, table=_int(_table(rng, B, P)), tree_base=_int(tree), commit_base=_int(tree + 1),
                 accept_len=_int(d), path=_int(path))
    else:
        R, V = c["R"], c["V"]
        x = normal(R, V, dtype=torch.float32) * 2.0
        # a few plausible tokens stand out of each row
        at = torch.randint(0, V, (R, 12), generator=g, device=dev)
        x.scatter_add_(1, at, 8 + 4 * torch.rand(R, 12, generator=g, device=dev))
        tokens = at[:, 0].to(torch.int32)
        if c["pad"]:
            tokens = torch.where(torch.as_tensor(_padded(c), device=dev), -1, tokens).to(torch.int32)
        s.update(logits=x.bfloat16() if c["dtype"] == "bf16" else x, tokens=tokens)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The library's cache handle, which a program keeps beside its pages."""
    import draft_token_verification_04_amd as sv

    if s["op"] == "attend":
        s["cache_"] = sv.PagedKV(s["k"], s["v"], s["k_scales"], s["v_scales"])
    elif s["op"] == "append":
        s["cache_"] = sv.PagedKV(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])


# ---- one pass --------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend_plain, "append": _append_plain, "commit": _commit_plain,
            "logprob": _logprob_plain}[state["op"]](state)


def _run_own(s):
    import draft_token_verification_04_amd as sv

    if s["op"] == "attend":
        r = sv.spec_attend_paged(s["q"], s["cache_"], s["table"], s["base"], parents=s["parents"],
                                 counts=s["counts"], scale=s["scale"], out=s["out"], lse=s["lse"])
        return {"out": r["out"], "lse": r["lse"], "status": r["status"]}
    if s["op"] == "append":
        r = sv.spec_append_kv_paged(s["q"], s["k"], s["v"], s["cache_"], s["table"], s["base"], s["positions"],
                                    q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, rope=s["rope"],
                                    interleaved=s["interleaved"], counts=s["counts"], q_out=s["q_out"])
        return {"q": r["q"], "status": r["status"], "k": s["k_pages"], "v": s["v_pages"],
                "ks": s["k_scales"], "vs": s["v_scales"]}
    if s["op"] == "commit":
        st = sv.spec_commit_tree_kv_paged(s["kv"], s["table"], s["tree_base"], s["commit_base"], s["accept_len"],
                                          s["path"], scales=s["scales"])
        return {"kv": s["kv"], "scales": s["scales"], "status": st}
    r = sv.spec_token_logprobs(s["logits"], s["tokens"], temperature=s["T"], top_k=s["k"])
    out = {"logprob": r["logprob"], "entropy": r["entropy"], "status": r["status"]}
    if s["k"]:
        out.update(top_ids=r["top_ids"], top_logprobs=r["top_logprobs"])
    return out


def _rows(pages, scales, table):
    """A request's cached rows in order, as floats: [B, Hkv, P * page, D]."""
    x = pages[table.long()].float()
    if scales is not None:
        x = x * scales[table.long()][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend_plain(s):
    B, N, H, Hkv, D = (s[k] for k in ("B", "N", "H", "Hkv", "D"))
    G = H // Hkv
    k, v = _rows(s["k"], s["k_scales"], s["table"]), _rows(s["v"], s["v_scales"], s["table"])
    L, dev = k.shape[2], k.device
    n = torch.arange(N, device=dev)
    if s["parents"] is None:
        sees = (n[:, None] >= n[None, :]).expand(B, N, N)
    else:
        up = (s["parents"][:, :, None] == n).float() + torch.eye(N, device=dev)
        sees = torch.linalg.matrix_power(up, 64) > 0
    t = torch.arange(L, device=dev)[None, :] - s["base"][:, None]  # [B, L]: place in the window
    inside = (t >= 0) & (t < N)
    at = t.clamp(0, N - 1).long()
    mask = (t < 0)[:, None, :] | (inside[:, None, :] & sees.gather(2, at[:, None, :].expand(B, N, L)))
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    w = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    w = w.view(B, Hkv, N, G, L).masked_fill(~mask[:, None, :, None, :], -math.inf).view(B, Hkv, N * G, L)
    top = w.amax(-1, keepdim=True)
    e = torch.exp(w - top)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / z
    lse = (top + torch.log(z))[..., 0].view(B, Hkv, N, G).transpose(1, 2).reshape(B, N, H)
    o = o.view(B, Hkv, N, G, D).transpose(1, 2).reshape(B, N, H, D).to(torch.bfloat16)
    if s["counts"] is not None:
        there = n[None, :] < s["counts"][:, None]
        o = torch.where(there[:, :, None, None], o, s["out"])
        lse = torch.where(there[:, :, None], lse, s["lse"])
    return {"out": o, "lse": lse, "status": torch.zeros(B, dtype=torch.int32, device=dev)}


def _turn(x, rope, positions, rot, interleaved):
    cs = rope[positions.long()][:, :, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append_plain(s):
    B, N, page = s["B"], s["N"], s["page"]

    def normed(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        return _turn(x, s["rope"], s["positions"], s["rot"], s["interleaved"])

    q = normed(s["q"], s["wq"]).to(torch.bfloat16)
    n = torch.arange(N, device=q.device)
    slot = s["base"][:, None].long() + n
    there = torch.ones(B, N, dtype=torch.bool, device=q.device)
    if s["counts"] is not None:
        there = n[None, :] < s["counts"][:, None]
        q = torch.where(there[:, :, None, None], q, s["q_out"])
    pg = s["table"].long().gather(1, slot // page)
    out = {"q": q, "status": torch.zeros(B, N, dtype=torch.int32, device=q.device)}
    for name, x in (("k", normed(s["k"], s["wk"])), ("v", s["v"].float())):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        if scales is not None:
            top = x.abs().amax(-1)
            old = scales[pg, :, slot % page]
            scales[pg, :, slot % page] = torch.where(there[..., None], top / 448, old)
            x = x * torch.where(top > 0, 448 / top, 0)[..., None]
        x = x.to(pages.dtype)
        # written as bytes or 16-bit words, so that every type can be stored by index
        raw, x = (pages.view(torch.uint8), x.view(torch.uint8)) if scales is not None else (pages, x)
        raw[pg, :, slot % page] = torch.where(there[..., None, None], x, raw[pg, :, slot % page])
        out[name], out[name + "s"] = pages, scales
    return out


def _commit_plain(s):
    N, page = s["N"], s["page"]
    k = torch.arange(N, device=s["kv"].device)
    moved = k[None, :] < s["accept_len"][:, None]
    into = s["commit_base"][:, None].long() + k
    # slots behind an accepted path are written with what they hold; those past the table with the last one's
    into = into.clamp_max(s["pages"] * page - 1)
    src = torch.where(moved, s["tree_base"][:, None].long() + s["path"].long(), into)
    table = s["table"].long()
    ps, pd = table.gather(1, src // page), table.gather(1, into // page)
    for x in (s["kv"].view(torch.uint8) if s["scales"] is not None else s["kv"], s["scales"]):
        if x is not None:
            x[:, pd, :, into % page] = x[:, ps, :, src % page]
    return {"kv": s["kv"], "scales": s["scales"],
            "status": torch.zeros(s["B"], dtype=torch.int32, device=table.device)}


def _logprob_plain(s):
    x, k, V = s["logits"].float(), s["k"], s["V"]
    there = s["tokens"] >= 0
    top = x.amax(1, keepdim=True)
    d = (x - top) / s["T"]
    e = torch.exp(d)
    z = e.sum(1, keepdim=True)
    lz = torch.log(z)
    lp = d.gather(1, s["tokens"].clamp_min(0).long()[:, None]) - lz
    ent = lz - (e * d).sum(1, keepdim=True) / z
    zero = torch.zeros((), device=x.device)
    out = {"logprob": torch.where(there, lp[:, 0], zero), "entropy": torch.where(there, ent[:, 0], zero),
           "status": torch.zeros(len(x), dtype=torch.int32, device=x.device)}
    if k:
        # whole keys that order by value and then by the lowest index
        b = (x + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, -2147483648 - b, b) * (1 << 20) - torch.arange(V, device=x.device)
        ids = key.topk(k, 1).indices
        lps = d.gather(1, ids) - lz
        out["top_ids"] = torch.where(there[:, None], ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(there[:, None], lps, -math.inf)
    return out


# ---- the same in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attend": _attend_exact, "append": _append_exact, "commit": _commit_exact,
            "logprob": _logprob_exact}[case["op"]](s)


def _read(pages, scales, table_row, slots, page):
    """Rows `slots` of one request in 64 bits: [n, Hkv, D]."""
    pg = table_row.long()[slots // page]
    x = pages.view(torch.uint8)[pg, :, slots % page].view(pages.dtype) if scales is not None else pages[pg, :, slots % page]
    x = x.double()
    return x * scales[pg, :, slots % page].double()[..., None] if scales is not None else x


def _attend_exact(s):
    B, N, H, Hkv, D, page = (s[k] for k in ("B", "N", "H", "Hkv", "D", "page"))
    G = H // Hkv
    base = s["base"].tolist()
    counts = s["counts"].tolist() if s["counts"] is not None else [N] * B
    par = s["parents"].tolist() if s["parents"] is not None else None
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(B):
        c, n0 = counts[b], base[b]
        slots = torch.arange(n0 + c, device=out.device)
        k = _read(s["k"], s["k_scales"], s["table"][b], slots, page)
        v = _read(s["v"], s["v_scales"], s["table"][b], slots, page)
        ok = np.zeros((c, n0 + c), bool)
        ok[:, :n0] = True
        for j in range(c):
            if par is None:
                ok[j, n0:n0 + j + 1] = True
            else:
                a = j
                while a >= 0:
                    ok[j, n0 + a] = True
                    a = par[b][a]
        blocked = torch.as_tensor(~ok, device=out.device)
        for h in range(Hkv):
            q = s["q"][b, :c, h * G:(h + 1) * G].double()  # [c, G, D]
            w = (q.reshape(c * G, D) @ k[:, h].T.contiguous()).view(c, G, -1) * s["scale"]
            w = w.masked_fill(blocked[:, None, :], -math.inf)
            z = torch.logsumexp(w, -1)
            out[b, :c, h * G:(h + 1) * G] = (torch.exp(w - z[..., None]).view(c * G, -1) @ v[:, h]).view(c, G, D)
            lse[b, :c, h * G:(h + 1) * G] = z
    return {"out": out, "lse": lse, "status": None}


def _e4m3(x):
    """The nearest e4m3 value, ties to even, of each |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _append_exact(s):
    B, N, H, Hkv, D, rot, page = (s[k] for k in ("B", "N", "H", "Hkv", "D", "rot", "page"))
    half = rot // 2
    i = torch.arange(half, device=s["q"].device)
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    counts = s["counts"].tolist() if s["counts"] is not None else [N] * B
    base = s["base"].tolist()
    q_out = s["q_out"].double()
    got = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    scales = {n: None if s[n + "_scales"] is None else s[n + "_scales"].double() for n in ("k", "v")}
    for b in range(B):
        c = counts[b]
        r = s["rope"][s["positions"][b, :c].long()].double()
        cos, sin = r[:, None, :half], r[:, None, half:]

        def through(x, w):
            y = x[b, :c].double()
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
            u, t = y[..., first].clone(), y[..., second].clone()
            y[..., first] = u * cos - t * sin
            y[..., second] = t * cos + u * sin
            return y

        q_out[b, :c] = through(s["q"], s["wq"])
        slots = base[b] + torch.arange(c, device=i.device)
        pg = s["table"][b].long()[slots // page]
        for name, y in (("k", through(s["k"], s["wk"])), ("v", s["v"][b, :c].double())):
            if scales[name] is not None:
                top = y.abs().max(-1).values
                scales[name][pg, :, slots % page] = top / 448
                y = _e4m3(y * (448 / top)[..., None])
            got[name][pg, :, slots % page] = y
    return {"q": q_out, "status": None, "k": got["k"], "v": got["v"], "ks": scales["k"], "vs": scales["v"]}


def _commit_exact(s):
    page = s["page"]
    d, path = s["accept_len"].tolist(), s["path"].tolist()
    tb, cb = s["tree_base"].tolist(), s["commit_base"].tolist()
    table = s["table"].tolist()
    fresh = []
    for x in (s["kv"], s["scales"]):
        if x is None:
            fresh.append(None)
            continue
        raw = x.view(torch.uint8) if x.element_size() == 1 else x
        y = raw.clone()
        for b in range(s["B"]):
            for k in range(d[b]):
                src, dst = tb[b] + path[b][k], cb[b] + k
                y[:, table[b][dst // page], :, dst % page] = raw[:, table[b][src // page], :, src % page]
        fresh.append(y.view(x.dtype))
    return {"kv": fresh[0], "scales": fresh[1], "status": None}


def _logprob_exact(s):
    R, V, k = s["R"], s["V"], s["k"]
    dev = s["logits"].device
    lp, ent = torch.zeros(R, dtype=torch.float64, device=dev), torch.zeros(R, dtype=torch.float64, device=dev)
    tops = torch.full((R, k), -math.inf, dtype=torch.float64, device=dev)
    rows = max(1, 40000000 // V)
    for r0 in range(0, R, rows):
        x = s["logits"][r0:r0 + rows].double() / s["T"]
        z = torch.logsumexp(x, 1)
        tok = s["tokens"][r0:r0 + rows].long()
        live = tok >= 0
        logp = x - z[:, None]
        lp[r0:r0 + rows] = torch.where(live, logp.gather(1, tok.clamp_min(0)[:, None])[:, 0], 0)
        ent[r0:r0 + rows] = torch.where(live, -(logp.exp() * logp).sum(1), 0)
        if k:
            tops[r0:r0 + rows] = torch.where(live[:, None], logp.topk(k, 1).values, -math.inf)
    out = {"logprob": lp, "entropy": ent, "status": None}
    if k:
        out.update(top_ids=None, top_logprobs=tops)
    return out
