"""CPU oracle of the paged-cache operators and the token log probabilities
(test infrastructure), in 64 bits with numpy, one request, row and head at a
time.  It shares no code with the library.

A cache is a pair of float64 arrays [num_pages, kv_heads, page_size, head_dim]
holding the values the stored elements stand for; slot s of request b is row
s % page_size of page table[b][s // page_size].
"""

from __future__ import annotations

import numpy as np


def bf16_values(a: np.ndarray) -> np.ndarray:
    """float64 values of bf16 bit patterns (uint16)."""
    with np.errstate(invalid="ignore"):  # NaN patterns
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values(a: np.ndarray) -> np.ndarray:
    """float64 values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, 0x7f and 0xff are NaN."""
    a = a.astype(np.int64)
    s, e, m = a >> 7, (a >> 3) & 15, a & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def row_of(table_row, slot: int, page_size: int, num_pages: int):
    """(page, row) of a slot, or None where the slot or its page does not exist."""
    if slot < 0 or slot // page_size >= len(table_row):
        return None
    page = int(table_row[slot // page_size])
    if page < 0 or page >= num_pages:
        return None
    return page, slot % page_size


def norm_and_turn(x, weight, eps, angles, rot, interleaved):
    """One head: x / sqrt(mean(x^2) + eps) * weight, then the rotation.  angles is
    the position's row of the table (rot/2 cosines, rot/2 sines) or None.
    Returns the result and, per value, the sum of the magnitudes that were
    added for it (what its rounding errors are relative to)."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y) + eps) * weight
    mag = np.abs(y)
    if angles is not None:
        half = rot // 2
        z, zm = y.copy(), mag.copy()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(angles[i]), float(angles[half + i])
            z[a], z[b] = y[a] * c - y[b] * s, y[b] * c + y[a] * s
            zm[a], zm[b] = abs(y[a] * c) + abs(y[b] * s), abs(y[b] * c) + abs(y[a] * s)
        y, mag = z, zm
    return y, mag


def ancestors(parents, n: int):
    """Tokens of the window that token n sees: itself and its ancestors."""
    seen = []
    while n >= 0:
        seen.append(n)
        n = int(parents[n])
    return sorted(seen)


def parents_ok(parents, count: int) -> bool:
    return all((int(parents[j]) == -1) if j == 0 else 0 <= int(parents[j]) < j for j in range(count))


def attend(q, k, v, table, base, counts, parents, scale):
    """q [B, N, H, D]; k, v caches (float64); parents [B, N] or None.

    Returns dict: out, lse, status, and for the tolerances of a comparison
    ``mean_abs`` (softmax-weighted mean of |v|), ``score_mag`` (the largest
    scale * sum |q_d k_d| of the row) and ``seen`` (bool [B, N]: rows in use)."""
    B, N, H, D = q.shape
    num_pages, Hkv, page_size, _ = k.shape
    G = H // Hkv
    out = np.zeros((B, N, H, D))
    lse = np.full((B, N, H), -np.inf)
    mean_abs, score_mag = np.zeros((B, N, H, D)), np.zeros((B, N, H))
    status, seen = np.zeros(B, np.int32), np.zeros((B, N), bool)
    for b in range(B):
        c = N if counts is None else min(max(int(counts[b]), 0), N)
        seen[b, :c] = True
        first = int(base[b])
        if first < 0 or first + c > table.shape[1] * page_size:
            status[b] = 1
            continue
        if parents is not None and not parents_ok(parents[b], c):
            status[b] = 2
            continue
        if c == 0:
            continue
        where = [row_of(table[b], s, page_size, num_pages) for s in range(first + c)]
        if any(w is None for w in where):
            status[b] = 1
            continue
        pg, rw = np.array([w[0] for w in where]), np.array([w[1] for w in where])
        for n in range(c):
            own = list(range(n + 1)) if parents is None else ancestors(parents[b], n)
            slots = np.array(list(range(first)) + [first + t for t in own])
            for h in range(H):
                kk, vv = k[pg[slots], h // G, rw[slots]], v[pg[slots], h // G, rw[slots]]
                with np.errstate(invalid="ignore", over="ignore"):
                    w = scale * (kk @ q[b, n, h])
                    score_mag[b, n, h] = np.max(scale * (np.abs(kk) @ np.abs(q[b, n, h])))
                    m = w.max()
                    e = np.exp(w - m)
                    out[b, n, h] = (e[:, None] * vv).sum(0) / e.sum()
                    mean_abs[b, n, h] = (e[:, None] * np.abs(vv)).sum(0) / e.sum()
                    lse[b, n, h] = m + np.log(e.sum())
    return dict(out=out, lse=lse, status=status, mean_abs=mean_abs, score_mag=score_mag, seen=seen)


def commit_paged(pages, scales, table, tree_base, commit_base, accept_len, path):
    """pages uint8 [G, num_pages, kv_heads, page_size, row_bytes], scales like it
    without the last dimension or None.  Returns (pages, scales, status) after
    the commit; every source row is read as it was on entry."""
    G, num_pages, _, page_size, _ = pages.shape
    B, N = path.shape
    out, souts = pages.copy(), None if scales is None else scales.copy()
    status = np.zeros(B, np.int32)
    for b in range(B):
        d = int(accept_len[b])
        p = [int(x) for x in path[b, :max(d, 0)]]
        if d < 0 or d > N - 1 or any(x < 1 or x >= N for x in p) or any(y <= x for x, y in zip(p, p[1:])):
            status[b] = 2
            continue
        src = [row_of(table[b], int(tree_base[b]) + x, page_size, num_pages) for x in p]
        dst = [row_of(table[b], int(commit_base[b]) + i, page_size, num_pages) for i in range(d)]
        if any(x is None for x in src + dst):
            status[b] = 1
            continue
        if d and tree_base[b] + 2 <= commit_base[b] < tree_base[b] + N:
            status[b] = 3
            continue
        for s, t in zip(src, dst):
            out[:, t[0], :, t[1]] = pages[:, s[0], :, s[1]]
            if scales is not None:
                souts[:, t[0], :, t[1]] = scales[:, s[0], :, s[1]]
    return out, souts, status


def token_logprobs(x, tokens, T, k):
    """x [R, V] float64 logits.  Returns logprob, entropy, top_ids, top_logprobs,
    status and ``spread``: sum p (d^2 + |d| + 1), d = log2 of p over the largest p,
    which bounds how far rounding of the terms moves the sums."""
    R, V = x.shape
    lp, ent, spread = np.zeros(R), np.zeros(R), np.zeros(R)
    ids, tops = np.full((R, k), -1, np.int64), np.full((R, k), -np.inf)
    status = np.zeros(R, np.int32)
    for r in range(R):
        t = None if tokens is None else int(tokens[r])
        if t == -1:
            continue
        m = x[r].max()
        order = np.lexsort((np.arange(V), -x[r]))[:k]
        ids[r] = order
        if m == -np.inf:
            if t is not None:
                lp[r] = -np.inf
                status[r] = 0 if 0 <= t < V else 1
            continue
        d = (x[r] - m) / T
        e = np.exp(d)
        z = e.sum()
        p = e / z
        f = np.where(np.isfinite(d), d, 0) / np.log(2)
        spread[r] = (p * (f * f + np.abs(f) + 1)).sum()
        ent[r] = np.log(z) - (e * np.where(np.isfinite(d), d, 0)).sum() / z
        logp = d - np.log(z)
        tops[r] = logp[order]
        if t is not None:
            ok = 0 <= t < V
            status[r] = 0 if ok else 1
            lp[r] = logp[t] if ok else -np.inf
    return dict(logprob=lp, entropy=ent, top_ids=ids, top_logprobs=tops, status=status, spread=spread)
