"""CPU oracle of the prompt operators (test infrastructure), in 64 bits with numpy:
the RMS norm with the residual's addition, the product of block-scaled operands, and
the cache write and causal attention of packed sequences.  It shares no code with the
library.  Caches are as in ``oracle.paged``."""

from __future__ import annotations

import numpy as np

from oracle.paged import norm_and_turn, row_of

BLOCK = 128


def rms_norm(x, residual, weight, eps):
    """(h, y): the sum and its norm."""
    h = np.array(x, dtype=np.float64)
    if residual is not None:
        h = h + residual
    y = np.empty_like(h)
    for t in range(len(h)):
        y[t] = h[t] / np.sqrt(np.mean(h[t] ** 2) + eps)
    return h, y if weight is None else y * weight


def block_scales(y):
    """[blocks, T]: max |y| / 448 of each row and 128 columns."""
    T, D = y.shape
    out = np.zeros((-(-D // BLOCK), T))
    for b in range(out.shape[0]):
        out[b] = np.abs(y[:, b * BLOCK:(b + 1) * BLOCK]).max(1) / 448
    return out


def linear(x, xs, w, ws):
    """x [M, K], xs [blocks of K, M], w [N, K], ws [blocks of N, blocks of K].  Returns
    the product, the sum of its terms' magnitudes, and the sum over the blocks of K of
    a bound of their largest term (what rounding errors are relative to)."""
    M, K = x.shape
    N = w.shape[0]
    out, mag, top = (np.zeros((M, N)) for _ in range(3))
    for b in range(-(-K // BLOCK)):
        k = slice(b * BLOCK, min((b + 1) * BLOCK, K))
        s = np.outer(xs[b], np.repeat(ws[:, b], BLOCK)[:N])
        out += s * (x[:, k] @ w[:, k].T)
        mag += np.abs(s) * (np.abs(x[:, k]) @ np.abs(w[:, k]).T)
        top += np.abs(s) * np.outer(np.abs(x[:, k]).max(1), np.abs(w[:, k]).max(1))
    return out, mag, top


def requests(starts, T):
    """(request, first token, tokens) of every request whose bounds are well formed."""
    return [(b, int(lo), int(hi - lo)) for b, (lo, hi) in enumerate(zip(starts, starts[1:])) if 0 <= lo <= hi <= T]


def append_rows(x, weight, eps, rope, rot, interleaved, positions, pair_axis, starts):
    """Every head of every token x [T, heads, D] through norm and rotation, positions
    [axes, T], pair_axis [rot / 2] or None.  Returns values and magnitudes (NaN for
    tokens outside every request)."""
    T, H, D = x.shape
    y, mag = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan)
    for _, first, n in requests(starts, T):
        for t in range(first, first + n):
            angles = None
            if rope is not None:
                axis = np.zeros(rot // 2, int) if pair_axis is None else np.asarray(pair_axis)
                at = positions[axis, t]
                i = np.arange(rot // 2)
                angles = np.concatenate([rope[at, i], rope[at, rot // 2 + i]]).astype(np.float64)
            for h in range(H):
                y[t, h], mag[t, h] = norm_and_turn(x[t, h], weight, eps, angles, rot, interleaved)
    return y, mag


def attend_packed(q, k, v, table, starts, base, scale):
    """q [T, H, D]; k, v caches in float64.  Returns dict as ``oracle.paged.attend``, with
    a leading dimension of 1: out [1, T, H, D], lse [1, T, H], mean_abs, score_mag, seen
    [1, T] (tokens of some request), and status [B]."""
    T, H, D = q.shape
    num_pages, Hkv, page_size, _ = k.shape
    out, mean_abs = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, score_mag = np.full((T, H), -np.inf), np.zeros((T, H))
    seen = np.zeros(T, bool)
    status = np.full(len(starts) - 1, 2, np.int32)
    for b, first, n in requests(starts, T):
        seen[first:first + n] = True
        before = 0 if base is None else int(base[b])
        status[b] = 0
        good = 0  # slots before the first that does not exist
        want = before + n if n else 0
        where = []
        if before >= 0:
            for s in range(want):
                r = row_of(table[b], s, page_size, num_pages)
                if r is None:
                    break
                where.append(r)
            good = len(where)
        if n and (before < 0 or good < want):
            status[b] = 1
        rows = max(0, min(n, good - before)) if before >= 0 else 0
        if rows == 0:
            continue
        at = slice(first, first + rows)
        pg, rw = np.array([w[0] for w in where]), np.array([w[1] for w in where])
        unseen = np.arange(good)[None, :] > before + np.arange(rows)[:, None]
        for h in range(H):
            kk, vv = k[pg, h * Hkv // H, rw], v[pg, h * Hkv // H, rw]
            with np.errstate(invalid="ignore", over="ignore"):
                w = np.where(unseen, -np.inf, scale * (q[at, h] @ kk.T))
                m = np.where(unseen, 0, scale * (np.abs(q[at, h]) @ np.abs(kk).T))
                score_mag[at, h] = m.max(1)
                top = w.max(1)
                e = np.exp(w - top[:, None])
                lse[at, h] = top + np.log(e.sum(1))
                if np.isfinite(vv).all():
                    out[at, h] = (e @ vv) / e.sum(1)[:, None]
                    mean_abs[at, h] = (e @ np.abs(vv)) / e.sum(1)[:, None]
                else:  # a masked slot's value reaches no row
                    for j in range(rows):
                        x = vv[:before + j + 1]
                        p = (e[j, :before + j + 1] / e[j].sum())[:, None]
                        out[first + j, h] = (p * x).sum(0)
                        mean_abs[first + j, h] = (p * np.abs(x)).sum(0)
    return dict(out=out[None], lse=lse[None], mean_abs=mean_abs[None], score_mag=score_mag[None], seen=seen[None],
                status=status)
