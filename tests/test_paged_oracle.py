"""The paged-cache and log-probability oracle (oracle/paged.py) against facts
fixed independently of it (CPU only)."""

import numpy as np
import pytest
import torch

from oracle import kv_commit, paged


def test_element_values_match_torch():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.e4m3_values(b), want, equal_nan=True)
    h = np.arange(0, 65536, 7, dtype=np.uint16)
    want = torch.from_numpy(h.view(np.int16)).view(torch.bfloat16).double().numpy()
    assert np.array_equal(paged.bf16_values(h), want, equal_nan=True)


def test_attention_of_a_chain_is_a_causal_softmax():
    # identity page tables: the cache read back is a dense [len, D] array
    rng = np.random.default_rng(0)
    B, N, H, Hkv, D, page, P = 2, 3, 4, 2, 8, 4, 3
    k, v = rng.normal(size=(2, B * P, Hkv, page, D))
    q = rng.normal(size=(B, N, H, D))
    table = np.arange(B * P).reshape(B, P)
    base = np.array([0, 7])
    o = paged.attend(q, k, v, table, base, None, None, 0.3)
    dense = lambda x, b: torch.from_numpy(x[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, P * page, D))
    for b in range(B):
        L = base[b] + N
        kk = dense(k, b)[:, :L].repeat_interleave(H // Hkv, 0)
        vv = dense(v, b)[:, :L].repeat_interleave(H // Hkv, 0)
        mask = torch.ones(N, L, dtype=torch.bool).tril(L - N)
        w = (torch.from_numpy(q[b]).transpose(0, 1) @ kk.transpose(1, 2) * 0.3).masked_fill(~mask, -torch.inf)
        want = (w.softmax(-1) @ vv).transpose(0, 1)
        np.testing.assert_allclose(o["out"][b], want.numpy(), rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(o["lse"][b], w.logsumexp(-1).T.numpy(), rtol=1e-12)
    assert o["status"].tolist() == [0, 0]


def test_tree_rows_see_their_ancestors_only():
    #   0 - 1 - 3 , 0 - 2 - 4 : a value of token 2 or 4 never reaches row 3
    par = np.array([[-1, 0, 0, 1, 2]])
    assert paged.ancestors(par[0], 3) == [0, 1, 3] and paged.ancestors(par[0], 4) == [0, 2, 4]
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(2, 1, 1, 8, 4))
    q = rng.normal(size=(1, 5, 1, 4))
    a = paged.attend(q, k, v, np.zeros((1, 1), int), np.zeros(1, int), None, par, 1.0)
    v2 = v.copy()
    v2[0, 0, 2] = np.inf
    v2[0, 0, 4] = np.nan
    c = paged.attend(q, k, v2, np.zeros((1, 1), int), np.zeros(1, int), None, par, 1.0)
    assert np.array_equal(a["out"][0, [0, 1, 3]], c["out"][0, [0, 1, 3]])
    assert not np.isfinite(c["out"][0, 2]).any() and not np.isfinite(c["out"][0, 4]).any()


def test_attention_status():
    z = np.zeros
    k = z((2, 1, 4, 4))
    q = z((1, 2, 1, 4))
    f = lambda table, base, par=None, counts=None: int(
        paged.attend(q, k, k, np.array([table]), np.array([base]), counts, par, 1.0)["status"][0])
    assert f([0, 1], 0) == 0 and f([0, 1], 6) == 0
    assert f([0, 1], 7) == 1 and f([0, 1], -1) == 1 and f([0, 2], 3) == 1 and f([0, 2], 1) == 0
    assert f([0, 1], 0, np.array([[-1, 1]])) == 2 and f([0, 1], 0, np.array([[0, 0]])) == 2
    assert f([0, 1], 0, np.array([[-1, 5]]), [1]) == 0  # rows behind the count are not looked at


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_differences_of_positions(interleaved):
    rng = np.random.default_rng(2)
    D, rot = 32, 16
    table = lambda p: np.concatenate([f(p * 100.0 ** (-np.arange(0, rot, 2) / rot)) for f in (np.cos, np.sin)])
    x, y = rng.normal(size=(2, D))
    turn = lambda u, p: paged.norm_and_turn(u, None, 0, table(p), rot, interleaved)[0]
    np.testing.assert_allclose(np.linalg.norm(turn(x, 9)), np.linalg.norm(x))
    np.testing.assert_allclose(turn(x, 9) @ turn(y, 4), turn(x, 25) @ turn(y, 20))
    assert np.array_equal(turn(x, 9)[rot:], x[rot:])
    # one pair by hand: a quarter turn takes (a, b) to (-b, a)
    ang = np.concatenate([np.ones(8), np.zeros(8)])
    ang[3], ang[8 + 3] = 0.0, 1.0
    t = paged.norm_and_turn(x, None, 0, ang, rot, interleaved)[0]
    i, j = (6, 7) if interleaved else (3, 11)
    assert t[i] == -x[j] and t[j] == x[i]


def test_norm_is_the_root_mean_square():
    x = np.array([3.0, -4.0, 0.0, 0.0])
    y, _ = paged.norm_and_turn(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0, None, 0, False)
    np.testing.assert_allclose(y, [3 / 2.5, -8 / 2.5, 0, 0])


def test_commit_agrees_with_the_contiguous_form():
    # one page table over shuffled pages; gathered back, the cache is contiguous
    rng = np.random.default_rng(3)
    G, B, Hkv, page, P, rb, N = 2, 5, 3, 16, 4, 16, 9
    table = rng.permutation(B * P).reshape(B, P)
    pages = rng.integers(0, 256, (G, B * P, Hkv, page, rb), dtype=np.uint8)
    scales = rng.normal(size=(G, B * P, Hkv, page)).astype(np.float32)
    d = np.array([0, 1, 4, 8, 3])
    path = np.full((B, N), -1)
    for b in range(B):
        path[b, :d[b]] = np.sort(rng.choice(np.arange(1, N), d[b], replace=False))
    tb = rng.integers(0, P * page - N, B)
    out, souts, st = paged.commit_paged(pages, scales, table, tb, tb + 1, d, path)
    dense = lambda x: x[:, table].transpose(0, 1, 2, 4, 3, 5).reshape(G, B, P * page, Hkv * rb)
    want, wst = kv_commit.commit_tree_kv(dense(pages), None, tb, tb + 1, d, path, N)
    assert np.array_equal(dense(out), want) and np.array_equal(st, wst)
    s4 = scales[..., None].view(np.uint8)
    sd = lambda x: x[:, table].transpose(0, 1, 2, 4, 3, 5).reshape(G, B, P * page, Hkv * 4)
    want, _ = kv_commit.commit_tree_kv(sd(s4), None, tb, tb + 1, d, path, N)
    assert np.array_equal(sd(souts[..., None].view(np.uint8)), want)


def test_log_probabilities():
    x = np.log(np.array([[0.1, 0.2, 0.3, 0.4], [0.25, 0.25, 0.25, 0.25]]))
    o = paged.token_logprobs(x, [2, 9], 1.0, 3)
    np.testing.assert_allclose(np.exp(o["logprob"]), [0.3, 0.0])
    np.testing.assert_allclose(o["entropy"], [-(np.exp(x[0]) * x[0]).sum(), np.log(4)])
    assert o["top_ids"].tolist() == [[3, 2, 1], [0, 1, 2]] and o["status"].tolist() == [0, 1]
    np.testing.assert_allclose(np.exp(o["top_logprobs"]), [[0.4, 0.3, 0.2], [0.25] * 3])
    # a temperature of 2 takes the square roots of the probabilities
    p = np.sqrt(np.exp(x[0]))
    np.testing.assert_allclose(paged.token_logprobs(x[:1], [0], 2.0, 0)["logprob"], [np.log(p[0] / p.sum())])
    # masked ids, a masked row, padding
    x = np.array([[0.0, -np.inf, 0.0], [-np.inf] * 3, [1.0, 2.0, 3.0]])
    o = paged.token_logprobs(x, [1, 0, -1], 1.0, 3)
    assert o["logprob"].tolist() == [-np.inf, -np.inf, 0] and o["top_ids"].tolist() == [[0, 2, 1], [0, 1, 2], [-1] * 3]
    np.testing.assert_allclose(o["entropy"], [np.log(2), 0, 0])
    assert (o["top_logprobs"][1:] == -np.inf).all() and o["top_logprobs"][0, 2] == -np.inf
