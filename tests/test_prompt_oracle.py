"""Pins of the prompt operators' oracle: against closed forms, plain numpy sums and the
window oracle, which was written apart from it."""

import numpy as np
import pytest

from oracle import paged, prompt


def test_norm_of_a_constant_row_is_its_sign():
    x = np.full((2, 16), -3.0)
    h, y = prompt.rms_norm(x, None, None, 0.0)
    assert (h == -3).all() and np.allclose(y, -1, atol=1e-15)
    h, y = prompt.rms_norm(x, np.full((2, 16), 5.0), np.arange(16.0), 0.0)
    assert (h == 2).all() and np.allclose(y, np.arange(16.0), atol=1e-15)


def test_block_scales_of_a_ragged_row():
    y = np.zeros((1, 130))
    y[0, 5], y[0, 129] = -448, 44.8
    assert np.allclose(prompt.block_scales(y)[:, 0], [1, 0.1])


def test_linear_against_the_scaled_operands():
    rng = np.random.default_rng(0)
    M, N, K = 3, 140, 272
    x, w = rng.normal(size=(M, K)), rng.normal(size=(N, K))
    xs, ws = rng.random((3, M)), rng.random((2, 3))
    big_x = x * np.repeat(xs.T, 128, 1)[:, :K]
    big_w = w * np.repeat(np.repeat(ws, 128, 0), 128, 1)[:N, :K]
    out, mag, top = prompt.linear(x, xs, w, ws)
    assert np.allclose(out, np.einsum("mk,nk->mn", big_x, big_w), rtol=1e-12, atol=1e-12)
    assert np.allclose(mag, np.einsum("mk,nk->mn", abs(big_x), abs(big_w)), rtol=1e-12)
    assert (top * 128 >= mag).all()
    least = sum(np.abs(big_x[:, None, k:k + 128] * big_w[None, :, k:k + 128]).max(2) for k in (0, 128, 256))
    assert (top >= least * (1 - 1e-12)).all()


@pytest.mark.parametrize("starts", [[0, 5, 5, 12], [2, 3, 9, 9]])
def test_packed_attention_is_that_of_windows(starts):
    rng = np.random.default_rng(1)
    H, Hkv, D, page, T = 4, 2, 8, 4, 13
    base = [3, 0, 6]
    k, v = rng.normal(size=(2, 20, Hkv, page, D))
    table = rng.permutation(20)[:15].reshape(3, 5)
    q = rng.normal(size=(T, H, D))
    o = prompt.attend_packed(q, k, v, table, starts, base, 0.3)
    for b in range(3):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        w = paged.attend(q[None, starts[b]:starts[b] + n], k, v, table[b:b + 1], [base[b]], None, None, 0.3)
        at = slice(starts[b], starts[b] + n)
        for name in ("out", "lse", "mean_abs", "score_mag"):
            assert np.allclose(o[name][0, at], w[name][0], rtol=1e-13, atol=1e-13), name
    assert (o["status"] == 0).all()
    assert (o["seen"][0] == (np.arange(T) >= starts[0]) & (np.arange(T) < starts[-1])).all()


def test_packed_attention_ends_at_the_first_missing_slot():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(2, 6, 1, 4, 8))
    q = rng.normal(size=(16, 1, 8))
    table = np.array([[0, 1, 6, 3], [2, 3, 4, 5]])
    o = prompt.attend_packed(q, k, v, table, [0, 12, 16], [0, -1], 0.3)
    assert o["status"].tolist() == [1, 1]
    assert np.isfinite(o["lse"][0, :8]).all() and (o["lse"][0, 8:] == -np.inf).all() and (o["out"][0, 8:] == 0).all()
    o = prompt.attend_packed(q, k, v, table, [0, 12, 4], [0, 0], 0.3)
    assert o["status"].tolist() == [1, 2]


def test_rotation_by_axes_is_the_rotation_of_each_part():
    rng = np.random.default_rng(3)
    T, D, rot = 4, 16, 16
    x = rng.normal(size=(T, 2, D))
    rope = rng.normal(size=(9, rot))
    pos = rng.integers(0, 9, (3, T))
    axis = np.array([0, 1, 2, 2, 1, 0, 0, 1])
    y, _ = prompt.append_rows(x, None, 0, rope, rot, False, pos, axis, [0, T])
    for a in range(3):
        z, _ = prompt.append_rows(x, None, 0, rope, rot, False, pos[a:a + 1], None, [0, T])
        mine = np.flatnonzero(axis == a)
        both = np.concatenate([mine, mine + 8])
        assert np.allclose(y[..., both], z[..., both], atol=1e-15)
