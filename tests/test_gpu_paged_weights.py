"""GPU tests of the precision spec_attend_paged states for its weights: two bf16
terms (2^-16 relative) where a wave holds one or two row tiles of 16, one (2^-8)
where it holds three.

A third of the slots have score 0 and values v, the others a score whose weight, half
and almost 2^-9, lies between two bf16 numbers, and values -v: the sums nearly
cancel, and the rounding of the second weight is what remains.  Tolerance: the
weight's rounding, 4 u (1 + |w|) twice for the exponent, (len + 64) u twice for the
sums (u = 2^-24), all of the weighted mean of |v|; then one bf16 rounding of the
small result."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import ints_to_dev, note
from oracle import paged
from paged_helpers import U, Cache, bf16_bits, bits_to_dev

pytestmark = pytest.mark.gpu

WEIGHT = 0.5 + 0.9 * 2.0 ** -9


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,N,base,terms", [
    (128, 4, 1, 1, 700, 2), (128, 4, 1, 1, 9000, 2),                    # one row tile, with and without a join
    (64, 8, 2, 8, 1000, 2), (128, 4, 2, 16, 2500, 2), (128, 2, 2, 31, 650, 2),  # two
    (128, 4, 2, 24, 700, 1), (64, 1, 1, 48, 1500, 1),                   # three
    (128, 4, 1, 16, 700, 2), (64, 8, 1, 16, 700, 2), (128, 4, 1, 32, 4000, 2),  # rows divided: one and two
    (128, 4, 1, 33, 700, 1), (64, 4, 1, 48, 700, 1),                    # three of nine and of twelve
    (256, 4, 1, 10, 800, 2)])
def test_weights_of_one_and_two_terms(kind, D, H, Hkv, N, base, terms):
    note(f"attend weights {kind} D={D} H={H} N={N} base={base}")
    rng = np.random.default_rng(D + N)
    P = -(-(base + N) // 16)
    table = rng.permutation(P)[None]
    cache = Cache(rng, P, Hkv, 16, D, kind)
    v = rng.choice([-1, 1], D) * 2.0 ** rng.integers(-2, 3, D)
    slot = np.empty((P, 16), np.int64)
    slot[table[0]] = np.arange(P * 16).reshape(P, 16)
    first = (slot % 3 == 0)[:, None, :, None]  # [page, 1, row, 1]
    k = np.zeros((P, Hkv, 16, D))
    k[..., :1] = np.where(first, 0, -1)
    vals = np.where(first, v, -v) * np.ones((P, Hkv, 16, D))
    for i, x in enumerate((k, vals)):
        if kind == "bf16":
            cache.host[i][:] = bf16_bits(x)
        else:
            cache.host[i][:] = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            cache.scales[i][:] = 1
        cache.values[i] = x
    q = np.zeros((1, N, H, D))
    q[..., 0] = 1
    scale = float(np.float32(-np.log(WEIGHT)))
    g = sv.spec_attend_paged(bits_to_dev(bf16_bits(q)), cache.upload(), ints_to_dev(table), ints_to_dev([base]), scale=scale)
    torch.cuda.synchronize()
    o = paged.attend(q, *cache.values, table, np.array([base]), None, None, scale)
    assert (g["status"].cpu().numpy() == 0).all()

    def tolerance(terms):
        tol = (2.0 ** (-8 * terms) + 2 * (4 * U * 2 + (base + N + 64) * U)) * o["mean_abs"]
        return tol + 2.0 ** -8 * (np.abs(o["out"]) + tol)

    off = np.abs(g["out"].double().cpu().numpy() - o["out"])
    assert (off <= tolerance(terms)).all(), (off.max(), tolerance(terms).min())
    # one term would not pass for two
    w = np.exp(-scale)
    rounded = float(paged.bf16_values(bf16_bits(np.array([w])))[0])
    n = base + 1 + np.arange(N)[None, :, None, None]
    a = (n + 2) // 3
    one = (a - (n - a) * rounded) / (a + (n - a) * w) * v
    assert (np.abs(one - o["out"]) > tolerance(2)).all()
