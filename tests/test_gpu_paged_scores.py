"""GPU tests of spec_attend_paged over the documented range of its scores.

Queries hold a power of two in value 0, one or nothing in value 1, and zeros
elsewhere; the keys' two values are chosen so that a score (q.k) is exact in fp32
whatever its size, and the weights follow from exact differences.  With u = 2^-24 and
c = scale log2(e) rounded to fp32, a difference of w (in scale q.k) is off by u |w|
for c and by 2 u |w| for the subtraction and the product (or one fma), the hardware
exponential by 4 u: each weight is within 4 u (1 + |w|) relative, and within 2^-8
more where it enters the second product as one bf16 term.  A weight with |w| > 104
counts for nothing (exp(-104) < 2^-150), so |w| is at most that, in the numerator and
in the sum; sums of `len` terms add (len + 64) u.  lse = w_max + log(sum): 4 u |lse|
for c, the product, the logarithm and the last rounding, and the sum's own error."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import ints_to_dev, note
from oracle import paged
from paged_helpers import U, Cache, bf16_bits, bits_to_dev, random_tree

pytestmark = pytest.mark.gpu


def _store(cache, i, values):
    """The keys' value i, exact in the cache's type."""
    if cache.kind == "bf16":
        cache.host[0][..., i] = bf16_bits(values)
    else:
        cache.host[0][..., i] = torch.from_numpy(values.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _run(rng, D, H, Hkv, N, kind, q0, k0, q1, k1, scale, base, counts=None, tree=False):
    """Scores +-q0 a + q1 b, a from k0 and b from k1."""
    B, page = len(base), 16
    P = -(-int(max(base) + N) // page)
    table = rng.permutation(B * P + 2)[:B * P].reshape(B, P)
    cache = Cache(rng, B * P + 2, Hkv, page, D, kind)
    shape = cache.host[0].shape[:3]
    a, b = rng.choice(k0, shape), rng.choice(k1, shape)
    _store(cache, 0, a)
    _store(cache, 1, b)
    if kind == "e4m3":
        cache.scales[0][:], cache.scales[1][:] = 1, 2.0 ** -7
        cache.values = [paged.e4m3_values(x) * s for x, s in zip(cache.host, (1, 2.0 ** -7))]
    else:
        cache.values[0] = paged.bf16_values(cache.host[0])
    assert np.array_equal(cache.values[0][..., 0], a) and np.array_equal(cache.values[0][..., 1], b)
    q = np.zeros((B, N, H, D))
    q[..., 0] = q0 * rng.choice([1, -1], (B, N, H))
    q[..., 1] = q1
    bits = bf16_bits(q)
    assert np.array_equal(paged.bf16_values(bits), q)
    parents = random_tree(rng, B, N) if tree else None
    kv = cache.upload()
    scale = float(np.float32(scale))
    g = sv.spec_attend_paged(bits_to_dev(bits), kv, ints_to_dev(table), ints_to_dev(base), scale=scale, lse=True,
                             counts=None if counts is None else ints_to_dev(counts),
                             parents=None if parents is None else ints_to_dev(parents))
    torch.cuda.synchronize()
    o = paged.attend(q, *cache.values, table, np.asarray(base), counts, parents, scale)
    assert (g["status"].cpu().numpy() == 0).all()
    seen, case = o["seen"], (q0, scale)
    out, lse = g["out"].double().cpu().numpy()[seen], g["lse"].double().cpu().numpy()[seen]
    assert np.isfinite(out).all() and np.isfinite(lse).all(), case
    assert (np.abs(o["lse"][seen]) < 1e29).all()
    sums = 4 * U * 105 + (max(base) + N + 64) * U
    tol = (2 * sums + 2.0 ** -8) * o["mean_abs"][seen]
    tol = tol + 2.0 ** -8 * (np.abs(o["out"][seen]) + tol) + 2.0 ** -126
    off = np.abs(out - o["out"][seen])
    assert (off <= tol).all(), (case, off.max(), tol.min())
    off = np.abs(lse - o["lse"][seen])
    assert (off <= 4 * U * np.abs(o["lse"][seen]) + sums).all(), (case, off.max())


# rows per KV head of one, two and three row tiles (slots divided) and of six and
# twelve (rows divided); head_dim 256; long enough for splits that are joined
SHAPES = [(128, 4, 2, 1), (64, 8, 2, 6), (128, 8, 2, 12), (128, 8, 2, 24), (64, 4, 1, 48), (256, 2, 1, 12)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,N", SHAPES)
def test_scores_from_small_to_the_largest(kind, D, H, Hkv, N):
    note(f"attend score sizes {kind} D={D} H={H} N={N}")
    rng = np.random.default_rng(D + N)
    steps, none = np.array([-8, -7.5, -4, -2, -1, -0.5, 0.5, 1, 2, 4, 6, 7, 7.5]), np.zeros(1)
    for power in (0, 10, 18, 22, 27, 30, 31, 32, 34, 40, 50, 64, 80, 92):
        _run(rng, D, H, Hkv, N, kind, 2.0 ** power, steps, 0, none, 1.0, [0, 40, 300], tree=N > 2)
    _run(rng, D, H, Hkv, N, kind, 2.0 ** 60, steps, 0, none, 3.7, [2500, 1100], counts=np.array([N, max(1, N - 2)]))
    _run(rng, D, H, Hkv, N, kind, 2.0 ** 100, steps, 0, none, 2.0 ** -60, [700, 90])
    _run(rng, D, H, Hkv, N, kind, 2.0 ** 4, steps, 0, none, 2.0 ** 60, [700, 90])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,N", SHAPES)
def test_large_scores_a_little_apart(kind, D, H, Hkv, N):
    # large scores whose weights are all in play, in tiles and splits that each have
    # their own largest; the last scale puts log2 of the weights on both sides of 2^20
    note(f"attend close large scores {kind} D={D} H={H} N={N}")
    rng = np.random.default_rng(D + N + 1)
    near, one = np.arange(0, 16) / 1.0, np.ones(1)
    for power in (4, 10, 13, 14, 16, 18, 19, 20, 21, 22):
        _run(rng, D, H, Hkv, N, kind, 2.0 ** power, one, 1, near, 0.4, [1300, 3, 530], tree=N > 2)
    for power, edge in ((20, 20), (20, 14), (20, 12), (22, 20)):
        _run(rng, D, H, Hkv, N, kind, 2.0 ** power, one, 1, near,
             2.0 ** edge * np.log(2) / (2.0 ** power + 7), [1300, 3, 530])
        _run(rng, D, H, Hkv, N, kind, 2.0 ** power, one, 1, near,
             2.0 ** edge * np.log(2) / (2.0 ** power - 7), [1300, 3, 530])
