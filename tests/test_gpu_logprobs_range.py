"""GPU tests of spec_token_logprobs over the range of its logits and temperatures:
rows masked with finite values, large common offsets, low temperatures.  Compared
with the 64-bit oracle; the tolerances are those of test_gpu_logprobs.py, whose
derivation assumes nothing about the size of a logit or of 1 / T."""

import numpy as np
import pytest

from gpu_helpers import note
from test_gpu_logprobs import _run

pytestmark = pytest.mark.gpu

MASKS = (-1e4, -1e5, -1e9, -1e10, -1e12, -1e20, -1e30, -1e35)


def _masked_rows(rng, V, mask):
    """Rows of ordinary logits under a mask: whole segments, a tail, all but a few
    tokens, all but one, everything."""
    x = rng.normal(size=(5, V)) * 4
    x[0, V // 3:V // 3 + 9000] = mask
    x[1, V - V // 4:] = mask
    x[2, rng.random(V) < 0.999] = mask
    x[3, np.arange(V) != V - 5] = mask
    x[4] = mask
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0.3, 0.6, 0.7, 0.8, 1.0, 1.3])
def test_finite_masks(dtype, T):
    note(f"logprobs finite masks {dtype} T={T}")
    rng = np.random.default_rng(int(T * 10))
    for V in (700, 20011):  # one segment and several
        x = np.concatenate([_masked_rows(rng, V, m) for m in MASKS])
        tokens = rng.integers(0, V, len(x))
        tokens[4::5] = V - 1
        _run(rng, len(x), V, dtype, T, 5, x=x, tokens=tokens)
    # rows that fill the card, where a wave takes a larger share of a row
    x = np.concatenate([_masked_rows(rng, 40009, m) for m in MASKS] * 7)
    _run(rng, len(x), 40009, dtype, T, 20, x=x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_low_temperatures(dtype):
    # the largest logit's distance to the next, over T, runs from much to nothing
    note(f"logprobs low temperatures {dtype}")
    rng = np.random.default_rng(17)
    for V in (50, 1500, 30011):
        for T in (0.02, 1e-3, 1e-4, 1e-5, 1e-6, 1e-7, 1e-10):
            x = rng.normal(size=(6, V)) * 4
            x[1] += 30
            x[2] = 1000 + x[2]
            x[3, rng.integers(0, V, 40)] = x[3].max()        # ties at the top
            x[4] = 17.3 + rng.integers(0, 4, V) * 2.0 ** -18  # a few steps apart
            x[5] *= -1e-3
            _run(rng, 6, V, dtype, T, 3, x=x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_offsets(dtype):
    # log probabilities do not change with an offset of the whole row
    note(f"logprobs large offsets {dtype}")
    rng = np.random.default_rng(19)
    for T in (0.7, 1.0):
        for off in (1e3, -1e4, 1.2e4, 3e4, -1e5, 1e6, -1e7):
            x = rng.integers(-64, 64, (3, 9001)) * 2.0 ** -3 + off
            _run(rng, 3, 9001, dtype, T, 5, x=x)
