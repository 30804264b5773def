"""GPU tests of the signs of what spec_token_logprobs returns: no probability above 1,
no negative entropy, exact zeros where one token has all the probability."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import f32_to_dev, ints_to_dev, note
from paged_helpers import bf16_bits, bits_to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_peaked_rows(dtype):
    note(f"logprobs signs {dtype}")
    rng = np.random.default_rng(23)
    R, V = 512, 3000
    for T in (0.01, 0.3, 1.0, 1.7):
        x = rng.normal(size=(R, V))
        at = rng.integers(0, V, R)
        # one token ahead of all others by 10 to 200 T
        x[np.arange(R), at] = x.max(1) + T * rng.uniform(10, 200, R)
        x += rng.uniform(-50, 50, R)[:, None]
        t = bits_to_dev(bf16_bits(x)) if dtype == "bf16" else f32_to_dev(x)
        top = t.float().argmax(1)
        g = sv.spec_token_logprobs(t, ints_to_dev(top.cpu().numpy()), temperature=T, top_k=2)
        torch.cuda.synchronize()
        assert (g["logprob"] <= 0).all() and (g["top_logprobs"] <= 0).all(), (T, g["logprob"].max().item())
        assert (g["entropy"] >= 0).all(), (T, g["entropy"].min().item())
    # a lone token: exactly 0
    x = np.full((64, V), -np.inf)
    x[np.arange(64), rng.integers(0, V, 64)] = rng.normal(size=64) * 30
    t = bits_to_dev(bf16_bits(x)) if dtype == "bf16" else f32_to_dev(x)
    g = sv.spec_token_logprobs(t, ints_to_dev(t.float().argmax(1).cpu().numpy()), temperature=0.7, top_k=1)
    for n in ("logprob", "entropy"):
        assert (g[n] == 0).all(), (n, g[n].abs().max().item())
    assert (g["top_logprobs"] == 0).all()
