"""GPU tests of spec_token_logprobs against the 64-bit oracle.

Tolerance: a term 2^d, d = (x - m) c, is off by 2^-22 (|d| + 1) relative (the
subtraction and the product round, the hardware exponential is good to one step),
so the sums of 2^d and 2^d d are off by at most 2^-22 times ``spread`` = sum
p (d^2 + |d| + 1) of the oracle, relative to the first sum; the pairwise sums over a
lane's 128 terms add 2^-20 spread; everything after is fp64, rounded once to fp32.
c itself is an fp32 number: 2^-24 of any difference of logits, so 2^-23 of the
result and of what separates it from the maximum."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, f32_to_dev, ints_to_dev, note
from oracle import paged
from paged_helpers import bf16_bits, bits_to_dev

pytestmark = pytest.mark.gpu


def _check(x, g, tokens, T, k):
    o = paged.token_logprobs(x, tokens, T, k)
    base = 2.0 ** -20 * o["spread"] + 2.0 ** -22

    def near(got, want, tol):
        got = got.cpu().numpy().astype(np.float64)
        same = (got == want) | (np.abs(got - want) <= tol) if want.size else np.ones(0, bool)
        assert same.all(), (np.argwhere(~same)[:4], got[~same][:4], want[~same][:4])

    with np.errstate(invalid="ignore"):
        if tokens is not None:
            near(g["logprob"], o["logprob"], base + 2.0 ** -22 * np.nan_to_num(np.abs(o["logprob"]), posinf=0))
        near(g["entropy"], o["entropy"], 2 * base + 2.0 ** -22 * o["entropy"])
        if k:
            assert np.array_equal(g["top_ids"].cpu().numpy(), o["top_ids"])
            near(g["top_logprobs"], o["top_logprobs"],
                 base[:, None] + 2.0 ** -22 * np.nan_to_num(np.abs(o["top_logprobs"]), posinf=0))
    if tokens is not None:
        assert np.array_equal(g["status"].cpu().numpy(), o["status"])


def _run(rng, R, V, dtype, T=1.0, k=5, x=None, tokens="random", offset=0):
    x = rng.normal(size=(R, V)) * 4 if x is None else x
    if dtype == "bf16":
        bits = bf16_bits(x)
        x = paged.bf16_values(bits)
        flat = np.concatenate([np.full(offset, 0x7f80, np.uint16), bits.reshape(-1)])
        t = bits_to_dev(flat)
    else:
        x32 = x.astype(np.float32)
        x = x32.astype(np.float64)
        t = f32_to_dev(np.concatenate([np.full(offset, np.inf), x32.reshape(-1)]))
    t = t[offset:].view(R, V)
    if isinstance(tokens, str):
        tokens = rng.integers(0, V, R)
    g = sv.spec_token_logprobs(t, None if tokens is None else ints_to_dev(tokens), temperature=T, top_k=k)
    torch.cuda.synchronize()
    _check(x, g, tokens, float(np.float32(T)), k)
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 33, 32), (5, 1000, 5), (4, 1001, 20), (1, 8191, 32),
                                   (1, 8192, 1), (2, 8193, 13), (3, 151937, 20), (2, 151936, 32), (700, 5003, 3)])
def test_sizes(dtype, R, V, k):
    note(f"logprobs {dtype} R={R} V={V} k={k}")
    _run(np.random.default_rng(V + k), R, V, dtype, 0.7, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(2, 400001), (32, 262145)])
def test_rows_of_more_segments_than_the_join_holds(dtype, R, V):
    note(f"logprobs {dtype} R={R} V={V}")
    _run(np.random.default_rng(V), R, V, dtype, 1.0, 20)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_every_place_on_the_16_byte_grid(dtype):
    # unaligned bases and odd row lengths; what lies around the rows is +inf
    note(f"logprobs alignment {dtype}")
    rng = np.random.default_rng(3)
    for off in range(9):
        _run(rng, 5, 515, dtype, 1.3, 4, offset=off)
        _run(rng, 1, 1, dtype, 1.0, 1, offset=off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_masks_and_orders(dtype):
    note(f"logprobs ties {dtype}")
    rng = np.random.default_rng(5)
    V = 20011
    low = -3.3e38
    rows = [np.zeros(V),                                    # all equal
            np.where(rng.random(V) < 0.999, -np.inf, rng.normal(size=V)),
            np.full(V, -np.inf),                            # nothing allowed
            np.full(V, low),                                # masked with the type's lowest value
            np.where(rng.random(V) < 0.99, low, rng.normal(size=V)),
            np.arange(V) * 0.5,                             # rising: every segment's best are its last
            -np.arange(V) * 0.5,
            rng.integers(-2, 3, V).astype(float),           # many ties
            np.where(np.arange(V) % 512 < 8, 5.0, 0.0) + rng.normal(size=V) * 0.01,  # one lane holds all the best
            np.where(np.arange(V) == V - 1, 0.0, -np.inf)]
    for k in (0, 1, 20, 32):
        _run(rng, len(rows), V, dtype, 1.0, k, x=np.array(rows))
    # the same rows where each wave takes a larger share of a row
    many = np.array(rows * 60)
    _run(rng, len(many), V, dtype, 1.0, 20, x=many)


def test_tokens_out_of_range_padding_and_absent():
    note("logprobs tokens")
    rng = np.random.default_rng(7)
    tokens = np.array([0, -1, 99, 100, -2, 2**31 - 1, -1, 50])
    g = _run(rng, 8, 100, "f32", 1.0, 3, tokens=tokens)
    assert g["status"].tolist() == [0, 0, 0, 1, 1, 1, 0, 0]
    g = _run(rng, 4, 300, "bf16", 1.0, 3, tokens=None)
    assert "logprob" not in g
    x = f32_to_dev(rng.normal(size=(4, 50)))
    g = sv.spec_token_logprobs(x, ints_to_dev([1, 2, 3, 4]), entropy=False, status=False)
    assert set(g) == {"logprob"}
    g = sv.spec_token_logprobs(x[:0], ints_to_dev([]), top_k=2)
    assert g["top_ids"].shape == (0, 2)
    for bad in (lambda: sv.spec_token_logprobs(x, ints_to_dev([1, 2])), lambda: sv.spec_token_logprobs(x.t()),
                lambda: sv.spec_token_logprobs(x, torch.zeros(4, device=dev()))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sv.spec_token_logprobs(x.half())
    for kw in (dict(top_k=33), dict(top_k=-1), dict(temperature=0.0)):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_token_logprobs(x, **kw)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_token_logprobs(x[:, :3].contiguous(), top_k=4)


def test_temperatures_and_agreement_with_the_sampler():
    # the sampler's own log-sum-exp of the same rows
    note("logprobs temperature")
    rng = np.random.default_rng(9)
    for T in (0.05, 0.7, 3.0, 100.0):
        g = _run(rng, 6, 3001, "f32", T, 8)
    x = rng.normal(size=(6, 1, 3001)).astype(np.float32)
    lse = sv.spec_verify_sample(f32_to_dev(x), None, None, None, f32_to_dev(np.full((6, 1), 0.5)), 0.7)["lse_target"]
    g = sv.spec_token_logprobs(f32_to_dev(x[:, 0]), ints_to_dev([5] * 6), temperature=0.7)
    want = x[:, 0, 5].astype(np.float64) / float(np.float32(0.7)) - lse[:, 0].double().cpu().numpy()
    assert np.abs(g["logprob"].cpu().numpy() - want).max() < 1e-5


def test_same_call_twice_gives_the_same_bits():
    note("logprobs repeated")
    rng = np.random.default_rng(11)
    x, t = bits_to_dev(bf16_bits(rng.normal(size=(64, 50021)) * 3)), ints_to_dev(rng.integers(0, 50021, 64))
    a = [sv.spec_token_logprobs(x, t, top_k=32) for _ in range(3)]
    torch.cuda.synchronize()
    for b in a[1:]:
        for k in a[0]:
            assert torch.equal(a[0][k], b[k])
