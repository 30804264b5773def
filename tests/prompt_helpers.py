"""Shared by the GPU tests of the prompt operators: seeded e4m3 operands, packed
sequences, and the comparisons with the 64-bit oracle.

Tolerances (u = 2^-24, fp32's half step; 2^-8, bf16's; e4m3: 2^-4 relative, or half of
the subnormal step 2^-9 times the scale):

* norm: the sum of D squares is off by at most D u relative, half of which reaches the
  inverse root; the sum h, the root, the division and two products by a few u each:
  (D / 2 + 16) u, then one rounding to the element type.
* linear, fp32 out: products of widened e4m3 values are exact; a block's 128 and the
  blocks' sums are added in fp32, two scale products and an fma round:
  (128 + blocks + 8) u of the terms' magnitudes.  bf16 out: the e4m3 matrix instruction
  cuts each of a block's 128 products at 2^-16 of the largest at worst: 2^-9 of the
  largest product, summed over the blocks, and the result's rounding, 2^-8.
* append and attend: as in ``paged_helpers``.
"""

from __future__ import annotations

import numpy as np
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, ints_to_dev
from oracle import paged, prompt
from paged_helpers import U, bf16_bits, bits_to_dev


def e4m3_bits(rng, shape, spread=1.0):
    """Random e4m3 bytes without NaN: Gaussian values of all magnitudes."""
    x = torch.from_numpy(rng.normal(size=shape) * spread * 100).clamp(-448, 448)
    return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def check_norm(x, residual, weight, eps, g, e4m3):
    """g: the call's outputs; x, residual, weight float64 on the host."""
    T, D = x.shape
    h, y = prompt.rms_norm(x, residual, weight, eps)
    off = (D / 2 + 16) * U
    if residual is not None:
        got = g["residual"].float().cpu().numpy().astype(np.float64)
        assert (np.abs(got - h) <= (2.0 ** -8 + 2 * U) * np.abs(h) + 2.0 ** -126).all()
    else:
        assert "residual" not in g
    got = g["out"].float().cpu().numpy().astype(np.float64)
    if not e4m3:
        assert (np.abs(got - y) <= (2.0 ** -8 + 2 * off) * np.abs(y) + 2.0 ** -126).all()
        return
    want = prompt.block_scales(y)
    scales = g["scales"].cpu().numpy().astype(np.float64)
    assert scales.shape == want.shape
    assert (np.abs(scales - want) <= 2 * off * want + 2.0 ** -126).all()
    s = np.repeat(scales.T, prompt.BLOCK, 1)[:, :D]
    assert (np.abs(got * s - y) <= (2.0 ** -4 + 4 * off) * np.abs(y) + 2.0 ** -10 * s * (1 + off) + 2.0 ** -126).all()


class LinearCase:
    def __init__(self, rng, M, N, K, pad=0, exact=False):
        kb, nb = -(-K // 128), -(-N // 128)
        self.shape = (M, N, K)
        if exact:  # small whole numbers and powers of two: every sum is exact in any order
            self.x = torch.from_numpy(rng.integers(-4, 5, (M, K)).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            self.w = torch.from_numpy(rng.integers(-4, 5, (N, K)).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            self.xs = np.exp2(rng.integers(-1, 2, (kb, M))).astype(np.float32)
            self.ws = np.exp2(rng.integers(-1, 2, (nb, kb))).astype(np.float32)
        else:
            self.x, self.w = e4m3_bits(rng, (M, K)), e4m3_bits(rng, (N, K))
            self.xs = np.exp(rng.normal(size=(kb, M))).astype(np.float32)
            self.ws = np.exp(rng.normal(size=(nb, kb))).astype(np.float32)
        self.pad = pad

    def upload(self):
        M, N, K = self.shape
        x = torch.zeros(M, K + self.pad, dtype=torch.uint8, device=dev())
        if self.pad:
            x[:, K:] = 0x7f  # NaN beside the rows
        x[:, :K] = torch.from_numpy(self.x).to(dev())
        xs = torch.full((self.xs.shape[0], M + self.pad), float("nan"), device=dev())
        xs[:, :M] = torch.from_numpy(self.xs).to(dev())
        return (x.view(torch.float8_e4m3fn)[:, :K], xs[:, :M], bits_to_dev(self.w), torch.from_numpy(self.ws).to(dev()))

    def check(self, out):
        M, N, K = self.shape
        x, w = paged.e4m3_values(self.x), paged.e4m3_values(self.w)
        want, mag, top = prompt.linear(x, self.xs.astype(np.float64), w, self.ws.astype(np.float64))
        got = out.float().cpu().numpy().astype(np.float64)
        if out.dtype == torch.float32:
            tol = (128 + self.xs.shape[0] + 8) * U * mag
        else:
            tol = 2.0 ** -9 * top + (128 + self.xs.shape[0] + 8) * U * mag
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        bad = ~(np.abs(got - want) <= tol + 2.0 ** -126)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


def run_packed(rng, cache, table, starts, base, T, H, scale=None, q=None, workspace=None, pad=0):
    """The call and the oracle on random queries; returns (call's outputs, oracle's) in
    the form that paged_helpers.check_attend compares."""
    D = cache.host[0].shape[-1]
    bits = bf16_bits(rng.normal(size=(T, H, D)) * 1.5) if q is None else q
    wide = torch.zeros(T, H * D + pad, dtype=torch.bfloat16, device=dev())
    wide[:, :H * D] = bits_to_dev(bits).reshape(T, H * D)
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full((T, H), 7.0, device=dev())
    g = sv.spec_attend_packed(wide[:, :H * D].unflatten(-1, (H, D)), cache.upload(), ints_to_dev(table), ints_to_dev(starts),
                              None if base is None else ints_to_dev(base), scale=scale, out=out, lse=lse,
                              workspace=workspace)
    torch.cuda.synchronize()
    o = prompt.attend_packed(paged.bf16_values(bits), *cache.values, table, starts, base,
                             D ** -0.5 if scale is None else scale)
    behind = ~o["seen"][0]
    assert (out.float().cpu().numpy()[behind] == 7).all() and (lse.cpu().numpy()[behind] == 7).all()
    return dict(out=g["out"][None], lse=g["lse"][None], status=g["status"]), o
