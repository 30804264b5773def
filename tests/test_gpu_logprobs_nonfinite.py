"""GPU tests of spec_token_logprobs on rows that hold NaN or +inf: their values are
NaN, the alternatives are those among the row's logits that are not NaN, and no
other row is touched."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, f32_to_dev, ints_to_dev, note
from oracle import paged
from paged_helpers import bf16_bits, bits_to_dev

pytestmark = pytest.mark.gpu


def _rows(rng, V):
    """(rows, whether each is of finite logits and -inf)."""
    nan, inf = np.nan, np.inf

    def row(fill=None):
        return rng.normal(size=V) * 3 if fill is None else np.full(V, fill)

    rows = [row(nan), row(), row(), row(), row(), row(-inf), row(-inf), row(1.0), row(), row(inf), row(-inf), row(),
            row(-1e30)]
    rows[1][:] = np.where(np.arange(V) < V - 3, nan, rows[1])   # a few numbers behind NaN segments
    rows[2][V // 2:V // 2 + 9000] = nan                         # a segment and more
    rows[3][V // 2] = nan                                       # one
    rows[4][V // 3] = inf
    rows[5][V - 1] = nan                                        # nothing but -inf beside it
    rows[6][V // 2] = inf
    rows[7][::2] = nan                                          # many ties at the top
    rows[8][::3] = -nan
    rows[8][1::3] = -inf
    rows[12][V // 4] = nan                                      # a mask value beside it
    return np.array(rows), np.array([not (np.isnan(x).any() or (x == inf).any()) for x in rows])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,copies", [(40, 1), (9000, 1), (30011, 1), (30011, 40)])
def test_nan_and_inf(dtype, V, copies):
    note(f"logprobs NaN and inf {dtype} V={V} x{copies}")
    rng = np.random.default_rng(V)
    x, fine = _rows(rng, V)
    x, fine = np.tile(x, (copies, 1)), np.tile(fine, copies)
    with np.errstate(invalid="ignore"):
        if dtype == "bf16":
            bits = bf16_bits(x)
            bits[np.isnan(x) & (np.arange(V) % 2 == 0)] = 0xffff  # NaN of either sign
            x, t = paged.bf16_values(bits), bits_to_dev(bits)
        else:
            x32 = x.astype(np.float32)
            x32.view(np.uint32)[np.isnan(x) & (np.arange(V) % 2 == 0)] = 0xffffffff
            x, t = x32.astype(np.float64), f32_to_dev(x32)
    R = len(x)
    tokens = rng.integers(0, V, R)
    outside = np.arange(R) % 13 == 3
    tokens[outside] = V + 5
    unread = np.arange(R) % 13 == 9
    tokens[unread] = -1
    k = min(V, 20)
    g = sv.spec_token_logprobs(t, ints_to_dev(tokens), top_k=k)
    torch.cuda.synchronize()
    g = {n: v.cpu().numpy() for n, v in g.items()}
    assert np.array_equal(g["status"], outside)
    want = np.full((R, k), -1)
    for r in range(R):
        live = np.flatnonzero(~np.isnan(x[r]))
        order = live[np.lexsort((live, -x[r][live]))][:k]
        if not unread[r]:
            want[r, :len(order)] = order
    assert np.array_equal(g["top_ids"], want)
    bad = ~fine & ~unread
    assert np.isnan(g["entropy"][bad]).all() and np.isnan(g["logprob"][bad & ~outside]).all()
    assert (g["logprob"][outside] == -np.inf).all()
    there = want >= 0
    assert np.isnan(g["top_logprobs"][bad[:, None] & there]).all()
    assert (g["top_logprobs"][~there] == -np.inf).all()
    assert (g["entropy"][unread] == 0).all() and (g["logprob"][unread] == 0).all()
    assert not any(np.isnan(g[n][fine]).any() for n in ("logprob", "entropy", "top_logprobs"))
    # the rows beside them are what they are alone
    alone = sv.spec_token_logprobs(t[torch.from_numpy(np.flatnonzero(fine)).to(t.device)].contiguous(),
                                   ints_to_dev(tokens[fine]), top_k=k)
    for n in ("logprob", "entropy"):
        assert np.allclose(alone[n].cpu().numpy(), g[n][fine], rtol=1e-5, atol=1e-5)
    # with neither tokens nor alternatives
    only = sv.spec_token_logprobs(t)
    assert np.array_equal(np.isnan(only["entropy"].cpu().numpy()), ~fine)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,R", [(40, 6), (9000, 6), (30011, 300)])
def test_signalling_nan(dtype, V, R):
    # patterns no arithmetic produces: NaN all the same, and ids of numbers
    note(f"logprobs signalling NaN {dtype} V={V} R={R}")
    rng = np.random.default_rng(V)
    x = bf16_bits(rng.normal(size=(R, V))) if dtype == "bf16" else rng.normal(size=(R, V)).astype(np.float32).view(np.uint32)
    a, b, c = (0x7f81, 0xff81, 0x7fbf) if dtype == "bf16" else (0x7f800001, 0xff800001, 0x7fbfffff)
    x[1, V // 2], x[2], x[3, ::2], x[4, V // 2:] = a, b, c, a
    if dtype == "bf16":
        t, v = bits_to_dev(x), paged.bf16_values(x)
    else:
        t = torch.from_numpy(x.view(np.int32)).to(dev()).view(torch.float32)
        with np.errstate(invalid="ignore"):
            v = x.view(np.float32).astype(np.float64)
    g = sv.spec_token_logprobs(t, ints_to_dev(np.zeros(R)), top_k=5)
    torch.cuda.synchronize()
    bad = np.isnan(v).any(1)
    assert bad[1:5].all() and bad.sum() == 4
    for n in ("logprob", "entropy"):
        assert np.array_equal(np.isnan(g[n].cpu().numpy()), bad)
    ids = g["top_ids"].cpu().numpy()
    for r in range(R):
        got = ids[r][ids[r] >= 0]
        assert not np.isnan(v[r, got]).any() and len(set(got.tolist())) == len(got)
        if not bad[r]:
            assert np.array_equal(ids[r], np.lexsort((np.arange(V), -v[r]))[:5])
