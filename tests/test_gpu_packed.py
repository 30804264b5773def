"""GPU tests of the packed-sequence operators (spec_append_kv_packed,
spec_attend_packed) against the 64-bit oracle and the window operators."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, ints_to_dev, note
from oracle import paged, prompt
from paged_helpers import U, Cache, bf16_bits, bits_to_dev, check_attend, to_bits
from prompt_helpers import run_packed

pytestmark = pytest.mark.gpu


def _table(rng, B, P, spare=3):
    return rng.permutation(B * P + spare)[:B * P].reshape(B, P), B * P + spare


# ---- attention -------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,page", [(64, 4, 4, 16), (128, 8, 2, 16), (256, 3, 1, 32), (128, 7, 1, 64),
                                          (64, 10, 2, 128), (128, 5, 5, 256)])
def test_packed_lengths(kind, D, H, Hkv, page):
    # empty, single, and lengths around a tile of slots and of rows; cached tokens before some
    note(f"packed {kind} D={D} H={H} Hkv={Hkv} page={page}")
    rng = np.random.default_rng(D + H + page)
    n = np.array([0, 1, 63, 64, 65, 0, 2, 31, 130, 17, 200, 33])
    base = np.array([0, 0, 0, 5, 64, 100, 127, 1, 0, 300, 61, 63])
    starts = np.concatenate([[3], 3 + np.cumsum(n)])
    T, B = int(starts[-1]) + 5, len(n)
    P = -(-int((n + base).max()) // page)
    table, pages = _table(rng, B, P)
    cache = Cache(rng, pages, Hkv, page, D, kind)
    g, o = run_packed(rng, cache, table, starts, base, T, H, pad=8 * (H % 3))
    assert (o["status"] == 0).all()
    check_attend(g, o, 400)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,H,Hkv,n,base", [(128, 4, 1, 700, 0), (64, 2, 2, 1100, 37), (256, 2, 1, 300, 900)])
def test_one_long_prompt(kind, D, H, Hkv, n, base):
    note(f"packed long {kind} D={D} n={n} base={base}")
    rng = np.random.default_rng(n)
    P = -(-(n + base) // 16)
    table, pages = _table(rng, 1, P)
    cache = Cache(rng, pages, Hkv, 16, D, kind)
    g, o = run_packed(rng, cache, table, [0, n], [base], n, H)
    check_attend(g, o, n + base)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_chunks_over_long_contexts_are_split_and_joined(kind):
    note(f"packed split {kind}")
    rng = np.random.default_rng(9)
    n, base = np.array([40, 1, 0, 25]), np.array([9000, 3000, 10, 4])
    starts = np.concatenate([[0], np.cumsum(n)])
    T, H, Hkv, page = int(starts[-1]), 4, 2, 32
    P = -(-9040 // page)
    table = np.zeros((4, P), np.int64)
    ids = rng.permutation(2 * P)
    for b, used in enumerate((P, 95, 1, 1)):
        table[b, :used], ids = ids[:used], ids[used:]
    table[1, 90] = 2 * P  # the second request's last slots lie on a page that does not exist
    cache = Cache(rng, 2 * P, Hkv, page, 128, kind)
    assert sv.attend_packed_workspace_bytes(T, 4, H, Hkv, 128, P, page, sv.SV_BF16 if kind == "bf16" else sv.SV_E4M3) > 256
    g, o = run_packed(rng, cache, table, starts, base, T, H)
    assert o["status"].tolist() == [0, 1, 0, 0]
    check_attend(g, o, 9040)


@pytest.mark.parametrize("kind,H,Hkv", [("bf16", 4, 2), ("e4m3", 4, 2), ("bf16", 130, 1), ("bf16", 300, 2)])
def test_many_requests_and_many_heads_of_one(kind, H, Hkv):
    # more requests than a wave holds at a time; row tiles that begin inside a token
    note(f"packed requests {kind} H={H}")
    rng = np.random.default_rng(H)
    n = rng.integers(0, 5, 150)
    n[130] = 70
    base = rng.integers(0, 60, 150)
    starts = np.concatenate([[0], np.cumsum(n)])
    table, pages = _table(rng, 150, 9)
    cache = Cache(rng, pages, Hkv, 16, 64, kind)
    g, o = run_packed(rng, cache, table, starts, base, int(starts[-1]), H)
    assert (o["status"] == 0).all()
    check_attend(g, o, 150)


def test_e4m3_rows_shared_by_eight_waves():
    # many row tiles of 256 rows, most of them partly filled; then parts of a long context
    note("packed eight waves")
    rng = np.random.default_rng(31)
    n, base = rng.integers(1, 20, 64), rng.integers(0, 40, 64)
    n[[5, 40]], base[[5, 40]] = [300, 257], [400, 3]
    starts = np.concatenate([[0], np.cumsum(n)])
    table, pages = _table(rng, 64, 22)
    cache = Cache(rng, pages, 16, 32, 128, "e4m3")
    g, o = run_packed(rng, cache, table, starts, base, int(starts[-1]), 16)
    check_attend(g, o, 700)
    table, pages = _table(rng, 1, 516)
    cache = Cache(rng, pages, 8, 32, 128, "e4m3")
    assert sv.attend_packed_workspace_bytes(500, 1, 8, 8, 128, 516, 32, sv.SV_E4M3) > 256
    g, o = run_packed(rng, cache, table, [0, 500], [16000], 500, 8)
    check_attend(g, o, 16500)


def test_without_base_and_at_the_first_token():
    note("packed no base")
    rng = np.random.default_rng(4)
    table, pages = _table(rng, 2, 4)
    cache = Cache(rng, pages, 1, 16, 64, "bf16")
    g, o = run_packed(rng, cache, table, [0, 50, 64], None, 64, 3)
    check_attend(g, o, 64)
    # the first token sees itself alone
    v = cache.values[1][table[0, 0], 0, 0]
    assert np.allclose(g["out"][0, 0].float().cpu().numpy(), v[None], rtol=2.0 ** -7, atol=2.0 ** -8)


def test_agrees_with_the_window_operator():
    note("packed against windows")
    rng = np.random.default_rng(5)
    B, N, H, Hkv, D, page = 3, 33, 8, 2, 128, 16
    table, pages = _table(rng, B, 12)
    cache = Cache(rng, pages, Hkv, page, D, "bf16")
    kv = cache.upload()
    base = np.array([100, 0, 47])
    q = bits_to_dev(bf16_bits(rng.normal(size=(B, N, H, D))))
    a = sv.spec_attend_paged(q, kv, ints_to_dev(table), ints_to_dev(base), lse=True)
    b = sv.spec_attend_packed(q.flatten(0, 1), kv, ints_to_dev(table), ints_to_dev([0, 33, 66, 99]), ints_to_dev(base), lse=True)
    # each within 2^-8 (weights) + 2^-8 (result) of the exact mean of values of up to about 4
    assert (a["out"].flatten(0, 1).float() - b["out"].float()).abs().max() <= 4 * 2.0 ** -6
    assert (a["lse"].flatten(0, 1) - b["lse"]).abs().max() <= 1e-4


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_tables_and_bounds(kind):
    note(f"packed bad {kind}")
    rng = np.random.default_rng(6)
    page, P = 16, 6
    # a bad page in the middle, a table that ends early, a negative base, decreasing bounds, bounds behind T, a good one
    starts = np.array([0, 90, 190, 200, 195, 205, 400])
    base = np.array([0, 10, -3, 0, 0, 0])
    table, pages = _table(rng, 6, P)
    table[0, 3] = -7
    table[5, 2] = pages
    cache = Cache(rng, pages, 2, page, 64, kind)
    g, o = run_packed(rng, cache, table, starts, base, 220, 4)
    assert o["status"].tolist() == [1, 1, 1, 2, 0, 2]
    check_attend(g, o, 100)


def test_overlapping_bounds_all_have_a_status():
    """Five requests of 128 tokens over the same 128, four rows a token: 20 row tiles where
    the sizes allow 4 + 9.  The first three fit."""
    note("packed overlap")
    rng = np.random.default_rng(29)
    cache = Cache(rng, 72, 1, 16, 64, "bf16")
    table = np.arange(72).reshape(9, 8)
    starts = np.array([0, 128] * 5)
    full = torch.full((9,), 7, dtype=torch.int32, device=dev())
    del full
    q = torch.zeros(128, 4, 64, dtype=torch.bfloat16, device=dev())
    g = sv.spec_attend_packed(q, cache.upload(), ints_to_dev(table), ints_to_dev(starts))
    assert g["status"].tolist() == [0, 2, 0, 2, 0, 2, 2, 2, 2]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_slots_that_are_not_finite_reach_no_row(kind, D):
    note(f"packed non-finite {kind} D={D}")
    rng = np.random.default_rng(7)
    page, H, Hkv = 16, 4, 2
    n, base = np.array([150, 40]), np.array([20, 0])
    starts = np.array([0, 150, 190])
    table, pages = _table(rng, 2, 11)
    cache = Cache(rng, pages, Hkv, page, D, kind)

    def put(b, s, which, d, bits, value):
        at = (table[b, s // page], 1, s % page, d)
        cache.host[which][at] = bits
        cache.values[which][at] = value

    nan, inf = ((0x7fc0, np.nan), (0x7f80, np.inf)) if kind == "bf16" else ((0x7f, np.nan), (0xff, np.nan))
    put(0, 100, 1, 3, *nan)       # a value that the later rows see
    put(0, 169, 1, D - 1, *inf)   # one that only the last row sees
    put(1, 30, 0, 5, *nan)        # a key
    for s in range(170, 176):     # behind the last token
        put(0, s, 0, 1, *nan)
        put(0, s, 1, 2, *inf)
    g, o = run_packed(rng, cache, table, starts, base, 190, H)
    check_attend(g, o, 170)
    out = g["out"][0].float().cpu().numpy()
    assert np.isfinite(out[:80]).all() and np.isnan(out[80:150, 2:, 3]).all() and np.isfinite(out[80:149, :, 4]).all()
    assert np.isfinite(out[150:180]).all() and np.isnan(out[180:, 2:]).all() and np.isfinite(out[180:, :2]).all()


@pytest.mark.parametrize("size", [1e3, 1e7, 1e12, 1e28])
def test_scores_of_any_size(size):
    # one slot's score far above the others: its value alone, whatever the size
    note(f"packed scores {size}")
    rng = np.random.default_rng(8)
    table, pages = _table(rng, 1, 10)
    cache = Cache(rng, pages, 1, 16, 64, "bf16")
    bits = bf16_bits(np.zeros((150, 2, 64)))
    bits[..., 0] = bf16_bits(np.array([size]))[0]
    for s in range(150):
        at = (table[0, s // 16], 0, s % 16, 0)
        cache.host[0][at] = bf16_bits(np.array([1.0 if s == 70 else -1.0 if s % 2 else 0.5]))[0]
        cache.values[0][at] = paged.bf16_values(cache.host[0][at])
    g, o = run_packed(rng, cache, table, [0, 150], None, 150, 2, scale=1.0, q=bits)
    v = cache.values[1][table[0, 70 // 16], 0, 70 % 16]
    out = g["out"][0].float().cpu().numpy()
    assert np.allclose(out[70:], np.broadcast_to(v, (80, 2, 64)), rtol=2.0 ** -7)
    lse = g["lse"][0].cpu().numpy()
    assert np.allclose(lse[70:], o["lse"][0, 70:], rtol=1e-6) and np.isfinite(lse).all()


def test_large_offsets():
    # pages beyond 2^32 bytes of the cache
    note("packed far pages")
    rng = np.random.default_rng(10)
    page, Hkv, D, far = 64, 8, 128, 40000
    k = torch.zeros(far, Hkv, page, D, dtype=torch.bfloat16, device=dev())
    v = torch.zeros_like(k)
    ids = np.array([[far - 1, 3, far - 7, 0]])
    small = Cache(rng, 4, Hkv, page, D, "bf16")
    for i, at in enumerate(ids[0]):
        k[at], v[at] = bits_to_dev(small.host[0][i]), bits_to_dev(small.host[1][i])
    q = bits_to_dev(bf16_bits(rng.normal(size=(220, 8, D))))
    a = sv.spec_attend_packed(q, sv.PagedKV(k, v), ints_to_dev(ids), ints_to_dev([0, 220]))
    b = sv.spec_attend_packed(q, small.upload(), ints_to_dev([[0, 1, 2, 3]]), ints_to_dev([0, 220]))
    assert torch.equal(a["out"], b["out"]) and int(a["status"][0]) == 0


# ---- append ----------------------------------------------------------------------------

def _append_inputs(rng, T, H, Hkv, D, rot, most, axes):
    x = bf16_bits(rng.normal(size=(T, H + 2 * Hkv, D)))
    wq, wk = (bf16_bits(1 + 0.2 * rng.normal(size=D)) for _ in range(2))
    angle = rng.random((most, rot // 2)) * 6.3
    rope = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    return x, wq, wk, rope, rng.integers(0, most, (axes, T)), rng.integers(0, axes, rot // 2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,rot,interleaved,axes", [(64, 64, False, 1), (128, 128, False, 3), (128, 64, True, 3),
                                                    (256, 128, False, 4), (128, 128, True, 2), (256, 256, True, 1)])
def test_append_packed(kind, D, rot, interleaved, axes):
    note(f"append packed {kind} D={D} rot={rot} il={interleaved} axes={axes}")
    rng = np.random.default_rng(D + rot + axes)
    H, Hkv, page = 5, 2, 16
    n, base = np.array([30, 0, 1, 17, 0, 50]), np.array([0, 4, 15, 16, 0, 33])
    starts = np.concatenate([[2], 2 + np.cumsum(n)])
    T = int(starts[-1]) + 3
    table, pages = _table(rng, len(n), 6)
    cache = Cache(rng, pages, Hkv, page, D, kind)
    x, wq, wk, rope, pos, axis = _append_inputs(rng, T, H, Hkv, D, rot, 70, axes)
    kv = cache.upload()
    xd = bits_to_dev(x)
    q_out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    g = sv.spec_append_kv_packed(xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], kv, ints_to_dev(table), ints_to_dev(starts),
                                 ints_to_dev(base), ints_to_dev(pos), q_weight=bits_to_dev(wq), k_weight=bits_to_dev(wk),
                                 eps=1e-6, rope=torch.from_numpy(rope).to(dev()), interleaved=interleaved,
                                 pair_axis=ints_to_dev(axis), q_out=q_out)
    assert (g["status"] == 0).all()
    v64 = paged.bf16_values(x)
    off = (D / 2 + 16) * U
    want, mag = prompt.append_rows(v64[:, :H], paged.bf16_values(wq), 1e-6, rope, rot, interleaved, pos, axis, starts)
    got = q_out.float().cpu().numpy().astype(np.float64)
    inside = np.zeros(T, bool)
    inside[starts[0]:starts[-1]] = True
    assert (got[~inside] == 7).all()
    assert (np.abs(got - want) <= off * mag + 2.0 ** -8 * (np.abs(want) + off * mag))[inside].all()
    ks, mags = prompt.append_rows(v64[:, H:H + Hkv], paged.bf16_values(wk), 1e-6, rope, rot, interleaved, pos, axis, starts)
    rows = [("k", ks, mags, kv.k_pages, kv.k_scales, 0), ("v", v64[:, H + Hkv:], np.abs(v64[:, H + Hkv:]), kv.v_pages, kv.v_scales, 1)]
    for name, want, mag, arr, scales, which in rows:
        bits = to_bits(arr)
        values = paged.bf16_values(bits) if kind == "bf16" else paged.e4m3_values(bits)
        left = np.ones(bits.shape[:3], bool)
        for b in range(len(n)):
            for j in range(n[b]):
                t, s = starts[b] + j, base[b] + j
                at = (table[b, s // page], slice(None), s % page)
                left[at] = False
                if kind == "bf16":
                    assert (np.abs(values[at] - want[t]) <= off * mag[t] + 2.0 ** -8 * (np.abs(want[t]) + off * mag[t])).all(), name
                else:
                    sc = scales[at].cpu().numpy().astype(np.float64)
                    top = np.abs(want[t]).max(-1)
                    assert (np.abs(sc * 448 - top) <= off * mag[t].max(-1) + 4 * U * top).all()
                    tol = off * mag[t] + 2.0 ** -4 * (np.abs(want[t]) + off * mag[t]) + 2.0 ** -9 * sc[:, None]
                    assert (np.abs(values[at] * sc[:, None] - want[t]) <= tol).all(), name
        assert np.array_equal(bits[left], cache.host[which][left])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N", [(3, 37), (2, 2500)])
def test_append_packed_equals_the_window_operator(kind, B, N):
    # one axis: the same bits as padded windows of equal length
    note(f"append packed against windows {kind} N={N}")
    rng = np.random.default_rng(N)
    H, Hkv, D, page = 4, 2, 128, 32
    x, wq, wk, rope, pos, _ = _append_inputs(rng, B * N, H, Hkv, D, 128, 3000, 1)
    base = np.array([5, 0, 64])[:B]
    P = -(-(N + 64) // page)
    table, pages = _table(rng, B, P)
    kw = dict(q_weight=bits_to_dev(wq), k_weight=bits_to_dev(wk), rope=torch.from_numpy(rope).to(dev()))
    xd = bits_to_dev(x)
    caches = [Cache(np.random.default_rng(0), pages, Hkv, page, D, kind).upload() for _ in range(2)]
    w = xd.view(B, N, H + 2 * Hkv, D)
    a = sv.spec_append_kv_paged(w[:, :, :H], w[:, :, H:H + Hkv], w[:, :, H + Hkv:], caches[0], ints_to_dev(table),
                                ints_to_dev(base), ints_to_dev(pos.reshape(B, N)), **kw)
    b = sv.spec_append_kv_packed(xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], caches[1], ints_to_dev(table),
                                 ints_to_dev(np.arange(B + 1) * N), ints_to_dev(base), ints_to_dev(pos[0]), **kw)
    assert torch.equal(a["q"].flatten(0, 1), b["q"])
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        p, q = getattr(caches[0], name), getattr(caches[1], name)
        assert p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_append_packed_bad_tokens_and_many_requests():
    note("append packed bad")
    rng = np.random.default_rng(11)
    H, Hkv, D, page, B = 2, 1, 64, 16, 300
    n = rng.integers(0, 4, B)
    starts = np.concatenate([[0], np.cumsum(n)])
    T = int(starts[-1])
    table, pages = _table(rng, B, 1)
    base = np.full(B, 3)
    base[7], base[9] = 15, -1  # runs out of its table; a slot below 0
    table[20, 0] = pages + 5
    x, wq, wk, rope, pos, axis = _append_inputs(rng, T, H, Hkv, D, 64, 40, 3)
    pos[1, starts[30]] = 40
    cache = Cache(rng, pages, Hkv, page, D, "bf16")
    kv, xd = cache.upload(), bits_to_dev(x)

    def call(axis):
        return sv.spec_append_kv_packed(xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], kv, ints_to_dev(table),
                                        ints_to_dev(starts), ints_to_dev(base), ints_to_dev(pos),
                                        rope=torch.from_numpy(rope).to(dev()), pair_axis=ints_to_dev(axis))

    want = np.zeros(T, int)
    for b in range(B):
        for j in range(n[b]):
            t, s = starts[b] + j, base[b] + j
            want[t] = 1 if s < 0 or s >= 16 or b == 20 else 0
            if want[t] == 0 and (pos[:, t] >= 40).any():
                want[t] = 2
    assert np.array_equal(call(axis)["status"].cpu().numpy(), want)
    before = kv.k_pages.clone()
    bad = axis.copy()
    bad[31] = 3
    st = call(bad)["status"].cpu().numpy()
    assert np.array_equal(st == 0, np.zeros(T, bool)) and torch.equal(before, kv.k_pages)


def test_refusals():
    cache = Cache(np.random.default_rng(0), 4, 2, 16, 64, "bf16").upload()
    q, k = torch.zeros(5, 4, 64, device=dev()).bfloat16(), torch.zeros(5, 2, 64, device=dev()).bfloat16()
    table, starts = ints_to_dev([[0, 1], [2, 3]]), ints_to_dev([0, 2, 5])
    rope, pos = torch.zeros(9, 64, device=dev()), ints_to_dev(np.zeros((3, 5)))
    ok = dict(q=q, cache=cache, page_table=table, starts=starts)
    for bad in (dict(q=q[0]), dict(q=q.float()), dict(q=q[..., :32]), dict(starts=starts[:2]), dict(starts=None),
                dict(starts=starts.long()), dict(base=starts), dict(page_table=table[0]), dict(out=q.float()),
                dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            sv.spec_attend_packed(**{**ok, **bad})
    ok.update(k=k, v=k, rope=rope, positions=pos, pair_axis=ints_to_dev(np.zeros(32)))
    sv.spec_append_kv_packed(**ok)
    for bad in (dict(k=k[:4]), dict(v=q), dict(positions=None), dict(positions=pos[:, :4]), dict(pair_axis=None),
                dict(pair_axis=ints_to_dev(np.zeros(31))), dict(rope=rope.double()), dict(q_weight=rope[0])):
        with pytest.raises(ValueError):
            sv.spec_append_kv_packed(**{**ok, **bad})
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_append_kv_packed(**{**ok, "positions": ints_to_dev(np.zeros((5, 5)))})
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_attend_packed(q[:, :3], cache, table, starts)
