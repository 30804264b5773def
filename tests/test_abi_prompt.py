"""Host-side checks of the prompt operators' entry points (CPU only: every call here is
refused, or empty, before a device is touched)."""

import ctypes
import os
import re

import pytest

import draft_token_verification_04_amd as sv
from test_abi_paged import BAD_CACHES, BAD_POINTERS, FAKE, INV, ODD, UNS, WS, _cache


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


NAN, INF = float("nan"), float("inf")


def _norm(lib, **kw):
    a = dict(x=FAKE, xs=256, r=None, w=FAKE, eps=1e-6, T=3, D=256, ro=None, out=FAKE, dt=sv.SV_E4M3, sc=FAKE)
    a.update(kw)
    return lib.spec_rms_norm(a["x"], a["xs"], a["r"], a["w"], a["eps"], a["T"], a["D"], a["ro"], a["out"], a["dt"],
                             a["sc"], None)


def test_norm_refusals(lib):
    for kw, want in [(dict(dt=sv.SV_F32), UNS), (dict(dt=9), UNS), (dict(T=-1), INV), (dict(D=0), INV),
                     (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(D=252), UNS),
                     (dict(D=sv.SV_MAX_NORM_COLS + 8, xs=1 << 20), UNS), (dict(T=1 << 24), UNS), (dict(x=None), INV),
                     (dict(out=None), INV), (dict(sc=None), INV), (dict(dt=sv.SV_BF16), INV), (dict(x=ODD), INV),
                     (dict(r=ODD), INV), (dict(w=ODD), INV), (dict(ro=ODD), INV), (dict(out=ODD), INV),
                     (dict(sc=ODD), INV), (dict(xs=248), INV), (dict(xs=260), INV), (dict(xs=1 << 33), UNS)]:
        assert _norm(lib, **kw) == want, kw
    assert _norm(lib, T=0, x=None, out=None) == sv.SV_OK


def _linear(lib, **kw):
    a = dict(x=FAKE, xs=256, s=FAKE, ss=8, w=FAKE, ws=FAKE, M=8, N=40, K=256, out=FAKE, dt=sv.SV_BF16, work=FAKE, wb=0)
    a.update(kw)
    return lib.spec_linear_e4m3(a["x"], a["xs"], a["s"], a["ss"], a["w"], a["ws"], a["M"], a["N"], a["K"], a["out"],
                                a["dt"], a["work"], a["wb"], None)


def test_linear_refusals(lib):
    for kw, want in [(dict(dt=sv.SV_E4M3), UNS), (dict(dt=-3), UNS), (dict(M=-1), INV), (dict(N=0), INV),
                     (dict(K=0), INV), (dict(K=248, xs=256), UNS), (dict(K=sv.SV_MAX_LINEAR_K + 16, xs=1 << 20), UNS),
                     (dict(M=1 << 30, N=1 << 30, ss=1 << 30), UNS), (dict(x=None), INV), (dict(s=None), INV),
                     (dict(w=None), INV), (dict(ws=None), INV), (dict(out=None), INV), (dict(work=None), INV),
                     (dict(x=ODD), INV), (dict(w=ODD), INV), (dict(out=ODD), INV), (dict(work=ODD), INV),
                     (dict(xs=240), INV), (dict(xs=264), INV), (dict(ss=7), INV), (dict(xs=1 << 33), UNS),
                     (dict(ss=1 << 33), UNS), (dict(), WS)]:
        assert _linear(lib, **kw) == want, kw
    assert _linear(lib, M=0, x=None, work=None) == sv.SV_OK
    f = lib.sv_linear_workspace_bytes
    need = f(8, 40, 256, sv.SV_BF16)
    assert need >= 256 and need % 256 == 0 and _linear(lib, wb=need - 1) == WS
    assert f(0, 40, 256, 1) == 0 and f(8, 0, 256, 1) == 0 and f(8, 40, 0, 1) == 0 and f(8, 40, 250, 1) == 0
    assert f(8, 40, 256, sv.SV_E4M3) == 0 and f(8, 40, sv.SV_MAX_LINEAR_K + 16, 1) == 0


def _append(lib, cache=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=4 * 128, ks=2 * 128, vs=2 * 128, wq=None, wk=None, eps=1e-6, rope=FAKE, rot=128,
             max_pos=100, il=0, pos=FAKE, axes=3, axis=FAKE, starts=FAKE, base=FAKE, T=7, B=2, H=4, table=FAKE, P=5,
             out=FAKE, st=None)
    a.update(kw)
    return lib.spec_append_kv_packed(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["wq"], a["wk"], a["eps"],
                                     a["rope"], a["rot"], a["max_pos"], a["il"], a["pos"], a["axes"], a["axis"],
                                     a["starts"], a["base"], a["T"], a["B"], a["H"], cache or _cache(), a["table"],
                                     a["P"], a["out"], a["st"], None)


def test_append_packed_refusals(lib):
    for c, want in BAD_CACHES:
        assert _append(lib, _cache(**c)) == want, c
    for c in BAD_POINTERS:
        assert _append(lib, _cache(**c)) == INV, c
    for kw, want in [(dict(B=-1), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(P=0), INV), (dict(eps=-1.0), INV),
                     (dict(eps=NAN), INV), (dict(rot=0), INV), (dict(rot=144), INV), (dict(rot=24), UNS),
                     (dict(max_pos=0), INV), (dict(axes=0), INV), (dict(axes=2, axis=None), INV),
                     (dict(axes=sv.SV_MAX_AXES + 1), UNS), (dict(P=1 << 28), UNS), (dict(T=1 << 24), UNS),
                     (dict(H=1 << 17), UNS), (dict(B=(1 << 31) - 1), UNS), (dict(q=None), INV), (dict(k=None), INV),
                     (dict(v=None), INV), (dict(starts=None), INV), (dict(table=None), INV), (dict(out=None), INV),
                     (dict(pos=None), INV), (dict(wq=FAKE), INV), (dict(wk=FAKE), INV), (dict(q=ODD), INV),
                     (dict(k=ODD), INV), (dict(v=ODD), INV), (dict(out=ODD), INV), (dict(rope=ODD), INV),
                     (dict(wq=ODD, wk=FAKE), INV), (dict(qs=500), INV), (dict(qs=504), INV), (dict(ks=128), INV),
                     (dict(vs=-256), INV), (dict(qs=1 << 33), UNS)]:
        assert _append(lib, **kw) == want, kw
    assert _append(lib, T=0, q=None, out=None) == sv.SV_OK


def _attend(lib, cache=None, **kw):
    a = dict(q=FAKE, qs=4 * 128, table=FAKE, P=5, starts=FAKE, base=None, T=7, B=2, H=4, scale=0.1, out=FAKE, lse=None,
             st=None, ws=FAKE, wsb=0)
    a.update(kw)
    return lib.spec_attend_packed(a["q"], a["qs"], cache or _cache(), a["table"], a["P"], a["starts"], a["base"], a["T"],
                                  a["B"], a["H"], a["scale"], a["out"], a["lse"], a["st"], a["ws"], a["wsb"], None)


def test_attend_packed_refusals(lib):
    for c, want in BAD_CACHES:
        assert _attend(lib, _cache(**c)) == want, c
    for c in BAD_POINTERS:
        assert _attend(lib, _cache(**c)) == INV, c
    for kw, want in [(dict(B=-1), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(H=3), INV), (dict(P=0), INV),
                     (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV),
                     (dict(P=1 << 28), UNS), (dict(T=1 << 30), UNS), (dict(H=1 << 18), UNS), (dict(B=1 << 30, T=1 << 28), UNS),
                     (dict(q=None), INV), (dict(table=None), INV), (dict(starts=None), INV), (dict(out=None), INV),
                     (dict(ws=None), INV), (dict(q=ODD), INV), (dict(out=ODD), INV), (dict(ws=ODD), INV),
                     (dict(qs=508), INV), (dict(qs=504), INV), (dict(qs=1 << 33), UNS), (dict(), WS)]:
        assert _attend(lib, **kw) == want, kw
    assert _attend(lib, scale=3e38, wsb=1 << 30) == UNS
    assert _attend(lib, B=0, q=None, ws=None) == sv.SV_OK
    f = lib.sv_attend_packed_workspace_bytes
    need = f(7, 2, 4, 2, 128, 5, 16, sv.SV_BF16)
    assert need >= 256 and need % 256 == 0 and _attend(lib, wsb=need - 1) == WS
    assert f(7, 0, 4, 2, 128, 5, 16, sv.SV_BF16) == 0 and f(7, 2, 5, 2, 128, 5, 16, sv.SV_BF16) == 0 and f(7, 2, 4, 2, 96, 5, 16, sv.SV_BF16) == 0
    assert f(-1, 2, 4, 2, 128, 5, 16, sv.SV_BF16) == 0 and f(7, 2, 4, 2, 128, 1 << 28, 16, sv.SV_BF16) == 0
    # few rows over a long table are split, within the bound; many rows are not
    assert 256 < f(200, 1, 32, 8, 128, 8192, 16, sv.SV_BF16) <= 513 << 20
    assert f(20000, 4, 32, 8, 128, 8192, 16, sv.SV_BF16) == 256
    assert f(64, 64, 64, 64, 256, 1 << 20, 16, sv.SV_BF16) <= 513 << 20


def test_the_largest_sizes_are_refused(lib):
    top = (1 << 31) - 1
    f = lib.sv_linear_workspace_bytes
    for m, n in [(1, top), (17, top), (64, top), (top, 1), (top, 64), (top, top), (300, top), (top - 300, 1), (1, top - 15)]:
        for dt in (sv.SV_BF16, sv.SV_F32):
            assert f(m, n, 16, dt) == 0, (m, n, dt)
            assert _linear(lib, M=m, N=n, K=16, ss=1 << 31, dt=dt) == UNS, (m, n, dt)
    for b in (top - 1, top - 63, 1 << 24):
        assert _append(lib, B=b) == UNS, b
    f = lib.sv_attend_packed_workspace_bytes
    for t, b in [(7, top), (0, top), (7, top - 63), (7, 1 << 24), (top, 1), (top, top)]:
        assert f(t, b, 4, 2, 128, 5, 16, sv.SV_BF16) == 0 and _attend(lib, T=t, B=b, wsb=1 << 40) == UNS, (t, b)


def test_constants_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "spec_verify.h")).read()
    consts = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(SV_[A-Z_]+)\s+(\d+)", text)}
    for name in ("SV_MAX_NORM_COLS", "SV_MAX_LINEAR_K", "SV_MAX_AXES"):
        assert getattr(sv, name) == consts[name], name
