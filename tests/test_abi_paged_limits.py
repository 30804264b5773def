"""Sizes whose launch would have 2^32 work items or more are refused on the host
(CPU only: every call here is refused before a device is touched; sizes that are
accepted are asked for through the workspace queries)."""

import pytest

import draft_token_verification_04_amd as sv
from test_abi_paged import UNS, _append, _attend, _cache, _commit, _logprobs

MOST = (1 << 24) - 1  # workgroups of 256


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_append_of_too_many_tokens(lib):
    for B, N in ((MOST + 1, 1), (1, MOST + 1), (1 << 12, 1 << 13), (1 << 20, 17), ((1 << 31) - 1, 1)):
        assert _append(lib, B=B, N=N) == UNS, (B, N)


def test_attention_of_too_many_workgroups(lib):
    f = lib.sv_attend_workspace_bytes
    for B, N, H, hkv, D, P in ((MOST + 1, 1, 1, 1, 128, 1), (MOST // 8 + 8, 1, 8, 8, 128, 1), (1 << 23, 1, 32, 8, 64, 4),
                               (1 << 21, 64, 2, 2, 256, 1)):
        assert _attend(lib, _cache(kv_heads=hkv, head_dim=D), B=B, N=N, H=H, qs=H * D, P=P, wsb=1 << 62) == UNS, (B, N, H)
        assert f(B, N, H, hkv, D, P, 16) == 0
    assert f(MOST - 7, 1, 1, 1, 128, 1, 16) == 256 and f(MOST // 8 - 1, 1, 8, 8, 128, 1, 16) == 256
    assert f(1 << 16, 1, 8, 1, 64, 512, 16) > 0


def test_commit_of_too_many_waves(lib):
    assert _commit(lib, B=1 << 27, G=1, h=1) == UNS      # a wave per request
    assert _commit(lib, B=1 << 26, G=5, h=1) == UNS
    assert _commit(lib, B=1 << 26, G=1, h=20) == UNS


def test_logprobs_of_too_many_rows(lib):
    f = lib.sv_token_logprobs_workspace_bytes
    for R, V, dt in ((MOST + 1, 1, sv.SV_BF16), (1 << 25, 50, sv.SV_F32), (1 << 24, 1000, sv.SV_F32),
                     (10_000_000, 70_000, sv.SV_BF16), (9_000_000, 60_000, sv.SV_F32)):
        assert f(R, V, dt, 0) == 0 and f(R, V, dt, 1) == 0, (R, V)
        assert _logprobs(lib, R=R, V=V, dt=dt, k=0, wsb=1 << 62) == UNS, (R, V)
    assert f(MOST, 1000, sv.SV_BF16, 0) > 0 and f(MOST, 1, sv.SV_F32, 1) > 0
    assert _logprobs(lib, R=MOST, V=1000, k=0, wsb=256) == sv.SV_ERR_WORKSPACE


def test_attention_workspace_is_bounded(lib):
    # page tables as wide as a model's longest context, not as the batch's longest request
    f = lib.sv_attend_workspace_bytes
    for B, N, H, hkv, D, slots in ((64, 1, 32, 8, 128, 131072), (256, 1, 32, 8, 128, 131072), (64, 33, 32, 8, 128, 131072),
                                   (256, 64, 64, 8, 128, 1 << 20), (512, 64, 64, 1, 256, 1 << 20), (1, 64, 128, 8, 128, 1 << 30),
                                   (4096, 8, 32, 8, 64, 1 << 18), (1, 1, 1, 1, 64, 1 << 30)):
        need = f(B, N, H, hkv, D, slots // 16, 16)
        assert 256 <= need <= 513 << 20, (B, N, H, need)
