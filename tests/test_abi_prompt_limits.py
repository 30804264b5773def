"""Host-side checks of the prompt operators' launch limits (CPU only: every call here is
refused before a device is touched)."""

import pytest

import draft_token_verification_04_amd as sv
from test_abi_paged import UNS, _cache
from test_abi_prompt import _attend, lib  # noqa: F401


# A workgroup of eight waves counts as two of 256 work items: single tokens of as many
# requests, each a row tile for every head.
@pytest.mark.parametrize("requests", [131072, 140000, 262143])
def test_workgroups_of_eight_waves_count_twice(lib, requests):  # noqa: F811
    c = _cache(kv_heads=64, page_size=16, head_dim=128, dt=sv.SV_E4M3, k_scale=1 << 20, v_scale=1 << 20)
    f = lib.sv_attend_packed_workspace_bytes
    assert f(requests, requests, 64, 64, 128, 1, 16, sv.SV_E4M3) == 0
    kw = dict(T=requests, B=requests, H=64, qs=64 * 128, P=1, wsb=1 << 40)
    assert _attend(lib, c, **kw) == UNS
    # what fits, and the same in bf16, whose workgroups have four waves
    assert f(131000, 131000, 64, 64, 128, 1, 16, sv.SV_E4M3) == 256
    assert f(requests, requests, 64, 64, 128, 1, 16, sv.SV_BF16) == 256
