"""GPU tests of spec_attend_paged with page tables far wider than the requests, as a
program keeps them whose graphs are captured for the longest context."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import note
from paged_helpers import Cache, check_attend, random_tree, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H,Hkv,D,N,slots", [
    (5, 8, 2, 128, 1, 1 << 17), (4, 4, 2, 64, 9, 1 << 17), (3, 8, 2, 128, 33, 1 << 17), (2, 2, 1, 256, 20, 1 << 17),
    (300, 2, 2, 64, 1, 1 << 20), (40, 16, 1, 128, 12, 1 << 20), (2, 4, 4, 128, 3, 1 << 30)])
def test_wide_tables(kind, B, H, Hkv, D, N, slots):
    note(f"attend wide table {kind} B={B} H={H} D={D} N={N} slots={slots}")
    rng = np.random.default_rng(B + N)
    page = 1024 if slots == 1 << 30 else 16
    P = slots // page
    base = rng.integers(0, 300, B)
    base[:2] = [2300, 1000]
    counts = rng.integers(1, N + 1, B)
    counts[0] = N
    used = -(-(base + counts) // page)
    table = np.full((B, P), -1, np.int32)
    ids = rng.permutation(int(used.sum()) + 3)
    for b in range(B):
        table[b, :used[b]], ids = ids[:used[b]], ids[used[b]:]
    cache = Cache(rng, int(used.sum()) + 3, Hkv, page, D, kind)
    assert sv.attend_workspace_bytes(B, N, H, Hkv, D, P, page) <= 513 << 20
    g, o = run_attend(rng, cache, table, base, N, H, counts=counts, parents=random_tree(rng, B, N) if N > 8 else None)
    assert (o["status"] == 0).all()
    check_attend(g, o, 2300 + N)
    torch.cuda.empty_cache()
