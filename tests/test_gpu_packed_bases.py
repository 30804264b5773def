"""GPU tests of the packed-sequence operators with numbers of cached tokens at the ends of
int32, and below 0."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, ints_to_dev, note
from oracle import paged
from paged_helpers import Cache, check_attend
from test_gpu_packed_edges import Case

pytestmark = pytest.mark.gpu
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", ["bf16 64", "eight waves"])
def test_bases_at_the_ends_of_int32(kind, form):
    note(f"packed edges base {kind} {form}")
    c = Case(form, 5)
    if kind != c.kind:
        c.cache, c.kind = Cache(c.rng, len(c.cache.host[0]), c.cache.host[0].shape[1], c.page, c.D, kind), kind
    for first, second in ((INT_MIN, INT_MAX), (INT_MIN + 1, INT_MAX - 3), (-1, INT_MIN), (INT_MAX, INT_MIN + 2)):
        c.base[:2] = first, second
        g, o = c.run()
        assert o["status"][:2].tolist() == [1, 1]
        check_attend(g, o, 2000)
        rows = slice(0, int(c.starts[2]))
        assert (g["out"][0, rows] == 0).all() and (g["lse"][0, rows] == -float("inf")).all()
        # the cache write: token j of a request takes slot base + j where there is one
        kv = c.cache.upload()
        before = [t.view(torch.uint8).clone() for t in (kv.k_pages, kv.v_pages)]
        x = torch.ones(c.T, c.H, c.D, dtype=torch.bfloat16, device=dev())
        k = torch.ones(c.T, c.cache.host[0].shape[1], c.D, dtype=torch.bfloat16, device=dev())
        table = np.where(np.arange(len(c.n))[:, None] < 2, c.table, -1)
        st = sv.spec_append_kv_packed(x, k, k, kv, ints_to_dev(table), ints_to_dev(c.starts), ints_to_dev(c.base))["status"]
        want = [int(paged.row_of(table[b], int(c.base[b]) + j, c.page, len(c.cache.host[0])) is None)
                for b in range(len(c.n)) for j in range(c.n[b])]
        assert st.tolist() == want and sum(want) >= c.T - c.n[0] + 1
        if all(want):
            assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(before, (kv.k_pages, kv.v_pages)))
