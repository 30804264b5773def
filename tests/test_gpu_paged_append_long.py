"""GPU test of spec_append_kv_paged on chunks of thousands of tokens, where a workgroup
walks all rows of its token."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_of_a_long_chunk_in_passes(kind):
    # from 4096 tokens a workgroup takes all of a token's rows: the same rows as
    # shorter calls write, token by token, padding and bad slots included
    note(f"append in passes {kind}")
    rng = np.random.default_rng(3)
    B, N, H, Hkv, D, page = 3, 1500, 40, 3, 128, 16
    P = -(-N // page) + 1
    x = torch.randn(B, N, H + 2 * Hkv, D, device=dev(), generator=torch.Generator(dev()).manual_seed(1)).bfloat16()
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    table = rng.permutation(B * P).reshape(B, P)
    table[1, 7] = B * P
    i32 = dict(dtype=torch.int32, device=dev())
    tab, base, counts = torch.tensor(table, **i32), torch.tensor([0, 5, 13], **i32), torch.tensor([N, N - 3, 700], **i32)
    pos = torch.tensor(rng.integers(0, 900, (B, N)), **i32)
    pos[0, 11] = 900
    rope = torch.randn(900, D, device=dev(), generator=torch.Generator(dev()).manual_seed(2))
    w = (torch.rand(2, D, device=dev(), generator=torch.Generator(dev()).manual_seed(4)) + 0.5).bfloat16()
    got = []
    for step in (N, 300):
        shape = (B * P, Hkv, page, D)
        pages = [torch.zeros(shape, dtype=torch.uint8 if kind == "e4m3" else torch.bfloat16, device=dev()) for _ in range(2)]
        scales = [torch.zeros(shape[:3], device=dev()) if kind == "e4m3" else None for _ in range(2)]
        views = [p.view(torch.float8_e4m3fn) if kind == "e4m3" else p for p in pages]
        cache = sv.PagedKV(*views, *scales)
        outs = torch.full((B, N, H, D), 7.0, dtype=torch.bfloat16, device=dev())
        status = []
        for n in range(0, N, step):
            cut = [t[:, n:n + step].contiguous() for t in (q, k, v)] if step < N else (q, k, v)
            part = torch.full((B, min(step, N - n), H, D), 7.0, dtype=torch.bfloat16, device=dev())
            r = sv.spec_append_kv_paged(*cut, cache, tab, base + n, pos[:, n:n + step].contiguous(), q_weight=w[0],
                                        k_weight=w[1], rope=rope, counts=(counts - n).contiguous(), q_out=part)
            outs[:, n:n + step] = part
            status.append(r["status"])
        torch.cuda.synchronize()
        got.append([outs, torch.cat(status, 1), *pages] + [s for s in scales if s is not None])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    st = got[0][1]
    assert st[0, 11] == 2 and (st[1, 107:123] == 1).all() and int(st.ne(0).sum()) == 17
