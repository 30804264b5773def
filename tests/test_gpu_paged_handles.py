"""GPU tests of PagedKV as a handle: what it was made from stays what calls use."""

import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, note

pytestmark = pytest.mark.gpu


def test_a_cache_handle_is_fixed():
    note("paged handle")
    k, v = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    kv = sv.PagedKV(k, v)
    for name in ("k_pages", "v_pages", "k_scales", "v_scales", "num_pages", "page_size", "head_dim", "device", "_c"):
        with pytest.raises(AttributeError):
            setattr(kv, name, torch.ones_like(k))
    assert kv.k_pages is k and kv.v_pages is v
    assert (kv.num_pages, kv.kv_heads, kv.page_size, kv.head_dim) == (4, 2, 16, 64)
