"""Shared prefixes whose stretches of work are single tiles of positions: a CTA goes through many of them, and of its two
streams the second has no tile in most.

A step over such prefixes, on one CTA and on many, against the float64 definition, with the same bits on every call and no wait
that runs out.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa
from test_gpu_prefix import _int32, _make, _reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grid", [1, 3, None])
@pytest.mark.parametrize("longest", [128, 400])
def test_many_stretches_of_one_tile(store, d, grid, longest):
    """Longest 128: only such stretches; 400: with ones of two to four tiles between them, in any order."""
    G, B, Hq, Hkv, S_q, page = 150, 300, 8, 2, 1, 16
    g = torch.Generator().manual_seed(longest + d)
    plens = torch.randint(0, longest + 1, (G,), generator=g).tolist()
    lens = torch.randint(0, 20, (B,), generator=g).tolist()
    of = torch.randint(-1, G, (B,), generator=g).tolist()
    cache, vals, ptab, table = _make(plens, lens, Hkv, page, d, store)
    Q = torch.randn((B, Hq, S_q, d), generator=g).to(torch.bfloat16)
    plan = tsa.SharedPrefixAttention(B, Hq, Hkv, S_q, d)
    if grid:
        plan.set_grid_limit(grid)
    args = (Q.cuda(), cache, ptab.cuda(), _int32(plens), table.cuda(), _int32(lens))
    O, LSE = plan(*args, prefix_of=_int32(of))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pu.check_decode(O, LSE, _reference(Q, vals, ptab, plens, of, table, page, lens, 1 / math.sqrt(d), tsa.MASK_CAUSAL), d)
    for _ in range(20):
        O2, LSE2 = plan(*args, prefix_of=_int32(of))
        assert torch.equal(O2, O) and torch.equal(LSE2, LSE)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
