"""Failure detection of the paged decode without a fault: a bounded wait that runs out.

The test hook makes the loading warps stop in front of a key block, with the blocks before it loaded or on their way.  The
computing warps' wait for it runs out after the (short) limit: the kernel records that in the cache's error word, waits for
its copies, frees what it holds and returns; the plan, the cache and the context stay usable.
"""
import time

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 16, 32, 64])
@pytest.mark.parametrize("withhold,grid", [(1, 1 << 20), (3, 1 << 20), (2, 5)])
def test_a_withheld_block_runs_out_and_the_plan_stays_usable(store, d, rows, withhold, grid):
    """Several units a CTA and cut units; the second call after the abort has the bits of the first."""
    lens, page = [3000, 0, 700, 1300], 32
    pages, scales, table, n = pu.make_pool(lens, 2, page, d, store, seed=1)
    cache = tsa.PagedCache(n, 2, page, d, dtype=store, pages=pages.cuda(), scales=None if scales is None else scales.cuda())
    Q = torch.randn((4, 2 * rows, 1, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    plan = tsa.PagedDecodeAttention(4, 2 * rows, 2, 1, d)
    plan.set_grid_limit(grid)
    want = plan(Q, cache, tab, ln)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    plan.set_watchdog(20_000_000, withhold=withhold)  # 20 ms
    start = time.monotonic()
    for _ in range(2):
        plan(Q, cache, tab, ln)
    assert cache.poll_device_error() == (tsa.ATTN_ERR_DEVICE_TIMEOUT, tsa.CACHE_ERR_WAIT)
    assert time.monotonic() - start < 2.0  # a wait that has run out ends the others
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    plan.set_watchdog(2_000_000_000)
    for _ in range(2):
        got = plan(Q, cache, tab, ln)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_watchdog_refusals():
    plan = tsa.PagedDecodeAttention(1, 1, 1, 1, 64)
    for args in ((0,), (-1,), (1000, -1)):
        with pytest.raises(tsa.AttnError) as e:
            plan.set_watchdog(*args)
        assert e.value.status == tsa.ATTN_ERR_INVALID_ARG
    assert tsa.attn_paged_set_watchdog(0, 1000) == tsa.ATTN_ERR_INVALID_ARG
