"""Selection over a cache that eviction has cut: the bounds of the pages that rows were moved to are computed again, all of
them, and follow later rows as before."""
import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 48)])
@pytest.mark.parametrize("into", ["other pages", "their own"])
def test_select_after_eviction(store, d, page, into):
    B, Hq, Hkv, wide, keep = 3, 4, 2, 20, 6
    lens, heavy, recent = [12 * page + 5, 3 * page, 9 * page - 1], 7 * page + 3, page + 9
    g = torch.Generator().manual_seed(41)
    total = 2 * B * wide
    cache = tsa.PagedCache(total, Hkv, page, d, dtype=store)
    order = torch.randperm(total, generator=g).to(torch.int32)
    table, other = order[:B * wide].view(B, wide), order[B * wide:].view(B, wide)

    def rows(n, heads=Hkv):
        return torch.randn((B, heads, n, d), generator=g).to(torch.bfloat16).cuda()

    bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
    n = _int32(lens)
    for t in (other, table):  # the other pages hold a sequence that has ended, with its bounds
        cache.write(rows(max(lens)), rows(max(lens)), t.cuda(), n, new_len=n)
        bounds.update(t.cuda(), n)
    weights.weights.copy_(torch.rand(weights.weights.shape, generator=g))
    stale = bounds.codes.clone()
    if into == "other pages":
        n, _ = weights.evict(table.cuda(), n, heavy, recent, to_table=other.cuda())
        table = other
    else:
        n, _ = weights.evict(table.cuda(), n, heavy, recent)
    assert torch.equal(bounds.codes, stale)  # (eviction does not touch them)
    tab = table.cuda()
    bounds.update(tab, n)
    step = tsa.PagedDecodeAttention(B, Hq, Hkv, 1, d)
    for _ in range(3):
        now = n.tolist()
        vals = pu.values(cache.pages, cache.scales)
        codes, exps = bounds.codes.cpu(), bounds.exponents.cpu()
        for b in range(B):
            for i in range(-(-now[b] // page)):
                c, e = cu.bounds(vals, table, page, b, now[b], i)
                assert torch.equal(codes[int(table[b, i])], c) and torch.equal(exps[int(table[b, i])], e)
        Q = rows(1, Hq)
        got, short = bounds.select(Q, tab, n, keep, sinks=1, recent=2)
        chosen, want_len = cu.select(Q.cpu(), codes, exps, table, page, now, keep, 1, 2)
        assert short.tolist() == want_len
        for b in range(B):
            for h in range(Hkv):
                assert got[b, h].tolist()[:len(chosen[b][h])] == table[b][torch.tensor(chosen[b][h])].tolist()
        pu.check_decode(*step(Q, cache, got, short), cu.decode_chosen(Q.cpu(), vals, table, page, now, chosen, d ** -0.5), d)
        n = n + 1
        cache.write(rows(1), rows(1), tab, n)
        bounds.update(tab, n, new_len=_int32([1] * B))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
