"""The operators for long contexts on the last pages of a large pool: offsets of keys and values beyond 2^32 bytes and 2^31
elements, of the bounds' codes beyond 2^31 (E4M3).  Each against its definition on those pages alone."""

import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

FAR = 80  # pages in use, the last of the pool


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _pool(store):
    """bf16: 4.6 GB of keys and values; E4M3: 36 GB, with 2.2 GB of codes of bounds and 1.1 GB of weights."""
    n_pages, page, d = (70000, 128, 128) if store == "bf16" else (17_500_000, 16, 64)
    dtype, scales = (torch.bfloat16, None) if store == "bf16" else (torch.uint8, torch.empty((n_pages, 1, page // 16, 2, 16), dtype=torch.uint8, device="cuda"))
    pages = torch.empty((n_pages, 1, 2, page, d), dtype=dtype, device="cuda")
    g = torch.Generator().manual_seed(51)
    x = torch.randn((FAR, 1, 2, page, d), generator=g)
    if store == "bf16":
        pages[-FAR:] = x.to(torch.bfloat16).cuda()
    else:
        codes, e = pu.quantise(x)
        pages[-FAR:] = codes.cuda()
        scales[-FAR:] = e.view(FAR, 1, 2, page // 16, 16).transpose(2, 3).contiguous().cuda()
        pages = pages.view(torch.float8_e4m3fn)
    return tsa.PagedCache(n_pages, 1, page, d, dtype=store, pages=pages, scales=scales), n_pages - FAR


def _values(cache):
    return pu.values(cache.pages[-FAR:], None if cache.scales is None else cache.scales[-FAR:])


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_last_pages_of_a_large_pool(store):
    cache, first = _pool(store)
    n_pages, _, page, d = cache.shape
    assert first * 2 * page * d * (2 if store == "bf16" else 1) > 2 ** 32
    order = torch.randperm(FAR, generator=torch.Generator().manual_seed(52)).to(torch.int32)
    table, other = order[:40].view(2, 20), order[40:].view(2, 20)  # local numbers
    tab, to = (table + first).cuda(), (other + first).cuda()
    lens, Hq, scale = [20 * page - 5, 11 * page + 1], 4, d ** -0.5
    n = _int32(lens)
    g = torch.Generator().manual_seed(53)
    Q = torch.randn((2, Hq, 1, d), generator=g).to(torch.bfloat16)
    vals = _values(cache)

    # ---- bounds, selection, attention over the chosen pages
    bounds = tsa.PageBounds(cache, codes=torch.empty((n_pages, 1, 2, d), dtype=torch.int8, device="cuda"),
                            exponents=torch.empty((n_pages, 1), dtype=torch.uint8, device="cuda"))
    assert store == "bf16" or first * 2 * d > 2 ** 31
    bounds.update(tab, n)
    codes, exps = bounds.codes[-FAR:].cpu(), bounds.exponents[-FAR:].cpu()
    for b in range(2):
        for i in range(-(-lens[b] // page)):
            c, e = cu.bounds(vals, table, page, b, lens[b], i)
            assert torch.equal(codes[int(table[b, i])], c) and torch.equal(exps[int(table[b, i])], e)
    got, short = bounds.select(Q.cuda(), tab, n, 6, 1, 2)
    chosen, want_len = cu.select(Q, codes, exps, table, page, lens, 6, 1, 2)
    assert short.tolist() == want_len
    for b in range(2):
        assert (got[b, 0].cpu() - first).tolist() == table[b][torch.tensor(chosen[b][0])].tolist()
    step = tsa.PagedDecodeAttention(2, Hq, 1, 1, d)
    pu.check_decode(*step(Q.cuda(), cache, got, short), cu.decode_chosen(Q, vals, table, page, lens, chosen, scale), d)

    # ---- the first sequence as the prefix of both: each attends to it, and to its own positions behind
    whole = torch.cat([table[:1, :19].expand(2, -1), table], dim=1)
    O, LSE = tsa.SharedPrefixAttention(2, Hq, 1, 1, d)(Q.cuda(), cache, tab[:1], _int32([19 * page]), tab, n)
    pu.check_decode(O, LSE, pu.decode(Q, vals, whole, page, [19 * page + x for x in lens], scale, 1, 0), d)

    # ---- weights
    weights = tsa.PageWeights(cache, torch.empty((n_pages, 1, page), device="cuda"))
    weights.weights[-FAR:] = torch.rand((FAR, 1, page), generator=g).cuda()
    before = weights.weights[-FAR:].cpu()
    O, LSE = step(Q.cuda(), cache, tab, n)
    weights.accumulate(Q.cuda(), LSE, tab, n, decay=0.5)
    want, err = cu.weigh(Q, LSE.cpu(), before, vals, table, page, lens, scale, 1, 0, 0.5)
    assert float(((weights.weights[-FAR:].cpu().double() - want).abs() - err).max()) <= 0

    # ---- eviction into other pages, then in place
    for src, dst, keep, recent in ((table, other, 9 * page + 3, page + 1), (other, None, 5 * page, 7)):
        vals, W = _values(cache), weights.weights[-FAR:].cpu()
        now = n.tolist()
        n, kept = weights.evict((src + first).cuda(), n, keep, recent, to_table=None if dst is None else (dst + first).cuda())
        dst = src if dst is None else dst
        after, W2 = _values(cache), weights.weights[-FAR:].cpu()
        for b, rows in enumerate(cu.evict(W, src, page, now, keep, recent)):
            j, i = torch.tensor(rows[0]), torch.arange(len(rows[0]))
            assert kept[b, 0].tolist() == rows[0] + [-1] * (keep + recent - len(rows[0])) and int(n[b]) == len(rows[0])
            p, q = src[b].long()[j // page], dst[b].long()[i // page]
            assert torch.equal(after[q, 0, :, i % page], vals[p, 0, :, j % page])
            assert torch.equal(W2[q, 0, i % page], W[p, 0, j % page])
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
