"""Bounds of pages' keys, the selection by them and attention over the selected pages, against definitions in whole
numbers and float64.

Slots behind a length and free pages hold NaN, and page-table entries that no position needs are out of range.
"""
import math

import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


def _cache(lens, Hkv, page, d, store, **kw):
    pages, scales, table, n = pu.make_pool(lens, Hkv, page, d, store, **kw)
    cache = tsa.PagedCache(n, Hkv, page, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    return cache, pu.values(pages, scales), table


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _check_bounds(bounds, vals, table, page, lens, news, before):
    codes, exps = before[0].clone(), before[1].clone()
    for b, n in enumerate(lens):
        fresh = min(n, news[b])
        if fresh <= 0:
            continue
        for i in range((n - fresh) // page, -(-n // page)):
            codes[int(table[b, i])], exps[int(table[b, i])] = cu.bounds(vals, table, page, b, n, i)
    assert torch.equal(bounds.exponents.cpu(), exps)
    assert torch.equal(bounds.codes.cpu(), codes)


def _marked(cache):
    bounds = tsa.PageBounds(cache)
    bounds.codes.fill_(55)
    bounds.exponents.fill_(77)
    return bounds, (bounds.codes.cpu(), bounds.exponents.cpu())


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_bounds_of_ragged_lengths(store, d, page):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 300, 700]
    cache, vals, table = _cache(lens, 3, page, d, store)
    for news in (None, [0, 1, 1, 4, 1, 1, 1, 2, 300, 129], [5, 0, 99, 0, -3, 63, 0, 0, 20, 701]):
        bounds, before = _marked(cache)
        bounds.update(table.cuda(), _int32(lens), None if news is None else _int32(news))
        assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
        _check_bounds(bounds, vals, table, page, lens, news or lens, before)


def test_bounds_of_many_sequences():
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 60, (600,), generator=g).tolist()
    cache, vals, table = _cache(lens, 2, 16, 64, "bf16")
    news = torch.randint(0, 20, (600,), generator=g).tolist()
    bounds, before = _marked(cache)
    bounds.update(table.cuda(), _int32(lens), _int32(news))
    _check_bounds(bounds, vals, table, 16, lens, news, before)


def test_bounds_of_extreme_keys():
    """Zeros, magnitudes at the limits of 127 * 2^k, the smallest and the largest bf16 numbers, infinities and NaN."""
    page, d = 16, 64
    pages = torch.zeros((9, 1, 2, page, d))
    pages[1, 0, 0, 3, 5] = 127.0
    pages[2, 0, 0, 3, 5] = -127.5  # above 127 by half a step of bf16: the next power
    pages[3, 0, 0, 0, 0] = 2.0 ** -133
    pages[4, 0, 0, 15, 63] = -3.3895313892515355e38
    pages[4, 0, 0, 14, 62] = 1.0
    pages[5, 0, 0, 2, 2] = math.inf
    pages[6, 0, 0, 2, 2] = math.nan
    pages[7, 0, 0, :, 1] = -2.0
    pages[8, 0, 0, 1, 1] = -math.inf
    cache = tsa.PagedCache(9, 1, page, d, pages=pages.to(torch.bfloat16).cuda())
    vals = pu.values(cache.pages, None)
    table = torch.arange(9, dtype=torch.int32)[None]
    bounds, before = _marked(cache)
    bounds.update(table.cuda(), _int32([9 * page]))
    _check_bounds(bounds, vals, table, page, [9 * page], [9 * page], before)
    assert bounds.exponents.cpu()[[5, 6, 8]].tolist() == [[255]] * 3


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,pages", [(16, 4), (64, 3), (144, 40)])
def test_bounds_of_rows_of_very_different_sizes(d, page, pages):
    """E4M3 rows whose exponents lie far apart, up to 14 apart and 15 apart; rows of zeros; a NaN code beside a usual
    exponent; few pages (a block each) and many (a warp each)."""
    g = torch.Generator().manual_seed(4)
    n = pages * page
    x = torch.randn((pages, 3, 2, page, d), generator=g)
    x[:, 0] *= torch.exp2(torch.randint(-60, 60, (pages, 2, page, 1), generator=g).float())
    x[:, 1] *= torch.exp2(torch.randint(0, 15, (pages, 2, page, 1), generator=g).float())
    x[:, 2, :, 3] = 0
    codes, e = pu.quantise(x)
    codes[0, 1, 0, 2, 5] = 0x7F
    codes[1, 0, 0, 3, 1] = 0xFF
    e[2, 1, 0, :9] = torch.tensor([100, 114, 113, 101, 107, 100, 114, 109, 110], dtype=torch.uint8)
    e[2, 1, 0, 9:] = 105
    e[2, 2, 0, :] = 90
    e[2, 2, 0, 4] = 105
    e[1, 2, 1, 7] = 255  # (a value's: no matter)
    cache = tsa.PagedCache(pages, 3, page, d, dtype="e4m3", pages=codes.view(torch.float8_e4m3fn).cuda(),
                           scales=e.view(pages, 3, 2, page // 16, 16).transpose(2, 3).contiguous().cuda())
    vals = pu.values(cache.pages, cache.scales)
    table = torch.arange(pages, dtype=torch.int32)[None]
    bounds, before = _marked(cache)
    bounds.update(table.cuda(), _int32([n - 1]))
    _check_bounds(bounds, vals, table, page, [n - 1], [n - 1], before)
    assert int(bounds.exponents[0, 1]) == 255 and int(bounds.exponents[1, 0]) == 255


def _sparse(lens, Hq, Hkv, S_q, d, page, store, keep, sinks, recent, seed=0, poke=None, q_scale=1.0):
    cache, vals, table = _cache(lens, Hkv, page, d, store, seed=seed)
    if poke:
        poke(cache, table)
        vals = pu.values(cache.pages, cache.scales)
    B = len(lens)
    g = torch.Generator().manual_seed(seed + 1)
    Q = (torch.randn((B, Hq, S_q, d), generator=g) * q_scale).to(torch.bfloat16)
    bounds = tsa.PageBounds(cache)
    tab, ln = table.cuda(), _int32(lens)
    bounds.update(tab, ln)
    got, short = bounds.select(Q.cuda(), tab, ln, keep, sinks, recent)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    chosen, want_len = cu.select(Q, bounds.codes.cpu(), bounds.exponents.cpu(), table, page, lens, keep, sinks, recent)
    want = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(Hkv):
            c = torch.tensor(chosen[b][h], dtype=torch.long)
            want[b, h, :len(c)] = table[b][c]
    assert short.tolist() == want_len
    assert torch.equal(got.cpu(), want)
    return cache, vals, table, Q, got, short, chosen


def _attend(lens, Hq, Hkv, S_q, d, page, store, keep, sinks=1, recent=2, **kw):
    cache, vals, table, Q, got, short, chosen = _sparse(lens, Hq, Hkv, S_q, d, page, store, keep, sinks, recent, **kw)
    O, LSE = tsa.PagedDecodeAttention(len(lens), Hq, Hkv, S_q, d)(Q.cuda(), cache, got, short)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pu.check_decode(O, LSE, cu.decode_chosen(Q, vals, table, page, lens, chosen, 1 / math.sqrt(d)), d)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_lengths(store, d, page):
    _attend([0, 1, 17, 3 * page, 4 * page, 4 * page + 1, 5 * page - 1, 1500, 2900], 8, 2, 1, d, page, store, 4)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,S_q", [(1, 1, 1), (3, 1, 1), (16, 2, 4), (64, 1, 1), (8, 8, 7), (10, 1, 5)])
def test_row_counts(store, Hq, Hkv, S_q):
    _attend([700, 40, 3], Hq, Hkv, S_q, 128, 16, store, 9)


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 1), (3, 2, 1), (3, 0, 3), (7, 0, 2), (30, 5, 1), (200, 0, 1)])
def test_shares_of_the_selection(keep, sinks, recent):
    """Nothing left to choose, nothing to keep first, and more than there is."""
    _attend([1000, 555, 96, 16], 4, 2, 1, 64, 16, "bf16", keep, sinks, recent)


@pytest.mark.parametrize("pages,Hkv", [(129, 1), (1000, 2), (5000, 1)])
def test_clusters_of_blocks(pages, Hkv):
    """Few sequences of many pages: up to eight blocks share a head's scores."""
    _sparse([pages * 16 - 3], 4 * Hkv, Hkv, 1, 64, 16, "bf16", 100, 1, 2)


def test_equal_scores_go_to_the_first_pages():
    def poke(cache, table):  # the keys of all full pages alike
        cache.pages[:, :, 0] = cache.pages[int(table[0, 3]), :, 0].clone()

    *_, chosen = _sparse([50 * 16], 8, 2, 1, 64, 16, "bf16", 10, 2, 1, poke=poke)
    assert chosen[0][0] == list(range(9)) + [49]


def test_pages_and_queries_that_are_not_finite():
    def poke(cache, table):
        cache.pages[int(table[0, 20]), 0, 0, 3, 7] = math.inf
        cache.pages[int(table[0, 30]), 1, 0, 3, 7] = math.nan

    *_, chosen = _sparse([50 * 16], 8, 2, 1, 64, 16, "bf16", 4, 1, 1, poke=poke)
    assert 20 in chosen[0][0] and 30 in chosen[0][1]
    cache, _, table, Q, *_ = _sparse([50 * 16], 8, 2, 1, 64, 16, "bf16", 6, 1, 1)
    bounds = tsa.PageBounds(cache)
    tab, ln = table.cuda(), _int32([50 * 16])
    bounds.update(tab, ln)
    for bad in (math.inf, -math.inf, math.nan):
        Qb = Q.clone()
        Qb[0, 1, 0, 3] = bad
        got, _ = bounds.select(Qb.cuda(), tab, ln, 6, 1, 1)
        assert got[0, 0].tolist() == table[0][[0, 1, 2, 3, 4, 49]].tolist()


def test_all_queries_zero_and_far_powers():
    _sparse([900], 4, 1, 1, 128, 16, "bf16", 12, 1, 1, q_scale=0.0)
    _sparse([900], 4, 1, 1, 128, 16, "bf16", 12, 1, 1, q_scale=2.0 ** 120)
    _sparse([900], 4, 1, 1, 128, 16, "bf16", 12, 1, 1, q_scale=2.0 ** -120)


def test_the_score_bounds_every_product():
    """No rounded query's product with a key of a page exceeds the page's score."""
    cache, vals, table, Q, *_ = _sparse([640], 4, 1, 1, 64, 16, "e4m3", 5, 1, 1)
    bounds = tsa.PageBounds(cache)
    bounds.update(table.cuda(), _int32([640]))
    c, e = bounds.codes.cpu().double(), bounds.exponents.cpu().double()
    q = Q[0, :, 0].double()
    q = torch.round(q * 2.0 ** -cu.power(float(q.abs().max())))
    for i in range(40):
        g = int(table[0, i])
        score = torch.maximum(q * c[g, 0, 0], q * c[g, 0, 1]).sum(-1).max() * 2.0 ** (e[g, 0] - 127)
        assert float((q @ vals[g, 0, 0].T).max()) <= float(score)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_a_table_for_each_head(store):
    """The decode over tables that differ from head to head, rows with strides of their own."""
    lens, page, d, Hq, Hkv = [500, 0, 77], 32, 64, 6, 3
    cache, vals, table = _cache(lens, Hkv, page, d, store)
    chosen = [[sorted(range(-(-n // page)), key=lambda i: (i * 7 + h) % 16) for h in range(Hkv)] for n in lens]
    for b, n in enumerate(lens):  # any order, but the last page stays last: it is not full
        for h in range(Hkv):
            last = -(-n // page) - 1
            chosen[b][h] = [i for i in chosen[b][h] if i != last] + ([last] if n else [])
    tab = torch.full((3, Hkv + 2, 20), 2 ** 30, dtype=torch.int32)
    for b in range(3):
        for h in range(Hkv):
            c = torch.tensor(chosen[b][h], dtype=torch.long)
            tab[b, h + 1, :len(c)] = table[b][c]
    g = torch.Generator().manual_seed(1)
    Q = torch.randn((3, Hq, 1, d), generator=g).to(torch.bfloat16)
    O, LSE = tsa.PagedDecodeAttention(3, Hq, Hkv, 1, d)(Q.cuda(), cache, tab.cuda()[:, 1:-1], _int32(lens))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pu.check_decode(O, LSE, cu.decode_chosen(Q, vals, table, page, lens, chosen, 1 / math.sqrt(d)), d)


@pytest.mark.parametrize("what", ["length", "negative", "page"])
def test_lengths_and_pages_that_are_not_followed(what):
    lens = [100, 900]
    cache, vals, table = _cache(lens, 2, 16, 64, "bf16")
    code = tsa.CACHE_ERR_PAGE if what == "page" else tsa.CACHE_ERR_POSITION
    bad = list(lens)
    if what == "page":
        table[0, 2] = 10 ** 6
    else:
        bad[0] = 16 * table.shape[1] + 1 if what == "length" else -1
    Q = torch.ones((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    bounds, before = _marked(cache)
    bounds.update(table.cuda(), _int32(bad))
    assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, code)
    got, short = bounds.select(Q, table.cuda(), _int32(bad), 5)
    assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, code)
    if what != "page":
        assert got[0].eq(-1).all() and int(short[0]) == 0
    # the other sequence's bounds are right
    for i in range(57):
        g = int(table[1, i])
        codes, exps = cu.bounds(vals, table, 16, 1, 900, i)
        assert torch.equal(bounds.codes[g].cpu(), codes) and torch.equal(bounds.exponents[g].cpu(), exps)


def test_far_pages_of_a_large_pool():
    """Offsets of codes and pages beyond 32 bits."""
    n_pages, page, d = 70000, 128, 128  # 70000 * 128 * 128 * 2 * 2 bytes: 4.6 GB; codes 18 MB
    cache = tsa.PagedCache(n_pages, 1, page, d)
    far = torch.arange(n_pages - 40, n_pages, dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((40, 1, 2, page, d), generator=g).to(torch.bfloat16)
    cache.pages[n_pages - 40:] = x.cuda()
    bounds, _ = _marked(cache)
    n = 40 * page - 5
    bounds.update(far[None].cuda(), _int32([n]))
    vals = pu.values(x, None)
    local = torch.arange(40, dtype=torch.int32)[None]
    for i in range(40):
        codes, exps = cu.bounds(vals, local, page, 0, n, i)
        assert torch.equal(bounds.codes[n_pages - 40 + i].cpu(), codes)
        assert torch.equal(bounds.exponents[n_pages - 40 + i].cpu(), exps)
