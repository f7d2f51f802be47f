"""Decode over shared prefixes, on the GPU against float64 definitions.

Slots behind a length and free pages hold NaN, and page-table entries that no position needs are out of range.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

FULL, CAUSAL = tsa.MASK_FULL, tsa.MASK_CAUSAL


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _join(x, y):
    """Softmax over two sets of keys from the results over each, as paged_util.decode gives them."""
    (o1, l1, a1, e1), (o2, l2, a2, e2) = x, y
    m = torch.maximum(l1, l2)
    base = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
    w1, w2 = torch.exp(l1 - base), torch.exp(l2 - base)
    s = w1 + w2
    d = torch.where(s == 0, torch.ones_like(s), s)
    w1, w2 = w1 / d, w2 / d
    return (o1 * w1[..., None] + o2 * w2[..., None], m + torch.log(s), a1 * w1[..., None] + a2 * w2[..., None],
            torch.maximum(e1, e2))


def _reference(Q, vals, ptab, plens, of, table, page, lens, scale, kind):
    B, Hq, S_q, d = Q.shape
    own = pu.decode(Q, vals, table, page, lens, scale, kind, 0)
    G = len(plens)
    rows = torch.tensor([g if 0 <= g < G else 0 for g in of])
    shared = pu.decode(Q, vals, ptab[rows], page, [plens[g] if 0 <= g < G else 0 for g in of], scale, 0, 0)
    return _join(shared, own)


def _make(plens, lens, Hkv, page, d, store, seed=0, **kw):
    pages, scales, tab, n = pu.make_pool(list(plens) + list(lens), Hkv, page, d, store, seed=seed, **kw)
    cache = tsa.PagedCache(n, Hkv, page, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    return cache, pu.values(pages, scales), tab[:len(plens)].contiguous(), tab[len(plens):].contiguous()


def _prefix(plens, lens, of, Hq, Hkv, S_q, d, page, store, kind=CAUSAL, grid=None, q_scale=1.0, k_scale=1.0, seed=0, reps=1,
            Q=None):
    cache, vals, ptab, table = _make(plens, lens, Hkv, page, d, store, seed, k_scale=k_scale)
    B = len(lens)
    g = torch.Generator().manual_seed(seed + 1)
    if Q is None:
        Q = (torch.randn((B, Hq, S_q, d), generator=g) * q_scale).to(torch.bfloat16)
    plan = tsa.SharedPrefixAttention(B, Hq, Hkv, S_q, d, kind=kind)
    if grid:
        plan.set_grid_limit(grid)
    outs = []
    for _ in range(reps):
        O = torch.full((B, Hq, S_q, d), math.nan, dtype=torch.bfloat16, device="cuda")
        LSE = torch.full((B, Hq, S_q), math.nan, device="cuda")
        plan(Q.cuda(), cache, ptab.cuda(), _int32(plens), table.cuda(), _int32(lens),
             prefix_of=None if of is None else _int32(of), O=O, LSE=LSE)
        outs.append((O, LSE))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    ref = _reference(Q, vals, ptab, plens, of or [0] * B, table, page, lens, 1 / math.sqrt(d), kind)
    for O, LSE in outs:
        pu.check_decode(O, LSE, ref, d)
        assert torch.equal(O, outs[0][0]) and torch.equal(LSE, outs[0][1])  # the same bits every call


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_prefix_lengths(store, d, page):
    for n in (1, 16, 127, 128, 129, 700):
        _prefix([n], [5, 1, 40], None, 8, 2, 1, d, page, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,S_q", [(1, 1, 1, 1), (2, 3, 1, 1), (3, 8, 8, 1), (16, 8, 1, 1), (17, 8, 1, 1), (5, 64, 1, 1),
                                          (40, 16, 2, 4), (7, 8, 8, 7), (33, 10, 1, 5)])
def test_row_counts(store, d, B, Hq, Hkv, S_q):
    """Rows of a prefix and kv head from one to several tiles of 128, tiles that a sequence's rows straddle."""
    _prefix([300], [(7 * b) % 60 + S_q for b in range(B)], None, Hq, Hkv, S_q, d, 16, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", [FULL, CAUSAL])
def test_groups_and_empty_parts(store, kind):
    """Several prefixes, one empty, one without sequences; sequences without a prefix, without positions of their own,
    without either, and with fewer of them than rows."""
    _prefix([200, 0, 77, 513], [0, 1, 2, 9, 0, 30, 150, 0, 4, 3], [0, 3, -1, 0, -1, 1, 3, 1, 3, 0], 6, 2, 3, 128, 32, store, kind)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("grid", [1, 2, 3, 7, 50, 304])
def test_grid_shares(store, grid):
    """Long shares over several units, and units cut between many CTAs; the same bits on every call."""
    _prefix([900, 1700], [30, 0, 400, 17, 5], [1, 0, 1, 1, 0], 40, 2, 1, 128, 16, store, grid=grid, reps=3)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_sharp_scores_move_the_reference(store):
    _prefix([3000], [77, 500], None, 8, 2, 1, 128, 64, store, q_scale=20.0, k_scale=2.0, grid=4)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_many_sequences_and_prefixes(store):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (300,), generator=g).tolist()
    plens = torch.randint(0, 90, (70,), generator=g).tolist()
    of = torch.randint(-1, 70, (300,), generator=g).tolist()
    _prefix(plens, lens, of, 4, 2, 1, 64, 16, store)


def test_as_many_prefixes_as_can_be():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 20, (1024,), generator=g).tolist()
    plens = torch.randint(0, 20, (1024,), generator=g).tolist()
    _prefix(plens, lens, torch.randperm(1024, generator=g).tolist(), 2, 1, 1, 64, 16, "bf16")
    _prefix([33], lens, None, 2, 1, 1, 64, 16, "e4m3")


def test_long_prefix():
    _prefix([20000], [100, 3], None, 16, 1, 1, 128, 128, "bf16")
    _prefix([20000], [100, 3], None, 16, 1, 1, 128, 128, "e4m3")


@pytest.mark.parametrize("page", [32, 80, 96, 128, 1024])
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_page_sizes(store, page):
    _prefix([1500], [3, 300], None, 8, 2, 1, 128, page, store)
    _prefix([77, 1025], [9, 200], [1, 1], 4, 2, 3, 64, page, store)


def test_one_sequence_is_a_decode_step():
    """Prefix and own positions together against the decode over one page table (pages that end with the prefix)."""
    page, n, m = 16, 320, 45
    cache, vals, ptab, table = _make([n], [m], 2, page, 128, "bf16")
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((1, 8, 1, 128), generator=g).to(torch.bfloat16).cuda()
    O, L = tsa.SharedPrefixAttention(1, 8, 2, 1, 128)(Q, cache, ptab.cuda(), _int32([n]), table.cuda(), _int32([m]))
    whole = torch.cat([ptab[:, :n // page], table[:, :3]], dim=1).contiguous().cuda()
    O2, L2 = tsa.PagedDecodeAttention(1, 8, 2, 1, 128)(Q, cache, whole, _int32([n + m]))
    # both are within 2^-8 (|O| + A) of the definition, A < 1.2 the mean of |v|
    assert float((O.double() - O2.double()).abs().max()) < 2.0 ** -7 * (float(O.abs().max()) + 1.2)
    assert float((L - L2).abs().max()) < 2.0 ** -12 + float(L.abs().max()) * 2.0 ** -21


def test_values_and_queries_that_are_not_finite():
    """A NaN in a value that all rows see, an infinity in a query: they stay with their sequences and heads."""
    cache, vals, ptab, table = _make([300, 100], [20, 20, 20], 2, 16, 64, "bf16")
    p = int(ptab[0, 3])
    cache.pages[p, 1, 1, 5, 9] = math.nan
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((3, 4, 1, 64), generator=g).to(torch.bfloat16)
    Q[2, 0, 0, 5] = math.inf
    O, L = tsa.SharedPrefixAttention(3, 4, 2, 1, 64)(Q.cuda(), cache, ptab.cuda(), _int32([300, 100]), table.cuda(),
                                                     _int32([20, 20, 20]), prefix_of=_int32([0, 1, 1]))
    O = O.cpu()
    assert O[0, 2:, 0, 9].isnan().all() and O[0, 2:].isfinite().sum() == 2 * 63
    assert O[0, :2].isfinite().all() and O[1].isfinite().all() and O[2, 1:].isfinite().all()
    assert O[2, 0].isnan().any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top", [100, 134, 135, 200])
def test_codes_and_exponents_of_all_kinds(d, top):
    """E4M3 prefixes of all codes, subnormal ones among them, with exponents up to `top` (one multiplication up to 134, two
    beyond), small keys and large values; then a NaN code beside a usual exponent, and a row of exponent 255."""
    page, n = 16, 200
    cache, vals, ptab, table = _make([n], [3, 9], 1, page, d, "e4m3")
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(0, 256, cache.pages.shape, generator=g).to(torch.uint8)
    codes = torch.where(codes & 0x7F == 0x7F, codes & 0x87, codes)
    exps = torch.randint(96, 112, cache.scales.shape, generator=g).to(torch.uint8)
    exps[:, :, :, 1] = torch.randint(top - 12, top + 1, exps[:, :, :, 1].shape, generator=g).to(torch.uint8)
    cache.pages.view(torch.uint8).copy_(codes.cuda())
    cache.scales.copy_(exps.cuda())
    Q = torch.randn((2, 4, 1, d), generator=g).to(torch.bfloat16)
    args = (Q.cuda(), cache, ptab.cuda(), _int32([n]), table.cuda(), _int32([3, 9]))
    plan = tsa.SharedPrefixAttention(2, 4, 1, 1, d)
    O, L = plan(*args)
    vals = pu.values(cache.pages, cache.scales)
    ref = _reference(Q, vals, ptab, [n], [0, 0], table, page, [3, 9], d ** -0.5, CAUSAL)
    # the own positions' weights: 2^-22 of the largest weight times the largest value factor, times codes up to 448
    coarse = torch.full((2, 4, 1), 128 * 448 * 2.0 ** -22 * 2.0 ** (top - 127), dtype=torch.float64)
    pu.check_decode(O, L, ref, d, more=coarse)
    cache.pages.view(torch.uint8)[int(ptab[0, 2]), 0, 1, 5, 7] = 0xFF
    O = plan(*args)[0].cpu()
    assert O[..., 7].isnan().all() and O.isfinite().sum() == O.numel() - 8
    cache.scales[int(ptab[0, 2]), 0, 0, 1, 6] = 255
    assert plan(*args)[0].isnan().all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("values", [[60, 130, 200, 90, 128], [200, 60, 61, 62, 63], [240, 1, 1, 1, 1], [1, 1, 1, 1, 240], [0, 0, 0, 0, 0]])
@pytest.mark.parametrize("grid", [None, 1])
def test_tiles_of_very_different_exponents(d, values, grid):
    """E4M3 prefixes whose tiles of 128 positions have value exponents far apart, keys' exponents spread within each tile, and
    queries from 2^-100 to 2^6: numbers are held in 16 bits relative to their row's or tile's exponent."""
    page, n, Hq = 16, 600, 8
    cache, _, ptab, table = _make([n], [0], 1, page, d, "e4m3")
    g = torch.Generator().manual_seed(21)
    codes = torch.randint(0, 256, cache.pages.shape, generator=g).to(torch.uint8)
    codes = torch.where(codes & 0x7F == 0x7F, codes & 0x87, codes)
    exps = torch.randint(100, 123, cache.scales.shape, generator=g).to(torch.uint8)  # (what is behind the end stays whatever)
    for j in range(n):
        exps[int(ptab[0, j // page]), :, j % page // 16, 1, j % 16] = max(0, values[j // 128] - j % 3)
    cache.pages.view(torch.uint8).copy_(codes.cuda())
    cache.scales.copy_(exps.cuda())
    Q = torch.randn((1, Hq, 1, d), generator=g) * 2.0 ** torch.tensor([-100, -40, -12, -4, -1, 0, 3, 6.0])[None, :, None, None]
    Q = Q.to(torch.bfloat16)
    plan = tsa.SharedPrefixAttention(1, Hq, 1, 1, d)
    if grid:
        plan.set_grid_limit(grid)
    O, L = plan(Q.cuda(), cache, ptab.cuda(), _int32([n]), table.cuda(), _int32([0]))
    vals = pu.values(cache.pages, cache.scales)
    ref = pu.decode(Q, vals, ptab, page, [n], d ** -0.5, FULL, 0)
    # A weight is an fp16 number relative to a reference M of weight times factor, at most twice 2^-7 of the largest of these:
    # half a step of the smallest is 2^-25, with a code of 448 off by 448 * 2^-31 of that largest, for each position.
    # Values below 2^-40 of the largest factor so far are off by half a step of theirs, 2^-25 - 7 - 40 of it.
    K, _ = pu.dense(vals, ptab, page, 0, n)
    p = torch.softmax(torch.einsum("hd,jd->hj", Q[0, :, 0].double(), K[0]) * d ** -0.5, -1)
    big, most = torch.zeros(Hq, dtype=torch.float64), 0.0
    for t in range(5):
        f = 2.0 ** (values[t] - 127)
        most = max(most, f)
        big = torch.maximum(big, p[:, 128 * t:128 * t + 128].amax(-1) * max(f, most * 2.0 ** -40))
    pu.check_decode(O, L, ref, d, more=(n * 448 * 2.0 ** -31 * big + most * 2.0 ** -72 + 2.0 ** -133)[None, :, None])
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("what", ["prefix length", "prefix page", "prefix number", "length", "page"])
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_numbers_that_are_not_followed(what, store):
    plens, lens, of = [300, 100], [20, 50], [0, 1]
    cache, vals, ptab, table = _make(plens, lens, 2, 16, 64, store)
    code = tsa.CACHE_ERR_PAGE if what.endswith("page") else tsa.CACHE_ERR_POSITION
    bad_p, bad_l, bad_of = list(plens), list(lens), list(of)
    if what == "prefix length":
        bad_p[0] = 16 * ptab.shape[1] + 1
    elif what == "length":
        bad_l[0] = -3
    elif what == "prefix number":
        bad_of[0] = 2
    elif what == "prefix page":
        ptab[0, 5] = -1
    else:
        table[0, 0] = 10 ** 6
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((2, 4, 1, 64), generator=g).to(torch.bfloat16)
    O, L = tsa.SharedPrefixAttention(2, 4, 2, 1, 64)(Q.cuda(), cache, ptab.cuda(), _int32(bad_p), table.cuda(), _int32(bad_l),
                                                     prefix_of=_int32(bad_of))
    assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, code)
    ref = _reference(Q, vals, ptab, plens, of, table, 16, lens, 0.125, CAUSAL)
    pu.check_decode(O[1:], L[1:], tuple(t[1:] for t in ref), 64)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_a_wait_that_runs_out(store):
    """A loading warp that stops: the step returns, the host learns of it, and the next step is right."""
    plens, lens = [5000], [40, 3]
    cache, vals, ptab, table = _make(plens, lens, 1, 16, 128, store)
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((2, 64, 1, 128), generator=g).to(torch.bfloat16)
    plan = tsa.SharedPrefixAttention(2, 64, 1, 1, 128)
    plan.set_grid_limit(2)
    args = (Q.cuda(), cache, ptab.cuda(), _int32(plens), table.cuda(), _int32(lens))
    plan.set_watchdog(20_000_000, 3)
    plan(*args)
    st, code = cache.poll_device_error()
    assert st == tsa.ATTN_ERR_DEVICE_TIMEOUT and code & tsa.CACHE_ERR_WAIT
    plan.set_watchdog(2_000_000_000, 0)
    O, L = plan(*args)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pu.check_decode(O, L, _reference(Q, vals, ptab, plens, [0, 0], table, 16, lens, 128 ** -0.5, CAUSAL), 128)
