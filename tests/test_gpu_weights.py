"""The attention weights of cached positions and eviction by them, against float64 and exact definitions."""
import math

import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

FULL, CAUSAL, WINDOW = tsa.MASK_FULL, tsa.MASK_CAUSAL, tsa.MASK_CAUSAL_SLIDING


def _cache(lens, Hkv, page, d, store, **kw):
    pages, scales, table, n = pu.make_pool(lens, Hkv, page, d, store, **kw)
    cache = tsa.PagedCache(n, Hkv, page, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    return cache, pu.values(pages, scales), table


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _weigh(lens, Hq, Hkv, S_q, d, page, store, kind=CAUSAL, window=0, decay=1.0, seed=0, scale=None, reps=1, q_scale=1.0,
           dead=()):
    first = [max(0, n - S_q - window) for n in lens] if kind == WINDOW and decay == 1.0 else None
    cache, vals, table = _cache(lens, Hkv, page, d, store, seed=seed, window_first=first)
    g = torch.Generator().manual_seed(seed + 1)
    B = len(lens)
    Q = (torch.randn((B, Hq, S_q, d), generator=g) * q_scale).to(torch.bfloat16)
    scale = scale or 1 / math.sqrt(d)
    LSE = pu.decode(Q, vals, table, page, lens, scale, kind, window)[1].float()
    for b, h, i in dead:
        LSE[b, h, i] = -math.inf
    W = torch.rand((cache.shape[0], Hkv, page), generator=g)
    for b, n in enumerate(lens):  # what new positions held before does not count
        for j in range(max(0, n - S_q), n):
            W[int(table[b, j // page]), :, j % page] = math.nan
    want, bound = W, None
    weights = tsa.PageWeights(cache, weights=W.cuda())
    for _ in range(reps):
        weights.accumulate(Q.cuda(), LSE.cuda(), table.cuda(), _int32(lens), scale=scale, kind=kind, window=window,
                           decay=decay)
        want, more = cu.weigh(Q, LSE, want, vals, table, page, lens, scale, kind, window, decay)
        bound = more if bound is None else bound * decay + more
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    got = weights.weights.cpu().double()
    bad = (got - want).abs() - bound
    assert float(bad.max()) <= 0, f"off by {float((got - want).abs().max()):.3e}, {float(bad.max()):.3e} past the bound"
    return got


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_lengths(store, d, page):
    _weigh([0, 1, 15, 16, 17, 31, 33, 127, 128, 900], 8, 2, 1, d, page, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,S_q", [(1, 1, 1), (3, 1, 1), (16, 1, 1), (17, 1, 1), (32, 1, 1), (16, 2, 4), (64, 1, 1),
                                        (8, 8, 7), (10, 1, 5)])
def test_row_counts(store, d, Hq, Hkv, S_q):
    _weigh([3, 70, 600], Hq, Hkv, S_q, d, 16, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,window", [(FULL, 0), (CAUSAL, 0), (WINDOW, 0), (WINDOW, 1), (WINDOW, 16), (WINDOW, 100),
                                         (WINDOW, 5000)])
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.0])
def test_masks_and_decay(store, kind, window, decay):
    """Among the lengths some shorter than S_q: rows that see nothing."""
    _weigh([0, 1, 2, 40, 129, 700], 6, 2, 3, 128, 32, store, kind, window, decay)


def test_released_pages_before_the_window():
    """Sequences whose first pages are gone, beside one whose page is the pool's first."""
    for seed in range(8):
        _weigh([255, 99, 128, 0, 17, 602, 1], 4, 4, 2, 64, 80, "bf16", kind=WINDOW, window=17, seed=seed)


def test_steps_add_up():
    _weigh([300, 20], 4, 2, 1, 64, 16, "bf16", decay=0.5, reps=1)
    a = _weigh([2000, 900, 30], 8, 2, 1, 128, 64, "bf16", seed=4)
    assert torch.equal(a, _weigh([2000, 900, 30], 8, 2, 1, 128, 64, "bf16", seed=4))  # the same bits every call


def test_weights_of_a_step_sum_to_its_rows():
    lens = [1777, 300]
    cache, vals, table = _cache(lens, 2, 64, 128, "bf16")
    g = torch.Generator().manual_seed(1)
    Q = torch.randn((2, 12, 2, 128), generator=g).to(torch.bfloat16).cuda()
    tab, ln = table.cuda(), _int32(lens)
    O, LSE = tsa.PagedDecodeAttention(2, 12, 2, 2, 128)(Q, cache, tab, ln)
    weights = tsa.PageWeights(cache)
    weights.accumulate(Q, LSE, tab, ln)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        w = weights.weights.cpu().double()[table[b].long()[j // 64], :, j % 64].sum(0)
        # 12 rows to a head; weights are off by E (d + 8) 2^-23 + 2^-19 at most (paged_util.check_decode), and
        # E = scale |q| . |k| is below 15 for 128 normal elements: 2^-12
        assert float((w - 12).abs().max()) < 12 * 2.0 ** -12


def test_rows_without_weight_and_sharp_scores():
    _weigh([200, 50], 8, 2, 2, 64, 16, "bf16", dead=[(0, 0, 0), (0, 1, 1), (0, 7, 0), (1, 3, 1)])
    _weigh([200, 50], 32, 1, 1, 64, 16, "e4m3", dead=[(0, i, 0) for i in range(32)])
    _weigh([3000, 77], 8, 2, 1, 128, 64, "bf16", q_scale=20.0)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    _weigh(torch.randint(0, 90, (300,), generator=g).tolist(), 4, 2, 1, 64, 16, "e4m3")


def test_long_sequence():
    _weigh([20000], 8, 1, 1, 128, 128, "bf16")
    _weigh([20000], 8, 1, 1, 128, 128, "e4m3")


def _evict(lens, Hkv, page, d, store, keep, recent, in_place, seed=0, make=None):
    cache, vals, table = _cache(lens, Hkv, page, d, store, seed=seed, spare=2 + sum(-(-min(n, keep + recent) // page) for n in lens))
    g = torch.Generator().manual_seed(seed + 5)
    n_pages = cache.shape[0]
    W = torch.rand((n_pages, Hkv, page), generator=g)
    W[torch.rand(W.shape, generator=g) < 0.3] = 0.25
    W[torch.rand(W.shape, generator=g) < 0.2] = 0.0
    if make:
        make(W, table)
    to = None
    if not in_place:
        used = {int(table[b, i]) for b, n in enumerate(lens) for i in range(-(-n // page))}
        free = [p for p in torch.randperm(n_pages, generator=g).tolist() if p not in used]
        to = torch.full((len(lens), max(1, -(-min(keep + recent, table.shape[1] * page) // page))), 2 ** 30, dtype=torch.int32)
        for b, n in enumerate(lens):
            for i in range(-(-min(n, keep + recent) // page)):
                to[b, i] = free.pop()
    before = [cache.pages.view(torch.uint8).cpu().clone(), None if cache.scales is None else cache.scales.cpu().clone()]
    weights = tsa.PageWeights(cache, weights=W.cuda())
    length, kept = weights.evict(table.cuda(), _int32(lens), keep, recent, to_table=None if to is None else to.cuda())
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    want = cu.evict(W, table, page, lens, keep, recent)
    pages, scales, Wn = before[0].clone(), None if before[1] is None else before[1].clone(), W.clone()
    where = table if to is None else to
    for b, n in enumerate(lens):
        for h in range(Hkv):
            j = torch.tensor(want[b][h], dtype=torch.long)
            i = torch.arange(len(j))
            row = torch.full((keep + recent,), -1, dtype=torch.int32)
            row[:len(j)] = j.int()
            assert torch.equal(kept[b, h].cpu(), row)
            sp, ss, dp, ds = table[b].long()[j // page], j % page, where[b].long()[i // page], i % page
            pages[dp, h, :, ds] = before[0][sp, h, :, ss]
            Wn[dp, h, ds] = W[sp, h, ss]
            if scales is not None:
                scales[dp, h, ds // 16, :, ds % 16] = before[1][sp, h, ss // 16, :, ss % 16]
    assert length.tolist() == [min(n, keep + recent) for n in lens]
    assert torch.equal(cache.pages.view(torch.uint8).cpu(), pages)
    assert torch.equal(weights.weights.cpu().view(torch.int32), Wn.view(torch.int32))
    if scales is not None:
        assert torch.equal(cache.scales.cpu(), scales)
    return kept


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48])
def test_eviction_of_ragged_lengths(store, d, page, in_place):
    _evict([0, 1, 16, 39, 40, 41, 100, 333, 1000], 3, page, d, store, 30, 10, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,recent", [(1, 0), (0, 1), (0, 50), (50, 0), (299, 0), (150, 149), (1, 298), (700, 13)])
def test_shares_that_stay(keep, recent, in_place):
    _evict([300, 299, 1], 2, 16, 64, "bf16", keep, recent, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_weights_that_are_equal_or_not_finite(in_place):
    def equal(W, table):
        W.fill_(0.5)

    def odd(W, table):
        g = torch.Generator().manual_seed(3)
        r = torch.rand(W.shape, generator=g)
        W[r < 0.1] = math.inf
        W[r > 0.97] = math.nan
        W[(r > 0.5) & (r < 0.6)] = -0.0
        W[(r > 0.6) & (r < 0.7)] = -1.5
        W[(r > 0.7) & (r < 0.72)] = -math.inf
        W[(r > 0.72) & (r < 0.74)] = 1e-42

    _evict([500, 90], 2, 16, 64, "bf16", 60, 7, in_place, make=equal)
    for keep in (20, 200, 450):
        _evict([500, 90], 2, 16, 64, "e4m3", keep, 7, in_place, make=odd)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("store,d", [("bf16", 128), ("e4m3", 64)])
def test_eviction_of_many_heads(store, d, in_place):
    """More heads than blocks that run at once."""
    _evict([(37 * b) % 90 for b in range(180)], 2, 16, d, store, 30, 11, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_of_a_long_sequence(in_place):
    """More weights than fit in shared memory, and several rounds of a block in place."""
    _evict([50000, 9000], 1, 128, 64, "bf16", 4000, 500, in_place)


def test_eviction_again_and_again_in_place():
    """A cache of bounded length: after each step the sequences are cut down to what stays."""
    page, Hkv, d, budget = 16, 2, 64, 40
    cache = tsa.PagedCache(8, Hkv, page, d)
    weights = tsa.PageWeights(cache)
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    step = tsa.PagedDecodeAttention(2, 4, Hkv, 1, d)
    held = [[[] for _ in range(Hkv)] for _ in range(2)]  # (key, value, weight) of each position
    for t in range(70):
        x = torch.randn((3, 2, 4, 1, d), generator=g).to(torch.bfloat16)
        K, V, Q = x[0, :, :Hkv], x[1, :, :Hkv], x[2]
        lens = lens + 1
        cache.write(K.cuda(), V.cuda(), table, lens)
        O, LSE = step(Q.cuda(), cache, table, lens)
        weights.accumulate(Q.cuda(), LSE, table, lens)
        for b in range(2):
            for h in range(Hkv):
                mine = held[b][h]
                mine.append([K[b, h, 0], V[b, h, 0], 0.0])
                k = torch.stack([m[0] for m in mine]).double()
                v = torch.stack([m[1] for m in mine]).double()
                p = torch.softmax(Q[b, 2 * h:2 * h + 2, 0].double() @ k.T / math.sqrt(d), -1)
                # the roundings of O and of the weights, and 2^-13 for the scores (E (d + 8) 2^-23 with E below 14)
                bound = (p @ v).abs() * 2.0 ** -8 + p @ v.abs() * (2.0 ** -8 + 2.0 ** -12)
                assert bool(((O[b, 2 * h:2 * h + 2, 0].cpu().double() - p @ v).abs() <= bound).all())
                for m, w in zip(mine, p.sum(0).tolist()):
                    m[2] += w
        lens, kept = weights.evict(table, lens, budget - 8, 8)
        for b in range(2):
            for h in range(Hkv):
                j = [i for i in kept[b, h].tolist() if i >= 0]
                if len(held[b][h]) > budget:
                    old = held[b][h][:-8]
                    assert j[-8:] == list(range(len(old), len(old) + 8))
                    # the one that goes is the lightest, up to the weights' errors (2^-13 of each)
                    gone = [m[2] for i, m in enumerate(old) if i not in j]
                    assert max(gone) <= min(old[i][2] for i in j[:-8]) * (1 + 2.0 ** -12)
                held[b][h] = [held[b][h][i] for i in j]
        assert int(lens.max()) <= budget
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("what", ["length", "negative", "page"])
def test_lengths_and_pages_that_are_not_followed(what):
    lens = [100, 200]
    cache, vals, table = _cache(lens, 2, 16, 64, "bf16", spare=20)
    code = tsa.CACHE_ERR_PAGE if what == "page" else tsa.CACHE_ERR_POSITION
    bad = list(lens)
    if what == "page":
        table[0, 2] = -5
    else:
        bad[0] = 16 * table.shape[1] + 1 if what == "length" else -1
    weights = tsa.PageWeights(cache)
    before = cache.pages.clone()
    Q = torch.ones((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    weights.accumulate(Q, torch.zeros((2, 4, 1), device="cuda"), table.cuda(), _int32(bad))
    assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, code)
    for to in (None, torch.full((2, 4), 10 ** 6, dtype=torch.int32).cuda()):
        length, kept = weights.evict(table.cuda(), _int32(bad), 30, 5, to_table=to)
        st, got = cache.poll_device_error()
        assert st == tsa.ATTN_ERR_INVALID_ARG and got & code
        assert length.tolist() == [35 if what == "page" else 0, 35]
        if what != "page":
            assert kept[0].eq(-1).all()
    # what belongs to nobody is as it was
    used = {int(table[b, i]) for b, n in enumerate(lens) for i in range(-(-n // 16))}
    free = [p for p in range(cache.shape[0]) if p not in used]
    assert torch.equal(cache.pages[free].view(torch.int16), before[free].view(torch.int16))
