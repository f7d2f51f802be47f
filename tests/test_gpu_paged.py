"""The paged cache and decode attention over it, on the GPU against float64 definitions.

Slots behind a length, free pages and pages a window has released hold NaN, and page-table entries that no position
needs are out of range: a kernel that uses one shows it.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

FULL, CAUSAL, WINDOW = tsa.MASK_FULL, tsa.MASK_CAUSAL, tsa.MASK_CAUSAL_SLIDING


def _cache(lens, Hkv, page, d, store, **kw):
    pages, scales, table, n = pu.make_pool(lens, Hkv, page, d, store, **kw)
    vals = pu.values(pages, scales)
    cache = tsa.PagedCache(n, Hkv, page, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    return cache, vals, table


def _decode(lens, Hq, Hkv, S_q, d, page, store, kind=CAUSAL, window=0, grid=None, q_scale=1.0, k_scale=1.0, seed=0,
            reps=1):
    first = [max(0, n - S_q - window) for n in lens] if kind == WINDOW else None
    cache, vals, table = _cache(lens, Hkv, page, d, store, seed=seed, window_first=first, k_scale=k_scale)
    g = torch.Generator().manual_seed(seed + 1)
    Q = (torch.randn((len(lens), Hq, S_q, d), generator=g) * q_scale).to(torch.bfloat16).cuda()
    plan = tsa.PagedDecodeAttention(len(lens), Hq, Hkv, S_q, d, kind=kind, window=window)
    if grid:
        plan.set_grid_limit(grid)
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    outs = []
    for _ in range(reps):
        O = torch.full_like(Q, math.nan)
        LSE = torch.full((len(lens), Hq, S_q), math.nan, device="cuda")
        plan(Q, cache, tab, ln, O=O, LSE=LSE)
        outs.append((O, LSE))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    ref = pu.decode(Q, vals, table, page, lens, 1 / math.sqrt(d), kind, window)
    for O, LSE in outs:
        pu.check_decode(O, LSE, ref, d)
        assert torch.equal(O, outs[0][0]) and torch.equal(LSE, outs[0][1])  # the same bits every call


RAGGED = [0, 1, 15, 16, 17, 31, 33, 64, 127, 500]


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_ragged_lengths(store, d, page):
    _decode(RAGGED, 8, 2, 1, d, page, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,S_q", [(1, 1, 1), (3, 1, 1), (8, 8, 1), (17, 1, 1), (32, 1, 1), (16, 2, 4), (64, 1, 1),
                                        (8, 8, 7), (12, 2, 5), (10, 1, 5)])
def test_row_counts(store, d, Hq, Hkv, S_q):
    """1 to 64 rows share a kv head: one, two and four warps to a ring."""
    _decode([3, 70, 260], Hq, Hkv, S_q, d, 16, store)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,window", [(FULL, 0), (WINDOW, 0), (WINDOW, 1), (WINDOW, 15), (WINDOW, 16), (WINDOW, 100),
                                         (WINDOW, 5000)])
@pytest.mark.parametrize("S_q", [1, 3])
def test_masks(store, kind, window, S_q):
    """Among the lengths some shorter than S_q: rows that see nothing."""
    _decode([0, 1, 2, 40, 129, 700], 6, 2, S_q, 128, 32, store, kind, window)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("grid", [1, 2, 3, 7, 50, 152])
@pytest.mark.parametrize("Hq,Hkv", [(8, 4), (40, 2)])
def test_grid_shares(store, grid, Hq, Hkv):
    """Long shares over several units, and units cut between many CTAs; the same bits on every call."""
    _decode([900, 0, 30, 1700], Hq, Hkv, 1, 128, 16, store, grid=grid, reps=3)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_sharp_scores_move_the_maximum(store):
    _decode([3000, 77], 8, 2, 1, 128, 64, store, q_scale=20.0, k_scale=2.0, grid=4)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_many_sequences(store):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    _decode(lens, 4, 2, 1, 64, 16, store)


def test_long_sequence():
    _decode([20000], 8, 1, 1, 128, 128, "bf16")
    _decode([20000], 8, 1, 1, 128, 128, "e4m3")


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [32, 80, 96, 128, 256, 1024])
def test_page_sizes(store, page):
    """Boxes of 16 to 128 positions, pages inside a tile, of a tile and of many."""
    _decode([1, 300, 1500], 8, 2, 1, 128, page, store)
    _decode([77, 513], 4, 2, 3, 64, page, store, WINDOW, 200)


@pytest.mark.parametrize("rows", [4, 16, 32, 64])
def test_spread_value_factors_and_a_dominant_key(rows):
    """Value rows of very different sizes, and one key that takes most of the weight: the small weights behind it must
    not be lost (both rounding terms of the E4M3 weights)."""
    lens, page, d = [1700, 257], 64, 128
    pages, scales, table, n = pu.make_pool(lens, 1, page, d, "e4m3", seed=9, v_spread=2.0)
    factors = torch.exp2(scales.transpose(2, 3).reshape(n, 1, 2, page).double() - 127)
    factors[scales.transpose(2, 3).reshape(n, 1, 2, page) == 255] = 0
    g = torch.Generator().manual_seed(3)
    Q = torch.randn((2, rows, 1, d), generator=g).to(torch.bfloat16)
    vals = pu.values(pages, scales)
    for b in range(2):  # position 5 of each sequence: a key along the first query
        k = (Q[b, 0, 0].float() * 0.9)[None]
        codes, e = pu.quantise(k)
        p = int(table[b, 0])
        pages.view(torch.uint8)[p, :, 0, 5] = codes
        scales[p, :, 0, 0, 5] = e
    vals = pu.values(pages, scales)
    cache = tsa.PagedCache(n, 1, page, d, dtype="e4m3", pages=pages.cuda(), scales=scales.cuda())
    O, LSE = tsa.PagedDecodeAttention(2, rows, 1, 1, d)(Q.cuda(), cache, table.cuda(),
                                                        torch.tensor(lens, dtype=torch.int32).cuda())
    scale = 1 / math.sqrt(d)
    more = pu.coarse_weights(Q, vals, factors, table, page, lens, scale)
    pu.check_decode(O, LSE, pu.decode(Q, vals, table, page, lens, scale, CAUSAL, 0), d, more)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_query_that_is_not_finite_stays_in_its_row(store, bad):
    lens = [300, 20]
    cache, vals, table = _cache(lens, 2, 16, 64, store, seed=2)
    Q = torch.randn((2, 6, 2, 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    plan = tsa.PagedDecodeAttention(2, 6, 2, 2, 64)
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want = plan(Q.cuda(), cache, tab, ln)
    Q[0, 4, 1, 7] = bad
    O, LSE = plan(Q.cuda(), cache, tab, ln)
    keep = torch.ones((2, 6, 2), dtype=torch.bool)
    keep[0, 4, 1] = False
    assert torch.equal(O.cpu()[keep], want[0].cpu()[keep]) and torch.equal(LSE.cpu()[keep], want[1].cpu()[keep])
    assert not bool(torch.isfinite(O[0, 4, 1].float()).any())


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(store):
    """A pool of more than 4 GiB whose sequence sits at its end."""
    d, Hkv, page = 128, 4, 64
    row = 2 * d if store == "bf16" else d
    n = (4 << 30) // (Hkv * 2 * page * row) + 50
    cache = tsa.PagedCache(n, Hkv, page, d, dtype=store)
    assert cache.pages.numel() * cache.pages.element_size() > 2 ** 32
    lens = [100, 90]
    table = torch.tensor([[n - 1, n - 4], [n - 2, 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    K, V = (torch.randn((2, Hkv, 100, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    cache.write(K, V, tab, ln, new_len=ln)
    Kd, Vd = cache.read(tab, ln, length=100)
    if store == "bf16":
        assert torch.equal(Kd[0], K[0]) and torch.equal(Vd[1, :, :90], V[1, :, :90])
    used = sorted(set(table.flatten().tolist()))
    small = {p: i for i, p in enumerate(used)}
    pages = cache.pages.view(torch.uint8)[used].cpu().view(cache.pages.dtype)
    vals = pu.values(pages, None if cache.scales is None else cache.scales[used])
    local = torch.tensor([[small[int(p)] for p in r] for r in table], dtype=torch.int32)
    Q = torch.randn((2, 8, 1, d), generator=g).to(torch.bfloat16).cuda()
    O, LSE = tsa.PagedDecodeAttention(2, 8, Hkv, 1, d)(Q, cache, tab, ln)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pu.check_decode(O, LSE, pu.decode(Q, vals, local, page, lens, 1 / math.sqrt(d), CAUSAL, 0), d)


def test_every_code_is_read_exactly():
    """One position, so O is its value row and each of the 256 codes and many exponents come through to bf16."""
    d = 128
    for exponents in ([127] * 4, [100, 130, 90, 160]):
        pages = torch.zeros((4, 1, 2, 16, d), dtype=torch.uint8)
        scales = torch.zeros((4, 1, 1, 2, 16), dtype=torch.uint8)
        codes = torch.arange(256, dtype=torch.uint8)
        codes = torch.where((codes & 0x7F) == 0x7F, torch.zeros_like(codes), codes)  # not the NaNs
        for p in range(4):
            pages[p, 0, 1, 0] = codes.view(2, 128)[p % 2]
            pages[p, 0, 0, 0] = codes.view(2, 128)[1 - p % 2]
            scales[p, 0, 0, :, 0] = exponents[p]
        vals = pu.values(pages.view(torch.float8_e4m3fn), scales)
        cache = tsa.PagedCache(4, 1, 16, d, dtype="e4m3", pages=pages.view(torch.float8_e4m3fn).cuda(),
                               scales=scales.cuda())
        Q = torch.zeros((4, 4, 1, d), dtype=torch.bfloat16)
        for h in range(4):  # scores that pick out single key elements
            Q[:, h, 0, 8 * h:8 * h + 3] = 1.0
        table = torch.arange(4, dtype=torch.int32)[:, None].cuda()
        lens = torch.ones(4, dtype=torch.int32).cuda()
        O, LSE = tsa.PagedDecodeAttention(4, 4, 1, 1, d, scale=1.0)(Q.cuda(), cache, table, lens)
        assert torch.equal(O.double().cpu(), vals[:, 0, 1, 0][:, None, None].expand(4, 4, 1, d))
        s = torch.einsum("bhsd,bd->bhs", Q.double(), vals[:, 0, 0, 0])
        assert float(((LSE.double().cpu() - s).abs() - s.abs() * 2.0 ** -21).max()) <= 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_non_finite_rows_stay_in_their_sequence(bad, store):
    """A value row that is not finite makes its own sequence and kv head not finite, and nothing else."""
    lens = [50, 60]
    pages, scales, table, n = pu.make_pool(lens, 2, 16, 64, "bf16", seed=4)
    pages[int(table[0, 1]), 1, 1, 3, 5] = bad
    if store == "e4m3":
        codes, e = pu.quantise(pages.float())
        pages, scales = codes.view(torch.float8_e4m3fn), e.view(n, 2, 2, 1, 16).transpose(2, 3).contiguous()
    cache = tsa.PagedCache(n, 2, 16, 64, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    Q = torch.randn((2, 4, 1, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    O, _ = tsa.PagedDecodeAttention(2, 4, 2, 1, 64)(Q, cache, table.cuda(),
                                                   torch.tensor(lens, dtype=torch.int32).cuda())
    O = O.float().cpu()
    assert bool(torch.isfinite(O[1]).all()) and bool(torch.isfinite(O[0, :2]).all())
    assert not bool(torch.isfinite(O[0, 2:, 0, 5]).any())


# ------------------------------------------------------------------------------------------------ cache
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,rot,layout", [(128, 128, "half"), (128, 64, "interleaved"), (64, 26, "half"),
                                          (64, 6, "interleaved"), (128, 0, "half")])
@pytest.mark.parametrize("S,Hq", [(1, 0), (1, 12), (37, 3)])
def test_write_and_read_back(store, d, rot, layout, S, Hq):
    B, Hkv, page = 4, 3, 48
    g = torch.Generator().manual_seed(S + d)
    news = [S, max(0, S // 2), 0, max(1, S - 3)]
    lens = [S + 20, 48, 33, max(1, S - 3)]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 1
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    order, at = torch.randperm(n_pages, generator=g).to(torch.int32), 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    cache = tsa.PagedCache(n_pages, Hkv, page, d, dtype=store)
    cache.pages.view(torch.uint8).fill_(0x11)
    if store == "e4m3":
        cache.scales.fill_(0x11)
    before = (cache.pages.clone(), None if cache.scales is None else cache.scales.clone())
    qkv = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
    qkv[0, 0, -1] = 0  # a row of zeros
    qkv[0, 0, -2, 3] = 300.0
    qkv = qkv.cuda()
    Q, K, V = (t.transpose(1, 2) for t in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]))
    rope = tsa.RotaryPositions(d, rot, layout=layout) if rot else None
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    Qr = cache.write(K, V, tab, ln, new_len=torch.tensor(news, dtype=torch.int32).cuda(), rope=rope,
                     Q=Q if Hq and rope else None)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    pos = torch.tensor(lens)[:, None] - torch.tensor(news)[:, None] + torch.arange(S)
    f, amp = pu.frequencies(rot) if rot else (torch.zeros(0, dtype=torch.float64), 1.0)
    k_ref, k_size = pu.rotate(K, pos, rot, layout, f, amp)
    if Qr is not None:
        q_ref, q_size = pu.rotate(Q, pos, rot, layout, f, amp)
        for b, n in enumerate(news):
            off = (Qr[b, :, :n].double().cpu() - q_ref[b, :, :n]).abs()
            assert not n or float((off - pu.rope_bound(q_ref, q_size, torch.bfloat16)[b, :, :n]).max()) <= 0
            assert bool((Qr[b, :, n:] == 0).all())
    vals = pu.values(cache.pages, cache.scales)
    written = torch.zeros((n_pages, page), dtype=torch.bool)
    for b, n in enumerate(news):
        for i in range(n):
            p, s = int(table[b, pos[b, i] // page]), int(pos[b, i] % page)
            written[p, s] = True
            k, v = vals[p, :, 0, s], vals[p, :, 1, s]
            want_k, want_v = k_ref[b, :, i], V[b, :, i].float().cpu()
            if store == "bf16":
                assert torch.equal(v, want_v.double())
                assert float(((k - want_k).abs() - pu.rope_bound(want_k, k_size[b, :, i], torch.bfloat16)).max()) <= 0
            else:
                codes, e = pu.quantise(want_v)
                assert torch.equal(cache.pages.view(torch.uint8)[p, :, 1, s].cpu(), codes)
                assert torch.equal(cache.scales[p, :, s // 16, 1, s % 16].cpu(), e)
                # a code is off by half a step: 2^-4 relative, or half the smallest step, 2^-10, times the factor
                f2 = torch.exp2(cache.scales[p, :, s // 16, 0, s % 16].double().cpu() - 127)[:, None]
                bound = want_k.abs() * 2.0 ** -4 + f2 * 2.0 ** -10 + k_size[b, :, i] * 2.0 ** -19
                assert float(((k - want_k).abs() - bound).max()) <= 0
                big = want_k.abs().amax(-1)
                assert bool((big <= 448 * f2[:, 0] * (1 + 2.0 ** -20)).all())
                assert bool(((big > 224 * f2[:, 0] * (1 - 2.0 ** -20)) | (big == 0)).all())
    # every other slot is as it was
    old = pu.values(*before) if store == "bf16" else before[0].view(torch.uint8).cpu()
    now = vals if store == "bf16" else cache.pages.view(torch.uint8).cpu()
    same = (old == now).all(-1).all(1).all(1)
    assert bool((same | written).all())
    if store == "e4m3":
        kept = (cache.scales.cpu() == 0x11).transpose(2, 3).reshape(n_pages, Hkv, 2, page).all(1).all(1)
        assert bool((kept | written).all())
    # read back: exactly what the rows stand for; behind the length as it was
    for first, length in ((0, max(lens) + 5), (17, 40)):
        Kd = torch.full((B, Hkv, length, d), 3.0, dtype=torch.bfloat16, device="cuda")
        Vd = torch.full((B, length, Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)  # strided
        cache.read(tab, ln, first=first, K=Kd, V=Vd)
        for b, n in enumerate(lens):
            m = max(0, min(length, n - first))
            if m:
                k, v = pu.dense(vals, table, page, b, first + m)
                assert torch.equal(Kd[b, :, :m].double().cpu(), k[:, first:])
                assert torch.equal(Vd[b, :, :m].double().cpu(), v[:, first:])
            assert bool((Kd[b, :, m:] == 3).all()) and bool((Vd[b, :, m:] == 3).all())
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,rot,layout,Hq", [(128, 128, "half", 0), (128, 96, "interleaved", 5), (64, 26, "half", 4)])
def test_more_tokens_than_the_grid_takes_at_once(store, d, rot, layout, Hq):
    """Prompts of thousands of tokens, ragged, appended behind others: every row against the definition."""
    lens, news, Hkv, page = [4100, 3500, 2900, 17], [4100, 3000, 2900, 0], 3, 80
    B, S = len(lens), max(news)
    need = [-(-n // page) for n in lens]
    g = torch.Generator().manual_seed(31)
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    cache = tsa.PagedCache(sum(need), Hkv, page, d, dtype=store)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    Q, K, V = (qkv[:, :, lo:hi].transpose(1, 2) for lo, hi in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    rope = tsa.RotaryPositions(d, rot, layout=layout)
    tab, ln, nw = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(news, dtype=torch.int32).cuda()
    Qr = cache.write(K, V, tab, ln, new_len=nw, rope=rope, Q=Q if Hq else None)
    Kd, Vd = cache.read(tab, ln, length=max(lens))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    f, amp = pu.frequencies(rot)
    for b, n in enumerate(news):
        if not n:
            continue
        pos = (lens[b] - n + torch.arange(n))[None]
        k_ref, k_size = pu.rotate(K[b:b + 1, :, :n], pos, rot, layout, f, amp)
        k, v = Kd[b:b + 1, :, lens[b] - n:lens[b]].double().cpu(), Vd[b:b + 1, :, lens[b] - n:lens[b]].double().cpu()
        v_ref = V[b:b + 1, :, :n].double().cpu()
        if store == "bf16":
            assert torch.equal(v, v_ref)
            bound = pu.rope_bound(k_ref, k_size, torch.bfloat16)
        else:
            codes, e = pu.quantise(v_ref.float())
            assert torch.equal(v, codes.view(torch.float8_e4m3fn).double() * torch.exp2(e.double() - 127)[..., None])
            # half a step of a code, 2^-4, or of the smallest ones, 2^-10 of the factor, which is below 2^-7 of the row's
            # largest (224 2^k < max): 2^-17 of that
            bound = k_ref.abs() * 2.0 ** -4 + k_ref.abs().amax(-1, keepdim=True) * 2.0 ** -17 + k_size * 2.0 ** -19
        assert float(((k - k_ref).abs() - bound).max()) <= 0
        if Hq:
            q_ref, q_size = pu.rotate(Q[b:b + 1, :, :n], pos, rot, layout, f, amp)
            off = (Qr[b:b + 1, :, :n].double().cpu() - q_ref).abs() - pu.rope_bound(q_ref, q_size, torch.bfloat16)
            assert float(off.max()) <= 0
    if Hq:
        for b, n in enumerate(news):
            assert bool((Qr[b, :, n:] == 0).all())


def test_written_rows_that_are_not_finite_read_back_as_nan():
    cache = tsa.PagedCache(2, 1, 16, 64, dtype="e4m3")
    K = torch.randn((1, 1, 3, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    V = K.clone()
    K[0, 0, 1, 7], V[0, 0, 2, 0] = math.inf, math.nan
    table, lens = torch.tensor([[1]], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    cache.write(K.cuda(), V.cuda(), table, lens)
    Kd, Vd = cache.read(table, lens, length=3)
    assert bool(torch.isnan(Kd[0, 0, 1]).all()) and bool(torch.isnan(Vd[0, 0, 2]).all())
    assert bool(torch.isfinite(Kd[0, 0, 0]).all()) and bool(torch.isfinite(Vd[0, 0, :2]).all())


@pytest.mark.parametrize("rot", [0, 64])
def test_a_bf16_cache_holds_infinities_as_they_are(rot):
    """Keys that are not rotated, elements behind the rotated ones and values are copied bit by bit."""
    cache = tsa.PagedCache(1, 2, 16, 128)
    K = torch.randn((1, 2, 5, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    K[0, 0, 2, 70], K[0, 1, 4, 127], K[0, 1, 0, 100] = math.inf, -math.inf, -0.0
    V = K.flip(3).contiguous()
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32).cuda()
    cache.write(K.cuda(), V.cuda(), table, lens, rope=tsa.RotaryPositions(128, rot) if rot else None)
    Kd, Vd = cache.read(table, lens, length=5)
    assert torch.equal(Vd.cpu().view(torch.int16), V.view(torch.int16))
    assert torch.equal(Kd.cpu()[..., rot:].contiguous().view(torch.int16), K[..., rot:].contiguous().view(torch.int16))
    assert bool(torch.isfinite(Kd[..., :rot]).all())


@pytest.mark.parametrize("power", [-130, -126, -100, 0, 100, 118])
def test_row_sizes(power):
    """Rows from the smallest to the largest bf16 magnitudes, and the 448 border."""
    x = torch.tensor([1.75, 1.7578125, 1.0, 1.9921875]).double() * 2.0 ** power
    V = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    V[0, :, 0, 5] = x.to(torch.bfloat16)
    V[0, :, 0, 6] = -x.to(torch.bfloat16) / 4
    cache = tsa.PagedCache(1, 4, 16, 64, dtype="e4m3")
    table, lens = torch.zeros((1, 1), dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    cache.write(V.cuda(), V.cuda(), table, lens)
    codes, e = pu.quantise(V[0, :, 0].float())
    assert torch.equal(cache.pages.view(torch.uint8)[0, :, 1, 0].cpu(), codes)
    assert torch.equal(cache.scales[0, :, 0, 1, 0].cpu(), e)
    Kd, _ = cache.read(table, lens, length=1)
    assert torch.equal(Kd[0, :, 0].double().cpu(), pu.values(cache.pages, cache.scales)[0, :, 0, 0])


# ------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_generation_steps_as_they_are_used(store):
    """Prompts written in ragged chunks, then steps of rotate + append + attend, captured once and replayed with the
    lengths moved on the device; an empty slot stays in the batch.  The last step equals the float64 operators on what
    the cache holds, and on a bf16 cache agrees with decode over the dense cache read back."""
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 128, 16, 20
    g = torch.Generator().manual_seed(8)
    prompt = [37, 0, 5]
    rope = tsa.RotaryPositions(d, scaling="yarn", factor=2.0, original_len=32)
    cache = tsa.PagedCache(16, Hkv, page, d, dtype=store)
    table = torch.tensor([[3, 9, 1, 12], [-1, -1, -1, -1], [4, 0, 7, 5]], dtype=torch.int32).cuda()
    S = max(prompt)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    news = torch.tensor(prompt, dtype=torch.int32).cuda()
    lens = news.clone()
    cache.write(qkv[:, :, Hq:Hq + Hkv].transpose(1, 2), qkv[:, :, Hq + Hkv:].transpose(1, 2), table, lens, new_len=news,
                rope=rope)
    plan = tsa.PagedDecodeAttention(B, Hq, Hkv, 1, d)
    one = torch.empty((B, 1, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    Q, K, V = (one[:, :, lo:hi].transpose(1, 2) for lo, hi in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    alive = torch.tensor([1, 0, 1], dtype=torch.int32).cuda()
    Qr = torch.empty((B, Hq, 1, d), dtype=torch.bfloat16, device="cuda")
    O, LSE = torch.empty_like(Qr), torch.empty((B, Hq, 1), device="cuda")

    def step():
        lens.add_(alive)
        cache.write(K, V, table, lens, new_len=alive, rope=rope, Q=Q, Q_out=Qr)
        plan(Qr, cache, table, lens, O=O, LSE=LSE)

    xs = torch.randn((steps, *one.shape), generator=g).to(torch.bfloat16).cuda()
    one.copy_(xs[0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        one.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        n = [p + (i + 1) * a for p, a in zip(prompt, (1, 0, 1))]
        assert lens.tolist() == n
        ref = pu.decode(Qr, pu.values(cache.pages, cache.scales), table.cpu(), page, n, 1 / math.sqrt(d), CAUSAL, 0)
        pu.check_decode(O, LSE, ref, d)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    # the dense decode over what is read back
    Kd, Vd = cache.read(table, lens, length=64)
    live = [0, 2]
    dec = tsa.DecodeAttention(2, Hq, Hkv, 1, 64, d)
    Od, Ld = dec(Qr[live].contiguous(), Kd[live].contiguous(), Vd[live].contiguous(), [n[b] for b in live])
    # each is within its rounding bounds of the exact result: two roundings of weights and of O each
    assert float((Od.float() - O[live].float()).abs().max()) <= 4 * 2.0 ** -8 * float(Vd.float().abs().max())
    assert float((Ld - LSE[live]).abs().max()) <= 1e-5


def test_one_plan_over_both_cache_types_and_changing_lengths():
    """What a call leaves in the plan's workspace (cut units, partial results) does not reach the next one."""
    Hq, Hkv, d, page = 12, 2, 64, 32
    plan = tsa.PagedDecodeAttention(3, Hq, Hkv, 2, d)
    Q = torch.randn((3, Hq, 2, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    for i, (lens, grid) in enumerate((([3000, 9, 1200], 304), ([40, 40, 40], 304), ([0, 0, 0], 304), ([1, 5000, 0], 5),
                                      ([2, 2, 700], 304))):
        plan.set_grid_limit(grid)
        for store in ("bf16", "e4m3"):
            cache, vals, table = _cache(lens, Hkv, page, d, store, seed=20 + i)
            O, LSE = plan(Q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
            pu.check_decode(O, LSE, pu.decode(Q, vals, table, page, lens, 1 / math.sqrt(d), CAUSAL, 0), d)
            assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, 2 ** 31 - 1])
def test_a_window_beyond_every_position(store, window):
    """The widest windows see what no window does, also with lengths below the number of rows."""
    lens = [0, 1, 2, 40, 700]
    cache, vals, table = _cache(lens, 2, 16, 64, store, seed=5)
    Q = torch.randn((5, 4, 4, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want = tsa.PagedDecodeAttention(5, 4, 2, 4, 64)(Q, cache, tab, ln)
    got = tsa.PagedDecodeAttention(5, 4, 2, 4, 64, kind=WINDOW, window=window)(Q, cache, tab, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_captured_behind_copies_and_another_stream(store):
    """In a graph the decode stands behind a copy of its lengths and behind a write from a second stream, and two calls of
    one plan stand behind one another; the replay sees what both left."""
    lens = [900, 33]
    cache, vals, table = _cache(lens, 2, 16, 128, store, seed=11)
    new = torch.tensor(lens, dtype=torch.int32).cuda()
    tab, ln = table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((2, 2, 8, 1, 128), generator=g).to(torch.bfloat16).cuda()
    K = torch.randn((2, 2, 1, 128), generator=g).to(torch.bfloat16).cuda()
    plan = tsa.PagedDecodeAttention(2, 8, 2, 1, 128)
    O, LSE = torch.empty_like(Q), torch.empty((2, 2, 8, 1), device="cuda")
    side = torch.cuda.Stream()

    def step():
        ln.copy_(new)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            cache.write(K, K, tab, ln)
        main.wait_stream(side)
        for i in range(2):
            plan(Q[i], cache, tab, ln, O=O[i], LSE=LSE[i])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shorter in (0, 20):
        new.sub_(shorter)
        ln.zero_()
        O.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        n = new.tolist()
        vals = pu.values(cache.pages, cache.scales)
        for i in range(2):
            pu.check_decode(O[i], LSE[i], pu.decode(Q[i], vals, table, 16, n, 1 / math.sqrt(128), CAUSAL, 0), 128)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_calls_behind_one_another_need_no_synchronisation(store):
    """Each call reads what the one before wrote, and writes what the one before that read, in the same few buffers: the
    same bits with and without waiting for each."""
    B, Hq, Hkv, d, page, room = 5, 16, 2, 128, 32, 1600
    g = torch.Generator().manual_seed(17)
    base = torch.randn((B, Hq + 2 * Hkv, 1, d), generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(B * room // page, generator=g).to(torch.int32).view(B, room // page).cuda()
    start = torch.tensor([1500, 0, 700, 31, 32], dtype=torch.int32).cuda()
    rope = tsa.RotaryPositions(d)

    def run(wait):
        cache = tsa.PagedCache(B * room // page, Hkv, page, d, dtype=store)
        plan = tsa.PagedDecodeAttention(B, Hq, Hkv, 1, d)
        x, lens = base.clone(), start.clone()
        Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        Qr, O = (torch.empty((B, Hq, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        LSE = torch.empty((B, Hq, 1), device="cuda")
        for _ in range(40):
            lens.add_(1)
            wait()
            cache.write(K, V, table, lens, rope=rope, Q=Q, Q_out=Qr)
            wait()
            plan(Qr, cache, table, lens, O=O, LSE=LSE)
            wait()
            cache.read(table, lens, K=K, V=V)  # the first position's rows become the next step's
            wait()
            rope(K, O, positions=lens[:, None], Q_out=K, K_out=Q)
            wait()
            rope.backward(Q, positions=lens[:, None], dQ=Q)
            wait()
        torch.cuda.synchronize()
        assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
        return x, O, LSE, cache.pages.view(torch.uint8).clone()

    want = run(torch.cuda.synchronize)
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            for _ in range(3):
                assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


def test_two_plans_on_two_streams():
    lens = [700, 90, 1300]
    cache, vals, table = _cache(lens, 2, 16, 128, "bf16", seed=6)
    tab, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(2)
    Qs = [torch.randn((3, 8, 1, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    plans = [tsa.PagedDecodeAttention(3, 8, 2, 1, 128) for _ in range(2)]
    want = [plans[i](Qs[i], cache, tab, ln) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(plans[i](Qs[i], cache, tab, ln, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for O, L in got[i]:
            assert torch.equal(O, want[i][0]) and torch.equal(L, want[i][1])


def test_bad_pages_and_lengths_are_reported():
    """Bounds are checked on the device: nothing outside the pool is read or written, the error word names the kind."""
    cache = tsa.PagedCache(4, 2, 16, 64)
    plan = tsa.PagedDecodeAttention(2, 4, 2, 1, 64)
    Q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    K = torch.ones((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    ok = torch.tensor([20, 5], dtype=torch.int32).cuda()
    for table, lens, code in ((good, [20, 33], tsa.CACHE_ERR_POSITION), (good, [2 ** 31 - 1, 1], tsa.CACHE_ERR_POSITION),
                              ([[0, 4], [2, 3]], [20, 5], tsa.CACHE_ERR_PAGE), ([[0, 1], [-1, 3]], [20, 5],
                                                                                tsa.CACHE_ERR_PAGE)):
        tab = torch.as_tensor(table, dtype=torch.int32).cuda()
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
        for call in (lambda: plan(Q, cache, tab, ln), lambda: cache.write(K, K, tab, ln),
                     lambda: cache.read(tab, ln, length=64)):
            call()
            assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, code)
            assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    plan(Q, cache, good, ok)  # the plan works on
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_negative_length_is_reported_by_the_decode():
    cache = tsa.PagedCache(1, 1, 16, 64)
    O, LSE = tsa.PagedDecodeAttention(1, 1, 1, 1, 64)(
        torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda"), cache,
        torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([-1], dtype=torch.int32).cuda())
    assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, tsa.CACHE_ERR_POSITION)


def test_expanded_inputs_and_dimensions_of_one():
    """Broadcast inputs are read as they are; the strides of dimensions of one do not matter."""
    cache = tsa.PagedCache(3, 2, 16, 64)
    K = torch.randn((1, 1, 4, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    tab = torch.tensor([[0], [1]], dtype=torch.int32).cuda()
    ln = torch.full((2,), 4, dtype=torch.int32, device="cuda")
    cache.write(K.expand(2, 2, 4, 64), K.expand(2, 2, 4, 64), tab, ln)
    Kd, Vd = cache.read(tab, ln, length=4)
    assert torch.equal(Kd, K.expand(2, 2, 4, 64)) and torch.equal(Vd, Kd)
    odd = torch.as_strided(K[0, 0, :1].clone(), (1, 1, 1, 64), (3, 5, 7, 1))
    cache.write(odd.expand(2, 2, 1, 64), odd.expand(2, 2, 1, 64), tab, ln)
    assert torch.equal(cache.read(tab, ln, first=3, length=1)[0], odd.expand(2, 2, 1, 64))
    with pytest.raises(ValueError):
        cache.read(tab, ln, K=Kd[:, :1].expand(2, 2, 4, 64), V=Vd)


def test_refusals():
    cache = tsa.PagedCache(4, 2, 16, 64)
    plan = tsa.PagedDecodeAttention(2, 4, 2, 1, 64)
    Q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    K = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    tab = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    ln = torch.ones(2, dtype=torch.int32, device="cuda")
    bad = [lambda: plan(Q, cache, tab.long(), ln), lambda: plan(Q, cache, tab, ln.long()),
           lambda: plan(Q, cache, tab, ln[:1]), lambda: plan(Q, cache, tab.cpu(), ln),
           lambda: plan(Q[:1], cache, tab, ln), lambda: plan(Q.float(), cache, tab, ln),
           lambda: plan(Q, tsa.PagedCache(4, 1, 16, 64), tab, ln), lambda: plan(Q, tsa.PagedCache(4, 2, 16, 128), tab, ln),
           lambda: cache.write(K, K[:, :1], tab, ln), lambda: cache.write(K.float(), K, tab, ln),
           lambda: cache.write(K, K, tab, ln, Q=Q), lambda: cache.write(K, K, tab, ln, rope=tsa.RotaryPositions(128)),
           lambda: cache.write(K, K, tab, ln, new_len=ln.long()), lambda: cache.read(tab, ln),
           lambda: cache.read(tab, ln, length=3, K=K), lambda: cache.read(tab, ln, first=-1, length=3),
           lambda: tsa.PagedCache(4, 2, 24, 64), lambda: tsa.PagedCache(0, 2, 16, 64),
           lambda: tsa.PagedCache(4, 2, 16, 96), lambda: tsa.PagedCache(4, 2, 16, 64, dtype="f32"),
           lambda: tsa.PagedCache(4, 2, 16, 64, pages=torch.zeros((4, 2, 2, 16, 64), device="cuda")),
           lambda: tsa.PagedDecodeAttention(2, 4, 3, 1, 64), lambda: tsa.PagedDecodeAttention(2, 128, 1, 1, 64),
           lambda: tsa.PagedDecodeAttention(2, 4, 2, 1, 96), lambda: tsa.PagedDecodeAttention(2, 4, 2, 0, 64),
           lambda: tsa.PagedDecodeAttention(2, 4, 2, 1, 64, kind=tsa.MASK_SLIDING),
           lambda: tsa.PagedDecodeAttention(2, 4, 2, 1, 64, kind=WINDOW, window=-1)]
    closed = tsa.RotaryPositions(64)
    closed.close()
    bad += [lambda: cache.write(K, K, tab, ln, rope=closed), lambda: cache.read(tab, ln, first=1 << 32, length=3),
            lambda: tsa.PagedDecodeAttention(2, 4, 2, 1, 64, kind=WINDOW, window=1 << 32),
            lambda: tsa.PagedDecodeAttention((1 << 32) + 2, 4, 2, 1, 64)]
    for call in bad:
        with pytest.raises((ValueError, tsa.AttnError)):
            call()
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
