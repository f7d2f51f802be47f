"""Selection by scores at the ends of the float32 range: they are compared exactly, whatever the bounds' powers of two are."""
import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _check(cache, codes, exps, table, n, Q, keep):
    bounds = tsa.PageBounds(cache, codes=codes.cuda(), exponents=exps.cuda())
    got, short = bounds.select(Q.cuda(), table.cuda(), _int32([n]), keep, 1, 1)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    page = cache.shape[2]
    chosen, want_len = cu.select(Q, codes, exps, table, page, [n], keep, 1, 1)
    assert short.tolist() == want_len
    for h in range(cache.shape[1]):
        assert got[0, h].tolist() == table[0][torch.tensor(chosen[0][h])].tolist()
    return chosen[0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lo,hi", [(1, 3), (230, 240), (247, 254), (250, 250), (1, 254)])
@pytest.mark.parametrize("most", [1, 127])
def test_powers_of_two_at_both_ends(d, lo, hi, most):
    """Codes up to `most` with exponents from lo to hi, pages of exponent 255 among them: 2^127 * 128 * 127^2 and its negative
    are scores, and 2^-126."""
    pages, Hkv, page = 300, 2, 16
    g = torch.Generator().manual_seed(d + lo + hi)
    codes = torch.randint(-most, most + 1, (pages, Hkv, 2, d), generator=g).sort(dim=2).values.to(torch.int8)
    codes[10:20] = most  # the largest score there is, and the smallest
    codes[20:30] = -most
    exps = torch.randint(lo, hi + 1, (pages, Hkv), generator=g).to(torch.uint8)
    exps[40] = 255
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    cache = tsa.PagedCache(pages, Hkv, page, d)
    for sign in (torch.ones(d), torch.randint(0, 2, (d,), generator=g) * 2.0 - 1):
        Q = (sign * torch.randint(1, 128, (1, 4, 1, d), generator=g)).to(torch.bfloat16)
        Q[..., 0] = 127.0
        for keep in (5, 60, 200):
            _check(cache, codes, exps, table, pages * page - 3, Q, keep)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_keys_of_far_powers(store):
    """Keys of about 2^118: every page's score is beyond 2^128, and they are still told apart."""
    pages, page, d = 60, 16, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn((pages, 1, 2, page, d), generator=g)
    x[:, :, 0] = (x[:, :, 0].abs() + 1) * 2.0 ** 117 * torch.linspace(0.5, 1.0, pages)[torch.randperm(pages, generator=g)][:, None, None, None]
    if store == "bf16":
        cache = tsa.PagedCache(pages, 1, page, d, pages=x.to(torch.bfloat16).cuda())
    else:
        codes, e = pu.quantise(x)
        cache = tsa.PagedCache(pages, 1, page, d, dtype="e4m3", pages=codes.view(torch.float8_e4m3fn).cuda(),
                               scales=e.view(pages, 1, 2, 1, 16).transpose(2, 3).contiguous().cuda())
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    n = pages * page
    bounds = tsa.PageBounds(cache)
    bounds.update(table.cuda(), _int32([n]))
    codes, exps = bounds.codes.cpu(), bounds.exponents.cpu()
    vals = pu.values(cache.pages, cache.scales)
    for i in range(pages):
        c, e = cu.bounds(vals, table, page, 0, n, i)
        assert torch.equal(codes[int(table[0, i])], c) and torch.equal(exps[int(table[0, i])], e)
    Q = (torch.rand((1, 4, 1, d), generator=g) + 0.5).to(torch.bfloat16)
    chosen = _check(cache, codes, exps, table, n, Q, 12)
    assert chosen[0][:11] != list(range(11))


def test_queries_that_are_not_finite_still_choose_unknown_pages_first():
    """Pages whose keys are not all finite have the largest score there is, for queries that are not finite too; the others are
    equal then, and the first of them follow."""
    pages, page, d = 50, 16, 64
    g = torch.Generator().manual_seed(6)
    codes = torch.randint(-127, 128, (pages, 1, 2, d), generator=g).sort(dim=2).values.to(torch.int8)
    exps = torch.full((pages, 1), 120, dtype=torch.uint8)
    exps[30] = exps[44] = 255
    table = torch.arange(pages, dtype=torch.int32)[None]
    cache = tsa.PagedCache(pages, 1, page, d)
    Q = torch.randn((1, 2, 1, d), generator=g).to(torch.bfloat16)
    Q[0, 1, 0, 9] = float("nan")
    assert _check(cache, codes, exps, table, pages * page, Q, 6)[0] == [0, 1, 2, 30, 44, 49]
