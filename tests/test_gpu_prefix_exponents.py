"""Shared prefixes over E4M3 pages whose rows' factors lie far apart within 128 positions.

Keys and values are held to 2^-32 of the largest factor 2^E among 128 positions (of values: at least 2^-40 of the largest factor
before them), so that rows whose exponent is up to 39 below the largest still count.  Rows with the large factors have no part in the
results here: the queries are zero where those keys are not, or their weights are nothing.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa
from test_gpu_prefix import _int32, _make

pytestmark = pytest.mark.gpu

PAGE, N, HQ = 16, 200, 4
LARGE = [5, 70, 130, 199]  # positions with the largest factor, in both tiles


def _step(d, k_codes, k_exps, v_codes, v_exps, Q, grid=None):
    """O, LSE and the float64 rows of one sequence behind a prefix of the given rows [N, d] and exponents [N]."""
    n = k_codes.shape[0]
    cache, _, ptab, table = _make([n], [0], 1, PAGE, d, "e4m3")
    codes, exps = cache.pages.view(torch.uint8).cpu(), cache.scales.cpu()
    for j in range(n):
        p, s = int(ptab[0, j // PAGE]), j % PAGE
        for kv, (c, e) in enumerate(((k_codes, k_exps), (v_codes, v_exps))):
            codes[p, 0, kv, s] = c[j].to(torch.float8_e4m3fn).view(torch.uint8)
            exps[p, 0, 0, kv, s] = int(e[j])
    cache.pages.view(torch.uint8).copy_(codes.cuda())
    cache.scales.copy_(exps.cuda())
    plan = tsa.SharedPrefixAttention(1, HQ, 1, 1, d)
    if grid:
        plan.set_grid_limit(grid)
    O, L = plan(Q.cuda(), cache, ptab.cuda(), _int32([n]), table.cuda(), _int32([0]))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    K, V = pu.dense(pu.values(cache.pages, cache.scales), ptab, PAGE, 0, n)
    return O[0, :, 0].double().cpu(), L[0, :, 0].double().cpu(), K[0], V[0]


def _check(O, L, K, V, Q, k_exps, v_exps, d):
    """A score is off by r: paged_util.check_decode's r, and 2^-32 of the largest key factor of the tile in every element that is
    not held exactly (rows up to 22 below the largest exponent are).  A weight is an fp16 number relative to a reference at least
    64 times below the largest product of weight and factor, `big`: off by 2^-11 of itself, or below 2^-20 of `big` by
    2^-31 of it, and never by more than itself.  Values: 2^-32 of their tile's factor."""
    n, scale = K.shape[0], d ** -0.5
    q = Q[0, :, 0].double()
    s = q @ K.T * scale
    size = (q.abs() @ K.abs().T * scale).amax(-1)
    held_k, held_v, factor_v, most = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64), 0.0
    for t in range(0, n, 128):
        tile = slice(t, min(n, t + 128))
        e = k_exps[tile].double()
        held_k[tile] = torch.where(e.max() - e > 22, 2.0 ** (e.max() - 127 - 32), torch.zeros_like(e))
        e = v_exps[tile].double()
        most = max(most, float(2.0 ** (e.max() - 127)))
        f = max(float(2.0 ** (e.max() - 127)), most * 2.0 ** -40)
        factor_v[tile] = f
        held_v[tile] = torch.where(math.log2(f) + 127 - e > 22, torch.full_like(e, f * 2.0 ** -32), torch.zeros_like(e))
    r = size * (d + 8) * 2.0 ** -23 + 2.0 ** -19 + scale * q.abs().sum(-1) * held_k.max()
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    want, A = p @ V, p @ V.abs()
    big = torch.zeros(HQ, dtype=torch.float64)
    for t in range(0, n, 128):
        big = torch.maximum(big, p[:, t:t + 128].amax(-1) * factor_v[t])
    off = torch.where(p * factor_v >= big[:, None] * 2.0 ** -20, p * 2.0 ** -11, torch.minimum(p, big[:, None] * 2.0 ** -31 / factor_v))
    bound = want.abs() * 2.0 ** -8 + (off @ V.abs() + (p @ held_v)[:, None] + torch.expm1(2 * r)[:, None] * A) * (1 + 2.0 ** -7) + 2.0 ** -133
    bad = (O - want).abs() - bound
    assert float(bad.max()) <= 0, (float((O - want).abs().max()), float(bound.min()), float(want.abs().max()))
    assert float(((L - lse).abs() - r - lse.abs() * 2.0 ** -22).max()) <= 0


def _queries(g, d):
    """Of magnitudes between 1/2 and 1 in the first half of the channels, zero in the others."""
    Q = (torch.rand((1, HQ, 1, d), generator=g) * 0.5 + 0.5) * (1.0 - 2.0 * torch.randint(0, 2, (1, HQ, 1, d), generator=g))
    Q[..., d // 2:] = 0
    return Q.to(torch.bfloat16)


def _codes(g, n, d, least=16.0, signs=True):
    x = least + (448 - least) * torch.rand((n, d), generator=g)
    return x * (1.0 - 2.0 * torch.randint(0, 2, (n, d), generator=g)) if signs else x


# 2^(e - E) times a code is exact up to 22 below; one factor up to 31; two up to 39; then nothing is left
APART = [0, 21, 22, 23, 30, 31, 32, 33, 36, 38]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", APART)
@pytest.mark.parametrize("grid", [None, 1])
def test_keys_far_below_the_largest_of_their_tile(d, apart, grid):
    g = torch.Generator().manual_seed(31 + apart)
    k, e = _codes(g, N, d), torch.full((N,), 118)
    k[LARGE, :d // 2] = 0
    e[LARGE] = 118 + apart
    v, ve = torch.randn((N, d), generator=g), torch.full((N,), 127)
    Q = _queries(g, d)
    O, L, K, V = _step(d, k, e, v, ve, Q, grid)
    _check(O, L, K, V, Q, e, ve, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", APART)
@pytest.mark.parametrize("grid", [None, 1])
def test_values_far_below_the_largest_of_their_tile(d, apart, grid):
    g = torch.Generator().manual_seed(32 + apart)
    Q = _queries(g, d)
    Q[...] = Q.abs()
    k, e = torch.rand((N, d), generator=g), torch.full((N,), 124)
    k[LARGE], e[LARGE] = -448.0, 130  # scores of -5000 and less: no weight
    v, ve = _codes(g, N, d, signs=False), torch.full((N,), 120)
    v[LARGE] = 1.0
    ve[LARGE] = 120 + apart
    O, L, K, V = _step(d, k, e, v, ve, Q, grid)
    _check(O, L, K, V, Q, e, ve, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", [39, 41, 50, 62, 63, 71, 72, 73, 76])
def test_values_far_below_those_of_the_tiles_before(d, apart):
    """One CTA goes through both tiles: the second's values are held to 2^-32 of 2^-40 of the first's factor."""
    g = torch.Generator().manual_seed(33 + apart)
    Q = _queries(g, d)
    Q[...] = Q.abs()
    n = 512
    k, e = torch.rand((n, d), generator=g), torch.full((n,), 124)
    k[:256], e[:256] = -448.0, 130
    v, ve = _codes(g, n, d, signs=False), torch.full((n,), 180 - apart)
    ve[:256] = 180
    O, L, K, V = _step(d, k, e, v, ve, Q, 1)
    _check(O, L, K, V, Q, e, ve, d)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_are_not_finite_beside_far_exponents(d):
    """Two factors leave a NaN a NaN: a NaN code in a row far below the largest exponent, and a row of exponent 255."""
    g = torch.Generator().manual_seed(34)
    k, e = _codes(g, N, d), torch.full((N,), 118)
    k[LARGE, :d // 2] = 0
    e[LARGE] = 118 + 34
    v, ve = torch.randn((N, d), generator=g), torch.full((N,), 127)
    ve[LARGE] = 127 + 34
    v[20, 7] = math.nan
    O, _, _, _ = _step(d, k, e, v, ve, _queries(g, d))
    assert bool(O[:, 7].isnan().all()) and int(O.isnan().sum()) == HQ
    ve[20] = 255
    v[20, 7] = 0
    O, _, _, _ = _step(d, k, e, v, ve, _queries(g, d))
    assert bool(O.isnan().all())
