"""The 16 significant bits of the paged decode's weights over bf16 pages (up to 32 rows to a kv head).

The values alternate in sign and nearly cancel, so that O's own rounding is small beside what a weight of eight bits would
leave: a kernel that dropped the second half of a weight fails.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

LENS, PAGE, HKV = [2, 6, 33, 700], 32, 2


def _inputs(rows, d):
    g = torch.Generator().manual_seed(rows + d)
    need = [-(-n // PAGE) for n in LENS]
    table = torch.full((len(LENS), max(need)), -1, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
    x = torch.randn((sum(need), HKV, 2, PAGE, d), generator=g)
    sign = 1.0 - 2.0 * (torch.arange(PAGE) % 2)  # (even page size: the sign goes by the position)
    x[:, :, 1] = sign[:, None] * (1.0 + 2.0 ** -5 * x[:, :, 1])
    pages = x.to(torch.bfloat16)
    Q = (0.1 * torch.randn((len(LENS), HKV * rows, 1, d), generator=g)).to(torch.bfloat16)
    return pages, table, Q


def _past_bound(O, ref, d):
    """How far O is past its bound.  A weight: 2^-16 of its rounding to two bf16 numbers (each leaves 2^-8 of what it
    rounds), and r of the score and of exp2, as paged_util.check_decode derives it; the same r in the sum that divides;
    then the rounding of O."""
    O_ref, _, A, E = ref
    r = (E * (d + 8) * 2.0 ** -23 + 2.0 ** -19)[..., None]
    return float(((O.double().cpu() - O_ref).abs() - (O_ref.abs() * 2.0 ** -8 + A * (2.0 ** -16 + 2 * r) * (1 + 2.0 ** -7))).max())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 8, 16, 17, 32])
@pytest.mark.parametrize("grid", [1 << 20, 3])
def test_weights_keep_sixteen_bits(rows, d, grid):
    pages, table, Q = _inputs(rows, d)
    cache = tsa.PagedCache(pages.shape[0], HKV, PAGE, d, pages=pages.cuda())
    plan = tsa.PagedDecodeAttention(len(LENS), HKV * rows, HKV, 1, d)
    plan.set_grid_limit(grid)
    O, _ = plan(Q.cuda(), cache, table.cuda(), torch.tensor(LENS, dtype=torch.int32).cuda())
    ref = pu.decode(Q, pu.values(pages, None), table, PAGE, LENS, 1 / math.sqrt(d), tsa.MASK_CAUSAL, 0)
    assert _past_bound(O, ref, d) <= 0
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 8, 16, 17, 32])
def test_eight_bits_would_not_pass(rows, d):
    """The definition with its weights rounded once to bf16 is past the bound; rounded to two bf16 numbers it is not."""
    pages, table, Q = _inputs(rows, d)
    vals = pu.values(pages, None)
    ref = pu.decode(Q, vals, table, PAGE, LENS, 1 / math.sqrt(d), tsa.MASK_CAUSAL, 0)
    for parts in (1, 2):
        O = torch.zeros_like(ref[0])
        for b, n in enumerate(LENS):
            K, V = pu.dense(vals, table, PAGE, b, n)
            s = torch.einsum("hgd,hjd->hgj", Q[b].double().view(HKV, rows, d), K) / math.sqrt(d)
            w = torch.exp(s - s.amax(-1, keepdim=True))
            held = w.to(torch.bfloat16).double()
            if parts == 2:
                held = held + (w - held).to(torch.bfloat16).double()
            O[b] = (torch.einsum("hgj,hjd->hgd", held, V) / w.sum(-1, keepdim=True)).view(HKV * rows, 1, d)
        assert (_past_bound(O.to(torch.bfloat16), ref, d) > 0) == (parts == 1)
