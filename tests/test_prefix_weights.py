"""The significant bits of the weights of a shared prefix: those of fp16 over E4M3 pages (11), of bf16 over bf16 pages (8).

The values alternate in sign and nearly cancel, so that O's own rounding is small beside what a weight of eight bits leaves:
weights of bf16 fail the bound of E4M3 pages.
"""
import math

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

PLENS, PAGE, HKV = [2, 6, 33, 700], 32, 2
HALF_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}


def _inputs(rows, members, d, store):
    g = torch.Generator().manual_seed(rows + d + members)
    need = [-(-n // PAGE) for n in PLENS]
    table = torch.full((len(PLENS), max(need)), -1, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
    x = torch.randn((sum(need), HKV, 2, PAGE, d), generator=g)
    sign = 1.0 - 2.0 * (torch.arange(PAGE) % 2)  # (even page size: the sign goes by the position)
    x[:, :, 1] = sign[:, None]
    if store == "bf16":
        pages, scales = x.to(torch.bfloat16), None
    else:
        codes, e = pu.quantise(x)
        pages = codes.view(torch.float8_e4m3fn)
        scales = e.view(sum(need), HKV, 2, PAGE // 16, 16).transpose(2, 3).contiguous()
    of = torch.arange(len(PLENS)).repeat(members)
    Q = (0.03 * torch.randn((of.numel(), HKV * rows, 1, d), generator=g)).to(torch.bfloat16)
    return pages, scales, table, of, Q


def _reference(Q, pages, scales, table, of, d):
    return pu.decode(Q, pu.values(pages, scales), table[of], PAGE, [PLENS[g] for g in of.tolist()], 1 / math.sqrt(d), tsa.MASK_FULL, 0)


def _past_bound(O, ref, d, half_step):
    """How far O is past its bound: half a step of a weight, and r of the score and of exp2, as paged_util.check_decode derives
    it; the same r in the sum that divides; then the rounding of O."""
    O_ref, _, A, E = ref
    r = (E * (d + 8) * 2.0 ** -23 + 2.0 ** -19)[..., None]
    return float(((O.double().cpu() - O_ref).abs() - (O_ref.abs() * 2.0 ** -8 + A * (half_step + 2 * r) * (1 + 2.0 ** -7))).max())


SHAPES = [(1, 1), (4, 1), (32, 1), (32, 5), (3, 60)]


@pytest.mark.gpu
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,members", SHAPES)
@pytest.mark.parametrize("grid", [1 << 20, 3])
def test_bits_of_the_weights(store, d, rows, members, grid):
    pages, scales, table, of, Q = _inputs(rows, members, d, store)
    cache = tsa.PagedCache(pages.shape[0], HKV, PAGE, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    B = of.numel()
    plan = tsa.SharedPrefixAttention(B, HKV * rows, HKV, 1, d)
    plan.set_grid_limit(grid)
    none = torch.zeros((B, 1), dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    O, _ = plan(Q.cuda(), cache, table.cuda(), torch.tensor(PLENS, dtype=torch.int32).cuda(), *none,
                prefix_of=of.to(torch.int32).cuda())
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    assert _past_bound(O, _reference(Q, pages, scales, table, of, d), d, HALF_STEP[store]) <= 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,members", SHAPES)
def test_weights_of_eight_bits_would_not_pass_over_e4m3(d, rows, members):
    """The definition with its weights rounded to bf16 is past the bound; rounded to fp16 it is not."""
    pages, scales, table, of, Q = _inputs(rows, members, d, "e4m3")
    vals = pu.values(pages, scales)
    ref = _reference(Q, pages, scales, table, of, d)
    for dtype in (torch.bfloat16, torch.float16):
        O = torch.zeros_like(ref[0])
        for b, g in enumerate(of.tolist()):
            K, V = pu.dense(vals, table, PAGE, g, PLENS[g])
            s = torch.einsum("hgd,hjd->hgj", Q[b].double().view(HKV, rows, d), K) / math.sqrt(d)
            w = torch.exp(s - s.amax(-1, keepdim=True))
            O[b] = (torch.einsum("hgj,hjd->hgd", w.to(dtype).double(), V) / w.sum(-1, keepdim=True)).view(HKV * rows, 1, d)
        assert (_past_bound(O.to(torch.bfloat16), ref, d, HALF_STEP["e4m3"]) > 0) == (dtype is torch.bfloat16)
