"""Host side of the entry points for long contexts over a paged cache (no GPU): refusals."""
import types

import pytest
import torch

import transformer_self_attention_gb300 as tsa

BAD = tsa.ATTN_ERR_INVALID_ARG


def test_null_handles_and_pointers_are_refused():
    assert tsa.attn_paged_forward_heads(0, 0, 16, 16, 1, 1, 1, 16, 16) == BAD
    assert tsa.attn_bounds_update(0, 16, 16, 1, 16, 1, 1, 16) == BAD
    assert tsa.attn_bounds_select(0, 16, 16, 1, 1, 1, 16, 16, 1, 1, 16, 4, 1, 1, 32, 32) == BAD


def _fake_cache(Hkv=2, page=16, d=64):
    """What the binding looks at before it calls the library."""
    cache = types.SimpleNamespace(shape=(8, Hkv, page, d), _device=-1, device="cpu", handle=None, pages=None, scales=None)
    cache._table = lambda table, lens: (table.shape[0], (0, 0, table.shape[1], 0))
    return cache


def test_selection_arguments_are_refused():
    bounds = tsa.PageBounds(_fake_cache(), codes=torch.zeros((8, 2, 2, 64), dtype=torch.int8),
                            exponents=torch.zeros((8, 2), dtype=torch.uint8))
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    Q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    for kw in (dict(keep=1), dict(keep=4, sinks=-1), dict(keep=4, recent=0), dict(keep=4, sinks=3, recent=2)):
        with pytest.raises(ValueError):
            bounds.select(Q, table, lens, **kw)
    for S_q, recent in ((2, 1), (17, 1), (18, 2)):
        with pytest.raises(ValueError):
            bounds.select(torch.zeros((1, 4, S_q, 64), dtype=torch.bfloat16), table, lens, keep=8, recent=recent)
    for bad in (Q.float(), Q[:, :3], Q[..., :32], Q[:, :, :0], Q.expand(2, 4, 1, 64), Q.transpose(1, 2)):
        with pytest.raises(ValueError):
            bounds.select(bad, table, lens, keep=4)
    with pytest.raises(ValueError):
        bounds.select(Q, table, lens, keep=2 ** 40)
    with pytest.raises(ValueError):
        tsa.PageBounds(_fake_cache(), codes=torch.zeros((8, 2, 2, 64), dtype=torch.uint8))


def test_weights_arguments_are_refused():
    assert tsa.attn_weights_accumulate(0, 16, 1, 1, 1, 16, 16, 1.0, 1, 0, 1.0, 16, 1, 1, 16) == BAD
    assert tsa.attn_weights_evict(0, 16, 1, 16, 1, 1, 16, 4, 1, 0, 0, 0, 32, 32) == BAD
    weights = tsa.PageWeights(_fake_cache(), weights=torch.zeros((8, 2, 16)))
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    Q, LSE = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16), torch.zeros((1, 4, 1))
    for q, lse in ((Q.float(), LSE), (Q[:, :3], LSE[:, :3]), (Q, LSE[:, :2]), (Q, LSE.double()), (Q[..., :32], LSE),
                   (Q.expand(2, 4, 1, 64), LSE)):
        with pytest.raises(ValueError):
            weights.accumulate(q, lse, table, lens)
    for kw in (dict(keep=-1), dict(keep=0), dict(keep=4, recent=-1), dict(keep=2 ** 31),
               dict(keep=40, to_table=torch.zeros((1, 2), dtype=torch.int32)),
               dict(keep=4, to_table=torch.zeros((2, 4), dtype=torch.int32))):
        with pytest.raises(ValueError):
            weights.evict(table, lens, **kw)
    with pytest.raises(ValueError):
        tsa.PageWeights(_fake_cache(), weights=torch.zeros((8, 16)))


@pytest.mark.parametrize("kw,status", [
    (dict(kind=tsa.MASK_CAUSAL_SLIDING), tsa.ATTN_ERR_UNSUPPORTED), (dict(kind=tsa.MASK_SLIDING), tsa.ATTN_ERR_UNSUPPORTED),
    (dict(kind=9), BAD), (dict(B=0), BAD), (dict(Hq=3), BAD), (dict(S_q=0), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(d=96), tsa.ATTN_ERR_UNSUPPORTED), (dict(B=1025), tsa.ATTN_ERR_UNSUPPORTED),
    (dict(S_q=33), tsa.ATTN_ERR_UNSUPPORTED)])
def test_prefix_create_refuses(kw, status):
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_prefix_create(**{**dict(B=2, Hq=4, Hkv=2, S_q=1, d=64, scale=0.1, kind=tsa.MASK_CAUSAL), **kw})
    assert e.value.status == status


def test_prefix_arguments_are_refused():
    assert tsa.attn_prefix_forward(0, 0, 16, 16, 1, 1, 16, 1, 0, 16, 1, 1, 16, 16) == BAD
    assert tsa.attn_prefix_set_grid_limit(0, 1) == BAD and tsa.attn_prefix_set_watchdog(0, 1) == BAD
    assert tsa.attn_prefix_destroy(0) == tsa.ATTN_OK
