"""Host side of the rotary, paged-cache and paged-decode entry points (no GPU): refusals, frequencies, the split."""
import numpy as np
import pytest

import paged_util as pu
import transformer_self_attention_gb300 as tsa


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), tsa.ATTN_ERR_INVALID_ARG), (dict(rot=3), tsa.ATTN_ERR_INVALID_ARG),
    (dict(rot=66), tsa.ATTN_ERR_INVALID_ARG), (dict(layout=2), tsa.ATTN_ERR_INVALID_ARG),
    (dict(scaling=4), tsa.ATTN_ERR_INVALID_ARG), (dict(base=1.0), tsa.ATTN_ERR_INVALID_ARG),
    (dict(base=float("nan")), tsa.ATTN_ERR_INVALID_ARG), (dict(scaling=1, factor=0.5), tsa.ATTN_ERR_INVALID_ARG),
    (dict(scaling=2, factor=2.0, rot=2), tsa.ATTN_ERR_INVALID_ARG),
    (dict(scaling=3, factor=2.0), tsa.ATTN_ERR_INVALID_ARG),  # no original length
    (dict(scaling=3, factor=2.0, original_len=8, beta_fast=1.0), tsa.ATTN_ERR_INVALID_ARG),
    (dict(amplitude=-1.0), tsa.ATTN_ERR_INVALID_ARG), (dict(d=72, rot=8), tsa.ATTN_ERR_UNSUPPORTED),
    (dict(d=272, rot=8), tsa.ATTN_ERR_UNSUPPORTED), (dict(d=0, rot=2), tsa.ATTN_ERR_INVALID_ARG)])
def test_rope_create_refuses(kw, status):
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_rope_create(**{**dict(d=64, rot=64), **kw})
    assert e.value.status == status


def test_rope_binding_refuses():
    for kw in (dict(layout="neox"), dict(scaling="dynamic"), dict(amplitude=0.0)):
        with pytest.raises(ValueError):
            tsa.RotaryPositions(64, **kw)


@pytest.mark.parametrize("rot,kw", [(64, {}), (26, dict(base=500000.0)), (2, dict(scaling="linear", factor=2.0)),
                                    (128, dict(scaling="ntk", factor=7.5)),
                                    (64, dict(scaling="yarn", factor=4.0, original_len=4096)),
                                    (64, dict(scaling="yarn", factor=16.0, original_len=100, beta_fast=8.0, beta_slow=0.25))])
def test_frequencies(rot, kw):
    f, amp = tsa.RotaryPositions(128, rot, **kw).frequencies()
    want, amp_want = pu.frequencies(rot, **kw)
    assert np.allclose(f, want.numpy(), rtol=1e-13, atol=0) and abs(amp - amp_want) < 1e-13
    assert tsa.RotaryPositions(128, rot, amplitude=0.5, **kw).frequencies()[1] == 0.5


def test_null_handles_and_pointers_are_refused():
    r = tsa.attn_rows(16, 64, 64, 64)
    bad = tsa.ATTN_ERR_INVALID_ARG
    assert tsa.attn_rope_forward(0, tsa.ATTN_BF16, 1, 1, 1, r, r) == bad
    h = tsa.attn_rope_create(64, 64)
    assert tsa.attn_rope_forward(h, tsa.ATTN_FP8_E4M3, 1, 1, 1, r, r) == bad
    assert tsa.attn_rope_forward(h, tsa.ATTN_BF16, 1, 1, 1, None, r) == bad
    assert tsa.attn_rope_forward(h, tsa.ATTN_BF16, 1, 1, 1, r, tsa.attn_rows(8, 64, 64, 64)) == bad
    assert tsa.attn_rope_forward(h, tsa.ATTN_BF16, 1, 1, 1, tsa.attn_rows(16, 64, 4, 64), r) == bad
    assert tsa.attn_rope_forward(h, tsa.ATTN_BF16, 1, 1, 1, r, r, Hk=1) == bad
    assert tsa.attn_rope_backward(h, tsa.ATTN_F32, 0, 1, 1, r, r) == bad
    assert tsa.attn_rope_forward(h, tsa.ATTN_BF16, 1, 0, 1, None, None) == tsa.ATTN_OK  # nothing to do
    assert tsa.attn_rope_destroy(h) == tsa.ATTN_OK and tsa.attn_rope_destroy(0) == tsa.ATTN_OK
    assert tsa.attn_cache_write(0, 1, 1, r, r, 16, 1, 1, 16) == bad
    assert tsa.attn_cache_read(0, 1, 1, 0, r, r, 16, 1, 1, 16) == bad
    assert tsa.attn_paged_forward(0, 0, 16, 16, 1, 1, 16, 16) == bad
    assert tsa.attn_cache_destroy(0) == tsa.ATTN_OK and tsa.attn_paged_destroy(0) == tsa.ATTN_OK


@pytest.mark.parametrize("args,status", [
    ((0, 1, 16, 64, tsa.ATTN_BF16, 16), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 1, 24, 64, tsa.ATTN_BF16, 16), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 1, 16, 64, tsa.ATTN_BF16, 0), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 1, 16, 64, tsa.ATTN_BF16, 8), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 1, 16, 64, tsa.ATTN_FP8_E4M3, 16), tsa.ATTN_ERR_INVALID_ARG),  # no scales
    ((1, 1, 16, 64, tsa.ATTN_F32, 16), tsa.ATTN_ERR_UNSUPPORTED),
    ((1, 1, 16, 96, tsa.ATTN_BF16, 16), tsa.ATTN_ERR_UNSUPPORTED),
    ((1, 1, 2048, 64, tsa.ATTN_BF16, 16), tsa.ATTN_ERR_UNSUPPORTED),
    ((1 << 30, 4, 16, 64, tsa.ATTN_BF16, 16), tsa.ATTN_ERR_UNSUPPORTED)])
def test_cache_create_refuses(args, status):
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_cache_create(*args)
    assert e.value.status == status


@pytest.mark.parametrize("args,status", [
    ((1, 4, 3, 1, 64, 1.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_INVALID_ARG),
    ((0, 4, 4, 1, 64, 1.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 4, 4, 1, 64, 0.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 4, 4, 1, 64, 1.0, 9), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 4, 4, 1, 64, 1.0, tsa.MASK_CAUSAL_SLIDING, -1), tsa.ATTN_ERR_INVALID_ARG),
    ((1, 4, 4, 1, 96, 1.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_UNSUPPORTED),
    ((1, 4, 4, 1, 64, 1.0, tsa.MASK_LOCAL_GLOBAL), tsa.ATTN_ERR_UNSUPPORTED),
    ((1, 65, 1, 1, 64, 1.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_UNSUPPORTED),
    ((1025, 4, 4, 1, 64, 1.0, tsa.MASK_CAUSAL), tsa.ATTN_ERR_UNSUPPORTED)])
def test_paged_create_refuses(args, status):
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_paged_create(*args)
    assert e.value.status == status


def test_split_refuses_a_cost_line_beyond_31_bits():
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_paged_split_host(1024, 64, 1, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL, 0, [1 << 24] * 1024, 304)
    assert e.value.status == tsa.ATTN_ERR_UNSUPPORTED


def test_split_of_the_widest_windows_and_lengths():
    """Differences of positions stay within 32 bits: the widest window sees everything, also in front of position 0."""
    for S_q in (1, 64):
        n_cta, parts = tsa.attn_paged_split_host(2, 1, S_q, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL_SLIDING, 2 ** 31 - 1,
                                                 [1, 100], 304)
        assert parts[:, 5].tolist() == [1, 7] and parts[:, 3].tolist() == [0, 0]
    n_cta, parts = tsa.attn_paged_split_host(1, 1, 1, 128, tsa.ATTN_FP8_E4M3, tsa.MASK_CAUSAL, 0, [1 << 30], 304)
    assert n_cta == 304 and int(parts[:, 4].max()) == 1 << 23
    for lens, status in (([(1 << 30) + 1], tsa.ATTN_ERR_UNSUPPORTED), ([-1], tsa.ATTN_ERR_INVALID_ARG)):
        with pytest.raises(tsa.AttnError) as e:
            tsa.attn_paged_split_host(1, 1, 1, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL, 0, lens, 304)
        assert e.value.status == status
    with pytest.raises(tsa.AttnError) as e:
        tsa.attn_paged_split_host(1, 1, 65, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL, 0, [1], 304)
    assert e.value.status == tsa.ATTN_ERR_UNSUPPORTED
    with pytest.raises(ValueError):  # fewer lengths than sequences
        tsa.attn_paged_split_host(3, 1, 1, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL, 0, [1], 304)


def test_numbers_beyond_32_bits_are_refused():
    for call in (lambda: tsa.RotaryPositions(64, rotary_dim=(1 << 32) + 32),
                 lambda: tsa.attn_rope_create(64, 64, scaling=3, factor=2.0, original_len=1 << 32),
                 lambda: tsa.attn_paged_create(1, 1, 1, 1, 64, 1.0, tsa.MASK_CAUSAL_SLIDING, 1 << 32),
                 lambda: tsa.attn_cache_create(1, 1, (1 << 32) + 16, 64, tsa.ATTN_BF16, 16)):
        with pytest.raises(ValueError):
            call()


def test_short_units_are_not_cut():
    """As many CTAs as units, one whole unit each, while the grid is large enough."""
    for lens in ([100], [1, 256, 17, 0, 90]):
        n_cta, parts = tsa.attn_paged_split_host(len(lens), 8, 1, 128, tsa.ATTN_BF16, tsa.MASK_CAUSAL, 0, lens, 304)
        assert n_cta == len(parts) == 8 * sum(n > 0 for n in lens)
        assert all(p[3] == 0 and p[4] == p[5] for p in parts.tolist())


def _cases():
    rng = np.random.default_rng(5)
    yield [0, 0, 0], 2, tsa.MASK_CAUSAL, 0, 152
    yield [1], 1, tsa.MASK_CAUSAL, 0, 152
    yield [100], 8, tsa.MASK_CAUSAL, 0, 152
    yield [1 << 20, 5, 0, 1 << 20], 8, tsa.MASK_CAUSAL, 0, 152
    yield [1 << 20] * 500, 50, tsa.MASK_CAUSAL, 0, 304  # a cost line of more than 2^30
    for _ in range(60):
        B = int(rng.integers(1, 60))
        lens = (rng.integers(0, 2, B) * np.exp(rng.uniform(0, 10, B))).astype(int).tolist()
        kind = [tsa.MASK_FULL, tsa.MASK_CAUSAL, tsa.MASK_CAUSAL_SLIDING][rng.integers(3)]
        yield lens, int(rng.integers(1, 9)), kind, int(rng.integers(0, 3000)), int(rng.integers(1, 305))


@pytest.mark.parametrize("lens,Hkv,kind,window,grid", list(_cases()))
@pytest.mark.parametrize("d,dtype", [(128, tsa.ATTN_BF16), (64, tsa.ATTN_FP8_E4M3)])
def test_split_covers_every_block_once(lens, Hkv, kind, window, grid, d, dtype):
    """Every visible key block of every unit in exactly one part; the CTAs named as a unit's first and last are those
    that hold its blocks, without a gap; a CTA leaves at most two units unfinished, which have different slots."""
    n_cta, parts = tsa.attn_paged_split_host(len(lens), Hkv, 1, d, dtype, kind, window, lens, grid)
    keys = {(128, tsa.ATTN_BF16): 16, (64, tsa.ATTN_FP8_E4M3): 128}[(d, dtype)]
    assert 0 <= n_cta <= grid
    want = {}
    for b, n in enumerate(lens):
        lo = max(0, n - 1 - window) // keys if kind == tsa.MASK_CAUSAL_SLIDING else 0
        if n:
            for h in range(Hkv):
                want[(b, h)] = -(-n // keys) - lo
    got, slots = {}, {}
    for cta, b, h, g0, g1, n, k0, k1 in parts.tolist():
        assert want[(b, h)] == n and 0 <= g0 < g1 <= n and 0 <= cta < n_cta
        got.setdefault((b, h), []).append((g0, g1, cta, k0, k1))
        if (g0, g1) != (0, n):
            slot = 2 * cta + (0 if g0 else 1)
            assert slot not in slots
            slots[slot] = (b, h)
            assert slot == 2 * cta + (cta == k0)  # how the joining CTA finds it
    assert set(got) == set(want)
    for unit, pieces in got.items():
        pieces.sort()
        assert pieces[0][0] == 0 and pieces[-1][1] == want[unit]
        assert all(a[1] == b[0] for a, b in zip(pieces, pieces[1:]))
        assert [p[2] for p in pieces] == list(range(pieces[0][3], pieces[0][4] + 1))
