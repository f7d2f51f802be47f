"""Rotary positions on the GPU against the float64 definition, the gradient against it and against differences."""
import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


def _pair(B, Hq, Hk, S, d, dtype, packed, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, S, Hq + Hk, d), generator=g).to(dtype).cuda()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    return (q, k) if packed else (q.contiguous(), k.contiguous())


def _check(rope, kw, rot, layout, Q, K, positions, back=False, **out):
    f, amp = pu.frequencies(rot, **kw)
    B, S = Q.shape[0], Q.shape[2]
    pos = torch.arange(S)[None].expand(B, S) if positions is None else positions.cpu().expand(B, S)
    refs = [pu.rotate(t, pos, rot, layout, f, amp, -1.0 if back else 1.0) for t in (Q, K) if t is not None]
    got = (rope.backward if back else rope)(Q, K, positions, **out)
    got = [got] if K is None else list(got)
    torch.cuda.synchronize()
    for y, (ref, size) in zip(got, refs):
        assert y.dtype == Q.dtype
        off = (y.double().cpu() - ref).abs() - pu.rope_bound(ref, size, Q.dtype)
        assert float(off.max()) <= 0, float(off.max())
        keep = ref[..., rot:]
        assert torch.equal(y.double().cpu()[..., rot:], keep)  # what is not rotated is copied
    return got


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 26), (128, 128), (128, 64), (128, 2), (128, 96), (16, 16), (48, 24),
                                   (80, 32), (256, 256), (240, 122)])
def test_widths_layouts_and_types(layout, dtype, d, rot):
    Q, K = _pair(2, 3, 2, 37, d, dtype, packed=True)
    rope = tsa.RotaryPositions(d, rot, layout=layout)
    for back in (False, True):
        _check(rope, {}, rot, layout, Q, K, None, back)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=4.0, original_len=2048),
                                dict(scaling="yarn", factor=1.0, original_len=1, beta_fast=4.0, beta_slow=0.5),
                                dict(base=500000.0)])
def test_scalings_and_far_positions(kw):
    Q, K = _pair(3, 4, 1, 5, 128, torch.float32, packed=False, seed=3)
    pos = torch.tensor([[0, 1, 2, 3, 4], [1 << 20, (1 << 20) + 1, 131071, 7, 1], [-3, 2 ** 31 - 1, -2 ** 31, 5, 6]],
                       dtype=torch.int32).cuda()
    rope = tsa.RotaryPositions(128, **kw)
    f, amp = rope.frequencies()
    ref, amp_ref = pu.frequencies(128, **kw)
    assert abs(amp - amp_ref) < 1e-12 and float((torch.tensor(f) / ref - 1).abs().max()) < 1e-13
    # the angle itself is known to 2^-52 of its size in the float64 reference: 2^31 * 2^-52 = 5e-7 rad, so the far
    # positions are compared against frequencies reduced exactly (a multiple of a turn more, on integers)
    from fractions import Fraction
    import math
    turn = Fraction(2 ** 64)
    B, H, S, d = Q.shape
    for t, y in zip((Q, K), rope(Q, K, pos)):
        x, y = t.double().cpu(), y.double().cpu()
        for b in range(B):
            for s in range(S):
                step = [int(math.ldexp(float(v) / (2 * math.pi), 64)) for v in f]
                ang = torch.tensor([float(Fraction((int(pos[b, s]) * st) % 2 ** 64) / turn) * 2 * math.pi for st in step],
                                   dtype=torch.float64)
                c, sn = torch.cos(ang) * amp, torch.sin(ang) * amp
                a, e = x[b, :, s, :d // 2], x[b, :, s, d // 2:]
                want = torch.cat([a * c - e * sn, a * sn + e * c], -1)
                size = torch.cat([(a.abs() + e.abs()) * amp] * 2, -1)
                assert float(((y[b, :, s] - want).abs() - pu.rope_bound(want, size, torch.float32)).max()) <= 0


@pytest.mark.parametrize("B,Hq,Hk,S", [(1, 1, 1, 1), (8, 64, 8, 1), (256, 4, 1, 1), (1, 5, 3, 700), (3, 33, 0, 129)])
@pytest.mark.parametrize("packed", [True, False])
def test_sizes_and_broadcast_positions(B, Hq, Hk, S, packed):
    Q, K = _pair(B, Hq, max(1, Hk), S, 128, torch.bfloat16, packed, seed=1)
    if Hk == 0:
        K = None
    rope = tsa.RotaryPositions(128)
    pos = torch.randint(0, 40000, (S,), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    _check(rope, {}, 128, "half", Q, K, pos)
    each = (torch.arange(B, dtype=torch.int32)[:, None] * 100 + torch.arange(S, dtype=torch.int32)).cuda()
    _check(rope, {}, 128, "half", Q, K, each)
    wide = torch.zeros((B, 2 * S), dtype=torch.int32, device="cuda")[:, ::2]
    wide.copy_(each)
    _check(rope, {}, 128, "half", Q, K, wide)  # strided positions


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 26), ("interleaved", 64)])
def test_in_place_and_strided_outputs(layout, rot):
    Q, K = _pair(2, 6, 2, 45, 128, torch.bfloat16, packed=True, seed=2)
    rope = tsa.RotaryPositions(128, rot, layout=layout)
    want = rope(Q, K)
    qkv = torch.full((2, 45, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = rope(Q, K, Q_out=qkv[:, :, :6].transpose(1, 2), K_out=qkv[:, :, 6:8].transpose(1, 2))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((qkv[:, :, 8:] == 7).all())  # nothing beside the rows is written
    rope(Q, K, Q_out=Q, K_out=K)
    assert torch.equal(Q, want[0]) and torch.equal(K, want[1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """The map is linear: <dy, R x1 - R x0> = <R^T dy, x1 - x0> up to the roundings of both sides."""
    rope = tsa.RotaryPositions(64, 48, layout=layout, scaling="yarn", factor=3.0, original_len=64)
    g = torch.Generator().manual_seed(9)
    x0, x1, dy = (torch.randn((1, 2, 9, 64), generator=g).cuda() for _ in range(3))
    dx = rope.backward(dy)
    y0, y1 = rope(x0), rope(x1)
    for h in range(2):
        for s in range(9):
            lhs = (dy * (y1 - y0))[0, h, s].double().sum()
            rhs = (dx * (x1 - x0))[0, h, s].double().sum()
            size = ((dy.abs() * (y0.abs() + y1.abs()))[0, h, s].sum() + (dx.abs() * (x1 - x0).abs())[0, h, s].sum())
            assert abs(float(lhs - rhs)) <= float(size) * 2.0 ** -18


@pytest.mark.parametrize("layout,d,rot", [("half", 128, 64), ("half", 64, 26), ("interleaved", 128, 64),
                                          ("interleaved", 64, 26)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_elements_that_are_not_finite_stay_in_their_pair(layout, d, rot, bad):
    """One in a pair makes that pair not finite; one behind the rotated elements is copied, and touches nothing else."""
    Q, K = _pair(1, 2, 1, 6, d, torch.bfloat16, packed=False, seed=9)
    Q[0, 0, 2, rot + 1] = bad
    Q[0, 1, 3, d - 2] = bad
    Q[0, 1, 4, 2] = bad  # of the pair (2, 2 + rot / 2), or (2, 3)
    rope = tsa.RotaryPositions(d, rot, layout=layout)
    for got in (rope(Q, K)[0], rope.backward(Q, K)[0]):
        odd = ~torch.isfinite(got)
        want = torch.zeros_like(odd)
        want[0, 0, 2, rot + 1] = want[0, 1, 3, d - 2] = True
        want[0, 1, 4, 2] = want[0, 1, 4, 2 + rot // 2 if layout == "half" else 3] = True
        assert torch.equal(odd, want)
        kept = got[..., rot:]
        assert torch.equal(torch.nan_to_num(kept, nan=7.0), torch.nan_to_num(Q[..., rot:], nan=7.0))


def test_empty_and_other_stream():
    rope = tsa.RotaryPositions(64)
    q = torch.empty((2, 3, 0, 64), dtype=torch.bfloat16, device="cuda")
    assert rope(q).shape == q.shape
    assert rope(torch.empty((0, 3, 5, 64), device="cuda")).shape == (0, 3, 5, 64)
    Q, K = _pair(2, 4, 4, 300, 64, torch.bfloat16, packed=False)
    want = rope(Q, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rope(Q, K, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_call_follows_its_positions():
    rope = tsa.RotaryPositions(128)
    Q, K = _pair(4, 8, 2, 1, 128, torch.bfloat16, packed=False)
    pos = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    Qo, Ko = torch.empty_like(Q), torch.empty_like(K)
    rope(Q, K, pos, Qo, Ko)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope(Q, K, pos, Qo, Ko)
    for p in (5, 70000):
        pos.fill_(p)
        graph.replay()
        want = rope(Q, K, pos)
        assert torch.equal(Qo, want[0]) and torch.equal(Ko, want[1])


def test_refusals():
    rope = tsa.RotaryPositions(64)
    Q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (Q.half(), Q[..., :32], Q.cpu(), torch.zeros((2, 4, 64, 8), device="cuda").transpose(2, 3)):
        with pytest.raises((ValueError, tsa.AttnError)):
            rope(bad)
    with pytest.raises(ValueError):
        rope(Q, Q[:1])
    with pytest.raises(ValueError):
        rope(Q, positions=torch.zeros((2, 8), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        rope(Q, positions=torch.zeros((2, 7), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):  # no query heads
        rope(Q[:, :0], Q)
    odd = torch.zeros(2 * 4 * 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4, 8, 64)
    with pytest.raises(tsa.AttnError) as e:  # rows off the 16-byte grid
        rope(odd)
    assert e.value.status == tsa.ATTN_ERR_INVALID_ARG
    with pytest.raises(tsa.AttnError):
        rope(torch.zeros((2, 4, 8, 68), dtype=torch.bfloat16, device="cuda")[..., :64])
