"""Plain float64 forms of the rotary, paged-cache and paged-decode operators, and builders of paged inputs."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(float64 [rot / 2], amplitude)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for p in range(rot // 2):
        f = base ** (-2.0 * p / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            r = original_len * f / (2 * math.pi)
            g = min(1.0, max(0.0, (r - beta_slow) / (beta_fast - beta_slow)))
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rotate(x, positions, rot, layout, freq, amp, sign=1.0):
    """x [B, H, S, d] turned by positions [B, S]; float64, and the bound (|a| + |b|) amp of each element's terms."""
    x = x.double().cpu()
    angle = sign * positions.double().cpu()[:, None, :, None] * freq
    c, s = torch.cos(angle) * amp, torch.sin(angle) * amp
    i = torch.arange(rot // 2)
    first, second = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., first], x[..., second]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * amp
    return y, size


def rope_bound(y, size, dtype):
    """|error| of a rotated element: cos and sin carry the float rounding of the angle in half turns (pi 2^-24),
    its cut at 2^-32 turns (1.5e-9) and sincospi's error (2^-23), the products and the sum three roundings; together
    under 2^-20 of the terms' size.  Then the rounding to the output type."""
    return y.abs() * EPS[dtype] + size * 2.0 ** -20


def quantise(x):
    """(codes uint8, exponent bytes uint8) of the rows of x (float32 CPU): the definition of an E4M3 cache row."""
    big = x.abs().amax(dim=-1)
    finite = torch.isfinite(x).all(dim=-1)
    m, e = torch.frexp(torch.where(finite, big, torch.ones_like(big)))  # 1/2 <= m < 1; 448 = 7/8 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    k = torch.where(big == 0, torch.full_like(k, -127), k)
    codes = (x.double() * torch.exp2(-k.double())[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(finite[..., None], codes, torch.full_like(codes, 0x7F))
    return codes, torch.where(finite, k + 127, torch.full_like(k, 255)).to(torch.uint8)


def values(pages, scales):
    """What a cache's rows stand for, float64 [n_pages, Hkv, 2, page, d] (CPU)."""
    x = pages.cpu().double()
    if scales is not None:
        e = scales.cpu().transpose(2, 3).reshape(x.shape[:-1]).double()
        x = x * torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))[..., None]
    return x


def make_pool(lens, Hkv, page, d, store, seed=0, spare=2, k_scale=1.0, window_first=None, v_spread=0.0):
    """(pages, scales, table, n_pages): CPU tensors; K and V of every position normal, every slot behind a length
    and every free page poisoned (NaN), unneeded table entries out of range.  window_first[b]: positions before it
    are poisoned too, their whole pages released (entries out of range).  v_spread: the value rows' sizes vary by
    e^(v_spread N(0, 1))."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
    table[:, -1] = 2 ** 30
    order = torch.randperm(n_pages, generator=g).tolist()
    x = torch.full((n_pages, Hkv, 2, page, d), math.nan)
    at = 0
    for b, n in enumerate(lens):
        first = window_first[b] if window_first else 0
        for i in range(need[b]):
            p = order[at]
            at += 1
            lo, hi = max(0, first - i * page), min(page, n - i * page)
            if hi <= lo:
                continue
            table[b, i] = p
            x[p, :, :, lo:hi] = torch.randn((Hkv, 2, hi - lo, d), generator=g)
            x[p, :, 0, lo:hi] *= k_scale
            if v_spread:
                x[p, :, 1, lo:hi] *= torch.exp(v_spread * torch.randn((Hkv, hi - lo, 1), generator=g))
    if store == "bf16":
        return x.to(torch.bfloat16), None, table, n_pages
    codes, e = quantise(x)
    e = e.view(n_pages, Hkv, 2, page // 16, 16).transpose(2, 3).contiguous()
    return codes.view(torch.float8_e4m3fn), e, table, n_pages


def dense(vals, table, page, b, n):
    """K and V [Hkv, n, d] of the first n positions of sequence b (rows of released pages come back as NaN)."""
    j = torch.arange(n)
    p = table[b].long()[j // page]
    ok = (p >= 0) & (p < vals.shape[0])
    x = vals[p.clamp(0, vals.shape[0] - 1), :, :, j % page]
    x[~ok] = math.nan
    return x[:, :, 0].transpose(0, 1), x[:, :, 1].transpose(0, 1)


def decode(Q, vals, table, page, lens, scale, kind, window):
    """Paged decode in float64 (kind: 0 full, 1 causal, 3 causal window).  Returns O, LSE, A (the weighted mean of
    |v|) and E (the largest sum scale |q_e k_e| over the visible keys), which bound the kernel's errors."""
    B, Hq, S_q, d = Q.shape
    Hkv = vals.shape[1]
    q = Q.double().cpu().view(B, Hkv, Hq // Hkv, S_q, d)
    O = torch.zeros(q.shape, dtype=torch.float64)
    A = torch.zeros_like(O)
    L = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64)
    E = torch.zeros(q.shape[:-1], dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, V = dense(vals, table, page, b, n)
        for i in range(S_q):
            t = n - S_q + i
            hi = n if kind == 0 else t + 1
            lo = max(0, t - window) if kind == 3 else 0
            if hi <= lo:
                continue
            k, v = K[:, lo:hi], V[:, lo:hi]
            s = torch.einsum("hgd,hjd->hgj", q[b, :, :, i], k) * scale
            E[b, :, :, i] = torch.einsum("hgd,hjd->hgj", q[b, :, :, i].abs(), k.abs()).amax(-1) * scale
            L[b, :, :, i] = torch.logsumexp(s, -1)
            p = torch.exp(s - L[b, :, :, i][..., None])
            O[b, :, :, i] = torch.einsum("hgj,hjd->hgd", p, v)
            A[b, :, :, i] = torch.einsum("hgj,hjd->hgd", p, v.abs())
    shape = (B, Hq, S_q)
    return O.view(*shape, d), L.view(shape), A.view(*shape, d), E.view(shape)


def coarse_weights(Q, vals, factors, table, page, lens, scale):
    """The second part of the weights' rounding over E4M3 pages, per row [B, Hq, S_q] (causal): a weight of one of 128
    positions is also off by 2^-22 of their largest weight times their largest value factor, times codes up to 448."""
    B, Hq, S_q, d = Q.shape
    Hkv = vals.shape[1]
    q = Q.double().cpu().view(B, Hkv, Hq // Hkv, S_q, d)
    out = torch.zeros(q.shape[:-1], dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, _ = dense(vals, table, page, b, n)
        j = torch.arange(n)
        f = factors[table[b].long()[j // page], :, 1, j % page].transpose(0, 1)  # [Hkv, n]
        for i in range(S_q):
            hi = n - S_q + i + 1
            if hi <= 0:
                continue
            p = torch.softmax(torch.einsum("hgd,hjd->hgj", q[b, :, :, i], K[:, :hi]) * scale, -1)
            for t in range(0, n, 128):
                if t < hi:
                    out[b, :, :, i] += 128 * 448 * 2.0 ** -22 * p[:, :, t:t + 128].amax(-1) * f[:, t:t + 128].amax(-1)[:, None]
    return out.view(B, Hq, S_q)


def check_decode(O, LSE, ref, d, more=None):
    """Elementwise bounds.  Scores: a float32 sum of d products, off by d 2^-24 of their absolute sum at most; exp2's
    argument and result a few 2^-23 of |score| log2 e and of itself, and the weights' float32 sum (errors of the same
    kind, in the mean) under 2^-19; so a weight is off by r = E (d + 8) 2^-23 + 2^-19 relative.  Weights are rounded
    to bf16 (2^-8), O once more."""
    O_ref, L_ref, A, E = ref
    O, LSE = O.double().cpu(), LSE.double().cpu()
    r = E * (d + 8) * 2.0 ** -23 + 2.0 ** -19
    assert torch.equal(torch.isneginf(LSE), torch.isneginf(L_ref))
    seen = ~torch.isneginf(L_ref)
    assert bool((O[~seen] == 0).all())
    assert bool(torch.isfinite(O).all()) and bool(torch.isfinite(LSE[seen]).all())
    bound = O_ref.abs() * 2.0 ** -8 + A * (2.0 ** -8 + 2 * r[..., None]) * (1 + 2.0 ** -7)
    if more is not None:
        bound = bound + more[..., None]
    bad = (O - O_ref).abs() - bound
    assert float(bad.max()) <= 0, f"O off by {float((O - O_ref).abs().max()):.3e}, {float(bad.max()):.3e} past its bound"
    off = (LSE - L_ref)[seen].abs() - (r[seen] + L_ref[seen].abs() * 2.0 ** -22)
    assert float(off.max()) <= 0 if off.numel() else True, f"LSE {float(off.max()):.3e} past its bound"
