"""Plain float64 forms of the operators for long contexts over a paged cache."""
import math

import torch

import paged_util as pu


def power(big):
    """The smallest k >= -126 with big <= 127 * 2^k (a python float)."""
    if big == 0:
        return -126
    k = math.ceil(math.log2(big / 127.0))
    while big > 127.0 * 2.0 ** k:
        k += 1
    while big <= 127.0 * 2.0 ** (k - 1):
        k -= 1
    return max(k, -126)


def bounds(vals, table, page, b, n, i):
    """(codes int8 [Hkv, 2, d], exponent bytes [Hkv]) of page i of sequence b with n positions; vals: paged_util.values."""
    x = vals[int(table[b, i]), :, 0, :min(page, n - i * page)]  # [Hkv, rows, d]
    Hkv, _, d = x.shape
    codes, exps = torch.zeros((Hkv, 2, d), dtype=torch.int8), torch.zeros(Hkv, dtype=torch.uint8)
    for h in range(Hkv):
        if not bool(torch.isfinite(x[h]).all()) or float(x[h].abs().max()) >= 2.0 ** 128:
            exps[h] = 255
            continue
        k = power(float(x[h].abs().max()))
        codes[h, 0] = torch.floor(x[h].amin(0) * 2.0 ** -k).to(torch.int8)
        codes[h, 1] = torch.ceil(x[h].amax(0) * 2.0 ** -k).to(torch.int8)
        exps[h] = k + 127
    return codes, exps


def select(Q, codes, exps, table, page, lens, keep, sinks, recent):
    """(chosen places [B][Hkv] lists, lengths): the definition in whole numbers."""
    B, Hq, S_q, d = Q.shape
    Hkv = codes.shape[1]
    chosen, out_len = [], []
    for b, n in enumerate(lens):
        pages = -(-n // page)
        out_len.append(n - max(0, pages - keep) * page)
        rows = []
        for h in range(Hkv):
            if pages <= keep:
                rows.append(list(range(pages)))
                continue
            q = Q[b].double().view(Hkv, -1, d)[h]
            if bool(torch.isfinite(q).all()):
                r = torch.round(q * 2.0 ** -power(float(q.abs().max())))
            else:
                r = torch.zeros_like(q)
            scores = []
            for i in range(sinks, pages - recent):
                g = int(table[b, i])
                c = codes[g, h].double()
                s = torch.maximum(r * c[0], r * c[1]).sum(-1).max()
                e = int(exps[g, h])
                scores.append((-math.inf if e == 255 else -float(s) * 2.0 ** (e - 127), i))
            best = sorted(i for _, i in sorted(scores)[:keep - sinks - recent])
            rows.append(list(range(sinks)) + best + list(range(pages - recent, pages)))
        chosen.append(rows)
    return chosen, out_len


def decode_chosen(Q, vals, table, page, lens, chosen, scale):
    """paged_util.decode's results (causal) over the chosen pages of each sequence and head."""
    B, Hq, S_q, d = Q.shape
    Hkv = vals.shape[1]
    outs = []
    for h in range(Hkv):
        group = Hq // Hkv
        wide = max([len(chosen[b][h]) for b in range(B)] + [1])
        tab = torch.zeros((B, wide), dtype=torch.int32)
        short = []
        for b, n in enumerate(lens):
            c = chosen[b][h]
            tab[b, :len(c)] = table[b][torch.tensor(c, dtype=torch.long)] if c else tab[b, :0]
            short.append(n - (-(-n // page) - len(c)) * page)
        outs.append(pu.decode(Q[:, h * group:(h + 1) * group], vals[:, h:h + 1], tab, page, short, scale, 1, 0))
    return tuple(torch.cat([o[i] for o in outs], dim=1) for i in range(4))


def weigh(Q, LSE, W, vals, table, page, lens, scale, kind, window, decay):
    """W [n_pages, Hkv, page] after a step (float64), and a bound on its float32 errors."""
    B, Hq, S_q, d = Q.shape
    Hkv = vals.shape[1]
    out, bound = W.double().clone(), torch.zeros(W.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, _ = pu.dense(vals, table, page, b, n)  # [Hkv, n, d]
        q = Q[b].double().view(Hkv, -1, S_q, d)
        lse = LSE[b].double().view(Hkv, -1, S_q)
        j = torch.arange(n)
        p, slot = table[b].long()[j // page], j % page
        held = (p >= 0) & (p < W.shape[0])  # (pages before every row's window may be gone: nobody's weights)
        p = p.clamp(0, W.shape[0] - 1)
        new = out[p, :, slot].T * decay  # [Hkv, n]
        new[:, max(0, n - S_q):] = 0
        err = new.abs() * 2.0 ** -24
        for i in range(S_q):
            t = n - S_q + i
            hi = n if kind == 0 else t + 1
            lo = max(0, t - window) if kind == 3 else 0
            if hi <= lo:
                continue
            s = torch.einsum("hgd,hjd->hgj", q[:, :, i], K[:, lo:hi]) * scale
            big = torch.einsum("hgd,hjd->hgj", q[:, :, i].abs(), K[:, lo:hi].abs()) * scale
            x = lse[:, :, i, None]
            live = x > -math.inf
            w = torch.where(live, torch.exp(s - torch.where(live, x, torch.zeros_like(x))), torch.zeros_like(s))
            # float32 sums of d products and the exponent's rounding: d + 8 half steps of what they are made of;
            # exp2 two more, and the sum over the rows one each
            r = (big * (d + 8) + torch.where(live, x.abs(), torch.zeros_like(x)) * 2) * 2.0 ** -23 + (2 + Hq * S_q) * 2.0 ** -24
            new[:, lo:hi] += w.sum(1)
            err[:, lo:hi] += (w * r).sum(1)
        p, slot = p[held], slot[held]
        out[p, :, slot] = new.T[held]
        bound[p, :, slot] = err.T[held] + out[p, :, slot].abs() * 2.0 ** -23
    return out, bound


def evict(W, table, page, lens, keep, recent):
    """Old positions [B][Hkv] of the positions that stay."""
    out = []
    for b, n in enumerate(lens):
        rows = []
        for h in range(W.shape[1]):
            old = max(0, n - recent)
            w = [float(W[int(table[b, i // page]), h, i % page]) for i in range(old)]
            key = [-math.inf if math.isnan(x) else -x for x in w]
            nan_first = sorted(range(old), key=lambda i: (not math.isnan(w[i]), key[i], i))
            rows.append(sorted(nan_first[:keep]) + list(range(old, n)) if n > keep + recent else list(range(n)))
        out.append(rows)
    return out
