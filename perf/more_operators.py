"""Operators for long contexts over a paged cache, in their plain form and as the library's calls.

Ways to read or hold less of a long context, over the pages that decode attention reads:

prefix   attention for a batch whose sequences share long prefixes: a prefix is read once for all of its
         sequences, and joined with what each of them holds for itself
sparse   attention over the pages that a cheap score selects for the new rows of a sequence and kv head: bounds of
         each page's keys (8-bit codes with a power of two), the largest score that they allow, the best pages
weigh    the attention weight that each cached position receives, summed over rows, heads of a group and steps
evict    the positions of largest weight, and the latest ones, moved to the front of other pages

``run`` with ``own`` false computes them from elementary torch operations in float32; with ``own`` true it makes the
library's calls.

Layout of a paged cache: pages [n_pages, Hkv, 2, page, d], keys at index 0 and values at index 1;
position j of sequence b is slot j % page of the page page_table[b, j // page].  An E4M3 cache holds
8-bit codes c and, per row of d codes, a biased exponent e (uint8, scales [n_pages, Hkv, page / 16,
2, 16]); the row stands for c * 2^(e - 127).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # A few users behind one short system prompt: the smallest call, its latency counts.
        _prefix("prefix_short", B=4, Hq=32, Hkv=8, S_q=1, d=128, page=16, prefix=500, own_min=1, own_max=60),
        # A long document that a batch of conversations asks about: the 32K GQA layout.
        _prefix("prefix_gqa_32k", B=32, Hq=64, Hkv=8, S_q=1, d=128, page=64, prefix=32768, own_min=64, own_max=1024),
        # Drafted tokens of several rows a sequence, or samples drawn from one prompt, over an 8-bit cache.
        _prefix("prefix_chunk_e4m3", B=16, Hq=32, Hkv=8, S_q=4, d=128, page=32, prefix=16000, own_min=16, own_max=512,
                store="e4m3"),
        # A busy server with several system prompts; some sequences have none, some nothing of their own yet.
        _prefix("prefix_groups", B=128, Hq=32, Hkv=4, S_q=1, d=64, page=16, prefix=8191, own_min=0, own_max=1024,
                groups=5),
        # One conversation of some length: bounds of the page in hand, selection, attention.
        _sparse("sparse_short", B=1, Hq=32, Hkv=8, S_q=1, d=128, page=16, len_min=1500, len_max=1500, keep=32),
        # Eight long ragged conversations of the 32K GQA layout, 2K positions of each read by a head.
        _sparse("sparse_gqa_32k", B=8, Hq=64, Hkv=8, S_q=1, d=128, page=64, len_min=16384, len_max=32768, keep=32),
        # Two prompts of up to 128K just written: bounds of all their pages, and the first step.
        _sparse("sparse_prompt_e4m3", B=2, Hq=32, Hkv=8, S_q=1, d=128, page=64, len_min=98304, len_max=131072,
                keep=64, new=131072, store="e4m3"),
        # Many conversations with four drafted rows each, short and ragged, some slots of the batch empty.
        _sparse("sparse_chunk4_many", B=64, Hq=32, Hkv=8, S_q=4, d=128, page=32, len_min=0, len_max=8192, keep=48),
        # The weights of one step of the 32K GQA layout.
        _weigh("weigh_gqa_32k", B=8, Hq=64, Hkv=8, S_q=1, d=128, page=64, len_min=16384, len_max=32768),
        # Four rows a sequence over an 8-bit cache, earlier weights fading.
        _weigh("weigh_chunk4_e4m3", B=16, Hq=32, Hkv=8, S_q=4, d=128, page=16, len_min=1024, len_max=8192,
               store="e4m3", decay=0.95),
        # Two short conversations cut down: the smallest call.
        _evict("evict_short", B=2, Hkv=2, d=64, page=16, len_min=300, len_max=300, keep=100, recent=28),
        # Long conversations cut down to 4K positions.
        _evict("evict_16k", B=8, Hkv=8, d=128, page=64, len_min=8192, len_max=16384, keep=3584, recent=512),
    ]


def _prefix(name, B, Hq, Hkv, S_q, d, page, prefix, own_min, own_max, store="bf16", groups=1, lens=1):
    return dict(name=name, op="prefix", B=B, Hq=Hq, Hkv=Hkv, S_q=S_q, d=d, page=page, prefix=prefix, len_min=own_min,
                len_max=own_max, store=store, groups=groups, lens=lens)


def _sparse(name, B, Hq, Hkv, S_q, d, page, len_min, len_max, keep, new=0, store="bf16", sinks=1, recent=2, lens=1):
    return dict(name=name, op="sparse", B=B, Hq=Hq, Hkv=Hkv, S_q=S_q, d=d, page=page, len_min=len_min,
                len_max=len_max, keep=keep, new=new or S_q, store=store, sinks=sinks, recent=recent, lens=lens)


def _weigh(name, B, Hq, Hkv, S_q, d, page, len_min, len_max, store="bf16", decay=1.0, window=-1, lens=1):
    return dict(name=name, op="weigh", B=B, Hq=Hq, Hkv=Hkv, S_q=S_q, d=d, page=page, len_min=len_min,
                len_max=len_max, store=store, decay=decay, window=window, lens=lens)


def _evict(name, B, Hkv, d, page, len_min, len_max, keep, recent, store="bf16", lens=1):
    return dict(name=name, op="evict", B=B, Hq=Hkv, Hkv=Hkv, S_q=1, d=d, page=page, len_min=len_min, len_max=len_max,
                keep=keep, recent=recent, store=store, lens=lens)


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm evenly spread."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "sparse", "weigh", "evict"])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    group, S_q = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 1, 2, 4])
    page, store = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "e4m3"])
    seed = rng.randint(1, 1 << 20)
    if op == "prefix":
        B = _spread(rng, 1, 128)
        groups = rng.choice([1, 1, 1, rng.randint(2, 6)])
        # rows times positions at most those of the largest listed case; the plain form's copies for each sequence too
        most = min(32768, 32 * 64 * 32768 * 128 // (B * Hkv * group * S_q * d))
        if groups > 1:
            most = min(most, 128 * 4 * 8192 * 64 // (B * Hkv * d), 8192)
        hi = _spread(rng, 1, min(1024, 32 * 8 * 1024 * 128 // (B * Hkv * d)))
        c = _prefix("", B, Hkv * group, Hkv, S_q, d, page, _spread(rng, 1, max(1, most)),
                    rng.choice([hi, max(1, hi // 8), 0]), hi, store, groups, seed)
    elif op == "sparse":
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 8, max(64, min(131072, 2 * 131072 * 8 * 128 // (B * Hkv * d))))
        recent = 1 + -(-(S_q - 1) // page) + rng.randint(0, 2)
        sinks = rng.randint(0, 2)
        c = _sparse("", B, Hkv * group, Hkv, S_q, d, page, rng.choice([hi, hi // 8, 0]), hi,
                    _spread(rng, sinks + recent, 64), rng.choice([0, 0, _spread(rng, 1, hi)]), store, sinks, recent,
                    seed)
    elif op == "weigh":
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 8, max(64, min(32768, 7 * 32768 * 8 * 128 // (B * Hkv * d))))
        c = _weigh("", B, Hkv * group, Hkv, S_q, d, page, rng.choice([hi, max(S_q, hi // 8), 0]), hi, store,
                   rng.choice([1.0, 0.875, rng.random()]), rng.choice([-1, -1, _spread(rng, 1, 8192)]), seed)
    else:
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 8, max(64, min(32768, 6 * 16384 * 8 * 128 // (B * Hkv * d))))
        c = _evict("", B, Hkv, d, page, rng.choice([hi, hi // 4, 0]), hi, _spread(rng, 1, hi), _spread(rng, 1, hi) - 1,
                   store, seed)
        c["keep"] = min(c["keep"], 4096)
        c["recent"] = min(c["recent"], 1024)
    del c["name"]
    return c


def _lens(case):
    """Cache lengths of a case's sequences: drawn evenly between its limits, one of them the largest."""
    r = random.Random(case["lens"])
    out = [r.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])]
    out[0] = case["len_max"]
    return out


def _prefixes(case):
    """(lengths of the prefixes, the prefix of each sequence): with several, -1 for about a sequence in eight."""
    G = case["groups"]
    r = random.Random(case["lens"] + 3)
    lens = [case["prefix"]] + [r.randint(case["prefix"] // 8, case["prefix"]) for _ in range(G - 1)]
    return lens, [0 if G == 1 or b == 0 else -1 if r.random() < 0.125 else r.randrange(G) for b in range(case["B"])]


def _pairs(n, S_q, window):
    """Query rows of a sequence of length n times the positions that they see."""
    total = 0
    for t in range(n - S_q, n):
        total += max(0, t + 1 if window < 0 else min(t, window) + 1)
    return total


def _selected(case, n):
    """(pages, positions) read of a sequence of length n."""
    pages = -(-n // case["page"])
    kept = min(pages, case["keep"])
    return kept, 0 if n == 0 else (kept - 1) * case["page"] + n - (pages - 1) * case["page"]


# ------------------------------------------------------------------------------------------- work
def work(case):
    B, Hq, Hkv, d, S_q, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "S_q", "page"))
    row = 2 * d if case["store"] == "bf16" else d + 1  # one key or value row as it is stored
    lens = _lens(case)
    if case["op"] == "evict":
        left = [min(n, case["keep"] + case["recent"]) for n in lens]
        # the weights of all positions, and the rows that stay, read and written with their weights and numbers
        return {"bytes": 4 * Hkv * sum(lens) + Hkv * sum(left) * (4 * row + 8), "flops": Hkv * sum(lens)}
    io = B * Hq * S_q * (4 * d + 4)  # queries, outputs and logarithms of sums
    if case["op"] == "weigh":
        seen = sum(n if case["window"] < 0 else n - max(0, n - S_q - case["window"]) for n in lens)
        pairs = sum(_pairs(n, S_q, case["window"]) for n in lens)
        return {"bytes": seen * Hkv * row + 8 * sum(lens) * Hkv + B * Hq * S_q * (2 * d + 4), "flops": 2 * d * pairs * Hq}
    if case["op"] == "prefix":
        pl, of = _prefixes(case)
        rows = sum(pl[g] for g in set(of) if g >= 0) + sum(lens)
        pairs = sum(_pairs(n, S_q, -1) + (S_q * pl[g] if g >= 0 else 0) for n, g in zip(lens, of))
        return {"bytes": 2 * rows * Hkv * row + io, "flops": 4 * d * pairs * Hq}
    pages = sum(-(-n // page) for n in lens)
    fresh = sum(n - max(0, n - case["new"]) // page * page for n in lens)  # positions of the pages that changed
    changed = sum(-(-n // page) - max(0, n - case["new"]) // page for n in lens)
    read = sum(_selected(case, n)[1] for n in lens)
    pairs = sum(_pairs(_selected(case, n)[1], S_q, -1) for n in lens)
    return {"bytes": Hkv * (fresh * row + (pages + changed) * (2 * d + 1) + 2 * read * row) + io,
            "flops": 4 * d * pairs * Hq + 4 * d * pages * Hq * S_q}


# ---------------------------------------------------------------------------------------- prepare
def _tables(many, page, gen):
    """Page tables of pages in random order for lists of lengths, -1 where none is needed, and the number of pages of
    the pool (a few stay free)."""
    need = [[-(-n // page) for n in lens] for lens in many]
    n_pages = sum(map(sum, need)) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    at, out = 0, []
    for lens in need:
        table = torch.full((len(lens), max(1, max(lens))), -1, dtype=torch.int32, device=DEV)
        for b, n in enumerate(lens):
            table[b, :n] = order[at:at + n]
            at += n
        out.append(table)
    return out, n_pages


def _fill(case, n_pages, gen):
    """A pool with everything in it that earlier steps wrote: keys with a few strong channels and a direction that the
    keys of a page share (neighbouring tokens are alike), values whose size differs from row to row."""
    Hkv, page, d = case["Hkv"], case["page"], case["d"]
    pages = torch.empty((n_pages, Hkv, 2, page, d), device=DEV,
                        dtype=torch.bfloat16 if case["store"] == "bf16" else torch.float8_e4m3fn)
    scales = None
    if case["store"] == "e4m3":
        scales = torch.empty((n_pages, Hkv, page // 16, 2, 16), dtype=torch.uint8, device=DEV)
    strong = torch.ones(d, device=DEV)
    strong[::16] = 3.0
    step = max(1, (1 << 26) // (Hkv * 2 * page * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        x = torch.randn((n, Hkv, 2, page, d), generator=gen, device=DEV)
        x[:, :, 0] += 0.75 * torch.randn((n, Hkv, 1, d), generator=gen, device=DEV)
        x[:, :, 0] *= strong
        x[:, :, 1] *= torch.exp(0.5 * torch.randn((n, Hkv, page, 1), generator=gen, device=DEV))
        if scales is None:
            pages[p:p + n] = x
        else:
            codes, e = _quantise(x)
            pages[p:p + n] = codes
            scales[p:p + n] = e.view(n, Hkv, 2, page // 16, 16).transpose(2, 3)
    return pages, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, Hq, Hkv, d, S_q, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "S_q", "page"))
    st = {"case": case}
    order = torch.randperm(B, generator=gen, device=DEV).tolist()
    lens = _lens(case)
    lens = [lens[i] for i in order]
    many = [lens]
    if case["op"] == "prefix":
        pl, of = _prefixes(case)
        of = [of[i] for i in order]
        many.append(pl)
        st["prefix_len"] = torch.tensor(pl, dtype=torch.int32, device=DEV)
        st["prefix_of"] = torch.tensor(of, dtype=torch.int32, device=DEV) if case["groups"] > 1 else None
    elif case["op"] == "evict":
        many.append([min(n, case["keep"] + case["recent"]) for n in lens])
    tables, n_pages = _tables(many, page, gen)
    st["table"], st["other"] = tables[0], tables[-1]  # the prefixes' table, or the table that rows are moved to
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["pages"], st["scales"] = _fill(case, n_pages, gen)
    st["Q"] = torch.randn((B, Hq, S_q, d), generator=gen, device=DEV).to(torch.bfloat16)
    if case["op"] == "sparse":
        # bounds of earlier pages, as they were left by the steps before
        st["codes"] = torch.zeros((n_pages, Hkv, 2, d), dtype=torch.int8, device=DEV)
        st["exps"] = torch.zeros((n_pages, Hkv), dtype=torch.uint8, device=DEV)
        st["news"] = torch.tensor([min(n, case["new"]) for n in lens], dtype=torch.int32, device=DEV)
        _update(st, case, torch.nonzero(_page_range(st, case, st["lens"]), as_tuple=True), st["lens"])
        st["changed"] = torch.nonzero(_page_range(st, case, st["news"]), as_tuple=True)
        for t in (st["codes"], st["exps"]):  # those that the call has to make
            t[st["table"][st["changed"]].long()] = 1
    elif case["op"] == "weigh":
        st["LSE"] = _lse(st, case)
        st["rows"] = torch.nonzero(torch.arange(st["table"].shape[1] * page, device=DEV)[None] < st["lens"][:, None],
                                   as_tuple=True)
    if case["op"] in ("weigh", "evict"):
        # weights that fall off over several orders of magnitude, among them equal ones and zeros
        w = torch.exp(2.0 * torch.randn((n_pages, Hkv, page), generator=gen, device=DEV))
        st["W"] = torch.where(w < 1.0, torch.floor(w * 64.0) / 64.0, w)
        if case["op"] == "weigh":  # what a step adds, a few times over
            st["W"] *= 2.0 * (Hq // Hkv) * S_q / max(1, case["len_max"])
    if case["op"] == "evict":
        stay = case["keep"] + case["recent"]
        left = st["lens"].clamp(max=stay)
        st["left"] = torch.nonzero(torch.arange(stay, device=DEV)[None] < left[:, None], as_tuple=True)
    if own:
        import transformer_self_attention_gb300 as tsa
        st["cache"] = tsa.PagedCache(n_pages, Hkv, page, d, dtype=case["store"], pages=st["pages"], scales=st["scales"])
        if case["op"] == "prefix":
            st["plan"] = tsa.SharedPrefixAttention(B, Hq, Hkv, S_q, d)
        elif case["op"] == "sparse":
            st["bounds"] = tsa.PageBounds(st["cache"], codes=st["codes"], exponents=st["exps"])
            st["plan"] = tsa.PagedDecodeAttention(B, Hq, Hkv, S_q, d)
        else:
            st["weights"] = tsa.PageWeights(st["cache"], weights=st["W"])
        if case["op"] == "weigh":
            st["kind"] = tsa.MASK_CAUSAL if case["window"] < 0 else tsa.MASK_CAUSAL_SLIDING
    return st


# -------------------------------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"prefix": _plain_prefix, "sparse": _plain_sparse, "weigh": _plain_weigh, "evict": _plain_evict}[case["op"]](
        st, case)


def _run_own(st, case):
    if case["op"] == "prefix":
        return list(st["plan"](st["Q"], st["cache"], st["other"], st["prefix_len"], st["table"], st["lens"],
                               prefix_of=st["prefix_of"]))
    if case["op"] == "sparse":
        bounds = st["bounds"]
        bounds.update(st["table"], st["lens"], st["news"])
        table, lens = bounds.select(st["Q"], st["table"], st["lens"], keep=case["keep"], sinks=case["sinks"],
                                    recent=case["recent"])
        return [st["codes"], st["exps"], table, lens] + list(st["plan"](st["Q"], st["cache"], table, lens))
    weights = st["weights"]
    if case["op"] == "weigh":
        weights.accumulate(st["Q"], st["LSE"], st["table"], st["lens"], decay=case["decay"], kind=st["kind"],
                           window=max(0, case["window"]))
        return [st["W"]]
    lens, kept = weights.evict(st["table"], st["lens"], keep=case["keep"], recent=case["recent"], to_table=st["other"])
    return [st["pages"], st["W"], lens, kept] + ([] if st["scales"] is None else [st["scales"]])


# ------------------------------------------------------------------------------------ plain forms
def _quantise(x):
    """E4M3 codes and biased exponents of the rows of x: the smallest power of two that brings the row's
    largest magnitude to at most 448."""
    big = x.abs().amax(dim=-1)
    m, e = torch.frexp(big)  # big = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    k = torch.where(big == 0, torch.full_like(k, -127), k)
    codes = (x * torch.exp2(-k[..., None].float())).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _power(big):
    """The smallest k with big <= 127 * 2^k, at least -126 (that for 0 too)."""
    m, e = torch.frexp(big)  # 127 = 127/128 2^7
    return torch.where(m <= 127.0 / 128.0, e - 7, e - 6).clamp(min=-126)


def _at(table, page, positions):
    """Page and slot of positions [B, S] (a page of -1 comes back as 0)."""
    index = (positions // page).clamp(0, table.shape[1] - 1).long()
    return table.gather(1, index).clamp(min=0).long(), (positions % page).long()


def _gather(st, table, page, S):
    """The first S positions of every row of a table, as float32 K and V [rows, Hkv, S, d]."""
    pos = torch.arange(S, device=DEV)[None].expand(table.shape[0], S)
    p, s = _at(table, page, pos)
    x = st["pages"][p, :, :, s].float()  # [rows, S, Hkv, 2, d]
    if st["scales"] is not None:
        e = st["scales"][p, :, s // 16, :, s % 16].float()
        x = x * torch.exp2(e - 127)[..., None]
    return x[:, :, :, 0].transpose(1, 2), x[:, :, :, 1].transpose(1, 2)


def _scores(q, K, case):
    """Scores [B, Hkv, group, S_q, S] of Q [B, Hq, S_q, d] against K [B or 1, Hkv, S, d]."""
    B, Hq, Hkv, S_q = case["B"], case["Hq"], case["Hkv"], case["S_q"]
    rows = q.float().reshape(B, Hkv, Hq // Hkv * S_q, case["d"])
    if K.shape[0] == 1:  # one set of keys for the rows of all sequences
        s = torch.matmul(rows.transpose(0, 1).reshape(Hkv, -1, case["d"]), K[0].transpose(-1, -2))
        s = s.view(Hkv, B, -1, K.shape[2]).transpose(0, 1)
    else:
        s = torch.matmul(rows, K.transpose(-1, -2))
    return s.reshape(B, Hkv, Hq // Hkv, S_q, -1) * (1.0 / math.sqrt(case["d"]))


def _weighted(p, V, case):
    """sum_j p_j v_j, [B, Hkv, group, S_q, d], for p like _scores' result."""
    B, Hkv, S = case["B"], case["Hkv"], V.shape[2]
    if V.shape[0] == 1:
        o = torch.matmul(p.reshape(B, Hkv, -1, S).transpose(0, 1).reshape(Hkv, -1, S), V[0])
        o = o.view(Hkv, B, -1, case["d"]).transpose(0, 1)
    else:
        o = torch.matmul(p.reshape(B, Hkv, -1, S), V)
    return o.reshape(B, Hkv, p.shape[2], p.shape[3], case["d"])


def _seen(st, case, lens, S, window=-1):
    """Which of S positions the rows of each sequence see: [B, 1, 1, S_q, S]."""
    t = (lens[:, None] - case["S_q"] + torch.arange(case["S_q"], device=DEV))[:, None, None, :, None]
    j = torch.arange(S, device=DEV)
    return (j <= t) if window < 0 else (j <= t) & (j >= t - window)


def _softmax_parts(s, seen):
    """(maximum, weights relative to it, their sum) over the last dimension; a row without a position has sum 0."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return m, p, p.sum(dim=-1, keepdim=True)


def _finish(m, l, o, case):
    o = o / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    shape = st_shape(case)
    return [o.reshape(shape).to(torch.bfloat16), lse.reshape(shape[:3])]


def st_shape(case):
    return case["B"], case["Hq"], case["S_q"], case["d"]


def _plain_prefix(st, case):
    page = case["page"]
    K, V = _gather(st, st["other"], page, case["prefix"])
    if case["groups"] == 1:
        has = st["prefix_len"][0]
    else:  # each sequence with its prefix
        of = st["prefix_of"].long()
        K, V = K[of.clamp(min=0)], V[of.clamp(min=0)]
        has = torch.where(of >= 0, st["prefix_len"][of.clamp(min=0)], torch.zeros_like(st["prefix_len"][:1]))
        has = has.view(-1, 1, 1, 1, 1)
    s = _scores(st["Q"], K, case)
    m1, p1, l1 = _softmax_parts(s, torch.arange(case["prefix"], device=DEV) < has)
    Ko, Vo = _gather(st, st["table"], page, st["table"].shape[1] * page)
    s = _scores(st["Q"], Ko, case)
    m2, p2, l2 = _softmax_parts(s, _seen(st, case, st["lens"], s.shape[-1]))
    m = torch.maximum(m1, m2)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    f1, f2 = torch.exp(m1 - base), torch.exp(m2 - base)
    o = _weighted(p1, V, case) * f1 + _weighted(p2, Vo, case) * f2
    return _finish(m, l1 * f1 + l2 * f2, o, case)


def _page_range(st, case, news):
    """[B, pages of a row]: whether a page holds some of the last news[b] positions of its sequence."""
    i = torch.arange(st["table"].shape[1], device=DEV)[None]
    lens = st["lens"][:, None]
    return (i * case["page"] < lens) & ((i + 1) * case["page"] > lens - news[:, None]) & (news[:, None] > 0)


def _update(st, case, where, news):
    """Bounds of the pages at `where`, (sequences, places in their rows of the table): codes of the smallest and the
    largest key element of each channel, rounded outwards, and the exponent of the two rows' power of two."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    b, i = where
    p = st["table"][b, i].long()
    x = st["pages"][p][:, :, 0].float()  # [n, Hkv, page, d]
    if st["scales"] is not None:
        e = st["scales"][p][:, :, :, 0].reshape(-1, Hkv, page).float()
        x = x * torch.exp2(e - 127)[..., None]
    inside = (i[:, None] * page + torch.arange(page, device=DEV) < st["lens"][b][:, None])[:, None, :, None]
    lo = torch.where(inside, x, torch.full_like(x, math.inf)).amin(dim=2)
    hi = torch.where(inside, x, torch.full_like(x, -math.inf)).amax(dim=2)
    k = _power(torch.maximum(lo.abs(), hi.abs()).amax(dim=-1))
    f = torch.exp2(-k.float())[..., None]
    st["codes"][p] = torch.stack([torch.floor(lo * f), torch.ceil(hi * f)], dim=2).to(torch.int8)
    st["exps"][p] = (k + 127).to(torch.uint8)


def _plain_sparse(st, case):
    B, Hq, Hkv, d, page, keep = (case[k] for k in ("B", "Hq", "Hkv", "d", "page", "keep"))
    _update(st, case, st["changed"], st["news"])
    # the queries of a kv head in 8 bits, with one power of two
    q = st["Q"].float().reshape(B, Hkv, -1, d)
    k = _power(q.abs().amax(dim=(2, 3)))
    q = torch.round(q * torch.exp2(-k.float())[..., None, None])
    # the largest product that the bounds allow, summed over the channels: whole numbers below 2^24
    p = st["table"].clamp(min=0).long()
    c = st["codes"][p].float().permute(0, 2, 1, 3, 4)  # [B, Hkv, pages, 2, d]
    s = torch.matmul(q.clamp(max=0), c[..., 0, :].transpose(-1, -2)) + torch.matmul(q.clamp(min=0), c[..., 1, :].transpose(-1, -2))
    s = s.amax(dim=2) * torch.exp2(st["exps"][p].permute(0, 2, 1).float() - 127)
    n = ((st["lens"] + page - 1) // page)[:, None, None]
    i = torch.arange(p.shape[1], device=DEV)
    s = torch.where((i < case["sinks"]) | (i >= n - case["recent"]), torch.full_like(s, math.inf), s)
    s = torch.where(i < n, s, torch.full_like(s, -math.inf))
    rank = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.full((B, Hkv, keep), 1 << 30, dtype=torch.long, device=DEV)
    best[..., :rank.shape[-1]] = torch.where(rank < n, rank, torch.full_like(rank, 1 << 30))
    best = torch.sort(best, dim=-1).values
    held = best < (1 << 30)
    table = st["table"][:, None].expand(B, Hkv, -1).gather(2, torch.where(held, best, torch.zeros_like(best)))
    table = torch.where(held, table, torch.full_like(table, -1))
    lens = (st["lens"] - (n[:, 0, 0] - keep).clamp(min=0) * page).to(torch.int32)
    # attention over the selected pages
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    x = st["pages"][table.clamp(min=0).long(), h].float()  # [B, Hkv, keep, 2, page, d]
    if st["scales"] is not None:
        e = st["scales"][table.clamp(min=0).long(), h].float()  # [B, Hkv, keep, page / 16, 2, 16]
        x = x * torch.exp2(e.transpose(3, 4).reshape(B, Hkv, keep, 2, page, 1) - 127)
    K, V = x[:, :, :, 0].reshape(B, Hkv, -1, d), x[:, :, :, 1].reshape(B, Hkv, -1, d)
    s = _scores(st["Q"], K, case)
    m, w, l = _softmax_parts(s, _seen(st, case, lens, s.shape[-1]))
    return [st["codes"], st["exps"], table, lens] + _finish(m, l, _weighted(w, V, case), case)


def _lse(st, case):
    """Logarithms of the sums, as the step before left them: a sequence at a time."""
    L = torch.full((case["B"], case["Hq"], case["S_q"]), -math.inf, device=DEV)
    one = dict(case, B=1)
    for b, n in enumerate(_lens_of(st)):
        if n:
            K, _ = _gather(st, st["table"][b:b + 1], case["page"], n)
            s = _scores(st["Q"][b:b + 1], K, one)
            m, _, l = _softmax_parts(s, _seen(st, one, st["lens"][b:b + 1], n, case["window"]))
            L[b] = (m + torch.log(l)).reshape(case["Hq"], case["S_q"])
    return L


def _lens_of(st):
    return st["lens"].tolist()


def _plain_weigh(st, case):
    page = case["page"]
    S = st["table"].shape[1] * page
    K, _ = _gather(st, st["table"], page, S)
    s = _scores(st["Q"], K, case)
    lse = st["LSE"].reshape(s.shape[:4])[..., None]
    seen = _seen(st, case, st["lens"], S, case["window"]) & (lse > -math.inf)
    w = torch.where(seen, torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))), torch.zeros_like(s))
    w = w.sum(dim=(2, 3))  # [B, Hkv, S]
    b, j = st["rows"]
    p, slot = st["table"][b, j // page].long(), j % page
    old = st["W"][p, :, slot] * case["decay"]
    old = torch.where((j < st["lens"][b] - case["S_q"])[:, None], old, torch.zeros_like(old))
    st["W"][p, :, slot] = old + w[b, :, j]
    return [st["W"]]


def _plain_evict(st, case):
    page, keep, recent, Hkv = case["page"], case["keep"], case["recent"], case["Hkv"]
    S, stay = st["table"].shape[1] * page, keep + recent
    pos = torch.arange(S, device=DEV)
    p, slot = _at(st["table"], page, pos[None].expand(case["B"], S))
    w = st["W"][p, :, slot].transpose(1, 2)  # [B, Hkv, S]
    n = st["lens"][:, None, None]
    w = torch.where(pos >= n - recent, torch.full_like(w, math.inf), w)
    w = torch.where(pos < n, w, torch.full_like(w, -math.inf))
    best = torch.full((case["B"], Hkv, stay), 1 << 30, dtype=torch.long, device=DEV)
    rank = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :stay]
    best[..., :rank.shape[-1]] = torch.where(rank < n, rank, torch.full_like(rank, 1 << 30))
    best = torch.sort(best, dim=-1).values
    kept = torch.where(best < (1 << 30), best, torch.full_like(best, -1)).to(torch.int32)
    b, i = st["left"]
    h = torch.arange(Hkv, device=DEV)[None]
    j = best[b, :, i]  # [rows, Hkv]
    src, at = st["table"][b[:, None], j // page].long(), j % page
    dst, to = st["other"][b, i // page].long()[:, None], (i % page)[:, None]
    pages = st["pages"] if st["scales"] is None else st["pages"].view(torch.uint8)
    pages[dst, h, :, to] = pages[src, h, :, at]
    if st["scales"] is not None:
        st["scales"][dst, h, to // 16, :, to % 16] = st["scales"][src, h, at // 16, :, at % 16]
    st["W"][dst, h, to] = st["W"][src, h, at]
    out = [st["pages"], st["W"], st["lens"].clamp(max=stay), kept]
    return out if st["scales"] is None else out + [st["scales"]]


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The outputs of ``run`` from the definitions in float64, sequence by sequence."""
    st = prepare(case, seed)
    return {"prefix": _exact_prefix, "sparse": _exact_sparse, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](
        st, case)


def _rows64(st, table, case, positions, h=None):
    """Keys and values [n, Hkv, 2, d] (of one head [n, 2, d]) at positions of the sequence with this table row."""
    page = case["page"]
    p, slot = table.long()[positions // page], positions % page
    if h is None:
        x = st["pages"][p, :, :, slot].double()
        e = None if st["scales"] is None else st["scales"][p, :, slot // 16, :, slot % 16]
    else:
        x = st["pages"][p, h, :, slot].double()
        e = None if st["scales"] is None else st["scales"][p, h, slot // 16, :, slot % 16]
    return x if e is None else x * torch.exp2(e.double() - 127)[..., None]


def _attend64(q, x, scale):
    """(logsumexp, output) of the rows q [Hkv, group, d] over x [n, Hkv, 2, d]."""
    s = torch.matmul(q, x[:, :, 0].permute(1, 2, 0)) * scale
    lse = torch.logsumexp(s, dim=-1)
    return lse, torch.matmul(torch.exp(s - lse[..., None]), x[:, :, 1].transpose(0, 1))


def _exact_prefix(st, case):
    B, Hq, Hkv, S_q, d = case["B"], case["Hq"], case["Hkv"], case["S_q"], case["d"]
    O = torch.zeros(st_shape(case), dtype=torch.float64, device=DEV)
    L = torch.full(O.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    of = [0] * B if st["prefix_of"] is None else st["prefix_of"].tolist()
    pl = st["prefix_len"].tolist()
    shared = [_rows64(st, st["other"][g], case, torch.arange(n, device=DEV)) for g, n in enumerate(pl)]
    for b, n in enumerate(_lens_of(st)):
        mine = _rows64(st, st["table"][b], case, torch.arange(n, device=DEV))
        x = mine if of[b] < 0 else torch.cat([shared[of[b]], mine])
        q = st["Q"][b].double().view(Hkv, Hq // Hkv, S_q, d)
        for i in range(S_q):
            upto = x.shape[0] - n + max(0, n - S_q + i + 1)
            if upto == 0:
                continue
            lse, o = _attend64(q[:, :, i], x[:upto], 1.0 / math.sqrt(d))
            O[b, :, i], L[b, :, i] = o.reshape(Hq, d), lse.reshape(Hq)
    return [O, L]


def _exact_sparse(st, case):
    B, Hq, Hkv, S_q, d, page, keep = (case[k] for k in ("B", "Hq", "Hkv", "S_q", "d", "page", "keep"))
    O = torch.zeros(st_shape(case), dtype=torch.float64, device=DEV)
    L = torch.full(O.shape[:3], -math.inf, dtype=torch.float64, device=DEV)

    def power(big):  # per row: the smallest k with big <= 127 2^k
        k = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big) * 2.0 ** -126) / 127.0))
        k = torch.where(big * torch.exp2(-k) > 127.0, k + 1, torch.where(big * torch.exp2(1 - k) <= 127.0, k - 1, k))
        return k.clamp(min=-126)

    for b, n in enumerate(_lens_of(st)):
        if n == 0:
            continue
        x = _rows64(st, st["table"][b], case, torch.arange(n, device=DEV))
        pages = -(-n // page)
        pad = x[-1:].expand(pages * page - n, -1, -1, -1)
        keys = torch.cat([x, pad])[:, :, 0].view(pages, page, Hkv, d)
        lo, hi = keys.amin(dim=1), keys.amax(dim=1)  # [pages, Hkv, d]
        f = torch.exp2(power(torch.maximum(-lo, hi).amax(dim=-1)))[..., None]
        lo, hi = torch.floor(lo / f) * f, torch.ceil(hi / f) * f
        q = st["Q"][b].double().view(Hkv, -1, d)
        g = torch.exp2(power(q.abs().amax(dim=(1, 2))))[:, None, None]
        r = torch.round(q / g)
        bound = torch.maximum(r[None] * lo[:, :, None], r[None] * hi[:, :, None]).sum(dim=-1).amax(dim=-1)
        for h in range(Hkv):
            score = bound[:, h].clone()
            score[:case["sinks"]] = math.inf
            score[max(0, pages - case["recent"]):] = math.inf
            best = torch.sort(torch.sort(score, descending=True, stable=True).indices[:keep]).values
            j = (best[:, None] * page + torch.arange(page, device=DEV)).flatten()
            j = j[j < n]
            rows = st["Q"][b].double().view(Hkv, Hq // Hkv, S_q, d)[h]
            for i in range(S_q):
                y = x[j[j <= n - S_q + i], h][:, None]
                if y.shape[0] == 0:
                    continue
                lse, o = _attend64(rows[None, :, i], y, 1.0 / math.sqrt(d))
                at = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                O[b, at, i], L[b, at, i] = o[0], lse[0]
    return [None, None, None, None, O, L]


def _exact_weigh(st, case):
    Hq, Hkv, S_q, d, page = (case[k] for k in ("Hq", "Hkv", "S_q", "d", "page"))
    W = st["W"].double()
    for b, n in enumerate(_lens_of(st)):
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        p, slot = st["table"][b].long()[j // page], j % page
        keys = _rows64(st, st["table"][b], case, j)[:, :, 0]
        q = st["Q"][b].double().view(Hkv, Hq // Hkv, S_q, d)
        lse = st["LSE"][b].double().view(Hkv, Hq // Hkv, S_q)
        w = W[p, :, slot] * case["decay"]
        w[max(0, n - S_q):] = 0
        for i in range(S_q):
            t = n - S_q + i
            lo = 0 if case["window"] < 0 else max(0, t - case["window"])
            if t < 0:
                continue
            s = torch.einsum("hgd,jhd->jhg", q[:, :, i], keys[lo:t + 1]) / math.sqrt(d)
            w[lo:t + 1] += torch.exp(s - lse[:, :, i]).sum(dim=-1)
        W[p, :, slot] = w
    return [W]


def _exact_evict(st, case):
    page, keep, recent, Hkv = case["page"], case["keep"], case["recent"], case["Hkv"]
    pages, W = st["pages"].double(), st["W"].double()
    for b, n in enumerate(_lens_of(st)):
        j = torch.arange(n, device=DEV)
        row, to = st["table"][b].long(), st["other"][b].long()
        w = W[row[j // page], :, j % page]  # [n, Hkv]
        old = max(0, n - recent)
        for h in range(Hkv):
            best = torch.sort(w[:old, h], descending=True, stable=True).indices[:keep]
            mine = torch.cat([torch.sort(best).values, j[old:]])
            i = torch.arange(mine.shape[0], device=DEV)
            dst, src = (to[i // page], h, slice(None), i % page), (row[mine // page], h, slice(None), mine % page)
            pages[dst] = pages[src]
            W[dst[0], h, dst[3]] = W[src[0], h, src[3]]
    out = [pages, W, None, None]
    return out if st["scales"] is None else out + [None]
