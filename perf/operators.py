"""The serving operators around decode attention, in their plain form and as the library's calls.

Three operators that are used together:

rope    rotary positions applied to Q and K (the first ``rot`` of d elements, half or interleaved
        pairs, frequencies scaled for long contexts), and the gradient of that rotation
cache   new keys and values written into pages (bf16, or E4M3 with one power-of-two scale per row),
        the keys rotated on the way, and the positions of a sequence read back as dense tensors
decode  attention of a few new rows per sequence over such pages

``run`` with ``own`` false computes them from elementary torch operations in float32 (angles in
float64); with ``own`` true it makes the library's calls.

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
        # One generation step of the long-context GQA layout: eight rows at far positions.
        _rope("rope_step", B=8, S=1, Hq=64, Hkv=8, d=128, rot=128, pos0=16384, packed=True),
        # Training or prompt pass of the causal 4K layout, Q and K as views of the packed projection.
        _rope("rope_prompt", B=2, S=4096, Hq=32, Hkv=32, d=128, rot=128, packed=True),
        # Gradients of the 16K layout: interleaved pairs, half of the head, context stretched 4 times.
        _rope("rope_grad", B=1, S=16384, Hq=32, Hkv=8, d=128, rot=64, layout="interleaved", scaling="yarn",
              factor=4.0, original=4096, backward=True),
        # Gradients in float32 on the small layout, odd length and odd number of pairs.
        _rope("rope_grad_f32", B=1, S=255, Hq=4, Hkv=4, d=64, rot=26, dtype="f32", backward=True),
        # A generation step's rows appended to a bf16 cache, queries and keys rotated in the call.
        _cache("append_bf16", B=16, S=1, Hq=32, Hkv=8, d=128, page=16, len_min=1, len_max=512),
        # A ragged chunk of four prompts written as E4M3, then the whole prefix read back for prefill.
        _cache("chunk_e4m3", B=4, S=2048, Hq=0, Hkv=8, d=128, page=64, len_min=2048, len_max=8192, store="e4m3",
               read=True),
        # The smallest step: one user with a short conversation.
        _decode("decode_one_short", B=1, Hq=32, Hkv=8, S_q=1, d=128, page=16, len_min=100, len_max=100),
        # Eight long ragged conversations of the 32K GQA layout, at both cache types.
        _decode("decode_gqa_32k", B=8, Hq=64, Hkv=8, S_q=1, d=128, page=64, len_min=16384, len_max=32768),
        _decode("decode_gqa_32k_e4m3", B=8, Hq=64, Hkv=8, S_q=1, d=128, page=64, len_min=16384, len_max=32768,
                store="e4m3"),
        # Every query head on one kv head: 32 rows against one cache.
        _decode("decode_mqa_16k", B=16, Hq=32, Hkv=1, S_q=1, d=128, page=32, len_min=2048, len_max=16384),
        # Four speculative rows per sequence over an 8-bit cache.
        _decode("decode_chunk4_e4m3", B=8, Hq=32, Hkv=8, S_q=4, d=128, page=16, len_min=1024, len_max=8192,
                store="e4m3"),
        # A busy server: many conversations, short and ragged, some slots of the batch empty.
        _decode("decode_many_short", B=256, Hq=32, Hkv=8, S_q=1, d=128, page=16, len_min=0, len_max=2048),
    ]


def _rope(name, B, S, Hq, Hkv, d, rot, layout="half", dtype="bf16", scaling="none", factor=1.0, original=0,
          base=10000.0, pos0=0, packed=False, backward=False):
    return dict(name=name, op="rope", B=B, S=S, Hq=Hq, Hkv=Hkv, d=d, rot=rot, layout=layout, dtype=dtype,
                scaling=scaling, factor=factor, original=original, base=base, pos0=pos0, packed=packed,
                backward=backward)


def _cache(name, B, S, Hq, Hkv, d, page, len_min, len_max, store="bf16", read=False, rot=0, layout="half", lens=1):
    return dict(name=name, op="cache", B=B, S=S, Hq=Hq, Hkv=Hkv, d=d, page=page, len_min=len_min, len_max=len_max,
                store=store, read=read, rot=rot or d, layout=layout, scaling="none", factor=1.0, original=0,
                base=10000.0, lens=lens)


def _decode(name, B, Hq, Hkv, S_q, d, page, len_min, len_max, store="bf16", window=-1, lens=1):
    return dict(name=name, op="decode", B=B, Hq=Hq, Hkv=Hkv, S_q=S_q, d=d, page=page, len_min=len_min,
                len_max=len_max, store=store, window=window, lens=lens)


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm evenly spread."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"]) if rot > 2 else "none"
        B = rng.randint(1, 8)
        S = _spread(rng, 1, max(1, 2 * 4096 * 64 * 128 // (B * Hkv * (group + 1) * d)))
        S = min(S, 65536)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            S = max(1, S // 2)
        c = _rope("", B, S, Hkv * group, Hkv, d, rot, rng.choice(["half", "interleaved"]), dtype, scaling,
                  1.0 if scaling == "none" else rng.uniform(1.5, 16.0),
                  rng.choice([2048, 4096, 8192]) if scaling == "yarn" else 0, rng.choice([10000.0, 500000.0]),
                  _spread(rng, 1, 1 << 20) - 1, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "cache":
        B, S = _spread(rng, 1, 64), _spread(rng, 1, 2048)
        S = min(S, max(1, 16384 // B))
        page = rng.choice([16, 32, 48, 64, 128])
        hi = S + _spread(rng, 1, 4096)
        c = _cache("", B, S, Hkv * group if rng.random() < 0.5 else 0, Hkv, d, page, S, min(hi, S + 65536 // B),
                   rng.choice(["bf16", "e4m3"]), rng.random() < 0.5, rng.choice([d, d // 2]),
                   rng.choice(["half", "interleaved"]), rng.randint(1, 1 << 20))
        if c["store"] == "e4m3":
            c["read"] = True
    else:
        B = _spread(rng, 1, 256)
        S_q = rng.choice([1, 1, 1, 2, 4])
        most = max(16, min(32768, 7 * 32768 * 8 * 128 // (B * Hkv * d)))
        hi = _spread(rng, 8, most)
        lo = rng.choice([hi, max(S_q, hi // 8), 0])
        c = _decode("", B, Hkv * group, Hkv, S_q, d, rng.choice([16, 32, 48, 64, 128]), lo, hi,
                    rng.choice(["bf16", "e4m3"]), rng.choice([-1, -1, _spread(rng, 1, 8192)]),
                    rng.randint(1, 1 << 20))
    del c["name"]
    return c


def _lens(case):
    """Cache lengths of a case's sequences, ascending in no order: drawn evenly between its limits."""
    r = random.Random(case["lens"])
    out = [r.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])]
    out[0] = case["len_max"]
    return out


def _news(case):
    """New rows of each sequence of a cache case: ragged, one sequence with all S of them."""
    r = random.Random(case["lens"] + 7)
    S = case["S"]
    return [S if b == 0 or S == 1 else r.randint(max(1, S // 2), S) for b in range(case["B"])]


# ------------------------------------------------------------------------------------------- work
def work(case):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        n = B * case["S"] * (Hq + Hkv)
        el = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * d * el + 4 * B * case["S"], "flops": 3 * n * case["rot"]}
    row = 2 * d if case["store"] == "bf16" else d + 1  # one key or value row as it is stored
    if case["op"] == "cache":
        new, lens = sum(_news(case)), sum(_lens(case))
        n = 2 * new * Hkv * (2 * d + row) + 2 * new * Hq * 2 * d
        if case["read"]:
            # the rows just written are among those read back; both directions of the readback are due
            n += 2 * lens * Hkv * (row + 2 * d)
        return {"bytes": n, "flops": 3 * new * (Hkv + Hq) * case["rot"] + 2 * new * Hkv * d}
    S_q, w = case["S_q"], case["window"]
    rows = pairs = 0
    for n in _lens(case):
        rows += n if w < 0 else n - max(0, n - S_q - w)
        for i in range(S_q):
            t = n - S_q + i
            pairs += max(0, t + 1 if w < 0 else min(t, w) + 1)
    return {"bytes": 2 * rows * Hkv * row + B * Hq * S_q * (4 * d + 4) + 4 * B, "flops": 4 * d * pairs * Hq}


# ---------------------------------------------------------------------------------------- prepare
def _table(lens, page, gen):
    """A page table of pages in random order for sequences of these lengths, -1 where none is needed, and
    the number of pages of the pool (a few stay free)."""
    need = [-(-n // page) for n in lens]
    wide = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _fill(case, n_pages, gen):
    """A pool with everything in it that earlier steps wrote: keys with a few strong channels, values whose
    size differs from row to row."""
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
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    st = {"case": case}
    if case["op"] == "rope":
        S = case["S"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["packed"]:  # views of one projection's output [B, S, heads, d]
            qkv = torch.randn((B, S, Hq + 2 * Hkv, d), generator=gen, device=DEV).to(dt)
            st["Q"], st["K"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            st["Q"] = torch.randn((B, Hq, S, d), generator=gen, device=DEV).to(dt)
            st["K"] = torch.randn((B, Hkv, S, d), generator=gen, device=DEV).to(dt)
        first = torch.randint(0, case["pos0"] + 1, (B, 1), generator=gen, device=DEV) + case["pos0"] // 2
        st["positions"] = (first + torch.arange(S, device=DEV)).to(torch.int32)
    else:
        order = torch.randperm(B, generator=gen, device=DEV).tolist()
        lens = _lens(case)
        lens = [lens[i] for i in order]
        st["table"], n_pages = _table(lens, case["page"], gen)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["pages"], st["scales"] = _fill(case, n_pages, gen)
        if case["op"] == "cache":
            S = case["S"]
            news = _news(case)
            st["news"] = torch.tensor([news[i] for i in order], dtype=torch.int32, device=DEV)
            st["new_rows"] = torch.nonzero(torch.arange(S, device=DEV)[None] < st["news"][:, None], as_tuple=True)
            qkv = torch.randn((B, S, Hq + 2 * Hkv, d), generator=gen, device=DEV).to(torch.bfloat16)
            st["Q"] = qkv[:, :, :Hq].transpose(1, 2) if Hq else None
            st["K"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
            st["V"] = qkv[:, :, Hq + Hkv:].transpose(1, 2)
            if case["read"]:  # the dense tensors that the next prefill call takes its keys and values from
                S_max = case["len_max"]
                st["Kd"] = torch.zeros((B, Hkv, S_max, d), dtype=torch.bfloat16, device=DEV)
                st["Vd"] = torch.zeros_like(st["Kd"])
        else:
            st["Q"] = torch.randn((B, Hq, case["S_q"], d), generator=gen, device=DEV).to(torch.bfloat16)
    if own:
        import transformer_self_attention_gb300 as tsa
        if case["op"] in ("rope", "cache"):
            st["rope"] = tsa.RotaryPositions(d, rotary_dim=case["rot"], layout=case["layout"], base=case["base"],
                                             scaling=case["scaling"], factor=case["factor"],
                                             original_len=case["original"])
        if case["op"] != "rope":
            st["cache"] = tsa.PagedCache(st["pages"].shape[0], Hkv, case["page"], d, dtype=case["store"],
                                         pages=st["pages"], scales=st["scales"])
        if case["op"] == "decode":
            kind = tsa.MASK_CAUSAL if case["window"] < 0 else tsa.MASK_CAUSAL_SLIDING
            st["plan"] = tsa.PagedDecodeAttention(B, Hq, Hkv, case["S_q"], d, kind=kind,
                                                  window=max(0, case["window"]))
    return st


# -------------------------------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "rope":
        c, s = _cos_sin(case, st["positions"])
        if case["backward"]:
            s = -s
        return [_rotate(t, c[:, None], s[:, None], case).to(t.dtype) for t in (st["Q"], st["K"])]
    if case["op"] == "cache":
        return _plain_cache(st, case)
    return _plain_decode(st, case)


def _run_own(st, case):
    if case["op"] == "rope":
        turn = st["rope"].backward if case["backward"] else st["rope"]
        return list(turn(st["Q"], st["K"], st["positions"]))
    cache = st["cache"]
    if case["op"] == "cache":
        Qr = cache.write(st["K"], st["V"], st["table"], st["lens"], new_len=st["news"], rope=st["rope"], Q=st["Q"])
        out = [] if Qr is None else [Qr]
        if case["read"]:
            return out + list(cache.read(st["table"], st["lens"], K=st["Kd"], V=st["Vd"]))
        return out + [cache.pages]
    return list(st["plan"](st["Q"], cache, st["table"], st["lens"]))


# ------------------------------------------------------------------------------------ plain forms
def _frequencies(case):
    """Angles per position of the rot / 2 pairs (float64) and the factor on the rotated elements."""
    rot, base, s = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk":  # the base raised so that the lowest frequency is divided by s
        base = base * s ** (rot / (rot - 2))
    f = torch.arange(rot // 2, dtype=torch.float64, device=DEV) * (-2.0 / rot)
    f = torch.exp(f * math.log(base))
    amp = 1.0
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "yarn":  # pairs that turn often within the old context keep their frequency
        turns = case["original"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / s * (1 - keep)
        amp = 0.1 * math.log(s) + 1.0
    return f, amp


def _cos_sin(case, positions, dtype=torch.float32):
    f, amp = _frequencies(case)
    angle = positions.to(torch.float64)[..., None] * f
    return (torch.cos(angle) * amp).to(dtype), (torch.sin(angle) * amp).to(dtype)


def _rotate(x, c, s, case):
    """x [..., d] with its pairs turned by the angles of c and s, in the type of c."""
    rot = case["rot"]
    x = x.to(c.dtype)
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    else:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _quantise(x):
    """E4M3 codes and biased exponents of the rows of x: the smallest power of two that brings the row's
    largest magnitude to at most 448."""
    big = x.abs().amax(dim=-1)
    m, e = torch.frexp(big)  # big = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    k = torch.where(big == 0, torch.full_like(k, -127), k)
    codes = (x * torch.exp2(-k[..., None].float())).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _at(table, page, positions):
    """Page and slot of positions [B, S] (a page of -1 comes back as 0)."""
    index = (positions // page).clamp(0, table.shape[1] - 1).long()
    return table.gather(1, index).clamp(min=0).long(), (positions % page).long()


def _gather(st, case, S, dtype):
    """The first S positions of every sequence, as stored: K and V [B, Hkv, S, d] in dtype."""
    pos = torch.arange(S, device=DEV)[None].expand(case["B"], S)
    p, s = _at(st["table"], case["page"], pos)
    x = st["pages"][p, :, :, s].to(dtype)  # [B, S, Hkv, 2, d]
    if st["scales"] is not None:
        e = st["scales"][p, :, s // 16, :, s % 16].to(dtype)
        x = x * torch.exp2(e - 127)[..., None]
    return x[:, :, :, 0].transpose(1, 2), x[:, :, :, 1].transpose(1, 2)


def _plain_cache(st, case):
    K, V, news, lens = st["K"], st["V"], st["news"], st["lens"]
    i = torch.arange(case["S"], device=DEV)[None]
    pos = (lens - news)[:, None] + i
    c, s = _cos_sin(case, pos)
    out = []
    if st["Q"] is not None:
        Qr = _rotate(st["Q"], c[:, None], s[:, None], case).to(torch.bfloat16)
        Qr = torch.where((i < news[:, None])[:, None, :, None], Qr, torch.zeros_like(Qr))
        out.append(Qr)
    new = torch.stack([_rotate(K, c[:, None], s[:, None], case), V.float()], dim=3)  # [B, Hkv, S, 2, d]
    new = new.permute(0, 2, 1, 3, 4)
    b, r = st["new_rows"]
    p, slot = _at(st["table"], case["page"], pos.clamp(min=0))
    p, slot, new = p[b, r], slot[b, r], new[b, r]
    if case["store"] == "bf16":
        st["pages"][p, :, :, slot] = new.to(torch.bfloat16)
    else:
        codes, e = _quantise(new)
        st["pages"].view(torch.uint8)[p, :, :, slot] = codes.view(torch.uint8)
        st["scales"][p, :, slot // 16, :, slot % 16] = e
    if not case["read"]:
        return out + [st["pages"]]
    S = case["len_max"]
    inside = (torch.arange(S, device=DEV)[None] < lens[:, None])[:, None, :, None]
    for dense, x in zip((st["Kd"], st["Vd"]), _gather(st, case, S, torch.float32)):
        dense.copy_(torch.where(inside, x.to(torch.bfloat16), dense))
        out.append(dense)
    return out


def _plain_decode(st, case):
    B, Hq, Hkv, S_q, d = case["B"], case["Hq"], case["Hkv"], case["S_q"], case["d"]
    S = st["table"].shape[1] * case["page"]
    K, V = _gather(st, case, S, torch.float32)
    q = st["Q"].float().reshape(B, Hkv, Hq // Hkv * S_q, d)
    s = torch.matmul(q, K.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s = s.view(B, Hkv, Hq // Hkv, S_q, S)
    t = (st["lens"][:, None] - S_q + torch.arange(S_q, device=DEV))[:, None, None, :, None]
    j = torch.arange(S, device=DEV)
    seen = j <= t
    if case["window"] >= 0:
        seen = seen & (j >= t - case["window"])
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, S), V).view(B, Hkv, -1, S_q, d) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    return [o.reshape(B, Hq, S_q, d).to(torch.bfloat16), lse.reshape(B, Hq, S_q)]


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The outputs of ``run`` from the definitions in float64, row by row or sequence by sequence."""
    st = prepare(case, seed)
    if case["op"] == "rope":
        sign = -1.0 if case["backward"] else 1.0
        return [_turned64(x, st["positions"], case, sign) for x in (st["Q"], st["K"])]
    if case["op"] == "cache":
        return _exact_cache(st, case)
    return _exact_decode(st, case)


def _turned64(x, positions, case, sign=1.0):
    """Each pair as a complex number times amp e^(i angle); x [B, H, S, d], positions [B, S]."""
    f, amp = _frequencies(case)
    rot = case["rot"]
    y = x.to(torch.float64).clone()
    first = slice(0, rot // 2) if case["layout"] == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if case["layout"] == "half" else slice(1, rot, 2)
    for b in range(x.shape[0]):
        angle = positions[b].double()[:, None] * f * sign
        z = torch.complex(y[b, ..., first].contiguous(), y[b, ..., second].contiguous())
        z = z * torch.polar(torch.full_like(angle, amp), angle)
        y[b, ..., first], y[b, ..., second] = z.real, z.imag
    return y


def _stored64(x, store):
    """Rows x (float64) as a cache holds them: themselves in bf16's stead, or their E4M3 values."""
    if store == "bf16":
        return x
    big = x.abs().amax(dim=-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 448.0))
    k = torch.where(big * torch.exp2(-k) > 448.0, k + 1, torch.where(big * torch.exp2(1 - k) <= 448.0, k - 1, k))
    k = k.clamp(-127, 127)
    y = (x * torch.exp2(-k)).abs()
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).double())  # four significant bits, down to 2^-9
    return torch.sign(x) * torch.round(y / step) * step * torch.exp2(k)


def _pages64(st, case):
    x = st["pages"].to(torch.float64)
    if st["scales"] is not None:
        e = st["scales"].transpose(2, 3).reshape(x.shape[:-1]).double()
        x = x * torch.exp2(e - 127)[..., None]
    return x


def _exact_cache(st, case):
    pages, page = _pages64(st, case), case["page"]
    pos = (st["lens"] - st["news"])[:, None] + torch.arange(case["S"], device=DEV)
    out = []
    if st["Q"] is not None:
        q = _turned64(st["Q"], pos, case)
        for b, n in enumerate(st["news"].tolist()):
            q[b, :, n:] = 0
        out.append(q)
    k = _stored64(_turned64(st["K"], pos, case), case["store"])
    v = _stored64(st["V"].double(), case["store"])
    for b, n in enumerate(st["news"].tolist()):
        j = pos[b, :n].long()
        p = st["table"][b].long()[j // page]
        pages[p, :, 0, j % page] = k[b, :, :n].transpose(0, 1)
        pages[p, :, 1, j % page] = v[b, :, :n].transpose(0, 1)
    if not case["read"]:
        return out + [pages]
    dense = [st["Kd"].double(), st["Vd"].double()]
    for b, n in enumerate(st["lens"].tolist()):
        j = torch.arange(n, device=DEV)
        p = st["table"][b].long()[j // page]
        for which in (0, 1):
            dense[which][b, :, :n] = pages[p, :, which, j % page].transpose(0, 1)
    return out + dense


def _exact_decode(st, case):
    B, Hq, Hkv, S_q, page = case["B"], case["Hq"], case["Hkv"], case["S_q"], case["page"]
    O = torch.zeros(st["Q"].shape, dtype=torch.float64, device=DEV)
    L = torch.full(st["Q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        p, slot = st["table"][b].long()[j // page], j % page
        x = st["pages"][p, :, :, slot].double()  # [n, Hkv, 2, d]
        if st["scales"] is not None:
            x = x * torch.exp2(st["scales"][p, :, slot // 16, :, slot % 16].double() - 127)[..., None]
        q = st["Q"][b].double().view(Hkv, Hq // Hkv, S_q, -1)
        for i in range(S_q):
            t = n - S_q + i
            lo = 0 if case["window"] < 0 else max(0, t - case["window"])
            if t < 0:
                continue
            y = x[lo:t + 1]
            s = torch.einsum("hgd,jhd->hgj", q[:, :, i], y[:, :, 0]) / math.sqrt(case["d"])
            lse = torch.logsumexp(s, dim=-1)
            o = torch.einsum("hgj,jhd->hgd", torch.exp(s - lse[..., None]), y[:, :, 1])
            O[b, :, i], L[b, :, i] = o.reshape(Hq, -1), lse.reshape(Hq)
    return [O, L]
