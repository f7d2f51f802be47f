"""The operators for long contexts over a paged cache as generation uses them: together, on other streams than the current
one, captured into graphs and replayed."""
import math

import pytest
import torch

import context_util as cu
import paged_util as pu
import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

CAUSAL = tsa.MASK_CAUSAL
STORES = pytest.mark.parametrize("store", ["bf16", "e4m3"])


def _int32(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


def _normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _vals(cache):
    return pu.values(cache.pages, cache.scales)


@STORES
@pytest.mark.parametrize("d", [64, 128])
def test_generation_over_selected_pages_with_a_bounded_cache(store, d):
    """Two prompts, then steps of S_q rows: rows are appended, bounds follow, pages are selected and attended to; every
    position's weight is added up over a full step, and a cache that has grown too long is cut down in place.  Every result
    against its definition on the cache as it then is."""
    B, Hq, Hkv, S_q, page, keep, heavy, recent = 2, 8, 2, 2, 16, 4, 100, 28
    g = torch.Generator().manual_seed(11)
    lens = [150, 70]
    cache = tsa.PagedCache(24, Hkv, page, d, dtype=store)
    bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
    table = torch.randperm(24, generator=g)[:2 * 11].view(2, 11).to(torch.int32)
    tab = table.cuda()
    rope = tsa.RotaryPositions(d)
    plan = tsa.PagedDecodeAttention(B, Hq, Hkv, S_q, d)
    n = _int32(lens)
    K, V = _normal(g, B, Hkv, 150, d), _normal(g, B, Hkv, 150, d)
    cache.write(K, V, tab, n, new_len=n, rope=rope)
    bounds.update(tab, n)
    for step in range(4):
        lens = [x + S_q for x in lens]
        n = n + S_q
        Q = cache.write(_normal(g, B, Hkv, S_q, d), _normal(g, B, Hkv, S_q, d), tab, n, rope=rope,
                        Q=_normal(g, B, Hq, S_q, d))
        bounds.update(tab, n, new_len=_int32([S_q] * B))
        vals = _vals(cache)
        codes, exps = bounds.codes.cpu(), bounds.exponents.cpu()
        for b in range(B):
            for i in range(-(-lens[b] // page)):
                c, e = cu.bounds(vals, table, page, b, lens[b], i)
                assert torch.equal(codes[int(table[b, i])], c) and torch.equal(exps[int(table[b, i])], e)
        got, short = bounds.select(Q, tab, n, keep, sinks=1, recent=2)
        chosen, want_len = cu.select(Q.cpu(), codes, exps, table, page, lens, keep, 1, 2)
        assert short.tolist() == want_len
        for b in range(B):
            for h in range(Hkv):
                assert got[b, h].tolist()[:len(chosen[b][h])] == table[b][torch.tensor(chosen[b][h])].tolist()
        O, LSE = plan(Q, cache, got, short)
        pu.check_decode(O, LSE, cu.decode_chosen(Q.cpu(), vals, table, page, lens, chosen, d ** -0.5), d)
        O, LSE = plan(Q, cache, tab, n)
        pu.check_decode(O, LSE, pu.decode(Q, vals, table, page, lens, d ** -0.5, CAUSAL, 0), d)
        before = weights.weights.cpu()
        weights.accumulate(Q, LSE, tab, n)
        seen, err = cu.weigh(Q.cpu(), LSE.cpu(), before, vals, table, page, lens, d ** -0.5, CAUSAL, 0, 1.0)
        assert float(((weights.weights.cpu().double() - seen).abs() - err).max()) <= 0
        W = weights.weights.cpu()
        n, kept = weights.evict(tab, n, heavy, recent, length=torch.empty_like(n))
        want = cu.evict(W, table, page, lens, heavy, recent)
        after = _vals(cache)
        for b in range(B):
            for h in range(Hkv):
                assert kept[b, h].tolist()[:len(want[b][h])] == want[b][h]
                j, i = torch.tensor(want[b][h]), torch.arange(len(want[b][h]))
                p, q = table[b].long()[j // page], table[b].long()[i // page]
                assert torch.equal(after[q, h, :, i % page], vals[p, h, :, j % page])
        lens = [min(x, heavy + recent) for x in lens]
        assert n.tolist() == lens
        bounds.update(tab, n)  # (rows have moved)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@STORES
@pytest.mark.parametrize("d,S_q", [(64, 1), (128, 3)])
def test_samples_of_one_prompt(store, d, S_q):
    """A prompt is written once; several continuations grow behind it in pages of their own.  Each step agrees with attention
    over the whole sequence, and with the paged decode step over a table of the prompt's and the own pages."""
    B, Hq, Hkv, page, prompt, steps = 5, 8, 2, 16, 128, 3
    g = torch.Generator().manual_seed(12)
    cache = tsa.PagedCache(8 + B * 2, Hkv, page, d, dtype=store)
    order = torch.randperm(8 + B * 2, generator=g).to(torch.int32)
    ptab, table = order[:8].view(1, 8), order[8:].view(B, 2)
    rope = tsa.RotaryPositions(d)
    plen = _int32([prompt])
    cache.write(_normal(g, 1, Hkv, prompt, d), _normal(g, 1, Hkv, prompt, d), ptab.cuda(), plen, rope=rope)
    plan, step = tsa.SharedPrefixAttention(B, Hq, Hkv, S_q, d), tsa.PagedDecodeAttention(B, Hq, Hkv, S_q, d)
    whole = torch.cat([ptab.expand(B, -1), table], dim=1).contiguous()
    for i in range(1, steps + 1):
        own, n = _int32([S_q * i] * B), _int32([prompt + S_q * i] * B)
        # (positions of the whole sequences: their last S_q rows are the new ones)
        Q = cache.write(_normal(g, B, Hkv, S_q, d), _normal(g, B, Hkv, S_q, d), whole.cuda(), n, rope=rope,
                        Q=_normal(g, B, Hq, S_q, d))
        O, LSE = plan(Q, cache, ptab.cuda(), plen, table.cuda(), own)
        ref = pu.decode(Q, _vals(cache), whole, page, n.tolist(), d ** -0.5, CAUSAL, 0)
        pu.check_decode(O, LSE, ref, d)
        pu.check_decode(*step(Q, cache, whole.cuda(), n), ref, d)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def _calls(store, page=16):
    """name -> call(stream, which): outputs from one of two sets of inputs."""
    B, Hq, Hkv, S_q, d, S = 3, 8, 2, 2, 128, 640
    g = torch.Generator().manual_seed(13)
    per = S // page
    made = []
    for _ in range(2):
        cache = tsa.PagedCache((2 * B + 1) * per, Hkv, page, d, dtype=store)
        table = torch.randperm((2 * B + 1) * per, generator=g).to(torch.int32).view(2 * B + 1, per).cuda()
        lens = _int32([S] * (2 * B + 1))
        cache.write(_normal(g, 2 * B + 1, Hkv, S, d), _normal(g, 2 * B + 1, Hkv, S, d), table, lens)
        bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
        bounds.update(table, lens)
        weights.weights.copy_(torch.rand(weights.weights.shape, generator=g))
        made.append((cache, bounds, weights, table, _normal(g, B, Hq, S_q, d)))
    n, one = _int32([S, S - 5, 300]), _int32([S])
    plan, step = tsa.SharedPrefixAttention(B, Hq, Hkv, S_q, d), tsa.PagedDecodeAttention(B, Hq, Hkv, S_q, d)
    picked = [m[1].select(m[4], m[3][:B], n, 8, 1, 2) for m in made]

    def weigh(stream, i):
        cache, _, _, table, Q = made[i]
        w = tsa.PageWeights(cache)
        LSE = torch.full((B, Hq, S_q), 5.0, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        w.accumulate(Q, LSE, table[:B], n, stream=stream)
        return (w.weights,)

    calls = {
        "select": lambda stream, i: made[i][1].select(made[i][4], made[i][3][:B], n, 8, 1, 2, stream=stream),
        "heads": lambda stream, i: step(made[i][4], made[i][0], *picked[i], stream=stream),
        "evict": lambda stream, i: made[i][2].evict(made[i][3][:B], n, 100, 20, to_table=made[i][3][B:2 * B], stream=stream),
        "prefix": lambda stream, i: plan(made[i][4], made[i][0], made[i][3][2 * B:], one, made[i][3][:B], n, stream=stream),
        "weigh": weigh,
    }
    torch.cuda.synchronize()
    return calls


OUTPUTS = ["select", "heads", "evict", "prefix"]


@STORES
@pytest.mark.parametrize("name", OUTPUTS)
def test_pending_work_of_the_current_stream_does_not_reach_the_outputs(name, store):
    """Blocks of the outputs' sizes are freed on the current stream while writes to them are still queued there."""
    call = _calls(store)[name]
    want = [t.clone() for t in call(None, 0)]
    shapes = [(t.shape, t.dtype) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    freed = [torch.empty(s, dtype=dt, device="cuda") for s, dt in shapes]
    for t in freed:
        t.fill_(7)
    del freed, t
    got = call(side, 0)
    side.synchronize()
    with torch.cuda.stream(side):
        early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for e, t, w in zip(early, got, want):
        assert torch.equal(e, w) and torch.equal(t, w)


@STORES
@pytest.mark.parametrize("name", OUTPUTS)
def test_outputs_freed_with_reads_pending_on_the_current_stream_are_not_reused(name, store):
    call = _calls(store)[name]
    want = [t.clone() for t in call(None, 0)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side, 0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    del got
    other = call(side, 1)  # its outputs must not lie where the copies are still to be read
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(copies, want))
    assert not torch.equal(other[-1 if name == "evict" else 0], want[-1 if name == "evict" else 0])


@STORES
def test_inputs_freed_on_the_current_stream_while_another_reads_them(store):
    calls = _calls(store)
    want = calls["weigh"](None, 0)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = calls["weigh"](side, 0)[0]  # (the logarithms of sums are a tensor that nobody keeps)
    for _ in range(4):
        torch.empty((3, 8, 2), device="cuda").fill_(-math.inf)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@STORES
def test_captured_steps_follow_lengths_tables_and_queries(store):
    """One graph of a step: append, bounds, selection, both attentions, weights, eviction into other pages.  It is replayed
    over lengths, tables and queries that change, and gives what the calls give one by one, bit for bit."""
    B, Hq, Hkv, d, page, S = 3, 8, 2, 64, 16, 320
    per = S // page
    pool = (2 * B + 1) * per
    g = torch.Generator().manual_seed(14)

    def state():
        gg = torch.Generator().manual_seed(15)
        cache = tsa.PagedCache(pool, Hkv, page, d, dtype=store)
        table = torch.arange(pool, dtype=torch.int32).view(2 * B + 1, per).cuda()
        cache.write(_normal(gg, 2 * B + 1, Hkv, S, d), _normal(gg, 2 * B + 1, Hkv, S, d), table, _int32([S] * (2 * B + 1)))
        bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
        bounds.update(table, _int32([S] * (2 * B + 1)))
        fixed = dict(K=_normal(gg, B, Hkv, 1, d), Q=_normal(gg, B, Hq, 1, d), table=table[:B].clone(), to=table[B:2 * B].clone(),
                     ptab=table[2 * B:].clone(), n=_int32([1] * B), new=_int32([1] * B),
                     plen=_int32([1]))
        plans = tsa.SharedPrefixAttention(B, Hq, Hkv, 1, d), tsa.PagedDecodeAttention(B, Hq, Hkv, 1, d)
        return cache, bounds, weights, fixed, plans

    def step(cache, bounds, weights, x, plans):
        cache.write(x["K"], x["K"], x["table"], x["n"], new_len=x["new"])
        bounds.update(x["table"], x["n"], new_len=x["n"])
        tab, short = bounds.select(x["Q"], x["table"], x["n"], 6, 1, 2)
        a = plans[1](x["Q"], cache, tab, short)
        b = plans[0](x["Q"], cache, x["ptab"], x["plen"], x["table"], x["n"])
        c = plans[1](x["Q"], cache, x["table"], x["n"])
        weights.accumulate(x["Q"], c[1], x["table"], x["n"], decay=0.9)
        e = weights.evict(x["table"], x["n"], 40, 30, to_table=x["to"])
        return (tab, short, *a, *b, *c, *e)

    eager, captured = state(), state()
    step(*captured)  # (kernels are loaded before the capture)
    captured[2].weights.zero_()
    step(*eager)
    eager[2].weights.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*captured)
    for i in range(5):
        new = dict(K=_normal(g, B, Hkv, 1, d), Q=_normal(g, B, Hq, 1, d),
                   table=torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda(),
                   n=_int32([[320, 1, 77], [0, 300, 96], [5, 16, 17], [128, 129, 0], [320, 320, 320]][i]),
                   plen=_int32([[0, 320, 1, 129, 64][i]]))
        new["new"] = new["n"].clamp(max=1)
        for s in (eager, captured):
            for k, v in new.items():
                s[3][k].copy_(v)
        want = step(*eager)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)
        assert torch.equal(eager[0].pages.view(torch.uint8), captured[0].pages.view(torch.uint8))
        assert torch.equal(eager[1].codes, captured[1].codes) and torch.equal(eager[2].weights, captured[2].weights)
    assert eager[0].poll_device_error() == captured[0].poll_device_error() == (tsa.ATTN_OK, 0)


@STORES
def test_two_captured_graphs_and_a_call_at_once(store):
    """Two graphs of the same shape, each over a handle of its own, are replayed on two streams beside calls on a third."""
    calls = [_calls(store) for _ in range(3)]
    want = {name: [t.clone() for t in calls[0][name](None, 0)] for name in OUTPUTS}
    for c in calls:
        for name in OUTPUTS:
            c[name](None, 0)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append({name: calls[i][name](None, 0) for name in OUTPUTS})
        graphs.append(graph)
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        got = {name: calls[2][name](streams[2], 0) for name in OUTPUTS}
        torch.cuda.synchronize()
        for o in (*outs, got):
            for name in OUTPUTS:
                assert all(torch.equal(a, b) for a, b in zip(o[name], want[name])), name


@STORES
def test_tables_of_other_strides(store):
    """One row of pages for all sequences (an expanded tensor), and rows and heads inside larger tables."""
    B, Hq, Hkv, d, page = 4, 4, 2, 64, 16
    g = torch.Generator().manual_seed(16)
    pages, scales, table, total = pu.make_pool([90], Hkv, page, d, store)
    cache = tsa.PagedCache(total, Hkv, page, d, dtype=store, pages=pages.cuda(),
                           scales=None if scales is None else scales.cuda())
    vals, Q = pu.values(pages, scales), _normal(g, B, Hq, 1, d)
    lens = [90, 90, 90, 90]
    same = table.cuda().expand(B, -1)
    bounds, step = tsa.PageBounds(cache), tsa.PagedDecodeAttention(B, Hq, Hkv, 1, d)
    bounds.update(same, _int32(lens))
    tab, short = bounds.select(Q, same, _int32(lens), 3)
    chosen = cu.select(Q.cpu(), bounds.codes.cpu(), bounds.exponents.cpu(), table.expand(B, -1), page, lens, 3, 1, 1)[0]
    want = cu.decode_chosen(Q.cpu(), vals, table.expand(B, -1), page, lens, chosen, d ** -0.5)
    wide = torch.full((B, 5, 9), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, 1:3, 2:5] = tab
    inside = wide[:, 1:3, 2:5]
    pu.check_decode(*step(Q, cache, inside, short), want, d)
    assert torch.equal(step(Q, cache, inside, short)[0], step(Q, cache, tab, short)[0])
    # one table for every head, given as an expanded one
    every = same[:, None].expand(B, Hkv, -1)
    assert torch.equal(step(Q, cache, every, _int32(lens))[0], step(Q, cache, same, _int32(lens))[0])
    plan = tsa.SharedPrefixAttention(B, Hq, Hkv, 1, d)
    O, L = plan(Q, cache, table.cuda(), _int32([90]), same, _int32([0] * B))
    pu.check_decode(O, L, pu.decode(Q, vals, table.expand(B, -1), page, lens, d ** -0.5, CAUSAL, 0), d)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_calls_that_are_refused():
    """Refusals of the library, which the binding passes on; nothing is launched."""
    cache = tsa.PagedCache(4, 2, 16, 64)
    bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
    table, n = torch.zeros((1, 2), dtype=torch.int32).cuda(), _int32([20])
    Q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    long = torch.zeros((1, 40961), dtype=torch.int32).cuda()
    L = torch.zeros((1, 4, 1), device="cuda")

    def refused(status, call):
        with pytest.raises(tsa.AttnError) as e:
            call()
        assert e.value.status == status

    refused(tsa.ATTN_ERR_UNSUPPORTED, lambda: bounds.select(Q, long, n, 4))
    refused(tsa.ATTN_ERR_UNSUPPORTED, lambda: bounds.select(Q, table, n, 40961))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.select(Q, table, n, 4, length=n))
    both = torch.zeros((1, 2, 3), dtype=torch.int32).cuda()  # (an output and an input, or two outputs, in one place)
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.select(Q, both.view(1, 6), n, 3, table=both))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.select(Q, table, n, 3, table=both, length=both.view(6)[:1]))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.select(Q, table, both.view(6)[:1], 3, table=both))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, both.view(6)[:1], 3, kept=both))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, n, 3, kept=both, length=both.view(6)[:1]))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, n, 3, to_table=both.view(1, 6), kept=both))
    many = torch.zeros((1, 4, 33, 64), dtype=torch.bfloat16, device="cuda")
    refused(tsa.ATTN_ERR_UNSUPPORTED, lambda: bounds.select(many, table, n, 8, recent=3))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, n, 4, length=n))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, n, 4, to_table=table))
    for kw in (dict(scale=0.0), dict(scale=math.nan), dict(decay=1.5), dict(decay=math.nan), dict(kind=7)):
        refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.accumulate(Q, L, table, n, **kw))
    for kind in (tsa.MASK_SLIDING, tsa.MASK_LOCAL_GLOBAL):
        refused(tsa.ATTN_ERR_UNSUPPORTED, lambda: weights.accumulate(Q, L, table, n, kind=kind, window=4))
    off = torch.zeros(2 * 4 * 2 * 16, device="cuda")[1:1 + 4 * 2 * 16].view(4, 2, 16)
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: tsa.PageWeights(cache, off).accumulate(Q, L, table, n))
    plan, step = tsa.SharedPrefixAttention(1, 4, 2, 1, 64), tsa.PagedDecodeAttention(1, 4, 2, 1, 64)
    other = tsa.PagedCache(4, 4, 16, 64)
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: plan(Q, other, table, n, table, n))
    for bad in (lambda: step(Q, cache, table[:, None].expand(1, 3, 2), n), lambda: plan(Q, cache, table, n, long[:, :0], n),
                lambda: plan(Q, cache, table.expand(2, 2), _int32([1, 1]), table, n), lambda: plan(Q.float(), cache, table, n, table, n),
                lambda: plan(Q, cache, table.cpu(), n, table, n), lambda: bounds.select(Q.cpu(), table, n, 4)):
        with pytest.raises(ValueError):
            bad()
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
    plan.close()
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: plan(Q, cache, table, n, table, n))
    cache.close()
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.update(table, n))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: bounds.select(Q, table, n, 4))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.accumulate(Q, L, table, n))
    refused(tsa.ATTN_ERR_INVALID_ARG, lambda: weights.evict(table, n, 4))


def test_calls_without_sequences():
    cache = tsa.PagedCache(4, 2, 16, 64)
    none, n = torch.zeros((0, 2), dtype=torch.int32).cuda(), _int32([])
    tsa.PageBounds(cache).update(none, n)
    tab, short = tsa.PageBounds(cache).select(torch.zeros((0, 4, 1, 64), dtype=torch.bfloat16, device="cuda"), none, n, 4)
    assert tab.shape == (0, 2, 4) and short.shape == (0,)
    w = tsa.PageWeights(cache)
    w.accumulate(torch.zeros((0, 4, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((0, 4, 1), device="cuda"), none, n)
    length, kept = w.evict(none, n, 3, 1)
    assert length.shape == (0,) and kept.shape == (0, 2, 4)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
