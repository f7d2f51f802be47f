"""Selections and evictions whose outputs share memory with an input, or with one another, at any offset are refused; outputs
that only touch them, or lie between the rows of a table, are not."""
import pytest
import torch

import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

B, HKV, PAGE, D, WIDE, KEEP, RECENT = 2, 2, 16, 64, 6, 10, 3


def _setup():
    cache = tsa.PagedCache(2 * B * WIDE, HKV, PAGE, D)
    bounds, weights = tsa.PageBounds(cache), tsa.PageWeights(cache)
    Q = torch.zeros((B, 4, 1, D), dtype=torch.bfloat16, device="cuda")
    pool = torch.arange(2 * B * WIDE, dtype=torch.int32, device="cuda").view(2, B, WIDE)
    return cache, bounds, weights, Q, pool[0].contiguous(), pool[1].contiguous()


def _place(shape, buf, at):
    n = 1
    for x in shape:
        n *= x
    return buf[at:at + n].view(shape)


def _in_buffer(t, buf, at):
    """The values of t in buf from `at` on."""
    out = _place(t.shape, buf, at)
    out.copy_(t)
    return out


def _refused(call):
    with pytest.raises(tsa.AttnError) as e:
        call()
    assert e.value.status == tsa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("what", ["lengths", "table", "to_table"])
@pytest.mark.parametrize("output", ["length", "big"])
def test_outputs_over_inputs(what, output):
    """The output begins in front of the input, inside it and behind it."""
    cache, bounds, weights, Q, table, to = _setup()
    lens = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    big = {"evict": (B, HKV, KEEP + RECENT), "select": (B, HKV, 3)}
    for call in ("evict", "select"):
        if call == "select" and what == "to_table":
            continue
        src = {"lengths": lens, "table": table, "to_table": to}[what]
        shape = (B,) if output == "length" else big[call]
        count = torch.Size(shape).numel()
        for at in range(100 - count - 1, 100 + src.numel() + 2):
            buf = torch.zeros(300, dtype=torch.int32, device="cuda")
            inside = _in_buffer(src, buf, 100)
            out = _place(shape, buf, at)
            t = inside if what == "table" else table
            n = inside if what == "lengths" else lens
            kw = {"length": out} if output == "length" else {"kept" if call == "evict" else "table": out}
            if call == "evict":
                go = lambda: weights.evict(t, n, KEEP, RECENT, to_table=inside if what == "to_table" else to, **kw)
            else:
                go = lambda: bounds.select(Q, t, n, 3, **kw)
            if at + count <= 100 or at >= 100 + src.numel():
                go()
                assert torch.equal(inside, src)
            else:
                _refused(go)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_outputs_over_one_another():
    cache, bounds, weights, Q, table, to = _setup()
    lens = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    for shape, call in (((B, HKV, KEEP + RECENT), lambda x, n: weights.evict(table, lens, KEEP, RECENT, to_table=to, length=n, kept=x)),
                        ((B, HKV, 3), lambda x, n: bounds.select(Q, table, lens, 3, table=x, length=n))):
        count = torch.Size(shape).numel()
        for at in range(20 - B - 1, 20 + count + 2):
            buf = torch.zeros(120, dtype=torch.int32, device="cuda")
            x, n = _place(shape, buf, 20), buf[at:at + B]
            if at + B <= 20 or at >= 20 + count:
                call(x, n)
            else:
                _refused(lambda: call(x, n))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_outputs_between_the_rows_of_a_table():
    """A table inside a wider buffer, whose gaps take the new lengths; a table of one row for all (an expanded one)."""
    cache, bounds, weights, Q, table, to = _setup()
    lens = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    want_t, want_n = bounds.select(Q, table, lens, 3)
    for gap in range(1, 9):
        buf = torch.zeros((B, WIDE + gap), dtype=torch.int32, device="cuda")
        buf[:, :WIDE] = table
        for at in range(WIDE, 2 * WIDE + gap):
            n = buf.view(-1)[at:at + B]
            if n.numel() < B:
                continue
            if at + B <= WIDE + gap or at >= 2 * WIDE + gap:
                got, short = bounds.select(Q, buf[:, :WIDE], lens, 3, length=n)
                assert torch.equal(got, want_t) and torch.equal(short, want_n) and torch.equal(buf[:, :WIDE], table)
            else:
                _refused(lambda: bounds.select(Q, buf[:, :WIDE], lens, 3, length=n))
    buf = torch.zeros(40, dtype=torch.int32, device="cuda")
    same = _in_buffer(table[0], buf, 10)[None].expand(B, -1)
    for at in range(10 - B, 10 + WIDE + 1):
        n = buf[at:at + B]
        if at + B <= 10 or at >= 10 + WIDE:
            bounds.select(Q, same, lens, 3, length=n)
        else:
            _refused(lambda: bounds.select(Q, same, lens, 3, length=n))
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)
