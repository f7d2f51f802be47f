"""Outputs that the rotary, cache and paged-decode calls allocate themselves, on another stream than the current one."""
import pytest
import torch

import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, S = 3, 8, 2, 128, 640


def _calls(store):
    """name -> call(stream, which): a tuple of outputs from one of two sets of inputs."""
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn((2, B, S, HQ + 2 * HKV, D), generator=g).to(torch.bfloat16).cuda()
    Q, K, V = (qkv[:, :, :, lo:hi].transpose(2, 3) for lo, hi in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    rope = tsa.RotaryPositions(D)
    caches = [tsa.PagedCache(B * S // 64, HKV, 64, D, dtype=store) for _ in range(2)]
    table = torch.randperm(B * S // 64, generator=g).to(torch.int32).view(B, S // 64).cuda()
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    for i in range(2):
        caches[i].write(K[i], V[i], table, lens)
    plan = tsa.PagedDecodeAttention(B, HQ, HKV, 2, D)
    q = Q[:, :, :, :2].contiguous()
    return {
        "rope": lambda stream, i: rope(Q[i], K[i], stream=stream),
        "rope backward": lambda stream, i: rope.backward(Q[i], K[i], stream=stream),
        "write": lambda stream, i: (caches[i].write(K[i], V[i], table, lens, rope=rope, Q=Q[i], stream=stream),),
        "read": lambda stream, i: caches[i].read(table, lens, length=S, stream=stream),
        "decode": lambda stream, i: plan(q[i], caches[i], table, lens, stream=stream),
    }


NAMES = ["rope", "rope backward", "write", "read", "decode"]


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", NAMES)
def test_pending_work_of_the_current_stream_does_not_reach_the_outputs(name, store):
    """Blocks of the outputs' sizes are freed on the current stream while writes to them are still queued there."""
    call = _calls(store)[name]
    want = [t.clone() for t in call(None, 0)]
    if name == "write":  # (its second call finds the same cache: keys that are written again)
        assert all(torch.equal(a, b) for a, b in zip(call(None, 0), want))
    shapes = [(t.shape, t.dtype) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    freed = [torch.empty(s, dtype=dt, device="cuda") for s, dt in shapes]
    for t in freed:
        t.fill_(7.0)
    del freed, t
    got = call(side, 0)
    side.synchronize()
    with torch.cuda.stream(side):
        early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for e, t, w in zip(early, got, want):
        assert torch.equal(e, w) and torch.equal(t, w)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", NAMES)
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
    assert not torch.equal(other[0], want[0])
