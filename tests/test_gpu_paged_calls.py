"""Calls of the paged cache at the edges of what its documentation allows."""
import pytest
import torch

import transformer_self_attention_gb300 as tsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,rot", [(0, 0), (0, 64), (6, 64)])
def test_an_append_of_no_rows_does_nothing(store, Hq, rot):
    cache = tsa.PagedCache(3, 2, 16, 64, dtype=store)
    before = cache.pages.view(torch.uint8).fill_(0x11).clone()
    table, lens = torch.zeros((2, 1), dtype=torch.int32).cuda(), torch.tensor([5, 0], dtype=torch.int32).cuda()
    K = torch.empty((2, 2, 0, 64), dtype=torch.bfloat16, device="cuda")
    Q = torch.empty((2, Hq, 0, 64), dtype=torch.bfloat16, device="cuda") if Hq else None
    out = cache.write(K, K, table, lens, rope=tsa.RotaryPositions(64, rot) if rot else None, Q=Q)
    assert out is None if Q is None else out.shape == Q.shape
    if Q is not None:  # and into an output that is given
        assert cache.write(K, K, table, lens, rope=tsa.RotaryPositions(64, rot), Q=Q, Q_out=Q) is Q
    Kd, Vd = cache.read(table, lens, length=0)
    assert Kd.shape == Vd.shape == (2, 2, 0, 64)
    assert torch.equal(cache.pages.view(torch.uint8), before)
    assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


def test_an_error_behind_a_poll_on_another_stream_is_recorded():
    """A new cache's first call, and a call directly behind a poll that cleared the word, on a stream that waits for no
    other: the clearing is done by then."""
    side = torch.cuda.Stream()
    K = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    bad, lens = torch.tensor([[9]], dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        cache = tsa.PagedCache(1, 1, 16, 64)  # (its pages' zeros may still be pending: the call writes none)
        for _ in range(5):
            cache.write(K, K, bad, lens, stream=side)
            assert cache.poll_device_error() == (tsa.ATTN_ERR_INVALID_ARG, tsa.CACHE_ERR_PAGE)
        assert cache.poll_device_error() == (tsa.ATTN_OK, 0)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_a_new_caches_zeros_come_before_the_first_write_on_another_stream(store):
    """The stream that allocates the pages is held up; the write runs on one that does not wait for it."""
    made, side = torch.cuda.Stream(), torch.cuda.Stream()
    K = torch.randn((1, 2, 40, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    table = torch.arange(40, dtype=torch.int32)[None, -3:].contiguous().cuda()
    lens = torch.tensor([40], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(made):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        cache = tsa.PagedCache(40, 2, 16, 64, dtype=store)
    cache.write(K, K, table, lens, stream=side)
    torch.cuda.synchronize()
    Kd, Vd = cache.read(table, lens, length=40)
    if store == "bf16":
        assert torch.equal(Kd, K) and torch.equal(Vd, K)
    else:  # half a step of a code, or of the smallest ones, 2^-10 of a factor that is below 2^-7 of the row's largest
        x = K.double()
        bound = x.abs() * 2.0 ** -4 + x.abs().amax(-1, keepdim=True) * 2.0 ** -17
        assert float(((Kd.double() - x).abs() - bound).max()) <= 0 and torch.equal(Kd, Vd)
    assert bool((cache.pages.view(torch.uint8)[:37] == 0).all())
