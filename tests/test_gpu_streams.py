"""Calls of the lossless cache on another stream than the current one: what the cache makes, fills or copies for a call
happens on that call's stream."""
import pytest
import torch

from lossless_compressed_kv_gaac_gb300.cache import LayerCache, _stream_object as stream_object

pytestmark = pytest.mark.gpu

BUSY = 40_000_000  # cycles that the current stream is kept busy: some 20 ms


def inputs(T=256, H=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    k, v = (torch.randn((1, T, H, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, 4 * H, 128), generator=g, device="cuda").to(torch.bfloat16)
    return k, v, q, torch.tensor([T - 3], dtype=torch.int32, device="cuda")


def cache(k, v, lens=None):
    c = LayerCache(1, k.shape[2], k.shape[1] // 64)
    c.calibrate(k[0], v[0])
    if lens is not None:
        c.encode(k, v, lens)
    return c


def streams():
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    return ((s, s), (t, t.cuda_stream))


def test_encode_reads_the_lengths_of_its_call():
    k, v, _, lens = inputs()
    right = cache(k, v, lens)
    for _, handle in streams():
        c = cache(k, v)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        c.encode(k, v, lens, stream=handle)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0 and torch.equal(c.seq_lens, lens)
        # the same entries but for the raw tiles' indices, which go in the order of arrival
        for x, y in zip(c.fields()[1:], right.fields()[1:]):
            assert torch.equal(x, y)
        k2, v2 = c.decompress(k.shape[1])
        n = int(lens)
        assert torch.equal(k2[:, :n], k[:, :n]) and torch.equal(v2[:, :n], v[:, :n])


def test_decompress_keeps_what_it_wrote():
    k, v, _, lens = inputs()
    c = cache(k, v, lens)
    for _, handle in streams():
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        k2, v2 = c.decompress(k.shape[1], stream=handle)
        torch.cuda.synchronize()
        n = int(lens)
        assert torch.equal(k2[:, :n], k[:, :n]) and torch.equal(v2[:, :n], v[:, :n])
        assert (k2[:, n:] == 0).all() and (v2[:, n:] == 0).all()


@pytest.mark.parametrize("bf16", [False, True])
def test_attention_takes_no_memory_in_use(bf16):
    k, v, q, lens = inputs()
    c = cache(k, v)
    c.encode(k, v, lens, raw=bf16)
    right = c.attention(q, 0.1, bf16=bf16)
    for s, handle in streams():
        torch.cuda.synchronize()
        used = torch.full_like(right, 7)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        seen = used.clone()
        del used
        out = c.attention(q, 0.1, bf16=bf16, stream=handle)
        torch.cuda.synchronize()
        assert (seen == 7).all() and torch.equal(out, right)
        torch.cuda._sleep(BUSY)
        seen = out.clone()
        del out
        with torch.cuda.stream(s):
            other = torch.full_like(right, 7)
        torch.cuda.synchronize()
        assert torch.equal(seen, right) and (other == 7).all()


def test_first_attention_on_a_side_stream_has_a_zeroed_workspace():
    k, v, q, lens = inputs(2048)
    right = cache(k, v, lens).attention(q, 0.1)
    for _, handle in streams():
        c = cache(k, v, lens)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        out = c.attention(q, 0.1, stream=handle)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0 and torch.equal(out, right)


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_raw_handle_of_the_default_stream(handle):
    """0 and 1 (the legacy default stream's names) are that stream, for what a call makes too; 2 is the thread's default
    stream, which waits for that one and makes it wait."""
    k, v, q, lens = inputs()
    c = cache(k, v, lens)
    right = c.attention(q, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        k2, v2 = c.decompress(k.shape[1], stream=handle)
        out = c.attention(q, 0.1, stream=handle)
    done = torch.cuda.default_stream().record_event()
    done.synchronize()
    assert not s.query()  # nothing of it waited for the current stream
    used = torch.full_like(k2, 7)  # the default stream's memory, of which the results' is a part
    n = int(lens)
    torch.cuda.synchronize()
    assert torch.equal(k2[:, :n], k[:, :n]) and torch.equal(v2[:, :n], v[:, :n]) and torch.equal(out, right)
    assert used.eq(7).all() and int(c.status.item()) == 0
    assert stream_object(handle, c.device).cuda_stream == 0 and stream_object(None, c.device) is None
