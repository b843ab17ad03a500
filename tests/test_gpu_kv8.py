"""The 8-bit paged cache on the GPU: append, decode attention and the page calls, alone and together."""
import math
import random

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from lossless_compressed_kv_gaac_gb300.cache import Kv8Cache
from tests import kv8_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4, E5 = G.FP8_E4M3, G.FP8_E5M2
SCALE = 1 / math.sqrt(128)


def rand(shape, dtype, seed=0, mul=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * mul).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(new):
    return ints([0] + torch.cumsum(torch.tensor(new), 0).tolist())


def ok(c):
    torch.cuda.synchronize()
    return int(c.status.item())


def kv_of(n, heads, dtype, seed):
    """Keys with uneven channels, values with others."""
    s = torch.exp(0.5 * rand((2, heads, 128), F32, 77))
    return ((rand((n, heads, 128), F32, seed) * s[0]).to(dtype), (rand((n, heads, 128), F32, seed + 1) * s[1]).to(dtype))


def filled(lens, heads, fmt=E4, dtype=BF16, seed=0, spare=3, max_blocks=None, shuffle=True):
    """A cache of sequences of these lengths, its pages scattered over the pool, and the tokens it was given."""
    B = len(lens)
    mb = max_blocks or max(1, max((n + 63) // 64 for n in lens))
    need = sum(n // 64 for n in lens)
    c = Kv8Cache(max(1, need + spare), B, heads, mb, fmt, dtype)
    k, v = kv_of(sum(lens), heads, dtype, seed)
    cu = cu_of(lens)
    c.reserve(cu)
    if shuffle and need:
        perm = torch.randperm(c.n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        c.table.copy_(torch.where(c.table >= 0, perm[c.table.clamp(min=0).long()], c.table))
        held = torch.zeros_like(c.refs)
        held[perm[:need].long()] = 1
        c.refs.copy_(held)
    c.append(k, v, cu, reserve=False)
    assert ok(c) == 0
    return c, k, v


def check_blocks(c, streams):
    """Every sequence's pages, scales and open block are those of its tokens ([2, n, heads, 128])."""
    lens = c.seq_lens.tolist()
    for b, x in streams.items():
        assert lens[b] == x.shape[1]
        full = lens[b] // 64
        ids = c.table[b, :full].long()
        blocks = x[:, :full * 64].reshape(2, full, 64, c.n_kv_heads, 128).permute(1, 3, 0, 2, 4)
        f8, s = U.quantise(blocks, c.fmt)
        assert U.f8_equal(c.pages[ids].view(U.FP8[c.fmt]), f8)
        assert torch.equal(c.scales[ids], s)
        assert torch.equal(c.tail[b, :, :, :lens[b] % 64], x[:, full * 64:].permute(2, 0, 1, 3))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("heads,steps", [(1, [[1], [62], [1], [1], [63], [200]]), (3, [[5, 0, 64], [59, 0, 1], [0, 130, 0]]),
                                         (8, [[63, 64, 65, 1], [1, 64, 63, 500], [128, 1, 1, 12]]),
                                         (2, [[7] * 70, [57] * 70, [1] * 70])])
def test_append_chunks(heads, steps, fmt, dtype):
    B = len(steps[0])
    total = [sum(s[b] for s in steps) for b in range(B)]
    c = Kv8Cache(sum(n // 64 for n in total) + 2, B, heads, max(n // 64 for n in total) + 1, fmt, dtype)
    got = {b: torch.zeros((2, 0, heads, 128), dtype=dtype, device="cuda") for b in range(B)}
    for i, new in enumerate(steps):
        k, v = kv_of(sum(new), heads, dtype, 10 * i)
        c.append(k, v, cu_of(new))
        at = 0
        for b, n in enumerate(new):
            got[b] = torch.cat([got[b], torch.stack([k[at:at + n], v[at:at + n]])], 1)
            at += n
        assert ok(c) == 0
        check_blocks(c, got)
    assert int((c.refs > 0).sum()) == sum(n // 64 for n in total)


def test_append_one_by_one_equals_at_once():
    lens = [64, 70, 130]
    a, k, v = filled(lens, 4, E5, F16, shuffle=False)
    b = Kv8Cache(a.n_pages, 3, 4, a.max_blocks, E5, F16)
    cu = [0, 64, 134]
    for t in range(130):
        new = [int(t < n) for n in lens]
        rows = [cu[i] + t for i in range(3) if new[i]]
        b.append(k[rows], v[rows], cu_of(new))
    assert ok(b) == 0
    for i, n in enumerate(lens):
        pa, pb = a.table[i, :n // 64].long(), b.table[i, :n // 64].long()
        assert torch.equal(a.pages[pa], b.pages[pb]) and torch.equal(a.scales[pa], b.scales[pb])
        assert torch.equal(a.tail[i, :, :, :n % 64], b.tail[i, :, :, :n % 64])


def test_append_single_form_and_strides():
    """Without cu_tokens; k and v slices of one projection's output with different token strides."""
    c, k, v = filled([62, 0, 127, 5], 2, max_blocks=3)
    tail, mine = c.tail.clone(), {b: U.tokens_of(c, b) for b in range(4)}
    for step in range(3):
        qkv = rand((4, 8, 128), BF16, step)
        other = rand((4, 6, 128), BF16, step + 5)
        c.append(qkv[:, 4:6], other[:, 2:4])
        for b in range(4):
            pos = int(c.seq_lens[b]) - 1
            if (pos + 1) % 64:
                assert torch.equal(c.tail[b, :, 0, pos % 64], qkv[b, 4:6]) and torch.equal(c.tail[b, :, 1, pos % 64], other[b, 2:4])
    assert ok(c) == 0 and c.seq_lens.tolist() == [65, 3, 130, 8]
    # rows that no new token took are as they were: sequence 0 filled its block (row 63 stays), then opened row 0
    assert torch.equal(c.tail[0, :, :, 1:62], tail[0, :, :, 1:62]) and torch.equal(c.tail[0, :, :, 63], tail[0, :, :, 63])
    assert torch.equal(c.tail[3, :, :, 8:], tail[3, :, :, 8:])
    assert torch.equal(U.tokens_of(c, 3)[:, :5], mine[3])


@pytest.mark.parametrize("fmt", [E4, E5])
def test_append_special_blocks(fmt):
    """Zeros, the type's extremes, subnormal magnitudes, NaN and infinities, each in a block of its own."""
    k = rand((64 * 8, 1, 128), BF16, 3)
    v = rand((64 * 8, 1, 128), BF16, 4)
    big, tiny = torch.finfo(BF16).max, 2.0 ** -133
    k[0:64] = 0
    v[0:64] = -0.0
    k[64:128] *= tiny
    v[64:128] = tiny
    k[130, 0, 7] = big
    v[130, 0, 7] = -big
    k[200, 0, 0], k[201, 0, 1], k[202, 0, 2] = math.nan, math.inf, -math.inf
    v[256:320] = math.inf
    k[256:320] = math.nan
    k[320:384] = 1.75  # the format's largest number in every place
    v[320:384] = -1.765625  # just above: the next scale
    c = Kv8Cache(8, 1, 1, 8, fmt, BF16)
    c.append(k, v, cu_of([512]))
    assert ok(c) == 0
    check_blocks(c, {0: torch.stack([k, v])})
    assert c.scales[c.table[0, 0].long()].eq(1).all()


def test_append_refused_on_the_device():
    c, _, _ = filled([60, 60, 64, 192], 2, max_blocks=3, spare=1)
    before = [t.clone() for t in c._tensors[:6]]
    k, v = kv_of(40, 2, BF16, 9)
    # sequence 0 lacks a page, 1 has one, 3 would pass the table
    c.table[1, 0] = -1
    c.table[0, 0] = -1
    free = int((c.refs == 0).nonzero()[0])
    c.table[1, 0] = free
    c.append(k, v, cu_of([10, 10, 10, 10]), reserve=False)
    assert ok(c) in (G.EPOOL, G.EINVAL)
    assert c.seq_lens.tolist() == [60, 70, 74, 192]
    assert torch.equal(c.tail[0], before[2][0]) and torch.equal(c.tail[3], before[2][3])
    # the sequence works again once it has a page
    c.status.zero_()
    c.refs[free] = 1
    c.release(ints([3]))
    c.append(k[:10], v[:10], cu_of([10, 0, 0, 0]))
    assert ok(c) == 0 and c.seq_lens.tolist() == [70, 70, 74, 0]
    # offsets that are not valid: nothing happens
    lens = c.seq_lens.tolist()
    for cu in ([0, 5, 3, 10, 10], [0, 10, 20, 30, 41], [-1, 10, 20, 30, 40]):
        c.status.zero_()
        c.append(k, v, ints(cu), reserve=False)
        assert ok(c) == G.EINVAL and c.seq_lens.tolist() == lens
    c.status.zero_()
    c.append(k, v, ints([20, 20, 20, 20, 30]), reserve=False)  # rows before the first offset belong to nobody
    assert ok(c) == 0 and c.seq_lens.tolist() == lens[:3] + [10]
    assert torch.equal(c.tail[3, :, 0, :10].transpose(0, 1), k[20:30])


def test_append_many_and_long():
    """More sequences than a warp looks up at once, and runs of many blocks."""
    lens = [(53 * i) % 200 for i in range(700)]
    c, k, v = filled(lens, 1)
    at = torch.cumsum(torch.tensor([0] + lens), 0).tolist()
    check_blocks(c, {b: torch.stack([k[at[b]:at[b + 1]], v[at[b]:at[b + 1]]]) for b in (0, 1, 31, 32, 33, 255, 256, 699)})
    c, k, v = filled([30011, 63, 20000], 4, E5, F16)
    check_blocks(c, {0: torch.stack([k[:30011], v[:30011]]), 1: torch.stack([k[30011:30074], v[30011:30074]]),
                     2: torch.stack([k[30074:], v[30074:]])})
    # chunks of many blocks behind open ones
    n = [9000, 1, 7777]
    k2, v2 = kv_of(sum(n), 4, F16, 60)
    d = Kv8Cache(c.n_pages + 300, 3, 4, c.max_blocks + 160, E5, F16)
    d.append(k, v, cu_of([30011, 63, 20000]))
    d.append(k2, v2, cu_of(n))
    assert ok(d) == 0
    check_blocks(d, {0: torch.stack([torch.cat([k[:30011], k2[:9000]]), torch.cat([v[:30011], v2[:9000]])]),
                     1: torch.stack([torch.cat([k[30011:30074], k2[9000:9001]]), torch.cat([v[30011:30074], v2[9000:9001]])]),
                     2: torch.stack([torch.cat([k[30074:], k2[9001:]]), torch.cat([v[30074:], v2[9001:]])])})


def test_append_empty_chunk():
    c, _, _ = filled([3, 64], 1)
    e = torch.empty((0, 1, 128), dtype=BF16, device="cuda")
    c.append(e, e, ints([0, 0, 0]))
    assert ok(c) == 0 and c.seq_lens.tolist() == [3, 64]


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt,dtype", [(E4, BF16), (E5, F16), (E4, F16), (E5, BF16)])
@pytest.mark.parametrize("lens,heads,group", [([1], 1, 1), ([64], 2, 4), ([65, 0, 63], 2, 8), ([777], 8, 2),
                                              ([5, 128, 129, 191, 192, 1000], 4, 5), ([4096, 1, 300, 2049], 2, 7),
                                              ([20000], 1, 8), ([63] * 40, 3, 3)])
def test_attention(lens, heads, group, fmt, dtype):
    c, _, _ = filled(lens, heads, fmt, dtype)
    q = rand((len(lens), heads * group, 128), dtype, 5)
    out = c.attention(q, SCALE)
    assert ok(c) == 0 and out.dtype == dtype
    U.check_attention(c, q, SCALE, out)
    full = torch.full(q.shape, math.nan, dtype=F32, device="cuda")
    assert c.attention(q, SCALE, out=full) is full
    U.check_attention(c, q, SCALE, full)
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()


def test_attention_many_short_sequences():
    """More (sequence, head) pairs than the GPU holds at once, ragged, with empty rows among them."""
    lens = [(37 * i) % 400 for i in range(300)]
    c, _, _ = filled(lens, 4)
    q = rand((300, 16, 128), BF16, 5)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    assert ok(c) == 0


@pytest.mark.parametrize("lens,heads,group", [
    ([70000], 1, 1), ([70000], 1, 3), ([40000, 39999], 1, 8),  # shared by most of the GPU: joined in teams
    ([100000] + [10] * 200, 1, 8), ([5] * 100 + [60001] + [130] * 100, 1, 5),  # the same among short ones
    ([64 * (i % 25) + 17 * (i % 3) for i in range(90)], 5, 2),  # up to 25 blocks, several heads side by side
    ([1] * 64, 8, 4), ([0] * 200, 2, 1), ([33] * 160 + [2000], 2, 8), ([1300] * 60, 3, 4), ([129, 0, 1] * 40, 16, 1)])
def test_attention_cuts(lens, heads, group):
    """Every way the blocks are cut over the GPU; twice the same bits."""
    c, _, _ = filled(lens, heads)
    q = rand((len(lens), heads * group, 128), BF16, 5)
    a = c.attention(q, SCALE)
    U.check_attention(c, q, SCALE, a)
    b = c.attention(q, SCALE)
    assert torch.equal(a, b) and ok(c) == 0
    assert all((a[i] == 0).all() for i, n in enumerate(lens) if n == 0)
    assert (c._ws[:3 * 152 * 4].view(torch.int32) == 0).all()  # counters are back at zero


def test_attention_thousands_of_sequences_and_many_heads():
    lens = [(29 * i) % 150 for i in range(6000)]
    c, _, _ = filled(lens, 1)
    q = rand((6000, 2, 128), BF16, 5)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    c, _, _ = filled([70, 0, 2000], 96, E5, F16)
    q = rand((3, 96 * 3, 128), F16, 5)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    assert ok(c) == 0


@pytest.mark.parametrize("batch", (31, 32, 33, 64, 65, 150, 255, 257, 1023, 1024, 1025, 2049))
def test_attention_sequence_counts(batch):
    """Where lengths are read by 32, by 256 and by 1,024; empty sequences at the ends, one long among them."""
    lens = [0 if i % 7 == 3 else (37 * i) % 131 for i in range(batch)]
    lens[0] = lens[-1] = 0
    lens[batch // 2] = 64 * 23 + 5
    c, _, _ = filled(lens, 1)
    q = rand((batch, 2, 128), BF16, batch)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    # Only the last has tokens; then none: the results are zeros.
    c, _, _ = filled([0] * (batch - 1) + [130], 1)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    c, _, _ = filled([0] * batch, 1)
    assert (c.attention(q, SCALE) == 0).all()
    assert ok(c) == 0


def test_attention_scales_far_apart():
    """V scales 2^-40 .. 2^40 apart between blocks, K scales 2^-6 .. 2^6, and scores that favour either end."""
    c, _, _ = filled([64 * 40 + 7] * 3, 2)
    e = torch.randint(-40, 41, c.scales.shape[:2], generator=torch.Generator().manual_seed(1)).cuda()
    c.scales[:, :, 1] = torch.exp2(e.float())
    c.scales[:, :, 0] = torch.exp2((e % 13 - 6).float() - 6)
    q = rand((3, 8, 128), BF16, 5)
    for scale in (SCALE, -SCALE, 0.0, 3.0):
        U.check_attention(c, q, scale, c.attention(q, scale, out=torch.empty(q.shape, device="cuda")))
    # scales that are not powers of two
    c.scales.mul_(torch.rand(c.scales.shape, device="cuda") + 0.5)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    assert ok(c) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_query_range(dtype):
    """Queries of 1e4 with a small scale and of 1e-4 with a large one; one row of zeros."""
    c, _, _ = filled([300, 64, 40], 2, E4, dtype)
    for mul in (1e4, 1e-4):
        q = rand((3, 8, 128), F32, 5)
        q = (q * mul).to(dtype)
        q[0, 3] = 0
        U.check_attention(c, q, SCALE / mul, c.attention(q, SCALE / mul))
    if dtype == BF16:
        q = (rand((3, 8, 128), F32, 5) * 1e30).to(dtype)
        U.check_attention(c, q, 1e-31, c.attention(q, 1e-31))
    assert ok(c) == 0


def test_attention_ignores_what_is_not_its_own():
    """Rows behind the open block's tokens, other pages and entries behind the length: NaN there changes nothing."""
    lens = [130, 1, 64, 0, 127]
    c, _, _ = filled(lens, 2, max_blocks=6)
    q = rand((5, 8, 128), BF16, 5)
    a = c.attention(q, SCALE)
    for b, n in enumerate(lens):
        c.tail[b, :, :, n % 64:] = math.nan if b % 2 else math.inf
        c.table[b, n // 64:] = 2 ** 31 - 1 if b % 2 else -7
    c.pages[c.refs == 0] = 0x7F
    c.scales[c.refs == 0] = math.nan
    assert torch.equal(c.attention(q, SCALE), a) and ok(c) == 0


def test_attention_nan_and_infinite_tokens():
    """A NaN in a head's key spoils that head's rows alone; an infinite logit makes its weight NaN as in a softmax."""
    c, k, v = filled([200, 200], 2)
    q = rand((2, 8, 128), BF16, 5)
    a = c.attention(q, SCALE)
    page = int(c.table[0, 1])
    c.pages[page, 1, 0, 3, 5] = 0x7F
    b = c.attention(q, SCALE)
    assert torch.isnan(b[0, 4:]).all() and torch.equal(b[0, :4], a[0, :4]) and torch.equal(b[1], a[1])
    c.pages[page, 1, 0, 3, 5] = 0
    c.tail[1, 0, 1, 2, 9] = math.nan  # V, token 194 of sequence 1, channel 9
    b = c.attention(q, SCALE)
    bad = torch.isnan(b)
    assert bad[1, :4, 9].all() and bad.sum() == 4


def test_attention_short_pairs_results():
    """Pairs that one group ends alone, between longer ones: every result type, and what is not finite stays put."""
    lens = [(53 * i) % 190 if i % 40 else 64 * 30 for i in range(161)]
    for fmt, dtype, group in ((E4, BF16, 4), (E5, F16, 8), (E4, F16, 1)):
        c, _, _ = filled(lens, 2, fmt, dtype)
        q = rand((161, 2 * group, 128), dtype, 6)
        for out in (dtype, torch.float32):
            U.check_attention(c, q, SCALE, c.attention(q, SCALE, torch.empty(q.shape, dtype=out, device="cuda")))
    c, _, _ = filled(lens, 2)
    q = rand((161, 8, 128), BF16, 6)
    a = c.attention(q, SCALE)
    assert torch.equal(a, c.attention(q, SCALE))
    b1 = next(b for b in range(60, 161) if 64 <= lens[b] < 128 and lens[b] % 64)
    b2 = next(b for b in range(b1 + 1, 161) if 64 < lens[b] < 190 and lens[b] % 64 > 3)
    c.pages[int(c.table[b1, 0]), 1, 0, 3, 5] = 0x7F  # a key of head 1
    c.tail[b2, 0, 1, 2, 9] = math.inf  # V of head 0, channel 9: infinite, or NaN by the weights' second part
    x = c.attention(q, SCALE)
    assert torch.isnan(x[b1, 4:]).all()
    assert not torch.isfinite(x[b2, :4, 9]).any()
    x[b1, 4:] = a[b1, 4:]
    x[b2, :4, 9] = a[b2, :4, 9]
    assert torch.equal(x, a)
    assert ok(c) == 0


def test_attention_bad_table_and_lengths():
    c, _, _ = filled([300, 300, 300], 2)
    q = rand((3, 8, 128), BF16, 5)
    a = c.attention(q, SCALE)
    good = c.table.clone()
    for bad in (c.n_pages, -1, 2 ** 31 - 1, -2 ** 31):
        c.table[1, 2] = bad
        b = c.attention(q, SCALE)
        assert ok(c) == G.EFORMAT
        c.status.zero_()
        assert torch.equal(b[0], a[0]) and torch.equal(b[2], a[2]) and torch.isfinite(b).all()
    c.table.copy_(good)
    for bad in (-1, 64 * c.max_blocks + 1, 2 ** 31 - 1, -2 ** 31):
        c.seq_lens[1] = bad
        b = c.attention(q, SCALE)
        assert ok(c) == G.EINVAL
        c.status.zero_()
        assert torch.equal(b[0], a[0]) and torch.equal(b[2], a[2]) and (b[1] == 0).all()
    c.seq_lens[1] = 300
    assert torch.equal(c.attention(q, SCALE), a) and ok(c) == 0


def test_attention_strided_queries_streams_and_graph():
    c, _, _ = filled([700, 33, 1500], 4)
    qkv = rand((3, 24, 128), BF16, 5)
    q = qkv[:, :16]
    a = c.attention(q.contiguous(), SCALE)
    assert torch.equal(c.attention(q, SCALE), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = c.attention(q, SCALE, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(b, a)
    out = torch.empty_like(a)
    g = torch.cuda.CUDAGraph()
    k1, v1 = kv_of(3, 4, BF16, 50)
    with torch.cuda.graph(g):
        c.append(k1, v1)
        c.attention(q, SCALE, out=out)
    h = torch.cuda.CUDAGraph()
    out2 = torch.empty_like(a)
    with torch.cuda.graph(h):  # a second graph over the same cache and workspace, replayed in turn
        c.attention(q, SCALE, out=out2)
    for step in range(3):
        g.replay()
        h.replay()
        assert ok(c) == 0 and c.seq_lens.tolist() == [701 + step, 34 + step, 1501 + step]
        U.check_attention(c, q, SCALE, out)
        assert torch.equal(out, out2)


def test_attention_offsets_past_32_bits():
    """A pool of more than 4 GB: pages at its end."""
    n = 36000
    c = Kv8Cache(n, 2, 8, 40, E4, BF16)
    k, v = kv_of(2 * 2000, 8, BF16, 1)
    c.reserve(ints([0, 2000, 4000]))
    c.refs.zero_()
    c.table.copy_(torch.where(c.table >= 0, n - 1 - c.table, c.table))
    c.refs[-62:] = 1
    c.append(k, v, ints([0, 2000, 4000]), reserve=False)
    q = rand((2, 16, 128), BF16, 5)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    moved = c.compact()
    assert moved[-62:].sort().values.tolist() == list(range(62))
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    check_blocks(c, {0: torch.stack([k[:2000], v[:2000]]), 1: torch.stack([k[2000:], v[2000:]])})
    assert ok(c) == 0


def test_attention_refusals():
    c, _, _ = filled([10, 10], 2)
    q = rand((2, 8, 128), BF16)
    for bad in (lambda: c.attention(q.half(), SCALE), lambda: c.attention(q[:1], SCALE), lambda: c.attention(q.cpu(), SCALE),
                lambda: c.attention(q[..., :64], SCALE), lambda: c.attention(q, SCALE, out=torch.empty_like(q)[:, :4]),
                lambda: c.attention(q, SCALE, out=q.half()), lambda: c.attention(q.transpose(0, 1), SCALE)):
        with pytest.raises(ValueError):
            bad()
    for n in (7, 36):
        with pytest.raises(G.GaacError) as e:
            c.attention(rand((2, n, 128), BF16), SCALE)
        assert e.value.status == G.EINVAL
    with pytest.raises(G.GaacError):
        c.attention(q, math.nan)
    with pytest.raises(ValueError):
        c.append(q[:, :2], q[:, :3])
    with pytest.raises(ValueError):
        c.append(q[:1, :2], q[:1, :2])
    with pytest.raises(ValueError):
        c.append(q[:, :2], q[:, :2], ints([0, 1]))
    with pytest.raises(ValueError):
        c.release(torch.tensor([0], device="cuda"))
    with pytest.raises(ValueError):
        c.fork(ints([0]), ints([0, 1]))
    with pytest.raises(ValueError):
        G.kv8_compact(c, ints([0]))


# ------------------------------------------------------------------ pages

def both(c, m, what, *args):
    """The call on the cache and on the plain model."""
    if what in ("reserve", "append"):
        new = args[0]
        if what == "append":
            k, v = kv_of(max(1, sum(new)), c.n_kv_heads, c.dtype, sum(new))
            c.append(k, v, cu_of(new), reserve=False)
        else:
            c.reserve(cu_of(new))
        getattr(m, what)(new)
    elif what == "compact":
        assert c.compact().tolist() == m.compact()
    else:
        getattr(c, what)(*(ints(a) for a in args))
        getattr(m, what)(*args)
    torch.cuda.synchronize()
    m.check(c)


@pytest.mark.parametrize("n_pages,batch,max_blocks", [(1, 1, 1), (7, 3, 4), (63, 5, 40), (8193, 40, 300), (20000, 70, 33)])
def test_page_calls_follow_the_model(n_pages, batch, max_blocks):
    rng = random.Random(n_pages)
    c, m = Kv8Cache(n_pages, batch, 1, max_blocks), U.Model(n_pages, batch, max_blocks)
    for step in range(24):
        what = rng.choice(["grow", "grow", "reserve", "release", "fork", "compact"])
        some = [rng.randrange(-1, batch + 1) for _ in range(rng.randrange(0, batch + 1))]
        if what in ("grow", "reserve"):
            most = rng.choice([1, 70, 64 * max_blocks // 3 + 1])
            new = [rng.randrange(most + 1) for _ in range(batch)]
            both(c, m, "reserve", new)
            if what == "grow":
                both(c, m, "append", new)
        elif what == "fork":
            both(c, m, "fork", some, [rng.randrange(-1, batch + 1) for _ in some])
        elif what == "release":
            both(c, m, "release", some)
        else:
            both(c, m, "compact")


def test_fork_shares_and_release_gives_back():
    c, k, v = filled([200, 0, 0, 0], 2, max_blocks=6, spare=10)
    q = rand((1, 8, 128), BF16, 5).expand(4, 8, 128).contiguous()
    c.fork(ints([0, 0, 0]), ints([1, 3, 2]))
    a = c.attention(q, SCALE)
    assert ok(c) == 0 and all(torch.equal(a[0], a[i]) for i in range(1, 4))
    assert int((c.refs > 0).sum()) == 3 and c.refs.max() == 4
    # the branches grow apart without touching one another
    own = {}
    for b in range(4):
        n = 30 + 40 * b
        kb, vb = kv_of(n, 2, BF16, 100 + b)
        new = [0] * 4
        new[b] = n
        c.append(kb, vb, cu_of(new))
        own[b] = torch.cat([torch.stack([k, v]), torch.stack([kb, vb])], 1)
    assert ok(c) == 0
    check_blocks(c, own)
    U.check_attention(c, q, SCALE, c.attention(q, SCALE))
    c.release(ints([0, 2, 0]))
    check_blocks(c, {1: own[1], 3: own[3]})
    c.compact()
    check_blocks(c, {1: own[1], 3: own[3]})
    c.release(ints([1, 3]))
    assert ok(c) == 0 and (c.refs == 0).all() and (c.table == -1).all() and (c.seq_lens == 0).all()


def test_fork_and_release_refusals():
    c, _, _ = filled([100, 64, 0, 0, 0], 1, max_blocks=4, spare=4)
    c.reserve(cu_of([0, 0, 64, 0, 0]))  # sequence 2: empty, but with a page reserved
    m = U.Model(c.n_pages, 5, 4)
    m.table, m.refs, m.lens = c.table.tolist(), c.refs.tolist(), c.seq_lens.tolist()
    for src, dst in (([0], [1]), ([0], [2]), ([0], [5]), ([-1], [3]), ([0, 1], [3, 3]), ([0, 3], [4, 1]), ([0], [0])):
        c.status.zero_()
        both(c, m, "fork", src, dst)
        assert ok(c) == G.EINVAL
    c.status.zero_()
    both(c, m, "release", [2, 2, -1])
    assert ok(c) == G.EINVAL
    c.status.zero_()
    c.table[0, 0] = c.n_pages
    c.fork(ints([0]), ints([2]))
    assert ok(c) == G.EFORMAT and int(c.seq_lens[2]) == 0
    c.status.zero_()
    c.release(ints([0]))
    assert ok(c) == G.EFORMAT and (c.table[0] == -1).all()


def test_pool_runs_out_and_recovers():
    c, m = Kv8Cache(5, 3, 1, 8), U.Model(5, 3, 8)
    new = [128, 128, 128]
    both(c, m, "reserve", new)
    assert ok(c) == G.EPOOL
    both(c, m, "append", new)  # the third sequence lacks a page and stays as it was
    assert c.seq_lens.tolist() == [128, 128, 0]
    c.status.zero_()
    both(c, m, "release", [0])
    both(c, m, "reserve", [0, 0, 128])
    both(c, m, "append", [0, 0, 128])
    assert ok(c) == 0 and c.seq_lens.tolist() == [0, 128, 128]
    c.reserve(ints([0, 600, 600, 600]))  # past the table
    assert ok(c) == G.EINVAL
    m.check(c)


def test_full_and_empty_pools_compact():
    c, m = Kv8Cache(9, 2, 1, 9), U.Model(9, 2, 9)
    both(c, m, "compact")
    both(c, m, "reserve", [320, 256])
    both(c, m, "append", [320, 256])
    both(c, m, "compact")
    assert ok(c) == 0


def test_page_calls_captured_and_on_another_stream():
    """A scheduler's step in a graph, replayed with other lists and lengths, and the same calls on a side stream."""
    c, m = Kv8Cache(300, 12, 1, 30), U.Model(300, 12, 30)
    done, src, dst, cu = ints([0, 1, 2]), ints([5, 5, 7]), ints([0, 1, 2]), ints([0] * 13)
    k, v = kv_of(2000, 1, BF16, 3)
    moved = ints([0] * 300)
    both(c, m, "reserve", [100] * 12)
    both(c, m, "append", [100] * 12)

    def step(stream=None):
        c.release(done, stream=stream)
        c.fork(src, dst, stream=stream)
        c.append(k, v, cu, stream=stream)
        G.kv8_compact(c, moved, stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = random.Random(1)
    for i in range(12):
        rows = rng.sample(range(12), 6)
        new = [rng.randrange(160) for _ in range(12)]
        lists = [rows[:3], [rng.choice(rows[3:]) for _ in range(3)], rows[:3]]
        for t, x in zip((done, src, dst, cu), lists + [cu_of(new)]):
            t.copy_(x if isinstance(x, torch.Tensor) else ints(x))
        if i % 3 == 2:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            step(s)
            torch.cuda.current_stream().wait_stream(s)
        else:
            g.replay()
        m.release(lists[0])
        m.fork(lists[1], lists[2])
        m.reserve(new)
        m.append(new)
        assert moved.tolist() == m.compact()
        m.check(c)
        # what does not fit is reported and leaves its sequence as it was, which the model follows
        c.status.zero_()


def test_append_rows_past_32_bits():
    """k and v are columns of a buffer of 2.4e9 elements: rows 60,000 elements apart."""
    buf = torch.zeros((40000, 60000), dtype=BF16, device="cuda")
    k, v = kv_of(40000, 1, BF16, 1)
    buf[:, 128:256], buf[:, 59872:] = k[:, 0], v[:, 0]
    c = Kv8Cache(640, 2, 1, 640, E4, BF16)
    c.append(buf[:, None, 128:256], buf[:, None, 59872:], ints([0, 100, 40000]))
    assert ok(c) == 0
    check_blocks(c, {0: torch.stack([k[:100], v[:100]]), 1: torch.stack([k[100:], v[100:]])})


def test_whole_flow_on_a_side_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c, _, _ = filled([300, 65, 0], 2)
        q = rand((3, 8, 128), BF16, 5)
        c.fork(ints([0]), ints([2]))
        out = c.attention(q, SCALE)
        c.release(ints([1]))
        c.compact()
        again = c.attention(q, SCALE)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out[0], again[0]) and torch.equal(out[2], again[2]) and (again[1] == 0).all()
    U.check_attention(c, q, SCALE, again)
    assert ok(c) == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,dtype", [(E4, BF16), (E5, F16)])
def test_serving_run(fmt, dtype):
    """Prefill, forks, decode steps with rotary positions in a captured graph, release, compact: the attention at
    every step against 64 bits over exactly the tokens that went in."""
    heads, group, B = 2, 4, 6
    w, ms = G.rope_frequencies(128, 1e6, "bands", 4.0, original_len=1024)
    turns = G.rope_turns(w, "cuda")
    c = Kv8Cache(64, B, heads, 12, fmt, dtype)
    seen = {}

    def take(k, v, new):
        at = 0
        for b, n in enumerate(new):
            seen[b] = torch.cat([seen.get(b, torch.zeros((2, 0, heads, 128), dtype=dtype, device="cuda")),
                                 torch.stack([k[at:at + n], v[at:at + n]])], 1)
            at += n

    new = [150, 64, 0, 3, 0, 0]
    q, (k, v) = rand((sum(new), heads * group, 128), dtype, 1), kv_of(sum(new), heads, dtype, 2)
    pos = torch.cat([torch.arange(n) for n in new]).cuda()
    k0 = k.clone()
    G.rope(q, k, pos, turns, mscale=ms)
    assert ((k.double() - U.rope_ref(k0, pos, w, mscale=ms)).abs() <= torch.finfo(dtype).eps * 4 * (k0.double().abs().amax())).all()
    c.append(k, v, cu_of(new))
    take(k, v, new)
    c.fork(ints([0, 0, 3]), ints([2, 4, 5]))
    seen.update({2: seen[0], 4: seen[0], 5: seen[3]})
    assert ok(c) == 0
    check_blocks(c, seen)
    # decode steps: one graph for rope, append and attention
    qs, ks, vs = rand((B, heads * group, 128), dtype), rand((B, heads, 128), dtype), rand((B, heads, 128), dtype)
    out = torch.empty_like(qs)

    def step():
        G.rope(qs, ks, c.seq_lens, turns, mscale=ms)
        c.append(ks, vs)
        c.attention(qs, SCALE, out=out)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(70):
        if i == 40:
            c.release(ints([1, 4]))
            seen[1] = seen[4] = torch.zeros((2, 0, heads, 128), dtype=dtype, device="cuda")
            c.compact()
        qs.copy_(rand((B, heads * group, 128), dtype, 100 + i))
        kn, vn = kv_of(B, heads, dtype, 300 + i)
        ks.copy_(kn)
        vs.copy_(vn)
        g.replay()
        take(ks, vs, [1] * B)
        if i % 13 == 0 or i == 41:
            U.check_attention(c, qs, SCALE, out)
            check_blocks(c, seen)
    assert ok(c) == 0
    check_blocks(c, seen)


@pytest.mark.parametrize("fmt,dtype", [(E4, BF16), (E5, BF16), (E4, F16), (E5, F16)])
@pytest.mark.parametrize("lens", [[777], [5, 0, 64, 130, 20000], [(53 * i) % 190 for i in range(161)]], ids=["one", "mixed", "short"])
def test_attention_16_bit_result_is_the_rounded_32_bit_one(lens, fmt, dtype):
    """The result's type changes its last rounding alone, none on the way to it."""
    c, _, _ = filled(lens, 2, fmt, dtype)
    q = rand((len(lens), 8, 128), dtype, 5)
    full = c.attention(q, SCALE, out=torch.empty(q.shape, dtype=F32, device="cuda"))
    assert torch.equal(c.attention(q, SCALE), full.to(dtype))
    # weights in two parts over the pages: 2^-22 of each is lost (2^-16 over an open block in bf16), whatever the result
    ref, bound = U.attention_ref(c, q, SCALE, 2.0 ** -16 if dtype == BF16 else 2.0 ** -20)
    half = torch.finfo(dtype).eps / 2
    err = (c.attention(q, SCALE).double() - ref).abs()
    assert (err <= bound * (1 + half) + half * ref.abs() + torch.finfo(dtype).tiny).all()
    assert ok(c) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,b", [([130], 0), ([70000], 0), ([30, 200, 64 * 9 + 50], 2), ([100 + i % 60 for i in range(161)], 60)],
                         ids=["one", "joined", "few", "short"])
def test_attention_infinite_values(lens, b, dtype):
    """V infinite in a channel: its weighted sum is, with the sign, however small the weight; NaN where both signs
    meet or a value is NaN.  In pages (E5M2) and in the open block; the other channels and rows keep their bits."""
    c, _, _ = filled(lens, 2, E5, dtype)
    q = rand((len(lens), 8, 128), dtype, 5)
    q[b, :4] = q[b, :1]  # the rows of head 0 alike
    types = (dtype, F32)
    plain = [c.attention(q, SCALE, out=torch.empty(q.shape, dtype=t, device="cuda")) for t in types]
    ids, n = c.table[b].tolist(), lens[b]
    inf8 = torch.tensor([math.inf, -math.inf, math.nan], device="cuda").to(U.FP8[E5]).view(torch.uint8).tolist()
    c.pages[ids[0], 0, 1, 5, 3] = inf8[0]
    c.pages[ids[0], 0, 1, 63, 64] = inf8[1]
    c.pages[ids[0], 0, 1, 2, 77] = inf8[0]
    c.pages[ids[0], 0, 1, 40, 77] = inf8[1]
    c.pages[ids[0], 0, 1, 9, 100] = inf8[2]
    c.tail[b, 0, 1, 1, 9] = math.inf  # the open block's second token
    c.tail[b, 0, 1, n % 64 - 1, 127] = -math.inf
    c.tail[b, 0, 1, n % 64:, 50] = math.inf  # behind its last
    for t, a in zip(types, plain):
        x = c.attention(q, SCALE, out=torch.empty(q.shape, dtype=t, device="cuda"))
        for ch, v in ((3, math.inf), (64, -math.inf), (9, math.inf), (127, -math.inf)):
            assert (x[b, :4, ch] == v).all(), (t, ch, x[b, :4, ch])
        assert torch.isnan(x[b, :4, 77]).all() and torch.isnan(x[b, :4, 100]).all()
        for ch in (3, 64, 9, 127, 77, 100):
            x[b, :4, ch] = a[b, :4, ch]
        assert torch.equal(x, a)
    assert ok(c) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("low", [5.0, 25.0, 40.0, 60.0, 100.0])
def test_attention_infinite_values_of_small_weight(low, dtype):
    """Token 5's logit is `low` powers of two below the others' (its weight is not 0 in 32 bits), in a page and in the
    open block; what is finite of such a token counts as before."""
    c = Kv8Cache(4, 2, 1, 4, E5, dtype)
    k, v = torch.zeros((2 * 100, 1, 128), dtype=dtype, device="cuda"), rand((2 * 100, 1, 128), dtype, 3)
    q = torch.zeros((2, 1, 128), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    at = (5, 100 + 70)  # sequence 0: in its page; sequence 1: in its open block
    for i in at:
        k[i, 0, 0] = -low
        v[i, 0, 9] = math.inf
    c.append(k, v, cu_of([100, 100]))
    scale = math.log(2.0)
    for t in (dtype, F32):
        x = c.attention(q, scale, out=torch.empty(q.shape, dtype=t, device="cuda"))
        assert (x[:, 0, 9] == math.inf).all(), x[:, 0, 9]
        assert torch.isfinite(x).sum() == x.numel() - 2
        c.tail[1, 0, 1, 6, 9] = 0.0
        page = c.pages[int(c.table[0, 0]), 0, 1, 5]
        page[9] = 0
        U.check_attention(c, q, scale, c.attention(q, scale, out=torch.empty(q.shape, dtype=t, device="cuda")))
        c.tail[1, 0, 1, 6, 9] = math.inf
        page[9] = 0x7C
    assert ok(c) == 0


BUSY = 40_000_000  # cycles that a stream is kept busy: some 20 ms


def side_streams():
    """A stream, as an object and as the raw handle of another."""
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    return ((s, s), (t, t.cuda_stream))


@pytest.mark.parametrize("what", ["attention", "compact"])
def test_results_on_a_side_stream_take_no_memory_in_use(what):
    """The result of a call with `stream` is not memory that the current stream's pending work still reads, nor is it
    given out again while the current stream reads it."""
    c, _, _ = filled([700, 33, 1500], 4)
    q = rand((3, 16, 128), BF16, 5)
    run = (lambda s: c.attention(q, SCALE, stream=s)) if what == "attention" else (lambda s: c.compact(stream=s))
    right = run(None)
    c.compact()
    right = run(None)  # of a compact pool, which a further compaction leaves as it is
    for s, handle in side_streams():
        torch.cuda.synchronize()
        used = torch.full_like(right, 7)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        seen = used.clone()
        del used  # its block is free for the current stream, which still has to read it
        out = run(handle)
        torch.cuda.synchronize()
        assert (seen == 7).all()
        assert torch.equal(out, right)
        # the other way round: read here, freed, and its memory asked for again there
        torch.cuda._sleep(BUSY)
        seen = out.clone()
        del out
        with torch.cuda.stream(s):
            other = torch.full_like(right, 7)
        torch.cuda.synchronize()
        assert torch.equal(seen, right) and (other == 7).all()


def test_append_with_bad_offsets_reserves_nothing():
    """Offsets that the append refuses as a whole, or tensors that it refuses, leave the table and the counts alone."""
    c, _, _ = filled([60, 60, 64, 0], 2, max_blocks=6, spare=12)
    k, v = kv_of(400, 2, BF16, 9)
    table, refs, lens = c.table.clone(), c.refs.clone(), c.seq_lens.clone()

    def same():
        return torch.equal(c.table, table) and torch.equal(c.refs, refs) and torch.equal(c.seq_lens, lens)

    for cu in ([0, 100, 50, 200, 400], [0, 100, 200, 300, 401], [-1, 100, 200, 300, 400], [0, 0, 0, 0, 2 ** 31 - 1],
               [0, 200, 100, 300, 200], [-2 ** 31, 0, 100, 200, 300]):
        c.append(k, v, ints(cu))
        assert ok(c) == G.EINVAL and same(), cu
        c.status.zero_()
    for cu in ([0, 100, 50, 200, 400], [-1, 100, 200, 300, 400], [0, 200, 100, 300, 200]):
        c.reserve(ints(cu))
        assert ok(c) == G.EINVAL and same(), cu
        c.status.zero_()
    for bad in (lambda: c.append(k, v[:300], cu_of([100, 100, 100, 100])), lambda: c.append(k, v.half(), cu_of([100] * 4)),
                lambda: c.append(k[:3], v[:3])):
        with pytest.raises(ValueError):
            bad()
        assert same()
    odd = torch.empty(400 * 256 + 1, dtype=BF16, device="cuda")[1:].view(400, 2, 128)
    with pytest.raises(G.GaacError):
        c.append(odd, v, cu_of([100] * 4))
    assert ok(c) == 0 and same()
    # good offsets still work, with rows before the first and behind the last that belong to nobody
    c.append(k, v, ints([30, 40, 40, 140, 300]))
    assert ok(c) == 0 and c.seq_lens.tolist() == [70, 60, 164, 160]
    assert torch.equal(c.tail[3, :, 0, :32].transpose(0, 1), k[268:300])


def test_bad_offsets_among_thousands_of_sequences():
    """One offset out of order, wherever it stands and whichever CTA finds it; the next call is not affected."""
    c = Kv8Cache(20000, 5000, 1, 4)
    k, v = kv_of(5000 * 64, 1, BF16, 1)
    good = 64 * torch.arange(5001, dtype=torch.int32, device="cuda")
    for at in (0, 1, 31, 32, 1024, 4999, 5000):
        cu = good.clone()
        cu[at] += 100 if at < 5000 else 1
        c.append(k, v, cu)
        assert ok(c) == G.EINVAL and (c.table == -1).all() and (c.refs == 0).all() and (c.seq_lens == 0).all()
        c.status.zero_()
    c.append(k, v, good)
    assert ok(c) == 0 and torch.equal(c.table[:, 0], torch.arange(5000, dtype=torch.int32, device="cuda"))
    assert (c.seq_lens == 64).all() and int(c.refs.sum()) == 5000


def test_readme_serving_loop():
    """The 8-bit cache's example as it stands in README.md: ended sequences take no further tokens."""
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md"), encoding="utf-8") as f:
        code, = [x for x in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "Kv8Cache" in x]
    new = [70 + i if i < 30 else 0 for i in range(32)]
    k, v = kv_of(sum(new), 8, BF16, 1)
    names = dict(q=rand((sum(new), 16, 128), BF16, 3), k=k, v=v, cu=cu_of(new), scale=SCALE,
                 positions=torch.cat([torch.arange(n) for n in new]).cuda(), src=ints([0, 5]), dst=ints([30, 31]),
                 finished=ints([3, 0, 31]))
    for i in (1, 2):
        names[f"q{i}"] = rand((32, 16, 128), BF16, 10 + i)
        names[f"k{i}"], names[f"v{i}"] = kv_of(32, 8, BF16, 20 + 2 * i)
    exec(compile(code, "README.md", "exec"), names)
    c = names["cache"]
    want = [n + 2 for n in new]
    want[30], want[31] = new[0] + 2, new[5] + 2
    for b in (3, 0, 31):
        want[b] = 0
    assert ok(c) == 0 and c.seq_lens.tolist() == want
    assert all((c.table[b] == -1).all() for b in (3, 0, 31))
    c.fork(ints([1]), ints([3]))  # an ended sequence's row takes a new one
    assert ok(c) == 0 and int(c.seq_lens[3]) == want[1]
    assert (names["out"][[0, 31]] == 0).all()
    assert names["k8"].shape == c.pages.shape


def test_two_attentions_at_once():
    """Two streams, a workspace each, one cache: the results of one after the other."""
    c, _, _ = filled([30000, 33, 1500, 0, 700], 4)
    q = [rand((5, 16, 128), BF16, s) for s in (5, 6)]
    right = [c.attention(x, SCALE) for x in q]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in q], [torch.empty_like(x) for x in q]
    ws = [torch.zeros(G.kv8_attention_workspace(), dtype=torch.uint8, device="cuda") for _ in q]
    torch.cuda.synchronize()
    for _ in range(50):
        for i in (0, 1):
            G.kv8_decode_attention(c, q[i], SCALE, outs[i], ws[i], c.status, streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, right)) and ok(c) == 0
    assert all((w[:3 * 4 * torch.cuda.get_device_properties(0).multi_processor_count] == 0).all() for w in ws)
