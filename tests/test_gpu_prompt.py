"""Attention of whole prompts against 64 bits: lengths, head groups, strides, what is masked and what is not finite."""
import math

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from lossless_compressed_kv_gaac_gb300.cache import Beams, Kv8Cache

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def offsets(lens, first=0):
    return (torch.tensor([0] + list(lens)).cumsum(0) + first).to(torch.int32).cuda()


def reference(q, k, v, lens, scale, first=0):
    """(out, lse, bound) in 64 bits.  bound: the error before the result is rounded.  Logits: 128 products summed in fp32,
    each addition off by 2^-23 at most (no rounding to nearest is assumed), a further 2^-19 for their scaling and the
    exponentials.  Weights are rounded to the inputs' type; in f16 those below 2^-14 of a reference that is at most the
    row's largest are off by 2^-25 of it.  The sum over j keys adds j roundings of 2^-23."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    g = q.shape[1] // k.shape[1]
    half = torch.finfo(q.dtype).eps / 2
    a = first
    for n in filter(None, lens):
        for h in range(q.shape[1]):
            x, y, z = q[a:a + n, h].double(), k[a:a + n, h // g].double(), v[a:a + n, h // g].double()
            s = x @ y.T * scale
            mask = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            s = s.masked_fill(mask, -INF)
            p = torch.softmax(s, -1)
            out[a:a + n, h] = p @ z
            lse[a:a + n, h] = torch.logsumexp(s, -1)
            size = (x.abs() @ y.abs().T).masked_fill(mask, 0)
            d = size.amax(-1, keepdim=True) * abs(scale) * (2.0 ** -16 + 2.0 ** -19)
            seen = torch.arange(1, n + 1, device="cuda")[:, None]
            bound[a:a + n, h] = (p @ z.abs()) * (half + 2.0 ** -19 + 2.05 * d + seen * 2.0 ** -23)
            if q.dtype == FP16:
                bound[a:a + n, h] += 2.0 ** -25 * z.abs().cumsum(0)
        a += n
    return out, lse, bound


def check(q, k, v, lens, scale=128 ** -0.5, first=0, out=None, cu=None):
    n = q.shape[0]
    lse = torch.full((n, q.shape[1]), NAN, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = G.prompt_attention(q, k, v, offsets(lens, first) if cu is None else cu, scale, out=out, lse=lse, status=status)
    assert int(status.item()) == 0
    want, want_lse, bound = reference(q, k, v, lens, scale, first)
    rows = slice(first, first + sum(lens))
    half = torch.finfo(q.dtype).eps / 2
    err = (out.double() - want).abs()[rows]
    tol = (bound * (1 + half) + half * want.abs())[rows] + torch.finfo(q.dtype).tiny
    assert out[rows].isfinite().all()
    assert (err <= tol).all(), (err / tol).max().item()
    if sum(lens):
        size = (q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()).item() * abs(scale)
        assert ((lse.double() - want_lse).abs()[rows] <= size * 2.0 ** -16 + 2.0 ** -16 * (1 + want_lse.abs()[rows])).all()
    return out


def qkv(g, n, hq, hkv, dtype=BF16):
    x = normal(g, n, hq + 2 * hkv, 128, dtype=dtype)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n", [1, 2, 31, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_lengths(n, dtype):
    check(*qkv(gen(n), n, 2, 1, dtype), [n])


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_groups(g):
    """Every number of heads to a kv-head, ragged sequences, some of them empty."""
    lens = [3, 0, 130, 1, 77, 0, 300, 128]
    check(*qkv(gen(g), sum(lens), 2 * g, 2, BF16 if g % 2 else FP16), lens)


@pytest.mark.parametrize("n,hq,hkv", [(3000, 4, 1), (2049, 8, 8), (1500, 16, 2)])
def test_long(n, hq, hkv):
    check(*qkv(gen(n), n, hq, hkv), [n])


def test_many_sequences():
    g = gen(2)
    lens = torch.randint(0, 40, (300,), generator=torch.Generator().manual_seed(3)).tolist()
    check(*qkv(g, sum(lens), 4, 2, FP16), lens)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 1e-8, 3.0])
def test_scales(scale):
    """Sharp ones make the running maximum jump, so that O is scaled on the way."""
    g = gen(4)
    q, k, v = qkv(g, 900, 4, 2)
    check(q * 0.5, k, v, [900], scale)


def test_growing_logits():
    """The maximum grows from block to block and within rows by far more than the slack of the reference."""
    g = gen(5)
    q, k, v = (x.clone() for x in qkv(g, 1100, 2, 1, FP16))
    k *= torch.linspace(0, 6, 1100, device="cuda")[:, None, None]
    check(q, k, v, [1100], 0.3)
    check(q, k.flip(0).contiguous(), v, [1100], 0.3)


def test_strides_and_given_rows():
    """Transposed memory, single heads with any stride, rows before, between and behind the sequences left alone."""
    g = gen(6)
    q, k, v = (normal(g, h, 400, 128).transpose(0, 1) for h in (4, 2, 2))
    out = torch.full((4, 400, 128), 7.0, dtype=BF16, device="cuda").transpose(0, 1)
    check(q, k, v, [100, 200], first=50, out=out)
    assert (out[:50] == 7).all() and (out[350:] == 7).all()
    wide = torch.full((400, 6, 128), 7.0, dtype=BF16, device="cuda")
    check(q, k, v, [400], out=wide[:, 1:5])
    assert (wide[:, 0] == 7).all() and (wide[:, 5] == 7).all()
    one = normal(g, 90, 1, 136)[:, :, :128]
    check(one, normal(g, 90, 1, 128), one.clone(), [90])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("hq", [1, 4])
def test_what_is_masked_has_no_influence(dtype, hq):
    """NaN and infinities in Q, K and V of later tokens, of other sequences and behind the last one."""
    g = gen(7)
    lens, n = [150, 70, 260], 600
    clean = [x.clone() for x in qkv(g, n, hq, 1, dtype)]
    out = check(*clean, lens)
    for bad in (NAN, INF, -INF):
        for at in (20, 149, 150, 219, 300, 479, 480, 599):
            q, k, v = (x.clone() for x in clean)
            q[at], k[at], v[at] = bad, bad, bad
            got = G.prompt_attention(q, k, v, offsets(lens), 128 ** -0.5)
            ends = [150, 220, 480, 600]
            end = next(e for e in ends if at < e)
            before = min(at, 480)
            assert torch.equal(got[:before], out[:before]) and torch.equal(got[end:480], out[end:480]), (bad, at)
            if at < 480:
                assert got[at].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n", [50, 400])
def test_infinite_values(dtype, n):
    """An infinite V makes its channel infinite for the rows that see it, both signs NaN, NaN stays; the others as they
    were."""
    g = gen(8)
    q, k, v = (x.clone() for x in qkv(g, n, 2, 1, dtype))
    q *= 0.3
    out = check(q, k, v, [n])
    for i, (at, ch, x) in enumerate([(3, 5, INF), (n // 2, 5, -INF), (n // 2 + 1, 100, INF), (n - 1, 64, NAN), (n - 2, 0, -INF)]):
        v[at, 0, ch] = x
    got = G.prompt_attention(q, k, v, offsets([n]), 128 ** -0.5)
    want = out.clone()
    want[3:, :, 5] = INF
    want[n // 2:, :, 5] = NAN
    want[n // 2 + 1:, :, 100] = INF
    want[n - 1:, :, 64] = NAN
    want[n - 2:, :, 0] = -INF
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(torch.nan_to_num(got, nan=0), torch.nan_to_num(want, nan=0))


def test_rows_without_weights():
    """All logits -infinity: 0, and -infinity in lse; the type's lowest numbers are ordinary ones."""
    q, k, v = (x.clone() for x in qkv(gen(9), 200, 2, 1))
    q.abs_()
    k[:60] = -INF
    lse = torch.empty(200, 2, device="cuda")
    out = G.prompt_attention(q, k, v, offsets([200]), 0.1, lse=lse)
    assert (out[:60] == 0).all() and (lse[:60] == -INF).all()
    assert out[60:].isfinite().all() and torch.equal(out[60], v[60].expand(2, 128))
    k[:60] = torch.finfo(BF16).min
    q[:] = 0
    check(q, k, v, [200], 0.1)


def test_bad_offsets_are_reported():
    g = gen(10)
    q, k, v = qkv(g, 100, 2, 1)
    for cu in ([0, 60, 50], [-1, 50, 100], [0, 50, 101]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((100, 2, 128), 3.0, dtype=BF16, device="cuda")
        G.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 0.1, out=out, status=status)
        assert int(status.item()) == G.EINVAL and (out == 3).all()
    out = torch.full((100, 2, 128), 3.0, dtype=BF16, device="cuda")
    G.prompt_attention(q, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), 0.1, out=out)
    assert (out == 3).all()
    assert G.prompt_attention(q[:0], k[:0], v[:0], torch.zeros(2, dtype=torch.int32, device="cuda"), 0.1).shape == (0, 2, 128)


def test_refusals():
    q, k, v = qkv(gen(11), 40, 4, 2)
    cu = offsets([40])
    for bad in (dict(q=q.float()), dict(k=k[:, :1].expand(40, 3, 128)), dict(v=v[:39]), dict(q=q.requires_grad_(False)[:, :, :64]),
                dict(cu=cu.long()), dict(out=torch.empty(40, 4, 128, device="cuda")), dict(lse=torch.empty(40, 2, device="cuda")),
                dict(k=k.cpu()), dict(status=torch.zeros(1, device="cuda"))):
        a = {**dict(q=q, k=k, v=v, cu=cu, out=None, lse=None, status=None), **bad}
        with pytest.raises((ValueError, G.GaacError)):
            G.prompt_attention(a["q"], a["k"], a["v"], a["cu"], 0.1, out=a["out"], lse=a["lse"], status=a["status"])
    whole = torch.empty(40, 4, 128, dtype=BF16, device="cuda")
    for args in ((whole, k, v, whole), (q, k[:, :1].expand(40, 2, 128), v, None)):
        with pytest.raises(G.GaacError):
            G.prompt_attention(*args[:3], cu, 0.1, out=args[3])
    with pytest.raises(G.GaacError):
        G.prompt_attention(q, k, v, cu, NAN)


def test_graph_stream_and_the_same_each_time():
    g = gen(12)
    lens = [500, 3, 260]
    q, k, v = (x.clone() for x in qkv(g, sum(lens), 8, 2))
    cu = offsets(lens)
    out = check(q, k, v, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    others = [G.prompt_attention(q, k, v, cu, 128 ** -0.5, stream=x) for x in (s, s.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in others)
    two = torch.cuda.Stream()
    two.wait_stream(torch.cuda.current_stream())
    pair = [G.prompt_attention(q, k, v, cu, 128 ** -0.5, stream=x) for x in (s, two) for _ in range(3)]  # at once
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in pair)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.prompt_attention(q, k, v, cu, 128 ** -0.5)
    q.copy_(normal(g, *q.shape))
    graph.replay()
    assert torch.equal(got, check(q, k, v, lens))


def test_offsets_past_32_bits():
    """Tokens a megabyte and more apart: q, k, v and out lie over 4 GB."""
    g = gen(14)
    wide = torch.zeros((2300, 1 << 20), dtype=BF16, device="cuda")
    parts = [wide[:, i * 4096:i * 4096 + h * 128].view(2300, h, 128) for i, h in enumerate((4, 2, 2, 4))]
    q, k, v, out = parts
    for x in (q, k, v):
        x.copy_(normal(g, *x.shape))
    got = check(q, k, v, [2300], out=out)
    assert got.data_ptr() == out.data_ptr() and int(wide[:, 4 * 4096:].abs().max()) == 0


def test_prompt_to_search():
    """Norms and rotation, prompt attention, append, fork, then steps of a search: the cache's attention of the last prompt
    token is the prompt attention's last row but for the cache's 8 bits, and every table stays consistent."""
    g = gen(13)
    groups, beams, hq, hkv, V = 2, 3, 8, 2, 3000
    lens = [200, 131]
    n = sum(lens)
    q, k, v = qkv(g, n, hq, hkv)
    w = normal(g, 128) * 0.1 + 1
    turns = G.rope_turns(G.rope_frequencies(128, 1e6)[0], "cuda")
    pos = torch.cat([torch.arange(x) for x in lens]).cuda()
    G.qk_norm_rope(q, k, w, w, pos, turns)
    cu = offsets(lens)
    out = check(q, k, v, lens)
    c = Kv8Cache(64, groups * beams, hkv, 8)
    cu6 = torch.tensor([0, 200, 200, 200, n, n, n], dtype=torch.int32, device="cuda")
    c.append(k, v, cu6)
    c.fork(torch.tensor([0, 0, 3, 3], dtype=torch.int32, device="cuda"), torch.tensor([1, 2, 4, 5], dtype=torch.int32, device="cuda"))
    last = q[cu[1:].long() - 1].repeat_interleave(beams, 0).contiguous()
    got = c.attention(last, 128 ** -0.5)
    want = out[cu[1:].long() - 1].repeat_interleave(beams, 0)
    assert (got.float() - want.float()).norm() <= 0.06 * want.float().norm()  # FP8 numbers: half steps of 2^-4
    head = torch.randn(hq * 128, V, generator=g, device="cuda") * 0.2
    embed = normal(g, V, hq + 2 * hkv, 128)
    scores = torch.full((groups, beams), -INF, device="cuda")
    scores[:, 0] = 0
    b = Beams(groups, beams, V)
    o = got
    for step in range(70):
        scores, parents, tokens = b.select(o.float().flatten(1) @ head, scores)
        c.reorder(parents)
        x = embed[tokens.flatten().long()]
        q1, k1, v1 = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        G.qk_norm_rope(q1, k1, w, w, c.seq_lens, turns)
        c.append(k1, v1)
        o = c.attention(q1.contiguous(), 128 ** -0.5)
    assert int(c.status.item()) == 0
    assert scores.isfinite().all() and (scores[:, 1:] <= scores[:, :-1]).all()
    assert c.seq_lens.tolist() == [270] * 3 + [201] * 3
    held = torch.bincount(c.table[c.table >= 0].long(), minlength=64)
    assert torch.equal(held, c.refs.long())
    c.release(torch.arange(6, dtype=torch.int32, device="cuda"))
    assert int(c.refs.abs().max()) == 0
    assert not math.isnan(o.float().sum().item())


def test_results_between_the_inputs_elements():
    """out as a slice of the projection that q, k and v are slices of, heads in turn with the queries' or tokens with the keys';
    what lies beside it is left alone, and an out that takes a channel of an input is refused."""
    g, n = gen(17), 150
    x = normal(g, n, 12, 128)
    rest = x[:, :8].clone()
    check(x[:, :4], x[:, 4:6], x[:, 6:8], [100, 50], out=x[:, 8:])
    assert torch.equal(x[:, :8], rest)
    for args in ((x[:, :4], x[:, 4:6], x[:, 6:8], x[:, 2:6]), (x[:, :4], x[:, 4:6], x[:, 6:8], x[:, 7:11])):
        with pytest.raises(G.GaacError):
            G.prompt_attention(*args[:3], offsets([n]), 0.1, out=args[3])
    x = normal(g, n, 3, 4, 128)
    rest = x[:, :, :3].clone()
    check(*(x[:, :, i] for i in range(3)), [n], out=x[:, :, 3])
    assert torch.equal(x[:, :, :3], rest)
    x = normal(g, 2, n, 4, 128).transpose(0, 1)
    rest = x[:, :, :3].clone()
    check(*(x[:, :, i] for i in range(3)), [n], out=x[:, :, 3])
    assert torch.equal(x[:, :, :3], rest)
    x = normal(g, 1, 8, 128)
    check(x[:, :2], x[:, 2:3], x[:, 3:4], [1], out=x[:, 4:6])


@pytest.mark.parametrize("hq,hkv,longest", [(16, 8, 1100), (16, 4, 2400), (8, 8, 1300), (2, 1, 8400)])
def test_more_keys_than_a_cache_holds(hq, hkv, longest):
    """Up to 32 sequences, some empty, with so many keys in all that the CTAs take one kv-head after the other, where there
    are 1,672 units of 256 / (hq / hkv) tokens or more too (the first two)."""
    lens = torch.randint(longest // 2, longest + 1, (32,), generator=torch.Generator().manual_seed(hq)).tolist()
    lens[3] = lens[17] = lens[31] = 0
    lens[5], lens[30] = 1, longest
    assert sum(lens) * hkv > 1.3 * 131072
    check(*qkv(gen(16), sum(lens), hq, hkv, FP16 if hq == 8 else BF16), lens)


@pytest.mark.parametrize("batch", [33, 100])
def test_bad_offsets_of_many_sequences_are_reported(batch):
    """More sequences than a warp has lanes, a bad offset among the first 32 or behind them."""
    q, k, v = qkv(gen(15), 400, 2, 1)
    good = torch.arange(batch + 1, dtype=torch.int32) * 4
    for at in (1, 20, batch - 1, batch):
        for bad in (-1, int(good[at - 1]) - 1, 401):
            cu = good.clone()
            cu[at] = bad
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out, lse = torch.full((400, 2, 128), 3.0, dtype=BF16, device="cuda"), torch.full((400, 2), 3.0, device="cuda")
            G.prompt_attention(q, k, v, cu.cuda(), 0.1, out=out, lse=lse, status=status)
            assert int(status.item()) == G.EINVAL and (out == 3).all() and (lse == 3).all(), (at, bad)
    check(q, k, v, [4] * batch)


@pytest.mark.parametrize("n", [100, 300])
def test_infinite_values_of_rows_without_weights(n):
    """A row whose logits are all -infinity is 0, whatever V is; a row behind them that has a weight sees an infinite V."""
    q, k, v = (x.clone() for x in qkv(gen(18), n, 2, 1))
    q.abs_()
    k[:n - 20] = -INF
    v[3, 0, 5] = v[n - 40, 0, 9] = INF
    out = G.prompt_attention(q, k, v, offsets([n]), 0.1)
    assert (out[:n - 20] == 0).all()
    ordinary = torch.ones(128, dtype=torch.bool, device="cuda")
    ordinary[[5, 9]] = False
    assert out[n - 20:, :, ordinary].isfinite().all() and not out[n - 20:, :, ~ordinary].isfinite().any()
