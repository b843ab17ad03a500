"""A beam search's selection over beams and vocabulary, and the reordering of a cache's sequences."""
import random

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from lossless_compressed_kv_gaac_gb300.cache import Beams, Kv8Cache
from tests import kv8_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def candidates(logits, scores, ended, end_token):
    """All candidates [batch, beams, vocab] in 64 bits; NaN counts as -infinity."""
    batch, beams = scores.shape
    x = logits.double().view(batch, beams, -1)
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1)
    dead = ~(scores.isfinite() & total.isfinite() & top[..., 0].isfinite())
    # Equal rows have equal sums, but torch adds up rows of other alignments in other orders: the logarithm to 2^-40.
    log = torch.round(torch.log(total) * 2.0 ** 40) * 2.0 ** -40
    c = scores.double()[..., None] + ((x - top) - log[..., None])  # a large maximum takes nothing from the sum
    if ended is not None:
        only = torch.full_like(c, -INF)
        only[..., end_token] = scores.double()
        c = torch.where(ended[..., None], only, c)
        dead = torch.where(ended, ~scores.isfinite(), dead)
    return torch.where(dead[..., None], -INF, c)


def check(logits, scores, n_out, ended=None, end_token=0, got=None):
    """The selection is the reference's.  A sum of exponentials is off by 2^-22 for each of them, 2^-23 times the
    mean distance from the maximum (below 16) and the roundings of 45 additions in a row: 2^-17 covers them.  Candidates
    closer than that may change places only between beams."""
    batch, beams = scores.shape
    vocab = logits.shape[1]
    if got is None:
        got = Beams(batch, beams, vocab, n_out, end_token).select(logits, scores, ended)
    out, parents, tokens = got
    c = candidates(logits, scores, ended, end_token).view(batch, -1)
    best, at = torch.sort(c, dim=-1, descending=True, stable=True)
    best, at = best[:, :n_out], at[:, :n_out]
    tol = 2.0 ** -17 + best.abs() * 2.0 ** -24
    assert torch.equal(best.isinf(), out.isinf())
    fine = best.isfinite()
    assert ((out.double() - best).abs() <= tol)[fine].all()
    assert (out[~fine] == -INF).all()
    flat = parents.long() * vocab + tokens
    assert (parents >= 0).all() and (parents < beams).all() and (tokens >= 0).all() and (tokens < vocab).all()
    for b in range(batch):
        assert len(set(flat[b].tolist())) == n_out
        mine = c[b, flat[b]]
        same = flat[b] == at[b]
        assert ((mine - best[b]).abs() <= tol[b])[~same].all() and same[~fine[b]].all()
        other = (flat[b] // vocab) != (at[b] // vocab)
        assert (same | other).all()
    return flat, at


@pytest.mark.parametrize("batch,beams,vocab,n_out,dtype", [
    (1, 1, 1, 1, "fp32"), (1, 1, 100, 64, "bf16"), (2, 4, 32000, 4, "fp32"), (3, 5, 50001, 10, "bf16"),
    (1, 8, 128511, 16, "fp16"), (2, 32, 777, 64, "bf16"), (5, 3, 8192, 6, "bf16"), (1, 2, 8185, 33, "fp16"),
    (2, 2, 8193, 32, "fp32"), (1, 1, 1 << 20, 64, "bf16"), (1, 32, 1 << 20, 64, "fp32"), (7, 1, 16385, 2, "fp16"),
    (1, 4, 2, 8, "fp32"), (70, 2, 4099, 4, "bf16")])
def test_select(batch, beams, vocab, n_out, dtype):
    g = gen(vocab + beams)
    logits = (4 * torch.randn((batch * beams, vocab), generator=g, device="cuda")).to(DT[dtype])
    scores = -10 * torch.rand((batch, beams), generator=g, device="cuda")
    check(logits, scores, n_out)
    ended = torch.rand((batch, beams), generator=g, device="cuda") < 0.4
    check(logits, scores, n_out, ended, vocab // 2)


@pytest.mark.parametrize("dtype", DT)
def test_select_ties(dtype):
    """Equal logits, equal beams, few distinct values, sorted vocabularies: ties go to the lowest place."""
    torch.manual_seed(4)
    dt = DT[dtype]
    scores = torch.zeros(2, 4, device="cuda")
    V = 20001
    for x in (torch.zeros(8, V), torch.randint(0, 2, (8, V)).float() - 0.0, -torch.zeros(8, V) * torch.randint(0, 2, (8, V)),
              torch.arange(V).float().expand(8, V) / 1000, -torch.arange(V).float().expand(8, V) / 1000,
              torch.randn(1, V).expand(8, V), torch.tensor([0.0, -0.0]).repeat(8, V)[:, :V]):
        x = x.to(dt).cuda().contiguous()
        for n_out in (1, 7, 40):
            flat, at = check(x, scores, n_out)
            assert torch.equal(flat, at)  # beams are alike bit for bit, so the sums are too


def test_select_masked_and_not_finite():
    g = gen(6)
    V = 9000
    x = torch.randn((12, V), generator=g, device="cuda")
    x[0] = -INF  # no token left
    x[1, 10:] = -INF  # ten left, in the first chunk
    x[2, :V - 3] = -INF
    x[3, 77] = torch.nan
    x[4, 8500] = INF
    x[5] = torch.finfo(torch.float32).min  # all alike, the type's lowest
    x[6, ::2] = torch.finfo(torch.float32).min
    scores = -torch.rand((3, 4), generator=g, device="cuda")
    scores[1, 2:] = -INF
    scores[2, 1:] = -INF  # a search's first step
    check(x, scores, 16)
    ended = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    ended[0, 1] = ended[2, 0] = ended[2, 2] = True
    for end in (0, 5, V - 1):
        flat, at = check(x, scores, 24, ended, end)
        assert torch.equal(flat[2], at[2])
    # nothing but -infinity: the lowest places
    scores[:] = -INF
    flat, at = check(x, scores, 10)
    assert torch.equal(flat, torch.arange(10, device="cuda").expand(3, 10))
    check(x, scores, 10, ended, 3)
    # fewer tokens than are wanted
    flat, at = check(x[:, :2].contiguous(), torch.zeros(3, 4, device="cuda"), 8)


@pytest.mark.parametrize("dtype", DT)
def test_select_runs(dtype):
    """Rows long enough for several runs of a CTA, with many beams: what comes late is far above or below what came early,
    masked starts, sorted rows, rows of few values."""
    g = gen(11)
    dt, V, rows = DT[dtype], 70001, 256
    x = torch.randn((rows, V), generator=g, device="cuda")
    x[0, :40000] = -INF
    x[1, 20000:] = -INF
    x[2, :33000] -= 900
    x[3, 33000:] -= 900
    x[4] = torch.arange(V, device="cuda") / 1000
    x[5] = -torch.arange(V, device="cuda") / 1000
    x[6] = torch.randint(0, 3, (V,), generator=g, device="cuda").float()
    x[7] = 5
    x[8, 8192:] = 7
    x[9, :] = -INF
    x[9, 69999] = -700
    x[10, 50000] = 300
    x[11] = (torch.arange(V, device="cuda") // 300) / 8
    scores = -torch.rand((rows // 8, 8), generator=g, device="cuda")
    for n_out in (8, 16, 64):
        check(x.to(dt), scores, n_out)
    each = torch.zeros((rows, 1), device="cuda")  # every row alone
    flat, at = check(x.to(dt), each, 33)
    assert torch.equal(flat, at)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_select_strided_rows(dtype, offset):
    """Rows of a wider tensor, at every alignment; what lies beside them is not looked at."""
    g = gen(8 + offset)
    wide = torch.full((6, 8200 + 13), 1e4, device="cuda").to(DT[dtype])
    x = wide[:, offset:offset + 8191]
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    check(x, -torch.rand((2, 3), generator=g, device="cuda"), 6)


def test_select_rows_past_32_bits():
    g = gen(12)
    x = torch.zeros((3, 1 << 30), dtype=torch.float16, device="cuda")[:, :9000]
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    check(x, torch.zeros((1, 3), device="cuda"), 5)


def test_select_in_a_graph_and_on_another_stream():
    g = gen(9)
    logits = torch.randn((8, 30000), generator=g, device="cuda").bfloat16()
    scores = -torch.rand((2, 4), generator=g, device="cuda")
    b = Beams(2, 4, 30000)
    want = b.select(logits, scores)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = b.select(logits, scores, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.select(logits, scores)
    logits.copy_(torch.randn((8, 30000), generator=g, device="cuda"))
    graph.replay()
    check(logits, scores, 4, got=out)
    for _ in range(20):  # one behind the other, the same each time
        again = b.select(logits, scores)
    assert all(torch.equal(x, y) for x, y in zip(out, again))


def model_reorder(m, beams, parents):
    """U.Model: sequences become what their parents were."""
    old = (list(m.lens), [list(r) for r in m.table])
    for s, p in enumerate(parents):
        src = s // beams * beams + p
        if not 0 <= p < beams or src == s:
            continue
        for i in range(m.max_blocks):
            if old[1][s][i] >= 0:
                m.refs[old[1][s][i]] -= 1
        full = old[0][src] // U.BLOCK
        m.table[s] = old[1][src][:full] + [-1] * (m.max_blocks - full)
        for page in m.table[s][:full]:
            m.refs[page] += 1
        m.lens[s] = old[0][src]


@pytest.mark.parametrize("groups,beams,heads,max_blocks,dtype", [
    (1, 1, 2, 4, "bf16"), (1, 2, 1, 3, "bf16"), (3, 4, 2, 8, "fp16"), (2, 5, 3, 300, "bf16"), (4, 8, 8, 20, "bf16"),
    (1, 16, 1, 5, "fp16"), (2, 32, 2, 4, "bf16"), (40, 3, 1, 2, "bf16")])
def test_reorder(groups, beams, heads, max_blocks, dtype):
    """Random appends, reserves and reorders against the tables as plain lists, and the open rows."""
    rng, g = random.Random(beams), gen(beams)
    n, dt = groups * beams, DT[dtype]
    n_pages = n * min(max_blocks, 12)
    c = Kv8Cache(n_pages, n, heads, max_blocks, dtype=dt)
    m = U.Model(n_pages, n, max_blocks)
    for step in range(4):
        new = [rng.randint(0, min(3 * U.BLOCK, max_blocks * U.BLOCK - m.lens[b])) for b in range(n)]
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        k, v = (torch.randn((sum(new), heads, 128), generator=g, device="cuda").to(dt) for _ in range(2))
        if m.reserve(new):
            m.append(new)
            c.append(k, v, cu)
        if step == 2:  # pages reserved ahead
            ahead = [1 if i % 3 == 0 and m.lens[i] % U.BLOCK == U.BLOCK - 1 else 0 for i in range(n)]
            m.reserve(ahead)
            c.reserve(torch.tensor([0] + ahead).cumsum(0).to(torch.int32).cuda())
        m.check(c)
        parents = [rng.randrange(beams) for _ in range(n)]
        tail, lens = c.tail.clone(), list(m.lens)
        c.reorder(torch.tensor(parents, dtype=torch.int32, device="cuda").view(groups, beams))
        model_reorder(m, beams, parents)
        m.check(c)
        assert int(c.status.item()) == 0
        for s, p in enumerate(parents):
            src = s // beams * beams + p
            r = lens[src] % U.BLOCK
            assert torch.equal(c.tail[s, :, :, :r], tail[src, :, :, :r])
            assert torch.equal(c.tail[s, :, :, r:], tail[s, :, :, r:])  # rows behind them as they were
    m.release(range(n))
    c.release(torch.arange(n, dtype=torch.int32, device="cuda"))
    m.check(c)
    assert int(c.refs.abs().max()) == 0


def test_reorder_refuses_on_the_device():
    """Bad parents, lengths and pages leave the rest as it should be."""
    c = Kv8Cache(16, 6, 1, 4)
    k = torch.randn(6 * 100, 1, 128, device="cuda").bfloat16()
    c.append(k, k, torch.arange(0, 700, 100, dtype=torch.int32, device="cuda"))
    t0 = c.table.clone()
    c.reorder(torch.tensor([[1, -1, 0], [3, 2, 2]], dtype=torch.int32, device="cuda"))
    assert int(c.status.item()) == G.EINVAL
    assert torch.equal(c.table, t0[[1, 1, 0, 3, 5, 5]])
    assert c.refs[t0[:, 0].long()].tolist() == [1, 2, 0, 1, 0, 2]
    c.status.zero_()
    c.seq_lens[4] = -5
    t1 = c.table.clone()
    c.reorder(torch.tensor([[0, 1, 2], [1, 1, 2]], dtype=torch.int32, device="cuda"))
    assert int(c.status.item()) == G.EFORMAT and torch.equal(c.table, t1)
    c.status.zero_()
    c.seq_lens[4] = 100
    c.table[4, 0] = 99
    c.reorder(torch.tensor([[0, 1, 2], [1, 1, 2]], dtype=torch.int32, device="cuda"))
    assert int(c.status.item()) == G.EFORMAT and c.table[3, 0] == 99 and c.refs[t0[3, 0]] == 0
    assert int(c._tensors[6][:6].abs().max()) == 0  # counters are zero between calls


def test_search_loop_in_a_graph():
    """Steps of select, reorder, append and attention, captured and replayed, are those made one by one."""
    groups, beams, heads, V = 2, 4, 2, 5000
    n = groups * beams

    def start(seed):
        g = gen(seed)
        c = Kv8Cache(256, n, heads, 8)
        k = torch.randn((groups * 150, heads, 128), generator=g, device="cuda").bfloat16()
        cu = torch.zeros(n + 1, dtype=torch.int32)
        cu[1:] = torch.repeat_interleave(torch.arange(1, groups + 1) * 150, beams)
        c.append(k, -k, cu.cuda())
        first = torch.arange(groups, dtype=torch.int32).repeat_interleave(beams - 1) * beams
        rest = torch.tensor([i for i in range(n) if i % beams], dtype=torch.int32)
        c.fork(first.cuda(), rest.cuda())
        st = {"c": c, "b": Beams(groups, beams, V), "table": torch.randn((V, heads, 128), generator=g, device="cuda").bfloat16(),
              "out": torch.randn((8 * 128, V), generator=g, device="cuda") * 0.1,
              "scores": torch.full((groups, beams), -INF, device="cuda"), "tokens": torch.zeros(n, dtype=torch.int64, device="cuda")}
        st["scores"][:, 0] = 0
        st["q"] = torch.randn((n, 8, 128), generator=g, device="cuda").bfloat16()
        return st

    def step(st):
        o = st["c"].attention(st["q"], 0.09).float().flatten(1)
        scores, parents, tokens = st["b"].select(o @ st["out"], st["scores"])
        st["scores"].copy_(scores)
        st["tokens"].copy_(tokens.flatten())
        st["c"].reorder(parents)
        k = st["table"][st["tokens"]]
        st["c"].append(k, -k)

    a, b = start(1), start(1)
    for _ in range(70):
        step(a)
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for _ in range(69):
        graph.replay()
    torch.cuda.synchronize()
    assert int(a["c"].status.item()) == 0 == int(b["c"].status.item())
    for x, y in ((a["scores"], b["scores"]), (a["tokens"], b["tokens"]), (a["c"].table, b["c"].table), (a["c"].refs, b["c"].refs)):
        assert torch.equal(x, y)
    held = torch.bincount(a["c"].table[a["c"].table >= 0].long(), minlength=256)
    assert torch.equal(held, a["c"].refs.long())
    assert a["c"].seq_lens.tolist() == [220] * n


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [70000, 70001])
def test_select_peak_in_a_later_run(V, dtype):
    """The largest logit 3 to 59 above the first run's, in a later run of the same CTA, with a step on the way in half of the
    rows; nothing else has weight.  The sum is off by 2^-22 for its exponentials (twice that of the small terms, 5% of it),
    three roundings of 2^-24 and the logarithm's 2^-25, together below 2^-21, the result by 2^-24 of itself."""
    rows = 256
    x = torch.full((rows, V), -300.0, device="cuda")
    gap = torch.linspace(3, 59, rows, device="cuda")
    x[:, 5] = -2.7
    x[:, 3 * 8192 + 77] = gap - 2.7
    x[::2, 8192 + 9] = gap[::2] / 2 - 5
    x = x.to(DT[dtype])
    scores = torch.zeros((rows, 1), device="cuda")
    out, _, tokens = Beams(rows, 1, V, 2).select(x, scores)
    best, at = candidates(x, scores, None, 0).view(rows, V).topk(2)
    assert torch.equal(tokens.long(), at)
    err = (out.double() - best).abs()
    assert (err <= 2.0 ** -21 + best.abs() * 2.0 ** -24).all(), err.max().item()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [70000, 70002])
def test_select_runs_of_aligned_rows(V, dtype):
    """Several runs of a CTA with rows on 16-byte and on 4-byte boundaries, which are loaded as vectors and as pairs."""
    g = gen(V)
    rows = 256
    x = torch.randn((rows, V), generator=g, device="cuda")
    x[0, :40000] = -INF
    x[1, 20000:] = -INF
    x[2, :33000] -= 900
    x[3] = torch.arange(V, device="cuda") / 1000
    x[4] = -torch.arange(V, device="cuda") / 1000
    x[5] = torch.randint(0, 3, (V,), generator=g, device="cuda").float()
    x[6] = 5
    x[7, V - 3:] = torch.tensor([9.0, 8.0, 9.0], device="cuda")  # in the last vector
    scores = -torch.rand((rows // 8, 8), generator=g, device="cuda")
    for n_out in (8, 40):
        check(x.to(DT[dtype]), scores, n_out)
    flat, at = check(x.to(DT[dtype]), torch.zeros((rows, 1), device="cuda"), 33)
    assert torch.equal(flat, at)
