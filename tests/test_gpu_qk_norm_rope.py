"""Norms of q and k with rotary positions in one pass, and the gradient, against 64 bits."""
import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from tests import kv8_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ref(x, w, pos, freq, eps=EPS, interleaved=False, mscale=1.0):
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    return U.rope_ref(y, pos, freq, interleaved, mscale), y


def pair_sums(y, rot, interleaved):
    """|a| + |b| of each turned channel's pair, |y| of the others: what an error of sine, cosine or norm acts on."""
    y = y.abs()
    s = y.clone()
    n = rot // 2
    ia = torch.arange(n) * 2 if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    both = y[..., ia] + y[..., ib]
    s[..., ia], s[..., ib] = both, both
    return s


def relative(dim):
    """fp32: the squares' sum is off by dim roundings at most, half of that in the root; 2^-22 for the root, 2^-21 for
    sine and cosine with their angle, three roundings of products and one of the sum: all below 2^-19 + dim 2^-25."""
    return 2.0 ** -19 + dim * 2.0 ** -25


def close(got, want, size, rel):
    """`got` is `want` but for errors of rel * size before the one rounding to got's type."""
    half = torch.finfo(got.dtype).eps / 2
    tol = size * rel * (1 + half) + half * want.abs() + torch.finfo(got.dtype).tiny
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), (err / tol).max().item()


CASES = [  # tokens, hq, hk, dim, rot, dtype, interleaved
    (1, 1, 1, 128, 128, "bf16", False), (32, 32, 8, 128, 128, "bf16", False), (777, 16, 8, 128, 64, "fp16", True),
    (5, 3, 1, 64, 64, "fp32", False), (33, 4, 2, 256, 128, "bf16", True), (9, 5, 5, 256, 256, "fp32", False),
    (7, 2, 3, 96, 32, "fp16", False), (6, 2, 1, 20, 6, "bf16", False), (3, 1, 2, 2, 2, "fp32", True),
    (11, 7, 1, 250, 250, "bf16", False), (4, 40, 8, 128, 2, "fp32", True), (2500, 8, 2, 64, 32, "bf16", False),
    (13, 2, 2, 24, 16, "fp16", False), (1, 6, 2, 34, 18, "fp16", True), (6000, 21, 5, 136, 112, "bf16", True),
    (6000, 21, 5, 136, 112, "fp16", False), (9000, 9, 1, 76, 32, "fp32", True), (40, 3, 7, 100, 92, "fp32", False)]


@pytest.mark.parametrize("n,hq,hk,dim,rot,dtype,inter", CASES)
def test_forward_and_gradient(n, hq, hk, dim, rot, dtype, inter):
    g, dt = gen(n + dim), DT[dtype]
    q, k = normal(g, n, hq, dim, dtype=dt), normal(g, n, hk, dim, dtype=dt) * 3
    wq, wk = (normal(g, dim, dtype=dt) + 1 for _ in range(2))
    pos = torch.randint(-5, 200000, (n,), generator=g, device="cuda")
    freq, _ = G.rope_frequencies(rot, 1e6)
    turns, m = G.rope_turns(freq, "cuda"), 1.25
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    G.qk_norm_rope(q, k, wq, wk, pos, turns, eps=EPS, q_out=qo, k_out=ko, interleaved=inter, mscale=m)
    for x, w, out in ((q, wq, qo), (k, wk, ko)):
        want, y = ref(x, w, pos, freq, EPS, inter, m)
        close(out, want, m * pair_sums(y, rot, inter), relative(dim))
    # in place
    q2, k2 = q.clone(), k.clone()
    G.qk_norm_rope(q2, k2, wq, wk, pos.int(), turns, eps=EPS, interleaved=inter, mscale=m)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # backward
    dq, dk = normal(g, n, hq, dim, dtype=dt), normal(g, n, hk, dim, dtype=dt)
    ws = torch.full((G.qk_norm_rope_workspace(dim),), 255, dtype=torch.uint8, device="cuda")
    dwq, dwk = (torch.full((dim,), torch.nan, device="cuda") for _ in range(2))
    G.qk_norm_rope_gradient(dq, dk, q, k, wq, wk, pos, turns, dwq, dwk, ws, eps=EPS, dq_out=qo, dk_out=ko,
                            interleaved=inter, mscale=m)
    for dz, x, w, dx, dw, heads in ((dq, q, wq, qo, dwq, hq), (dk, k, wk, ko, dwk, hk)):
        gr = U.rope_ref(dz, pos, freq, inter, m, inverse=True)
        size = m * pair_sums(dz.double(), rot, inter)
        check_gradient(gr, size, x, w, dx, dw, dim, n * heads)
        # autograd of the forward's definition gives the same
        xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
        ax, aw = torch.autograd.grad(ref(xd, wd, pos, freq, EPS, inter, m)[0], (xd, wd), dz.double())
        check_gradient(gr, size, x, w, dx, dw, dim, n * heads, ax, aw)
    # in place of the results' gradients, or of x; the same each time
    z2, d2 = dq.clone(), dwq.clone()
    G.qk_norm_rope_gradient(z2, dk, q, k, wq, wk, pos, turns, dwq, dwk, ws, eps=EPS, dk_out=k2, interleaved=inter, mscale=m)
    assert torch.equal(z2, qo) and torch.equal(k2, ko) and torch.equal(d2, dwq)
    q2.copy_(q)
    G.qk_norm_rope_gradient(dq, None, q2, None, wq, None, pos, turns, None, None, ws, eps=EPS, dq_out=q2,
                            interleaved=inter, mscale=m)
    assert torch.equal(q2, qo)


def check_gradient(gr, size, x, w, dx, dw, dim, rows, want_x=None, want_w=None):
    """gr: the result's gradient turned back, in 64 bits, off by `size` times the rotation's error.  The mean of h x r is
    a sum of dim terms; dw one of `rows` (in whatever order, off by a rounding for each)."""
    x = x.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    w = torch.ones(x.shape[-1], dtype=torch.float64, device="cuda") if w is None else w.double()
    h, hs = gr * w, size * w.abs()
    want = r * (h - x * r * (h * x * r).mean(-1, keepdim=True)) if want_x is None else want_x
    bound = r * (hs + x.abs() * r * (hs * x.abs() * r).mean(-1, keepdim=True))
    close(dx, want, bound, 2 * relative(dim) + dim * 2.0 ** -24)
    if dw is not None:
        want = (gr * x * r).flatten(0, -2).sum(0) if want_w is None else want_w
        close(dw, want, (size * x.abs() * r).flatten(0, -2).sum(0), relative(dim) + rows * 2.0 ** -24)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """Along one direction, central differences of the kernel's own fp32 results at a step of 2^-7: their roundings
    (2^-19 + 64 * 2^-25 of each result, twice, over the two steps), and the third derivative's part, 2^-14 / 6 of it:
    for heads of unit size that is below 2^-9 of the sum of the magnitudes."""
    g = gen(5)
    n, h, dim = 3, 2, 64
    x, u, dz = (normal(g, n, h, dim) for _ in range(3))
    w, uw = normal(g, dim) + 1, normal(g, dim)
    pos = torch.arange(n, device="cuda")
    turns = G.rope_turns(G.rope_frequencies(dim, 100.0)[0], "cuda")
    ws = torch.empty(G.qk_norm_rope_workspace(dim), dtype=torch.uint8, device="cuda")
    dx, dw, step = torch.empty_like(x), torch.empty_like(w), 2.0 ** -7
    G.qk_norm_rope_gradient(dz, None, x, None, w, None, pos, turns, dw, None, ws, eps=0.01, dq_out=dx, interleaved=inter)

    def at(s, t):
        y = x + s * u
        G.qk_norm_rope(y, None, w + t * uw, None, pos, turns, eps=0.01, interleaved=inter)
        return (y.double() * dz.double())

    size = at(0, 0).abs().sum()
    for d, want in (((step, 0), (dx.double() * u.double()).sum()), ((0, step), (dw.double() * uw.double()).sum())):
        got = (at(*d) - at(-d[0], -d[1])).sum() / (2 * step)
        assert abs(got - want) <= 2.0 ** -9 * size + 2.0 ** -9 * abs(want), (got, want)


def test_weights_and_strides():
    """fp32 weights, none at all, slices of one projection, batches with a stride, positions for each batch row."""
    g = gen(1)
    B, n, hq, hk, dim = 3, 21, 4, 2, 128
    freq, _ = G.rope_frequencies(dim)
    turns = G.rope_turns(freq, "cuda")
    qkv = normal(g, B, n + 2, hq + 2 * hk, dim, dtype=torch.bfloat16)[:, :n]
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    pos = torch.randint(0, 5000, (B, n), generator=g, device="cuda")
    before = qkv.clone()
    w = normal(g, dim)
    G.qk_norm_rope(q, k, w, None, pos, turns)
    for x, x0, wt in ((q, before[:, :, :hq], w), (k, before[:, :, hq:hq + hk], None)):
        want, y = ref(x0, wt, pos, freq)
        close(x, want, pair_sums(y, dim, False), relative(dim))
    assert torch.equal(qkv[:, :, hq + hk:], before[:, :, hq + hk:])
    # one position list for all batches; an odd base address takes single elements
    flat = normal(g, 5 * 2 * 64 + 1, dtype=torch.float16)
    a = flat[1:].view(5, 2, 64)
    a0, freq = a.clone(), G.rope_frequencies(64)[0]
    G.qk_norm_rope(a, None, None, None, torch.arange(5, device="cuda"), G.rope_turns(freq, "cuda"))
    want, y = ref(a0, None, torch.arange(5), freq)
    close(a, want, pair_sums(y, 64, False), relative(64))
    # transposed memory: [heads, tokens, dim]
    t = normal(g, 4, 9, 128, dtype=torch.bfloat16).transpose(0, 1)
    t0 = t.clone()
    z = normal(g, 9, 4, 128, dtype=torch.bfloat16)
    ws = torch.empty(G.qk_norm_rope_workspace(128), dtype=torch.uint8, device="cuda")
    dw = torch.empty(128, device="cuda")
    freq = G.rope_frequencies(128)[0]
    p9 = torch.arange(9, device="cuda")
    out = torch.empty_like(z)
    G.qk_norm_rope_gradient(z, None, t, None, None, None, p9, turns, dw, None, ws, dq_out=out)
    gr = U.rope_ref(z, p9, freq, inverse=True)
    check_gradient(gr, pair_sums(z.double(), 128, False), t0, None, out, dw, 128, 36)


def test_offsets_past_32_bits():
    g = gen(9)
    # two buffers: an output that lies between the elements of another tensor is refused, as one that overlaps it
    x, z = (torch.zeros((2200, 1 << 20), dtype=torch.bfloat16, device="cuda")[:, :256].view(2200, 2, 128) for _ in range(2))
    x.copy_(normal(g, 2200, 2, 128))
    z.copy_(normal(g, 2200, 2, 128))
    x0, z0, pos, freq = x.clone(), z.clone(), torch.arange(2200, device="cuda"), G.rope_frequencies(128)[0]
    turns = G.rope_turns(freq, "cuda")
    ws, dw = torch.empty(G.qk_norm_rope_workspace(128), dtype=torch.uint8, device="cuda"), torch.empty(128, device="cuda")
    G.qk_norm_rope_gradient(z, None, x, None, None, None, pos, turns, dw, None, ws)
    check_gradient(U.rope_ref(z0, pos, freq, inverse=True), pair_sums(z0.double(), 128, False), x0, None, z, dw, 128, 4400)
    G.qk_norm_rope(x, None, None, None, pos, turns)
    want, y = ref(x0, None, pos, freq, EPS)
    close(x, want, pair_sums(y, 128, False), relative(128))


def test_special_heads():
    """Zeros stay zeros; NaN and infinities stay in their head; no tokens: weight gradients of zero."""
    g = gen(2)
    x = normal(g, 4, 3, 128, dtype=torch.bfloat16)
    x[0, 1] = 0
    x[1, 2, 5] = torch.inf
    x[2, 0, 7] = torch.nan
    turns = G.rope_turns(G.rope_frequencies(128)[0], "cuda")
    p = torch.arange(4, device="cuda")
    y = torch.empty_like(x)
    G.qk_norm_rope(x, None, None, None, p, turns, q_out=y)
    assert (y[0, 1] == 0).all()
    assert y[2, 0].isnan().all() and y[1, 2].isnan().any()
    fine = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    fine[1, 2] = fine[2, 0] = False
    assert y[fine].isfinite().all()
    e = torch.empty(0, 3, 128, device="cuda")
    ws = torch.empty(G.qk_norm_rope_workspace(128), dtype=torch.uint8, device="cuda")
    dw, dk = torch.full((2, 128), torch.nan, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    G.qk_norm_rope(e, e.clone(), None, None, none, turns)
    G.qk_norm_rope_gradient(e, e.clone(), e, e.clone(), None, None, none, turns, dw, dk, ws)
    assert (dw == 0).all() and (dk == 0).all()


def test_graph_and_other_stream():
    g = gen(3)
    q, k = normal(g, 64, 8, 128, dtype=torch.bfloat16), normal(g, 64, 2, 128, dtype=torch.bfloat16)
    w = normal(g, 128, dtype=torch.bfloat16)
    turns = G.rope_turns(G.rope_frequencies(128)[0], "cuda")
    pos = torch.arange(64, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dw = torch.empty(2, 128, device="cuda")
    ws = torch.empty(G.qk_norm_rope_workspace(128), dtype=torch.uint8, device="cuda")

    def both(stream=None):
        G.qk_norm_rope(q, k, w, w, pos, turns, q_out=qo, k_out=ko, stream=stream)
        G.qk_norm_rope_gradient(qo, ko, q, k, w, w, pos, turns, dw[0], dw[1], ws, stream=stream)
        return [t.clone() for t in (qo, ko, dw)]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    G.qk_norm_rope(q, k, w, w, pos, turns, q_out=qo, k_out=ko, stream=s)
    G.qk_norm_rope_gradient(qo, ko, q, k, w, w, pos, turns, dw[0], dw[1], ws, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (qo, ko, dw)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    q.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(both(), replayed))


UNTURNED = [(128, 64, "bf16", False), (128, 64, "fp16", True), (256, 128, "fp32", False), (64, 32, "fp32", True),
            (34, 18, "fp16", True), (20, 6, "bf16", False), (76, 32, "fp32", True), (128, 2, "bf16", True)]


@pytest.mark.parametrize("dim,rot,dtype,inter", UNTURNED)
def test_infinity_in_a_channel_that_is_not_turned(dim, rot, dtype, inter):
    """Token t has one in channel rot + t: that becomes NaN (infinity over infinity), the others of its head 0."""
    g, dt = gen(dim), DT[dtype]
    n = dim - rot
    x = normal(g, n, 2, dim, dtype=dt)
    t = torch.arange(n, device="cuda")
    x[t, 1, rot + t] = torch.inf
    w = normal(g, dim, dtype=dt) + 3
    freq = G.rope_frequencies(rot, 1e4)[0]
    y = torch.empty_like(x)
    G.qk_norm_rope(x, None, w, None, t, G.rope_turns(freq, "cuda"), q_out=y, interleaved=inter)
    want, size = ref(x, w, t, freq, EPS, inter)
    close(y[:, 0], want[:, 0], pair_sums(size, rot, inter)[:, 0], relative(dim))
    assert torch.equal(y[:, 1].isnan(), want[:, 1].isnan()) and (torch.nan_to_num(y[:, 1], nan=0) == 0).all()


@pytest.mark.parametrize("dim,rot,dtype,inter", UNTURNED)
def test_gradient_with_infinities_in_channels_that_are_not_turned(dim, rot, dtype, inter):
    """One in a head's dz reaches the head's dx and its own channel of dw, one in x likewise: other heads' dx and other channels
    of dw are what they are without it (an infinite x leaves 0 of its head's part)."""
    g, dt = gen(dim + 1), DT[dtype]
    n, heads = 5, 3
    x, dz = normal(g, n, heads, dim, dtype=dt), normal(g, n, heads, dim, dtype=dt)
    w = normal(g, dim, dtype=dt) + 3
    pos, turns = torch.arange(n, device="cuda"), G.rope_turns(G.rope_frequencies(rot, 1e4)[0], "cuda")
    ws = torch.empty(G.qk_norm_rope_workspace(dim), dtype=torch.uint8, device="cuda")

    def gradient(dz, x):
        dx, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
        G.qk_norm_rope_gradient(dz, None, x, None, w, None, pos, turns, dw, None, ws, dq_out=dx, interleaved=inter)
        return dx, dw

    others = torch.ones(n, heads, dtype=torch.bool, device="cuda")
    others[2, 1] = False
    dx0, dw0 = gradient(dz, x)
    silent = dz.clone()
    silent[2, 1] = 0
    dx1, dw1 = gradient(silent, x)
    for ch in range(rot, dim):
        rest = torch.arange(dim, device="cuda") != ch
        bad = dz.clone()
        bad[2, 1, ch] = -torch.inf
        dx, dw = gradient(bad, x)
        assert torch.equal(dx[others], dx0[others]) and not dx[2, 1].isfinite().any()
        assert torch.equal(dw[rest], dw0[rest]) and dw[ch].isinf()
        bad = x.clone()
        bad[2, 1, ch] = torch.inf
        dx, dw = gradient(dz, bad)
        assert torch.equal(dx[others], dx1[others])
        assert torch.equal(dw[rest], dw1[rest]) and dw[ch].isnan()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [256, 250])
def test_weight_gradient_is_fp32_for_16_bit_inputs(dim, dtype):
    """x = 1 and eps = 0, dz is 1 in the first of each pair and 0 in the second: dw is the angles' cosines and -sines.  An angle
    is off by 2^-25 of half a turn, its functions by 2^-24: 2^-22.6 together; the root by 2^-22 (two units in the last
    place) and the two products by 2^-24 each, of the value."""
    dt, pairs = DT[dtype], dim // 2
    x, dz = torch.ones((1, 1, dim), dtype=dt, device="cuda"), torch.zeros((1, 1, dim), dtype=dt, device="cuda")
    dz[..., :pairs] = 1
    freq = G.rope_frequencies(dim, 1e4)[0]
    turns = G.rope_turns(freq, "cuda")
    ws, dx, dw = torch.empty(G.qk_norm_rope_workspace(dim), dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty(dim, device="cuda")
    for pos in torch.randint(0, 100000, (100,), generator=torch.Generator().manual_seed(dim)).tolist():
        p = torch.tensor([pos], device="cuda")
        G.qk_norm_rope_gradient(dz, None, x, None, None, None, p, turns, dw, None, ws, eps=0.0, dq_out=dx)
        want = U.rope_ref(dz, p, freq, inverse=True)[0, 0]
        err = (dw.double() - want).abs()
        assert (err <= 2.0 ** -22.6 + 1.5 * 2.0 ** -22 * want.abs()).all(), err.max().item()
