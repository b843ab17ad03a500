"""Rotary positions on the GPU against the formula in 64 bits."""
import math

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from tests import kv8_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def tolerance(x, ref, w, interleaved, mscale):
    """Rounding of the result (half a step), and of the computation in fp32: the angle is off by 2^-33 turns and by
    its conversion (2^-24 of half a turn), sin and cos by 2 ulp, the two products and their sum by 2^-24 each:
    below 2^-20 of the pair's magnitude."""
    n = w.numel()
    mag = torch.zeros_like(ref)
    a = x.double().abs()
    ia = torch.arange(n) * 2 if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    mag[..., ia] = mag[..., ib] = (a[..., ia] + a[..., ib]) * abs(mscale)
    half = torch.finfo(x.dtype).eps / 2
    return half * ref.abs() + 2.0 ** -20 * mag + torch.finfo(x.dtype).tiny * half * 2


def check(x, out, pos, w, interleaved=False, mscale=1.0, inverse=False):
    ref = U.rope_ref(x, pos, w, interleaved, mscale, inverse)
    tol = tolerance(x, ref, w, interleaved, mscale)
    assert ((out.double() - ref).abs() <= tol).all()
    rot = 2 * w.numel()
    assert torch.equal(out[..., rot:], x[..., rot:])


def rand(shape, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [(1, 1, 1, 2, 2), (1, 8, 1, 128, 128), (3, 5, 3, 128, 64), (7, 4, 2, 64, 32),
                                                  (65, 4, 4, 256, 256), (9, 3, 1, 10, 6), (33, 2, 2, 96, 12), (257, 8, 2, 80, 80),
                                                  (2, 2, 1, 130, 2), (1000, 16, 8, 128, 128)])
def test_shapes(tokens, hq, hk, dim, rot, dtype, interleaved):
    q, k = rand((tokens, hq, dim), dtype, 1), rand((tokens, hk, dim), dtype, 2)
    pos = torch.randint(0, 1 << 20, (tokens,), dtype=torch.int32, device="cuda")
    w, _ = G.rope_frequencies(rot, 1e6)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    G.rope(q, k, pos, G.rope_turns(w, "cuda"), q_out=qo, k_out=ko, interleaved=interleaved)
    check(q, qo, pos, w, interleaved)
    check(k, ko, pos, w, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_one_tensor_and_multiplier(interleaved):
    q = rand((5, 3, 128), BF16)
    x = q.clone()
    pos = torch.tensor([0, 1, 2, 1000, 5], dtype=torch.int64, device="cuda")
    w, m = G.rope_frequencies(64, 1e4, "bands", 8.0, original_len=2048)
    G.rope(q, None, pos, G.rope_turns(w, "cuda"), interleaved=interleaved, mscale=m)
    check(x, q, pos, w, interleaved, m)


def test_batched_and_strided():
    """q and k as slices of one projection's output, in place; positions [batch, tokens] and [tokens]."""
    w, _ = G.rope_frequencies(128)
    t = G.rope_turns(w, "cuda")
    for shape in ((2, 9), (9,)):
        qkv = rand((2, 9, 12, 128), F16)
        x = qkv.clone()
        pos = torch.randint(0, 5000, shape, device="cuda")
        G.rope(qkv[:, :, :8], qkv[:, :, 8:10], pos, t)
        p = pos.expand(2, 9)
        check(x[:, :, :8], qkv[:, :, :8], p, w)
        check(x[:, :, 8:10], qkv[:, :, 8:10], p, w)
        assert torch.equal(qkv[:, :, 10:], x[:, :, 10:])
    # heads before tokens, positions with a stride, an odd offset (2-byte aligned)
    big = rand((4 * 6 * 128 + 1,), BF16)
    x = big[1:].view(4, 6, 128).transpose(0, 1)
    out = torch.empty((4, 6, 128), dtype=BF16, device="cuda").transpose(0, 1)
    pos = torch.arange(12, dtype=torch.int32, device="cuda")[::2]
    G.rope(x, None, pos, t, q_out=out)
    check(x, out, pos, w)
    # one token repeated (a broadcast input)
    x = rand((1, 2, 128), BF16).expand(6, 2, 128)
    out = torch.empty((6, 2, 128), dtype=BF16, device="cuda")
    G.rope(x, None, pos, t, q_out=out)
    check(x, out, pos, w)


def test_far_and_negative_positions():
    """The turn is exact modulo one however far the position: 64-bit positions against exact arithmetic."""
    w, _ = G.rope_frequencies(8, 1e4)
    t = G.rope_turns(w, "cuda")
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 12 + 7, -10 ** 15, 2 ** 62]
    x = torch.zeros((len(pos), 1, 8), dtype=F32, device="cuda")
    x[..., :4] = 1.0
    out = torch.empty_like(x)
    G.rope(x, None, torch.tensor(pos, device="cuda"), t, q_out=out)
    for i, p in enumerate(pos):
        for j, f in enumerate(t.tolist()):
            turn = (p * f % 2 ** 64) / 2 ** 64
            # one conversion of the fraction (2^-25 of a turn's half, 2 pi of it), 2 ulp of the function, 2^-33 turns
            assert abs(out[i, 0, j].item() - math.cos(2 * math.pi * turn)) < 2.0 ** -21
            assert abs(out[i, 0, j + 4].item() - math.sin(2 * math.pi * turn)) < 2.0 ** -21


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    """inverse is the adjoint, and the directional difference of the forward call."""
    w, m = G.rope_frequencies(64, 1e4, "bands", 4.0, original_len=4096)
    t = G.rope_turns(w, "cuda")
    x, g, d = (rand((17, 3, 128), F32, s) for s in (1, 2, 3))
    pos = torch.arange(1000, 1017, device="cuda")

    def f(v, inverse=False):
        out = torch.empty_like(v)
        G.rope(v, None, pos, t, q_out=out, interleaved=interleaved, mscale=m, inverse=inverse)
        return out

    grad = f(g, True)
    ref = U.rope_ref(g, pos, w, interleaved, m, inverse=True)
    assert ((grad.double() - ref).abs() <= tolerance(g, ref, w, interleaved, m)).all()
    # differences: f is linear, so (f(x + d) - f(x - d)) / 2 . g = grad . d up to fp32 roundings of 6528 terms,
    # each below 2^-19 of its magnitude
    diff = ((f(x + d).double() - f(x - d).double()) / 2 * g.double()).sum().item()
    terms = 4 * (m * (x.abs() + d.abs()).double() * g.abs().double()).sum().item()
    assert abs(diff - (grad.double() * d.double()).sum().item()) <= 2.0 ** -19 * terms


def test_special_values_and_empty():
    w, _ = G.rope_frequencies(128)
    t = G.rope_turns(w, "cuda")
    x = rand((2, 1, 128), BF16)
    x[0, 0, 3] = math.nan
    out = torch.empty_like(x)
    pos = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    G.rope(x, None, pos, t, q_out=out)
    bad = torch.isnan(out)
    assert bad[0, 0, 3] and bad[0, 0, 67] and bad.sum() == 2
    e = torch.empty((0, 4, 128), dtype=BF16, device="cuda")
    G.rope(e, None, torch.empty(0, dtype=torch.int32, device="cuda"), t)


def test_refusals():
    w, _ = G.rope_frequencies(128)
    t = G.rope_turns(w, "cuda")
    q, pos = rand((4, 2, 128), BF16), torch.arange(4, device="cuda")
    k = rand((4, 1, 128), BF16)
    for bad in (lambda: G.rope(q, k.float(), pos, t), lambda: G.rope(q, k[:3], pos, t), lambda: G.rope(q, k, pos.float(), t),
                lambda: G.rope(q, k, pos[:3], t), lambda: G.rope(q, k, pos, t.int()), lambda: G.rope(q, k, pos.cpu(), t),
                lambda: G.rope(q, k, pos, t, q_out=q[:, :1]), lambda: G.rope(q, None, pos, t, k_out=k),
                lambda: G.rope(q.transpose(1, 2), None, pos, t), lambda: G.rope(q.view(4, 256), None, pos, t),
                lambda: G.rope(q.double(), None, pos, t)):
        with pytest.raises(ValueError):
            bad()
    buf = rand((5, 2, 128), BF16)
    for bad in (lambda: G.rope(buf[1:], None, pos, t, q_out=buf[:4]),  # overlapping
                lambda: G.rope(q, None, pos, t, q_out=q[:1].expand(4, 2, 128)),  # repeated output
                lambda: G.rope(rand((4, 2, 64), BF16), None, pos, t)):  # more pairs than the head has
        with pytest.raises(G.GaacError) as e:
            bad()
        assert e.value.status == G.EINVAL


def test_captured_and_on_another_stream():
    w, _ = G.rope_frequencies(128)
    t = G.rope_turns(w, "cuda")
    q, k = rand((8, 4, 128), BF16), rand((8, 2, 128), BF16)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    G.rope(q, k, pos, t, q_out=qo, k_out=ko, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(q, qo, pos, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.rope(q, k, pos, t, q_out=qo, k_out=ko)
    for step in range(2):
        pos.add_(1000)
        q.copy_(rand((8, 4, 128), BF16, 10 + step))
        g.replay()
        check(q, qo, pos, w)
        check(k, ko, pos, w)


def test_more_elements_than_32_bits():
    """A tensor of 2.3e9 elements, in place; rows at its beginning, at 2^31 elements and at its end."""
    n = 70000
    x = torch.empty((n, 256, 128), dtype=BF16, device="cuda")
    rows = [0, 1, 65535, 65536, n - 1]
    for i in rows:
        x[i] = rand((256, 128), BF16, i)
    before = x[rows].clone()
    pos = torch.arange(n, device="cuda")
    w, _ = G.rope_frequencies(128)
    G.rope(x, None, pos, G.rope_turns(w, "cuda"))
    check(before, x[rows], pos[rows], w)


def test_refuses_to_cut_a_graph():
    """Tensors that autograd follows are refused while it records, since no gradient would come back; inside a Function
    and without recording the calls run, and inverse is the gradient."""
    w, m = G.rope_frequencies(64, 1e4, "bands", 4.0, original_len=4096)
    t = G.rope_turns(w, "cuda")
    x, g = rand((17, 3, 128), F32, 1), rand((17, 3, 128), F32, 2)
    pos = torch.arange(1000, 1017, device="cuda")
    leaf = x.clone().requires_grad_()
    for bad in (lambda: G.rope(leaf, None, pos, t), lambda: G.rope(leaf * 2, None, pos, t),
                lambda: G.rope(leaf, None, pos, t, q_out=torch.empty_like(x)),
                lambda: G.rope(x, leaf, pos, t, k_out=torch.empty_like(x)),
                lambda: G.rope(x, None, pos, t, q_out=leaf), lambda: G.rope(x, x.clone(), pos, t, k_out=leaf)):
        with pytest.raises(ValueError, match="autograd"):
            bad()
    assert torch.equal(leaf.detach(), x)
    with torch.no_grad():
        out = torch.empty_like(x)
        G.rope(leaf, None, pos, t, q_out=out, mscale=m)
    check(x, out, pos, w, mscale=m)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            y = torch.empty_like(v)
            G.rope(v, None, pos, t, q_out=y, mscale=m)
            return y

        @staticmethod
        def backward(ctx, gy):
            gx = torch.empty_like(gy)
            G.rope(gy.contiguous(), None, pos, t, q_out=gx, mscale=m, inverse=True)
            return gx

    y = Rope.apply(leaf)
    y.backward(g)
    assert torch.equal(y.detach(), out)
    check(g, leaf.grad, pos, w, mscale=m, inverse=True)
