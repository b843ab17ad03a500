"""What the entry points of a generation loop refuse on the host, before any launch."""
import ctypes
import math

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from tests.test_kv8_host import BAD_CACHES, EINVAL, GOOD, ODD, OK, cache, lib  # noqa: F401

MORE = GOOD + (1 << 24)


def norm_call(lib, n=1, gradient=False, **kw):  # noqa: F811
    d = dict(x=GOOD, dz=MORE, out=GOOD, weight=None, dweight=None, n_heads=2, x_seq=0, x_tok=256, x_head=128, dz_seq=0, dz_tok=256,
             dz_head=128, out_seq=0, out_tok=256, out_head=128)
    a = dict(dtype=0, wtype=0, n_seq=1, n_tok=4, dim=128, rot=128, pos=GOOD, bits=32, ps=0, pt=1, turns=GOOD, m=1.0, eps=1e-6,
             flags=0, ws=GOOD, ws_bytes=1 << 30)
    d.update({k: v for k, v in kw.items() if k in d})
    a.update({k: v for k, v in kw.items() if k in a})
    t = (G.gaac_norm_tensor * 2)()
    for i, e in enumerate(t):
        for k, v in d.items():
            setattr(e, k, v if not isinstance(v, tuple) else v[i])
    args = [t, n, a["dtype"], a["wtype"], a["n_seq"], a["n_tok"], a["dim"], a["rot"], a["pos"], a["bits"], a["ps"], a["pt"],
            a["turns"], a["m"], a["eps"], a["flags"]]
    if gradient:
        return lib.gaac_qk_norm_rope_gradient(*args, a["ws"], a["ws_bytes"], None)
    return lib.gaac_qk_norm_rope(*args, None)


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("bad", [
    dict(n=0), dict(n=3), dict(dtype=3), dict(wtype=1), dict(wtype=-1), dict(n_tok=-1), dict(n_seq=-1), dict(dim=1),
    dict(dim=258, x_head=258, out_head=258, x_tok=516, out_tok=516), dict(rot=3), dict(rot=0), dict(rot=130), dict(bits=16),
    dict(ps=-1), dict(pt=-1), dict(pos=None), dict(turns=None), dict(turns=ODD), dict(pos=GOOD + 2), dict(m=math.nan), dict(m=math.inf),
    dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(flags=2), dict(flags=4), dict(x=None), dict(out=None), dict(x=GOOD + 1),
    dict(n_heads=0), dict(x_tok=-256), dict(out_tok=-256), dict(out_tok=0), dict(out_head=64), dict(out_tok=128), dict(out=GOOD + 16),
    dict(out_tok=512), dict(x_tok=0), dict(weight=GOOD + 1), dict(weight=GOOD + 2, wtype=2), dict(x_tok=1 << 60), dict(out=MORE, x=MORE + 64)],
    ids=str)
def test_norm_refusals(lib, gradient, bad):  # noqa: F811
    assert norm_call(lib, **{"n": 1, **bad}, gradient=gradient) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(dz=None), dict(dz=GOOD + 16), dict(dz=MORE + 1), dict(dz_tok=-1), dict(ws=None), dict(ws=GOOD + 8), dict(ws_bytes=100),
    dict(dweight=GOOD + 2), dict(out=MORE + 8)], ids=str)
def test_norm_gradient_refusals(lib, bad):  # noqa: F811
    assert norm_call(lib, gradient=True, **bad) == EINVAL


def test_norm_refuses_tensors_that_share_their_first_element(lib):  # noqa: F811
    far = [GOOD + (i << 24) for i in range(4)]
    assert norm_call(lib, n=2, x=(far[0], far[1]), out=(far[2], far[2])) == EINVAL
    assert norm_call(lib, n=2, x=(far[0], far[1]), out=(far[1], far[2])) == EINVAL
    assert norm_call(lib, n=2, gradient=True, x=(far[0], far[1]), dz=(far[2], far[3]), out=(far[3], far[1])) == EINVAL
    assert norm_call(lib, n=2, gradient=True, x=(far[0], far[1]), dz=(far[2], far[3]), out=(far[2], far[3]),
                     dweight=(GOOD, GOOD)) == EINVAL


def test_norm_nothing_to_do(lib):  # noqa: F811
    assert norm_call(lib, n_tok=0) == OK
    assert lib.gaac_qk_norm_rope_workspace(1) == 0 == lib.gaac_qk_norm_rope_workspace(300)
    assert lib.gaac_qk_norm_rope_workspace(128) >= 152 * 2 * 128 * 4


def test_select_refusals(lib):  # noqa: F811
    good = dict(logits=GOOD, dtype=0, row=1000, scores=GOOD, ended=None, end=0, batch=2, beams=4, vocab=1000, n_out=4, out=GOOD,
                parents=GOOD, tokens=GOOD, ws=GOOD, ws_bytes=1 << 30)
    for bad in (dict(logits=None), dict(logits=GOOD + 1), dict(logits=GOOD + 2, dtype=2), dict(dtype=3), dict(row=999), dict(row=1 << 41),
                dict(scores=None), dict(scores=GOOD + 2), dict(ended=GOOD, end=-1), dict(ended=GOOD, end=1000), dict(batch=-1),
                dict(beams=0), dict(beams=33), dict(vocab=0), dict(vocab=(1 << 20) + 1, row=1 << 21), dict(n_out=0), dict(n_out=65),
                dict(vocab=1, n_out=5), dict(out=None), dict(out=GOOD + 2), dict(parents=None), dict(tokens=None), dict(tokens=GOOD + 1),
                dict(ws=None), dict(ws=ODD), dict(ws_bytes=64), dict(batch=1 << 30)):
        assert lib.gaac_beam_select(*{**good, **bad}.values(), None) == EINVAL, bad
    assert lib.gaac_beam_select(*{**good, "batch": 0}.values(), None) == OK
    for sizes in ((0, 1, 1, 1), (1, 33, 1, 1), (1, 1, 0, 1), (1, 1, 1 << 21, 1), (1, 1, 9, 65)):
        assert lib.gaac_beam_workspace(*sizes) == 0
    assert lib.gaac_beam_workspace(2, 4, 9000, 5) >= 2 * 4 * 2 * (5 * 8 + 8)


def test_reorder_refusals(lib):  # noqa: F811
    f = lib.gaac_kv8_reorder
    for bad in BAD_CACHES:
        assert f(cache(**bad), GOOD, 2, None, None) == EINVAL
    for args in ((None, 2), (GOOD + 2, 2), (GOOD, 0), (GOOD, 3), (GOOD, 33)):
        assert f(cache(), *args, None, None) == EINVAL, args
    assert f(cache(), GOOD, 1, None, None) == OK  # no other parent to have


def test_python_refusals():
    z = torch.zeros
    i32, i64 = dict(dtype=torch.int32), dict(dtype=torch.int64)
    with pytest.raises(ValueError, match="device"):
        G.qk_norm_rope(z(4, 2, 128), None, None, None, z(4, **i32), z(64, **i64))
    with pytest.raises(ValueError, match="autograd"):
        G.qk_norm_rope(z(4, 2, 128), None, z(128, requires_grad=True), None, z(4, **i32), z(64, **i64))
    with pytest.raises(ValueError, match="gradient"):
        G.qk_norm_rope_gradient(z(4, 2, 128), None, z(4, 2, 128), z(4, 2, 128), None, None, z(4, **i32), z(64, **i64), None, None, z(4))
    with pytest.raises(ValueError, match="CUDA"):
        G.beam_select(z(4, 10), z(2, 2), z(2, 2), z(2, 2, **i32), z(2, 2, **i32), z(4))
    with pytest.raises(ValueError, match="autograd"):
        G.beam_select(z(4, 10, requires_grad=True), z(2, 2), z(2, 2), z(2, 2, **i32), z(2, 2, **i32), z(4))

    class Fake:
        _index, _ref, batch, n_pages, _own_status = -1, None, 4, 8, (None, 0)

    for bad in (z(2, 2), z(4, **i32), z(2, 3, **i32), z(2, 4, **i32)[:, ::2]):
        with pytest.raises(ValueError, match="parents"):
            G.kv8_reorder(Fake(), bad)


def test_struct_matches_the_header():
    assert ctypes.sizeof(G.gaac_norm_tensor) == 5 * 8 + 8 + 9 * 8


def prompt_call(lib, **kw):  # noqa: F811
    d = dict(q=GOOD, k=MORE, v=2 * MORE, out=3 * MORE, lse=None, q_tok=1024, q_head=128, k_tok=256, k_head=128, v_tok=256, v_head=128,
             out_tok=1024, out_head=128)
    a = dict(dtype=0, n=100, hq=8, hkv=2, cu=GOOD, batch=3, scale=0.1)
    d.update({k: v for k, v in kw.items() if k in d})
    a.update({k: v for k, v in kw.items() if k in a})
    p = G.gaac_prompt(*(d[n] for n, _ in G.gaac_prompt._fields_))
    return lib.gaac_prompt_attention(ctypes.byref(p), *a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(n=-1), dict(n=2 ** 31 - 100), dict(hq=0), dict(hq=7), dict(hq=18), dict(hkv=0), dict(hq=1025, hkv=1025),
    dict(cu=None), dict(cu=GOOD + 2), dict(batch=-1), dict(batch=65536), dict(scale=math.nan), dict(scale=math.inf), dict(q=None), dict(k=None),
    dict(v=None), dict(out=None), dict(q=GOOD + 8), dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(lse=GOOD + 2), dict(q_tok=127), dict(k_tok=0),
    dict(v_head=64), dict(q_tok=1028), dict(k_head=132), dict(out_tok=1 << 39), dict(out=GOOD), dict(out=MORE), dict(out_tok=512),
    dict(out_head=1024, out_tok=1024)], ids=str)
def test_prompt_refusals(lib, bad):  # noqa: F811
    assert prompt_call(lib, **bad) == EINVAL


def test_prompt_nothing_to_do(lib):  # noqa: F811
    assert lib.gaac_prompt_attention(None, 0, 4, 2, 1, GOOD, 1, 0.1, None, None) == EINVAL
    assert prompt_call(lib, n=0) == OK and prompt_call(lib, batch=0) == OK


def test_prompt_refuses_on_the_host():
    z = torch.zeros
    cu = z(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        G.prompt_attention(z(4, 2, 128).bfloat16(), z(4, 1, 128).bfloat16(), z(4, 1, 128).bfloat16(), cu, 0.1)
    with pytest.raises(ValueError, match="autograd"):
        G.prompt_attention(z(4, 2, 128, requires_grad=True), z(4, 1, 128), z(4, 1, 128), cu, 0.1)


def test_outputs_that_autograd_follows_are_refused():
    z = torch.zeros
    q, k, cu = z(4, 2, 128, dtype=torch.bfloat16), z(4, 1, 128, dtype=torch.bfloat16), z(2, dtype=torch.int32)
    for kw in (dict(out=q.clone().requires_grad_()), dict(lse=z(4, 2, requires_grad=True))):
        with pytest.raises(ValueError, match="autograd"):
            G.prompt_attention(q, k, k, cu, 0.1, **kw)
        with pytest.raises(ValueError, match="CUDA"), torch.no_grad():
            G.prompt_attention(q, k, k, cu, 0.1, **kw)
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="autograd"):
        G.beam_select(z(4, 10), z(2, 2), z(2, 2, requires_grad=True), z(2, 2, **i), z(2, 2, **i), z(4))


SIZE = 2 * 100 * 1024  # bytes of prompt_call's q and out
APART = dict(q_tok=2048, out_tok=2048)  # rows with room for another tensor's heads


@pytest.mark.parametrize("bad", [
    dict(out=GOOD + 16), dict(out=GOOD + 256), dict(out=GOOD + 2048), dict(out=GOOD + SIZE - 16), dict(q=3 * MORE + 256), dict(out=MORE + 256),
    dict(out=2 * MORE + 100 * 512 - 16), dict(**APART, out=GOOD + 2048 - 16), dict(**APART, out=GOOD + 2048 + 16),
    dict(q_tok=2048, out=GOOD + 2048), dict(q_head=256, q_tok=2048, out_head=256, out_tok=2048, out=GOOD + 512),
    dict(q_head=256, q_tok=2048, out_head=256, out_tok=2048, out=GOOD + 128), dict(n=1, out=GOOD + 256), dict(n=1, out=GOOD + 2048 - 16),
    dict(lse=GOOD), dict(lse=GOOD - 4), dict(lse=MORE + 512), dict(lse=3 * MORE + SIZE - 4), dict(lse=3 * MORE - 100 * 8 * 4 + 4)], ids=str)
def test_prompt_refuses_results_that_overlap(lib, bad):  # noqa: F811
    assert prompt_call(lib, **bad) == EINVAL


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.36e38])
def test_prompt_refuses_scales_that_overflow(lib, scale):  # noqa: F811
    """scale * log2 e has to be a number of fp32."""
    assert prompt_call(lib, scale=scale) == EINVAL
