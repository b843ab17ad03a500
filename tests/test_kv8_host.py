"""The rotary and 8-bit-cache entry points on the host: refusals before any launch, and the frequency tables."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import lossless_compressed_kv_gaac_gb300 as G
from tests import kv8_util as U

OK, EINVAL = 0, 1
GOOD, ODD = 0x10000, 0x10004  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from lossless_compressed_kv_gaac_gb300 import build

    build.build()
    return G.lib()


def cache(**kw):
    f = dict(pages=GOOD, scales=GOOD, tail=GOOD, table=GOOD, refs=GOOD, seq_lens=GOOD, work=GOOD, n_pages=8, batch=2,
             n_kv_heads=4, max_blocks=3, fmt=G.FP8_E4M3, dtype=0)
    f.update(kw)
    return ctypes.byref(G.gaac_kv8(*(f[n] for n, _ in G.gaac_kv8._fields_)))


BAD_CACHES = [dict(pages=None), dict(scales=None), dict(tail=None), dict(table=None), dict(refs=None),
              dict(seq_lens=None), dict(work=None), dict(n_pages=0), dict(batch=0), dict(batch=65536),
              dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(max_blocks=0), dict(fmt=2), dict(fmt=-1), dict(dtype=2),
              dict(pages=ODD), dict(tail=ODD), dict(refs=ODD), dict(work=ODD), dict(scales=ODD), dict(table=GOOD + 2),
              dict(seq_lens=GOOD + 1), dict(n_pages=2 ** 31 // (128 * 4))]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=lambda d: "{}={}".format(*next(iter(d.items()))))
def test_bad_caches_refused_by_every_call(lib, bad):
    c = cache(**bad)
    assert lib.gaac_kv8_append(c, GOOD, GOOD, 2, 512, 512, None, None, None) == EINVAL
    assert lib.gaac_kv8_decode_attention(c, GOOD, 8, 1024, 0.1, GOOD, 0, GOOD, 1 << 30, None, None) == EINVAL
    assert lib.gaac_kv8_reserve(c, None, None, None) == EINVAL
    assert lib.gaac_kv8_release(c, GOOD, 1, None, None) == EINVAL
    assert lib.gaac_kv8_fork(c, GOOD, GOOD, 1, None, None) == EINVAL
    assert lib.gaac_kv8_compact(c, GOOD, None) == EINVAL


def test_append_refusals(lib):
    f = lib.gaac_kv8_append
    assert f(None, GOOD, GOOD, 2, 512, 512, None, None, None) == EINVAL
    for args in ((None, GOOD, 2, 512, 512, None), (GOOD, None, 2, 512, 512, None), (ODD, GOOD, 2, 512, 512, None),
                 (GOOD, ODD, 2, 512, 512, None), (GOOD, GOOD, 3, 512, 512, None), (GOOD, GOOD, -1, 512, 512, GOOD),
                 (GOOD, GOOD, 2, 511, 512, None), (GOOD, GOOD, 2, 512, 504, None), (GOOD, GOOD, 2, 516, 512, None),
                 (GOOD, GOOD, 1 << 31, 512, 512, GOOD), (GOOD, GOOD, 2, 512, 512, GOOD + 2)):
        assert f(cache(), *args, None, None) == EINVAL, args
    assert f(cache(), None, None, 0, 0, 0, GOOD, None, None) == OK  # nothing to append


def test_attention_refusals(lib):
    f = lib.gaac_kv8_decode_attention
    need = 1 << 30
    for args in ((None, 8, 1024, 0.1, GOOD, 0, GOOD, need), (ODD, 8, 1024, 0.1, GOOD, 0, GOOD, need),
                 (GOOD, 7, 1024, 0.1, GOOD, 0, GOOD, need), (GOOD, 0, 1024, 0.1, GOOD, 0, GOOD, need),
                 (GOOD, 36, 8192, 0.1, GOOD, 0, GOOD, need), (GOOD, 8, 1016, 0.1, GOOD, 0, GOOD, need),
                 (GOOD, 8, 1028, 0.1, GOOD, 0, GOOD, need), (GOOD, 8, 1024, math.nan, GOOD, 0, GOOD, need),
                 (GOOD, 8, 1024, math.inf, GOOD, 0, GOOD, need), (GOOD, 8, 1024, 0.1, None, 0, GOOD, need),
                 (GOOD, 8, 1024, 0.1, ODD, 0, GOOD, need), (GOOD, 8, 1024, 0.1, GOOD, 1, GOOD, need),
                 (GOOD, 8, 1024, 0.1, GOOD, 0, None, need), (GOOD, 8, 1024, 0.1, GOOD, 0, ODD, need),
                 (GOOD, 8, 1024, 0.1, GOOD, 0, GOOD, 8)):
        assert f(cache(), *args, None, None) == EINVAL, args


def test_attention_refuses_more_blocks_than_it_counts(lib):
    big = cache(batch=60000, n_kv_heads=16, max_blocks=3000, n_pages=64)
    assert lib.gaac_kv8_decode_attention(big, GOOD, 16, 2048, 0.1, GOOD, 0, GOOD, 1 << 30, None, None) == EINVAL


def test_page_call_refusals(lib):
    assert lib.gaac_kv8_reserve(cache(), GOOD + 2, None, None) == EINVAL
    assert lib.gaac_kv8_release(cache(), None, 1, None, None) == EINVAL
    assert lib.gaac_kv8_release(cache(), GOOD, -1, None, None) == EINVAL
    assert lib.gaac_kv8_release(cache(), None, 0, None, None) == OK
    assert lib.gaac_kv8_fork(cache(), GOOD, None, 1, None, None) == EINVAL
    assert lib.gaac_kv8_fork(cache(), GOOD, GOOD, 3, None, None) == EINVAL  # more pairs than sequences
    assert lib.gaac_kv8_fork(cache(), None, None, 0, None, None) == OK
    assert lib.gaac_kv8_compact(cache(), None, None) == EINVAL
    assert lib.gaac_kv8_workspace(0, 8) == 0 and lib.gaac_kv8_workspace(2, 0) == 0
    assert lib.gaac_kv8_workspace(2, 8) >= 4 * (2 + 2 * 8)


def rope_call(lib, n=1, **kw):
    d = dict(x=GOOD, out=GOOD, n_heads=2, x_seq=0, x_tok=256, x_head=128, out_seq=0, out_tok=256, out_head=128)
    a = dict(dtype=0, n_seq=1, n_tok=4, dim=128, rot=128, pos=GOOD, bits=32, ps=0, pt=1, turns=GOOD, m=1.0, flags=0)
    d.update({k: v for k, v in kw.items() if k in d})
    a.update({k: v for k, v in kw.items() if k in a})
    t = (G.gaac_rope_tensor * 2)()
    for e in t:
        for k, v in d.items():
            setattr(e, k, v)
    return lib.gaac_rope(t, n, a["dtype"], a["n_seq"], a["n_tok"], a["dim"], a["rot"], a["pos"], a["bits"], a["ps"],
                         a["pt"], a["turns"], a["m"], a["flags"], None)


@pytest.mark.parametrize("bad", [
    dict(n=0), dict(n=3), dict(dtype=3), dict(n_tok=-1), dict(n_seq=-1), dict(dim=1), dict(dim=5000, rot=2),
    dict(rot=3), dict(rot=0), dict(rot=130), dict(bits=16), dict(ps=-1), dict(pt=-1), dict(pos=None), dict(turns=None),
    dict(turns=ODD), dict(pos=GOOD + 2), dict(m=math.nan), dict(m=math.inf), dict(flags=4), dict(x=None), dict(out=None),
    dict(x=GOOD + 1), dict(n_heads=0), dict(x_tok=-256), dict(out_tok=-256), dict(out_tok=0), dict(out_head=64),
    dict(out_tok=128), dict(out=GOOD + 16), dict(out_tok=512), dict(x_tok=0)], ids=str)
def test_rope_refusals(lib, bad):
    assert rope_call(lib, **{"n": 1, **bad}) == EINVAL


def test_rope_nothing_to_do(lib):
    assert rope_call(lib, n_tok=0) == OK


def test_python_refuses_host_tensors_and_shapes():
    z = torch.zeros
    with pytest.raises(ValueError):
        G.rope(z(4, 2, 128), None, z(4, dtype=torch.int32), z(64, dtype=torch.int64))
    with pytest.raises(ValueError):
        G.Kv8(z(8, 4, 2, 64, 128, dtype=torch.uint8), z(8, 4, 2), z(2, 4, 2, 64, 128, dtype=torch.bfloat16),
              z(2, 3, dtype=torch.int32), z(8, dtype=torch.int32), z(2, dtype=torch.int32), G.FP8_E4M3)
    for args in ((127,), (0,), (64, -1.0), (64, 1e4, "linear", 0.0), (64, 1e4, "cubic"), (64, 1e4, "bands", 4.0),
                 (64, 1.0, "bands", 4.0, 4096), (64, 1e4, "bands", 4.0, 4096, 1.0, 2.0), (2, 1e4, "base", 2.0)):
        with pytest.raises(ValueError):
            G.rope_frequencies(*args)
    with pytest.raises(ValueError):
        G.rope_turns(torch.tensor([math.inf]))
    with pytest.raises(ValueError):
        G.rope_turns(z(2, 2))


def test_frequencies():
    w, m = G.rope_frequencies(128, 1e6)
    assert m == 1.0 and w.dtype == torch.float64
    assert torch.allclose(w, 1e6 ** (-torch.arange(64, dtype=torch.float64) / 64), rtol=1e-14)
    lin, _ = G.rope_frequencies(128, 1e6, "linear", 4.0)
    assert torch.equal(lin, w / 4.0)
    base, _ = G.rope_frequencies(128, 1e4, "base", 8.0)
    plain, _ = G.rope_frequencies(128, 1e4)
    assert base[0] == 1.0 and abs(base[-1] * 8.0 / plain[-1] - 1) < 1e-12  # slowest pair slowed by the factor
    assert (base[1:] < plain[1:]).all()
    band, mb = G.rope_frequencies(128, 1e4, "bands", 16.0, original_len=4096)
    assert abs(mb - (0.1 * math.log(16.0) + 1)) < 1e-15
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(band[turns > 40], plain[turns > 40])  # turning often: kept (32 turns, rounded to whole pairs)
    assert torch.allclose(band[turns < 0.8], plain[turns < 0.8] / 16.0, rtol=1e-14)
    assert ((band <= plain) & (band >= plain / 16.0 * (1 - 1e-14))).all() and (band[1:] < band[:-1]).all()
    assert G.rope_frequencies(128, 1e4, "bands", 1.0, original_len=4096)[1] == 1.0


def test_turns_are_the_fraction_of_a_turn():
    w, _ = G.rope_frequencies(64, 1e4)
    t = [x % 2 ** 64 for x in G.rope_turns(w).tolist()]
    for x, f in zip(w.tolist(), t):
        # 53 bits of w / (2 pi) in double: relative error below 2^-51
        assert abs(Fraction(f, 2 ** 64) - Fraction(x / (2 * math.pi))) < Fraction(1, 2 ** 64) + Fraction(x) / 2 ** 52
    # negative frequencies turn backwards
    neg = G.rope_turns(-w).tolist()
    assert all((a + b) % 2 ** 64 == 0 for a, b in zip(neg, G.rope_turns(w).tolist()))


def test_plain_forms_agree_with_hand_values():
    """The oracle's own pins: a block whose largest number is 448, 449 and 3.5 * 2^-130, and a quarter turn."""
    x = torch.zeros(1, 64, 128, dtype=torch.float64)
    for top, e in ((448.0, 0), (449.0, 1), (1.0, -8), (1.75, -8), (1.76, -7), (2.0 ** -133, -126), (3.0e38, 120)):
        x[0, 3, 5] = top
        f8, s = U.quantise(x, 0)
        assert s.item() == 2.0 ** e, top
        assert f8.float().abs().max().item() <= 448.0
    assert U.quantise(x * 0, 1)[1].item() == 1.0
    y = U.rope_ref(torch.tensor([[[1.0, 0.0, 5.0]]]), torch.tensor([1]), torch.tensor([math.pi / 2], dtype=torch.float64))
    assert torch.allclose(y, torch.tensor([[[0.0, 1.0, 5.0]]], dtype=torch.float64), atol=1e-15)


@pytest.mark.parametrize("rot,theta,factor,original,fast,slow", [
    (128, 1e4, 4.0, 131072, 32.0, 1.0), (128, 1e4, 4.0, 262144, 32.0, 1.0), (128, 1e4, 8.0, 65536, 32.0, 1.0),
    (64, 1e4, 2.0, 1 << 20, 16.0, 2.0), (128, 1e6, 4.0, 32768, 32.0, 1.0), (128, 1e4, 16.0, 4096, 32.0, 1.0)])
def test_band_frequencies_follow_the_ramp(rot, theta, factor, original, fast, slow):
    """The share of each pair that is kept, from its definition; above all where every pair turns more than `slow` times
    within original_len, so that the ramp ends behind the last pair."""
    w, _ = G.rope_frequencies(rot, theta, "bands", factor, original_len=original, fast=fast, slow=slow)
    first = rot * math.log(original / (2 * math.pi * fast)) / (2 * math.log(theta))
    end = rot * math.log(original / (2 * math.pi * slow)) / (2 * math.log(theta))
    for j in range(rot // 2):
        plain = theta ** (-2 * j / rot)
        share = (j - math.floor(first)) / (math.ceil(end) - math.floor(first))
        kept = 1 - min(1.0, max(0.0, share))
        assert abs(w[j].item() - (plain * kept + plain / factor * (1 - kept))) <= 1e-12 * plain, j
        if plain * original / (2 * math.pi) > slow * 1.5 and j < math.ceil(end) - 1:
            assert w[j].item() > plain / factor * (1 + 1e-9)  # turns more often than slow: not the whole factor


def test_reserve_append_refuses_what_append_refuses(lib):
    f = lib.gaac_kv8_reserve_append
    for bad in BAD_CACHES:
        assert f(cache(**bad), GOOD, GOOD, 2, 512, 512, None, None, None) == EINVAL
    for args in ((None, GOOD, 2, 512, 512, None), (GOOD, None, 2, 512, 512, None), (ODD, GOOD, 2, 512, 512, None),
                 (GOOD, ODD, 2, 512, 512, None), (GOOD, GOOD, 3, 512, 512, None), (GOOD, GOOD, -1, 512, 512, GOOD),
                 (GOOD, GOOD, 2, 511, 512, None), (GOOD, GOOD, 2, 512, 504, None), (GOOD, GOOD, 2, 516, 512, None),
                 (GOOD, GOOD, 1 << 31, 512, 512, GOOD), (GOOD, GOOD, 2, 512, 512, GOOD + 2)):
        assert f(cache(), *args, None, None) == EINVAL, args
    assert f(cache(), None, None, 0, 0, 0, GOOD, None, None) == OK  # nothing to append


def test_rope_refuses_to_cut_a_graph_before_it_looks_at_devices():
    q, pos, t = torch.zeros(4, 2, 128, requires_grad=True), torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
    with pytest.raises(ValueError, match="autograd"):
        G.rope(q, None, pos, t)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        G.rope(q, None, pos, t)


def test_rope_refuses_q_and_k_that_share_their_first_element(lib):
    """The second tensor's output is the first's, or one's output is the other's input: some element would be turned
    twice, or read after it has been."""
    other, third, fourth = GOOD + (1 << 20), GOOD + (2 << 20), GOOD + (3 << 20)
    t = (G.gaac_rope_tensor * 2)()

    def call(x0, o0, x1, o1):
        for e, x, o in ((t[0], x0, o0), (t[1], x1, o1)):
            e.x, e.out, e.n_heads, e.x_seq, e.x_tok, e.x_head = x, o, 2, 0, 256, 128
            e.out_seq, e.out_tok, e.out_head = 0, 256, 128
        return lib.gaac_rope(t, 2, 0, 1, 4, 128, 128, GOOD, 32, 0, 1, GOOD, 1.0, 0, None)

    for args in ((GOOD, GOOD, GOOD, GOOD), (GOOD, other, third, other), (GOOD, other, other, third),
                 (GOOD, third, other, GOOD), (GOOD, GOOD, other, GOOD)):
        assert call(*args) == EINVAL, args


@pytest.mark.parametrize("index,status", [(0, torch.zeros(1, dtype=torch.int32)), (-1, torch.zeros(1)),
                                          (-1, torch.zeros(0, dtype=torch.int32))], ids=["host", "type", "empty"])
def test_a_status_that_the_kernels_cannot_write_is_refused(index, status):
    class Fake:  # a cache on device `index` (-1: the host's tensors pass for its own) that never reaches the library
        _index, _ref, batch, n_pages, _own_status = index, None, 2, 8, (None, 0)

    with pytest.raises(ValueError, match="status"):
        G.kv8_reserve(Fake(), None, status)
