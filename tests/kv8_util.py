"""Plain 64-bit forms of the operators around the 8-bit paged cache, shared by its tests.

They run on any device and use no code of the library."""
from __future__ import annotations

import math

import torch

BLOCK, D = 64, 128
FP8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
TOP = {0: 8, 1: 15}


def rope_ref(x, pos, w, interleaved=False, mscale=1.0, inverse=False):
    """x [..., tokens, heads, dim], pos [..., tokens], w float64 [pairs]: the rotated x in 64 bits."""
    n = w.numel()
    ang = pos.double().cpu()[..., None] * w.double().cpu()
    c, s = (mscale * torch.cos(ang)).to(x.device)[..., None, :], (mscale * torch.sin(ang)).to(x.device)[..., None, :]
    if inverse:
        s = -s
    y = x.double().clone()
    ia = torch.arange(n) * 2 if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def quantise(x, fmt):
    """FP8 bits and scales of blocks x [..., 64, 128]."""
    x = x.double()
    mag = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    top = mag.amax(dim=(-2, -1))
    scale = torch.ones_like(top)
    flat, out = top.flatten().tolist(), []
    for a in flat:
        if a == 0.0:
            out.append(1.0)
            continue
        e = math.frexp(a)[1] - 1 - TOP[fmt] - 1
        while a > 1.75 * 2.0 ** (TOP[fmt] + e):
            e += 1
        out.append(2.0 ** max(e, -126))
    scale = torch.tensor(out, dtype=torch.float64, device=x.device).view(top.shape)
    y = (x / scale[..., None, None]).float()  # exact: at most 11 significant bits
    f8 = y.to(FP8[fmt])
    if fmt == 1:
        f8 = torch.where(torch.isinf(x), x.float().to(FP8[1]).float(), f8.float()).to(FP8[1])
    return f8, scale.float()


def f8_equal(a, b):
    """The same FP8 numbers (NaN of any bits being one number)."""
    a, b = a.float(), b.float()
    return torch.equal(torch.nan_to_num(a, nan=1e30), torch.nan_to_num(b, nan=1e30)) and \
        torch.equal(torch.signbit(a) & ~a.isnan(), torch.signbit(b) & ~b.isnan())


def tokens_of(cache, b):
    """K and V [2, len, heads, 128] in 64 bits of sequence b, read from its pages and open block."""
    n = int(cache.seq_lens[b])
    ids = cache.table[b, :n // BLOCK].long()
    x = cache.pages[ids].view(FP8[cache.fmt]).double() * cache.scales[ids].double()[..., None, None]
    x = x.permute(2, 0, 3, 1, 4).reshape(2, -1, cache.n_kv_heads, D)
    tail = cache.tail[b, :, :, :n % BLOCK].double().permute(1, 2, 0, 3)
    return torch.cat([x, tail], 1)


def attention_ref(cache, q, scale, weights=2.0 ** -11):
    """(out, bound) in 64 bits: the attention of q [batch, q_heads, 128], and for every element the error that a
    computation in 32 bits with weights off by `weights` may have before its result is rounded.

    Logits: 128 products in fp32 are off by at most 128 * 2^-24 of the sum of their magnitudes, a further 2^-20 of
    that covers scaling them and splitting off their maxima, and 2^-19 the exponentials and the sums.  An error d of a logit changes each weight by a factor of about 1 + d, in numerator and denominator."""
    B, hq, _ = q.shape
    g = hq // cache.n_kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b in range(B):
        k, v = tokens_of(cache, b)
        if k.shape[0] == 0:
            continue
        for h in range(cache.n_kv_heads):
            rows = slice(h * g, (h + 1) * g)
            qb = q[b, rows].double()
            s = qb @ k[:, h].T * scale
            p = torch.softmax(s, -1)
            out[b, rows] = p @ v[:, h]
            d = (qb.abs() @ k[:, h].abs().T).amax(-1, keepdim=True) * abs(scale) * (2.0 ** -17 + 2.0 ** -20)
            bound[b, rows] = (p @ v[:, h].abs()) * (weights + 2.0 ** -19 + 2.05 * d)
    return out, bound


def check_attention(cache, q, scale, out):
    """Weights: one f16 (2^-11, a whole step to be generous) for a bf16 result; in two parts for others, each rounded
    to 11 bits of what is left (2^-22, below 2^-20), or to bf16's 8 (2^-18, below 2^-16) over a bf16 open block."""
    weights = 2.0 ** -11 if out.dtype == torch.bfloat16 else 2.0 ** -16 if cache.dtype == torch.bfloat16 else 2.0 ** -20
    ref, bound = attention_ref(cache, q, scale, weights)
    half = torch.finfo(out.dtype).eps / 2
    tol = bound * (1 + half) + half * ref.abs() + torch.finfo(out.dtype).tiny
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"error {worst:.3f} of the bound"
    return worst


class Model:
    """The page tables as plain Python: what reserve, release, fork, append (lengths) and compact have to leave."""

    def __init__(self, n_pages, batch, max_blocks):
        self.n_pages, self.batch, self.max_blocks = n_pages, batch, max_blocks
        self.table = [[-1] * max_blocks for _ in range(batch)]
        self.refs = [0] * n_pages
        self.lens = [0] * batch

    def reserve(self, new):
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        ok = True
        for b in range(self.batch):
            n = self.lens[b] + new[b]
            if n > self.max_blocks * BLOCK:
                ok = False
                continue
            for i in range(self.lens[b] // BLOCK, n // BLOCK):
                if self.table[b][i] < 0:
                    if free:
                        self.table[b][i] = free.pop(0)
                        self.refs[self.table[b][i]] = 1
                    else:
                        ok = False
        return ok

    def append(self, new):
        for b in range(self.batch):
            n = self.lens[b] + new[b]
            if n <= self.max_blocks * BLOCK and all(self.table[b][i] >= 0 for i in range(self.lens[b] // BLOCK, n // BLOCK)):
                self.lens[b] = n

    def release(self, seqs):
        for b in seqs:
            if 0 <= b < self.batch:
                for i in range(self.max_blocks):
                    if self.table[b][i] >= 0:
                        self.refs[self.table[b][i]] -= 1
                    self.table[b][i] = -1
                self.lens[b] = 0

    def fork(self, src, dst):
        before = (list(self.lens), [list(r) for r in self.table])
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < self.batch and 0 <= d < self.batch) or s in dst or d in dst[:i]:
                continue
            if before[0][d] or any(p >= 0 for p in before[1][d]):
                continue
            self.lens[d] = self.lens[s]
            for j in range(self.lens[s] // BLOCK):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in range(self.n_pages - 1, n - 1, -1) if self.refs[p] > 0]
        to = [p if self.refs[p] > 0 else -1 for p in range(self.n_pages)]
        for m, h in zip(movers, holes):
            to[m] = h
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.table = [[to[p] if p >= 0 else -1 for p in r] for r in self.table]
        return to

    def check(self, cache):
        assert cache.seq_lens.tolist() == self.lens
        assert cache.refs.tolist() == self.refs
        assert cache.table.tolist() == self.table
