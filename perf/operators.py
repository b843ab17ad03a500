"""Cases for the operators around the 8-bit paged KV cache: rotary positions, the quantising append, decode
attention, the turnover of a cache's pages (release, fork, reserve) and compaction.

Every case is one pass as a serving loop makes it.  `own` selects the framework's kernels; otherwise the pass is
written out in elementary torch operations.

The cache of one layer (block = 64 tokens, head width 128):
  pages   uint8 [n_pages, kv_heads, 2 (K, V), 64, 128]: FP8 bits; the value is the FP8 number times the scale
  scales  fp32 [n_pages, kv_heads, 2]: a power of two for each block of tokens, head and K|V
  tail    [batch, kv_heads, 2, 64, 128] in the model's type: the tokens of the block that is still open
  table   int32 [batch, max_blocks] page of each block, -1 where there is none
  refs    int32 [n_pages] sequences that hold the page
  seq_lens int32 [batch]
"""
import math

import torch

own = False

BLOCK, D = 64, 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}  # the largest finite value is 1.75 * 2^TOP


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a single chat just started: launch and merge latency
        {"name": "attention 1 x 777, 16q/8kv", "op": "attention", "batch": 1, "lo": 777, "hi": 777, "hq": 16, "hkv": 8,
         "fmt": "e4m3", "dtype": "bf16"},
        # continuous batching: 32 sequences of very different lengths
        {"name": "attention 32 x 4096-32768, 16q/8kv", "op": "attention", "batch": 32, "lo": 4096, "hi": 32768,
         "hq": 16, "hkv": 8, "fmt": "e5m2", "dtype": "fp16"},
        # one long document: the work of few rows split over a long axis
        {"name": "attention 1 x 65536, 32q/8kv", "op": "attention", "batch": 1, "lo": 65536, "hi": 65536, "hq": 32,
         "hkv": 8, "fmt": "e4m3", "dtype": "bf16"},
        # a decode step of a batch: one token each, some blocks full
        {"name": "append 32 x 1 token", "op": "append", "batch": 32, "prior": 1023, "new": 1, "hkv": 8, "fmt": "e4m3",
         "dtype": "bf16"},
        # prefill chunks of uneven lengths behind sequences with an open block
        {"name": "append 8 chunks of up to 24000", "op": "append", "batch": 8, "prior": 200, "new": 24000, "hkv": 8,
         "fmt": "e5m2", "dtype": "bf16"},
        # a decode step's queries and keys
        {"name": "rope decode 32, 32q/8kv", "op": "rope", "tokens": 32, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "inverse": False, "far": 131072},
        # prefill of a long prompt
        {"name": "rope prefill 32768, 32q/8kv", "op": "rope", "tokens": 32768, "hq": 32, "hk": 8, "dim": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "inverse": False, "far": 32768},
        # a training step's gradient: part of the head, interleaved pairs, long context
        {"name": "rope gradient 4999, 16q/8kv, half the head", "op": "rope", "tokens": 4999, "hq": 16, "hk": 8,
         "dim": 128, "rot": 64, "dtype": "fp16", "interleaved": True, "inverse": True, "far": 1000000},
        # a scheduler step of a small server: some sequences end, prompts are forked into their rows, all grow
        {"name": "turnover 32 rows, 8192 pages", "op": "turnover", "batch": 32, "max_blocks": 512, "n_pages": 8192,
         "share": 0.25, "new": 16, "hkv": 8, "dtype": "bf16"},
        # the same of a large server that admits chunks
        {"name": "turnover 256 rows, 65536 pages", "op": "turnover", "batch": 256, "max_blocks": 2048,
         "n_pages": 65536, "share": 0.25, "new": 2048, "hkv": 4, "dtype": "bf16"},
        # a small pool defragmented between requests
        {"name": "compact 257 pages", "op": "compact", "batch": 4, "n_pages": 257, "live": 0.4, "hkv": 8,
         "fmt": "e4m3"},
        # a pool of 1 GB before it is shrunk
        {"name": "compact 8192 pages", "op": "compact", "batch": 64, "n_pages": 8192, "live": 0.5, "hkv": 8,
         "fmt": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "append", "rope", "rope", "turnover", "compact"])
    fmt, dtype = rng.choice(["e4m3", "e5m2"]), rng.choice(["bf16", "fp16"])
    if op == "attention":
        batch = _log(rng, 1, 64)
        hkv = rng.choice([1, 2, 4, 8])
        top = min(65536, 65536 * 8 // (batch * hkv))
        hi = _log(rng, 1, 256) if rng.random() < 0.25 else _log(rng, 256, top)
        lo = hi if rng.random() < 0.3 else max(1, hi // rng.choice([2, 8, 64]))
        return {"op": op, "batch": batch, "lo": lo, "hi": hi, "hq": hkv * rng.choice([1, 2, 4, 5, 8]), "hkv": hkv,
                "fmt": fmt, "dtype": dtype}
    if op == "append":
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 65536 // batch))
        return {"op": op, "batch": batch, "prior": _log(rng, 1, 2000), "new": new, "hkv": rng.choice([1, 2, 3, 4, 8]),
                "fmt": fmt, "dtype": dtype}
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 16384), "hq": hk * rng.choice([1, 2, 4]), "hk": hk, "dim": dim,
                "rot": dim // rng.choice([1, 1, 2, 4]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.3, "far": _log(rng, 1000, 4000000)}
    if op == "turnover":
        batch = _log(rng, 4, 256)
        max_blocks = _log(rng, 32, 65536 // batch)
        return {"op": op, "batch": batch, "max_blocks": max_blocks,
                "n_pages": _log(rng, batch * max_blocks // 2, batch * max_blocks), "share": rng.uniform(0.1, 0.5),
                "new": _log(rng, 1, 64 * max_blocks // 8), "hkv": rng.choice([1, 2, 4]), "dtype": dtype}
    return {"op": op, "batch": _log(rng, 1, 64), "n_pages": _log(rng, 64, 6000), "live": rng.uniform(0.1, 0.9),
            "hkv": rng.choice([1, 2, 4, 8]), "fmt": fmt}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _host_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _channel_scales(g, hkv):
    """Keys: uneven channels with a few strong ones; values: milder."""
    sk = torch.exp(0.5 * torch.randn(hkv, D, generator=g, device="cuda"))
    sk[:, torch.randperm(D, generator=g, device="cuda")[:4]] *= 5.0
    sv = torch.exp(0.5 * torch.randn(hkv, D, generator=g, device="cuda"))
    return torch.stack([sk, sv], 1)  # [hkv, 2, D]


def _quantise(x, fmt):
    """FP8 numbers and power-of-two scales of blocks x [..., 64, 128] (fp32): the smallest power of two that brings
    the block's largest finite magnitude to 1.75 * 2^TOP or below; 1 for a block of zeros."""
    mag = x.abs()
    amax = torch.where(torch.isfinite(mag), mag, 0.0).amax(dim=(-2, -1))
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1)
    e = (ex - 1 - TOP[fmt] + (mant > 0.875).to(ex.dtype)).clamp(min=-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 1.0)
    return (x / scale[..., None, None]).to(FP8[fmt]), scale


def _pages(g, n_pages, hkv, fmt):
    pages = torch.empty((n_pages, hkv, 2, BLOCK, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_pages, hkv, 2), dtype=torch.float32, device="cuda")
    chan = _channel_scales(g, hkv)
    for i in range(0, n_pages, 512):
        n = min(512, n_pages - i)
        x = torch.randn((n, hkv, 2, BLOCK, D), generator=g, device="cuda") * chan[None, :, :, None, :]
        f8, s = _quantise(x, fmt)
        pages[i:i + n], scales[i:i + n] = f8.view(torch.uint8), s
    return pages, scales, chan


def _table(g, batch, max_blocks, blocks, n_pages):
    """Pages of a shuffled pool given to the first blocks[b] blocks of each sequence."""
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(max_blocks, device="cuda")[None, :] < blocks.cuda()[:, None]
    n = int(blocks.sum())
    table[held] = perm[:n]
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[perm[:n].long()] = 1
    return table, refs


def _handle(st, fmt, dtype):
    """The cache object of a program that uses the framework, around the state's buffers."""
    from lossless_compressed_kv_gaac_gb300 import FP8_E4M3, FP8_E5M2
    from lossless_compressed_kv_gaac_gb300.cache import Kv8Cache

    return Kv8Cache.over(st["pages"], st["scales"], st["tail"], st["table"], st["refs"], st["seq_lens"],
                         fmt=FP8_E4M3 if fmt == "e4m3" else FP8_E5M2)


def _inv_freq(rot):
    return 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2.0 / rot)


def prepare(case, seed):
    g, hg = _gen(seed), _host_gen(seed)
    op = case["op"]
    dt = DTYPES[case.get("dtype", "bf16")]
    st = {"case": case}
    if op == "rope":
        n = case["tokens"]
        st["q"] = torch.randn((n, case["hq"], case["dim"]), generator=g, device="cuda").to(dt)
        st["k"] = torch.randn((n, case["hk"], case["dim"]), generator=g, device="cuda").to(dt)
        # a prompt's consecutive positions, or a batch's scattered ones
        if n > 256:
            first = int(torch.randint(0, max(1, case["far"] - n) + 1, (1,), generator=hg))
            pos = torch.arange(first, first + n, device="cuda")
        else:
            pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
        st["pos"] = pos.to(torch.int32)
        st["inv_freq"] = _inv_freq(case["rot"])
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if own:
            from lossless_compressed_kv_gaac_gb300 import rope_turns

            st["turns"] = rope_turns(st["inv_freq"])
        return st
    batch, hkv = case["batch"], case["hkv"]
    if op == "attention":
        lens = torch.randint(case["lo"], case["hi"] + 1, (batch,), generator=hg)
        full = lens // BLOCK
        max_blocks = max(1, (case["hi"] + BLOCK - 1) // BLOCK)
        n_pages = int(full.sum()) + 3
        st["pages"], st["scales"], chan = _pages(g, n_pages, hkv, case["fmt"])
        st["table"], st["refs"] = _table(g, batch, max_blocks, full, n_pages)
        st["tail"] = (torch.randn((batch, hkv, 2, BLOCK, D), generator=g, device="cuda") * chan[None, :, :, None]).to(dt)
        st["seq_lens"] = lens.to(torch.int32).cuda()
        st["q"] = torch.randn((batch, case["hq"], D), generator=g, device="cuda").to(dt)
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
    elif op == "append":
        prior = torch.randint(0, case["prior"] + 1, (batch,), generator=hg)
        new = torch.full((batch,), 1) if case["new"] == 1 else torch.randint(0, case["new"] + 1, (batch,), generator=hg)
        if case["new"] == 1:  # one in eight sequences fills its block with this token
            fills = prior | (BLOCK - 1)
            prior = torch.where((torch.arange(batch) % 8 == 0) & (fills <= case["prior"]), fills, prior)
        else:
            new[int(torch.randint(0, batch, (1,), generator=hg))] = case["new"]
        blocks = (prior + new) // BLOCK  # what append fills has its pages already
        max_blocks = (case["prior"] + case["new"]) // BLOCK + 2
        n_pages = batch * ((case["prior"] + case["new"]) // BLOCK) + 3
        st["pages"], st["scales"], chan = _pages(g, n_pages, hkv, case["fmt"])
        st["table"], st["refs"] = _table(g, batch, max_blocks, blocks, n_pages)
        st["tail0"] = (torch.randn((batch, hkv, 2, BLOCK, D), generator=g, device="cuda") * chan[None, :, :, None]).to(dt)
        st["lens0"] = prior.to(torch.int32).cuda()
        st["tail"], st["seq_lens"] = st["tail0"].clone(), st["lens0"].clone()
        total = int(new.sum())
        kv = torch.randn((total, hkv, 2, D), generator=g, device="cuda") * chan[None]
        st["k"], st["v"] = kv[:, :, 0].to(dt).contiguous(), kv[:, :, 1].to(dt).contiguous()
        cu = torch.zeros(batch + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(new, 0)
        st["cu"] = cu.cuda()
    elif op == "turnover":
        max_blocks, n_pages = case["max_blocks"], case["n_pages"]
        top = max(1, min(n_pages // (2 * batch), max_blocks - (case["new"] + BLOCK - 1) // BLOCK - 1))
        lens = torch.randint(0, top * BLOCK + 1, (batch,), generator=hg)
        st["pages"] = torch.empty((n_pages, hkv, 2, BLOCK, D), dtype=torch.uint8, device="cuda")  # contents play no part
        st["scales"] = torch.ones((n_pages, hkv, 2), dtype=torch.float32, device="cuda")
        st["table"], st["refs"] = _table(g, batch, max_blocks, lens // BLOCK, n_pages)
        st["tail"] = torch.randn((batch, hkv, 2, BLOCK, D), generator=g, device="cuda").to(dt)
        st["seq_lens"] = lens.to(torch.int32).cuda()
        perm = torch.randperm(batch, generator=hg)
        n = max(1, int(case["share"] * batch))
        st["done"] = perm[:n].to(torch.int32).cuda()
        parents = perm[n:][torch.randint(0, batch - n, (n,), generator=hg)]
        st["src"], st["dst"] = parents.to(torch.int32).cuda(), st["done"].clone()
        new = torch.randint(0, case["new"] + 1, (batch,), generator=hg)
        cu = torch.zeros(batch + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(new, 0)
        st["cu"] = cu.cuda()
    else:  # compact
        n_pages = case["n_pages"]
        n_live = max(1, int(case["live"] * n_pages))
        share = n_live // batch
        blocks = torch.full((batch,), share)
        blocks[0] += n_live - share * batch
        max_blocks = int(blocks.max()) + 1
        st["pages"], st["scales"], chan = _pages(g, n_pages, hkv, case["fmt"])
        st["table0"], st["refs0"] = _table(g, batch, max_blocks, blocks, n_pages)
        if batch > 1 and share > 1:  # the second sequence shares the first one's opening blocks
            old = st["table0"][1, :share // 2].long()
            st["refs0"][old] = 0
            st["table0"][1, :share // 2] = st["table0"][0, :share // 2]
            st["refs0"][st["table0"][0, :share // 2].long()] = 2
        st["table"], st["refs"] = st["table0"].clone(), st["refs0"].clone()
        st["tail"] = torch.zeros((batch, hkv, 2, BLOCK, D), dtype=dt, device="cuda")
        st["seq_lens"] = (blocks * BLOCK).to(torch.int32).cuda()
    if own:
        st["cache"] = _handle(st, case.get("fmt", "e4m3"), case.get("dtype", "bf16"))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_rope(st):
    from lossless_compressed_kv_gaac_gb300 import rope

    rope(st["q"], st["k"], st["pos"], st["turns"], q_out=st["q_out"], k_out=st["k_out"],
         interleaved=st["case"]["interleaved"], inverse=st["case"]["inverse"])
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_attention(st):
    return st["cache"].attention(st["q"], st["scale"], out=st["out"])


def _own_append(st):
    # back to the lengths (and, for chunks, the open blocks) before the pass, then the append
    st["seq_lens"].copy_(st["lens0"])
    if st["case"]["new"] == 1:
        st["cache"].append(st["k"], st["v"], reserve=False)
    else:
        st["tail"].copy_(st["tail0"])
        st["cache"].append(st["k"], st["v"], st["cu"], reserve=False)
    return {"pages": st["pages"].view(FP8[st["case"]["fmt"]]), "scales": st["scales"], "tail": st["tail"],
            "seq_lens": st["seq_lens"]}


def _own_turnover(st):
    c = st["cache"]
    c.release(st["done"])
    c.fork(st["src"], st["dst"])
    c.reserve(st["cu"])
    return {"table": st["table"], "refs": st["refs"], "seq_lens": st["seq_lens"], "tail": st["tail"]}


def _own_compact(st):
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    moved_to = st["cache"].compact()
    return {"moved_to": moved_to, "table": st["table"], "refs": st["refs"],
            "pages": st["pages"].view(FP8[st["case"]["fmt"]]), "scales": st["scales"]}


def _plain_rope(st):
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    ang = st["pos"].double()[:, None] * st["inv_freq"][None]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if case["inverse"]:
        sin = -sin
    return {"q": _rotate(st["q"], cos, sin, rot, half, case["interleaved"]),
            "k": _rotate(st["k"], cos, sin, rot, half, case["interleaved"])}


def _rotate(x, cos, sin, rot, half, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_attention(st):
    case = st["case"]
    B, hkv, hq = case["batch"], case["hkv"], case["hq"]
    blocks = st["table"].shape[1]
    at = st["table"].clamp(min=0).long()
    f8 = st["pages"][at.flatten()].view(FP8[case["fmt"]])
    kv = f8.float() * st["scales"][at.flatten()][..., None, None]  # [B * blocks, hkv, 2, 64, 128]
    kv = kv.view(B, blocks, hkv, 2, BLOCK, D)
    # the open block comes from the tail
    full = st["seq_lens"].long() // BLOCK
    is_open = (torch.arange(blocks, device=full.device)[None] == full[:, None])[:, :, None, None, None, None]
    kv = torch.where(is_open, st["tail"].float()[:, None], kv)
    valid = torch.arange(blocks * BLOCK, device=full.device)[None] < st["seq_lens"][:, None]  # [B, T]
    kv = torch.where(valid.view(B, blocks, 1, 1, BLOCK, 1), kv, 0.0)
    k = kv[:, :, :, 0].permute(0, 2, 1, 3, 4).reshape(B, hkv, blocks * BLOCK, D)
    v = kv[:, :, :, 1].permute(0, 2, 1, 3, 4).reshape(B, hkv, blocks * BLOCK, D)
    q = st["q"].float().view(B, hkv, hq // hkv, D) * st["scale"]
    s = torch.where(valid[:, None, None], torch.matmul(q, k.transpose(-1, -2)), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-37)
    return o.reshape(B, hq, D).to(st["q"].dtype)


def _plain_append(st):
    case = st["case"]
    B, hkv, fmt = case["batch"], case["hkv"], case["fmt"]
    st["seq_lens"].copy_(st["lens0"])
    st["tail"].copy_(st["tail0"])
    dev = st["k"].device
    old = st["seq_lens"].long()
    cu = st["cu"].long()
    now = old + cu[1:] - cu[:-1]
    # a buffer of whole blocks from each sequence's open block on: its old tokens, then the new ones
    first = old // BLOCK
    n_blk = torch.where(now > old, (now + BLOCK - 1) // BLOCK - first, 0)
    at = torch.cumsum(n_blk, 0) - n_blk  # first block of each sequence in the buffer
    total_blk = int(st["k"].shape[0]) // BLOCK + 2 * B
    buf = torch.zeros((total_blk, hkv, 2, BLOCK, D), dtype=torch.float32, device=dev)
    # blocks without new tokens go to a spare one at the end, which nothing reads
    buf = torch.cat([buf, buf[:1]])
    buf[torch.where(now > old, at, total_blk)] = st["tail"].float()
    tok = torch.arange(st["k"].shape[0], device=dev)
    of = torch.searchsorted(cu, tok, right=True) - 1
    pos = old[of] + tok - cu[of]
    kv = torch.stack([st["k"], st["v"]], 2).float()  # [tokens, hkv, 2, D]
    buf[at[of] + pos // BLOCK - first[of], :, :, pos % BLOCK] = kv
    # full blocks are quantised into their pages
    b_of = torch.searchsorted(at + n_blk, torch.arange(total_blk, device=dev), right=True).clamp(max=B - 1)
    blk = first[b_of] + torch.arange(total_blk, device=dev) - at[b_of]
    sealed = (torch.arange(total_blk, device=dev) < n_blk.sum()) & (blk < now[b_of] // BLOCK)
    src = sealed.nonzero().flatten()
    dst = st["table"][b_of[src], blk[src]].long()
    f8, scale = _quantise(buf[src], fmt)
    st["pages"][dst] = f8.view(torch.uint8)
    st["scales"][dst] = scale
    # the open block: rows below the new length, those behind it as they were
    last = at + now // BLOCK - first
    rows = buf[last.clamp(max=total_blk)].to(st["tail"].dtype)
    fresh = torch.arange(BLOCK, device=dev)[None] < (now % BLOCK)[:, None]
    fresh &= (now > old)[:, None]
    st["tail"].copy_(torch.where(fresh[:, None, None, :, None], rows, st["tail"]))
    st["seq_lens"].copy_(now.to(torch.int32))
    return {"pages": st["pages"].view(FP8[fmt]), "scales": st["scales"], "tail": st["tail"],
            "seq_lens": st["seq_lens"]}


def _count(refs, ids, by):
    """refs[id] += by for every id >= 0."""
    ids = ids.flatten().long()
    refs.scatter_add_(0, ids.clamp(min=0), torch.where(ids >= 0, by, 0).to(refs.dtype))


def _plain_turnover(st):
    table, refs, lens, tail = st["table"], st["refs"], st["seq_lens"], st["tail"]
    max_blocks = table.shape[1]
    done, src, dst = st["done"].long(), st["src"].long(), st["dst"].long()
    # sequences that ended give their pages back
    _count(refs, table[done], -1)
    table[done] = -1
    lens[done] = 0
    # prompts forked: full blocks shared, the open block copied
    n = lens[src].long()
    col = torch.arange(max_blocks, device=table.device)
    rows = torch.where(col[None] < (n // BLOCK)[:, None], table[src], -1)
    table[dst] = rows
    _count(refs, rows, 1)
    lens[dst] = n.to(torch.int32)
    keep = torch.arange(BLOCK, device=table.device)[None] < (n % BLOCK)[:, None]
    tail[dst] = torch.where(keep[:, None, None, :, None], tail[src], tail[dst])
    # pages for the blocks that the next tokens fill: the lowest free ones, in order of sequence and block
    n = lens.long()
    grown = n + (st["cu"][1:] - st["cu"][:-1]).long()
    need = (col[None] >= (n // BLOCK)[:, None]) & (col[None] < (grown // BLOCK)[:, None]) & (table < 0)
    rank = torch.cumsum(need.flatten().long(), 0) - 1
    order = torch.argsort((refs > 0).to(torch.int32), stable=True)
    have = (refs == 0).sum()
    give = need.flatten() & (rank < have)
    page = order[rank.clamp(min=0, max=refs.numel() - 1)]
    refs.scatter_add_(0, page, give.to(refs.dtype))
    table.copy_(torch.where(give, page.to(torch.int32), table.flatten()).view_as(table))
    return {"table": table, "refs": refs, "seq_lens": lens, "tail": tail}


def _plain_compact(st):
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    table, refs = st["table"], st["refs"]
    n = refs.numel()
    page = torch.arange(n, device=refs.device)
    live = refs > 0
    n_live = live.sum()
    holes = (~live & (page < n_live)).nonzero().flatten()  # lowest first
    movers = (live & (page >= n_live)).nonzero().flatten().flip(0)  # highest first
    moved_to = torch.where(live, page, -1).to(torch.int32)
    moved_to[movers] = holes.to(torch.int32)
    st["pages"][holes] = st["pages"][movers]
    st["scales"][holes] = st["scales"][movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, moved_to[table.clamp(min=0).long()], table))
    return {"moved_to": moved_to, "table": table, "refs": refs,
            "pages": st["pages"].view(FP8[st["case"]["fmt"]]), "scales": st["scales"]}


_OWN = {"rope": _own_rope, "attention": _own_attention, "append": _own_append, "turnover": _own_turnover,
        "compact": _own_compact}
_PLAIN = {"rope": _plain_rope, "attention": _plain_attention, "append": _plain_append, "turnover": _plain_turnover,
          "compact": _plain_compact}


# ------------------------------------------------------------------ what a pass cannot do without

def _mean_len(case):
    return (case["lo"] + case["hi"]) / 2


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", "bf16")]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        return {"bytes": 2 * n * size + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * (case["hq"] + case["hk"]) * case["rot"]}
    B, hkv = case["batch"], case["hkv"]
    if op == "attention":
        # mean lengths; the open block's half is small beside the pages and counted at their width
        t = B * _mean_len(case)
        return {"bytes": t * hkv * 2 * D + t / BLOCK * (4 + 8 * hkv) + 2 * B * case["hq"] * D * size,
                "flops": 4 * t * case["hq"] * D}
    if op == "append":
        t = B * (1 if case["new"] == 1 else case["new"] / 2) + (case["new"] / 2 if case["new"] > 1 else 0)
        # read once in the model's type; written in 8 bits where a block fills, in the model's type where it stays open
        sealed = t if case["new"] > BLOCK else 0
        return {"bytes": t * hkv * 2 * D * size + (sealed + (t - sealed) * size) * hkv * 2 * D,
                "flops": 4 * t * hkv * 2 * D}
    if op == "turnover":
        n = max(1, int(case["share"] * B))
        rows = B * case["max_blocks"] * 4
        # the ended and forked rows, the counts of the pool once, the open blocks copied
        return {"bytes": 4 * n * case["max_blocks"] * 4 + case["n_pages"] * 4 + n * hkv * 2 * 32 * D * size * 2
                + min(rows, B * (case["new"] // (2 * BLOCK)) * 8), "flops": 0}
    n_pages, live = case["n_pages"], case["live"]
    moved = n_pages * live * (1 - live)
    return {"bytes": 2 * moved * hkv * 2 * (BLOCK * D + 4) + 12 * n_pages, "flops": 0}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time."""
    op = case["op"]
    if op in ("turnover", "compact"):
        return None  # whole numbers and copies
    st = prepare(case, seed)
    if op == "rope":
        out = {}
        sign = -1.0 if case["inverse"] else 1.0
        for name in ("q", "k"):
            x = st[name].double()
            y = x.clone()
            for j in range(case["rot"] // 2):
                a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + case["rot"] // 2)
                ang = st["pos"].double() * 1e6 ** (-2.0 * j / case["rot"])
                c, s = torch.cos(ang)[:, None], sign * torch.sin(ang)[:, None]
                y[..., a] = c * x[..., a] - s * x[..., b]
                y[..., b] = s * x[..., a] + c * x[..., b]
            out[name] = y
        return out
    fp8 = FP8[case["fmt"]]
    if op == "attention":
        B, hq, hkv = case["batch"], case["hq"], case["hkv"]
        out = torch.zeros((B, hq, D), dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(st["seq_lens"][b])
            for h in range(hkv):
                ids = st["table"][b, :n // BLOCK].long()
                kv = st["pages"][ids, h].view(fp8).double() * st["scales"][ids, h].double()[..., None, None]
                tail = st["tail"][b, h, :, :n % BLOCK].double()
                k = torch.cat([kv[:, 0].reshape(-1, D), tail[0]])
                v = torch.cat([kv[:, 1].reshape(-1, D), tail[1]])
                if n:
                    rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                    s = (st["q"][b, rows].double() @ k.T) * st["scale"]
                    out[b, rows] = torch.softmax(s, -1) @ v
        return out
    # append: block by block; a page's number is the token's value over the block's scale, before its rounding
    if case["batch"] * case["new"] > 400000:
        return None
    pages, scales, tail = st["pages"].view(fp8).double(), st["scales"].double(), st["tail0"].double()
    lens, cu = st["lens0"].tolist(), st["cu"].tolist()
    after = []
    for b in range(case["batch"]):
        old, n = lens[b], cu[b + 1] - cu[b]
        after.append(old + n)
        if n == 0:
            continue
        r = old % BLOCK
        for kind, name in ((0, "k"), (1, "v")):
            x = torch.cat([st["tail0"][b, :, kind, :r].double().transpose(0, 1), st[name][cu[b]:cu[b + 1]].double()])
            full = (r + n) // BLOCK
            if full:
                ids = st["table"][b, old // BLOCK:old // BLOCK + full].long()
                y = x[:full * BLOCK].view(full, BLOCK, -1, D).transpose(1, 2)  # [blocks, hkv, 64, D]
                top = y.abs().amax(dim=(-2, -1)) / 1.75
                # the smallest power of two with largest magnitude / scale <= 1.75 * 2^TOP
                sc = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300))) - TOP[case["fmt"]])
                sc = torch.where(top > 0, sc, 1.0)
                pages[ids, :, kind] = y / sc[..., None, None]
                scales[ids, :, kind] = sc
            rest = x[full * BLOCK:]
            tail[b, :, kind, :rest.shape[0]] = rest.transpose(0, 1)
    return {"pages": pages, "scales": scales, "tail": tail, "seq_lens": None}
