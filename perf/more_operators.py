"""Cases for the operators of a generation loop around the 8-bit paged KV cache: norms and rotary positions of queries
and keys in one pass, the gradient of that, attention over whole prompts, a beam search's selection, and the reordering
of a cache's sequences that follows it.

Every case is one pass as a serving or training loop makes it.  `own` selects the framework's kernels; otherwise the
pass is written out in elementary torch operations.

Beams: sequence g * beams + i of a cache is beam i of search g.
"""
import math

import torch

own = False

BLOCK, D = 64, 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's queries and keys: launch latency
        {"name": "norm+rope decode 32 32q/8kv", "op": "norm", "tokens": 32, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "far": 131072},
        # prefill of a long prompt
        {"name": "norm+rope prefill 32768 32q/8kv", "op": "norm", "tokens": 32768, "hq": 32, "hk": 8, "dim": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "far": 32768},
        # a training step's gradient: an odd number of tokens, half of the head turned, interleaved pairs
        {"name": "norm+rope gradient 4999 16q/8kv half", "op": "norm_grad", "tokens": 4999, "hq": 16, "hk": 8,
         "dim": 128, "rot": 64, "dtype": "fp16", "interleaved": True, "far": 1000000},
        # the same of a larger batch
        {"name": "norm+rope gradient 16384 32q/8kv", "op": "norm_grad", "tokens": 16384, "hq": 32, "hk": 8,
         "dim": 128, "rot": 128, "dtype": "bf16", "interleaved": False, "far": 32768},
        # one short chat: few tiles, latency
        {"name": "prompt 1 x 777 16q/8kv", "op": "prompt", "batch": 1, "lo": 777, "hi": 777, "hq": 16, "hkv": 8,
         "dtype": "bf16"},
        # a batch of short and middling prompts admitted together
        {"name": "prompt 32 x 1-2048 16q/8kv", "op": "prompt", "batch": 32, "lo": 1, "hi": 2048, "hq": 16, "hkv": 8,
         "dtype": "fp16"},
        # few longer ones of very different lengths, an odd number of heads to a kv-head
        {"name": "prompt 8 x 300-5000 20q/4kv", "op": "prompt", "batch": 8, "lo": 300, "hi": 5000, "hq": 20,
         "hkv": 4, "dtype": "bf16"},
        # one long document
        {"name": "prompt 1 x 16384 32q/8kv", "op": "prompt", "batch": 1, "lo": 16384, "hi": 16384, "hq": 32,
         "hkv": 8, "dtype": "bf16"},
        # one search of four beams over a small vocabulary: latency
        {"name": "select 1 x 4 32000", "op": "select", "batch": 1, "beams": 4, "n_out": 4, "vocab": 32000,
         "dtype": "fp32", "ended": 0.0},
        # a batch of searches over a large, odd one, some beams ended, twice the beams wanted
        {"name": "select 32 x 8 128511", "op": "select", "batch": 32, "beams": 8, "n_out": 16, "vocab": 128511,
         "dtype": "bf16", "ended": 0.1},
        # four searches of four beams behind a short prompt
        {"name": "reorder 4 x 4 up to 1000 tokens", "op": "reorder", "batch": 4, "beams": 4, "tokens": 1000,
         "max_blocks": 64, "hkv": 8, "dtype": "bf16"},
        # a batch of searches behind long ones
        {"name": "reorder 32 x 8 up to 30000 tokens", "op": "reorder", "batch": 32, "beams": 8, "tokens": 30000,
         "max_blocks": 512, "hkv": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "prompt", "prompt", "prompt", "select", "select", "reorder"])
    if op in ("norm", "norm_grad"):
        dim = rng.choice([64, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 16384), "hq": hk * rng.choice([1, 2, 4]), "hk": hk, "dim": dim,
                "rot": dim // rng.choice([1, 1, 2, 4]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "interleaved": rng.random() < 0.5, "far": _log(rng, 1000, 4000000)}
    if op == "prompt":
        hkv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(12000, 16384 / math.sqrt(batch)))
        lo = hi if rng.random() < 0.3 else max(1, hi // rng.choice([2, 8, 64]))
        return {"op": op, "batch": batch, "lo": lo, "hi": hi, "hq": hkv * rng.choice([1, 2, 3, 4]), "hkv": hkv,
                "dtype": rng.choice(["bf16", "fp16"])}
    if op == "select":
        batch, beams = _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 5, 8])
        return {"op": op, "batch": batch, "beams": beams, "n_out": beams * rng.choice([1, 2]),
                "vocab": _log(rng, 100, 128000), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "ended": rng.choice([0.0, 0.2])}
    batch, beams = _log(rng, 1, 32), rng.choice([2, 3, 4, 5, 8])
    max_blocks = _log(rng, 4, 512)
    return {"op": op, "batch": batch, "beams": beams, "tokens": _log(rng, 1, max_blocks * BLOCK - 1),
            "max_blocks": max_blocks, "hkv": rng.choice([1, 2, 4, 8]), "dtype": rng.choice(["bf16", "fp16"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _host_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g, hg = _gen(seed), _host_gen(seed)
    st = {"case": case}
    return {"norm": _prepare_norm, "norm_grad": _prepare_norm, "prompt": _prepare_prompt, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](st, case, g, hg)


def _prepare_norm(st, case, g, hg):
    n, dim, dt = case["tokens"], case["dim"], DTYPES[case["dtype"]]
    # heads of uneven magnitude with a few strong channels, as projections give them
    for name, heads in (("q", case["hq"]), ("k", case["hk"])):
        size = torch.exp(0.5 * torch.randn((heads, dim), generator=g, device="cuda"))
        st[name] = (torch.randn((n, heads, dim), generator=g, device="cuda") * size).to(dt)
        st[name + "_weight"] = (1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dt)
        st[name + "_out"] = torch.empty_like(st[name])
        if case["op"] == "norm_grad":
            st["d" + name] = torch.randn((n, heads, dim), generator=g, device="cuda").to(dt)
            st["d" + name + "_weight"] = torch.empty(dim, dtype=torch.float32, device="cuda")
    # a prompt's consecutive positions, or a batch's scattered ones
    if n > 256:
        first = int(torch.randint(0, max(1, case["far"] - n) + 1, (1,), generator=hg))
        pos = torch.arange(first, first + n, device="cuda")
    else:
        pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
    st["pos"] = pos.to(torch.int32)
    st["inv_freq"] = 1e6 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") * 2.0 / case["rot"])
    if own:
        from lossless_compressed_kv_gaac_gb300 import qk_norm_rope_workspace, rope_turns

        st["turns"] = rope_turns(st["inv_freq"])
        st["workspace"] = torch.empty(qk_norm_rope_workspace(dim), dtype=torch.uint8, device="cuda")
    return st


def _prepare_prompt(st, case, g, hg):
    batch, hq, hkv = case["batch"], case["hq"], case["hkv"]
    # one of the longest, the others at random but for their sum, which is the same for every seed
    lens = torch.randint(case["lo"], case["hi"] + 1, (batch,), generator=hg)
    lens[0] = case["hi"]
    rest = case["hi"] + (batch - 1) * (case["lo"] + case["hi"]) // 2 - int(lens.sum())
    for i in range(1, batch):
        change = max(case["lo"] - int(lens[i]), min(case["hi"] - int(lens[i]), rest))
        lens[i] += change
        rest -= change
    lens = lens[torch.randperm(batch, generator=hg)]
    cu = torch.zeros(batch + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(lens, 0)
    st["cu"], st["longest"] = cu.cuda(), int(lens.max())
    # q, k and v are slices of one projection's output
    qkv = torch.randn((int(cu[-1]), hq + 2 * hkv, D), generator=g, device="cuda")
    qkv[:, hq:hq + hkv] *= torch.exp(0.5 * torch.randn((hkv, D), generator=g, device="cuda"))
    qkv = qkv.to(DTYPES[case["dtype"]])
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    st["out"] = torch.empty((qkv.shape[0], hq, D), dtype=qkv.dtype, device="cuda")
    st["scale"] = 1.0 / math.sqrt(D)
    return st


def _prepare_select(st, case, g, hg):
    batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
    st["logits"] = (3.0 * torch.randn((batch * beams, vocab), generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    st["scores"] = -10.0 * torch.rand((batch, beams), generator=g, device="cuda")
    st["ended"] = torch.rand((batch, beams), generator=g, device="cuda") < case["ended"]
    st["end_token"] = int(torch.randint(0, vocab, (1,), generator=hg))
    if own:
        from lossless_compressed_kv_gaac_gb300.cache import Beams

        st["beams"] = Beams(batch, beams, vocab, n_out=case["n_out"], end_token=st["end_token"])
    return st


def _prepare_reorder(st, case, g, hg):
    batch, beams, hkv, max_blocks = case["batch"], case["beams"], case["hkv"], case["max_blocks"]
    n = batch * beams
    # the beams of a search are as long as one another, share their prompt's pages and have a few of their own
    length = torch.randint(case["tokens"] // 2, case["tokens"] + 1, (batch,), generator=hg)
    full = length // BLOCK
    apart = torch.minimum(full, torch.randint(0, 5, (batch,), generator=hg))
    per = full + (beams - 1) * apart  # pages of a search
    first = torch.cumsum(per, 0) - per
    n_pages = batch * (case["tokens"] // BLOCK + 4 * (beams - 1)) + 3
    perm = torch.randperm(n_pages, generator=hg)
    col, beam = torch.arange(max_blocks)[None, None], torch.arange(beams)[None, :, None]
    shared = (full - apart)[:, None, None]
    at = first[:, None, None] + torch.where(col < shared, col, shared + beam * apart[:, None, None] + col - shared)
    held = (col < full[:, None, None]).expand(batch, beams, max_blocks)
    table = torch.where(held, perm[at.clamp(max=n_pages - 1)], -1).view(n, max_blocks)
    refs = torch.bincount(table[table >= 0], minlength=n_pages)
    st["table"], st["refs"] = table.to(torch.int32).cuda(), refs.to(torch.int32).cuda()
    st["seq_lens"] = length[:, None].expand(batch, beams).reshape(-1).to(torch.int32).cuda()
    st["pages"] = torch.empty((n_pages, hkv, 2, BLOCK, D), dtype=torch.uint8, device="cuda")  # contents play no part
    st["scales"] = torch.ones((n_pages, hkv, 2), dtype=torch.float32, device="cuda")
    st["tail"] = torch.randn((n, hkv, 2, BLOCK, D), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    # good beams are continued several times, some not at all
    st["parents"] = torch.randint(0, beams, (batch, beams), generator=hg, dtype=torch.int32).cuda()
    if own:
        from lossless_compressed_kv_gaac_gb300.cache import Kv8Cache

        st["cache"] = Kv8Cache.over(st["pages"], st["scales"], st["tail"], st["table"], st["refs"], st["seq_lens"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_norm(st):
    from lossless_compressed_kv_gaac_gb300 import qk_norm_rope

    qk_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"], st["pos"], st["turns"], eps=EPS, q_out=st["q_out"],
                 k_out=st["k_out"], interleaved=st["case"]["interleaved"])
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_norm_grad(st):
    from lossless_compressed_kv_gaac_gb300 import qk_norm_rope_gradient

    qk_norm_rope_gradient(st["dq"], st["dk"], st["q"], st["k"], st["q_weight"], st["k_weight"], st["pos"], st["turns"],
                          st["dq_weight"], st["dk_weight"], st["workspace"], eps=EPS, dq_out=st["q_out"],
                          dk_out=st["k_out"], interleaved=st["case"]["interleaved"])
    return {"q": st["q_out"], "k": st["k_out"], "q_weight": st["dq_weight"], "k_weight": st["dk_weight"]}


def _own_prompt(st):
    from lossless_compressed_kv_gaac_gb300 import prompt_attention

    return prompt_attention(st["q"], st["k"], st["v"], st["cu"], st["scale"], out=st["out"])


def _own_select(st):
    scores, parents, tokens = st["beams"].select(st["logits"], st["scores"], ended=st["ended"])
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _own_reorder(st):
    st["cache"].reorder(st["parents"])
    return {"table": st["table"], "refs": st["refs"], "seq_lens": st["seq_lens"], "tail": st["tail"]}


def _turn(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] with its first rot channels turned; cos, sin [tokens, 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _angles(st):
    ang = st["pos"].double()[:, None] * st["inv_freq"][None]
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]


def _plain_norm(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(y, cos, sin, case["rot"], case["interleaved"]).to(x.dtype)

    return {"q": one(st["q"], st["q_weight"]), "k": one(st["k"], st["k_weight"])}


def _plain_norm_grad(st):
    case = st["case"]
    cos, sin = _angles(st)

    def one(dy, x, w):
        y = x.float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        n = y * r
        g = _turn(dy.float(), cos, -sin, case["rot"], case["interleaved"])
        dw = (g * n).flatten(0, 1).sum(0, dtype=torch.float64).float()
        h = g * w.float()
        return (r * (h - n * (h * n).mean(-1, keepdim=True))).to(x.dtype), dw

    dq, dq_weight = one(st["dq"], st["q"], st["q_weight"])
    dk, dk_weight = one(st["dk"], st["k"], st["k_weight"])
    return {"q": dq, "k": dk, "q_weight": dq_weight, "k_weight": dk_weight}


def _plain_prompt(st):
    case = st["case"]
    hq, hkv, top = case["hq"], case["hkv"], st["longest"]
    cu, dt = st["cu"].long(), st["q"].dtype
    # padded to the longest prompt: row i of sequence b is token cu[b] + i
    i = torch.arange(top, device=cu.device)
    real = i[None] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(real, cu[:-1, None] + i[None], 0)
    q = st["q"].float()[at].view(-1, top, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)  # [B, hkv, g, T, D]
    k = st["k"].float()[at].transpose(1, 2)[:, :, None]
    v = torch.where(real[..., None, None], st["v"].float()[at], 0.0).transpose(1, 2)[:, :, None]
    s = torch.matmul(q * st["scale"], k.transpose(-1, -2))
    s.masked_fill_(i[None] > i[:, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(-1, top, hq, D)[real].to(dt)


def _plain_select(st):
    case = st["case"]
    batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
    x = st["logits"].double().view(batch, beams, vocab)
    top = x.amax(-1, keepdim=True)
    c = st["scores"].double()[..., None] + (x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
    # an ended beam goes on as it is, with the end token alone
    kept = torch.arange(vocab, device=x.device) == st["end_token"]
    c = torch.where(st["ended"][..., None], torch.where(kept, st["scores"].double()[..., None], -math.inf), c)
    best, at = torch.sort(c.view(batch, -1), dim=-1, descending=True, stable=True)
    best, at = best[:, :case["n_out"]], at[:, :case["n_out"]]
    return {"scores": best.float(), "parents": (at // vocab).to(torch.int32), "tokens": (at % vocab).to(torch.int32)}


def _plain_reorder(st):
    table, refs, lens, tail = st["table"], st["refs"], st["seq_lens"], st["tail"]
    batch, beams = st["parents"].shape
    of = torch.arange(batch, device=table.device)[:, None] * beams + st["parents"].long()
    of = of.flatten()
    n = lens[of].long()
    col = torch.arange(table.shape[1], device=table.device)
    rows = torch.where(col[None] < (n // BLOCK)[:, None], table[of], -1)
    for ids, by in ((table, -1), (rows, 1)):
        ids = ids.flatten().long()
        refs.scatter_add_(0, ids.clamp(min=0), torch.where(ids >= 0, by, 0).to(refs.dtype))
    # the open block's rows; those behind them as they were
    keep = (torch.arange(BLOCK, device=table.device)[None] < (n % BLOCK)[:, None])[:, None, None, :, None]
    tail.copy_(torch.where(keep, tail[of], tail))
    table.copy_(rows)
    lens.copy_(n)
    return {"table": table, "refs": refs, "seq_lens": lens, "tail": tail}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "prompt": _own_prompt, "select": _own_select,
        "reorder": _own_reorder}
_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "prompt": _plain_prompt, "select": _plain_select,
          "reorder": _plain_reorder}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op in ("norm", "norm_grad"):
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        turned = case["tokens"] * (case["hq"] + case["hk"]) * case["rot"]
        if op == "norm":
            return {"bytes": 2 * n * size + 4 * case["tokens"], "flops": 4 * n + 3 * turned}
        return {"bytes": 3 * n * size + 4 * case["tokens"] + 8 * case["dim"], "flops": 10 * n + 3 * turned}
    if op == "prompt":
        B, lo, hi = case["batch"], case["lo"], case["hi"]
        # the mean of t and of t (t + 1) / 2 over the lengths
        mean, square = (lo + hi) / 2, ((hi - lo + 1) ** 2 - 1) / 12 + ((lo + hi) / 2) ** 2
        tokens = hi + (B - 1) * mean
        pairs = (hi * (hi + 1) + (B - 1) * (square + mean)) / 2
        return {"bytes": tokens * 2 * (case["hq"] + case["hkv"]) * D * size + 4 * B,
                "flops": 4 * pairs * case["hq"] * D}
    rows = case["batch"] * case["beams"]
    if op == "select":
        return {"bytes": rows * (case["vocab"] * size * (1 - case["ended"]) + 5) + case["batch"] * case["n_out"] * 12,
                "flops": 4 * rows * case["vocab"]}
    # open blocks are half full, a beam in `beams` stays as it is; the last few of a row's pages differ
    moved = rows * (1 - 1 / case["beams"])
    tokens = 0.75 * case["tokens"]
    return {"bytes": 2 * moved * (min(tokens, 32) * case["hkv"] * 2 * D * size + tokens / BLOCK * 4 + 4), "flops": 0}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions in 64 bits."""
    op = case["op"]
    if op == "reorder":
        return None  # whole numbers and copies
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm, "prompt": _exact_prompt, "select": _exact_select}[op](st, case)


def _exact_norm(st, case):
    """Pair by pair; the gradient by differentiating that."""
    out = {}
    for name in ("q", "k"):
        grad = case["op"] == "norm_grad"
        x = st[name].double().requires_grad_(grad)
        w = st[name + "_weight"].double().requires_grad_(grad)
        n = w * x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS)
        half = case["rot"] // 2
        j = torch.arange(half, device=x.device)
        ia, ib = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
        z = torch.polar(torch.ones_like(st["inv_freq"]).expand(case["tokens"], half).contiguous(),
                        torch.outer(st["pos"].double(), 1e6 ** (-2.0 * j.double() / case["rot"])))
        turned = torch.complex(n[..., ia], n[..., ib]) * z[:, None]
        y = n.clone()
        y[..., ia] = turned.real
        y[..., ib] = turned.imag
        if grad:
            out[name], out[name + "_weight"] = torch.autograd.grad(y, (x, w), st["d" + name].double())
        else:
            out[name] = y
    return out


def _exact_prompt(st, case):
    """One sequence and kv-head at a time, some hundreds of queries of each."""
    hq, hkv = case["hq"], case["hkv"]
    per = hq // hkv
    out = torch.zeros((st["q"].shape[0], hq, D), dtype=torch.float64, device="cuda")
    cu = st["cu"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(hkv):
            k, v = st["k"][a:b, h].double(), st["v"][a:b, h].double()
            for i in range(a, b, 1024):
                e = min(b, i + 1024)
                q = st["q"][i:e, h * per:(h + 1) * per].double().transpose(0, 1)
                s = (q @ k[:e - a].T) * st["scale"]
                s = s + torch.triu(torch.full((e - i, e - a), -math.inf, dtype=torch.float64, device="cuda"), i - a + 1)
                out[i:e, h * per:(h + 1) * per] = (torch.softmax(s, -1) @ v[:e - a]).transpose(0, 1)
    return out


def _exact_select(st, case):
    """The largest candidates' values, search by search."""
    values = []
    for b in range(case["batch"]):
        rows = torch.log_softmax(st["logits"][b * case["beams"]:(b + 1) * case["beams"]].double(), -1)
        rows = rows + st["scores"][b].double()[:, None]
        rows = torch.cat([st["scores"][b, i:i + 1].double() if st["ended"][b, i] else rows[i]
                          for i in range(case["beams"])])
        values.append(torch.cat([rows, torch.full((case["n_out"],), -math.inf, dtype=torch.float64, device="cuda")])
                      .topk(case["n_out"]).values)
    return {"scores": torch.stack(values), "parents": None, "tokens": None}
