"""The serving operators around the sparse attention layer, as cases to measure.

Four operators: the norm and position rotation of queries and keys
(``rope``), appending keys and values to the paged 8-bit cache (``append``),
attention over that cache for new tokens (``cache``), and causal attention
over packed prompts (``prompt``).  ``run`` computes them in elementary torch
operations, or with ``own`` set through libssa's entry points.

Head counts and dimensions are those of the layer's workloads (32 query heads
over 8 kv-heads, 8 over 1, 8 over 8; d = 64 and 128; 64- and 128-key blocks).
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E_MIN, E_MAX = -40, 120          # exponents that a page's scale may have


def _heads(hq, hkv, d):
    return {"hq": hq, "hkv": hkv, "d": d}


def listed():
    return [
        # one new token for each of 64 sequences: latency of a launch
        {"name": "rope decode 64", "op": "rope", "tokens": 64, **_heads(32, 8, 128), "rot": 128, "layout": "half",
         "dtype": "bf16", "far": 262144, "stretch": 1.0},
        # an odd prompt in float32: a quarter of the head left as it is, neighbouring pairs
        {"name": "rope f32 5003", "op": "rope", "tokens": 5003, **_heads(8, 8, 64), "rot": 48, "layout": "pairs",
         "dtype": "f32", "far": 5003, "stretch": 1.0},
        # a 128K prompt whose frequencies are stretched for positions past the trained length
        {"name": "rope 128K stretched", "op": "rope", "tokens": 131072, **_heads(32, 8, 128), "rot": 128,
         "layout": "half", "dtype": "bf16", "far": 1048576, "stretch": 8.0},
        # a decode step of 64 sequences: one token each, pages partly filled
        {"name": "append decode 64", "op": "append", "seqs": 64, "tokens": 64, "have": 4096, **_heads(32, 8, 128),
         "page": 64, "rot": 128, "layout": "half", "dtype": "bf16"},
        # a few tokens for each of 37 sequences (drafts), 128-token pages, float32 activations
        {"name": "append drafts f32", "op": "append", "seqs": 37, "tokens": 37 * 5, "have": 1000, **_heads(8, 8, 64),
         "page": 128, "rot": 32, "layout": "pairs", "dtype": "f32"},
        # the prompts of 7 sequences of different lengths, into fresh and partly filled pages
        {"name": "append prompts 64K", "op": "append", "seqs": 7, "tokens": 65536, "have": 300, **_heads(32, 8, 128),
         "page": 64, "rot": 128, "layout": "half", "dtype": "bf16"},
        # one long sequence: few rows, a long axis to split
        {"name": "cache 1 x 128K", "op": "cache", "seqs": 1, "new": 1, "longest": 131072, **_heads(32, 8, 128),
         "page": 64, "topk": 0, "window": 0},
        # a decode batch of 64 ragged sequences
        {"name": "cache 64 x 16K", "op": "cache", "seqs": 64, "new": 1, "longest": 16384, **_heads(32, 8, 128),
         "page": 64, "topk": 0, "window": 0},
        # the layer's own decode: 32 selected blocks and a window of 256 keys, for each of 64 sequences
        {"name": "cache 64 x 16K selected", "op": "cache", "seqs": 64, "new": 1, "longest": 16384,
         **_heads(32, 8, 128), "page": 64, "topk": 32, "window": 256},
        # short prompts packed together, one-token sequences among them
        {"name": "prompt short 23", "op": "prompt", "seqs": 23, "tokens": 1111, **_heads(8, 8, 64)},
        # three prompts packed, four query heads per kv-head
        {"name": "prompt 8K", "op": "prompt", "seqs": 3, "tokens": 8192, **_heads(32, 8, 128)},
        # one long prompt, eight query heads on one kv-head
        {"name": "prompt 16K", "op": "prompt", "seqs": 1, "tokens": 16384, **_heads(8, 1, 128)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "cache", "prompt"])
    hq, hkv = rng.choice([(32, 8), (8, 8), (8, 1), (8, 4), (16, 2)])
    d = rng.choice([64, 128])
    c = {"op": op, **_heads(hq, hkv, d)}
    if op == "rope":
        c.update(tokens=_log(rng, 1, 65536), rot=rng.choice([16, 32, 48, 64, d]), layout=rng.choice(["half", "pairs"]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), far=_log(rng, 16, 1 << 20),
                 stretch=rng.choice([1.0, 2.0, 8.0, 32.0]))
    elif op == "append":
        seqs = _log(rng, 1, 64)
        c.update(seqs=seqs, tokens=seqs + _log(rng, 1, 32768), have=_log(rng, 1, 2048), page=rng.choice([64, 128]),
                 rot=rng.choice([32, 64, d]), layout=rng.choice(["half", "pairs"]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op == "cache":
        seqs = _log(rng, 1, 64)
        topk = rng.choice([0, 0, 0, 8, 32])
        c.update(seqs=seqs, new=rng.choice([1, 1, 1, 2, 5]), longest=_log(rng, 64, min(131072, 524288 // seqs)),
                 page=rng.choice([64, 128]), topk=topk, window=rng.choice([64, 200, 256]) if topk else 0)
    else:
        seqs = _log(rng, 1, 24)
        c.update(seqs=seqs, tokens=seqs + _log(rng, 16, 4096))
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed, dev="cuda"):
    return torch.Generator(device=dev).manual_seed(seed)


def _split(total, parts):
    """`parts` lengths of at least 1 that sum to `total`, of different sizes."""
    w = torch.rand(parts, generator=_gen(parts, "cpu")).double() + 0.05
    n = 1 + ((total - parts) * w / w.sum()).long()
    n[-1] += total - int(n.sum())
    return n


def _lengths(c):
    """(tokens already in the cache, new tokens) of each sequence: a case's
    sizes are its own, whatever the seed."""
    if c["op"] == "append":
        new = _split(c["tokens"], c["seqs"])
        return torch.randint(0, 2 * c["have"], (c["seqs"],), generator=_gen(c["have"], "cpu")), new
    have = (c["longest"] * (0.25 + 0.75 * torch.rand(c["seqs"], generator=_gen(c["longest"], "cpu")))).long()
    have[0] = c["longest"]
    return (have - c["new"]).clamp_min(0), torch.full((c["seqs"],), c["new"])


def _starts(n):
    return torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(torch.int32)


def _frequencies(rot, base=10000.0, stretch=1.0, trained=32768, fast=32.0, slow=1.0):
    """Angle per position of each rotated pair, in float64.  A stretch above
    1 divides the frequencies that turn less than `slow` times over the
    trained length by it, keeps those that turn more than `fast` times and
    blends between them; the rotated vectors are then scaled by the returned
    factor."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if stretch == 1.0:
        return f, 1.0
    at = lambda t: rot * math.log(trained / (t * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f * keep + f / stretch * (1.0 - keep), 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    c = case
    g, h = _gen(seed), _gen(seed, "cpu")
    dev = "cuda"
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    s = {"case": c}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] in ("rope", "append"):
        f, m = _frequencies(c["rot"], stretch=c.get("stretch", 1.0))
        s.update(freq=f.to(dev), mscale=m, eps=1e-6, q_weight=1.0 + 0.1 * randn(d), k_weight=1.0 + 0.1 * randn(d))
    if c["op"] in ("rope", "append", "prompt"):
        # one projection's output: the heads of q, k and v side by side
        T = c["tokens"]
        x = torch.empty(T, hq + 2 * hkv, d, device=dev, dtype=dt)
        x.normal_(generator=g)
        x[:, hq + hkv:] *= torch.exp(0.5 * randn(1, hkv, 1)).to(dt)
        s.update(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:])
    if c["op"] == "rope":
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=dev, dtype=torch.int32)
        s["q_out"] = torch.empty(c["tokens"], hq, d, device=dev, dtype=dt)
        s["k_out"] = torch.empty(c["tokens"], hkv, d, device=dev, dtype=dt)
    if c["op"] in ("append", "cache"):
        n, P = c["seqs"], c["page"]
        have, new = _lengths(c)
        pages = (have + new + P - 1) // P
        width = int(pages.max())
        pool = int(pages.sum()) + 3
        order = torch.randperm(pool, generator=h).to(torch.int32)[:int(pages.sum())]
        first = pages.cumsum(0) - pages
        at = first[:, None] + torch.arange(width)
        table = torch.where(torch.arange(width) < pages[:, None], order[at.clamp_max(len(order) - 1)], -1)
        cache = torch.randint(0, 256, (2, pool, hkv, P, d), generator=g, device=dev, dtype=torch.uint8)
        # codes of normal values whose largest is near the end of the range
        cache = _codes_of_normals(cache)
        scale = torch.exp2(torch.randint(-8, -5, (2, pool, hkv), generator=g, device=dev).float())
        s.update(table=table.to(dev), kc=cache[0], vc=cache[1], ks=scale[0], vs=scale[1],
                 start=have.to(torch.int32).to(dev), cu=_starts(new).to(dev), length=(have + new).to(torch.int32).to(dev))
    if c["op"] == "cache":
        s["q"] = randn(n, c["new"], hq, d).to(torch.bfloat16)
        s["out"] = torch.empty(n, c["new"], hq, d, device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.empty(n, c["new"], hq, device=dev)
        s["idx"] = None
        if c["topk"]:
            s["idx"] = _selection(c, have, g)
    if c["op"] == "prompt":
        s["cu"] = _starts(_split(c["tokens"], c["seqs"])).to(dev)
        s["out"] = torch.empty(c["tokens"], hq, d, device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.empty(c["tokens"], hq, device=dev)
    if own:
        _plan(s)
    return s


def _codes_of_normals(b):
    """Random bytes to e4m3 codes of values spread like a normal of deviation 100: a table of 256 quantiles."""
    u = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
    t = (100.0 * math.sqrt(2.0) * torch.erfinv(2 * u - 1)).clamp(-448, 448).float().to(E4M3).view(torch.uint8)
    return t.to(b.device)[b.to(torch.int32)]


def _selection(c, have, g):
    """What the router gives each new token: distinct fully visible blocks in ascending order, padded with -1."""
    n, new, hkv, k, P = c["seqs"], c["new"], c["hkv"], c["topk"], c["page"]
    pos = have.to("cuda")[:, None] + torch.arange(new, device="cuda")
    visible = (pos + 1) // P
    width = max(int(visible.max()), k)
    r = torch.rand(n, new, hkv, width, generator=g, device="cuda")
    r = r.masked_fill(torch.arange(width, device="cuda") >= visible[:, :, None, None], -1.0)
    best, at = r.topk(k, dim=-1)
    at = at.masked_fill(best < 0, width).sort(dim=-1).values
    return torch.where(at >= width, -1, at).to(torch.int32).contiguous()


# ---------------------------------------------------------------- the framework's calls

def _plan(s):
    from content_routed_block_ssa_b200 import ssa
    c = s["case"]
    s["ssa"] = ssa
    heads = dict(h_q=c["hq"], h_kv=c["hkv"], d=c["d"])
    if c["op"] == "rope":
        s["p"] = ssa.make_rope_params(c["tokens"], **heads, rot=c["rot"], layout=c["layout"], dtype=c["dtype"],
                                      eps=s["eps"], mscale=s["mscale"], q_stride=s["q"].stride(0),
                                      k_stride=s["k"].stride(0))
    elif c["op"] == "append":
        s["p"] = ssa.make_append_params(n_tokens=c["tokens"], n_seq=c["seqs"], max_pages=s["table"].shape[1],
                                        n_pages=s["kc"].shape[0], page=c["page"], h_kv=c["hkv"], d=c["d"],
                                        rot=c["rot"], layout=c["layout"], dtype=c["dtype"], eps=s["eps"],
                                        mscale=s["mscale"], k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
    elif c["op"] == "cache":
        s["p"] = ssa.make_cache_attn_params(n_seq=c["seqs"], n_q=c["new"], **heads, page=c["page"],
                                            n_pages=s["kc"].shape[0], max_pages=s["table"].shape[1], topk=c["topk"],
                                            window=c["window"])
        s["ws"] = ssa.byte_buffer(ssa.ssa_cache_attn_workspace_size(s["p"]))
    else:
        s["p"] = ssa.make_prompt_params(n_seq=c["seqs"], n_q=c["tokens"], n_kv=c["tokens"], **heads,
                                        q_stride=s["q"].stride(0), k_stride=s["k"].stride(0),
                                        v_stride=s["v"].stride(0))


def _run_own(s):
    ssa, op, p = s["ssa"], s["case"]["op"], s["p"]
    if op == "rope":
        ssa.ssa_qk_rope(p, s["q"], s["k"], s["q_weight"], s["k_weight"], s["freq"], s["pos"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "append":
        ssa.ssa_cache_append(p, s["k"], s["v"], s["k_weight"], s["freq"], s["cu"], s["start"], s["table"],
                             s["kc"], s["vc"], s["ks"], s["vs"])
        return s["kc"].view(E4M3), s["vc"].view(E4M3), s["ks"], s["vs"]
    if op == "cache":
        ssa.ssa_cache_attn(p, s["q"], s["table"], s["length"], s["kc"], s["vc"], s["ks"], s["vs"], s["idx"],
                           s["out"], s["lse"], ws=s["ws"])
    else:
        ssa.ssa_prompt_attn(p, s["q"], s["k"], s["v"], s["cu"], s["cu"], s["out"], s["lse"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- plain forms

def _rotated(x, w, freq, pos, m, eps, layout):
    """The norm over each head and the rotation of its first dims, in float32."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a = pos.double()[:, None] * freq
    cos, sin = (a.cos() * m).float()[:, None], (a.sin() * m).float()[:, None]
    r = 2 * freq.numel()
    if layout == "half":
        u, v = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    else:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, clamped."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _append(x, page, slot, codes, scale):
    """x [T, h, d] into the pages' codes and scales, at (page, slot) of each token."""
    e_tok = _exponent(x.abs().amax(-1))
    touched, of = torch.unique(page, return_inverse=True)
    e_new = torch.full((len(touched), x.shape[1]), E_MIN, device=x.device, dtype=e_tok.dtype)
    e_new.index_reduce_(0, of, e_tok, "amax")
    anew = torch.zeros(len(touched), device=x.device, dtype=torch.bool)
    anew[of[slot == 0]] = True
    first = torch.full_like(touched, codes.shape[2]).index_reduce_(0, of, slot, "amin")
    e_old = torch.frexp(scale[touched])[1] - 1
    e = torch.where(anew[:, None], e_new, torch.maximum(e_old, e_new))
    old = codes[touched].view(E4M3).float()
    grown = torch.exp2((e_old - e).clamp_max(0).float())[:, :, None, None]
    before = (torch.arange(codes.shape[2], device=x.device) < first[:, None])[:, None, :, None]
    codes[touched] = torch.where(before, old * grown, old).to(E4M3).view(torch.uint8)
    scale[touched] = torch.exp2(e.float())
    codes[page, :, slot] = (x * torch.exp2(-e[of].float())[:, :, None]).to(E4M3).view(torch.uint8)


def _visible(s, keys):
    """Which of a sequence's keys each (sequence, new token, kv-head) attends."""
    c = s["case"]
    j = torch.arange(keys, device="cuda")
    pos = (s["length"][:, None] - c["new"] + torch.arange(c["new"], device="cuda"))[:, :, None, None]
    if s["idx"] is None:
        return j <= pos
    chosen = torch.zeros(*s["idx"].shape[:3], keys // c["page"] + 1, device="cuda", dtype=torch.bool)
    chosen.scatter_(3, torch.where(s["idx"] < 0, keys // c["page"], s["idx"]).long(), True)
    return chosen[..., :-1].repeat_interleave(c["page"], -1) | ((j <= pos) & (j > pos - c["window"]))


def _softmax_product(scores, values, eq):
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    l = p.sum(-1, keepdim=True)
    return torch.einsum(eq, p / l, values), (m + torch.log(l)).squeeze(-1)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, G = c["op"], c["hq"] // c["hkv"]
    if op == "rope":
        q = _rotated(s["q"], s["q_weight"], s["freq"], s["pos"], s["mscale"], s["eps"], c["layout"])
        k = _rotated(s["k"], s["k_weight"], s["freq"], s["pos"], s["mscale"], s["eps"], c["layout"])
        return q.to(s["q"].dtype), k.to(s["k"].dtype)
    if op == "append":
        t = torch.arange(c["tokens"], device="cuda", dtype=torch.int32)
        seq = torch.searchsorted(s["cu"], t, right=True) - 1
        pos = s["start"][seq] + t - s["cu"][seq]
        page, slot = s["table"][seq, pos // c["page"]].long(), (pos % c["page"]).long()
        k = _rotated(s["k"], s["k_weight"], s["freq"], pos, s["mscale"], s["eps"], c["layout"])
        _append(k, page, slot, s["kc"], s["ks"])
        _append(s["v"].float(), page, slot, s["vc"], s["vs"])
        return s["kc"].view(E4M3), s["vc"].view(E4M3), s["ks"], s["vs"]
    if op == "cache":
        at = s["table"].clamp_min(0).long()
        n, w = at.shape
        keys = w * c["page"]
        k = (s["kc"][at].view(E4M3).float() * s["ks"][at][..., None, None]).transpose(1, 2).reshape(n, c["hkv"], keys, c["d"])
        v = (s["vc"][at].view(E4M3).float() * s["vs"][at][..., None, None]).transpose(1, 2).reshape(n, c["hkv"], keys, c["d"])
        q = s["q"].float().view(n, c["new"], c["hkv"], G, c["d"])
        x = torch.einsum("nihgd,nhjd->nihgj", q, k) / math.sqrt(c["d"])
        x = x.masked_fill(~_visible(s, keys)[:, :, :, None], -math.inf)
        o, lse = _softmax_product(x, v, "nihgj,nhjd->nihgd")
        return o.reshape(n, c["new"], c["hq"], c["d"]).to(torch.bfloat16), lse.reshape(n, c["new"], c["hq"])
    T = c["tokens"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], t, right=True)
    q = s["q"].float().view(T, c["hkv"], G, c["d"])
    x = torch.einsum("ihgd,jhd->hgij", q, s["k"].float()) / math.sqrt(c["d"])
    x = x.masked_fill_((seq[:, None] != seq) | (t > t[:, None]), -math.inf)
    o, lse = _softmax_product(x, s["v"].float(), "hgij,jhd->ihgd")
    return o.reshape(T, c["hq"], c["d"]).to(torch.bfloat16), lse.reshape(c["hq"], T).t().contiguous()


# ---------------------------------------------------------------- what it costs at least

def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    es = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rope":
        return {"bytes": 2 * c["tokens"] * (hq + hkv) * d * es, "flops": c["tokens"] * (hq + hkv) * d * 7}
    if c["op"] == "append":
        return {"bytes": c["tokens"] * hkv * d * (2 * es + 2), "flops": c["tokens"] * hkv * d * 10}
    if c["op"] == "cache":
        length = sum(_lengths(c))
        rows = c["seqs"] * c["new"]
        pairs = length * c["new"]
        if c["topk"]:   # each new token's own blocks and window
            pairs = pairs.clamp_max(c["new"] * (c["topk"] * c["page"] + c["window"]))
        keys = int(torch.minimum(length, pairs).sum())
        return {"bytes": 2 * keys * hkv * d + rows * hq * d * 4 + rows * hq * 4, "flops": 4 * int(pairs.sum()) * hq * d}
    n = _split(c["tokens"], c["seqs"])
    pairs = int((n * (n + 1) // 2).sum())
    return {"bytes": c["tokens"] * ((2 * hq + 2 * hkv) * d * 2 + hq * 4), "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _turned(x, w, freq, pos, m, eps, layout):
    """Each rotated pair as a complex number times m e^(i pos f)."""
    x = x.double()
    x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * w.double()
    z = torch.polar(torch.full_like(freq, m).expand(len(pos), -1).contiguous(), pos.double().outer(freq))[:, None]
    r = 2 * freq.numel()
    head = x[..., :r]
    pair = (head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if layout == "half" else head.unflatten(-1, (r // 2, 2))).contiguous()
    turned = torch.view_as_real(torch.view_as_complex(pair) * z)
    x[..., :r] = (turned.transpose(-1, -2) if layout == "half" else turned).flatten(-2)
    return x


def _exact_append(x, page, slot, codes, scale):
    value = codes.view(E4M3).double()
    scale = scale.double()
    for p in page.unique().tolist():
        at = (page == p).nonzero()[:, 0]
        xs, sl = x[at], slot[at]
        top = xs.abs().amax((0, 2))
        s = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(E_MIN, E_MAX))
        if not bool((sl == 0).any()):
            s = torch.maximum(s, scale[p])
            old = value[p][:, :int(sl.min())]
            old.copy_((old * (scale[p] / s)[:, None, None]).float().to(E4M3))
        scale[p] = s
        value[p][:, sl] = (xs / s[:, None]).transpose(0, 1)
    return value, scale


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    G, d = c["hq"] // c["hkv"], c["d"]
    if c["op"] == "rope":
        return tuple(_turned(s[n], s[n + "_weight"], s["freq"], s["pos"], s["mscale"], s["eps"], c["layout"]) for n in "qk")
    if c["op"] == "append":
        cu, start, table = s["cu"].tolist(), s["start"].tolist(), s["table"].cpu()
        pos = torch.cat([torch.arange(b, b + j - i) for b, i, j in zip(start, cu, cu[1:])])
        page = torch.cat([table[n, torch.arange(b, b + j - i) // c["page"]] for n, (b, i, j) in enumerate(zip(start, cu, cu[1:]))])
        page, slot, pos = page.cuda().long(), (pos % c["page"]).cuda(), pos.cuda()
        k = _turned(s["k"], s["k_weight"], s["freq"], pos, s["mscale"], s["eps"], c["layout"])
        kv, ks = _exact_append(k, page, slot, s["kc"], s["ks"])
        vv, vs = _exact_append(s["v"].double(), page, slot, s["vc"], s["vs"])
        return kv, vv, ks, vs
    if c["op"] == "cache":
        n, new, P = c["seqs"], c["new"], c["page"]
        o = torch.zeros(n, new, c["hq"], d, device="cuda", dtype=torch.float64)
        lse = torch.zeros(n, new, c["hq"], device="cuda", dtype=torch.float64)
        for a in range(n):
            L = int(s["length"][a])
            pages = s["table"][a, :(L + P - 1) // P].long()
            k, v = ((x[pages].view(E4M3).double() * y[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
                    for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            j = torch.arange(L, device="cuda")
            for i in range(new):
                p = L - new + i
                see = (j <= p).expand(c["hkv"], L)
                if s["idx"] is not None:
                    see = ((j[None, :, None] // P) == s["idx"][a, i][:, None, :]).any(-1) | ((j <= p) & (j > p - c["window"]))
                q = s["q"][a, i].double().view(c["hkv"], G, d)
                x = (q @ k.transpose(1, 2) / math.sqrt(d)).masked_fill(~see[:, None], -math.inf)
                o[a, i] = (x.softmax(-1) @ v).flatten(0, 1)
                lse[a, i] = x.logsumexp(-1).flatten()
        return o, lse
    o = torch.zeros(c["tokens"], c["hq"], d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(c["tokens"], c["hq"], device="cuda", dtype=torch.float64)
    cu = s["cu"].tolist()
    for i, j in zip(cu, cu[1:]):
        future = torch.ones(j - i, j - i, device="cuda", dtype=torch.bool).triu(1)
        for a in range(c["hq"]):
            x = (s["q"][i:j, a].double() @ s["k"][i:j, a // G].double().t() / math.sqrt(d)).masked_fill_(future, -math.inf)
            lse[i:j, a] = x.logsumexp(-1)
            o[i:j, a] = x.softmax(-1) @ s["v"][i:j, a // G].double()
    return o, lse
