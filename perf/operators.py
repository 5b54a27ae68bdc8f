"""The paged-cache operators as measured work: their plain forms and the library's calls.

Four operators: per-head norm with rotation, append to a paged cache, attention of one
new token over it, attention of ragged chunks over it.  A case names its operator in
``"op"``; lengths of ragged batches are spread over ``lo .. hi`` by a fixed rule and
shuffled by the seed.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------

def _norm(name, **k):
    return dict({"name": name, "op": "norm", "dtype": "bf16", "D": 128, "style": "interleaved",
                 "axes": 1, "pairs": 64, "far": 4096, "head_major": False}, **k)


def _append(name, **k):
    return dict({"name": name, "op": "append", "dtype": "bf16", "D": 128, "page": 16, "style": "half",
                 "pairs": 64, "old": 0, "packed": True}, **k)


def _read(name, op, **k):
    return dict({"name": name, "op": op, "dtype": "bf16", "D": 128, "page": 16, "window": 0, "prefix": 0,
                 "cap": 0.0, "slopes": False, "causal": True}, **k)


def listed():
    return [
        # a 480P chunk (3 latent frames of 1560 tokens, 12 heads): queries and keys normed, rotated on
        # (frame, row, column) and laid out head by head, as the chunk step takes them
        _norm("norm chunk 480p", tokens=4680, hq=12, hk=12, axes=3, head_major=True),
        # one token of a 40-head model: latency
        _norm("norm one token", tokens=1, hq=40, hk=40, style="half", far=200000),
        # a serving batch, one new token per sequence, at far positions
        _append("append tokens", seqs=64, lo=1, hi=1, hq=32, hk=8, old=30000),
        # odd little prompts, 32-bit activations, small pages, part of the head rotated
        _append("append prompts fp32", seqs=3, lo=37, hi=701, hq=12, hk=4, D=64, page=8, style="interleaved",
                pairs=11, old=77, dtype="fp32", packed=False),
        # long prompts
        _append("append prompts", seqs=8, lo=500, hi=4001, hq=32, hk=8, page=64, pairs=32),
        # the first tokens of one conversation: latency
        _read("decode short", "decode", seqs=1, lo=131, hi=131, hq=32, hk=8),
        # a serving batch with ragged lengths
        _read("decode batch", "decode", seqs=64, lo=17, hi=8191, hq=32, hk=8),
        # one very long document
        _read("decode long", "decode", seqs=1, lo=200001, hi=200001, hq=32, hk=8, page=128),
        # sliding window behind a few sink tokens, capped scores, 32-bit, every head its own keys
        _read("decode window fp32", "decode", seqs=16, lo=901, hi=20011, hq=16, hk=16, D=64, page=32,
              window=1024, prefix=64, cap=30.0, dtype="fp32"),
        # short pieces of many sequences in one batch: window, cap and distance bias
        _read("attend pieces", "attend", seqs=12, lo=50, hi=3001, qlo=1, qhi=97, hq=16, hk=2, D=64, window=512,
              prefix=16, cap=50.0, slopes=True),
        # a 480P chunk over its history and itself (18 + 3 frames), no order within the chunk
        _read("attend chunk 480p", "attend", seqs=1, lo=32760, hi=32760, qlo=4680, qhi=4680, hq=12, hk=12,
              page=128, causal=False),
        # two long prompts, one of them behind a cached part, with an always-visible prefix
        _read("attend prompts", "attend", seqs=2, lo=4096, hi=9001, qlo=4096, qhi=4501, hq=32, hk=8, page=64,
              prefix=500),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "decode", "attend"])
    dt = "fp32" if rng.random() < 0.25 else "bf16"
    D = rng.choice([64, 128])
    style = rng.choice(["interleaved", "half"])
    pairs = rng.choice([D // 2, D // 4, 16]) if style == "half" else rng.randint(1, D // 2)
    hk = rng.choice([1, 2, 3, 4, 5, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "norm":
        c = _norm("", tokens=_log(rng, 1, 20000), hq=hk * group, hk=hk, D=D, dtype=dt, style=style, pairs=pairs,
                  far=_log(rng, 100, 1000000), axes=1 if pairs < 3 else rng.choice([1, 2, 3]),
                  head_major=rng.random() < 0.5)
        big = 2 * c["tokens"] * (c["hq"] + c["hk"]) * D * 4
        if big > 400e6:
            c["tokens"] = max(1, int(c["tokens"] * 400e6 / big))
    elif op == "append":
        s = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 20000 // s))
        c = _append("", seqs=s, lo=rng.randint(1, hi), hi=hi, hq=hk * group, hk=hk, D=D, dtype=dt, page=page,
                    style=style, pairs=pairs, old=_log(rng, 1, 2000), packed=rng.random() < 0.5)
        big = 2 * s * hi * (c["hq"] + 2 * hk) * D * 4
        if big > 400e6:
            c["hi"] = max(1, int(hi * 400e6 / big))
            c["lo"] = min(c["lo"], c["hi"])
    else:
        window = rng.choice([0, 0, 0, 1, 100, 1024])
        more = dict(hq=hk * group, hk=hk, D=D, dtype=dt, page=page, window=window,
                    prefix=rng.choice([0, 0, 1, 4, 300]), cap=rng.choice([0.0, 0.0, 30.0]),
                    slopes=rng.random() < 0.25)
        s = _log(rng, 1, 128) if op == "decode" else _log(rng, 1, 16)
        if op == "decode":
            hi = _log(rng, 1, max(1, 300000 // s))
            c = _read("", "decode", seqs=s, lo=rng.randint(1, hi), hi=hi, **more)
        else:
            hi = _log(rng, 1, max(1, 20000 // s))
            qhi = rng.randint(1, min(hi, 2000))
            c = _read("", "attend", seqs=s, lo=rng.randint(qhi, hi), hi=hi, qlo=rng.randint(1, qhi), qhi=qhi,
                      causal=rng.random() < 0.75, **more)
            pairs_n = s * qhi * hi * c["hq"] * (4 if dt == "fp32" else 1)
            if pairs_n > 1e9:  # the scores of the plain form stay within memory
                f = math.sqrt(1e9 / pairs_n)
                c["hi"], c["qhi"] = max(1, int(hi * f)), max(1, int(qhi * f))
                c["qhi"] = min(c["qhi"], c["hi"])
                c["qlo"] = min(c["qlo"], c["qhi"])
                c["lo"] = max(c["qhi"], min(c["lo"], c["hi"]))
    del c["name"]
    return c


# ---- sizes of a case -----------------------------------------------------------------

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spaced on a square-root scale (many short, few long)."""
    if n == 1:
        return [hi]
    return [lo + int(round((hi - lo) * (i / (n - 1)) ** 2)) for i in range(n)]


def _q_lens(c):
    if c["op"] == "decode":
        return [1] * c["seqs"]
    if c["op"] == "append":
        return _spread(c["lo"], c["hi"], c["seqs"])
    return _spread(c["qlo"], c["qhi"], c["seqs"])


def _kv_lens(c):
    if c["op"] == "append":
        return [q + c["old"] - (7 * i) % (c["old"] // 2 + 1) for i, q in enumerate(_q_lens(c))]
    return _spread(c["lo"], c["hi"], c["seqs"])


def _axis_pairs(c):
    """The video split of 64 pairs is 22 + 21 + 21: the first axis takes what does not divide."""
    n, p = c.get("axes", 1), c["pairs"]
    return [p - (n - 1) * (p // n)] + [p // n] * (n - 1)


def _visible(c, q, kv):
    """(query, key) pairs that attend, and keys that any query sees, of one sequence."""
    pos = torch.arange(kv - q, kv, dtype=torch.int64)
    hi = pos if c["causal"] else torch.full_like(pos, kv - 1)
    lo = (pos - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(pos)
    pre = min(c["prefix"], kv)
    n = (hi - torch.maximum(lo, torch.full_like(lo, pre)) + 1).clamp(min=0) + pre
    low = int(lo[0])
    return int(n.sum()), kv if pre >= low else kv - low + pre


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    D = c["D"]
    if c["op"] == "norm":
        n = c["tokens"] * (c["hq"] + c["hk"]) * D
        return {"bytes": 2 * n * e, "flops": 10 * n}
    if c["op"] == "append":
        t = sum(_q_lens(c))
        return {"bytes": 2 * t * (c["hq"] + 2 * c["hk"]) * D * e, "flops": 10 * t * (c["hq"] + c["hk"]) * D}
    pairs = keys = 0
    for q, kv in zip(_q_lens(c), _kv_lens(c)):
        a, b = _visible(c, q, kv)
        pairs, keys = pairs + a, keys + b
    t = sum(_q_lens(c))
    return {"bytes": (2 * t * c["hq"] + 2 * keys * c["hk"]) * D * e, "flops": 4 * D * c["hq"] * pairs}


# ---- inputs --------------------------------------------------------------------------

def _rand(g, shape, dt, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std + mean).to(dt)


def _rope_inputs(c, g, s):
    n = c["pairs"]
    s["pairs"] = _axis_pairs(c)
    s["omega"] = torch.cat([10000.0 ** (-torch.arange(m, dtype=torch.float64) / m) for m in s["pairs"]]).to(DEV).float()
    s["q_weight"] = _rand(g, (c["D"],), torch.float32, 0.1, 1.0)
    s["k_weight"] = _rand(g, (c["D"],), torch.float32, 0.1, 1.0)
    s["pair_axis"] = torch.repeat_interleave(torch.arange(len(s["pairs"]), device=DEV),
                                             torch.tensor(s["pairs"], device=DEV), output_size=n)


def _batch(c, g, s):
    """Ragged batch over a paged cache: lengths, pages in random order, stale rows behind the lengths."""
    order = torch.randperm(c["seqs"], generator=g, device=DEV).cpu().tolist()
    q = [_q_lens(c)[i] for i in order]
    kv = [_kv_lens(c)[i] for i in order]
    page = c["page"]
    need = [-(-n // page) for n in kv]
    width, pages = max(need), sum(need) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    s["table"] = table.to(DEV)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu_q"] = torch.tensor([0] + q, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
    s["tokens"], s["qmax"], s["kmax"] = sum(q), max(q), width * page
    s["q_lens"], s["kv_lens"] = q, kv
    shape = (pages, c["hk"], page, c["D"])
    s["k_cache"] = _rand(g, shape, DT[c["dtype"]])
    s["v_cache"] = _rand(g, shape, DT[c["dtype"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, D = DT[c["dtype"]], c["D"]
    s = {"case": c}
    if c["op"] == "norm":
        t = s["tokens"] = c["tokens"]
        _rope_inputs(c, g, s)
        s["positions"] = torch.randint(0, c["far"], (len(s["pairs"]), t), generator=g, device=DEV, dtype=torch.int32)
        s["q"] = _rand(g, (t, c["hq"], D), dt, 2.0)
        s["k"] = _rand(g, (t, c["hk"], D), dt, 2.0)
        if c["head_major"]:
            s["q_out"] = torch.empty((c["hq"], t, D), dtype=dt, device=DEV)
            s["k_out"] = torch.empty((c["hk"], t, D), dtype=dt, device=DEV)
        else:
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        _batch(c, g, s)
        t = s["tokens"]
        if c["op"] == "append":
            _rope_inputs(c, g, s)
            rows = _rand(g, (t, c["hq"] + 2 * c["hk"], D), dt, 2.0)  # one projection, as a model's layer leaves it
            s["q"], s["k"], s["v"] = rows.split([c["hq"], c["hk"], c["hk"]], dim=1)
            if not c["packed"]:
                s["q"], s["k"], s["v"] = s["q"].contiguous(), s["k"].contiguous(), s["v"].contiguous()
            s["q_out"] = torch.empty((t, c["hq"], D), dtype=dt, device=DEV)
        else:
            s["q"] = _rand(g, (t, c["hq"], D), dt, 1.5)
            s["out"] = torch.empty((t, c["hq"], D), dtype=dt, device=DEV)
            s["prefix_len"] = torch.full((c["seqs"],), c["prefix"], dtype=torch.int32, device=DEV) if c["prefix"] else None
            s["slopes"] = (2.0 ** (-8.0 * (torch.arange(c["hq"], device=DEV, dtype=torch.float32) + 1) / c["hq"])
                           if c["slopes"] else None)
    if own:
        import kv_cache_compression_fkv_b200 as fkv
        s["fkv"] = fkv
        if c["op"] in ("norm", "append"):
            s["rope"] = fkv.make_rope(s["omega"], axis_pairs=s["pairs"], style=c["style"], norm=True, eps=EPS,
                                      q_weight=s["q_weight"], k_weight=s["k_weight"])
        if c["op"] != "norm":
            s["cache"] = fkv.PagedCache(s["k_cache"], s["v_cache"], s["table"], num_q_heads=c["hq"],
                                        softcap=c.get("cap", 0.0), window=c.get("window", 0),
                                        causal=c.get("causal", True), alibi_slopes=s.get("slopes"))
            s["ws"] = s["cache"].workspace()
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    fkv, c = s["fkv"], s["case"]
    if c["op"] == "norm":
        q_out, k_out = s["q_out"], s["k_out"]
        if c["head_major"]:
            q_out, k_out = q_out.transpose(0, 1), k_out.transpose(0, 1)
        fkv.qk_norm_rope(s["rope"], s["q"], s["k"], s["positions"], q_out, k_out)
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        fkv.paged_append(s["cache"], s["kv_len"], s["k"], s["v"], s["ws"], cu_q=s["cu_q"], rope=s["rope"],
                         q=s["q"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "decode":
        fkv.paged_decode(s["cache"], s["kv_len"], s["q"], s["out"], s["ws"], prefix_len=s["prefix_len"])
    else:
        fkv.paged_attend(s["cache"], s["kv_len"], s["cu_q"], s["q"], s["out"], s["ws"], prefix_len=s["prefix_len"])
    return {"out": s["out"]}


def _rotated(x, weight, s, c, angle):
    """Norm and rotation of [tokens, heads, D] rows, angles [tokens, pairs] in 64 bits."""
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    n = c["pairs"]
    if c["style"] == "half":
        x0, x1, rest = y[..., :n], y[..., n:2 * n], y[..., 2 * n:]
        out = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos, rest], -1)
    else:
        x0, x1, rest = y[..., 0:2 * n:2], y[..., 1:2 * n:2], y[..., 2 * n:]
        out = torch.cat([torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2), rest], -1)
    return out.to(x.dtype)


def _token_places(s):
    """Sequence and cache position of every token."""
    t = torch.arange(s["tokens"], device=DEV)
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    q_len = cu[1:] - cu[:-1]
    return b, s["kv_len"].long()[b] - q_len[b] + t - cu[b], t - cu[b]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        angle = s["positions"].double()[s["pair_axis"]].t() * s["omega"].double()
        q, k = _rotated(s["q"], s["q_weight"], s, c, angle), _rotated(s["k"], s["k_weight"], s, c, angle)
        if c["head_major"]:
            q, k = q.transpose(0, 1).contiguous(), k.transpose(0, 1).contiguous()
        return {"q": q, "k": k}
    if c["op"] == "append":
        b, p, _ = _token_places(s)
        angle = p.double().unsqueeze(1) * s["omega"].double()
        q, k = _rotated(s["q"], s["q_weight"], s, c, angle), _rotated(s["k"], s["k_weight"], s, c, angle)
        page, row = s["table"].long()[b, p // c["page"]], p % c["page"]
        s["k_cache"][page, :, row] = k
        s["v_cache"][page, :, row] = s["v"]
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"out": _attention_plain(s, c)}


def _dense(cache, table):
    """[sequences, heads, positions, D] of a paged cache, in 32 bits (unused pages read as page 0, masked later)."""
    x = cache[table.clamp(min=0).long()].float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attention_plain(s, c):
    hk, D, G, qm = c["hk"], c["D"], c["hq"] // c["hk"], s["qmax"]
    n = c["seqs"]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    i = torch.arange(qm, device=DEV)
    q_len = cu[1:] - cu[:-1]
    at = (cu[:-1].unsqueeze(1) + i).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[at].view(n, qm, hk, G, D).permute(0, 2, 3, 1, 4).reshape(n, hk, G * qm, D)
    z = torch.matmul(q, _dense(s["k_cache"], s["table"]).transpose(2, 3)).view(n, hk, G, qm, -1)
    z = z * (1.0 / math.sqrt(D))
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    j = torch.arange(z.shape[-1], device=DEV)
    p = ((kv - q_len).unsqueeze(1) + i).unsqueeze(-1)  # [n, qm, 1]
    if c["slopes"]:
        z = z + s["slopes"].view(1, hk, G, 1, 1) * (j - p).float().view(n, 1, 1, qm, -1)
    near = torch.ones_like(p * j, dtype=torch.bool)
    if c["causal"]:
        near = near & (j <= p)
    if c["window"]:
        near = near & (j > p - c["window"])
    if s["prefix_len"] is not None:
        near = near | (j < s["prefix_len"].view(n, 1, 1))
    near = (near & (j < kv.view(n, 1, 1))).view(n, 1, 1, qm, -1)
    z = z.masked_fill(~near, -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    del z
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(n, hk, G * qm, -1), _dense(s["v_cache"], s["table"])).view(n, hk, G, qm, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, qm, hk * G, D)
    b, _, k = _token_places(s)
    return o[b, k].to(s["q"].dtype)


# ---- the definition in 64 bits ---------------------------------------------------------

def _turned(x, w, omega, pos, pairs, style):
    x = x.double().clone()
    x /= ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    x *= w.double()
    first = list(range(pairs)) if style == "half" else list(range(0, 2 * pairs, 2))
    second = [i + pairs for i in first] if style == "half" else [i + 1 for i in first]
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.ones_like(pos), pos * omega.double())[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        pos = torch.cat([s["positions"][a].double()[:, None].expand(-1, m) for a, m in enumerate(s["pairs"])], 1)
        got = {x: _turned(s[x], s[x + "_weight"], s["omega"], pos, c["pairs"], c["style"]) for x in "qk"}
        return {x: v.transpose(0, 1).contiguous() if c["head_major"] else v for x, v in got.items()}
    ps, table = c["page"], s["table"].cpu().tolist()
    if c["op"] == "append":
        pos = torch.cat([torch.arange(kv - q, kv) for q, kv in zip(s["q_lens"], s["kv_lens"])]).to(DEV).double()
        pos = pos[:, None].expand(-1, c["pairs"])
        k = _turned(s["k"], s["k_weight"], s["omega"], pos, c["pairs"], c["style"])
        kc, vc, t = s["k_cache"].double(), s["v_cache"].double(), 0
        for b, (q, kv) in enumerate(zip(s["q_lens"], s["kv_lens"])):
            p = kv - q
            while p < kv:  # rows up to the end of the page
                m = min(kv, (p // ps + 1) * ps) - p
                kc[table[b][p // ps], :, p % ps:p % ps + m] = k[t:t + m].transpose(0, 1)
                vc[table[b][p // ps], :, p % ps:p % ps + m] = s["v"][t:t + m].double().transpose(0, 1)
                p, t = p + m, t + m
        return {"q": _turned(s["q"], s["q_weight"], s["omega"], pos, c["pairs"], c["style"]), "k_cache": kc,
                "v_cache": vc}
    out, t, G = [], 0, c["hq"] // c["hk"]
    for b, (q, kv) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        pages = table[b][:-(-kv // ps)]
        j = torch.arange(kv, device=DEV)
        i = torch.arange(kv - q, kv, device=DEV)[:, None]
        see = (j <= i) if c["causal"] else torch.ones_like(j <= i)
        if c["window"]:
            see = see & (i - j < c["window"])
        see = see | (j < c["prefix"])
        heads = []
        for h in range(c["hq"]):
            k = s["k_cache"][pages, h // G].reshape(-1, c["D"])[:kv].double()
            v = s["v_cache"][pages, h // G].reshape(-1, c["D"])[:kv].double()
            z = s["q"][t:t + q, h].double() @ k.t() / math.sqrt(c["D"])
            z = torch.tanh(z / c["cap"]) * c["cap"] if c["cap"] else z
            z = z - s["slopes"][h].double() * (i - j) if c["slopes"] else z
            z[~see] = -math.inf
            heads.append(torch.softmax(z, -1) @ v)
        out.append(torch.stack(heads, 1))
        t += q
    return {"out": torch.cat(out)}
