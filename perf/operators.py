"""Cases, plain forms and 64-bit definitions of three operators that stand between the QKV projection and the output
projection of a transformer block: rotary positions, norms of queries and keys with the rotation, and attention under masks.

Tensors are [B, N, heads, head_dim]; where a case says "fused", they are views of one [B, N, (hq + 2 hk) * d] projection output."""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _rope(name, dtype, B, N, h, d, rot, layout, axes, scaling, start, fused):
    return {"name": name, "op": "rope", "dtype": dtype, "B": B, "N": N, "h": h, "d": d, "rot": rot, "layout": layout,
            "axes": axes, "scaling": scaling, "start": start, "fused": fused}


def _norm(name, dtype, B, N, hq, hk, d, rot, layout, axes, scaling, start, norm):
    return {"name": name, "op": "qk_norm_rope", "dtype": dtype, "B": B, "N": N, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "layout": layout, "axes": axes, "scaling": scaling, "start": start, "norm": norm}


def _attn(name, dtype, B, Nq, Nk, hq, hk, d, causal=False, prefix=False, docs=0, lens=False, cap=0.0, bias=False,
          spread=1.0, layout=1):
    return {"name": name, "op": "masked_attention", "dtype": dtype, "B": B, "Nq": Nq, "Nk": Nk, "hq": hq, "hk": hk,
            "d": d, "causal": causal, "prefix": prefix, "docs": docs, "lens": lens, "cap": cap, "bias": bias,
            "spread": spread, "layout": layout}


def listed():
    return [
        # the queries of one new token, far into a long context
        _rope("rope_one_token", "bf16", 1, 1, 16, 64, 64, "half", 1, "none", 70001, False),
        # a batch of clips of 8 slots of 16 x 16 patches: three axes of 10 pairs, 4 dims left, q inside a fused projection
        _rope("rope_clips_3_axes", "f16", 4, 2048, 16, 64, 60, "interleaved", 3, "none", 0, True),
        # a long prompt whose heads are turned in their first half, context stretched by frequency
        _rope("rope_long_half_head", "bf16", 1, 18432, 32, 128, 64, "half", 1, "yarn", 4096, False),
        # one new token for each of 32 requests, shared key heads
        _norm("norm_step_32", "bf16", 32, 1, 16, 4, 128, 128, "half", 1, "linear", 30000, "rms"),
        # ViT-L clips of 16 frames with a leading token: norm with mean and bias, three axes
        _norm("norm_clips_3_axes", "f16", 4, 3137, 16, 16, 64, 60, "interleaved", 3, "none", 0, "layer"),
        # predictor heads of 32, an odd number of tokens, 32-bit values, part of the head turned
        _norm("norm_odd_f32", "f32", 3, 1025, 12, 12, 32, 20, "half", 1, "ntk", 11, "rms"),
        # one query of one stream against a short cache
        _attn("attn_step_one", "bf16", 1, 1, 257, 16, 16, 64, causal=True, lens=True),
        # one new token for each of 16 requests over long ragged caches, shared key heads, capped
        _attn("attn_step_cache", "bf16", 16, 1, 8192, 32, 8, 128, causal=True, lens=True, cap=30.0, spread=3.0),
        # clips of unequal lengths packed into one row, rows behind the last left over
        _attn("attn_packed_clips", "f16", 1, 12548, 12548, 16, 16, 64, docs=24, layout=3),
        # prompts: a bidirectional prefix, causal behind it, capped, shared key heads
        _attn("attn_prefix_cap", "bf16", 4, 2048, 2048, 16, 4, 128, causal=True, prefix=True, cap=50.0, spread=3.0),
        # a clip of 64 frames (8192 tokens) with a penalty on distance
        _attn("attn_long_bias", "f16", 1, 8192, 8192, 16, 16, 64, bias=True),
        # padded batch of an odd length, heads of 80
        _attn("attn_padded_odd", "bf16", 5, 1369, 1369, 16, 16, 80, lens=True, layout=2),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "qk_norm_rope", "masked_attention", "masked_attention"])
    if op == "masked_attention":
        dtype = rng.choice(["f16", "bf16"])
        d = rng.choice([32, 64, 64, 80, 96, 128, 128])
        hk = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        hq = hk * rng.choice([1, 1, 2, 4])
        cap = rng.choice([0.0, 0.0, 20.0, 50.0])
        bias = rng.random() < 0.3
        spread = rng.choice([1.0, 3.0]) if cap else 1.0
        layout = rng.randrange(1, 1000)
        if rng.random() < 0.4:  # few queries over a cache
            B = _between(rng, 1, 32)
            Nq = rng.choice([1, 1, 1, 2, 5, 8])
            Nk = _between(rng, 16, 16384)
            while B * Nk * hk * d > 1 << 26:
                B = max(1, B // 2)
                Nk = max(16, Nk * 3 // 4)
            c = _attn("", dtype, B, Nq, Nk, hq, hk, d, causal=True, lens=True, cap=cap, bias=bias, spread=spread,
                      layout=layout)
        else:
            N = _between(rng, 20, 8192)
            B = _between(rng, 1, 16)
            while B * N * N * hq * max(d, 64) > 1 << 36:
                if B > 1:
                    B //= 2
                else:
                    N = N * 3 // 4
            kind = rng.choice(["full", "causal", "prefix", "docs", "lens"])
            docs = min(_between(rng, 2, 64), N // 4) if kind == "docs" else 0
            c = _attn("", dtype, B, N, N, hq, hk, d, causal=kind in ("causal", "prefix"), prefix=kind == "prefix",
                      docs=docs, lens=kind == "lens", cap=cap, bias=bias, spread=spread, layout=layout)
    else:
        dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
        d = rng.choice([32, 64, 64, 80, 128, 128])
        axes = rng.choice([1, 1, 3])
        rot = {32: [32, 20, 30], 64: [64, 32, 60], 80: [80, 40, 78], 128: [128, 64, 126]}[d]
        rot = rot[2] if axes == 3 else rng.choice(rot[:2])
        layout = rng.choice(["half", "interleaved"])
        scaling = "none" if axes == 3 else rng.choice(["none", "linear", "ntk", "yarn"])
        h = rng.choice([1, 3, 8, 12, 16, 32])
        B = _between(rng, 1, 32)
        N = 1 if rng.random() < 0.3 else _between(rng, 2, 16384)
        hk = h if rng.random() < 0.5 else max(1, h // 4)
        while 2 * B * N * (h if op == "rope" else h + hk) * d * TYPES[dtype].itemsize > 300e6:
            B = max(1, B // 2)
            N = N * 3 // 4
        start = rng.choice([0, 0, 1000, 100000, 1000000])
        if op == "rope":
            c = _rope("", dtype, B, N, h, d, rot, layout, axes, scaling, start, rng.random() < 0.5)
        else:
            c = _norm("", dtype, B, N, h, hk, d, rot, layout, axes, scaling, start, rng.choice(["rms", "layer"]))
    del c["name"]
    return c


# ---------------------------------------------------- what a case lays down
FACTOR, ORIGINAL, FAST, SLOW = 8.0, 8192, 32.0, 1.0


def _frequencies(case):
    """(radians per position, axis) of each pair, and the factor on cosine and sine."""
    axes, pairs = case["axes"], case["rot"] // 2
    n = pairs // axes
    base = 10000.0
    if case["scaling"] == "ntk":
        base *= FACTOR ** (n / (n - 1.0))
    freq = [base ** (-i / n) for i in range(n)] * axes
    axis = [a for a in range(axes) for _ in range(n)]
    factor = 1.0
    if case["scaling"] == "linear":
        freq = [f / FACTOR for f in freq]
    if case["scaling"] == "yarn":
        keep = [min(1.0, max(0.0, (ORIGINAL * f / (2 * math.pi) - SLOW) / (FAST - SLOW))) for f in freq]
        freq = [f * (g + (1 - g) / FACTOR) for f, g in zip(freq, keep)]
        factor = 1.0 + 0.1 * math.log(FACTOR)
    return freq, axis, factor


def _positions(case):
    """[N], or [3, N] of slot, row and column on a grid of 16 columns and 16 rows."""
    n = torch.arange(case["N"], device="cuda")
    if case["axes"] == 1:
        return n + case["start"]
    return torch.stack([n // 256 + case["start"], n // 16 % 16, n % 16])


def _lens(case):
    r = random.Random(case["layout"])
    n = [r.randint(max(case["Nq"] if case["causal"] else 1, case["Nk"] // 2), case["Nk"]) for _ in range(case["B"])]
    return n if case["lens"] else [case["Nk"]] * case["B"]


def _documents(case):
    """Offsets of each row's documents, one of them empty, a few tokens behind the last."""
    r = random.Random(case["layout"])
    rows = []
    for _ in range(case["B"]):
        used = case["Nk"] - min(case["Nk"] // 8, 100)
        cuts = r.sample(range(1, used), case["docs"] - 1)
        rows.append(sorted([0, cuts[0], used] + cuts))
    return rows


def _prefixes(case):
    r = random.Random(case["layout"] + 1)
    return [r.randint(0, case["Nk"] // 2) for _ in range(case["B"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, by=1.0, to=dtype):
        return torch.randn(*shape, generator=g, device="cuda").mul_(by).to(to)

    s = {"case": case}
    B, d = case["B"], case["d"]
    if case["op"] == "masked_attention":
        Nq, Nk, hq, hk = case["Nq"], case["Nk"], case["hq"], case["hk"]
        if Nq == Nk:  # views of one projection output
            qkv = normal(B, Nq, (hq + 2 * hk) * d)
            qkv[..., :hq * d] *= case["spread"]
            q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], -1))
        else:         # new tokens against a cache
            q, k, v = normal(B, Nq, hq, d, by=case["spread"]), normal(B, Nk, hk, d), normal(B, Nk, hk, d)
        s |= {"q": q, "k": k, "v": v, "lens": None, "start": None, "prefix": None, "docs": None, "slopes": None}
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        if case["lens"]:
            s["lens"] = ints(_lens(case))
            if Nq != Nk:
                s["start"] = s["lens"] - Nq
        if case["prefix"]:
            s["prefix"] = ints(_prefixes(case))
        if case["docs"]:
            s["docs"] = ints(_documents(case))
        if case["bias"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
        return s
    N = case["N"]
    freq, axis, factor = _frequencies(case)
    s["pos"] = _positions(case)
    s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
    s["axis"], s["factor"] = axis, factor
    if own:
        import jepa_video_encoder_b200 as jb
        n = len(freq) // case["axes"]
        scaling = {"none": None, "linear": {"type": "linear", "factor": FACTOR}, "ntk": {"type": "ntk", "factor": FACTOR},
                   "yarn": {"type": "yarn", "factor": FACTOR, "original": ORIGINAL, "fast": FAST, "slow": SLOW}}
        s["plan"] = jb.rope_plan(case["rot"], layout=case["layout"], sections=[n] * case["axes"],
                                 scaling=scaling[case["scaling"]])
    if case["op"] == "rope":
        h = case["h"]
        s["x"] = normal(B, N, 3, h, d)[:, :, 0] if case["fused"] else normal(B, N, h, d)
        return s
    hq, hk = case["hq"], case["hk"]
    qkv = normal(B, N, (hq + 2 * hk) * d, by=1.5)
    s["q"], s["k"], _ = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], -1))
    s["qw"], s["kw"] = (1 + normal(d, by=0.1, to=torch.float32) for _ in range(2))
    s["qb"], s["kb"] = (normal(d, by=0.1, to=torch.float32) if case["norm"] == "layer" else None for _ in range(2))
    return s


# -------------------------------------------------------------- plain forms
def _turn(x, s):
    """Rotate 32-bit x [B, N, h, d] by its positions; the angles in 64 bits, as far positions need."""
    case = s["case"]
    rot = case["rot"]
    pos = s["pos"].double().reshape(-1, case["N"])
    angle = pos[s["axis"]].T * s["freq"]                       # [N, pairs]
    c, n = (t.float()[:, None] * s["factor"] for t in (angle.cos(), angle.sin()))
    out = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * n, a * n + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * n, a * n + b * c
    return out


def _normed(x, w, b):
    x = x.float()
    if b is not None:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    return x if b is None else x + b


def _plain_attention(s):
    case, q, k, v = s["case"], s["q"].float(), s["k"].float(), s["v"].float()
    B, Nq, Nk, g = case["B"], case["Nq"], case["Nk"], case["hq"] // case["hk"]
    k, v = k.repeat_interleave(g, 2), v.repeat_interleave(g, 2)
    p = q.transpose(1, 2) @ k.permute(0, 2, 3, 1)              # [B, hq, Nq, Nk]
    p *= 1.0 / math.sqrt(case["d"])
    if case["cap"]:
        p = torch.tanh(p / case["cap"]).mul_(case["cap"])
    i, j = torch.arange(Nq, device="cuda"), torch.arange(Nk, device="cuda")
    i = (i + Nk - Nq).expand(B, Nq) if s["start"] is None else i + s["start"][:, None]
    if case["bias"]:
        p -= s["slopes"][:, None, None] * (i[:, None, :, None] - j).abs()
    ok = (j < (Nk if s["lens"] is None else s["lens"][:, None])).expand(B, Nk)[:, None, :]
    if case["causal"]:
        under = j <= i[:, :, None]
        ok = ok & (under if s["prefix"] is None else under | (j < s["prefix"][:, None, None]))
    if case["docs"]:
        doc = torch.searchsorted(s["docs"], j.int().expand(B, Nk).contiguous(), right=True)
        ok = ok & (doc[:, :, None] == doc[:, None, :]) & (doc[:, :, None] < s["docs"].shape[1])
    ok = ok[:, None]
    p = p.masked_fill_(~ok, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v.transpose(1, 2)) / torch.where(total == 0, 1.0, total)
    return out.transpose(1, 2).to(s["q"].dtype)


def run(state):
    s = state
    case = s["case"]
    if own:
        import jepa_video_encoder_b200 as jb
        if case["op"] == "rope":
            return jb.rope(s["x"], s["pos"], s["plan"])
        if case["op"] == "qk_norm_rope":
            return jb.qk_norm_rope(s["q"], s["k"], s["pos"], s["plan"], s["qw"], s["kw"], q_bias=s["qb"], k_bias=s["kb"],
                                   norm=case["norm"], eps=1e-6)
        return jb.masked_attention(s["q"], s["k"], s["v"], cap=case["cap"], slopes=s["slopes"], causal=case["causal"],
                                   prefix=s["prefix"], doc_offsets=s["docs"], kv_len=s["lens"], q_start=s["start"])
    if case["op"] == "rope":
        return _turn(s["x"].float(), s).to(s["x"].dtype)
    if case["op"] == "qk_norm_rope":
        return (_turn(_normed(s["q"], s["qw"], s["qb"]), s).to(s["q"].dtype),
                _turn(_normed(s["k"], s["kw"], s["kb"]), s).to(s["k"].dtype))
    return _plain_attention(s)


# ------------------------------------------------------------ what it needs
def _intervals(case):
    """[lo, hi) of the keys that each query row of each batch row reads."""
    Nq, Nk = case["Nq"], case["Nk"]
    lens, prefix = _lens(case), _prefixes(case)
    for b in range(case["B"]):
        start = lens[b] - Nq if case["lens"] and Nq != Nk else Nk - Nq
        if case["docs"]:
            offsets = _documents(case)[b]
            for lo, hi in zip(offsets, offsets[1:]):
                for _ in range(hi - lo):
                    yield b, lo, hi
            continue
        for i in range(Nq):
            hi = lens[b]
            if case["causal"]:
                hi = min(hi, max(start + i + 1, prefix[b] if case["prefix"] else 0))
            yield b, 0, max(0, hi)


def work(case):
    size = TYPES[case["dtype"]].itemsize
    B, d = case["B"], case["d"]
    if case["op"] == "masked_attention":
        pairs, top = 0, [0] * B
        for b, lo, hi in _intervals(case):
            pairs += hi - lo
            top[b] = max(top[b], hi)
        return {"bytes": size * d * (2 * B * case["Nq"] * case["hq"] + 2 * sum(top) * case["hk"]),
                "flops": 4 * d * case["hq"] * pairs}
    heads = case["h"] if case["op"] == "rope" else case["hq"] + case["hk"]
    values = B * case["N"] * heads * d
    turned = 3 * B * case["N"] * heads * case["rot"]
    return {"bytes": 2 * values * size + 8 * case["N"] * case["axes"],
            "flops": turned + (0 if case["op"] == "rope" else 4 * values)}


# --------------------------------------------------------------- in 64 bits
def _turned_exactly(x, case, pos):
    """Each pair as a complex number, times factor * e^(i angle)."""
    freq, axis, factor = _frequencies(case)
    at = pos.double().reshape(case["axes"], -1)
    angle = torch.stack([at[a] * f for a, f in zip(axis, freq)], -1)
    by = torch.polar(torch.full_like(angle, factor), angle)[:, None]
    rot, half = case["rot"], case["rot"] // 2
    first = x[..., :rot]
    if case["layout"] == "half":
        z = torch.complex(first[..., :half].contiguous(), first[..., half:].contiguous()) * by
        z = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_real(torch.view_as_complex(first.contiguous().unflatten(-1, (half, 2))) * by).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned_exactly(s["x"].double(), case, s["pos"])
    if case["op"] == "qk_norm_rope":
        got = []
        for x, w, b in ((s["q"], s["qw"], s["qb"]), (s["k"], s["kw"], s["kb"])):
            x = x.double()
            mean = x.mean(-1, keepdim=True) if case["norm"] == "layer" else torch.zeros_like(x[..., :1])
            y = (x - mean) / ((x - mean).square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            got.append(_turned_exactly(y + (0 if b is None else b.double()), case, s["pos"]))
        return tuple(got)
    if case["B"] * case["hq"] * case["Nq"] * case["Nk"] > 4e9:
        return None
    B, Nq, Nk, hq, d = case["B"], case["Nq"], case["Nk"], case["hq"], case["d"]
    lo, hi = torch.zeros(B, Nq, dtype=torch.int64), torch.zeros(B, Nq, dtype=torch.int64)
    seen = [0] * B
    for b, low, high in _intervals(case):
        lo[b, seen[b]], hi[b, seen[b]] = low, high
        seen[b] += 1
    lo, hi = lo.cuda(), hi.cuda()
    out = torch.zeros(B, Nq, hq, d, dtype=torch.float64, device="cuda")
    key, lens = torch.arange(Nk, device="cuda"), _lens(case)
    for b in range(B):
        first = lens[b] - Nq if case["lens"] and Nq != Nk else Nk - Nq
        away = (torch.arange(Nq, device="cuda")[:, None] + first - key).abs().double()
        barred = (key < lo[b][:, None]) | (key >= hi[b][:, None])
        for h in range(hq):
            kv = h * case["hk"] // hq
            score = s["q"][b, :, h].double() @ s["k"][b, :, kv].double().T / math.sqrt(d)
            if case["cap"]:
                score = case["cap"] * torch.tanh(score / case["cap"])
            if case["bias"]:
                score = score - float(s["slopes"][h]) * away
            weight = torch.softmax(score.masked_fill(barred, -math.inf), -1).nan_to_num(0.0)
            out[b, :, h] = weight @ s["v"][b, :, kv].double()
    return out
