"""The per-head operators on the GPU against plain implementations in 64
bits.  Error bounds, with u = eps / 2 of the output's type:

rotation: the angle is off by half a rounding of a value up to 1 half-turn
(2^-25 half-turns, pi * 2^-25 rad), cosine and sine by 2 units of 2^-23 and
their product with the factor by 2^-24 relative, the two products and their
sum by 3 * 2^-24: under 2^-21 of factor * (|x0| + |x1|), plus u |result|.

norms: mean and mean square are sums of d <= 256 terms in f32 by lanes and a
tree (at most 13 additions in a row), so the statistics are off by 2^-20
relative and the mean by 2^-20 of the largest |x|; y is off by under 2^-18 of
(|x|max / std) |w| + |b|; this passes through the rotation with |cos| + |sin|
<= sqrt 2.

attention: products of 16-bit values are exact in f32, so a score's error is
at most (d + 4) 2^-23 of scale * sum |q k| plus 2^-22 of its own terms (cap,
bias, the exp2 argument); a relative error e of every weight moves the result
by at most 2 e A, A = sum p |v| / sum p; the exponential adds 2^-15, the
rounding of p to the type u, the sums N 2^-23, f16 weights under 2^-14 an
absolute 2^-25 each (against a row sum of at least 1), and the result
u |result|."""
import math

import numpy as np
import pytest

from tests.gpu_common import need_cuda, orc, torch

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def u(dtype):
    return torch.finfo(dtype).eps / 2


def _ok():
    assert jb.op_sync_status() == 0


def _randn(seed, *shape, dtype=torch.float16, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * by).to(dtype).cuda()


# ================================================================= rotation
def ref_turn(x, pos, plan):
    """x f64 [B, N, h, d] turned by integer positions pos [axes, B, N]."""
    n_pairs = plan.rot_dim // 2
    axis = [a for a, n in enumerate(plan.sections) for _ in range(n)]
    ang = torch.stack([pos[a].double() * w for a, w in zip(axis, plan.inv_freq)], -1).to(x.device)[:, :, None]
    c, s = torch.cos(ang) * plan.factor, torch.sin(ang) * plan.factor
    out = x.clone()
    i0 = torch.arange(n_pairs) if plan.layout == "half" else 2 * torch.arange(n_pairs)
    i1 = i0 + n_pairs if plan.layout == "half" else i0 + 1
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i0] * s + x[..., i1] * c
    size = torch.zeros_like(x)
    size[..., i0] = size[..., i1] = plan.factor * (x[..., i0].abs() + x[..., i1].abs())
    return out, size


def assert_turned(got, x, pos, plan, extra=0.0):
    want, size = ref_turn(x, pos, plan)
    err = (got.double() - want).abs()
    tol = u(got.dtype) * want.abs() + 2.0 ** -21 * size + extra
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"worst {((err - tol).max()).item():.3e} over"
    rest = slice(plan.rot_dim, None)
    if not torch.is_tensor(extra) and extra == 0.0:
        assert torch.equal(got[..., rest].double(), x[..., rest])


def _positions(axes, B, N, start, batched, dtype):
    n = torch.arange(N) + start
    if axes == 1:
        pos = n
        full = pos.expand(1, B, N)
        if batched:
            pos = pos + 1000 * torch.arange(B)[:, None]
            full = pos[None]
    else:
        pos = torch.stack([n // 35 + start, n // 5 % 7, n % 5])
        full = pos[:, None].expand(3, B, N)
        if batched:
            pos = pos[:, None] + torch.arange(B)[:, None]
            full = pos
    return pos.to(dtype).cuda(), full.to(torch.int64)


ROPE_CASES = [
    # dtype, B, N, h, d, rot, layout, sections, scaling, start
    ("bf16", 1, 1, 1, 64, 64, "half", None, None, 0),
    ("f16", 2, 37, 16, 64, 60, "interleaved", (10, 10, 10), None, 0),
    ("bf16", 1, 131, 5, 128, 64, "half", None, {"type": "yarn", "factor": 8.0, "original": 4096}, 70001),
    ("f32", 3, 33, 12, 32, 20, "half", None, {"type": "ntk", "factor": 4.0}, 11),
    ("f16", 2, 9, 3, 80, 80, "half", None, {"type": "linear", "factor": 8.0}, 10 ** 6),
    ("f32", 1, 65, 2, 256, 256, "interleaved", None, None, -50),
    ("bf16", 1, 5, 2, 256, 130, "half", None, None, 3),
    ("f16", 1, 7, 3, 17, 6, "interleaved", (1, 1, 1), None, 2),
    ("f32", 2, 3, 1, 2, 2, "half", None, None, 123456789),
    ("bf16", 4, 50, 7, 96, 96, "interleaved", None, None, 0),
    ("f16", 1, 300, 33, 64, 2, "half", None, None, 0),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}x{c[4]}-{c[5]}{c[6]}")
@pytest.mark.parametrize("batched,ints", [(False, torch.int64), (True, torch.int32)])
def test_rope(case, batched, ints):
    need_cuda()
    dtype, B, N, h, d, rot, layout, sections, scaling, start = case
    plan = jb.rope_plan(rot, layout=layout, sections=sections, scaling=scaling)
    x = _randn(N + d, B, N, h, d, dtype=TYPES[dtype])
    pos, full = _positions(len(plan.sections), B, N, start, batched, ints)
    before = x.clone()
    got = jb.rope(x, pos, plan)
    _ok()
    assert torch.equal(x, before)
    assert_turned(got, x.double(), full, plan)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("how", ["slice", "heads_first", "batch_broadcast", "odd_offset", "odd_stride"])
def test_rope_strides(dtype, how):
    """Views of a fused projection, head-major tensors, a broadcast batch, and
    starts and strides that no wide load fits."""
    need_cuda()
    B, N, h, d = 2, 21, 4, 64
    dt = TYPES[dtype]
    if how == "slice":
        x = _randn(1, B, N, 3, h, d, dtype=dt)[:, :, 1]
    elif how == "heads_first":
        x = _randn(2, B, h, N, d, dtype=dt).transpose(1, 2)
    elif how == "batch_broadcast":
        x = _randn(3, 1, N, h, d, dtype=dt).expand(B, N, h, d)
    elif how == "odd_offset":
        x = _randn(4, B * N * h * d + 1, dtype=dt)[1:].view(B, N, h, d)
    else:
        x = _randn(5, B, N, h, d + 1, dtype=dt)[..., :d]
    plan = jb.rope_plan(48)
    pos, full = _positions(1, B, N, 5, False, torch.int64)
    got = jb.rope(x, pos, plan)
    _ok()
    assert_turned(got, x.double(), full, plan)
    out = torch.full((B, N, h, d + 3), 7.0, dtype=dt, device="cuda")     # an output with strides of its own
    jb.rope(x, pos, plan, out=out[..., 1:d + 1])
    _ok()
    assert torch.equal(out[..., 1:d + 1], got)
    assert (out[..., 0] == 7).all() and (out[..., d + 1:] == 7).all()


def test_rope_in_place_and_beside():
    """In place on q inside a fused buffer: k and v stay as they are."""
    need_cuda()
    qkv = _randn(6, 2, 40, 3, 4, 64, dtype=torch.bfloat16)
    before = qkv.clone()
    plan = jb.rope_plan(64, layout="interleaved")
    pos, full = _positions(1, 2, 40, 9, False, torch.int32)
    q = qkv[:, :, 0]
    assert jb.rope(q, pos, plan, out=q) is q
    _ok()
    assert_turned(q, before[:, :, 0].double(), full, plan)
    assert torch.equal(qkv[:, :, 1:], before[:, :, 1:])


def test_rope_matches_the_encoders_rotation():
    """The three-axis plan is the rotation that the encoder's QKV product
    applies, by its oracle."""
    need_cuda()
    slots, rows, cols = 3, 4, 5
    n = np.arange(slots * rows * cols)
    grid = np.stack([n // (rows * cols), n // cols % rows, n % cols])
    x = _randn(7, 1, len(n), 2, 64, dtype=torch.float32)
    plan = jb.rope_plan(60, layout="interleaved", sections=(10, 10, 10))
    got = jb.rope(x, torch.from_numpy(grid).cuda(), plan)
    _ok()
    want = orc.rope(x[0].double().cpu().numpy().transpose(1, 0, 2), grid.T.astype(np.float64))
    err = np.abs(got[0].double().cpu().numpy().transpose(1, 0, 2) - want)
    assert err.max() <= 2.0 ** -20 * np.abs(want).max() * 2


def test_rope_values_that_are_not_finite_stay_in_their_pairs():
    need_cuda()
    x = _randn(8, 1, 4, 2, 64, dtype=torch.float16)
    x[0, 1, 0, 3] = float("nan")
    x[0, 2, 1, 63] = float("inf")
    plan = jb.rope_plan(60, layout="interleaved")
    got = jb.rope(x, torch.arange(4).cuda(), plan)
    _ok()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[0, 1, 0, 2:4] = True
    want[0, 2, 1, 63] = True
    assert torch.equal(bad, want)


def test_rope_empty():
    need_cuda()
    plan = jb.rope_plan(64)
    for shape in ((0, 4, 2, 64), (2, 0, 2, 64), (2, 4, 0, 64)):
        x = torch.empty(shape, dtype=torch.float16, device="cuda")
        assert jb.rope(x, torch.arange(shape[1]).cuda(), plan).shape == shape
    _ok()


# ==================================================================== norms
def ref_norm(x, w, b, kind, eps):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    std = ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    y = (x - mean) / std * w.double()
    size = x.abs().amax(-1, keepdim=True) / std * w.double().abs() + (x - mean).abs() / std * w.double().abs()
    if b is not None:
        y, size = y + b.double(), size + b.double().abs()
    return y, 2.0 ** -18 * size


def _norm_tolerance(extra, plan):
    """The norm's error through the rotation: each output takes in both of its
    pair's."""
    if plan is None:
        return extra
    n = plan.rot_dim // 2
    i0 = torch.arange(n) if plan.layout == "half" else 2 * torch.arange(n)
    i1 = i0 + n if plan.layout == "half" else i0 + 1
    out = extra.clone()
    out[..., i0] = out[..., i1] = plan.factor * (extra[..., i0] + extra[..., i1])
    return out


NORM_CASES = [
    # dtype, B, N, hq, hk, d, rot, layout, sections, norm, bias, per head
    ("bf16", 3, 1, 16, 4, 128, 128, "half", None, "rms", False, False),
    ("f16", 2, 45, 4, 4, 64, 60, "interleaved", (10, 10, 10), "layer", True, False),
    ("f32", 1, 33, 12, 12, 32, 20, "half", None, "rms", True, True),
    ("bf16", 1, 70, 8, 1, 80, 40, "half", None, "layer", False, True),
    ("f16", 2, 5, 3, 6, 256, 64, "interleaved", None, "rms", False, False),
    ("f32", 2, 17, 1, 2, 96, 0, "half", None, "layer", True, False),
    ("f16", 1, 3, 2, 1, 7, 4, "half", None, "rms", False, False),
    ("bf16", 1, 9, 5, 0, 64, 64, "half", None, "rms", False, False),
    ("f16", 1, 9, 0, 2, 64, 64, "half", None, "rms", False, False),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}+{c[4]}x{c[5]}-{c[6]}-{c[9]}")
def test_qk_norm_rope(case):
    need_cuda()
    dtype, B, N, hq, hk, d, rot, layout, sections, norm, bias, per_head = case
    dt = TYPES[dtype]
    qkv = _randn(d + N, B, N, (hq + 2 * hk) * d, dtype=dt, by=2.0)
    q, k = qkv[..., :hq * d].unflatten(-1, (hq, d)), qkv[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    plan = jb.rope_plan(rot, layout=layout, sections=sections) if rot else None
    pos, full = _positions(len(plan.sections), B, N, 77, True, torch.int64) if rot else (None, None)
    par = [_randn(50 + i, *((n, d) if per_head else (d,)), dtype=torch.float32, by=0.3) + (1 if i < 2 else 0)
           for i, n in enumerate((hq, hk, hq, hk))]
    qb, kb = (par[2], par[3]) if bias else (None, None)
    before = qkv.clone()
    got = jb.qk_norm_rope(q, k, pos, plan, par[0], par[1], q_bias=qb, k_bias=kb, norm=norm, eps=1e-5)
    _ok()
    assert torch.equal(qkv, before)
    for g, x, w, b in ((got[0], q, par[0], qb), (got[1], k, par[1], kb)):
        if not g.numel():
            continue
        y, extra = ref_norm(x.double(), w, b, norm, 1e-5)
        if plan is None:
            assert ((g.double() - y).abs() <= u(dt) * y.abs() + extra).all()
        else:
            assert_turned(g, y, full, plan, _norm_tolerance(extra, plan))
    # in place, and into the rows of a cache
    cache = torch.zeros(B, N + 3, hk, d, dtype=dt, device="cuda")
    jb.qk_norm_rope(q, k, pos, plan, par[0], par[1], q_bias=qb, k_bias=kb, norm=norm, eps=1e-5, q_out=q,
                    k_out=cache[:, 2:N + 2])
    _ok()
    assert torch.equal(q, got[0]) and torch.equal(cache[:, 2:N + 2], got[1])
    assert not cache[:, :2].any() and not cache[:, N + 2:].any()
    assert torch.equal(qkv[..., hq * d:], before[..., hq * d:])


def test_qk_norm_rope_extreme_rows():
    """A row of zeros (eps alone under the root), one large common offset
    (LayerNorm's centred squares), and a head with an infinity: its row is not
    finite, the others are as without it."""
    need_cuda()
    q = _randn(9, 1, 4, 2, 64, dtype=torch.float32)
    q[0, 0, 0] = 0
    q[0, 1, 0] += 1000.0
    k = q.clone()
    w = torch.ones(64, device="cuda")
    clean, _ = jb.qk_norm_rope(q, k, None, None, w, w, norm="layer", eps=1e-6)
    y, extra = ref_norm(q.double(), w, None, "layer", 1e-6)
    assert ((clean.double() - y).abs() <= u(torch.float32) * y.abs() + extra).all()
    assert not clean[0, 0, 0].any()
    q[0, 2, 1, 5] = float("inf")
    got, _ = jb.qk_norm_rope(q, k, None, None, w, w, norm="layer", eps=1e-6)
    _ok()
    bad = ~torch.isfinite(got).all(-1)
    assert bad[0, 2, 1] and bad.sum() == 1
    keep = ~bad
    assert torch.equal(got[keep], clean[keep])


# ================================================================ attention
def ref_attention(q, k, v, scale, cap=0.0, slopes=None, allowed=None, pos=None):
    """f64 result [B, Nq, hq, d] and the error bound; allowed bool [B, Nq, Nk],
    pos int64 [B, Nq]."""
    dt = q.dtype
    B, Nq, hq, d = q.shape
    Nk, g = k.shape[1], hq // k.shape[2]
    q, k, v = q.double(), k.double().repeat_interleave(g, 2), v.double().repeat_interleave(g, 2)
    seen = allowed.any(1)                                                  # keys some row reads
    k = torch.where(seen[:, :, None, None], k, 0.0)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * scale
    ds = torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs()) * abs(scale) * (d + 4) * 2.0 ** -23
    if cap:
        s = cap * torch.tanh(s / cap)
        ds = ds + cap * 2.0 ** -21
    if slopes is not None:
        far = (pos[:, :, None] - torch.arange(Nk, device=q.device)).abs().double()
        bias = slopes.double()[:, None, None] * far[:, None]
        s, ds = s - bias, ds + bias * 2.0 ** -22
    ds = ds + s.abs() * 2.0 ** -22
    ok = allowed[:, None]
    s = torch.where(ok, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.where(ok, torch.exp(s - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = torch.einsum("bhij,bjhd->bihd", p, v)
    size = torch.einsum("bhij,bjhd->bihd", p, v.abs())
    worst = torch.where(ok, ds, 0.0).amax(-1).transpose(1, 2)[..., None]   # [B, Nq, hq, 1]
    tol = size * (2 * (worst + 2.0 ** -15 + u(dt)) + Nk * 2.0 ** -23) + u(dt) * out.abs()
    if dt == torch.float16:
        tol = tol + 2.0 ** -25 * (allowed.sum(-1)[:, :, None, None] * v.abs().amax() + 1)
    return out, tol


def allow(B, Nq, Nk, causal=False, prefix=None, docs=None, kv_len=None, q_start=None):
    """(allowed [B, Nq, Nk], positions [B, Nq], written [B, Nq]) element by
    element from the definition."""
    a = np.zeros((B, Nq, Nk), bool)
    pos = np.zeros((B, Nq), np.int64)
    written = np.ones((B, Nq), bool)
    j = np.arange(Nk)
    for b in range(B):
        for i in range(Nq):
            if docs is not None:
                pos[b, i] = i
                t = [t for t in range(len(docs[b]) - 1) if docs[b][t] <= i < docs[b][t + 1]]
                written[b, i] = bool(t)
                if t:
                    lo, hi = docs[b][t[0]], docs[b][t[0] + 1]
                    ok = (j >= lo) & (j < hi)
                    if causal:
                        ok &= (j <= i) | (j < lo + (prefix[b][t[0]] if prefix is not None else 0))
                    a[b, i] = ok
                continue
            pos[b, i] = (Nk - Nq if q_start is None else q_start[b]) + i
            ok = j < (Nk if kv_len is None else kv_len[b])
            if causal:
                ok = ok & ((j <= pos[b, i]) | (j < (prefix[b] if prefix is not None else 0)))
            a[b, i] = ok
    return torch.from_numpy(a).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(written).cuda()


def _ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _qkv(seed, B, Nq, Nk, hq, hk, d, dtype, by=1.0):
    return (_randn(seed, B, Nq, hq, d, dtype=dtype, by=by), _randn(seed + 1, B, Nk, hk, d, dtype=dtype),
            _randn(seed + 2, B, Nk, hk, d, dtype=dtype))


def check_attention(q, k, v, scale=None, cap=0.0, slopes=None, mask=None, out=None, **call):
    mask = {} if mask is None else mask
    B, Nq, hq, d = q.shape
    Nk = k.shape[1]
    got = jb.masked_attention(q, k, v, scale=scale, cap=cap, slopes=slopes, causal=mask.get("causal", False),
                              prefix=_ints(mask.get("prefix")), doc_offsets=_ints(mask.get("docs")),
                              kv_len=_ints(mask.get("kv_len")), q_start=_ints(mask.get("q_start")), out=out, **call)
    _ok()
    allowed, pos, written = allow(B, Nq, Nk, **mask)
    want, tol = ref_attention(q, k, v, 1 / math.sqrt(d) if scale is None else scale, cap, slopes, allowed, pos)
    err = (got.double() - want).abs()
    rows = written[:, :, None, None].expand_as(err)
    assert torch.isfinite(got[rows]).all()
    assert (err[rows] <= tol[rows]).all(), f"worst {(err / tol)[rows].max().item():.3f} of the bound"
    return got, written


LENGTHS = [(1, 1), (1, 2), (5, 5), (64, 64), (127, 127), (128, 128), (129, 129), (257, 257), (300, 300), (1, 300),
           (3, 1000), (8, 513), (16, 70), (17, 260), (40, 333), (130, 7), (600, 200)]


@pytest.mark.parametrize("Nq,Nk", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d,hq,hk", [("f16", 64, 3, 3), ("bf16", 128, 4, 2)])
def test_attention_lengths(Nq, Nk, causal, dtype, d, hq, hk):
    """From one token to several tiles, odd sizes, more queries than keys
    (causal: the first queries then read nothing)."""
    need_cuda()
    q, k, v = _qkv(Nq + Nk, 2, Nq, Nk, hq, hk, d, TYPES[dtype])
    got, _ = check_attention(q, k, v, mask=dict(causal=causal))
    if causal and Nq > Nk:
        assert not got[:, :Nq - Nk].any()


@pytest.mark.parametrize("Nq", [1, 40])
def test_attention_without_keys(Nq):
    need_cuda()
    q = _randn(15, 2, Nq, 4, 64)
    none = torch.empty(2, 0, 2, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 3.0)
    assert jb.masked_attention(q, none, none, out=out) is out and not out.any()
    assert not jb.masked_attention(q, none, none, causal=True, cap=5.0).any()
    _ok()


@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 72, 80, 96, 104, 120])
@pytest.mark.parametrize("Nq,Nk", [(150, 150), (1, 300)])
def test_attention_head_dims(d, Nq, Nk):
    need_cuda()
    for dtype in (torch.float16, torch.bfloat16):
        q, k, v = _qkv(d, 2, Nq, Nk, 4, 2, d, dtype)
        check_attention(q, k, v, mask=dict(causal=Nq == 1))


@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 1), (8, 2), (12, 4), (32, 2)])
@pytest.mark.parametrize("Nq,Nk", [(140, 140), (1, 200), (4, 200)])
def test_attention_shared_key_heads(hq, hk, Nq, Nk):
    need_cuda()
    q, k, v = _qkv(hq, 1, Nq, Nk, hq, hk, 64, torch.bfloat16)
    check_attention(q, k, v, mask=dict(causal=True))


SHAPES = [(2, 1, 300), (2, 5, 270), (2, 260, 260)]


@pytest.mark.parametrize("B,Nq,Nk", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("cap,by,scale", [(30.0, 1.0, None), (5.0, 8.0, None), (50.0, 3.0, 0.5), (0.5, 4.0, None)])
def test_attention_cap(B, Nq, Nk, dtype, cap, by, scale):
    """Scores far under the cap, and most of them at it."""
    need_cuda()
    for d in (64, 128):
        q, k, v = _qkv(3, B, Nq, Nk, 4, 4, d, dtype, by=by)
        check_attention(q, k, v, scale=scale, cap=cap, mask=dict(causal=True))


@pytest.mark.parametrize("B,Nq,Nk", SHAPES)
@pytest.mark.parametrize("causal,cap", [(False, 0.0), (True, 0.0), (True, 20.0)])
def test_attention_distance_bias(B, Nq, Nk, causal, cap):
    need_cuda()
    for d in (64, 128):
        q, k, v = _qkv(4, B, Nq, Nk, 4, 2, d, torch.float16)
        slopes = torch.tensor([0.5, 0.03, 0.0, -0.01], device="cuda")
        check_attention(q, k, v, cap=cap, slopes=slopes, mask=dict(causal=causal))


@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_prefix(dtype, d):
    need_cuda()
    q, k, v = _qkv(5, 4, 300, 300, 2, 1, d, dtype)
    check_attention(q, k, v, mask=dict(causal=True, prefix=[0, 1, 129, 300]))
    check_attention(q, k, v, mask=dict(causal=True, prefix=[200, 5000, -3, 60], kv_len=[150, 300, 40, 61],
                                       q_start=[0, 0, 0, 0]))
    q1 = q[:, :2]
    check_attention(q1, k, v, mask=dict(causal=True, prefix=[200, 0, 3, 60], q_start=[100, 4, 298, 0]))


@pytest.mark.parametrize("Nq,Nk", [(1, 400), (4, 400), (200, 400), (400, 400)])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_lengths_per_clip(Nq, Nk, dtype, d):
    """Ragged clips, an empty one, one token, a length past the buffer; the
    rest of the cache holds NaN and infinities."""
    need_cuda()
    lens = [400, 0, 1, 129, 64, 9999]
    q, k, v = _qkv(6, 6, Nq, Nk, 4, 2, d, dtype)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
        v[b, n:, :, ::2] = float("nan")
    got, _ = check_attention(q, k, v, mask=dict(kv_len=lens))
    assert not got[1].any()
    start = [min(n, Nk) - Nq for n in lens]
    check_attention(q, k, v, mask=dict(kv_len=lens, q_start=start, causal=True), cap=20.0,
                    slopes=torch.tensor([0.1, 0.2, 0.0, 0.05], device="cuda"))


DOCS = [[0, 130, 130, 131, 200, 290], [0, 0, 0, 0, 5, 300], [10, 20, 40, 256, 257, 299], [0, 300, 300, 300, 300, 300]]


@pytest.mark.parametrize("causal,prefix", [(False, None), (True, None),
                                           (True, [[60, 3, 1, 0, 500], [0, 0, 0, 2, 100], [1, 2, 3, 4, 5], [299, 0, 0, 0, 0]])])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_documents(causal, prefix, dtype, d):
    """Documents of unequal lengths, empty ones, boundaries inside and at tile
    edges; rows outside every document are left as they were."""
    need_cuda()
    q, k, v = _qkv(7, 4, 300, 300, 4, 2, d, dtype)
    mask = dict(causal=causal, prefix=prefix, docs=DOCS)
    got, written = check_attention(q, k, v, mask=mask, cap=15.0, slopes=torch.tensor([0.1, 0.0, 0.5, 0.01], device="cuda"))
    assert not got[~written].any()
    out = torch.full_like(q, 3.0)
    kept, _ = check_attention(q, k, v, mask=mask, cap=15.0, slopes=torch.tensor([0.1, 0.0, 0.5, 0.01], device="cuda"), out=out)
    assert kept is out and (out[~written] == 3.0).all() and torch.equal(out[written], got[written])


@pytest.mark.parametrize("N", [1, 7, 31, 33, 60])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_documents_of_few_tokens(N, dtype, d):
    """Packed rows short enough for the few-query kernel, with rows outside
    every document."""
    need_cuda()
    q, k, v = _qkv(16, 2, N, N, 4, 2, d, dtype)
    docs = [[0, N // 3, N // 3, N - N // 4], [N // 5, N // 2, N // 2, N]]
    for mask in (dict(docs=docs), dict(docs=docs, causal=True), dict(docs=docs, causal=True, prefix=[[2, 0, 3], [1, 0, 99]])):
        out = torch.full_like(q, 3.0)
        _, written = check_attention(q, k, v, mask=mask, cap=9.0, out=out)
        assert (out[~written] == 3.0).all()


def test_attention_many_short_documents():
    need_cuda()
    rng = np.random.default_rng(1)
    cuts = np.sort(rng.choice(np.arange(1, 1000), 199, replace=False))
    q, k, v = _qkv(8, 1, 1000, 1000, 2, 2, 64, torch.float16)
    check_attention(q, k, v, mask=dict(docs=[[0] + cuts.tolist() + [1000]], causal=True))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_masked_values_never_arrive(value, dtype, d):
    """One token's key and value are not finite: the rows that may not read it
    are as if it were zero, in the tile that holds it too."""
    need_cuda()
    for Nq, Nk, bad, mask in ((300, 300, 140, dict(causal=True)), (300, 300, 140, dict(docs=[[0, 141, 300]])),
                              (4, 300, 298, dict(causal=True)), (300, 300, 299, dict(causal=True))):
        q, k, v = _qkv(9, 1, Nq, Nk, 2, 2, d, dtype)
        k[0, bad], v[0, bad] = 0, 0
        call = dict(causal=mask.get("causal", False), doc_offsets=_ints(mask.get("docs")))
        clean = jb.masked_attention(q, k, v, **call)
        v[0, bad] = value
        only_v = jb.masked_attention(q, k, v, **call)
        k[0, bad] = value
        both = jb.masked_attention(q, k, v, **call)
        _ok()
        allowed, _, _ = allow(1, Nq, Nk, **mask)
        free = ~allowed[0, :, bad]
        assert free.any() and (~free).any()
        want, tol = ref_attention(q, torch.where(torch.isfinite(k), k, 0), torch.where(torch.isfinite(v), v, 0),
                                  1 / math.sqrt(d), allowed=allow(1, Nq, Nk, **mask)[0])
        for got in (clean, only_v, both):
            assert ((got.double() - want).abs() <= tol)[0, free].all()
        assert not torch.isfinite(only_v[0, ~free]).all(-1).any()


def test_attention_values_that_are_read_arrive():
    """A score of NaN makes its row NaN; large finite scores do not overflow."""
    need_cuda()
    for Nq in (1, 200):
        q, k, v = _qkv(10, 1, Nq, 200, 1, 1, 64, torch.bfloat16)
        k[0, 150, 0, 3] = float("nan")
        got = jb.masked_attention(q, k, v)
        assert torch.isnan(got).all()
        capped = jb.masked_attention(q, k, v, cap=10.0)
        assert torch.isnan(capped).all()
        q, k, v = _qkv(11, 1, Nq, 200, 1, 1, 64, torch.bfloat16)
        check_attention(q * 300, k * 300, v)
        check_attention(q * 300, k * 300, v, cap=30.0)
        _ok()


@pytest.mark.parametrize("Nq", [2, 200])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_attention_scores_of_minus_infinity(Nq, dtype, d):
    """A row whose every allowed score is -inf is 0 / 0; one score of -inf
    beside finite ones counts nothing."""
    need_cuda()
    q, k, v = _qkv(12, 1, Nq, 200, 1, 1, d, dtype)
    q = q.abs() + 0.5
    k[0, :, 0] = 0
    k[0, 100:, 0, 0] = -float("inf")
    got = jb.masked_attention(q, k, v, kv_len=_ints([150]))
    want, tol = ref_attention(q, torch.where(torch.isfinite(k), k, 0), v, 1 / math.sqrt(d),
                              allowed=allow(1, Nq, 200, kv_len=[100])[0])
    assert ((got.double() - want).abs() <= tol).all()
    k[0, :, 0, 0] = -float("inf")
    assert torch.isnan(jb.masked_attention(q, k, v, kv_len=_ints([150]))).all()
    _ok()


@pytest.mark.parametrize("causal,docs", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 96)])
def test_attention_more_work_than_the_device_holds(causal, docs, dtype, d):
    """More pieces of work than SMs, of unequal lengths: every one is done,
    once, whichever CTA takes it."""
    need_cuda()
    B, N, h = 5, 700, 16
    q, k, v = _qkv(13, B, N, N, h, h, d, dtype)
    rng = np.random.default_rng(2)
    off = [[0] + sorted(rng.choice(np.arange(1, N), 5, replace=False).tolist()) + [N] for _ in range(B)]
    mask = dict(causal=causal) | (dict(docs=off) if docs else {})
    got, _ = check_attention(q, k, v, mask=mask)
    call = dict(causal=causal, doc_offsets=_ints(off) if docs else None)
    for _ in range(5):
        out = torch.full_like(q, float("nan"))
        assert torch.equal(jb.masked_attention(q, k, v, out=out, **call), got)
    _ok()


def test_attention_wait_bound():
    """A bound of 0 makes the first wait that is not over give up: the call
    unwinds, the status says so, and the next call works."""
    need_cuda()
    q, k, v = _qkv(14, 3, 600, 600, 32, 32, 64, torch.float16)
    want = jb.masked_attention(q, k, v)
    _ok()
    jb.op_set_timeout_ns(0)
    jb.masked_attention(q, k, v)
    st = jb.op_sync_status()
    jb.op_set_timeout_ns(4_000_000_000)
    assert st == jb._abi.ERR_TIMEOUT
    _ok()
    assert torch.equal(jb.masked_attention(q, k, v), want)
    _ok()


FIRST_CALL = """
import torch
import jepa_video_encoder_b200 as jb
q = torch.ones(2, {Nq}, 4, 64, dtype=torch.float16, device="cuda")
k = torch.ones(2, 900, 4, 64, dtype=torch.float16, device="cuda")
plan = jb.rope_plan(64)
pos = torch.arange({Nq}, device="cuda")
w = torch.ones(64, device="cuda")
out = torch.zeros_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a, b = jb.qk_norm_rope(q, jb.rope(q, pos, plan), pos, plan, w, w)
    jb.masked_attention(a, k, k, causal=True, out=out)
g.replay()
torch.cuda.synchronize()
assert jb.op_sync_status() == 0
assert (out == 1).all(), out
"""


@pytest.mark.parametrize("Nq", [1, 900])
def test_first_call_of_a_process_captured(Nq):
    """Nothing needs a warm-up call outside the capture."""
    need_cuda()
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(Nq=Nq)], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("Nq,Nk", [(200, 200), (2, 200)])
@pytest.mark.parametrize("how", ["fused", "heads_first", "broadcast_batch", "broadcast_head", "padded_rows", "reversed_layout"])
def test_attention_strides(Nq, Nk, how):
    need_cuda()
    B, h, d, dt = 2, 4, 64, torch.float16
    if how == "fused":
        qkv = _randn(1, B, Nk, 3, h, d, dtype=dt)
        q, k, v = qkv[:, :Nq, 0], qkv[:, :, 1], qkv[:, :, 2]
    elif how == "heads_first":
        q, k, v = (_randn(i, B, h, n, d, dtype=dt).transpose(1, 2) for i, n in ((2, Nq), (3, Nk), (4, Nk)))
    elif how == "broadcast_batch":
        q = _randn(5, B, Nq, h, d, dtype=dt)
        k, v = (_randn(i, 1, Nk, h, d, dtype=dt).expand(B, Nk, h, d) for i in (6, 7))
    elif how == "broadcast_head":
        q = _randn(8, B, Nq, h, d, dtype=dt)
        k, v = (_randn(i, B, Nk, 1, d, dtype=dt).expand(B, Nk, h, d) for i in (9, 10))
    elif how == "padded_rows":
        q, k, v = (_randn(i, B, n, h, d + 24, dtype=dt)[..., 8:d + 8] for i, n in ((11, Nq), (12, Nk), (13, Nk)))
    else:
        q, k, v = (_randn(i, h, n, B, d, dtype=dt).permute(2, 1, 0, 3) for i, n in ((14, Nq), (15, Nk), (16, Nk)))
    got, _ = check_attention(q, k, v, mask=dict(causal=True))
    out = torch.full((B, h, Nq, d + 8), 5.0, dtype=dt, device="cuda")
    view = out[..., :d].transpose(1, 2)
    jb.masked_attention(q, k, v, causal=True, out=view)
    _ok()
    assert torch.equal(view, got) and (out[..., d:] == 5).all()


def test_attention_offsets_past_32_bits():
    """A cache whose clips lie 2^31 elements apart."""
    need_cuda()
    B, Nk, h, d = 2, 130, 2, 64
    far = 1 << 31
    buf = torch.empty(far + Nk * h * d, dtype=torch.float16, device="cuda")
    k = buf.as_strided((B, Nk, h, d), (far, h * d, d, 1))
    k.copy_(_randn(20, B, Nk, h, d))
    v = _randn(21, B, Nk, h, d)
    for Nq in (1, 130):
        check_attention(_randn(22, B, Nq, h, d), k, v)
        check_attention(_randn(22, B, Nq, h, d), v, k)
    del buf, k


@pytest.mark.parametrize("Nq,Nk", [(1, 700), (300, 300)])
def test_attention_is_repeatable_and_capturable(Nq, Nk):
    """The same bits from a second call, from a graph's replays on new values,
    and from two graphs in flight on two streams."""
    need_cuda()
    sets = [_qkv(30 + i, 2, Nq, Nk, 4, 2, 64, torch.bfloat16) for i in range(2)]
    want = [jb.masked_attention(*s, causal=True) for s in sets]
    assert torch.equal(want[0], jb.masked_attention(*sets[0], causal=True))
    graphs = []
    for i in range(2):
        ins = [t.clone() for t in sets[i]]
        out = torch.empty_like(ins[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            jb.masked_attention(*ins, causal=True, out=out)
        graphs.append((g, ins, out, torch.cuda.Stream()))
    for turn in range(3):
        for i, (g, ins, out, st) in enumerate(graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                for t, s in zip(ins, sets[(i + turn) % 2]):
                    t.copy_(s)
                g.replay()
        torch.cuda.synchronize()
        for i, (_, _, out, _) in enumerate(graphs):
            assert torch.equal(out, want[(i + turn) % 2])
    _ok()


def test_operators_on_a_stream_that_is_given():
    need_cuda()
    st = torch.cuda.Stream()
    q, k, v = _qkv(40, 1, 150, 150, 2, 2, 64, torch.float16)
    plan = jb.rope_plan(64)
    pos = torch.arange(150).cuda()
    w = torch.ones(64, device="cuda")
    want = jb.masked_attention(*jb.qk_norm_rope(q, jb.rope(k, pos, plan), pos, plan, w, w), v)
    st.wait_stream(torch.cuda.current_stream())
    a = jb.rope(k, pos, plan, stream=st)
    b = jb.qk_norm_rope(q, a, pos, plan, w, w, stream=st)
    c = jb.masked_attention(*b, v, stream=st)
    d = jb.masked_attention(q, k, v, doc_offsets=_ints([[0, 70, 140]]), stream=st)
    st.synchronize()
    assert torch.equal(c, want) and not d[:, 140:].any()
    assert jb.op_sync_status(st) == 0


def test_refusals_on_the_device():
    need_cuda()
    q, k, v = _qkv(50, 1, 8, 8, 2, 2, 64, torch.float16)
    with pytest.raises(ValueError, match="overlaps"):
        jb.masked_attention(q, k, v, out=q)
    with pytest.raises(ValueError, match="forward only"):
        jb.masked_attention(q.clone().requires_grad_(), k, v)
    with torch.no_grad():
        jb.masked_attention(q.clone().requires_grad_(), k, v)
    for bad in (dict(kv_len=torch.zeros(1, device="cuda")), dict(kv_len=_ints([1, 2])), dict(q_start=torch.zeros(1, dtype=torch.int32)),
                dict(doc_offsets=_ints([0, 8])), dict(doc_offsets=_ints([[0, 8]]), kv_len=_ints([8])),
                dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(1, 2, device="cuda")),
                dict(slopes=torch.zeros(2, dtype=torch.float16, device="cuda")), dict(causal=True, prefix=_ints([[1]])),
                dict(out=torch.empty(1, 8, 2, 32, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            jb.masked_attention(q, k, v, **bad)
    plan = jb.rope_plan(64)
    pos = torch.arange(8).cuda()
    for bad in (lambda: jb.rope(q, pos.cpu(), plan), lambda: jb.rope(q[..., :32], pos, plan), lambda: jb.rope(q, pos[:7], plan),
                lambda: jb.rope(q.double(), pos, plan), lambda: jb.rope(q[:, 1:], pos[1:], plan, out=q[:, :-1]),
                lambda: jb.qk_norm_rope(q, k.float(), pos, plan, v, v), lambda: jb.qk_norm_rope(q, k, None, plan, q, k)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        jb.qk_norm_rope(q, k, pos, plan, w.half(), w)
    with pytest.raises(ValueError):
        jb.qk_norm_rope(q, k, pos, None, w, w)
    with pytest.raises(ValueError, match="overlaps"):
        jb.qk_norm_rope(q, k, pos, plan, w, w, q_out=k)
    _ok()


# ============================================================ all of a block
@pytest.mark.parametrize("step", [False, True])
def test_block_of_operators(step):
    """QKV projection, norms with rotation, attention, output projection, as a
    block runs them; a prompt, then single tokens over the cache it left.
    Each stage is checked against f64 of that stage's own inputs."""
    need_cuda()
    B, N, h, d, D = 2, 150, 4, 64, 256
    x = _randn(60, B * N, D)
    Wq, Wo = _randn(61, 3 * D, D, by=0.06), _randn(62, D, D, by=0.06)
    w = [_randn(63 + i, d, dtype=torch.float32, by=0.1) + 1 for i in range(2)]
    plan = jb.rope_plan(d, layout="half")
    qkv = torch.empty(B * N, 3 * D, dtype=torch.float16, device="cuda")
    jb.linear(x, Wq, jb.synth.DT_F16, 3 * D, None, jb._abi.EPI_F16, qkv)
    q, k, v = qkv.view(B, N, 3, h, d).unbind(2)
    cache_k = torch.full((B, N + 10, h, d), float("nan"), dtype=torch.float16, device="cuda")
    cache_v = cache_k.clone()
    cache_v[:, :N] = v
    pos = torch.arange(N).cuda()
    qn, _ = jb.qk_norm_rope(q, k, pos, plan, *w, k_out=cache_k[:, :N])
    if not step:
        att, _ = check_attention(qn, cache_k, cache_v, mask=dict(causal=True, kv_len=[N] * B, q_start=[0] * B))
    else:
        for t in range(N - 3, N):   # the same tokens again, one at a time
            qt, kt = jb.qk_norm_rope(q[:, t:t + 1], k[:, t:t + 1], pos[t:t + 1], plan, *w)
            assert torch.equal(qt, qn[:, t:t + 1]) and torch.equal(kt, cache_k[:, t:t + 1])
            check_attention(qt, cache_k, cache_v, mask=dict(causal=True, kv_len=[t + 1] * B, q_start=[t] * B))
        att = jb.masked_attention(qn, cache_k, cache_v, causal=True, kv_len=_ints([N] * B), q_start=_ints([0] * B))
    y, extra = ref_norm(q.double(), w[0], None, "rms", 1e-6)
    assert_turned(qn, y, torch.arange(N).expand(1, B, N), plan, _norm_tolerance(extra, plan))
    out = torch.empty(B * N, D, dtype=torch.float32, device="cuda")
    jb.linear(att.reshape(B * N, D), Wo, jb.synth.DT_F16, D, None, jb._abi.EPI_F32, out)
    _ok()
    a, o = att.reshape(B * N, D).double(), Wo.double()
    assert ((out.double() - a @ o.T).abs() <= D * 2.0 ** -22 * (a.abs() @ o.abs().T) + 1e-30).all()
