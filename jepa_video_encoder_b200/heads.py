"""Per-head operators of a transformer block, between its QKV projection and
its output projection: rotary positions (rope), norms of queries and keys with
the rotation in the same pass (qk_norm_rope), and attention under masks
(masked_attention).

Operands are CUDA tensors [B, N, heads, head_dim] with a contiguous last axis,
views of one projection output or of a cache included.  The calls are
asynchronous on ``stream`` (default: the current stream), allocate nothing but
an output that was not given, keep nothing between calls, and can be captured
into CUDA graphs.  With a ``stream`` that is not the current one the operands
may be dropped as soon as the call returns: their memory is not given out
again before the stream has passed it.  Their contents must be ready on it
(stream.wait_stream), and an output that was not given belongs to it.

The operators are forward only: a tensor that requires grad is
refused while autograd records, and so is one that carries a tangent.
"""
from __future__ import annotations

import math
from array import array
from dataclasses import dataclass, field
from typing import Any, Optional, Sequence, Tuple

import torch
import torch.autograd.forward_ad as fwAD

from . import _abi
from ._abi import check, load_library

_ROPE = _abi.packer(_abi.RopeArgs)
_QK = _abi.packer(_abi.QkNormRopeArgs)
_ATTN = _abi.packer(_abi.MaskedAttentionArgs)
_LAYOUTS = {"half": _abi.ROPE_HALF, "interleaved": _abi.ROPE_INTERLEAVED}
_NORMS = {"rms": _abi.NORM_RMS, "layer": _abi.NORM_LAYER}
_NO_ROPE = (0, 0, 0, 0, 0, 0, 0, 0, 0, 0.0)
# the current stream's address without a Stream object, which costs more than
# the rest of a call's checks together
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: _abi.BF16}


# ---------------------------------------------------------------- operands
def check_forward_only(t, name: str) -> None:
    """Refuse a tensor that autograd follows in reverse mode (while it
    records) or in forward mode (a tangent of the current level)."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: the per-head operators are forward only (call them under "
                         "torch.no_grad() or on detached tensors)")
    if fwAD._current_level >= 0 and fwAD.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} has a tangent: the per-head operators do not carry one on (call them on its primal)")


def _check_cuda(t, name: str, device: int) -> None:
    if t.get_device() != device:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    if t.requires_grad or fwAD._current_level >= 0:
        check_forward_only(t, name)


def check_heads(t, name: str, dtype=None, shape: Optional[Sequence[int]] = None, granule: int = 1):
    """Validate the layout of a [B, N, heads, head_dim] operand: four axes,
    the last one contiguous; ``dtype`` and ``shape`` where they are set by
    another operand; with ``granule`` g > 1 a data pointer and strides that
    are multiples of g elements.  Returns (shape, (address, strides of the
    first three axes))."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    have = t.shape
    if len(have) != 4:
        raise ValueError(f"{name} must be [B, N, heads, head_dim], got {list(have)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and have != shape and tuple(have) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(have)}")
    sb, sn, sh, one = t.stride()
    if one != 1 and have[3] > 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    at = t.data_ptr()
    if granule > 1:
        if at % (granule * t.element_size()):
            raise ValueError(f"{name} must start at a multiple of {granule * t.element_size()} bytes")
        if (sb | sn | sh) % granule:
            for n, s in zip(have, (sb, sn, sh)):
                if n > 1 and s % granule:
                    raise ValueError(f"{name}'s strides must be multiples of {granule} elements, got {t.stride()}")
            sb, sn, sh = (s if n > 1 else 0 for n, s in zip(have, (sb, sn, sh)))  # an axis of one has no stride
    return have, (at, sb, sn, sh)


def _span(t) -> int:
    """Elements from a view's first to behind its last."""
    return 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))


def check_output(out, name: str, inputs) -> None:
    """Validate an output that the caller gave: no two of its elements in one
    place, and no overlap with ``inputs``, a list of (tensor, name, may be the
    output itself).  Views whose ranges of memory interleave count as
    overlapping unless they lie in separate columns of a common step."""
    axes = sorted((s, n) for n, s in zip(out.shape, out.stride()) if n > 1)
    reach = 1
    for s, n in axes:
        if s < reach:
            raise ValueError(f"{name} has elements that share memory (strides {out.stride()})")
        reach = s * (n - 1) + reach
    for t, what, same_ok in inputs:
        if t is None or not t.numel() or not out.numel():
            continue
        if out.untyped_storage().data_ptr() != t.untyped_storage().data_ptr():
            continue
        if same_ok and out.data_ptr() == t.data_ptr() and out.dtype == t.dtype and \
                all(a == b for n, a, b in zip(out.shape, out.stride(), t.stride()) if n > 1):
            continue
        o0, t0 = out.data_ptr(), t.data_ptr()
        o1, t1 = o0 + _span(out) * out.element_size(), t0 + _span(t) * t.element_size()
        if o1 <= t0 or t1 <= o0:
            continue
        if not _columns_apart(out, t):
            raise ValueError(f"{name} overlaps {what}")


def _columns_apart(a, b) -> bool:
    """Whether two views lie in separate columns of some common step: a stride
    of one of them by which every larger stride of both is a whole number of
    steps, as with slices of one projection output (the step of a token) and
    with the heads of q, k and v in turn (the step of a head)."""
    size = a.element_size()
    if a.dtype != b.dtype or (b.data_ptr() - a.data_ptr()) % size:
        return False
    axes = [[(n, s) for n, s in zip(x.shape, x.stride()) if n > 1] for x in (a, b)]
    for step in {s for x in axes for _, s in x if s > 1}:
        inside = [[(n, s) for n, s in x if s % step] for x in axes]
        if any(s > step for x in inside for _, s in x):
            continue
        wide = [1 + sum((n - 1) * s for n, s in x) for x in inside]
        off = (b.data_ptr() - a.data_ptr()) // size % step
        if wide[0] <= off and off + wide[1] <= step:
            return True
    return False


def _launch(t, stream):
    """(current device, raw stream) of a call on tensor t."""
    if not t.is_cuda:
        raise ValueError(f"expected CUDA tensors, got one on {t.device}")
    device = torch.cuda.current_device()
    if stream is None:
        return device, _raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, but the current device is cuda:{device}")
    return device, stream.cuda_stream


def _hold(device: int, raw: int, stream, tensors) -> None:
    """Tell the allocator that a stream other than the current one, whose
    memory they are, uses these tensors."""
    if raw != _raw_stream(device):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _new(like, shape, stream, zero: bool = False):
    """A contiguous output like an operand [B, N, h, d], owned by the stream
    that writes it, and its (address, strides)."""
    make = torch.zeros_like if zero else torch.empty_like
    if stream is None:
        out = make(like, memory_format=torch.contiguous_format)
    else:
        with torch.cuda.stream(stream):
            out = make(like, memory_format=torch.contiguous_format)
    _, N, h, d = shape
    return out, (out.data_ptr(), N * h * d, h * d, d)


# -------------------------------------------------------------- rotary plan
@dataclass(frozen=True)
class RopePlan:
    """Frequencies of a rotation (rope_plan makes it; a program keeps it; it
    serves every device).  Pairs of dims turn by position * inv_freq
    radians.  The arrays that go to the library are made from these numbers
    here, in every copy and unpickled plan anew, so that a plan passes the
    addresses of its own arrays."""
    rot_dim: int
    layout: str
    sections: Tuple[int, ...]
    inv_freq: Tuple[float, ...]   # radians per unit of position, one a pair
    factor: float                 # on cosine and sine
    turns: Any = field(init=False, repr=False, compare=False)   # uint64 [pairs]: inv_freq / 2 pi as binary fractions
    axis: Any = field(init=False, repr=False, compare=False)    # uint8 [pairs]
    addresses: Tuple[int, int] = field(init=False, repr=False, compare=False)   # of turns and axis

    def __post_init__(self):
        if self.layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {self.layout!r}")
        if not 2 <= self.rot_dim <= 256 or self.rot_dim % 2:
            raise ValueError(f"rot_dim must be even, at least 2 and at most 256, got {self.rot_dim}")
        if not 1 <= len(self.sections) <= 3 or min(self.sections) < 1 or sum(self.sections) != self.rot_dim // 2:
            raise ValueError(f"sections must be 1 to 3 positive counts of pairs that add up to {self.rot_dim // 2}, "
                             f"got {self.sections}")
        if len(self.inv_freq) != self.rot_dim // 2 or not all(math.isfinite(w) for w in self.inv_freq):
            raise ValueError(f"inv_freq must be {self.rot_dim // 2} finite numbers")
        turns = array("Q", rope_turns(self.inv_freq))
        axis = array("B", [a for a, n in enumerate(self.sections) for _ in range(n)])
        object.__setattr__(self, "turns", turns)
        object.__setattr__(self, "axis", axis)
        object.__setattr__(self, "addresses", (turns.buffer_info()[0], axis.buffer_info()[0]))

    def __reduce__(self):
        return RopePlan, (self.rot_dim, self.layout, self.sections, self.inv_freq, self.factor)


def rope_frequencies(rot_dim: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None,
                     scaling: Optional[dict] = None):
    """(inverse frequencies, axis of each pair, factor on cosine and sine).

    The pairs form one section per position axis (default: one section of
    rot_dim / 2).  Pair i of a section of n turns by base^(-i/n) radians per
    position.  ``scaling`` stretches that for long contexts, with "factor" f:
      {"type": "linear"}: every frequency / f;
      {"type": "ntk"}: base * f^(n/(n-1)), so that the slowest pair turns f
        times slower and the fastest as before;
      {"type": "yarn", "original": L, "fast": 32, "slow": 1, "magnitude": m}: a
        pair that makes r turns within the L positions of training keeps its
        frequency for r >= fast, has it divided by f for r <= slow, and is
        blended linearly in r between; cosine and sine are multiplied by m
        (default 1 + 0.1 ln f)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    sections = (rot_dim // 2,) if sections is None else tuple(int(n) for n in sections)
    if not 1 <= len(sections) <= 3 or min(sections) < 1 or sum(sections) != rot_dim // 2:
        raise ValueError(f"sections must be 1 to 3 positive counts of pairs that add up to {rot_dim // 2}, got {sections}")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError(f"base must be positive, got {base}")
    kind, f, factor = None, 1.0, 1.0
    if scaling is not None:
        kind, f = scaling.get("type"), float(scaling.get("factor", 1.0))
        known = {"linear": set(), "ntk": set(), "yarn": {"original", "fast", "slow", "magnitude"}}
        if kind not in known:
            raise ValueError(f"scaling type must be one of {sorted(known)}, got {kind!r}")
        if set(scaling) - known[kind] - {"type", "factor"}:
            raise ValueError(f"unknown keys in scaling: {sorted(set(scaling) - known[kind] - {'type', 'factor'})}")
        if not (f > 0 and math.isfinite(f)):
            raise ValueError(f"scaling factor must be positive, got {f}")
    freq, axis = [], []
    for a, n in enumerate(sections):
        b = base
        if kind == "ntk":
            if n < 2:
                raise ValueError("ntk scaling needs sections of two pairs or more")
            b = base * f ** (n / (n - 1))
        freq += [b ** (-i / n) for i in range(n)]
        axis += [a] * n
    if kind == "linear":
        freq = [w / f for w in freq]
    elif kind == "yarn":
        if "original" not in scaling:
            raise ValueError('yarn scaling needs "original", the positions of training')
        length, fast, slow = float(scaling["original"]), float(scaling.get("fast", 32.0)), float(scaling.get("slow", 1.0))
        if not (length > 0 and fast > slow >= 0):
            raise ValueError("yarn scaling needs original > 0 and fast > slow >= 0")
        keep = [min(1.0, max(0.0, (length * w / (2 * math.pi) - slow) / (fast - slow))) for w in freq]
        freq = [w * (g + (1 - g) / f) for w, g in zip(freq, keep)]
        factor = float(scaling.get("magnitude", 1.0 + 0.1 * math.log(f)))
    return tuple(freq), tuple(axis), factor


def rope_turns(inv_freq: Sequence[float]):
    """Radians per position as 64-bit words: the fraction of a turn per
    position times 2^64, rounded, modulo 2^64."""
    return [int(round(math.ldexp(math.fmod(w / (2 * math.pi), 1.0), 64))) % (1 << 64) for w in inv_freq]


def rope_plan(rot_dim: int, *, layout: str = "half", base: float = 10000.0, sections: Optional[Sequence[int]] = None,
              scaling: Optional[dict] = None) -> RopePlan:
    """Plan of a rotation of the first rot_dim dims of every head.

    layout "half": pair i is dims (i, i + rot_dim / 2); "interleaved": dims
    (2i, 2i + 1).  sections: pairs of each position axis (the encoder's own
    3-D rotation is rope_plan(60, layout="interleaved", sections=(10, 10,
    10))).  base, scaling: see rope_frequencies."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    if rot_dim > 256:
        raise ValueError(f"rot_dim must be at most 256, got {rot_dim}")
    freq, _, factor = rope_frequencies(rot_dim, base, sections, scaling)
    sections = (rot_dim // 2,) if sections is None else tuple(int(n) for n in sections)
    return RopePlan(rot_dim, layout, sections, freq, factor)


def check_positions(positions, n_axes: int, B: int, N: int) -> Tuple[int, int, int]:
    """Validate positions: int32 or int64, [N] or [B, N] for one axis, [axes,
    N] or [axes, B, N] for more, the token axis contiguous.  Returns (is
    int64, axis stride, batch stride)."""
    if not isinstance(positions, torch.Tensor):
        raise TypeError(f"positions must be a torch.Tensor, got {type(positions).__name__}")
    if positions.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"positions must be int32 or int64, got {positions.dtype}")
    shape = positions.shape
    lead = () if n_axes == 1 else (n_axes,)
    if shape == lead + (N,):
        batched = False
    elif shape == lead + (B, N):
        batched = True
    else:
        raise ValueError(f"positions must be {list(lead + (N,))} or {list(lead + (B, N))}, got {list(shape)}")
    if N > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return (1 if positions.dtype == torch.int64 else 0, positions.stride(0) if n_axes > 1 else 0,
            positions.stride(-2) if batched else 0)


def _rope_words(plan: RopePlan, positions, B: int, N: int, d: int, device: int):
    if not isinstance(plan, RopePlan):
        raise TypeError(f"plan must be a RopePlan, got {type(plan).__name__}")
    if plan.rot_dim > d:
        raise ValueError(f"the plan turns {plan.rot_dim} dims of heads that have {d}")
    axes = len(plan.sections)
    i64, stride_axis, stride_b = check_positions(positions, axes, B, N)
    _check_cuda(positions, "positions", device)
    return (plan.rot_dim, _LAYOUTS[plan.layout], axes, i64, positions.data_ptr(), stride_axis, stride_b,
            *plan.addresses, plan.factor)


def _float_type(t, name: str) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    return _DTYPES[t.dtype]


def rope(x, positions, plan: RopePlan, out=None, stream=None):
    """Rotary positions: x [B, N, heads, head_dim] float16, bfloat16 or
    float32, head_dim up to 256 -> a tensor like x.

    positions: integer tensor [N] (every clip the same) or [B, N], with
    several axes [axes, N] or [axes, B, N].  out: the tensor to write; x
    itself turns x in place."""
    shape, at_x = check_heads(x, "x")
    B, N, H, d = shape
    dtype = _float_type(x, "x")
    device, raw = _launch(x, stream)
    _check_cuda(x, "x", device)
    if not 1 <= d <= 256:
        raise ValueError(f"head_dim must be 1 to 256, got {d}")
    words = _rope_words(plan, positions, B, N, d, device)
    if out is None:
        out, at_out = _new(x, shape, stream)
    else:
        at_out = check_heads(out, "out", x.dtype, shape)[1]
        _check_cuda(out, "out", device)
        check_output(out, "out", [(x, "x", True), (positions, "positions", False)])
    if not (B and N and H):
        return out
    if stream is not None:
        _hold(device, raw, stream, (x, positions, out))
    check(load_library().jepa_b200_op_rope(_ROPE.pack(*at_x, *at_out, dtype, B, N, H, d, *words), raw), "rope")
    return out


def _weight(t, name: str, heads: int, d: int, device: int) -> Tuple[int, int]:
    """(address, elements from one head's values to the next's) of a float32
    vector [d] or table [heads, d]."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if (shape != (d,) and shape != (heads, d)) or (d > 1 and strides[-1] != 1):
        raise ValueError(f"{name} must be [{d}] or [{heads}, {d}] with a contiguous last axis, got {list(shape)}")
    if t.get_device() != device or t.requires_grad or fwAD._current_level >= 0:
        _check_cuda(t, name, device)
    return t.data_ptr(), strides[0] if len(shape) == 2 else 0


def qk_norm_rope(q, k, positions, plan: Optional[RopePlan], q_weight, k_weight, *, q_bias=None, k_bias=None,
                 norm: str = "rms", eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Norm of every head of q [B, N, hq, d] and k [B, N, hk, d], then the
    rotation, in one launch.  Returns (q_out, k_out), tensors like q and k.

    norm "rms": x / sqrt(mean(x^2) + eps) * weight (+ bias); "layer": (x -
    mean) / sqrt(var + eps) * weight (+ bias).  Weights and biases: float32
    [d], or [heads, d] of their own.  plan None (positions then None too):
    no rotation.  q_out, k_out: the tensors to write; q and k themselves for
    an update in place, or rows of a cache."""
    shape, at_q = check_heads(q, "q")
    dtype = _float_type(q, "q")
    k_shape, at_k = check_heads(k, "k", q.dtype)
    B, N, hq, d = shape
    hk = k_shape[2]
    if tuple(k_shape) != (B, N, hk, d):
        raise ValueError(f"k must be [{B}, {N}, heads, {d}] like q, got {list(k.shape)}")
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}, got {norm!r}")
    if not (eps >= 0):
        raise ValueError(f"eps must not be negative, got {eps}")
    if not 1 <= d <= 256:
        raise ValueError(f"head_dim must be 1 to 256, got {d}")
    device, raw = _launch(q, stream)
    _check_cuda(q, "q", device)
    _check_cuda(k, "k", device)
    if q_weight is None or k_weight is None:
        raise TypeError("q_weight and k_weight must be tensors")
    qw, qw_h = _weight(q_weight, "q_weight", hq, d, device)
    kw, kw_h = _weight(k_weight, "k_weight", hk, d, device)
    qb, qb_h = _weight(q_bias, "q_bias", hq, d, device)
    kb, kb_h = _weight(k_bias, "k_bias", hk, d, device)
    if plan is None:
        if positions is not None:
            raise ValueError("positions need a plan")
        words = _NO_ROPE
    else:
        words = _rope_words(plan, positions, B, N, d, device)
    def others():
        return [(positions, "positions", False), (q_weight, "q_weight", False), (k_weight, "k_weight", False),
                (q_bias, "q_bias", False), (k_bias, "k_bias", False)]

    if q_out is None:
        q_out, at_qo = _new(q, shape, stream)
    else:
        at_qo = check_heads(q_out, "q_out", q.dtype, shape)[1]
        _check_cuda(q_out, "q_out", device)
        check_output(q_out, "q_out", [(q, "q", True), (k, "k", False)] + others())
    if k_out is None:
        k_out, at_ko = _new(k, k_shape, stream)
    else:
        at_ko = check_heads(k_out, "k_out", q.dtype, k_shape)[1]
        _check_cuda(k_out, "k_out", device)
        check_output(k_out, "k_out", [(k, "k", True), (q, "q", False), (q_out, "q_out", False)] + others())
    if not (B and N and (hq or hk)):
        return q_out, k_out
    if stream is not None:
        _hold(device, raw, stream, (q, k, positions, q_weight, k_weight, q_bias, k_bias, q_out, k_out))
    check(load_library().jepa_b200_op_qk_norm_rope(
        _QK.pack(*at_q, *at_k, *at_qo, *at_ko, dtype, B, N, hq, hk, d, _NORMS[norm], eps, qw, qb, kw, kb, qw_h, qb_h,
                 kw_h, kb_h, *words), raw), "qk_norm_rope")
    return q_out, k_out


def _per_clip(t, name: str, shape, device: int) -> int:
    """Device address of an int32 tensor that a kernel indexes per clip."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)}, got {t.dtype} {list(t.shape)}")
    _check_cuda(t, name, device)
    return t.data_ptr()


def masked_attention(q, k, v, *, scale: Optional[float] = None, cap: Optional[float] = None, slopes=None,
                     causal: bool = False, prefix=None, doc_offsets=None, kv_len=None, q_start=None, out=None,
                     stream=None):
    """Attention of q [B, Nq, hq, d] over k, v [B, Nk, hk, d] (float16 or
    bfloat16, d a multiple of 8 up to 128, hq a multiple of hk: query head h
    reads key head h * hk // hq) -> [B, Nq, hq, d].

    Query row i of clip b stands at position p = q_start[b] + i among the
    keys (int32 [B]; default Nk - Nq: the queries are the last tokens).
      s = scale * q.k (default 1 / sqrt(d)); cap c: s = c * tanh(s / c);
      slopes float32 [hq]: s -= slopes[h] * |p - j| for key j;
      kv_len int32 [B]: only keys j < kv_len[b] (a padded batch, a cache);
      causal: only keys j <= p; prefix int32 [B]: or j < prefix[b];
      doc_offsets int32 [B, n + 1] (needs Nq = Nk, no kv_len or q_start): a
        row of n documents one after another, document t the tokens
        doc_offsets[b, t] .. doc_offsets[b, t + 1] - 1 (never decreasing;
        equal offsets make an empty one), each reading itself alone; prefix
        is then [B, n] and counts from each document's start.
    Rows that may read no key are zeros.  Rows outside every document are
    left as they are in ``out``, and are zeros where out is not given.  Keys
    and values that a row may not read do not reach it, whatever they hold."""
    shape, at_q = check_heads(q, "q", granule=8)
    dtype = _DTYPES.get(q.dtype, 0)
    if not dtype:
        raise ValueError(f"q must be float16 or bfloat16, got {q.dtype}")
    k_shape, at_k = check_heads(k, "k", q.dtype, granule=8)
    _, at_v = check_heads(v, "v", q.dtype, k_shape, granule=8)
    B, Nq, hq, d = shape
    Bk, Nk, hk, dk = k_shape
    if Bk != B or dk != d:
        raise ValueError(f"k must be [{B}, Nk, heads, {d}] like q, got {list(k_shape)}")
    if hq < 1 or hk < 1 or hq % hk:
        raise ValueError(f"q's heads must be a multiple of k's, got {hq} and {hk}")
    if not 8 <= d <= 128 or d % 8:
        raise ValueError(f"head_dim must be a multiple of 8 from 8 to 128, got {d}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    cap = 0.0 if cap is None else float(cap)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    if not (cap >= 0 and math.isfinite(cap)):
        raise ValueError(f"cap must be finite and not negative, got {cap}")
    if prefix is not None and not causal:
        raise ValueError("prefix needs causal")
    device, raw = _launch(q, stream)
    _check_cuda(q, "q", device)
    _check_cuda(k, "k", device)
    _check_cuda(v, "v", device)
    n_docs = 0
    if doc_offsets is not None:
        if kv_len is not None or q_start is not None:
            raise ValueError("doc_offsets exclude kv_len and q_start")
        if Nq != Nk:
            raise ValueError(f"doc_offsets need as many queries as keys, got {Nq} and {Nk}")
        if not isinstance(doc_offsets, torch.Tensor) or doc_offsets.dim() != 2 or doc_offsets.shape[1] < 2:
            raise ValueError("doc_offsets must be an int32 tensor [B, n + 1] with n >= 1")
        n_docs = doc_offsets.shape[1] - 1
    at_docs = _per_clip(doc_offsets, "doc_offsets", (B, n_docs + 1), device)
    at_prefix = _per_clip(prefix, "prefix", (B, n_docs) if n_docs else (B,), device)
    at_len = _per_clip(kv_len, "kv_len", (B,), device)
    at_start = _per_clip(q_start, "q_start", (B,), device)
    at_slopes = 0
    if slopes is not None:
        at_slopes, _ = _weight(slopes, "slopes", 1, hq, device)
        if slopes.dim() != 1:
            raise ValueError(f"slopes must be [{hq}], got {list(slopes.shape)}")
    if out is None:
        out, at_out = _new(q, shape, stream, zero=n_docs > 0)
    else:
        at_out = check_heads(out, "out", q.dtype, shape, granule=8)[1]
        _check_cuda(out, "out", device)
        check_output(out, "out", [(q, "q", False), (k, "k", False), (v, "v", False), (prefix, "prefix", False),
                                  (doc_offsets, "doc_offsets", False), (kv_len, "kv_len", False),
                                  (q_start, "q_start", False), (slopes, "slopes", False)])
    if not (B and Nq):
        return out
    if stream is not None:
        _hold(device, raw, stream, (q, k, v, slopes, prefix, doc_offsets, kv_len, q_start, out))
    check(load_library().jepa_b200_op_masked_attention(
        _ATTN.pack(*at_q, *at_k, *at_v, *at_out, dtype, B, Nq, Nk, hq, hk, d, scale, cap,
                   1 if causal else 0, n_docs, at_slopes, at_prefix, at_docs, at_len, at_start), raw),
        "masked_attention")
    return out
