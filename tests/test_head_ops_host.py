"""The per-head operators on the CPU: rotary frequencies and their 64-bit
turn fractions, the argument structures, and every refusal of the binding and
of the C entry points (invalid arguments are rejected before any device
work, so no GPU is needed)."""
import copy
import ctypes
import dataclasses
import math
import pathlib
import pickle
import random
import subprocess

import pytest
import torch
import torch.autograd.forward_ad as fwAD

import jepa_video_encoder_b200 as jb
from jepa_video_encoder_b200 import _abi, build, heads

STRUCTS = {"jepa_b200_rope_args": _abi.RopeArgs, "jepa_b200_qk_norm_rope_args": _abi.QkNormRopeArgs,
           "jepa_b200_masked_attention_args": _abi.MaskedAttentionArgs, "jepa_b200_heads": _abi.Heads,
           "jepa_b200_rope": _abi.Rope}


def _cpu(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


# ------------------------------------------------------------- frequencies
def test_frequencies_of_one_axis():
    freq, axis, factor = heads.rope_frequencies(8)
    assert freq == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15) and axis == (0,) * 4 and factor == 1.0


def test_frequencies_of_three_axes_are_the_encoders():
    freq, axis, _ = heads.rope_frequencies(60, sections=(10, 10, 10))
    assert axis == (0,) * 10 + (1,) * 10 + (2,) * 10
    for a in range(3):
        assert freq[10 * a:10 * a + 10] == pytest.approx([10000.0 ** (-2 * i / 20) for i in range(10)], rel=1e-15)


def test_scalings():
    plain, _, _ = heads.rope_frequencies(64)
    linear, _, f = heads.rope_frequencies(64, scaling={"type": "linear", "factor": 4.0})
    assert linear == pytest.approx([w / 4 for w in plain], rel=1e-15) and f == 1.0
    ntk, _, f = heads.rope_frequencies(64, scaling={"type": "ntk", "factor": 4.0})
    assert ntk[0] == plain[0] and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-12) and f == 1.0
    yarn, _, f = heads.rope_frequencies(64, scaling={"type": "yarn", "factor": 4.0, "original": 4096})
    assert f == pytest.approx(1 + 0.1 * math.log(4))
    for w, y in zip(plain, yarn):
        turns = 4096 * w / (2 * math.pi)
        if turns >= 32:
            assert y == w
        elif turns <= 1:
            assert y == pytest.approx(w / 4, rel=1e-15)
        else:
            assert w / 4 < y < w
    assert heads.rope_frequencies(64, scaling={"type": "yarn", "factor": 4.0, "original": 4096, "magnitude": 1.0})[2] == 1.0


@pytest.mark.parametrize("kw", [
    dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, sections=(2, 1)), dict(rot_dim=8, sections=(1, 1, 1, 1)),
    dict(rot_dim=8, sections=(4, 0)), dict(rot_dim=8, base=0.0), dict(rot_dim=8, scaling={"type": "other"}),
    dict(rot_dim=8, scaling={"type": "linear", "factor": 0.0}), dict(rot_dim=8, scaling={"type": "linear", "slow": 1}),
    dict(rot_dim=2, scaling={"type": "ntk", "factor": 2.0}), dict(rot_dim=8, scaling={"type": "yarn", "factor": 2.0}),
    dict(rot_dim=8, scaling={"type": "yarn", "factor": 2.0, "original": 64, "fast": 1.0, "slow": 2.0})])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        heads.rope_frequencies(**kw)


@pytest.mark.parametrize("pos", [0, 1, -1, 70001, 10 ** 6, -(10 ** 6), 2 ** 31 - 1])
def test_turn_fractions_hold_far_positions(pos):
    """position * turns mod 2^64 against the angle in exact rational terms:
    the word is off by at most half a unit of 2^-64 of a turn and by the
    rounding of w / 2 pi in f64 (2 * 2^-53 of the fraction w / 2 pi <= 1/6)."""
    from fractions import Fraction
    freq, _, _ = heads.rope_frequencies(64)
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for w, word in zip(freq, heads.rope_turns(freq)):
        got = Fraction((pos * word) % 2 ** 64, 2 ** 64)
        want = (Fraction(w) * pos / two_pi) % 1
        diff = abs(got - want)
        diff = min(diff, 1 - diff)
        assert diff <= abs(pos) * (Fraction(1, 2 ** 65) + Fraction(w) / two_pi * Fraction(2, 2 ** 53))


# ------------------------------------------------------- argument structures
def test_structures_match_the_header(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "jepa_b200.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", f"{build.ROOT}/include", str(src), "-o", str(exe)], check=True)
    said = dict(x.rsplit(" ", 1) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for name, cls in STRUCTS.items():
        assert int(said[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(said[f"{name}.{f}"]) == getattr(cls, f).offset


@pytest.mark.parametrize("cls", [_abi.RopeArgs, _abi.QkNormRopeArgs, _abi.MaskedAttentionArgs])
def test_packed_bytes_are_the_structure(cls):
    """Values 1, 2, 3, ... in order of the fields land in those fields."""
    pack = _abi.packer(cls)

    def leaves(c):
        for name, typ in c._fields_:
            if issubclass(typ, ctypes.Structure):
                yield from ((name,) + x for x in leaves(typ))
            else:
                yield (name,)

    names = list(leaves(cls))
    got = cls.from_buffer_copy(pack.pack(*range(1, len(names) + 1)))
    for i, path in enumerate(names):
        v = got
        for f in path:
            v = getattr(v, f)
        assert v == i + 1, path


# ------------------------------------------------------ refusals in Python
def test_host_tensors_and_shapes_are_refused():
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        jb.masked_attention(_cpu(1, 4, 2, 64), _cpu(1, 4, 2, 64), _cpu(1, 4, 2, 64))
    for bad in (_cpu(4, 2, 64), _cpu(1, 4, 64, 2).transpose(2, 3), "x"):
        with pytest.raises((ValueError, TypeError)):
            heads.check_heads(bad, "x")
    with pytest.raises(ValueError, match="multiples of 8"):
        heads.check_heads(_cpu(1, 4, 2, 68)[..., :64], "x", granule=8)
    with pytest.raises(ValueError, match="start at"):
        heads.check_heads(_cpu(1, 4, 2, 72)[..., 1:65], "x", granule=8)
    heads.check_heads(_cpu(1, 1, 1, 68)[..., :64], "x", granule=8)        # no axis steps by 68
    heads.check_heads(_cpu(2, 4, 2, 64)[:, :, :1], "x", torch.float16, (2, 4, 1, 64), 8)


@pytest.mark.parametrize("kw,match", [
    (dict(q=_cpu(1, 4, 2, 64, dtype=torch.float32)), "float16 or bfloat16"),
    (dict(k=_cpu(1, 4, 2, 64, dtype=torch.bfloat16)), "must be"),
    (dict(v=_cpu(1, 5, 2, 64)), "must be"),
    (dict(k=_cpu(2, 4, 2, 64), v=_cpu(2, 4, 2, 64)), "like q"),
    (dict(k=_cpu(1, 4, 3, 64), v=_cpu(1, 4, 3, 64)), "multiple of k's"),
    (dict(q=_cpu(1, 4, 2, 136), k=_cpu(1, 4, 2, 136), v=_cpu(1, 4, 2, 136)), "head_dim"),
    (dict(scale=float("inf")), "scale"), (dict(cap=-1.0), "cap"), (dict(cap=float("nan")), "cap"),
    (dict(prefix=torch.zeros(1, dtype=torch.int32)), "needs causal")])
def test_masked_attention_refuses(kw, match):
    args = dict(q=_cpu(1, 4, 2, 64), k=_cpu(1, 4, 2, 64), v=_cpu(1, 4, 2, 64)) | kw
    with pytest.raises(ValueError, match=match):
        jb.masked_attention(args.pop("q"), args.pop("k"), args.pop("v"), **args)


def test_positions():
    i = torch.arange(6)
    assert heads.check_positions(i, 1, 2, 6) == (1, 0, 0)
    assert heads.check_positions(i.int().expand(2, 6), 1, 2, 6) == (0, 0, 0)
    assert heads.check_positions(torch.zeros(2, 6, dtype=torch.int32), 1, 2, 6) == (0, 0, 6)
    assert heads.check_positions(torch.zeros(3, 6, dtype=torch.int32), 3, 2, 6) == (0, 6, 0)
    assert heads.check_positions(torch.zeros(3, 2, 6, dtype=torch.int64), 3, 2, 6) == (1, 12, 6)
    for bad, axes in ((i.float(), 1), (i, 3), (torch.zeros(2, 6, dtype=torch.int64), 3), (torch.zeros(6, 2).long().t(), 1),
                      (torch.zeros(5).long(), 1), (torch.zeros(12).long()[::2], 1)):
        with pytest.raises(ValueError):
            heads.check_positions(bad, axes, 2, 6)
    with pytest.raises(TypeError):
        heads.check_positions([0, 1], 1, 2, 6)


def test_outputs_that_overlap_are_refused():
    qkv = _cpu(2, 4, 6, 64)
    q, k = qkv[:, :, :2], qkv[:, :, 2:4]
    heads.check_output(q, "out", [(q, "q", True), (k, "k", False)])       # in place, beside k's columns
    heads.check_output(qkv[:, :1, :2], "out", [(qkv[:, :1, 2:4], "k", False)])   # one token a clip
    with pytest.raises(ValueError, match="overlaps"):
        heads.check_output(q, "out", [(q, "q", False)])
    with pytest.raises(ValueError, match="overlaps"):
        heads.check_output(qkv[:, :, 1:3], "out", [(q, "q", True)])
    with pytest.raises(ValueError, match="overlaps"):
        heads.check_output(qkv[:, 1:3, :2], "out", [(qkv[:, :2, :2], "q", True)])
    with pytest.raises(ValueError, match="share memory"):
        heads.check_output(_cpu(1, 4, 2, 64).expand(2, 4, 2, 64), "out", [])
    with pytest.raises(ValueError, match="share memory"):
        heads.check_output(_cpu(400).as_strided((1, 4, 2, 64), (0, 64, 32, 1)), "out", [])
    heads.check_output(_cpu(2, 2, 4, 64).transpose(1, 2), "out", [])


def test_views_that_interleave_are_told_apart():
    """Columns of any common step: heads of q, k and v in turn, with and
    without more tokens and clips; views that do meet are refused."""
    for B, N in ((2, 4), (1, 4), (2, 1), (1, 1)):
        x = _cpu(B, N, 3, 3, 64)          # [heads, q / k / v, head_dim]
        q, k, v = x.unbind(3)
        heads.check_output(q, "q_out", [(q, "q", True), (k, "k", False), (v, "v", False)])
        heads.check_output(v, "out", [(q, "q", False), (k, "k", False)])
        heads.check_output(x[..., 1, 32:], "out", [(x[..., 1, :32], "x", False)])    # halves of a head
        for a, b in ((x[..., 0, :], x[..., 0, :32]), (x[..., 0, 16:48], x[..., 0, :32])):
            with pytest.raises(ValueError, match="overlaps"):
                heads.check_output(a, "out", [(b, "x", False)])
    x = _cpu(2, 4, 6, 64)
    with pytest.raises(ValueError, match="overlaps"):
        heads.check_output(x[:, :, ::2], "out", [(x[:, :, 2:5], "x", False)])
    heads.check_output(x[:, :, ::2], "out", [(x[:, :, 1::2], "x", False)])
    flat = _cpu(4096)
    a, b = flat.as_strided((1, 4, 2, 8), (0, 24, 8, 1)), flat.as_strided((1, 4, 2, 8), (0, 32, 8, 1), 16)
    with pytest.raises(ValueError, match="overlaps"):     # other steps: b's second row lies in a's third
        heads.check_output(a, "out", [(b, "x", False)])


def test_apart_means_no_element_in_common():
    """The rule against the elements themselves, for strided views at random:
    never apart where one is shared."""
    rng, told = random.Random(3), 0
    flat = _cpu(1 << 14)
    for _ in range(3000):
        views = []
        row = rng.choice([8, 12, 24, 48])
        for _ in range(2):
            shape = [rng.choice([1, 2, 3]) for _ in range(3)] + [rng.choice([1, 4, 8])]
            strides = [rng.choice([0, row, 2 * row, 96, 5]) for _ in range(3)] + [1]
            views.append(flat.as_strided(shape, strides, rng.randrange(64)))
        idx = [set(torch.arange(1 << 14).as_strided(v.shape, v.stride(), v.storage_offset()).flatten().tolist()) for v in views]
        if heads._columns_apart(*views):
            told += 1
            assert not idx[0] & idx[1], [(v.shape, v.stride(), v.storage_offset()) for v in views]
    assert told > 50


# ------------------------------------------------------------- forward only
def test_tensors_that_autograd_follows_are_refused():
    """Reverse mode where it records, forward mode within its level; a plain
    tensor beside a dual one passes."""
    x = torch.zeros(2, 3)
    heads.check_forward_only(x, "x")
    with pytest.raises(ValueError, match="forward only"):
        heads.check_forward_only(x.clone().requires_grad_(), "x")
    with torch.no_grad():
        heads.check_forward_only(x.clone().requires_grad_(), "x")
    with fwAD.dual_level():
        dual = fwAD.make_dual(x.clone(), torch.ones(2, 3))
        heads.check_forward_only(x, "x")
        with pytest.raises(ValueError, match="tangent"):
            heads.check_forward_only(dual, "x")
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):   # which does not stop forward mode
            heads.check_forward_only(dual, "x")
    heads.check_forward_only(x, "x")


# --------------------------------------------------------- copies of a plan
def _own_addresses(plan):
    assert plan.addresses == (plan.turns.buffer_info()[0], plan.axis.buffer_info()[0])
    assert len(plan.turns) == len(plan.axis) == plan.rot_dim // 2


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p)), dataclasses.replace])
def test_a_copied_plan_holds_its_own_numbers(how):
    """The addresses that go to the library are those of the copy's arrays,
    not of the original's, which may be gone."""
    plan = jb.rope_plan(60, layout="interleaved", sections=(10, 10, 10), scaling={"type": "linear", "factor": 4.0})
    got = how(plan)
    _own_addresses(plan)
    _own_addresses(got)
    assert got == plan and list(got.turns) == list(plan.turns) and list(got.axis) == list(plan.axis)
    for name in ("rot_dim", "layout", "sections", "inv_freq", "factor"):
        assert getattr(got, name) == getattr(plan, name)


def test_a_module_with_a_plan_is_copied():
    m = torch.nn.Module()
    m.plan = jb.rope_plan(64)
    twin = copy.deepcopy(m)
    _own_addresses(twin.plan)
    assert twin.plan.turns is not m.plan.turns


def test_a_plan_whose_numbers_are_replaced():
    """The arrays follow the frequencies; what does not fit is refused."""
    plan = jb.rope_plan(8)
    slow = dataclasses.replace(plan, inv_freq=tuple(f / 2 for f in plan.inv_freq), factor=0.5)
    _own_addresses(slow)
    assert list(slow.turns) == heads.rope_turns(slow.inv_freq) and slow.factor == 0.5
    for bad in (dict(inv_freq=plan.inv_freq[:3]), dict(sections=(3,)), dict(sections=(1, 1, 1, 1)), dict(sections=(4, 0)),
                dict(rot_dim=10), dict(rot_dim=7), dict(rot_dim=258), dict(layout="other"), dict(inv_freq=(1.0, 0.1, 0.01, math.nan))):
        with pytest.raises(ValueError):
            dataclasses.replace(plan, **bad)


# ------------------------------------------------------- refusals of the ABI
@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load_library()


BUF = ctypes.create_string_buffer(4096)
AT = (ctypes.addressof(BUF) + 63) & ~63


def _h(at=AT, sb=512, sn=128, sh=64):
    return _abi.Heads(at, sb, sn, sh)


def _attn(**kw):
    a = _abi.MaskedAttentionArgs(q=_h(), k=_h(), v=_h(), out=_h(), dtype=1, B=1, Nq=4, Nk=4, heads_q=2, heads_kv=2,
                                 head_dim=64, scale=0.125)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), _abi.ERR_DTYPE), (dict(dtype=8), _abi.ERR_DTYPE),
    (dict(head_dim=60), _abi.ERR_SHAPE), (dict(head_dim=136), _abi.ERR_SHAPE), (dict(head_dim=0), _abi.ERR_SHAPE),
    (dict(heads_kv=0), _abi.ERR_SHAPE), (dict(heads_q=3, heads_kv=2), _abi.ERR_SHAPE),
    (dict(B=-1), _abi.ERR_SHAPE), (dict(Nq=-1), _abi.ERR_SHAPE), (dict(Nk=-4), _abi.ERR_SHAPE),
    (dict(cap=-1.0), _abi.ERR_ARG), (dict(cap=float("nan")), _abi.ERR_ARG), (dict(scale=float("nan")), _abi.ERR_ARG),
    (dict(causal=2), _abi.ERR_ARG), (dict(prefix=AT), _abi.ERR_ARG), (dict(n_docs=1), _abi.ERR_ARG),
    (dict(doc_offsets=AT), _abi.ERR_ARG), (dict(n_docs=1, doc_offsets=AT, kv_len=AT), _abi.ERR_ARG),
    (dict(n_docs=1, doc_offsets=AT, Nk=5), _abi.ERR_ARG), (dict(kv_len=AT + 2), _abi.ERR_ARG),
    (dict(q=_h(0)), _abi.ERR_ARG), (dict(k=_h(AT + 8)), _abi.ERR_ARG), (dict(v=_h(sn=100)), _abi.ERR_ARG),
    (dict(q=_h(sb=-8)), _abi.ERR_ARG), (dict(out=_h(sn=0)), _abi.ERR_ARG), (dict(out=_h(sh=8)), _abi.ERR_ARG)])
def test_masked_attention_entry_refuses(lib, kw, status):
    assert lib.jepa_b200_op_masked_attention(ctypes.byref(_attn(**kw)), None) == status


@pytest.mark.parametrize("kw", [dict(scale=math.inf), dict(scale=-math.inf), dict(cap=math.inf)])
def test_masked_attention_entry_refuses_infinities(lib, kw):
    """As the binding does: an infinite scale or cap times a score of zero has
    no value."""
    assert lib.jepa_b200_op_masked_attention(ctypes.byref(_attn(B=0, **kw)), None) == _abi.ERR_ARG


def test_masked_attention_entry_empty(lib):
    assert lib.jepa_b200_op_masked_attention(None, None) == _abi.ERR_ARG
    assert lib.jepa_b200_op_masked_attention(ctypes.byref(_attn(B=0)), None) == 0
    assert lib.jepa_b200_op_masked_attention(ctypes.byref(_attn(Nq=0)), None) == 0


def _rope(**kw):
    r = _abi.Rope(rot_dim=64, layout=0, n_axes=1, pos_i64=1, pos=AT, turns=AT, factor=1.0)
    a = _abi.RopeArgs(x=_h(), out=_h(), dtype=1, B=1, N=4, heads=2, head_dim=64, rope=r)
    for n, v in kw.items():
        if hasattr(a, n):
            setattr(a, n, v)
        else:
            setattr(a.rope, n, v)
    return a


ROPE_BAD = [(dict(dtype=2), _abi.ERR_DTYPE), (dict(head_dim=0), _abi.ERR_SHAPE), (dict(head_dim=257), _abi.ERR_SHAPE),
            (dict(B=-1), _abi.ERR_SHAPE), (dict(B=65536, N=65536), _abi.ERR_SHAPE), (dict(rot_dim=66), _abi.ERR_SHAPE),
            (dict(rot_dim=3), _abi.ERR_SHAPE), (dict(rot_dim=-2), _abi.ERR_SHAPE), (dict(n_axes=4), _abi.ERR_SHAPE),
            (dict(n_axes=0), _abi.ERR_SHAPE), (dict(n_axes=3), _abi.ERR_ARG), (dict(layout=2), _abi.ERR_ARG),
            (dict(pos=0), _abi.ERR_ARG), (dict(turns=0), _abi.ERR_ARG),
            (dict(pos=AT + 4), _abi.ERR_ARG), (dict(pos_i64=2), _abi.ERR_ARG), (dict(pos_stride_b=-1, B=2), _abi.ERR_ARG),
            (dict(x=_h(0)), _abi.ERR_ARG), (dict(x=_h(AT + 1)), _abi.ERR_ARG), (dict(out=_h(sn=8)), _abi.ERR_ARG)]


@pytest.mark.parametrize("kw,status", ROPE_BAD)
def test_rope_entry_refuses(lib, kw, status):
    assert lib.jepa_b200_op_rope(ctypes.byref(_rope(**kw)), None) == status


def test_rope_entry_empty(lib):
    assert lib.jepa_b200_op_rope(None, None) == _abi.ERR_ARG
    for kw in (dict(B=0), dict(N=0), dict(heads=0)):
        assert lib.jepa_b200_op_rope(ctypes.byref(_rope(**kw)), None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), _abi.ERR_DTYPE), (dict(norm=2), _abi.ERR_ARG), (dict(eps=-1.0), _abi.ERR_ARG),
    (dict(eps=float("nan")), _abi.ERR_ARG), (dict(q_weight=0), _abi.ERR_ARG), (dict(k_weight=AT + 2), _abi.ERR_ARG),
    (dict(q_bias=AT + 1), _abi.ERR_ARG), (dict(q_weight_stride_h=-64), _abi.ERR_ARG), (dict(head_dim=300), _abi.ERR_SHAPE),
    (dict(k=_h(0)), _abi.ERR_ARG), (dict(k_out=_h(sn=1)), _abi.ERR_ARG), (dict(B=0), 0), (dict(heads_q=0, heads_k=0), 0)])
def test_qk_norm_rope_entry_refuses(lib, kw, status):
    a = _abi.QkNormRopeArgs(q=_h(), k=_h(), q_out=_h(), k_out=_h(), dtype=1, B=1, N=4, heads_q=2, heads_k=2,
                            head_dim=64, eps=1e-6, q_weight=AT, k_weight=AT)
    for n, v in kw.items():
        setattr(a, n, v)
    assert lib.jepa_b200_op_qk_norm_rope(ctypes.byref(a), None) == status


# ------------------------------------------------------------ kernel sources
def test_cluster_barriers_are_met_by_whole_warps():
    """The aligned cluster barrier stands in one function alone, behind a
    barrier of the warp: lanes reach it from loops of unequal length."""
    csrc = pathlib.Path(build.CSRC)
    found = {p.name: p.read_text().count("barrier.cluster") for p in sorted(csrc.iterdir()) if p.suffix in (".cu", ".cuh")}
    assert {n: c for n, c in found.items() if c} == {"common.cuh": 2}
    body = (csrc / "common.cuh").read_text()
    body = body[body.index("void cluster_sync()"):]
    body = body[:body.index("}")]
    assert -1 < body.find("__syncwarp();") < body.find("barrier.cluster.arrive")
