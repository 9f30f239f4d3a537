"""Score caps from far under the scores to far over them: cap * tanh(s / cap)
loses nothing to the cap's size, so that a huge cap is no cap.

Bound, with u = eps / 2 of the output's type: a score's dot product is off by
(d + 4) 2^-23 of scale * sum |q k|; its capped value, relative to itself, by
the polynomial of tanh(z) / z (5.9e-7 with 6 terms; 6.9e-6 with 5, bf16) and
five roundings of 2^-24, under 2^-20 (2^-17), or beyond |z| = 1 by the
exponent's rounding, z 2^-23 of a term that is at most e^-2z, under 2^-20 too;
by 2^-22 in the exponent's argument.  A score's error e moves the result by at
most 2 e A, A = sum p |v| / sum p; the exponential adds 2^-15, the rounding of p
to the type u, the sums N 2^-23; f16 weights under 2^-14 an absolute 2^-25 each;
the result u |result|."""
import math

import pytest

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _ok, _qkv, u

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu


def _reference(q, k, v, scale, cap):
    dt, d = q.dtype, q.shape[3]
    g = q.shape[2] // k.shape[2]
    q, k, v = q.double(), k.double().repeat_interleave(g, 2), v.double().repeat_interleave(g, 2)
    s = cap * torch.tanh(torch.einsum("bihd,bjhd->bhij", q, k) * (scale / cap))
    ds = torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs()) * scale * (d + 4) * 2.0 ** -23
    ds = ds + s.abs() * ((2.0 ** -17 if dt == torch.bfloat16 else 2.0 ** -20) + 2.0 ** -22)
    p = torch.softmax(s, -1)
    out = torch.einsum("bhij,bjhd->bihd", p, v)
    size = torch.einsum("bhij,bjhd->bihd", p, v.abs())
    worst = ds.amax(-1).transpose(1, 2)[..., None]
    tol = size * (2 * (worst + 2.0 ** -15 + u(dt)) + k.shape[1] * 2.0 ** -23) + u(dt) * out.abs()
    return out, tol + (2.0 ** -25 * (k.shape[1] * v.abs().amax() + 1) if dt == torch.float16 else 0.0)


@pytest.mark.parametrize("Nq", [1, 5, 200])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("cap", [2.0, 30.0, 600.0, 1e3, 1e5, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("by,scale", [(3.0, None), (8.0, 0.01), (2.0, 3.0)])
def test_cap_of_any_size(Nq, dtype, cap, by, scale):
    need_cuda()
    for d in (64, 128):
        q, k, v = _qkv(110 + d, 2, Nq, 300, 4, 2, d, dtype, by=by)
        real = 1 / math.sqrt(d) if scale is None else scale
        got = jb.masked_attention(q, k, v, scale=scale, cap=cap)
        _ok()
        want, tol = _reference(q, k, v, real, cap)
        err = (got.double() - want).abs()
        assert torch.isfinite(got).all()
        worst = (err / tol).max().item()
        assert worst <= 1, worst


@pytest.mark.parametrize("Nq", [1, 200])
@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("cap", [5.0, 1e6])
def test_cap_with_scales_that_are_not_positive(Nq, scale, cap):
    """Scale 0 averages the values; a negative one turns the order round."""
    need_cuda()
    for dtype in (torch.float16, torch.bfloat16):
        q, k, v = _qkv(120, 1, Nq, 300, 2, 2, 64, dtype, by=2.0)
        got = jb.masked_attention(q, k, v, scale=scale, cap=cap)
        _ok()
        want, tol = _reference(-q, k, v, -scale, cap)
        assert ((got.double() - want).abs() <= tol).all()
