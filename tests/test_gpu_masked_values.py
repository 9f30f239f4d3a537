"""Attention under masks: what a row may not read, or what a row gives no
weight, does not reach it, however large.  The comparisons are bit for bit
with the same call on zeros in those places: a weight of zero times a finite
value is zero, so nothing may differ."""
import math

import pytest

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _ints, _ok, _qkv, allow

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


def _slopes(on):
    return torch.tensor([0.1, 0.0, -0.02, 0.5], device="cuda") if on else None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("slopes,cap", [(False, 0.0), (True, 0.0), (False, 20.0), (True, 20.0)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_finite_values_at_masked_keys(dtype, d, slopes, cap, sign):
    """Every key from the 141st on holds the type's largest value (or its
    negative): the rows that read none of them, in the tiles that do hold
    them too, are as with zeros."""
    need_cuda()
    first, N = 141, 300
    for mask in (dict(causal=True), dict(docs=[[0, first, N]]), dict(docs=[[0, first, N]], causal=True, prefix=[[50, 9]]),
                 dict(causal=True, prefix=[60])):
        q, k, v = _qkv(70 + d, 1, N, N, 4, 2, d, dtype)
        call = dict(causal=mask.get("causal", False), prefix=_ints(mask.get("prefix")), doc_offsets=_ints(mask.get("docs")),
                    slopes=_slopes(slopes), cap=cap)
        v[:, first:] = 0
        want = jb.masked_attention(q, k, v, **call)
        v[:, first:] = sign * torch.finfo(dtype).max
        got = jb.masked_attention(q, k, v, **call)
        _ok()
        free = ~allow(1, N, N, **mask)[0][0, :, first:].any(-1)
        assert free.sum() == first
        same = torch.equal(got[0, free], want[0, free])
        assert same


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slopes", [False, True])
def test_largest_finite_values_at_scores_far_below(dtype, d, slopes):
    """Keys that a row does read, 500 below its other scores: e^-500 of the
    type's largest value is nothing, in tiles that no mask cuts too."""
    need_cuda()
    N = 384
    q, k, v = _qkv(90 + d, 1, N, N, 4, 2, d, dtype)
    q[..., 0] = 8.0
    low = torch.arange(N, device="cuda") % 3 == 1
    k[..., 0] = torch.where(low, -80.0 * math.sqrt(d), 0.0).to(dtype)[None, :, None]   # scores of -640 beside ones within some 20 of 0
    v[:, low] = 0
    want = jb.masked_attention(q, k, v, slopes=_slopes(slopes))
    v[:, low] = torch.finfo(dtype).max
    got = jb.masked_attention(q, k, v, slopes=_slopes(slopes))
    _ok()
    same = torch.equal(got, want)
    assert same
