"""Projections whose heads hold q, k and v in turn: [B, N, heads, 3, d]."""
import pytest

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _ok, _randn

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 128), (torch.float32, 32), (torch.float16, 24)])
@pytest.mark.parametrize("B,N", [(2, 37), (3, 1), (1, 1)])
def test_in_place_on_interleaved_heads(dtype, d, B, N):
    """q and k turned and normalised where they lie give what copies give, and
    v stays as it was."""
    need_cuda()
    x = _randn(d + N, B, N, 4, 3, d, dtype=dtype)
    before = x.clone()
    q, k, v = x.unbind(3)
    plan, pos = jb.rope_plan(d), torch.arange(N, device="cuda") + 5
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    want = jb.qk_norm_rope(q.contiguous(), k.contiguous(), pos, plan, w, w)
    got = jb.qk_norm_rope(q, k, pos, plan, w, w, q_out=q, k_out=k)
    _ok()
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, before[..., 2, :])
    turned = jb.rope(before[..., 0, :].contiguous(), pos, plan)
    x.copy_(before)
    jb.rope(q, pos, plan, out=q)
    _ok()
    assert torch.equal(q, turned) and torch.equal(x[..., 1:, :], before[..., 1:, :])
    if dtype != torch.float32:
        out = jb.masked_attention(q, k, v, causal=True)
        into = torch.zeros(B, N, 4, 2, d, dtype=dtype, device="cuda")
        jb.masked_attention(q, k, v, causal=True, out=into[..., 1, :])
        _ok()
        assert torch.equal(into[..., 1, :], out) and not into[..., 0, :].any()
