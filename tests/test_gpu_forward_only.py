"""The per-head operators refuse operands whose tangents they would drop."""
import pytest
import torch.autograd.forward_ad as fwAD

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _ints, _qkv

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu


def _dual(t):
    return fwAD.make_dual(t, torch.ones_like(t))


def test_dual_tensors_are_refused():
    """In every place of a float operand; the same calls on plain tensors,
    within the level too, work."""
    need_cuda()
    q, k, v = _qkv(1, 1, 8, 8, 2, 2, 64, torch.float16)
    w, b, slopes = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"), torch.ones(2, device="cuda")
    plan, pos = jb.rope_plan(64), torch.arange(8).cuda()
    ops = {
        "rope": (lambda x, out: jb.rope(x, pos, plan, out=out), dict(x=q, out=torch.empty_like(q))),
        "norm": (lambda q, k, w, b, o: jb.qk_norm_rope(q, k, pos, plan, w, w, q_bias=b, k_bias=b, q_out=o),
                 dict(q=q, k=k, w=w, b=b, o=torch.empty_like(q))),
        "attention": (lambda q, k, v, slopes, out: jb.masked_attention(q, k, v, slopes=slopes, kv_len=_ints([8]), out=out),
                      dict(q=q, k=k, v=v, slopes=slopes, out=torch.empty_like(q))),
    }
    with fwAD.dual_level():
        for call, args in ops.values():
            call(**args)
            for name, t in args.items():
                with pytest.raises(ValueError, match="tangent"):
                    call(**(args | {name: _dual(t)}))
    assert jb.op_sync_status() == 0
