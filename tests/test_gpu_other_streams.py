"""Per-head operators on a stream that is given: operands that the caller
drops, whose memory other tensors want at once, keep their values until the
stream has read them."""
import pytest

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _ints, _ok, _qkv

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu

WAIT = 50_000_000   # clocks that the stream is busy with something else: some 30 ms


def _operands():
    q, k, v = _qkv(5, 2, 96, 96, 4, 2, 64, torch.float16)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    return dict(q=q, k=k, v=v, w=w, b=w * 0.25, pos=torch.arange(96, device="cuda") + 7,
                slopes=torch.tensor([0.1, 0.2, 0.0, 0.3], device="cuda"), kv_len=_ints([60, 96]), q_start=_ints([3, 0]),
                prefix=_ints([20, 5]))


CALLS = {
    "rope": lambda t, plan, **kw: [jb.rope(t["q"], t["pos"], plan, **kw)],
    "norm": lambda t, plan, **kw: list(jb.qk_norm_rope(t["q"], t["k"], t["pos"], plan, t["w"], t["w"], q_bias=t["b"],
                                                       k_bias=t["b"], norm="layer", **kw)),
    "attention": lambda t, plan, **kw: [jb.masked_attention(t["q"], t["k"], t["v"], slopes=t["slopes"], causal=True,
                                                            prefix=t["prefix"], kv_len=t["kv_len"], q_start=t["q_start"],
                                                            **kw)],
}


@pytest.mark.parametrize("name", CALLS)
def test_operands_dropped_after_the_call(name):
    need_cuda()
    plan, side = jb.rope_plan(64), torch.cuda.Stream()
    want = CALLS[name](_operands(), plan)
    _ok()
    ops = _operands()
    shapes = [(t.shape, t.dtype) for t in ops.values()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = CALLS[name](ops, plan, stream=side)
    del ops
    taken = [torch.zeros(s, dtype=t, device="cuda") for s, t in shapes for _ in range(4)]   # wants the same blocks
    torch.cuda.synchronize()
    assert jb.op_sync_status(side) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(taken) == 4 * len(shapes)


def test_two_streams_inside_a_capture():
    """A call on a stream that joined the capture, its operands made and
    dropped within it."""
    need_cuda()
    plan = jb.rope_plan(64)
    ops = _operands()
    want = CALLS["rope"](ops, plan)[0] * 2
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = ops["q"] * 2
        side.wait_stream(torch.cuda.current_stream())
        y = jb.rope(x, ops["pos"], plan, stream=side)
        del x
        z = torch.zeros_like(want)   # may not take x's memory
        torch.cuda.current_stream().wait_stream(side)
        out.copy_(y + z)
        del y
    for _ in range(2):
        out.zero_()
        g.replay()
        _ok()
        # doubling commutes with every rounding of the rotation but those under f16's normal range
        assert torch.allclose(out, want, rtol=0, atol=2.0 ** -23)
