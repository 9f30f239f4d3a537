"""The device status of the single-kernel calls."""
import pytest

from tests.gpu_common import need_cuda, torch
from tests.test_gpu_head_ops import _qkv, _randn

import jepa_video_encoder_b200 as jb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["linear", "attention"])
def test_status_is_cleared_of_every_call_at_once(first):
    """A GEMM and an attention call whose waits run out before one look at the
    status: it says so, and the next look, after work that succeeded, is
    clean."""
    need_cuda()
    a, w = _randn(1, 256, 1024), _randn(2, 512, 1024)
    out = torch.empty(256, 512, dtype=torch.float32, device="cuda")
    q, k, v = _qkv(3, 3, 600, 600, 32, 32, 64, torch.float16)

    def linear():
        jb.linear(a, w, jb.synth.DT_F16, 512, None, jb._abi.EPI_F32, out)

    def attention():
        return jb.masked_attention(q, k, v)

    want = attention()
    assert jb.op_sync_status() == 0
    jb.op_set_timeout_ns(0)
    try:
        for call in (linear, attention) if first == "linear" else (attention, linear):
            call()
        torch.cuda.synchronize()
    finally:
        jb.op_set_timeout_ns(4_000_000_000)
    assert jb.op_sync_status() == jb._abi.ERR_TIMEOUT
    linear()
    got = attention()
    assert jb.op_sync_status() == 0
    assert torch.equal(got, want)
    assert ((out.double() - a.double() @ w.double().T).abs() <= 1024 * 2.0 ** -22 * (a.double().abs() @ w.double().abs().T)).all()


def test_rows_computed_anew_do_not_run_out_of_time():
    """A value that is not finite sends the rows that read it through the
    definition, which takes longer than the wait bound set here; the CTAs that
    go on to another item wait for theirs meanwhile."""
    need_cuda()
    q, k, v = _qkv(9, 1, 2048, 2048, 40, 40, 64, torch.float16)
    v[0, 7] = float("inf")
    want = jb.masked_attention(q, k, v)
    assert jb.op_sync_status() == 0
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    jb.op_set_timeout_ns(2_000_000)
    try:
        start.record()
        got = jb.masked_attention(q, k, v)
        end.record()
        status = jb.op_sync_status()
    finally:
        jb.op_set_timeout_ns(4_000_000_000)
    assert status == 0
    assert start.elapsed_time(end) > 2
    assert torch.equal(got, want) and not torch.isfinite(got).any()
