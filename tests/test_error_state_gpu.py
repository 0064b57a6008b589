"""A launch that the CUDA runtime refuses is reported, and leaves nothing behind that a later,
correct call would report in its place.

The refusal is made on the host: a stream that is captured and then synchronized has an
invalidated capture, and takes no launch until the capture has ended.  torch does not get over
that, so it happens in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))


def refused_then_right():
    import torch

    import mxfp8_quantization_moe_mx_b200 as mxq

    def u8(*shape):
        return torch.empty(shape, dtype=torch.uint8, device="cuda")

    x = torch.randn(64, 64, device="cuda").bfloat16()
    y, q, s, t, fs = torch.empty_like(x), u8(64, 64), u8(64, 2), u8(64, 64), torch.empty(1, 64, device="cuda")
    blocked = u8(mxq.mx_scales_blocked_bytes(1, 64, 2))
    offs = torch.tensor([64], dtype=torch.int32, device="cuda")
    ids = torch.zeros(64, dtype=torch.int32, device="cuda")
    plan = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (8, 64, 64)]
    calls = [lambda: mxq.mx_quantize(x, mxq.ROW, q_row=q, s_row=s),
             lambda: mxq.mx_dequantize(q, s, 1, 64, 64, mxq.ROW, y),
             lambda: mxq.mxq_transpose_u8(q, t),
             lambda: mxq.mx_scales_to_blocked(s, blocked),
             lambda: mxq.fp8_per_group_rowwise_quant(x, offs, mxq.COL_MAJOR, q, fs)]
    for call in calls:  # loads every kernel
        call()
    mxq.moe_plan(ids, *plan)
    torch.cuda.synchronize()
    for call in calls:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph.capture_begin()
            try:
                side.synchronize()
                raise SystemExit("the capture was not invalidated")
            except RuntimeError:
                pass
            try:
                mxq.moe_plan(ids, *plan, stream=side)
                raise SystemExit("the launch was not refused")
            except mxq.MxqError:
                pass
            try:
                graph.capture_end()
            except RuntimeError:
                pass
        call()
    torch.cuda.synchronize()


def test_a_refused_launch_is_not_reported_twice():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    code = (f"import sys; sys.path[:0] = [{TESTS!r}, {os.path.dirname(TESTS)!r}]\n"
            f"from _gpu import ensure_lib; ensure_lib()\n"
            f"import test_error_state_gpu as t; t.refused_then_right()")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
