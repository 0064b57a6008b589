"""The bounded waits of the norm's gradient, made to give up on purpose: a CTA that gives up
leaves its remaining rows of grad_x unwritten, grad_weight is NaN throughout (its sums lack
those rows), and the CTA is counted.

No GPU fault is involved: giving up is an ordinary branch of the kernel, and every copy still
lands before its CTA exits."""
import pytest
import torch

import mxfp8_quantization_moe_mx_b200 as mxq
from _gpu import CANARY, ensure_lib

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_lib()
    yield
    mxq.mxq_set_wait_limit_ns(mxq.WAIT_LIMIT_DEFAULT_NS)


def operands(M, D, with_res):
    g = torch.Generator().manual_seed(M + D)
    gy, h, gres = (torch.randn(M, D, generator=g).to(BF).cuda() for _ in range(3))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(BF).cuda()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    ws = torch.empty(mxq.rmsnorm_backward_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")

    def run(limit):
        """(grad_x's bits, grad_weight, CTAs that gave up); the workspace holds an earlier call's sums."""
        gx, gw = torch.empty_like(h), torch.empty(D, device="cuda")
        gx.view(torch.uint8).fill_(CANARY)
        before = mxq.mxq_wait_timeouts()
        mxq.mxq_set_wait_limit_ns(limit)
        try:
            mxq.rmsnorm_backward(gy, h, w, rstd, gx, gw, ws, grad_res=gres if with_res else None)
            torch.cuda.synchronize()
        finally:
            mxq.mxq_set_wait_limit_ns(mxq.WAIT_LIMIT_DEFAULT_NS)
        return gx.view(torch.int16), gw, mxq.mxq_wait_timeouts() - before
    return run


@pytest.mark.parametrize("M,D,with_res", [(1, 64, False), (7, 512, True), (60, 5120, True), (9, 16384, True),
                                          (31, 1056, False)])
def test_every_wait_gives_up(M, D, with_res):
    run = operands(M, D, with_res)
    gx, gw, n = run(mxq.WAIT_LIMIT_DEFAULT_NS)
    assert n == 0 and torch.isfinite(gw).all()
    bits, lost, n = run(0)
    assert n == M  # a row per CTA
    assert (bits.view(torch.uint8) == CANARY).all()
    assert torch.isnan(lost).all()
    again, gw2, n = run(mxq.WAIT_LIMIT_DEFAULT_NS)
    assert n == 0 and torch.equal(again, gx) and torch.equal(gw2, gw)


@pytest.mark.parametrize("limit", [1, 300, 1000])
@pytest.mark.parametrize("M,D", [(3000, 512), (2000, 5120)])
def test_some_waits_give_up(M, D, limit):
    """Limits near a copy's own time: some CTAs give up, some of them after several rows.  A row
    is written whole and right or not at all."""
    run = operands(M, D, True)
    gx, gw, _ = run(mxq.WAIT_LIMIT_DEFAULT_NS)
    for _ in range(5):
        bits, got, n = run(limit)
        untouched = (bits.view(torch.uint8) == CANARY).all(1)
        assert ((bits == gx).all(1) | untouched).all()
        if n:
            assert untouched.any() and torch.isnan(got).all()
        else:
            assert torch.equal(bits, gx) and torch.equal(got, gw)
    again, gw2, n = run(mxq.WAIT_LIMIT_DEFAULT_NS)
    assert n == 0 and torch.equal(again, gx) and torch.equal(gw2, gw)
