"""The mixture-of-experts operators as a model calls them (mxfp8_quantization_moe_mx_b200.moe):
gradients through autograd against the formulas in 64 bits, and the calls that the
documentation allows around them.

Tolerances: those of tests/test_moe_gpu.py for one operator; a chain adds its operators'."""
import numpy as np
import pytest
import torch

import _moe_ref as ref
import mxfp8_quantization_moe_mx_b200 as mxq
from _gpu import ensure_lib
from mxfp8_quantization_moe_mx_b200 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_lib()
    yield
    assert mxq.mxq_wait_timeouts() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def near(got, want, mag, rel):
    got, want, mag = (t.detach().double().cpu() for t in (got, want, mag))
    assert ((got - want).abs() <= rel * mag + 2.0 ** -8 * want.abs() + 1e-30).all(), (got - want).abs().max()


def plain_norm(x, w, residual, eps=1e-5):
    h = x if residual is None else x + residual
    return h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * w, h


@pytest.mark.parametrize("wdt", [BF, torch.float32])
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_gradients(wdt, with_res):
    g = gen(1)
    # sums that bf16 holds exactly, so that the 64-bit form sees the same stream
    x = (torch.randint(-64, 65, (300, 352), generator=g) / 32).to(BF).cuda().requires_grad_()
    r = (torch.randint(-64, 65, (300, 352), generator=g) / 32).to(BF).cuda().requires_grad_() if with_res else None
    w = (1 + 0.2 * torch.randn(352, generator=g)).to(wdt).cuda().requires_grad_()
    gy, gr = torch.randn(300, 352, generator=g).to(BF).cuda(), torch.randn(300, 352, generator=g).to(BF).cuda()
    n = moe.rmsnorm(x, w, residual=r)
    ((n.y * gy).sum() + (n.res * gr).sum()).backward()
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    rd = r.detach().double().requires_grad_() if with_res else None
    y, h = plain_norm(xd, wd, rd)
    ((y * gy.double()).sum() + (h * gr.double()).sum()).backward()
    mag = gy.abs().double() * w.abs().double() * 4 + gr.abs().double() + 1
    if with_res:
        near(x.grad, xd.grad, mag, 2.0 ** -15)
        near(r.grad, rd.grad, mag, 2.0 ** -15)
    else:  # two gradients reach x and are added in bf16: half a step of each and of the sum
        near(x.grad, xd.grad, mag, 2.0 ** -7)
    step = 2.0 ** -8 if wdt == BF else 0.0
    terms = (gy.double() * h.detach() * torch.rsqrt(h.detach().square().mean(1, keepdim=True) + 1e-5)).abs().sum(0)
    assert ((w.grad.double() - wd.grad).abs() <= 2.0 ** -16 * terms + step * wd.grad.abs()).all()


def test_norm_gradient_of_the_stream_alone_and_of_expanded_gradients():
    x = torch.randn(5, 64, generator=gen(2)).to(BF).cuda().requires_grad_()
    r = torch.randn(5, 64, generator=gen(3)).to(BF).cuda().requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    moe.rmsnorm(x, w, residual=r).res.sum().backward()  # a gradient of stride 0
    assert (x.grad == 1).all() and (r.grad == 1).all() and w.grad is None
    x.grad = r.grad = None
    moe.rmsnorm(x, w, residual=r).y.sum().backward()
    h = (x.detach().float() + r.detach().float()).to(BF).double().requires_grad_()
    plain_norm(h, w.detach().double(), None)[0].sum().backward()
    near(x.grad, h.grad, torch.full_like(h, 4.0), 2.0 ** -15)
    assert torch.equal(x.grad, r.grad)


@pytest.mark.parametrize("score,renorm", [(mxq.SOFTMAX, False), (mxq.SOFTMAX, True), (mxq.SIGMOID, False),
                                          (mxq.SIGMOID, True)])
def test_route_gradients(score, renorm):
    g = gen(4)
    x = torch.randn(50, 33, generator=g).cuda().requires_grad_()
    bias = (0.1 * torch.randn(33, generator=g)).cuda().requires_grad_()
    gw = torch.randn(50, 4, generator=g).cuda()
    w, ids = moe.route(x, 4, bias=bias, score=score, renorm=renorm, scale=2.0)
    assert not ids.requires_grad
    (w * gw).sum().backward()
    xd = x.detach().double().requires_grad_()
    p = torch.softmax(xd, 1) if score == mxq.SOFTMAX else torch.sigmoid(xd)
    p = p.gather(1, ids.long())
    if renorm:
        p = p / p.sum(1, keepdim=True)
    (2.0 * p * gw.double()).sum().backward()
    assert bias.grad is None
    assert ((x.grad.double() - xd.grad).abs() <= 2.0 ** -16 * 2 * gw.abs().sum(1, keepdim=True).double()).all()


def test_route_of_strided_logits_and_no_rows():
    x = torch.randn(40, 20, generator=gen(5)).cuda()
    w, ids = moe.route(x.T, 3)
    w2, ids2 = moe.route(x.T.contiguous(), 3)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    w, ids = moe.route(x[:0], 3)
    assert w.shape == ids.shape == (0, 3)
    p = moe.plan(ids, 20)
    assert (p.offs == 0).all() and p.src.numel() == 0
    y = moe.rmsnorm(x[:0].to(BF).new_zeros(0, 32), torch.ones(32, device="cuda"))
    assert y.y.shape == (0, 32) and y.s.shape == (0, 1)


def test_a_training_step_through_norm_router_and_experts():
    """Loss and gradients of a small layer with bf16 experts: this library's norm, routing and
    row plan between torch's products, against the same layer in 64 bits with the same
    choices."""
    T, D, E, k = 200, 64, 8, 2
    g = gen(6)
    x = (torch.randint(-32, 33, (T, D), generator=g) / 16).to(BF).cuda().requires_grad_()
    r = (torch.randint(-32, 33, (T, D), generator=g) / 16).to(BF).cuda()
    w = torch.ones(D, device="cuda", requires_grad=True)
    router = (torch.randn(E, D, generator=g) / D ** 0.5).cuda().requires_grad_()
    mats = (torch.randn(E, D, D, generator=g) / D ** 0.5).cuda()

    n = moe.rmsnorm(x, w, residual=r)
    weights, ids = moe.route(n.y.float() @ router.T, k, renorm=True)
    p = moe.plan(ids, E)
    rows = n.y.float()[p.src.long() // k]
    expert = torch.searchsorted(p.offs, torch.arange(T * k, device="cuda"), right=True)
    out = torch.einsum("md,mnd->mn", rows, mats[expert])
    y = (out[p.rows.long()] * weights[:, :, None]).sum(1)
    loss = (y * y).mean()
    loss.backward()

    xd, rd = x.detach().double().requires_grad_(), r.double()
    wd, routerd = w.detach().double().requires_grad_(), router.detach().double().requires_grad_()
    yd, _ = plain_norm(xd, wd, rd)
    # the norm leaves in bf16: the same rounding, its gradient passed straight through
    yb = yd + (n.y.detach().double() - yd).detach()
    pr = torch.softmax((yb @ routerd.T).gather(1, ids.long()), 1)
    od = torch.einsum("td,tknd->tkn", yb, mats.double()[ids.long()])
    lossd = ((od * pr[:, :, None]).sum(1) ** 2).mean()
    lossd.backward()
    assert abs(float(loss.detach()) - float(lossd.detach())) <= 1e-5 * float(lossd.detach())
    # fp32 products of 64 terms and the router's gradient: 2^-14 of the largest; x's gradient
    # passes bf16 once (gradient of y) and is rounded to it: 2^-7
    for a, b, tol in ((router.grad, routerd.grad, 2.0 ** -12), (w.grad, wd.grad, 2.0 ** -7), (x.grad, xd.grad, 2.0 ** -7)):
        assert (a.double() - b).abs().max() <= tol * b.abs().max()


def test_backward_in_a_graph():
    """Forward and backward captured and replayed on new inputs give the eager gradients."""
    T, D, E, k = 64, 128, 16, 2
    g = gen(7)
    x = torch.randn(T, D, generator=g).to(BF).cuda()
    w = torch.ones(D, device="cuda")
    router = (torch.randn(E, D, generator=g) / D ** 0.5).cuda()

    def step(x):
        xs, ws, rs = (t.detach().requires_grad_() for t in (x, w, router))
        n = moe.rmsnorm(xs, ws, residual=x)
        weights, ids = moe.route(n.y.float() @ rs.T, k)
        loss = (weights * weights).sum() + n.res.float().square().mean()
        return (*torch.autograd.grad(loss, (xs, ws, rs)), ids)

    static = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(static)
    for seed in (8, 9):
        new = torch.randn(T, D, generator=gen(seed)).to(BF).cuda()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(new)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams with buffers of their own do not disturb each other."""
    T, E, k = 30000, 64, 2
    xs = [torch.randn(T, E, generator=gen(s)).cuda() for s in (1, 2)]
    want = [(*moe.route(x, k), *moe.plan(moe.route(x, k)[1], E)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                w, ids = moe.route(x, k)
                got.append((w, ids, *moe.plan(ids, E)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_experts_held_in_four_bits():
    g = gen(10)
    G, N, K = 3, 256, 384
    weights = (0.05 * torch.randn(G, N, K, generator=g)).to(BF).cuda()
    experts = moe.Mxfp4Experts(weights)
    for sizes in ([1, 0, 0], [2, 5, 1], [200, 0, 300]):
        M = sum(sizes)
        x = torch.randn(M, K, generator=g).to(BF).cuda()
        offs = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
        out = experts(x, offs)
        a = ref.f4_values(*ref.f4_quantize(x.double().cpu().numpy()))
        at = 0
        for e, n in enumerate(sizes):
            b = ref.f4_values(*ref.f4_quantize(weights[e].double().cpu().numpy()))
            want, mag = a[at:at + n] @ b.T, np.abs(a[at:at + n]) @ np.abs(b).T
            got = out[at:at + n].double().cpu().numpy()
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * mag)
            at += n
    with pytest.raises(mxq.MxqError, match="gradient"):
        experts(x.requires_grad_(), offs)
    with torch.no_grad():
        experts(x, offs)
    for bad in (torch.zeros(2, 100, 384), torch.zeros(2, 256, 100)):
        with pytest.raises(mxq.MxqError):
            moe.Mxfp4Experts(bad.to(BF).cuda())
    with pytest.raises(mxq.MxqError):
        experts(x.detach()[:, :128], offs)


def test_two_products_at_once():
    """The few-row and the many-row product on two streams, several times over."""
    g = gen(12)
    few = moe.Mxfp4Experts((0.05 * torch.randn(8, 512, 1024, generator=g)).to(BF).cuda())
    many = moe.Mxfp4Experts((0.05 * torch.randn(2, 2560, 1024, generator=g)).to(BF).cuda())
    jobs = [(few, torch.randn(16, 1024, generator=g).to(BF).cuda(),
             torch.arange(2, 18, 2, dtype=torch.int32, device="cuda")),
            (many, torch.randn(1500, 1024, generator=g).to(BF).cuda(),
             torch.tensor([700, 1500], dtype=torch.int32, device="cuda"))]
    want = [e(x, o) for e, x, o in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        got = []
        for (e, x, o), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append([e(x, o) for _ in range(3)])
        torch.cuda.synchronize()
        for outs, w in zip(got, want):
            assert all(torch.equal(u, w) for u in outs)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their last rows as a call on those rows alone."""
    D = 16384
    M = (1 << 31) // D + 300
    x = torch.empty(M, D, dtype=BF, device="cuda")
    x[:4].normal_()
    x[4:-4] = 1.0
    x[-4:].normal_()
    w = torch.ones(D, device="cuda")
    q, s = (torch.empty(M, n, dtype=torch.uint8, device="cuda") for n in (D, D // 32))
    y, r = torch.empty_like(x), torch.empty(M, device="cuda")
    mxq.rmsnorm_mx_quantize(x, w, 1e-5, q, s, y=y, rstd=r)
    for part in (slice(0, 4), slice(M - 4, M)):
        n = moe.rmsnorm(x[part], w)
        assert torch.equal(n.y, y[part]) and torch.equal(n.q, q[part]) and torch.equal(n.s, s[part])
    gx, gw = torch.empty_like(x), torch.empty(D, device="cuda")
    ws = torch.empty(mxq.rmsnorm_backward_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    mxq.rmsnorm_backward(y, x, w, r, gx, gw, ws)
    part, gw4 = torch.empty(4, D, dtype=BF, device="cuda"), torch.empty_like(gw)
    mxq.rmsnorm_backward(y[-4:], x[-4:], w, r[-4:], part, gw4, ws)
    assert torch.equal(part, gx[-4:])
    del gx, y, q, s
    codes, scales = (torch.empty(M, n, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 32))
    mxq.mxfp4_quantize(x, codes, scales)
    back = torch.empty_like(x)
    mxq.mxfp4_dequantize(codes, scales, back)
    c4, s4, b4 = torch.empty_like(codes[:4]), torch.empty_like(scales[:4]), torch.empty_like(back[:4])
    mxq.mxfp4_quantize(x[-4:], c4, s4)
    mxq.mxfp4_dequantize(c4, s4, b4)
    assert torch.equal(c4, codes[-4:]) and torch.equal(s4, scales[-4:]) and torch.equal(b4, back[-4:])
    tiles = torch.empty(mxq.mx_scales_blocked_bytes(1, M, D // 32), dtype=torch.uint8, device="cuda")
    again = torch.empty_like(codes)
    mxq.mxfp4_quantize(x, again, sf_blocked=tiles)
    assert torch.equal(again[-4:], c4)
    want = torch.empty_like(tiles)
    mxq.mx_scales_to_blocked(scales, want)
    assert torch.equal(tiles, want)
    del x, back, codes, again, tiles, want
    T, E = (1 << 31) // 256 + 77, 256
    logits = torch.zeros(T, E, dtype=BF, device="cuda")
    logits[-9:].normal_()
    wt, ids = moe.route(logits, 4)
    w9, i9 = moe.route(logits[-9:], 4)
    assert torch.equal(wt[-9:], w9) and torch.equal(ids[-9:], i9)
    assert (ids[:-9] == torch.arange(4, dtype=torch.int32, device="cuda")).all()
