"""The mixture-of-experts operators on the GPU against their plain 64-bit forms.

Tolerances, fixed before the first run (u = 2^-24, the relative half step of fp32):
  route weights   the score's error: |l - max| u for the rounded argument (logits here stay
                  within 40 of the maximum), 4 u for exp (2 units in the last place), 37 u
                  for the sum (chains of 32 + 5 additions), 6 u for the divisions and
                  products: 87 u < 2^-17 relative; below 2^-120 the scores underflow.
  route gradient  2^-16 of the sum of its terms' magnitudes (two such scores and a sum of at
                  most 32 terms), and half a step (2^-8) for bf16 output.
  norm            mean of squares: chains of 32 + 5 + 5 additions and the products: 50 u;
                  1 / sqrt halves it: rstd within 2^-18; y = h r w two roundings more, and
                  half a step of bf16 (2^-8).
  norm gradient   the mean of products the same way, so 2^-17 of the terms' magnitudes and
                  half a step of bf16; the weight's gradient: a CTA adds M / 148 rows at
                  most at these sizes (34 of them), then up to 592 / 8 + 8 partial sums,
                  and n = h r carries rstd's error: 2^-16 of the magnitudes' sum.
  fp4             exact.  The product: 2^-8 |ref| + K 2^-23 sum |a b| as for MXFP8 (bf16
                  rounding and any order of fp32 additions, both doubled).
"""
import itertools

import numpy as np
import pytest
import torch

import _moe_ref as ref
import mxfp8_quantization_moe_mx_b200 as mxq
import oracle
from _gpu import bits_of, ensure_lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_lib()
    yield
    assert mxq.mxq_wait_timeouts() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def empty(dt, *shape):
    """Device memory with a pattern in it."""
    t = torch.empty(shape, dtype=dt, device="cuda")
    t.view(torch.uint8).fill_(0xA5)
    return t


# ---- routing ---------------------------------------------------------------------------------------

def gpu_route(x, k, bias=None, **kw):
    w, i = empty(F32, x.shape[0], k), empty(torch.int32, x.shape[0], k)
    mxq.moe_route(x.cuda(), w, i, bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    return i.cpu().numpy(), f64(w)


def check_route(x, k, bias=None, score="softmax", n_groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0):
    ids, w = gpu_route(x, k, bias, score=mxq.SIGMOID if score == "sigmoid" else mxq.SOFTMAX, n_groups=n_groups,
                       top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale)
    rid, rw = ref.route(f64(x), None if bias is None else f64(bias), score, n_groups, top_groups, group_top, k,
                        renorm, scale)
    assert np.array_equal(ids, rid)
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    assert np.all(w[ids < 0] == 0)
    fine = ~np.isnan(rw)
    assert np.all(np.abs(w - rw)[fine] <= 2.0 ** -17 * np.abs(rw[fine]) + 2.0 ** -120)
    return ids


SHAPES = [(1, 1, 1), (1, 5, 3), (2, 31, 31), (3, 32, 1), (9, 33, 7), (5, 64, 32), (17, 100, 8), (8, 128, 8),
          (13, 160, 6), (7, 256, 8), (6, 511, 10), (4, 1000, 16), (5, 1024, 32)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_route_shapes(T, E, k, dt):
    for n, (score, renorm, with_bias) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True),
                                                                    (False, True))):
        g = gen(1000 * n + E)
        x = (2.0 * torch.randn(T, E, generator=g)).to(dt)
        b = 0.1 * torch.randn(E, generator=g) if with_bias else None
        check_route(x, k, b, score=score, renorm=renorm, scale=1.0 if n % 2 else 2.5)


@pytest.mark.parametrize("E,n_groups,top_groups,k", [(4, 2, 1, 2), (64, 8, 3, 6), (60, 4, 2, 5), (96, 32, 7, 12),
                                                     (256, 8, 4, 8), (255, 5, 2, 9), (992, 31, 1, 32), (64, 32, 2, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, n_groups, top_groups, k, score):
    for n, (dt, gt, with_bias) in enumerate(itertools.product((BF, F32), (1, 2), (False, True))):
        g = gen(100 * n + E)
        x = (2.0 * torch.randn(21, E, generator=g)).to(dt)
        b = 0.2 * torch.randn(E, generator=g) if with_bias else None
        ids = check_route(x, k, b, score=score, n_groups=n_groups, top_groups=top_groups, group_top=gt, renorm=True)
        if k > top_groups * (E // n_groups):
            assert (ids < 0).any()  # the kept groups have fewer experts than k


def test_route_masked_rows_and_experts():
    g = gen(7)
    x = torch.randn(12, 70, generator=g)
    x[0] = -np.inf                     # nothing is left
    x[1, 5:] = -np.inf                 # fewer than k
    x[2, :69] = -np.inf                # one
    x[3, ::2] = -np.inf
    x[4] = torch.finfo(BF).min         # the lowest finite value is an ordinary one
    x[5, 10:] = torch.finfo(BF).min
    b = 0.1 * torch.randn(70, generator=g)
    b[[3, 9]] = -np.inf
    for dt, bias, score, (n, top, gt) in itertools.product((BF, F32), (None, b), ("softmax", "sigmoid"),
                                                           ((1, 1, 1), (7, 2, 1), (7, 3, 2))):
        for renorm in (False, True):
            check_route(x.to(dt), 8, bias, score=score, n_groups=n, top_groups=top, group_top=gt, renorm=renorm)


def test_route_ties_go_to_the_lower_index():
    x = torch.zeros(6, 96)
    x[1] = torch.arange(96) % 3
    x[2] = -(torch.arange(96) // 2).float()
    x[3, ::2] = -0.0                                    # equal to +0
    x[4] = 50.0 + (torch.arange(96) % 4)                # sigmoid is 1 in 64 bits for all of them
    x[5, 40:] = 1.0
    zero = torch.zeros(96)
    for dt, bias, score, (n, top, gt) in itertools.product((BF, F32), (None, zero), ("softmax", "sigmoid"),
                                                           ((1, 1, 1), (8, 3, 1), (8, 3, 2))):
        if bias is not None and score == "sigmoid":
            y = x[:4]                                   # the 64-bit scores of row 4 tie, exactly or not by rounding
        else:
            y = x
        check_route(y.to(dt), 8, bias, score=score, n_groups=n, top_groups=top, group_top=gt)


def test_route_order_of_close_candidates():
    """Candidates that differ by less than 32 bits resolve: logits one step apart whose
    biases all but undo the difference, so that the order is decided in 64 bits."""
    g = gen(11)
    E = 64
    x = torch.randn(200, E, generator=g)
    base = torch.randn(200, 1, generator=g)
    x[:, 8:24] = base + torch.arange(16) * 2.0 ** -23
    b = torch.zeros(E)
    b[8:24] = 1.0 + torch.randperm(16, generator=g) * 2.0 ** -23
    for score in ("softmax", "sigmoid"):
        check_route(x, 12, b, score=score)
        check_route(x, 8, b, score=score, n_groups=8, top_groups=2, group_top=2)


@pytest.mark.parametrize("k", [4, 12, 20, 32])
def test_route_candidate_with_a_large_score_among_small_ones(k):
    """One expert takes most of the softmax and its bias brings it down among the others: its
    candidate's error in 32 bits is a thousand times its neighbours', and sweeps past them."""
    g = gen(13)
    E, T = 64, 600
    x = 0.5 * torch.randn(1, E, generator=g).repeat(T, 1)
    x[:, 5] = 7.0 + torch.arange(T) * 2.0 ** -19
    b = 0.05 * torch.rand(E, generator=g)
    p = torch.softmax(x[T // 2].double(), 0)
    c = torch.sort(p + b, descending=True).values
    for place in (k - 1, k, k // 2):
        b[5] = 0.0
        b[5] = float(c[place + 1] - p[5])
        check_route(x, k, b)


def test_route_large_biases_that_cancel_in_groups():
    g = gen(12)
    x = torch.randn(100, 32, generator=g)
    b = torch.empty(32)
    b[0::2], b[1::2] = 64.0, -64.0 + 2.0 ** -18 * torch.arange(16)
    check_route(x, 4, b, score="sigmoid", n_groups=16, top_groups=3, group_top=2)


def test_route_rows_with_nan_and_inf_show():
    x = torch.randn(6, 40, generator=gen(3))
    x[0, 7] = np.nan
    x[1, 39] = np.inf
    x[2, 3] = np.nan
    x[2, 4] = -np.inf
    b = torch.zeros(40)
    nb = b.clone()
    nb[5] = np.nan
    for bias in (None, b, nb):
        for score in ("softmax", "sigmoid"):
            y = x.clone()
            if bias is nb:
                y[4, 5] = -np.inf  # masked: its bias does not matter
            check_route(y, 3, bias, score=score)


def test_route_infinite_bias_forces_the_choice():
    x = torch.randn(5, 40, generator=gen(4))
    b = torch.zeros(40)
    b[[30, 2, 17]] = np.inf
    for score in ("softmax", "sigmoid"):
        ids = check_route(x, 5, b, score=score)
        assert (ids[:, :3] == [2, 17, 30]).all()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("score,renorm", list(itertools.product(("softmax", "sigmoid"), (False, True))))
def test_route_backward(T, E, k, dt, score, renorm):
    g = gen(E + T)
    x = (2.0 * torch.randn(T, E, generator=g)).to(dt)
    x[0, : E // 2] = -np.inf
    if T > 2:
        x[2] = -np.inf
    code = mxq.SIGMOID if score == "sigmoid" else mxq.SOFTMAX
    ids, _ = gpu_route(x, k, score=code, renorm=renorm, scale=1.5)
    gw = torch.randn(T, k, generator=g)
    out = empty(dt, T, E)
    mxq.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), gw.cuda(), out, score=code, renorm=renorm,
                           scale=1.5)
    want, mag = ref.route_grad(f64(x), ids, f64(gw), score, renorm, 1.5)
    half = 2.0 ** -8 if dt == BF else 2.0 ** -24
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -16 * mag + half * np.abs(want) + 2.0 ** -120)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_route_backward_where_one_expert_has_nearly_all(score, renorm):
    """Weights near 1 and 0: the difference g_j - sum g_m r_m is small beside its terms.  Each
    entry, to 2^-16 of the sum of the magnitudes of its own uncancelled terms
    r_j r_m |g_j - g_m| (and p_j p_e |g_j| for the unchosen)."""
    g = gen(31)
    T, E, k = 64, 24, 4
    x = torch.randn(T, E, generator=g)
    if score == "softmax":
        x[:, 3] += torch.linspace(8.0, 16.0, T)
    else:
        x[:, 3] = 4.0
        x[:, :3] -= 10.0
        x[:, 4:] -= torch.linspace(8.0, 16.0, T)[:, None]
    code = mxq.SIGMOID if score == "sigmoid" else mxq.SOFTMAX
    ids, _ = gpu_route(x, k, score=code, renorm=renorm)
    gw = torch.randn(T, k, generator=g)
    out = empty(F32, T, E)
    mxq.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), gw.cuda(), out, score=code, renorm=renorm)
    want, _ = ref.route_grad(f64(x), ids, f64(gw), score, renorm, 1.0)
    z, w = f64(x), f64(gw)
    for t in range(T):
        p = ref.scores(z[t], score)
        mag = np.zeros(E)
        r = p[ids[t]] / (p[ids[t]].sum() if renorm else 1.0)
        f = 1.0 - p[ids[t]] if score == "sigmoid" else 1.0
        mag[ids[t]] = f * r * (r[None, :] * np.abs(w[t][:, None] - w[t][None, :])).sum(1)
        if not renorm:
            rest = np.delete(np.arange(E), ids[t])
            mag[ids[t]] += r * np.abs(w[t]) * p[rest].sum()
            mag[rest] = p[rest] * (np.abs(w[t]) * r).sum()
        assert np.all(np.abs(f64(out)[t] - want[t]) <= 2.0 ** -16 * mag + 2.0 ** -120)


def test_route_backward_against_differences():
    """The gradient of a fixed choice against central differences of the 64-bit weights."""
    g = gen(21)
    x = torch.randn(4, 24, generator=g)
    gw = torch.randn(4, 5, generator=g)
    for score, renorm in itertools.product(("softmax", "sigmoid"), (False, True)):
        code = mxq.SIGMOID if score == "sigmoid" else mxq.SOFTMAX
        ids, _ = gpu_route(x, 5, score=code, renorm=renorm)
        out = empty(F32, 4, 24)
        mxq.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), gw.cuda(), out, score=code, renorm=renorm)

        def value(z):
            tot = 0.0
            for t in range(4):
                p = ref.scores(z[t], score)[ids[t]]
                if renorm:
                    p = p / p.sum()
                tot += (p * f64(gw)[t]).sum()
            return tot
        z, h = f64(x), 1e-5
        num = np.zeros_like(z)
        for t, e in itertools.product(range(4), range(24)):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            num[t, e] = (value(up) - value(dn)) / (2 * h)
        # differences: h^2 / 6 times a third derivative (below 1), and 2^-52 / h of rounding
        assert np.all(np.abs(f64(out) - num) <= 1e-9 + 2.0 ** -16 * np.abs(f64(gw)).max())


def test_route_backward_repeated_and_foreign_indices():
    """An index that comes twice counts twice; indices outside the experts are skipped."""
    x = torch.randn(3, 20, generator=gen(5))
    ids = np.array([[4, 4, 4, 7], [-1, 20, 3, 1 << 30], [0, 19, 0, -5]], np.int32)
    gw = torch.randn(3, 4, generator=gen(6))
    for score, renorm in itertools.product(("softmax", "sigmoid"), (False, True)):
        out = empty(F32, 3, 20)
        mxq.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), gw.cuda(), out,
                               score=mxq.SIGMOID if score == "sigmoid" else mxq.SOFTMAX, renorm=renorm)
        want, mag = ref.route_grad(f64(x), ids, f64(gw), score, renorm, 1.0)
        assert np.all(np.abs(f64(out) - want) <= 2.0 ** -16 * mag + 2.0 ** -24 * np.abs(want) + 2.0 ** -120)


@pytest.mark.parametrize("dt", [BF, F32])
def test_route_of_rows_off_the_wide_boundaries(dt):
    """Logits and gradients that start anywhere: slices of larger tensors."""
    for E, skip in ((64, 1), (256, 3), (128, 5), (16, 7)):
        big = torch.randn(9 * E + 16, generator=gen(E)).to(dt).cuda()
        x = big[skip:skip + 9 * E].view(9, E)
        w, ids = empty(F32, 9, 4), empty(torch.int32, 9, 4)
        mxq.moe_route(x, w, ids)
        w2, ids2 = empty(F32, 9, 4), empty(torch.int32, 9, 4)
        mxq.moe_route(x.clone(), w2, ids2)
        assert torch.equal(w, w2) and torch.equal(ids, ids2)
        gw = torch.randn(9, 4, generator=gen(1)).cuda()
        buf = empty(dt, 9 * E + 16)
        mxq.moe_route_backward(x, ids, gw, buf[skip:skip + 9 * E].view(9, E))
        want = empty(dt, 9, E)
        mxq.moe_route_backward(x.clone(), ids, gw, want)
        assert torch.equal(buf[skip:skip + 9 * E].view(9, E), want)
        rest = torch.cat((buf[:skip], buf[skip + 9 * E:])).view(torch.uint8)
        assert (rest == 0xA5).all()


def test_route_many_rows_are_all_written():
    """More rows than one pass of the grid covers; every row against the plain rule."""
    T, E, k = 30011, 16, 1
    x = torch.randn(T, E, generator=gen(8)).to(BF)
    ids, w = gpu_route(x, k, score=mxq.SIGMOID)
    z = f64(x)
    assert np.array_equal(ids[:, 0], z.argmax(1))
    p = 1 / (1 + np.exp(-z.max(1)))
    assert np.all(np.abs(w[:, 0] - p) <= 2.0 ** -17 * p)


# ---- plan --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (1, 8, 128), (7, 3, 5), (256, 8, 16), (255, 8, 300),
                                   (257, 8, 16), (1000, 6, 1024), (1024, 8, 256), (1025, 8, 256), (2049, 8, 256),
                                   (3001, 7, 64), (9000, 2, 3), (40000, 3, 1024)])
@pytest.mark.parametrize("kind", ["spread", "one", "none", "foreign"])
def test_plan(T, k, E, kind):
    g = gen(T + E)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if kind == "one":
        ids.fill_(E - 1)
    elif kind == "none":
        ids.fill_(-1)
    elif kind == "foreign":
        ids[torch.rand(T, k, generator=g) < 0.3] = -1
        ids[torch.rand(T, k, generator=g) < 0.1] = E
        ids[torch.rand(T, k, generator=g) < 0.1] = -(1 << 31)
        ids[torch.rand(T, k, generator=g) < 0.1] = (1 << 31) - 1
    n = T * k
    need = mxq.moe_plan_workspace_bytes(n, E)
    ws = empty(torch.uint8, need + 64)
    offs, rows, src = empty(torch.int32, E), empty(torch.int32, T, k), empty(torch.int32, n)
    mxq.moe_plan(ids.cuda(), offs, rows, src, ws[:need] if need else None)
    want = ref.plan(ids.numpy(), E)
    for got, w in zip((offs, rows, src), want):
        assert np.array_equal(got.cpu().numpy().reshape(-1), w)
    assert (ws[need:] == 0xA5).all()  # nothing past the workspace


def test_plan_refuses_a_small_workspace():
    ids = torch.zeros(50000, dtype=torch.int32, device="cuda")
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (8, 50000, 50000)]
    with pytest.raises(mxq.MxqError, match="workspace"):
        mxq.moe_plan(ids, *out)
    with pytest.raises(mxq.MxqError, match="workspace"):
        mxq.moe_plan(ids, *out, torch.empty(8, dtype=torch.uint8, device="cuda"))


# ---- norm ------------------------------------------------------------------------------------------------

def norm_inputs(M, D, wdt, seed, residual=True):
    g = gen(seed)
    x = (torch.randn(M, D, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(BF)
    r = torch.randn(M, D, generator=g).to(BF) if residual else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(wdt)
    return x, r, w


def gpu_norm(x, r, w, eps, y=True, rstd=True, res=True):
    M, D = x.shape
    o = {"q": empty(torch.uint8, M, D), "s": empty(torch.uint8, M, D // 32)}
    if y:
        o["y"] = empty(BF, M, D)
    if rstd:
        o["rstd"] = empty(F32, M)
    if res:
        o["res_out"] = empty(BF, M, D)
    mxq.rmsnorm_mx_quantize(x.cuda(), w.cuda(), eps, residual=None if r is None else r.cuda(), **o)
    torch.cuda.synchronize()
    return o


def check_norm(x, r, w, eps=1e-5):
    o = gpu_norm(x, r, w, eps)
    h = x if r is None else (x.float() + r.float()).to(BF)
    assert np.array_equal(bits_of(o["res_out"]), bits_of(h))
    z = f64(h)
    rstd = 1 / np.sqrt((z * z).mean(1) + eps)
    assert np.all(np.abs(f64(o["rstd"]) - rstd) <= 2.0 ** -18 * rstd)
    y = z * rstd[:, None] * f64(w)
    assert np.all(np.abs(f64(o["y"]) - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y) + 2.0 ** -133)
    # the codes are those of the norm's own bf16 output, byte for byte
    q = oracle.mx_quantize(bits_of(o["y"]), oracle.ROW)
    assert np.array_equal(o["q"].cpu().numpy(), q["q_row"])
    assert np.array_equal(o["s"].cpu().numpy(), q["s_row"])


@pytest.mark.parametrize("M,D", [(1, 32), (3, 64), (2, 96), (5, 256), (7, 288), (4, 512), (3, 1056), (9, 2048),
                                 (13, 5120), (5, 8192), (4, 8224), (3, 16352), (2, 16384), (700, 544), (1500, 5120)])
@pytest.mark.parametrize("wdt", [BF, F32])
def test_norm(M, D, wdt):
    for residual in (True, False):
        check_norm(*norm_inputs(M, D, wdt, M + D, residual))


def test_norm_without_the_optional_outputs():
    x, r, w = norm_inputs(6, 320, BF, 2)
    a = gpu_norm(x, r, w, 1e-6)
    b = gpu_norm(x, r, w, 1e-6, y=False, rstd=False, res=False)
    for k in b:
        assert torch.equal(a[k], b[k])


def test_norm_updates_the_residual_stream_in_place():
    for M in (6, 900):
        x, r, w = norm_inputs(M, 5120, BF, 3)
        a = gpu_norm(x, r, w, 1e-6)
        for at in ("x", "residual"):
            xd, rd = x.cuda(), r.cuda()
            q, s = empty(torch.uint8, M, 5120), empty(torch.uint8, M, 160)
            mxq.rmsnorm_mx_quantize(xd, w.cuda(), 1e-6, q, s, residual=rd, res_out=xd if at == "x" else rd)
            assert torch.equal(a["q"], q) and torch.equal(a["s"], s)
            assert torch.equal(a["res_out"], xd if at == "x" else rd)


def test_norm_of_zero_tiny_and_spoilt_rows():
    x, _, w = norm_inputs(8, 128, F32, 4, False)
    x[0] = 0
    x[1] = 1e-38
    x[2, 5] = np.nan
    x[3, 70] = np.inf
    x[4] = 3e38                        # the sum of squares overflows: r is 0
    x[5, :64] = 0                      # zero blocks
    o = gpu_norm(x, None, w, 1e-5)
    q = oracle.mx_quantize(bits_of(o["y"]), oracle.ROW)
    assert np.array_equal(o["q"].cpu().numpy(), q["q_row"])
    assert np.array_equal(o["s"].cpu().numpy(), q["s_row"])
    y = f64(o["y"])
    assert np.all(y[0] == 0) and np.all(y[4] == 0) and np.isnan(y[2]).all()
    assert np.isnan(y[3, 70]) and np.all(np.delete(y[3], 70) == 0)
    assert (o["s"][2] == 255).all()
    check_norm(x[5:], None, w)


@pytest.mark.parametrize("M,D", [(1, 32), (3, 96), (5, 512), (7, 1056), (13, 5120), (3, 16384), (2, 8224),
                                 (640, 544), (5000, 256)])
@pytest.mark.parametrize("wdt", [BF, F32])
def test_norm_backward(M, D, wdt):
    for with_res in (True, False):
        h, e, w = norm_inputs(M, D, wdt, 3 * M + D)
        g = (0.1 * torch.randn(M, D, generator=gen(M))).to(BF)
        z, gy, wt = f64(h), f64(g), f64(w)
        rstd = torch.from_numpy(1 / np.sqrt((z * z).mean(1) + 1e-5)).float()
        r = f64(rstd)[:, None]
        gx, gw = empty(BF, M, D), empty(F32, D)
        need = mxq.rmsnorm_backward_workspace_bytes(M, D)
        ws = empty(torch.uint8, need + 64)
        mxq.rmsnorm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda(), gx, gw, ws[:need],
                             grad_res=e.cuda() if with_res else None)
        torch.cuda.synchronize()
        n, gn = z * r, gy * wt
        mean = (gn * n).mean(1, keepdims=True)
        want = r * (gn - n * mean) + (f64(e) if with_res else 0)
        mag = r * (np.abs(gn) + np.abs(n) * np.abs(gn * n).mean(1, keepdims=True)) + (np.abs(f64(e)) if with_res else 0)
        assert np.all(np.abs(f64(gx) - want) <= 2.0 ** -17 * mag + 2.0 ** -8 * np.abs(want))
        assert np.all(np.abs(f64(gw) - (gy * n).sum(0)) <= 2.0 ** -16 * np.abs(gy * n).sum(0))
        assert (ws[need:] == 0xA5).all()


def test_norm_backward_in_place_and_without_rows():
    h, e, w = norm_inputs(9, 640, BF, 5)
    g = torch.randn(9, 640, generator=gen(1)).to(BF).cuda()
    rstd = (1 / (f64(h) ** 2).mean(1) ** 0.5).astype(np.float32)
    args = h.cuda(), w.cuda(), torch.from_numpy(rstd).cuda()
    ws = empty(torch.uint8, mxq.rmsnorm_backward_workspace_bytes(9, 640))
    gx, gw = empty(BF, 9, 640), empty(F32, 640)
    mxq.rmsnorm_backward(g, *args, gx, gw, ws, grad_res=e.cuda())
    for at in ("g", "e"):
        a, b, gw2 = g.clone(), e.cuda(), empty(F32, 640)
        mxq.rmsnorm_backward(a, *args, a if at == "g" else b, gw2, ws, grad_res=b)
        assert torch.equal(gx, a if at == "g" else b) and torch.equal(gw, gw2)
    none = torch.empty(0, 640, dtype=BF, device="cuda")
    mxq.rmsnorm_backward(none, none, args[1], args[2][:0], none, gw, ws[:0])
    assert (gw == 0).all()


# ---- fp4 --------------------------------------------------------------------------------------------------

def f4_inputs(rows, cols, seed):
    """bf16 values over the whole exponent range, with zero blocks, subnormals, exact ties,
    infinities and NaN."""
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp2(torch.randint(-40, 40, (rows, cols // 32, 1), generator=g).float()).expand(-1, -1, 32).reshape(x.shape)
    x = x.to(BF)
    blocks = x.view(-1, 32)
    n = blocks.shape[0]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.96875, 4.0, 0.0, -0.0, -0.25, -2.5, -5.0])
    special = [torch.zeros(32), torch.cat((ties, -ties)), torch.cat((ties, ties)) * 2.0 ** -120,
               torch.full((32,), 1e-40), torch.cat((ties, ties)) * 2.0 ** 124, torch.full((32,), -0.0)]
    for i, s in enumerate(special):
        if n > 2 * i:
            blocks[2 * i] = s.to(BF)
    if n > 20:
        blocks[13, 5], blocks[15, 31], blocks[17, 0] = np.nan, -np.inf, np.inf
    return x


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (16, 512), (130, 544), (257, 1056), (5, 5120)])
def test_fp4_quantize_and_back(rows, cols):
    x = f4_inputs(rows, cols, rows + cols)
    code, s = ref.f4_quantize(f64(x))
    q, sd = empty(torch.uint8, rows * cols // 2 + 64), empty(torch.uint8, rows * cols // 32 + 64)
    qv, sv = q[:rows * cols // 2].view(rows, -1), sd[:rows * cols // 32].view(rows, -1)
    mxq.mxfp4_quantize(x.cuda(), qv, sv)
    assert np.array_equal(sv.cpu().numpy(), s)
    assert np.array_equal(qv.cpu().numpy(), ref.f4_pack(code))
    y = empty(BF, rows, cols)
    mxq.mxfp4_dequantize(qv, sv, y)
    want = ref.f4_values(code, s)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want).to(BF)  # exact but for what overflows
    got, nan = y.cpu(), torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    assert torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))
    assert (q[rows * cols // 2:] == 0xA5).all() and (sd[rows * cols // 32:] == 0xA5).all()


@pytest.mark.parametrize("cols", [32, 160, 512, 544, 1056])
def test_fp4_scales_in_tiles_per_matrix(cols):
    x = torch.stack([f4_inputs(140, cols, i) for i in range(3)])
    q, s = empty(torch.uint8, 3, 140, cols // 2), empty(torch.uint8, 3, 140, cols // 32)
    sf = empty(torch.uint8, mxq.mx_scales_blocked_bytes(3, 140, cols // 32) + 64)
    mxq.mxfp4_quantize(x.cuda(), q, s, sf_blocked=sf)
    want = [ref.f4_quantize(f64(m)) for m in x]
    assert np.array_equal(q.cpu().numpy(), np.stack([ref.f4_pack(c) for c, _ in want]))
    assert np.array_equal(s.cpu().numpy(), np.stack([t for _, t in want]))
    assert np.array_equal(sf[:-64].cpu().numpy(), np.concatenate([ref.blocked(t) for _, t in want]))
    assert (sf[-64:] == 0xA5).all()
    again = torch.empty_like(sf)
    mxq.mx_scales_to_blocked(s, again)
    assert torch.equal(again[:-64], sf[:-64])


@pytest.mark.parametrize("sizes", [[1], [0, 0], [3, 0, 128, 129, 1], [300], [0, 5, 0, 0, 7], [1] * 70])
def test_fp4_scales_in_tiles_per_group(sizes):
    M, cols, G = sum(sizes) + 5, 288, len(sizes)
    offs = np.cumsum(sizes).astype(np.int32)
    x = f4_inputs(M, cols, M)
    q = empty(torch.uint8, M, cols // 2)
    sf = empty(torch.uint8, mxq.mx_scales_blocked_bytes(1, M, cols // 32, G) + 64)
    mxq.mxfp4_quantize(x.cuda(), q, sf_blocked=sf, offs=torch.from_numpy(offs).cuda())
    code, s = ref.f4_quantize(f64(x))
    have = int(offs[-1])
    assert np.array_equal(q.cpu().numpy()[:have], ref.f4_pack(code)[:have])
    assert (q[have:] == 0xA5).all()          # rows in no group are left alone
    want = ref.blocked(s, offs)
    assert np.array_equal(sf.cpu().numpy()[:want.size], want)
    assert (sf[want.size:] == 0xA5).all()


def f4_operands(M, N, K, G, offs, seed, special=False):
    g = gen(seed)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(BF)
    w = (0.05 * torch.randn(G, N, K, generator=g)).to(BF)
    if special and M > 1:
        x[M // 2, K - 1] = np.nan  # its block's scale is NaN: the row's outputs are NaN, no other's
    xd, wd, od = x.cuda(), w.cuda(), torch.from_numpy(np.asarray(offs, np.int32)).cuda()
    qa, qb = empty(torch.uint8, M, K // 2), empty(torch.uint8, G, N, K // 2)
    sfa = empty(torch.uint8, mxq.mx_scales_blocked_bytes(1, M, K // 32, G))
    sfb = empty(torch.uint8, mxq.mx_scales_blocked_bytes(G, N, K // 32))
    mxq.mxfp4_quantize(xd, qa, sf_blocked=sfa, offs=od)
    mxq.mxfp4_quantize(wd, qb, sf_blocked=sfb)
    return x, w, (qa, sfa, qb, sfb, od)


def check_product(M, N, K, offs, seed=0, special=False):
    G = len(offs)
    x, w, ops = f4_operands(M, N, K, G, offs, seed, special)
    out = empty(BF, M, N)
    mxq.mxfp4_grouped_gemm(*ops, out)
    torch.cuda.synchronize()
    got = f64(out)
    a = ref.f4_values(*ref.f4_quantize(f64(x)))
    inside = np.zeros(M, bool)
    for g, (s, e) in enumerate(ref.groups(offs, M)):
        if e == s:
            continue
        inside[s:e] = True
        b = ref.f4_values(*ref.f4_quantize(f64(w[g])))
        want, mag = a[s:e] @ b.T, np.abs(a[s:e]) @ np.abs(b).T
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got[s:e]), nan)
        tol = 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * mag
        bad = np.abs(got[s:e] - want)[~nan] > tol[~nan]
        assert not bad.any(), f"group {g}: {bad.sum()} of {bad.size} outputs outside"
    raw = bits_of(out)
    assert np.all(raw[~inside] == 0xA5A5), "rows in no group were written"


@pytest.mark.parametrize("M,N,K,sizes", [
    (1, 256, 128, [1]),                              # one token, half a stage
    (1, 256, 256, [1]),
    (1, 512, 2176, [0, 0, 1]),                       # more stages than the ring, an odd half
    (9, 256, 384, [3, 0, 5]),                        # one row behind
    (33, 256, 512, [33]),                            # a token tile and one row
    (40, 512, 640, [8, 8, 8, 9, 7]),
    (128, 256, 1024, [31, 1, 0, 96]),                # tiles at every offset of a scale tile
    (150, 256, 256, [1, 140, 9, 0]),                 # a group larger than one scale tile
    (70, 256, 256, [1] * 70),
])
def test_fp4_product_of_few_rows(M, N, K, sizes):
    check_product(M, N, K, np.cumsum(sizes), seed=M + K)


@pytest.mark.parametrize("M,N,K,sizes", [
    (130, 256, 128, [65, 60]),
    (300, 512, 384, [128, 0, 100, 72]),
    (385, 256, 640, [129, 127, 129]),
])
def test_fp4_product_of_some_rows(M, N, K, sizes):
    check_product(M, N, K, np.cumsum(sizes), seed=M + K)


@pytest.mark.parametrize("M,N,K,sizes", [
    (256, 256, 256, [256]),
    (320, 256, 128, [200, 120]),
    # enough units for the 256 x 256 tiles (more than one wave of the 128 x 128 ones)
    (256, 9984, 128, [256]),                         # half a stage
    (1024, 2560, 640, [129, 1, 257, 383, 230]),      # ragged, odd numbers of tiles
    (700, 4096, 1920, [650, 40]),                    # more stages than the ring
    (1037, 2560, 256, [300, 0, 700]),                # rows behind the last group
])
def test_fp4_product_of_many_rows(M, N, K, sizes):
    check_product(M, N, K, np.cumsum(sizes), seed=M + K)


@pytest.mark.parametrize("M,N", [(20, 256), (200, 256), (800, 256), (800, 2560)])
def test_fp4_product_offsets_and_nan(M, N):
    check_product(M, N, 640, [M // 3, M // 4, 5 * M], seed=M, special=True)   # decreasing, then past the end
    check_product(M, N, 384, [-7, 0, M // 2], seed=M, special=True)
    check_product(M, N, 256, [0, 0, 0], seed=M)


def test_fp4_product_more_units_than_processors():
    rng = np.random.default_rng(3)
    for lo, hi, N in ((0, 5, 1024), (40, 130, 512), (100, 300, 512)):
        sizes = rng.integers(lo, hi, size=45)
        sizes[[3, 17, 18, 44]] = 0
        check_product(int(sizes.sum()) + 7, N, 384, np.cumsum(sizes), seed=lo)


def test_fp4_product_many_groups():
    """More groups than the table in shared memory holds, and as many."""
    for G in (1100, 1024):
        sizes = np.zeros(G, int)
        sizes[[0, 3, 700, 1010, G - 1]] = [2, 1, 130, 5, 9]
        check_product(int(sizes.sum()), 256, 128, np.cumsum(sizes))


# ---- a layer ------------------------------------------------------------------------------------------------

def layer(x, res, w, router, experts, k):
    """norm -> router -> plan -> 4-bit product of the routed rows -> weighted sum."""
    T, D = x.shape
    E, N = router.shape[0], experts.shape[1]
    dev = x.device
    o = {n: torch.empty(s, dtype=d, device=dev) for n, s, d in (
        ("q", (T, D), torch.uint8), ("s", (T, D // 32), torch.uint8), ("y", (T, D), BF), ("res_out", (T, D), BF))}
    mxq.rmsnorm_mx_quantize(x, w, 1e-5, residual=res, **o)
    logits = o["y"].float() @ router.T
    wt = torch.empty(T, k, device=dev)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    mxq.moe_route(logits, wt, ids, renorm=True)
    offs = torch.empty(E, dtype=torch.int32, device=dev)
    rows, src = torch.empty_like(ids), torch.empty(T * k, dtype=torch.int32, device=dev)
    need = mxq.moe_plan_workspace_bytes(T * k, E)
    mxq.moe_plan(ids, offs, rows, src, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    tokens = o["y"][src.long() // k]
    qa = torch.empty(T * k, D // 2, dtype=torch.uint8, device=dev)
    sfa = torch.empty(mxq.mx_scales_blocked_bytes(1, T * k, D // 32, E), dtype=torch.uint8, device=dev)
    qb = torch.empty(E, N, D // 2, dtype=torch.uint8, device=dev)
    sfb = torch.empty(mxq.mx_scales_blocked_bytes(E, N, D // 32), dtype=torch.uint8, device=dev)
    mxq.mxfp4_quantize(tokens, qa, sf_blocked=sfa, offs=offs)
    mxq.mxfp4_quantize(experts, qb, sf_blocked=sfb)
    prod = torch.empty(T * k, N, dtype=BF, device=dev)
    mxq.mxfp4_grouped_gemm(qa, sfa, qb, sfb, offs, prod)
    return o, logits, wt, ids, (prod[rows.long()].float() * wt[:, :, None]).sum(1)


@pytest.mark.parametrize("T", [1, 24, 700])
def test_the_operators_together(T):
    D, E, N, k = 512, 16, 256, 3
    g = gen(T)
    x, res, w = norm_inputs(T, D, BF, T)
    router = torch.randn(E, D, generator=g) / D ** 0.5
    experts = (0.05 * torch.randn(E, N, D, generator=g)).to(BF)
    o, logits, wt, ids, out = layer(x.cuda(), res.cuda(), w.cuda(), router.cuda(), experts.cuda(), k)
    rid, rw = ref.route(f64(logits), None, "softmax", 1, 1, 1, k, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), rid)
    y = f64(o["y"])
    a = ref.f4_values(*ref.f4_quantize(y))
    want, tol = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        b = ref.f4_values(*ref.f4_quantize(f64(experts[e])))
        t, j = np.nonzero(rid == e)
        v, m = a[t] @ b.T, np.abs(a[t]) @ np.abs(b).T
        want[t] += v * rw[t, j][:, None]
        tol[t] += rw[t, j][:, None] * (2.0 ** -8 * np.abs(v) + D * 2.0 ** -23 * m + 2.0 ** -16 * np.abs(v))
    # three weighted fp32 terms are added: within 2^-22 of their magnitudes, which 2^-16 covers
    assert np.all(np.abs(f64(out) - want) <= tol)


@pytest.mark.parametrize("T", [40, 5000])
def test_the_operators_in_a_graph_on_their_own_stream(T):
    """The whole chain captured into a CUDA graph and replayed on new inputs."""
    T, D, E, N, k = T, 512, 8, 256, 2
    x, res, w = norm_inputs(T, D, BF, 1)
    g = gen(2)
    router = (torch.randn(E, D, generator=g) / D ** 0.5).cuda()
    experts = (0.05 * torch.randn(E, N, D, generator=g)).to(BF).cuda()
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(xd, rd, wd, router, experts, k)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = layer(xd, rd, wd, router, experts, k)
    for seed in (5, 6):
        x2, r2, _ = norm_inputs(T, D, BF, seed)
        xd.copy_(x2)
        rd.copy_(r2)
        graph.replay()
        torch.cuda.synchronize()
        want = layer(x2.cuda(), r2.cuda(), wd, router, experts, k)
        for a, b in zip((got[0]["q"], got[0]["s"], *got[2:]), (want[0]["q"], want[0]["s"], *want[2:])):
            assert torch.equal(a, b)


def test_the_operators_on_a_given_stream():
    x, r, w = norm_inputs(500, 1024, BF, 9)
    want = gpu_norm(x, r, w, 1e-5)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    o = {n: empty(t.dtype, *t.shape) for n, t in want.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mxq.rmsnorm_mx_quantize(xd, wd, 1e-5, residual=rd, stream=side, **o)
    side.synchronize()
    for n in want:
        assert torch.equal(want[n], o[n])
