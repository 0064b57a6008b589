"""A padded batch through a mixture-of-experts layer, written as the package's documentation
writes it: slots that are routed nowhere have row -1, and the products leave the rows behind
the last group unwritten, whatever lies there.  The steps are taken from the documentation's
own text, so that what it says is what runs."""
import inspect
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import _moe_ref as ref
from mxfp8_quantization_moe_mx_b200 import moe

BF = torch.bfloat16


def documented_steps():
    """The layer in the module's documentation, as lines of Python."""
    lines = inspect.cleandoc(moe.__doc__).splitlines()
    first = next(i for i, line in enumerate(lines) if line.startswith("    n = "))
    last = next(i for i, line in enumerate(lines) if line.startswith("    y = "))
    return [line.strip() for line in lines[first:last + 1]]


def combine(out, rows, weights):
    """The steps behind the product."""
    steps = documented_steps()
    names = {"out": out, "p": SimpleNamespace(rows=rows), "weights": weights}
    exec("\n".join(steps[1 + next(i for i, s in enumerate(steps) if s.startswith("out = ")):]), names)
    return names["y"]


@pytest.mark.parametrize("spoilt", [float("nan"), float("inf")])
def test_the_combination_ignores_rows_that_no_product_wrote(spoilt):
    out = torch.randn(6, 8, generator=torch.Generator().manual_seed(1))
    rows = torch.tensor([[2, 0], [-1, -1], [1, -1]], dtype=torch.int32)
    weights = torch.tensor([[0.75, 0.25], [0.0, 0.0], [1.0, 0.0]])
    out[3:] = spoilt
    out, weights = out.requires_grad_(), weights.requires_grad_()
    y = combine(out, rows, weights)
    want = torch.stack([0.75 * out[2] + 0.25 * out[0], torch.zeros(8), out[1]])
    assert torch.equal(y, want)
    y.sum().backward()
    assert (out.grad[3:] == 0).all() and torch.isfinite(out.grad).all() and torch.isfinite(weights.grad).all()


def test_the_combination_of_a_batch_without_any_routed_slot():
    y = combine(torch.full((4, 8), float("nan")), torch.full((2, 2), -1, dtype=torch.int32), torch.zeros(2, 2))
    assert (y == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 24, 700])
def test_a_padded_batch(T):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from _gpu import ensure_lib

    ensure_lib()
    D, E, N, k = 512, 16, 256, 3
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=g).to(BF).cuda()
    weight = torch.ones(D, device="cuda")
    router = (torch.randn(E, D, generator=g) / D ** 0.5).cuda()
    mats = (0.05 * torch.randn(E, N, D, generator=g)).to(BF).cuda()
    pad = torch.arange(T, device="cuda") % 4 == 3  # whole tokens
    few = torch.arange(T, device="cuda") % 4 == 1  # tokens that may go to one expert only
    seen = []

    def route(logits, k, **how):
        logits = logits.masked_fill(pad[:, None], float("-inf"))
        one = few[:, None] & (torch.arange(E, device="cuda") != 2)
        seen.append(logits.masked_fill(one, float("-inf")))
        return moe.route(seen[0], k, **how)

    experts = moe.Mxfp4Experts(mats)
    names = {"moe": SimpleNamespace(rmsnorm=moe.rmsnorm, plan=moe.plan, route=route), "x": x, "weight": weight,
             "stream": x, "router": router, "k": k, "E": E,
             "experts": lambda rows, offs: experts(rows, offs, out=torch.full((T * k, N), float("nan"), dtype=BF,
                                                                              device="cuda"))}
    exec("\n".join(documented_steps()), names)
    y = names["y"].double().cpu().numpy()
    assert (y[pad.cpu().numpy()] == 0).all()

    rid, rw = ref.route(seen[0].double().cpu().numpy(), None, "softmax", 1, 1, 1, k, True, 1.0)
    assert np.array_equal(names["ids"].cpu().numpy(), rid) and (rid < 0).any() and (rid >= 0).any()
    a = ref.f4_values(*ref.f4_quantize(names["n"].y.double().cpu().numpy()))
    want, tol = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        b = ref.f4_values(*ref.f4_quantize(mats[e].double().cpu().numpy()))
        t, j = np.nonzero(rid == e)
        v, m = a[t] @ b.T, np.abs(a[t]) @ np.abs(b).T
        want[t] += v * rw[t, j][:, None]
        # half a step of bf16, fp32 accumulation of D terms, and the weight's and the sum's fp32
        tol[t] += rw[t, j][:, None] * (2.0 ** -8 * np.abs(v) + D * 2.0 ** -23 * m + 2.0 ** -16 * np.abs(v))
    assert np.all(np.abs(y - want) <= tol)
