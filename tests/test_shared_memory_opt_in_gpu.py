"""Sizes whose dynamic shared memory stays below 48 KB while, with the kernel's static shared
memory, it passes them: the launch needs the opt-in to larger shared memory all the same.

The opt-in belongs to the kernel and outlives the call, so that an earlier call of a larger
size would hide a missing one: every family of cases runs in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))


def routing():
    """64 E bytes a CTA for the groups, and 3456 static: 714 experts fit, 715 to 736 do not
    (64 * 736 = 46 KB)."""
    import torch

    from test_moe_gpu import check_route, gen

    for dt in (torch.float32, torch.bfloat16):
        for E, n_groups in ((714, 7), (715, 5), (720, 8), (736, 8), (744, 8)):
            x = (2.0 * torch.randn(9, E, generator=gen(E))).to(dt)
            b = 0.2 * torch.randn(E, generator=gen(E + 1))
            check_route(x, 8, b, score="sigmoid", n_groups=n_groups, top_groups=3, group_top=2, renorm=True)

def per_group():
    """Average group sizes whose tile, with 288 to 1840 bytes of static memory, passes 48 KB."""
    import numpy as np

    import mxfp8_quantization_moe_mx_b200 as mxq
    import oracle
    from _gpu import bits_of, gpu_per_group, same_f32
    from mxfp8_quantization_moe_mx_b200 import workloads as wl

    for n, G, layout, width, cluster in ((2400, 3, mxq.ROW_MAJOR, 64, 8), (5460, 2, mxq.ROW_MAJOR, 32, 8),
                                         (2849, 3, mxq.COL_MAJOR, 16, 2), (5460, 2, mxq.COL_MAJOR, 32, 8),
                                         (5740, 2, mxq.COL_MAJOR, 16, 4), (11500, 2, mxq.COL_MAJOR, 16, 8)):
        M, K = n * G, 96
        plan = mxq.fp8_per_group_rowwise_plan(M, K, G, layout)
        assert (plan["kernel"], plan["slab_cols"], plan["cluster"]) == ("tile", width, cluster), plan
        x = wl.stress(seed=n, M=M, K=K, n_groups=3, n_empty=0)["x"]
        offs = (n * np.arange(1, G + 1)).astype(np.int32)
        qr, sr = oracle.per_group_quant(bits_of(x), offs, layout)
        q, s = gpu_per_group(x, offs, layout)
        assert same_f32(s, sr) and np.array_equal(q, qr), (n, G, layout)


def run(family):
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    code = (f"import sys; sys.path[:0] = [{TESTS!r}, {os.path.dirname(TESTS)!r}]\n"
            f"from _gpu import ensure_lib; ensure_lib()\n"
            f"import test_shared_memory_opt_in_gpu as t; t.{family}()")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_grouped_routing_first_in_a_process():
    run("routing")


def test_per_group_first_in_a_process():
    run("per_group")
