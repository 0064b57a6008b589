"""One kernel launched from two host threads at once, at two sizes that want different amounts
of shared memory: no launch is refused, and the results are those of one thread.

The threads call the C ABI itself, so that little but the launches runs between the calls."""
import threading

import numpy as np
import pytest
import torch

import mxfp8_quantization_moe_mx_b200 as mxq
from _gpu import ensure_lib

pytestmark = pytest.mark.gpu
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
CALLS = 4000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def at_once(jobs):
    """jobs: (call on a raw stream -> status, its outputs).  Each alone, then all at once, CALLS
    times each; the same bits."""
    L, device = mxq.lib(), torch.cuda.current_device()
    streams = [torch.cuda.Stream() for _ in jobs]
    want = []
    for (call, outs), s in zip(jobs, streams):
        s.wait_stream(torch.cuda.current_stream())
        assert call(s.cuda_stream) == 0, L.mxq_last_cuda_error()
        s.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.view(U8).fill_(0xA5)
    torch.cuda.synchronize()
    start, refused = threading.Barrier(len(jobs)), [0] * len(jobs)

    def work(i):
        torch.cuda.set_device(device)
        call, raw = jobs[i][0], streams[i].cuda_stream
        start.wait()
        for _ in range(CALLS):
            refused[i] += call(raw) != 0

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(jobs)
    for (_, outs), w in zip(jobs, want):
        assert all(torch.equal(o.view(U8), v.view(U8)) for o, v in zip(outs, w))


def norm_gradient(M, D, seed):
    L, g = mxq.lib(), gen(seed)
    gy, h, gres = (torch.randn(M, D, generator=g).to(BF).cuda() for _ in range(3))
    w, r = (1 + torch.rand(n, generator=g).cuda() for n in (D, M))
    gx, gw = torch.empty_like(h), torch.empty(D, device="cuda")
    ws = torch.empty(mxq.rmsnorm_backward_workspace_bytes(M, D), dtype=U8, device="cuda")
    p = [t.data_ptr() for t in (gy, h, w, r, gres, gx, gw, ws)]

    def call(raw, keep=(gy, h, w, r, gres, ws)):
        return L.rmsnorm_backward(p[0], p[1], p[2], 1, p[3], p[4], M, D, p[5], p[6], p[7], raw)
    return call, [gx, gw]


def plan(n, E, seed):
    L = mxq.lib()
    ids = torch.randint(-1, E, (n,), generator=gen(seed), dtype=I32).cuda()
    offs, rows, src = (torch.empty(m, dtype=I32, device="cuda") for m in (E, n, n))

    def call(raw, keep=ids):
        return L.moe_plan(ids.data_ptr(), n, E, offs.data_ptr(), rows.data_ptr(), src.data_ptr(), None, raw)
    return call, [offs, rows, src]


def route(T, E, n_groups, seed):
    L, k = mxq.lib(), 8
    x = torch.randn(T, E, generator=gen(seed)).cuda()
    b = (0.1 * torch.randn(E, generator=gen(seed + 1))).cuda()
    w, ids = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=I32, device="cuda")

    def call(raw, keep=(x, b)):
        return L.moe_route(x.data_ptr(), 1, T, E, b.data_ptr(), mxq.SIGMOID, n_groups, 2, 2, k, 1, 1.0, w.data_ptr(),
                           ids.data_ptr(), raw)
    return call, [w, ids]

def per_group(M, K, G, seed):
    L = mxq.lib()
    x = torch.randn(M, K, generator=gen(seed)).to(BF).cuda()
    offs = (torch.arange(1, G + 1, dtype=I32) * (M // G)).cuda()
    q, s = torch.empty(M, K, dtype=U8, device="cuda"), torch.empty(G, K, device="cuda")

    def call(raw, keep=(x, offs)):
        return L.fp8_per_group_rowwise_quant(x.data_ptr(), M, K, offs.data_ptr(), G, mxq.ROW_MAJOR, q.data_ptr(),
                                             s.data_ptr(), raw)
    return call, [q, s]


def test_norm_gradients():
    # 600 rows: more than one per CTA, so that the order of the weight gradient's sums is the grid's
    at_once([norm_gradient(8, 16384, 1), norm_gradient(600, 1056, 2)])


def test_plans():
    at_once([plan(500, 1024, 3), plan(300, 400, 4)])


def test_grouped_routing():
    at_once([route(16, 1024, 8, 5), route(16, 768, 8, 6)])


def test_per_group():
    sizes = (1150, 64, 2), (800, 64, 2)  # 575 and 400 rows a group: 80 and 58 KB of tile
    for M, K, G in sizes:
        plan = mxq.fp8_per_group_rowwise_plan(M, K, G, mxq.ROW_MAJOR)
        assert (plan["kernel"], plan["slab_cols"], plan["cluster"]) == ("tile", 64, 1), plan
    at_once([per_group(*size, seed) for seed, size in enumerate(sizes)])
