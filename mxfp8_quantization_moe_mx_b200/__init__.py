"""B200-native MXFP8 / per-group FP8 quantization for MoE expert-parallel training.

Thin Python binding over the C ABI of ``libmxq.so`` (declared in ``include/mxq.h``).
Functions carry the C names and only marshal arguments: they check that the torch
tensors they are given are CUDA tensors of the right dtype, shape and contiguity,
pass their device pointers and the current CUDA stream to the C entry point, and raise
``MxqError`` on a non-zero status.  Every step of the computation runs in the CUDA
kernels; there is no CPU or PyTorch fallback, and the first call raises if the
library has not been built.

Operations (see include/mxq.h for the exact arithmetic and layouts):
  mx_quantize / mx_dequantize -- the local quantize and dequantize around the MXFP8
    expert-parallel all-to-all (torchtitan "[mxfp8 MoE training] Support mxfp8 all to
    all in expert parallel", Summary).
  fp8_per_group_rowwise_quant -- per-group rowwise FP8 scaling (torchao "[moe
    training] fix uncoalesced global accesses in per group rowwise scaling kernel").
  moe_route / moe_route_backward / moe_plan -- the experts of each token, the gradient of
    the router's logits, and the rows of the grouped products.
  rmsnorm_mx_quantize / rmsnorm_backward -- residual addition, RMS norm and MXFP8 output.
  mxfp4_quantize / mxfp4_dequantize / mxfp4_grouped_gemm -- 4-bit codes and their product.
``mxfp8_quantization_moe_mx_b200.moe`` has the differentiable forms.
"""
from __future__ import annotations

import ctypes
import os

import torch

ROW, COL = 1, 2
ROW_MAJOR, COL_MAJOR = 0, 1
SOFTMAX, SIGMOID = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")
_LIB = None


class MxqError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """Load libmxq.so (built in-tree by ``build.py``).  Raises if it is missing."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise MxqError(f"{LIB_PATH} is missing: build it with "
                           "`python -m mxfp8_quantization_moe_mx_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        L.mx_quantize.argtypes = [vp, i64, i64, i64, ci, vp, vp, vp, vp, vp]
        L.mx_dequantize.argtypes = [vp, vp, i64, i64, i64, ci, vp, vp]
        L.fp8_per_group_rowwise_quant.argtypes = [vp, i64, i64, vp, i32, ci, vp, vp, vp]
        L.mx_e4m3_encode_f32.argtypes = [vp, i64, vp, vp]
        L.mxq_transpose_u8.argtypes = [vp, i64, i64, i64, vp, vp]
        L.mxq_transpose_u8.restype = ci
        L.mx_scales_to_blocked.argtypes = [vp, i64, i64, i64, vp, i32, vp, vp]
        L.mx_scales_to_blocked.restype = ci
        L.mx_scales_blocked_bytes.argtypes = [i64, i64, i64, i32]
        L.mx_scales_blocked_bytes.restype = i64
        L.fp8_per_group_rowwise_quant_batched.argtypes = [vp, i64, i64, i64, ci, vp, vp, vp]
        L.fp8_per_group_rowwise_quant_batched.restype = ci
        L.mx_grouped_gemm.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp]
        L.mx_grouped_gemm.restype = ci
        cf = ctypes.c_float
        L.moe_route.argtypes = [vp, ci, i64, i64, vp, ci, i32, i32, i32, i32, ci, cf, vp, vp, vp]
        L.moe_route_backward.argtypes = [vp, ci, i64, i64, vp, i32, vp, ci, ci, cf, vp, vp]
        L.moe_plan.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.rmsnorm_mx_quantize.argtypes = [vp, vp, vp, ci, i64, i64, cf, vp, vp, vp, vp, vp, vp]
        L.rmsnorm_backward.argtypes = [vp, vp, vp, ci, vp, vp, i64, i64, vp, vp, vp, vp]
        L.mxfp4_quantize.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, i32, vp]
        L.mxfp4_dequantize.argtypes = [vp, vp, i64, i64, vp, vp]
        L.mxfp4_grouped_gemm.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp]
        for f in (L.moe_route, L.moe_route_backward, L.moe_plan, L.rmsnorm_mx_quantize, L.rmsnorm_backward,
                  L.mxfp4_quantize, L.mxfp4_dequantize, L.mxfp4_grouped_gemm):
            f.restype = ci
        L.moe_plan_workspace_bytes.argtypes = L.rmsnorm_backward_workspace_bytes.argtypes = [i64, i64]
        L.moe_plan_workspace_bytes.restype = L.rmsnorm_backward_workspace_bytes.restype = i64
        for f in (L.mx_quantize, L.mx_dequantize, L.fp8_per_group_rowwise_quant,
                  L.mx_e4m3_encode_f32):
            f.restype = ci
        L.mxq_status_string.argtypes = [ci]
        L.mxq_status_string.restype = ctypes.c_char_p
        L.mxq_last_cuda_error.argtypes = []
        L.mxq_last_cuda_error.restype = ctypes.c_char_p
        L.mxq_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.mxq_wait_timeouts.restype = ci
        L.mxq_wait_abandoned.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.mxq_wait_abandoned.restype = ci
        L.mxq_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.mxq_set_wait_limit_ns.restype = ci
        ip = ctypes.POINTER(ci)
        L.fp8_per_group_rowwise_plan.argtypes = [i64, i64, i32, ci, ci, ip, ip, ip, ip, ip]
        L.fp8_per_group_rowwise_plan.restype = ci
        _LIB = L
    return _LIB


def _check(status: int) -> None:
    if status != 0:
        L = lib()
        msg = L.mxq_status_string(status).decode()
        if status == 5:
            msg += ": " + L.mxq_last_cuda_error().decode()
        raise MxqError(msg)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str, numel: int | None = None) -> int:
    if not isinstance(t, torch.Tensor):
        raise MxqError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise MxqError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise MxqError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MxqError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise MxqError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _bsc(x: torch.Tensor):
    if x.dim() == 2:
        return 1, x.shape[0], x.shape[1]
    if x.dim() == 3:
        return x.shape[0], x.shape[1], x.shape[2]
    raise MxqError("expected a (rows, cols) or (batch, rows, cols) tensor")


# ---- MX quantize / dequantize -----------------------------------------------------------

def mx_quantize(x: torch.Tensor, axes: int, q_row=None, s_row=None, q_col=None, s_col=None,
                stream=None) -> None:
    """x: bf16 (rows, cols) or (batch, rows, cols).  Outputs (uint8, preallocated):
    q_row (b, rows, cols), s_row (b, rows, cols/32), q_col (b, cols, rows),
    s_col (b, cols, rows/32)."""
    batch, rows, cols = _bsc(x)
    px = _dev(x, torch.bfloat16, "x")
    n = batch * rows * cols
    pr = sr = pc = sc = None
    if axes & ROW:
        pr = _dev(q_row, torch.uint8, "q_row", n)
        sr = _dev(s_row, torch.uint8, "s_row", n // 32)
    if axes & COL:
        pc = _dev(q_col, torch.uint8, "q_col", n)
        sc = _dev(s_col, torch.uint8, "s_col", n // 32)
    _check(lib().mx_quantize(px, batch, rows, cols, axes, pr, sr, pc, sc, _stream(stream)))


def mx_dequantize(q: torch.Tensor, s: torch.Tensor, batch: int, rows: int, cols: int,
                  axis: int, y: torch.Tensor, stream=None) -> None:
    n = batch * rows * cols
    pq = _dev(q, torch.uint8, "q", n)
    ps = _dev(s, torch.uint8, "s", n // 32)
    py = _dev(y, torch.bfloat16, "y", n)
    _check(lib().mx_dequantize(pq, ps, batch, rows, cols, axis, py, _stream(stream)))


def empty_mx_outputs(x: torch.Tensor, axes: int):
    """Allocate the uint8 outputs mx_quantize writes for ``x`` (device memory)."""
    batch, rows, cols = _bsc(x)
    kw = dict(dtype=torch.uint8, device=x.device)
    out = {}
    if axes & ROW:
        out["q_row"] = torch.empty((batch, rows, cols), **kw)
        out["s_row"] = torch.empty((batch, rows, cols // 32), **kw)
    if axes & COL:
        out["q_col"] = torch.empty((batch, cols, rows), **kw)
        out["s_col"] = torch.empty((batch, cols, rows // 32), **kw)
    return out


# ---- per-group rowwise --------------------------------------------------------------------

def fp8_per_group_rowwise_quant(x: torch.Tensor, offs: torch.Tensor, out_layout: int,
                                q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """x: bf16 (M, K); offs: int32 (G,) end offsets on the device; q: uint8 (M, K) for
    ROW_MAJOR or (K, M) for COL_MAJOR; scales: fp32 (G, K)."""
    if x.dim() != 2:
        raise MxqError("x must be (M, K)")
    M, K = x.shape
    G = offs.numel()
    px = _dev(x, torch.bfloat16, "x")
    po = _dev(offs, torch.int32, "offs")
    pq = _dev(q, torch.uint8, "q", M * K)
    ps = _dev(scales, torch.float32, "scales", G * K)
    _check(lib().fp8_per_group_rowwise_quant(px, M, K, po, G, out_layout, pq, ps, _stream(stream)))


def fp8_per_group_rowwise_quant_batched(x: torch.Tensor, out_layout: int, q: torch.Tensor, scales: torch.Tensor,
                                        stream=None) -> None:
    """x: bf16 (E, M, K), every matrix its own group; q: uint8 (E, M, K) for ROW_MAJOR or
    (E, K, M) for COL_MAJOR; scales: fp32 (E, K)."""
    if x.dim() != 3:
        raise MxqError("x must be (E, M, K)")
    E, M, K = x.shape
    px = _dev(x, torch.bfloat16, "x")
    pq = _dev(q, torch.uint8, "q", E * M * K)
    ps = _dev(scales, torch.float32, "scales", E * K)
    _check(lib().fp8_per_group_rowwise_quant_batched(px, E, M, K, out_layout, pq, ps, _stream(stream)))


def mx_e4m3_encode_f32(x: torch.Tensor, q: torch.Tensor, stream=None) -> None:
    """fp32 -> E4M3 with the convert every kernel uses (RNE, saturating to 448)."""
    n = x.numel()
    px = _dev(x, torch.float32, "x")
    pq = _dev(q, torch.uint8, "q", n)
    _check(lib().mx_e4m3_encode_f32(px, n, pq, _stream(stream)))


PLAN_KERNELS = {0: "none", 1: "tile", 2: "pair", 3: "stream"}


def fp8_per_group_rowwise_plan(M: int, K: int, G: int, out_layout: int, n_sm: int = 0) -> dict:
    """The kernel and tile shape fp8_per_group_rowwise_quant launches for these sizes
    (host only).  Returns {kernel, slab_cols, cluster, tile_rows, threads}."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    _check(lib().fp8_per_group_rowwise_plan(M, K, G, out_layout, n_sm, *[ctypes.byref(v) for v in vals]))
    kernel, w, cl, rows, threads = (v.value for v in vals)
    return {"kernel": PLAN_KERNELS[kernel], "slab_cols": w, "cluster": cl, "tile_rows": rows, "threads": threads}


WAIT_LIMIT_DEFAULT_NS = 2_000_000_000


def mxq_wait_timeouts() -> int:
    """Number of kernel CTAs that gave up a bounded wait since the library was loaded
    (0 in a healthy run).  Synchronizes the device."""
    n = ctypes.c_uint(0)
    _check(lib().mxq_wait_timeouts(ctypes.byref(n)))
    return n.value


def mxq_wait_abandoned() -> int:
    """Of those, the CTAs whose copies in flight did not land after giving up either
    (0 in a healthy run).  Synchronizes the device."""
    n = ctypes.c_uint(0)
    _check(lib().mxq_wait_abandoned(ctypes.byref(n)))
    return n.value


def mxq_set_wait_limit_ns(ns: int) -> None:
    """Limit of the bounded waits of the per-group kernels and the norm's gradient for later
    launches (0: give up at once, to exercise the give-up path)."""
    _check(lib().mxq_set_wait_limit_ns(int(ns)))


# ---- layouts for the scaled grouped GEMM ---------------------------------------------------

def mxq_transpose_u8(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """uint8 (rows, cols) or (batch, rows, cols) -> dst (.., cols, rows)."""
    batch, rows, cols = _bsc(src)
    ps = _dev(src, torch.uint8, "src")
    pd = _dev(dst, torch.uint8, "dst", batch * rows * cols)
    _check(lib().mxq_transpose_u8(ps, batch, rows, cols, pd, _stream(stream)))


def mx_scales_blocked_bytes(batch: int, rows: int, n_k: int, G: int = 0) -> int:
    n = int(lib().mx_scales_blocked_bytes(batch, rows, n_k, G))
    if n < 0:
        raise MxqError("invalid sizes for the blocked scale layout")
    return n


def mx_scales_to_blocked(s: torch.Tensor, out: torch.Tensor, offs: torch.Tensor | None = None,
                         stream=None) -> None:
    """E8M0 scales uint8 (rows, n_k) or (batch, rows, n_k) -> out (flat uint8 of
    mx_scales_blocked_bytes), tiled for the block-scaled MMA; with offs (int32 end
    offsets on the device) every group's rows padded to whole 128-row tiles."""
    batch, rows, n_k = _bsc(s)
    G = 0 if offs is None else offs.numel()
    ps = _dev(s, torch.uint8, "s")
    po = None if offs is None else _dev(offs, torch.int32, "offs")
    pout = _dev(out, torch.uint8, "out")
    if out.numel() < mx_scales_blocked_bytes(batch, rows, n_k, G):
        raise MxqError("out is smaller than mx_scales_blocked_bytes")
    _check(lib().mx_scales_to_blocked(ps, batch, rows, n_k, po, G, pout, _stream(stream)))


# ---- MXFP8 grouped GEMM -------------------------------------------------------------------------

def mx_grouped_gemm(qa: torch.Tensor, sfa_blocked: torch.Tensor, qb: torch.Tensor, sfb_blocked: torch.Tensor,
                    offs: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """qa uint8 (M, K) E4M3 tokens; sfa_blocked: their scales from mx_scales_to_blocked
    with offs; qb uint8 (G, N, K) expert weights; sfb_blocked: their scales from
    mx_scales_to_blocked (per matrix); offs int32 (G,) end offsets; out bf16 (M, N)."""
    if qa.dim() != 2 or qb.dim() != 3:
        raise MxqError("qa must be (M, K) and qb (G, N, K)")
    M, K = qa.shape
    G, N, K2 = qb.shape
    if K2 != K or offs.numel() != G:
        raise MxqError("qa, qb and offs disagree on K or G")
    pa = _dev(qa, torch.uint8, "qa")
    pb = _dev(qb, torch.uint8, "qb")
    psa = _dev(sfa_blocked, torch.uint8, "sfa_blocked")
    psb = _dev(sfb_blocked, torch.uint8, "sfb_blocked")
    if sfa_blocked.numel() < mx_scales_blocked_bytes(1, M, K // 32, G):
        raise MxqError("sfa_blocked is smaller than mx_scales_blocked_bytes(1, M, K/32, G)")
    if sfb_blocked.numel() < mx_scales_blocked_bytes(G, N, K // 32, 0):
        raise MxqError("sfb_blocked is smaller than mx_scales_blocked_bytes(G, N, K/32, 0)")
    po = _dev(offs, torch.int32, "offs")
    pout = _dev(out, torch.bfloat16, "out", M * N)
    _check(lib().mx_grouped_gemm(pa, psa, pb, psb, po, G, M, N, K, pout, _stream(stream)))


# ---- the operators of a mixture-of-experts layer --------------------------------------------------

def _refuse(t, dtype, name: str, numel, dev: int) -> None:
    """Raise what is wrong with an argument that _arg has not accepted."""
    _dev(t, dtype, name, numel)
    raise MxqError(f"{name} is on {t.device}, the other tensors are on cuda:{dev}")


def _arg(t: torch.Tensor, dtype, name: str, numel: int, dev: int) -> int:
    """The pointer of a contiguous tensor of numel elements on CUDA device dev."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() == numel and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, name, numel, dev)


def _opt(t, dtype, name: str, numel: int, dev: int):
    return None if t is None else _arg(t, dtype, name, numel, dev)


def _first(t: torch.Tensor, name: str) -> int:
    """The device of a call: that of its first tensor."""
    try:
        dev = t.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        raise MxqError(f"{name} must be a CUDA tensor")
    return dev


def _type_of(t, name: str) -> int:
    d = getattr(t, "dtype", None)
    if d is torch.bfloat16:
        return 0
    if d is torch.float32:
        return 1
    raise MxqError(f"{name} must be a bfloat16 or float32 tensor")


_DTYPES = (torch.bfloat16, torch.float32)
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(f, dev: int, stream, *args) -> None:
    """f(*args, stream) on device dev: on its current stream unless one is given."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = f(*args, _stream(stream))
    elif stream is None and _RAW_STREAM is not None:
        status = f(*args, _RAW_STREAM(dev))
    else:
        status = f(*args, _stream(stream))
    if status:
        _check(status)


def _tiles_bytes(batch: int, rows: int, n_k: int, G: int) -> int:
    """mx_scales_blocked_bytes, for sizes that the call itself checks."""
    tiles = (rows + 127 * G) // 128 if G else batch * ((rows + 127) // 128)
    return tiles * ((n_k + 3) // 4) * 512


def _two(t: torch.Tensor, name: str, what: str) -> tuple[int, int]:
    try:
        rows, cols = t.shape
    except (AttributeError, ValueError):
        raise MxqError(f"{name} must be {what}") from None
    return rows, cols


def moe_route(logits: torch.Tensor, weights: torch.Tensor, ids: torch.Tensor, bias: torch.Tensor | None = None,
              score: int = SOFTMAX, n_groups: int = 1, top_groups: int = 1, group_top: int = 1,
              renorm: bool = False, scale: float = 1.0, stream=None) -> None:
    """logits bf16 or fp32 (T, E); bias fp32 (E,) or None; weights fp32 (T, k) and ids int32
    (T, k) receive the k experts of each token and their weights."""
    T, E = _two(logits, "logits", "(T, E)")
    k = _two(ids, "ids", "(T, k)")[1]
    dev, ty = _first(logits, "logits"), _type_of(logits, "logits")
    _run(lib().moe_route, dev, stream, _arg(logits, _DTYPES[ty], "logits", T * E, dev), ty, T, E,
         _opt(bias, torch.float32, "bias", E, dev), score, n_groups, top_groups, group_top, k, 1 if renorm else 0,
         scale, _arg(weights, torch.float32, "weights", T * k, dev), _arg(ids, torch.int32, "ids", T * k, dev))


def moe_route_backward(logits: torch.Tensor, ids: torch.Tensor, grad_weights: torch.Tensor,
                       grad_logits: torch.Tensor, score: int = SOFTMAX, renorm: bool = False, scale: float = 1.0,
                       stream=None) -> None:
    """The gradient of moe_route's logits: logits and ids as there, grad_weights fp32
    (T, k), grad_logits (T, E) of the logits' type (written whole)."""
    T, E = _two(logits, "logits", "(T, E)")
    k = _two(ids, "ids", "(T, k)")[1]
    dev, ty = _first(logits, "logits"), _type_of(logits, "logits")
    _run(lib().moe_route_backward, dev, stream, _arg(logits, _DTYPES[ty], "logits", T * E, dev), ty, T, E,
         _arg(ids, torch.int32, "ids", T * k, dev), k, _arg(grad_weights, torch.float32, "grad_weights", T * k, dev),
         score, 1 if renorm else 0, scale, _arg(grad_logits, _DTYPES[ty], "grad_logits", T * E, dev))


def moe_plan_workspace_bytes(n: int, E: int) -> int:
    b = lib().moe_plan_workspace_bytes(n, E)
    if b < 0:
        raise MxqError("invalid sizes for moe_plan")
    return b


def moe_plan(ids: torch.Tensor, offs: torch.Tensor, rows: torch.Tensor, src: torch.Tensor,
             workspace: torch.Tensor | None = None, stream=None) -> None:
    """ids int32 (any shape, n slots); offs int32 (E,) receives the experts' end offsets,
    rows int32 (n) the row of each slot, src int32 (n) the slot of each row; workspace
    uint8 of moe_plan_workspace_bytes(n, E) (None where that is 0)."""
    dev = _first(ids, "ids")
    n, E = ids.numel(), offs.numel()
    size = 0 if workspace is None else workspace.numel()
    if size < moe_plan_workspace_bytes(n, E):
        raise MxqError("workspace is smaller than moe_plan_workspace_bytes")
    i32 = torch.int32
    _run(lib().moe_plan, dev, stream, _arg(ids, i32, "ids", n, dev), n, E, _arg(offs, i32, "offs", E, dev),
         _arg(rows, i32, "rows", n, dev), _arg(src, i32, "src", n, dev),
         _opt(workspace, torch.uint8, "workspace", size, dev))


def rmsnorm_mx_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float, q: torch.Tensor, s: torch.Tensor,
                        residual: torch.Tensor | None = None, res_out: torch.Tensor | None = None,
                        y: torch.Tensor | None = None, rstd: torch.Tensor | None = None, stream=None) -> None:
    """x, residual bf16 (M, D); weight bf16 or fp32 (D,); q uint8 (M, D) and s uint8
    (M, D/32) receive the MXFP8 norm of x + residual; optional outputs: res_out bf16 (M, D)
    the sum (may be x or residual itself), y bf16 (M, D) the norm, rstd fp32 (M,)."""
    M, D = _two(x, "x", "(M, D)")
    dev, ty, n = _first(x, "x"), _type_of(weight, "weight"), M * D
    bf, u8 = torch.bfloat16, torch.uint8
    _run(lib().rmsnorm_mx_quantize, dev, stream, _arg(x, bf, "x", n, dev), _opt(residual, bf, "residual", n, dev),
         _arg(weight, _DTYPES[ty], "weight", D, dev), ty, M, D, eps, _opt(res_out, bf, "res_out", n, dev),
         _opt(y, bf, "y", n, dev), _arg(q, u8, "q", n, dev), _arg(s, u8, "s", n // 32, dev),
         _opt(rstd, torch.float32, "rstd", M, dev))


def rmsnorm_backward_workspace_bytes(M: int, D: int) -> int:
    b = lib().rmsnorm_backward_workspace_bytes(M, D)
    if b < 0:
        raise MxqError("invalid sizes for rmsnorm_backward")
    return b


def rmsnorm_backward(grad_y: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     grad_x: torch.Tensor, grad_weight: torch.Tensor, workspace: torch.Tensor,
                     grad_res: torch.Tensor | None = None, stream=None) -> None:
    """grad_y, h (the forward pass's res_out, or its x), grad_res bf16 (M, D); rstd fp32
    (M,); grad_x bf16 (M, D) and grad_weight fp32 (D,) receive the gradients; workspace
    uint8 of rmsnorm_backward_workspace_bytes(M, D)."""
    M, D = _two(grad_y, "grad_y", "(M, D)")
    dev, ty, n = _first(grad_y, "grad_y"), _type_of(weight, "weight"), M * D
    bf, f32 = torch.bfloat16, torch.float32
    size = workspace.numel()
    if size < rmsnorm_backward_workspace_bytes(M, D):
        raise MxqError("workspace is smaller than rmsnorm_backward_workspace_bytes")
    _run(lib().rmsnorm_backward, dev, stream, _arg(grad_y, bf, "grad_y", n, dev), _arg(h, bf, "h", n, dev),
         _arg(weight, _DTYPES[ty], "weight", D, dev), ty, _arg(rstd, f32, "rstd", M, dev),
         _opt(grad_res, bf, "grad_res", n, dev), M, D, _arg(grad_x, bf, "grad_x", n, dev),
         _arg(grad_weight, f32, "grad_weight", D, dev), _arg(workspace, torch.uint8, "workspace", size, dev))


def mxfp4_quantize(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor | None = None,
                   sf_blocked: torch.Tensor | None = None, offs: torch.Tensor | None = None, stream=None) -> None:
    """x bf16 (rows, cols) or (batch, rows, cols) -> q uint8 (.., cols/2) E2M1 code pairs,
    with the E8M0 scales plain in s uint8 (.., cols/32), or in the tensor cores' tiles in
    sf_blocked uint8 (mx_scales_blocked_bytes), or both; with offs (int32 end offsets) the
    tiles are laid out per group, and rows in no group are left out."""
    batch, rows, cols = _bsc(x)
    dev, n, u8 = _first(x, "x"), batch * rows * cols, torch.uint8
    G = 0 if offs is None else offs.numel()
    size = 0
    if sf_blocked is not None:
        size = sf_blocked.numel()
        if size < _tiles_bytes(batch, rows, cols // 32, G):
            raise MxqError("sf_blocked is smaller than mx_scales_blocked_bytes")
    elif s is None:
        raise MxqError("mxfp4_quantize needs s or sf_blocked for the scales")
    if offs is not None and (sf_blocked is None or G == 0):
        raise MxqError("offs needs sf_blocked and at least one group")
    _run(lib().mxfp4_quantize, dev, stream, _arg(x, torch.bfloat16, "x", n, dev), batch, rows, cols,
         _arg(q, u8, "q", n // 2, dev), _opt(s, u8, "s", n // 32, dev), _opt(sf_blocked, u8, "sf_blocked", size, dev),
         _opt(offs, torch.int32, "offs", G, dev), G)


def mxfp4_dequantize(q: torch.Tensor, s: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """q uint8 (.., cols/2) and s uint8 (.., cols/32) from mxfp4_quantize -> y bf16
    (rows, cols) or (batch, rows, cols)."""
    batch, rows, cols = _bsc(y)
    dev, n = _first(y, "y"), batch * rows * cols
    _run(lib().mxfp4_dequantize, dev, stream, _arg(q, torch.uint8, "q", n // 2, dev),
         _arg(s, torch.uint8, "s", n // 32, dev), batch * rows, cols, _arg(y, torch.bfloat16, "y", n, dev))


def mxfp4_grouped_gemm(qa: torch.Tensor, sfa_blocked: torch.Tensor, qb: torch.Tensor, sfb_blocked: torch.Tensor,
                       offs: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """qa uint8 (M, K/2) tokens and sfa_blocked their scales, from mxfp4_quantize with offs;
    qb uint8 (G, N, K/2) expert matrices and sfb_blocked their scales, from mxfp4_quantize;
    offs int32 (G,) end offsets; out bf16 (M, N)."""
    if qa.dim() != 2 or qb.dim() != 3:
        raise MxqError("qa must be (M, K/2) and qb (G, N, K/2)")
    M, Kb = qa.shape
    G, N, Kb2 = qb.shape
    if Kb2 != Kb or offs.numel() != G:
        raise MxqError("qa, qb and offs disagree on K or G")
    K, dev, u8 = 2 * Kb, _first(qa, "qa"), torch.uint8
    na, nb = sfa_blocked.numel(), sfb_blocked.numel()
    if na < _tiles_bytes(1, M, K // 32, G):
        raise MxqError("sfa_blocked is smaller than mx_scales_blocked_bytes(1, M, K/32, G)")
    if nb < _tiles_bytes(G, N, K // 32, 0):
        raise MxqError("sfb_blocked is smaller than mx_scales_blocked_bytes(G, N, K/32, 0)")
    _run(lib().mxfp4_grouped_gemm, dev, stream, _arg(qa, u8, "qa", M * Kb, dev),
         _arg(sfa_blocked, u8, "sfa_blocked", na, dev), _arg(qb, u8, "qb", G * N * Kb, dev),
         _arg(sfb_blocked, u8, "sfb_blocked", nb, dev), _arg(offs, torch.int32, "offs", G, dev), G, M, N, K,
         _arg(out, torch.bfloat16, "out", M * N, dev))
