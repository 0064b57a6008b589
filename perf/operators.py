"""The operators around a mixture-of-experts layer: what is measured, and their plain forms.

  route    scores of a router -> the k experts of each token and their weights, with the
           gradient of the logits
  plan     the experts of each token -> end offsets of the experts' groups of rows, and
           the row of every (token, slot) and back
  norm     residual addition, root-mean-square norm and MXFP8 quantization of the result,
           with the gradients
  fp4      MXFP4 quantization and back to bf16 (the values the 4-bit codes stand for)
  experts  the tokens' MXFP4 quantization and their product with the MXFP4 matrices of
           their experts

`run` computes an operator in elementary torch operations where `own` is false and with
this package's calls where it is true.
"""
import math

import torch

own = False

F4_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- the cases ----------------------------------------------------------------------------------

def _route(name, T, E, k, score, bias, groups, keep, group_top, renorm, scale, dtype, grad, masked):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "keep": keep, "group_top": group_top, "renorm": renorm, "scale": scale, "dtype": dtype, "grad": grad,
            "masked": masked}


def listed():
    return [
        # eight sequences that each decode one token; the call is all latency
        _route("route-step", 8, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, "bf16", False, False),
        # local batch 8 x sequence 8192 tokens, node-limited choice with a balancing bias
        _route("route-groups", 65536, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "f32", False, False),
        # a training step's forward and backward pass, some experts masked, some tokens padding
        _route("route-train", 16640, 128, 6, "softmax", False, 1, 1, 1, False, 1.0, "bf16", True, True),
        # the rows of a decoding step's tokens
        {"name": "plan-step", "op": "plan", "T": 8, "k": 8, "E": 128, "padding": 0.0},
        # the rows of a training batch, one token in fifty padding
        {"name": "plan-batch", "op": "plan", "T": 65536, "k": 8, "E": 256, "padding": 0.02},
        # thirteen decoding sequences, the norm before the router (it reads y in bf16 too)
        {"name": "norm-step", "op": "norm", "M": 13, "D": 5120, "residual": True, "y": True, "wtype": "bf16",
         "grad": False},
        # the dispatch payload of a training step: local batch 8 x sequence 8192, dim 5120
        {"name": "norm-batch", "op": "norm", "M": 65536, "D": 5120, "residual": True, "y": False, "wtype": "bf16",
         "grad": False},
        # the backward pass of a norm with a gradient on its residual stream
        {"name": "norm-grad", "op": "norm", "M": 16640, "D": 5120, "residual": True, "y": True, "wtype": "f32",
         "grad": True},
        # tokens to 4 bits and back
        {"name": "fp4-tokens", "op": "fp4", "batch": 1, "rows": 16640, "cols": 5120},
        # sixteen experts' weights to 4 bits and back
        {"name": "fp4-weights", "op": "fp4", "batch": 16, "rows": 8192, "cols": 5120},
        # a decoding step: 24 rows over 16 experts, every expert's weights read once
        {"name": "experts-step", "op": "experts", "M": 24, "G": 16, "N": 8192, "K": 5120, "rest": 0},
        # a ragged batch over 16 experts, three rows behind the last group
        {"name": "experts-batch", "op": "experts", "M": 16411, "G": 16, "N": 8192, "K": 5120, "rest": 3},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("route", "plan", "norm", "fp4", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log(rng, 4, 512 // groups)
        T = _log(rng, 1, min(65536, 65536 * 256 // E))
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(10, E // groups * keep))
        c = _route("", T, E, k, rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, groups, keep,
                   rng.randint(1, 2), rng.random() < 0.5, rng.choice((1.0, 2.5)), rng.choice(("bf16", "f32")),
                   rng.random() < 0.5, rng.random() < 0.3)
        del c["name"]
        return c
    if op == "plan":
        return {"op": "plan", "T": _log(rng, 4, 65536), "k": rng.randint(1, 8), "E": _log(rng, 8, 512),
                "padding": rng.choice((0.0, 0.02, 0.25))}
    if op == "norm":
        D = 32 * _log(rng, 16, 512)
        grad = rng.random() < 0.4
        return {"op": "norm", "M": _log(rng, 1, min(65536, (16640 if grad else 65536) * 5120 // D)), "D": D,
                "residual": rng.random() < 0.7, "y": rng.random() < 0.5, "wtype": rng.choice(("bf16", "f32")),
                "grad": grad}
    if op == "fp4":
        cols = 32 * _log(rng, 4, 512)
        batch = rng.choice((1, 1, 3, 8))
        return {"op": "fp4", "batch": batch, "rows": _log(rng, 1, min(65536, 8192 * 16 * 5120 // (cols * batch))),
                "cols": cols}
    N, K = 256 * _log(rng, 4, 32), 128 * _log(rng, 8, 64)
    G = _log(rng, 1, min(64, 16 * 8192 * 5120 // (N * K)))
    M = _log(rng, 1, min(16384, 16384 * 8192 * 5120 // (N * K)))
    return {"op": "experts", "M": M, "G": G, "N": N, "K": K, "rest": min(M // 2, rng.choice((0, 0, 1, 17)))}


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        b = T * E * size + 8 * T * k + (4 * E if case["bias"] else 0)
        if case["grad"]:
            b += T * E * size + 4 * T * k
        return {"bytes": b, "flops": (8 if case["grad"] else 4) * T * E}
    if op == "plan":
        n = case["T"] * case["k"]
        return {"bytes": 12 * n + 4 * case["E"], "flops": 0}
    if op == "norm":
        n, M, D = case["M"] * case["D"], case["M"], case["D"]
        w = D * (2 if case["wtype"] == "bf16" else 4)
        if case["grad"]:  # grad_y, h, grad_x, and the residual stream's gradient; grad_weight in 32 bits
            return {"bytes": n * (6 + (2 if case["residual"] else 0)) + 4 * M + w + 4 * D, "flops": 10 * n}
        b = n * 2 + n + n // 32 + w + 4 * M
        b += (4 * n if case["residual"] else 0) + (2 * n if case["y"] else 0)
        return {"bytes": b, "flops": 6 * n}
    if op == "fp4":  # the codes and their scales are written and read, too: they are what is kept
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 4 * n}
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    used = min(G, M)  # the matrices that are read are those of the groups that have rows
    return {"bytes": 2 * M * K + used * N * (K // 2 + K // 32) + 2 * M * N + 4 * G, "flops": 2 * M * N * K}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _token_values(g, rows, cols):
    """Hidden states: every token its own scale, a few outlying entries."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    far = torch.randint(0, rows * cols, (max(1, rows * cols // 1000),), generator=g, device="cuda")
    x.view(-1)[far] *= 20.0
    return x.to(torch.bfloat16)


def _blocked(s):
    """E8M0 scales (batch, rows, n) in the tensor cores' tiles of 128 rows x 4 scales,
    missing rows and scales zero."""
    b, r, n = s.shape
    R, C = (r + 127) // 128, (n + 3) // 4
    full = torch.zeros((b, R * 128, C * 4), dtype=torch.uint8, device=s.device)
    full[:, :r, :n] = s
    return full.view(b, R, 4, 32, C, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _randn(g, T, E) * 1.5 + 0.5 * _randn(g, 1, E)
        if case["masked"]:  # experts that may not be used, and tokens that are padding
            x[:, torch.rand(E, generator=g, device="cuda") < 0.05] = -math.inf
            x[torch.rand(T, generator=g, device="cuda") < 0.02] = -math.inf
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["logits"] = x.to(dt)
        st["bias"] = 0.05 * _randn(g, E) if case["bias"] else None
        st["grad_weights"] = _randn(g, T, k)
        st["weights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["grad_logits"] = torch.empty((T, E), dtype=dt, device="cuda")
    elif op == "plan":
        T, k, E = case["T"], case["k"], case["E"]
        # experts of unlike popularity, each token's k different ones
        pull = _randn(g, T, E) + _randn(g, 1, E)
        ids = torch.topk(pull, k, dim=1).indices.to(torch.int32)
        ids[torch.rand(T, generator=g, device="cuda") < case["padding"]] = -1
        st["ids"] = ids.contiguous()
        st["offs"] = torch.empty(E, dtype=torch.int32, device="cuda")
        st["rows"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["src"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        # room for the call's intermediate counts, as its workspace rule has it at most
        st["workspace"] = torch.empty(4 * E * (T * k // 2048 + 2), dtype=torch.uint8, device="cuda")
    elif op == "norm":
        M, D = case["M"], case["D"]
        st["x"] = _token_values(g, M, D)
        st["residual"] = _token_values(g, M, D) if case["residual"] else None
        w = 1.0 + 0.2 * _randn(g, D)
        st["weight"] = w.to(torch.bfloat16 if case["wtype"] == "bf16" else torch.float32)
        st["eps"] = 1e-5
        if case["grad"]:
            # what the forward pass kept: the normed stream and 1 / rms of its rows
            st["h"] = st.pop("x")
            st["rstd"] = torch.rsqrt(st["h"].double().square().mean(1) + st["eps"]).float()
            st["grad_y"] = (0.01 * _randn(g, M, D)).to(torch.bfloat16)
            st["grad_res"] = (0.01 * _randn(g, M, D)).to(torch.bfloat16) if case["residual"] else None
            st["residual"] = None
            st["grad_x"] = torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
            st["grad_weight"] = torch.empty(D, dtype=torch.float32, device="cuda")
            st["workspace"] = torch.empty(4 * D * min(M, 1184), dtype=torch.uint8, device="cuda")
        else:
            e = lambda dt, *s: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
            st["q"], st["s"] = e(torch.uint8, M, D), e(torch.uint8, M, D // 32)
            st["rstd"] = e(torch.float32, M)
            st["res_out"] = e(torch.bfloat16, M, D) if case["residual"] else None
            st["y"] = e(torch.bfloat16, M, D) if case["y"] else None
    elif op == "fp4":
        b, r, c = case["batch"], case["rows"], case["cols"]
        st["x"] = torch.empty((b, r, c), dtype=torch.bfloat16, device="cuda")
        for i in range(b):
            st["x"][i] = _token_values(g, r, c) if b == 1 else (0.02 * _randn(g, r, c)).to(torch.bfloat16)
        st["q"] = torch.empty((b, r, c // 2), dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty((b, r, c // 32), dtype=torch.uint8, device="cuda")
        st["y"] = torch.empty((b, r, c), dtype=torch.bfloat16, device="cuda")
    else:
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        st["x"] = _token_values(g, M, K)
        # every group a share of the rows (one row at least while there are enough), the rest behind
        have = max(0, M - case["rest"])
        pick = torch.randint(0, G, (have,), generator=g, device="cuda")
        pick[:min(G, have)] = torch.arange(min(G, have), device="cuda")
        sizes = torch.bincount(pick, minlength=G)
        st["offs"] = torch.cumsum(sizes, 0).to(torch.int32)
        st["most"] = max(1, int(sizes.max()))  # rows of the largest group, a number its program knows
        st["qb"] = torch.empty((G, N, K // 2), dtype=torch.uint8, device="cuda")
        st["sb"] = torch.empty((G, N, K // 32), dtype=torch.uint8, device="cuda")
        for i in range(G):
            w = (0.02 * _randn(g, N, K)).to(torch.bfloat16)
            codes, st["sb"][i] = _fp4_codes(w.float())
            st["qb"][i] = codes[:, 0::2] | codes[:, 1::2] << 4
        st["sfb"] = _blocked(st["sb"])
        st["qa"] = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
        st["sfa"] = torch.zeros((M + 127 * G + 127) // 128 * ((K // 32 + 3) // 4) * 512, dtype=torch.uint8,
                                device="cuda")
        st["out"] = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------------------

def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


# ---- plain forms

def _p_route(st):
    c = st["case"]
    k, E, T = c["k"], c["E"], c["T"]
    # in 64 bits: the choice compares scores that lie close together
    x = st["logits"].double()
    dead = x == -math.inf
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
        e, top = p, None
    else:
        top = x.max(1, keepdim=True).values
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        e = torch.exp(x - top)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total == 0, torch.ones_like(total), total)
    none = torch.full_like(x, -math.inf)
    by = x if st["bias"] is None else torch.where(dead, none, p + st["bias"].double())
    if c["groups"] > 1:
        value = p if st["bias"] is None else by
        value = torch.where(dead, none, value).view(T, c["groups"], -1)
        best = torch.sort(value, dim=2, descending=True).values[:, :, :c["group_top"]]
        some = best[:, :, 0] > -math.inf
        score = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        if c["group_top"] == 1 and st["bias"] is None:
            score = x.view(T, c["groups"], -1).max(2).values
        score = torch.where(some, score, torch.full_like(score, -math.inf))
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        by = torch.where(open_.repeat_interleave(E // c["groups"], 1), by, none)
    order = torch.sort(by, dim=1, descending=True, stable=True)
    ids, ok = order.indices[:, :k], order.values[:, :k] > -math.inf
    picked = torch.where(ok, p.gather(1, ids), torch.zeros((), dtype=torch.float64, device=x.device))
    if not c["renorm"]:
        w = picked * c["scale"]
    elif c["score"] == "sigmoid":
        w = picked / (picked.sum(1, keepdim=True) + 1e-20) * c["scale"]
    else:
        near = torch.where(ok, x.gather(1, ids), none[:, :k])
        high = near.max(1, keepdim=True).values
        near = torch.exp(near - torch.where(high == -math.inf, torch.zeros_like(high), high))
        total = near.sum(1, keepdim=True)
        w = near / torch.where(total == 0, torch.ones_like(total), total) * c["scale"]
    out = {"weights": w.float(), "ids": torch.where(ok, ids, torch.full_like(ids, -1)).to(torch.int32)}
    if c["grad"]:
        gw = torch.where(ok, st["grad_weights"].double() * c["scale"], torch.zeros((), dtype=torch.float64,
                                                                                  device=x.device))
        r = w / c["scale"]
        spot = torch.zeros_like(x)
        if c["renorm"]:
            part = gw - (gw * r).sum(1, keepdim=True)
            if c["score"] == "softmax":
                gx = spot.scatter_add_(1, ids, r * part)
            else:
                gx = spot.scatter_add_(1, ids, r * part * (1.0 - picked))
        elif c["score"] == "softmax":
            gx = spot.scatter_add_(1, ids, gw * picked) - p * (gw * picked).sum(1, keepdim=True)
        else:
            gx = spot.scatter_add_(1, ids, gw * picked * (1.0 - picked))
        out["grad_logits"] = gx.to(st["logits"].dtype)
    return out


def _p_plan(st):
    ids, E = st["ids"], st["case"]["E"]
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True)
    live = order.values < E
    src = torch.where(live, order.indices, torch.full_like(flat, -1))
    at = torch.empty_like(flat).scatter_(0, order.indices, torch.arange(n, device=flat.device))
    rows = torch.where(flat < 0, torch.full_like(flat, -1), at)
    ends = torch.cumsum(torch.zeros(E + 1, dtype=torch.int64, device=flat.device).scatter_add_(
        0, key, torch.ones_like(key)), 0)[:E]
    return {"offs": ends.to(torch.int32), "rows": rows.view(ids.shape).to(torch.int32), "src": src.to(torch.int32)}


def _mx8(y):
    """MXFP8 blocks of 32 along the rows: E4M3 codes and E8M0 scales."""
    M, D = y.shape
    blocks = y.float().view(M, D // 32, 32)
    top = blocks.abs().amax(2)
    ex = torch.frexp(top).exponent - 1  # floor(log2)
    b = torch.where(top > 0, torch.clamp(ex - 8, -127, 127) + 127, torch.zeros_like(ex))
    v = torch.ldexp(blocks, (127 - b).unsqueeze(2)).clamp(-448.0, 448.0)
    return v.to(torch.float8_e4m3fn).view(M, D), b.to(torch.uint8)


def _p_norm(st):
    c = st["case"]
    w = st["weight"].float()
    if c["grad"]:
        h, gy, r = st["h"].float(), st["grad_y"].float(), st["rstd"].unsqueeze(1)
        n = h * r
        gn = gy * w
        gx = r * (gn - n * (gn * n).mean(1, keepdim=True))
        if st["grad_res"] is not None:
            gx = gx + st["grad_res"].float()
        return {"grad_x": gx.to(torch.bfloat16), "grad_weight": (gy * n).sum(0)}
    h = st["x"].float()
    out = {}
    if st["residual"] is not None:
        out["res"] = (h + st["residual"].float()).to(torch.bfloat16)
        h = out["res"].float()
    r = torch.rsqrt(h.square().mean(1) + st["eps"])
    y = (h * r.unsqueeze(1) * w).to(torch.bfloat16)
    q, s = _mx8(y)
    out |= {"q": q, "s": s.view(torch.float8_e8m0fnu), "rstd": r}
    if c["y"]:
        out["y"] = y
    return out


def _fp4_codes(x):
    """MXFP4 blocks of 32 along the rows of x (rows, cols) in 32 bits: a 4-bit code for each
    value, and the blocks' E8M0 scales."""
    rows, cols = x.shape
    blocks = x.view(rows, cols // 32, 32)
    top = blocks.abs().amax(2)
    ex = torch.frexp(top).exponent - 1
    b = torch.where(top > 0, torch.clamp(ex - 2, -127, 127) + 127, torch.zeros_like(ex))
    v = torch.ldexp(blocks, (127 - b).unsqueeze(2))
    a = v.abs().clamp(max=6.0)
    # codes 0..4 are halves up to 2, then 3, 4, 6: nearest, ties to the even code
    code = torch.where(a <= 2.0, torch.round(2.0 * a),
                       torch.where(a <= 4.0, torch.round(a) + 2.0, torch.round(0.5 * a) + 4.0))
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code.view(rows, cols), b.to(torch.uint8)


def _fp4_values(code, s):
    """The values of 4-bit codes (..., cols) under E8M0 scales (..., cols / 32), in 32 bits."""
    grid = torch.tensor(F4_GRID + tuple(-v for v in F4_GRID), device=code.device)
    v = grid[code.int()]
    return torch.ldexp(v.view(*s.shape, 32), (s.int() - 127).unsqueeze(-1)).view(code.shape)


def _p_fp4(st):
    x = st["x"].view(-1, st["case"]["cols"]).float()
    code, s = _fp4_codes(x)
    return {"values": _fp4_values(code, s).to(torch.bfloat16).view(st["x"].shape)}


def _p_experts(st):
    c = st["case"]
    M, G = c["M"], c["G"]
    code, s = _fp4_codes(st["x"].float())
    a = _fp4_values(code, s)
    qb = st["qb"]
    w = _fp4_values(torch.stack((qb & 15, qb >> 4), -1).view(G, c["N"], c["K"]), st["sb"])
    # the rows of each group side by side, as many as the largest has; those past a group's end count nothing
    ends = st["offs"].long()
    starts = torch.cat((ends.new_zeros(1), ends[:-1]))
    at = starts.unsqueeze(1) + torch.arange(st["most"], device=a.device)
    there = at < ends.unsqueeze(1)
    prod = torch.bmm(a[at.clamp(max=M - 1)], w.transpose(1, 2)).to(torch.bfloat16)
    out = torch.zeros_like(st["out"])
    out[at[there]] = prod[there]
    return {"out": out}


_plain = {"route": _p_route, "plan": _p_plan, "norm": _p_norm, "fp4": _p_fp4, "experts": _p_experts}


# ---- this package's calls

def _o_route(st):
    import mxfp8_quantization_moe_mx_b200 as mxq
    c = st["case"]
    score = mxq.SIGMOID if c["score"] == "sigmoid" else mxq.SOFTMAX
    mxq.moe_route(st["logits"], st["weights"], st["ids"], bias=st["bias"], score=score, n_groups=c["groups"],
                  top_groups=c["keep"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"])
    out = {"weights": st["weights"], "ids": st["ids"]}
    if c["grad"]:
        mxq.moe_route_backward(st["logits"], st["ids"], st["grad_weights"], st["grad_logits"], score=score,
                               renorm=c["renorm"], scale=c["scale"])
        out["grad_logits"] = st["grad_logits"]
    return out


def _o_plan(st):
    import mxfp8_quantization_moe_mx_b200 as mxq
    mxq.moe_plan(st["ids"], st["offs"], st["rows"], st["src"], st["workspace"])
    return {"offs": st["offs"], "rows": st["rows"], "src": st["src"]}


def _o_norm(st):
    import mxfp8_quantization_moe_mx_b200 as mxq
    c = st["case"]
    if c["grad"]:
        mxq.rmsnorm_backward(st["grad_y"], st["h"], st["weight"], st["rstd"], st["grad_x"], st["grad_weight"],
                             st["workspace"], grad_res=st["grad_res"])
        return {"grad_x": st["grad_x"], "grad_weight": st["grad_weight"]}
    mxq.rmsnorm_mx_quantize(st["x"], st["weight"], st["eps"], st["q"], st["s"], residual=st["residual"],
                            res_out=st["res_out"], y=st["y"], rstd=st["rstd"])
    out = {"q": st["q"].view(torch.float8_e4m3fn), "s": st["s"].view(torch.float8_e8m0fnu), "rstd": st["rstd"]}
    if st["residual"] is not None:
        out["res"] = st["res_out"]
    if c["y"]:
        out["y"] = st["y"]
    return out


def _o_fp4(st):
    import mxfp8_quantization_moe_mx_b200 as mxq
    mxq.mxfp4_quantize(st["x"], st["q"], st["s"])
    mxq.mxfp4_dequantize(st["q"], st["s"], st["y"])
    return {"values": st["y"]}


def _o_experts(st):
    import mxfp8_quantization_moe_mx_b200 as mxq
    mxq.mxfp4_quantize(st["x"], st["qa"], sf_blocked=st["sfa"], offs=st["offs"])
    mxq.mxfp4_grouped_gemm(st["qa"], st["sfa"], st["qb"], st["sfb"], st["offs"], st["out"])
    return {"out": st["out"]}


_own = {"route": _o_route, "plan": _o_plan, "norm": _o_norm, "fp4": _o_fp4, "experts": _o_experts}


# ---- the definitions in 64 bits ------------------------------------------------------------------------

def _e_route(st):
    c = st["case"]
    x = st["logits"].to(torch.float64).requires_grad_(True)
    T, E, k = c["T"], c["E"], c["k"]
    alive = torch.isfinite(x.detach())
    safe = torch.where(alive, x, torch.full_like(x, -1e5))  # its score is zero
    some = alive.any(1, keepdim=True)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(safe)
    else:
        p = torch.softmax(safe, 1) * (alive & some)
    rank = (safe if st["bias"] is None else p + st["bias"].to(torch.float64)).detach().clone()
    rank[~alive] = -math.inf
    if c["groups"] > 1:
        v = (p if st["bias"] is None else p + st["bias"].to(torch.float64)).detach().clone()
        v[~alive] = -math.inf
        if st["bias"] is None and c["group_top"] == 1:
            v = rank.clone()
        v = v.view(T, c["groups"], E // c["groups"])
        score = torch.zeros(T, c["groups"], dtype=torch.float64, device=x.device)
        for j in range(c["group_top"]):
            m, i = v.max(2)
            score += torch.where(m == -math.inf, m if j == 0 else torch.zeros_like(m), m)
            v = v.scatter(2, i.unsqueeze(2), -math.inf)
        # a group is kept if fewer than `keep` others stand before it
        g = torch.arange(c["groups"], device=x.device)
        before = (score.unsqueeze(1) > score.unsqueeze(2)) | ((score.unsqueeze(1) == score.unsqueeze(2))
                                                             & (g.view(1, 1, -1) < g.view(1, -1, 1)))
        kept = before.sum(2) < c["keep"]
        rank = torch.where(kept.unsqueeze(2), rank.view(T, c["groups"], -1),
                           torch.full((), -math.inf, dtype=torch.float64, device=x.device)).reshape(T, E)
    chosen, ok = [], []
    place = torch.arange(E, device=x.device)
    for _ in range(k):
        m = rank.max(1, keepdim=True).values
        i = torch.where(rank == m, place, E).min(1, keepdim=True).values
        chosen.append(i)
        ok.append(m > -math.inf)
        rank = rank.scatter(1, i, -math.inf)
    i, ok = torch.cat(chosen, 1), torch.cat(ok, 1)
    w = p.gather(1, i) * ok
    if c["renorm"] and c["score"] == "sigmoid":
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    elif c["renorm"]:
        w = torch.softmax(torch.where(ok, safe.gather(1, i), torch.full_like(w, -1e9)), 1) * ok
    w = w * c["scale"]
    out = {"weights": w.detach(), "ids": None}
    if c["grad"]:
        (gx,) = torch.autograd.grad(w, x, st["grad_weights"].to(torch.float64))
        out["grad_logits"] = torch.where(alive, gx, torch.zeros_like(gx))
    return out


def _floor_power(top, down):
    """2 ** (floor(log2(top)) - down), at least 2 ** -127, from the exponent's bits."""
    ex = (top.view(torch.int64) >> 52) - 1023 - down
    return (ex.clamp(-127, 127) + 1023 << 52).view(torch.float64)


def _e_norm(st):
    c = st["case"]
    w = st["weight"].to(torch.float64)
    if c["grad"]:
        h, gy = st["h"].to(torch.float64), st["grad_y"].to(torch.float64)
        r = st["rstd"].to(torch.float64)[:, None]
        dot = (gy * w * h).sum(1, keepdim=True)
        gx = r * gy * w - h * r ** 3 * dot / c["D"]
        if st["grad_res"] is not None:
            gx += st["grad_res"].to(torch.float64)
        return {"grad_x": gx, "grad_weight": torch.einsum("md,md,m->d", gy, h, r[:, 0])}
    h, out = st["x"].to(torch.float64), {}
    if st["residual"] is not None:
        out["res"] = h + st["residual"].to(torch.float64)
        h = out["res"].to(torch.bfloat16).to(torch.float64)  # the sum is kept, and normed, in bf16
    r = 1.0 / torch.sqrt((h * h).sum(1) / c["D"] + st["eps"])
    y = h * r[:, None] * w
    blocks = y.to(torch.bfloat16).to(torch.float64).view(c["M"], -1, 32)
    scale = _floor_power(blocks.abs().amax(2), 8)
    # a code stands for the value under the scale, up to its rounding
    out |= {"q": (blocks / scale[..., None]).clamp(-448, 448).view(c["M"], -1), "s": scale, "rstd": r}
    if c["y"]:
        out["y"] = y
    return out


def _e_values(x):
    """The nearest value of the 4-bit grid under each block's scale, in 64 bits."""
    blocks = x.to(torch.float64).view(-1, 32)
    top = blocks.abs().amax(1, keepdim=True)
    scale = _floor_power(top, 2)
    v = (blocks / scale).abs()
    got = torch.zeros_like(v)
    grid = F4_GRID
    for i in range(1, 8):  # the border between two neighbours belongs to the one of even index
        border = (grid[i - 1] + grid[i]) / 2
        got = torch.where((v >= border) if i % 2 == 0 else (v > border), torch.full_like(v, grid[i]), got)
    return (torch.copysign(got, blocks) * scale).view(x.shape)


def _e_fp4(st):
    return {"values": torch.stack([_e_values(m).to(torch.float32) for m in st["x"]])}


def _e_experts(st):
    c = st["case"]
    a = _e_values(st["x"])
    out = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=a.device)
    grid = torch.tensor(F4_GRID, dtype=torch.float64, device=a.device)
    start = 0
    for g, end in enumerate(st["offs"].tolist()):
        if end > start:
            q = st["qb"][g].to(torch.int64)
            pairs = [grid[n & 7] * torch.where(n >= 8, -1.0, 1.0) for n in (q % 16, q // 16)]
            scale = (st["sb"][g].to(torch.int64) + (1023 - 127) << 52).view(torch.float64)
            w = torch.stack(pairs, 2).view(c["N"], -1, 32) * scale[..., None]
            out[start:end] = a[start:end] @ w.view(c["N"], c["K"]).T
        start = max(start, end)
    return {"out": out}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    return {"route": _e_route, "norm": _e_norm, "fp4": _e_fp4, "experts": _e_experts}[case["op"]](prepare(case, seed))
