"""Plain 64-bit forms of the mixture-of-experts operators, for the tests: numpy on the host,
row by row where that says the rule most plainly."""
import numpy as np

F4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scores(x, score):
    """x (E,) float64 without NaN: the scores, 0 for masked experts."""
    live = x > -np.inf
    p = np.zeros_like(x)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            p[live] = 1.0 / (1.0 + np.exp(-x[live]))
    elif live.any():
        e = np.exp(x[live] - x[live].max())
        p[live] = e / e.sum()
    return p


def route_row(x, bias, score, n_groups, top_groups, group_top, k, renorm, scale):
    """One row: (ids, weights)."""
    E = len(x)
    spoilt = np.isnan(x).any() or (score == "softmax" and np.isposinf(x).any())
    if bias is not None:
        spoilt = spoilt or (np.isnan(bias) & (x != -np.inf)).any()
    if spoilt:
        return np.arange(k), np.full(k, np.nan)
    p = scores(x, score)
    c = x.copy() if bias is None else np.where(x == -np.inf, -np.inf, p + bias)
    ok = c > -np.inf
    if n_groups > 1:
        gs = E // n_groups
        v = np.where(ok, p, -np.inf) if bias is None and group_top == 2 else c
        val = np.full(n_groups, -np.inf)
        for g in range(n_groups):
            best = [t for t in sorted(v[g * gs:(g + 1) * gs], reverse=True)[:group_top] if t > -np.inf]
            if best:
                val[g] = sum(best[1:], best[0])
        kept = [g for g in sorted(range(n_groups), key=lambda g: (-val[g], g))[:top_groups] if val[g] > -np.inf]
        ok &= np.isin(np.arange(E) // gs, kept)
    order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if ok[e]][:k]
    ids = np.full(k, -1)
    ids[:len(order)] = order
    w = np.zeros(k)
    w[:len(order)] = p[order]
    if renorm and score == "sigmoid":
        w = w / (w.sum() + 1e-20)
    elif renorm and order:
        e = np.exp(x[order] - x[order].max())
        w[:len(order)] = e / e.sum()
    return ids, w * scale


def route(x, bias, score, n_groups, top_groups, group_top, k, renorm, scale):
    rows = [route_row(r, bias, score, n_groups, top_groups, group_top, k, renorm, scale) for r in x]
    return (np.array([r[0] for r in rows]).reshape(len(x), k), np.array([r[1] for r in rows]).reshape(len(x), k))


def route_grad(x, ids, g, score, renorm, scale):
    """The gradient of the logits for given choices, and the sum of its terms' magnitudes."""
    out, mag = np.zeros_like(x), np.zeros_like(x)
    for t in range(len(x)):
        p = scores(x[t], score)
        slot = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < x.shape[1]]
        e, gt = ids[t, slot], scale * g[t, slot]
        if renorm:
            if score == "softmax":
                top = x[t, e].max() if slot and x[t, e].max() > -np.inf else 0.0
                r = np.exp(x[t, e] - top)
                r = r / r.sum() if r.sum() > 0 else r
                f = np.ones(len(slot))
            else:
                r = p[e] / (p[e].sum() + 1e-20)
                f = 1.0 - p[e]
            np.add.at(out[t], e, r * f * (gt - (gt * r).sum()))
            np.add.at(mag[t], e, r * f * (abs(gt) + (abs(gt) * r).sum()))
        elif score == "sigmoid":
            np.add.at(out[t], e, gt * p[e] * (1.0 - p[e]))
            np.add.at(mag[t], e, abs(gt) * p[e] * (1.0 - p[e]))
        else:
            np.add.at(out[t], e, gt * p[e])
            np.add.at(mag[t], e, abs(gt) * p[e])
            out[t] -= p * (gt * p[e]).sum()
            mag[t] += p * (abs(gt) * p[e]).sum()
    return out, mag


def plan(ids, E):
    flat = ids.reshape(-1)
    rows, src, offs = np.full(flat.size, -1), [], []
    for e in range(E):
        for i in np.flatnonzero(flat == e):
            rows[i] = len(src)
            src.append(i)
        offs.append(len(src))
    return np.array(offs), rows, np.array(src + [-1] * (flat.size - len(src)), dtype=np.int64)


def f4_quantize(x):
    """x (rows, cols) float64 holding bf16 values -> codes (rows, cols) and E8M0 scales."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(2)
    top = np.where(bad[..., None], 0.0, np.abs(b)).max(2)
    with np.errstate(divide="ignore"):
        ex = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
    s = np.clip(ex, -127, 127) + 127
    v = np.abs(np.where(bad[..., None], 0.0, b)) * np.exp2(127.0 - s)[..., None]
    # the nearest of the eight magnitudes, of two equally near ones the even one
    d = np.abs(v[..., None] - F4)
    near = d.min(-1, keepdims=True) == d
    code = np.where(near[..., 0::2].any(-1), 2 * near[..., 0::2].argmax(-1), 2 * near[..., 1::2].argmax(-1) + 1)
    code = np.where(bad[..., None], 7, code) | np.signbit(b) * 8
    return code.reshape(rows, cols).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def f4_pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def f4_values(code, s):
    v = F4[code & 7] * np.where(code & 8, -1.0, 1.0)
    sc = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (v.reshape(*s.shape, 32) * sc[..., None]).reshape(code.shape)


def groups(offs, M):
    """The clamp rule of the end offsets: (start, end) of each group."""
    out, last = [], 0
    for o in offs:
        end = min(max(int(o), last), M)
        out.append((last, end))
        last = end
    return out


def blocked(s, offs=None):
    """E8M0 scales (rows, n) in tiles of 128 rows x 4, each group on a fresh tile; the rows
    that the tiles' padding holds are 0."""
    n = s.shape[1]
    parts = [(0, s.shape[0])] if offs is None else groups(offs, s.shape[0])
    C = (n + 3) // 4
    out = []
    for a, e in parts:
        R = (e - a + 127) // 128
        full = np.zeros((R * 128, C * 4), np.uint8)
        full[:e - a, :n] = s[a:e]
        out.append(full.reshape(R, 4, 32, C, 4).transpose(0, 3, 2, 1, 4).reshape(-1))
    return np.concatenate(out)
