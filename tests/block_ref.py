"""Plain 64-bit forms of the operators of include/moe_block.h, and the error bounds of the fp32
arithmetic that computes them. u = 2^-24 is the largest relative error of one fp32 rounding."""
import numpy as np
import torch

U = 2.0 ** -24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
TINY = 2.0 ** -100          # what may be flushed, and bounded logistic tails


def half(bf16):
    return BF16_HALF if bf16 else U


# ----------------------------------------------------------------------------------- routing --
def scores(logits, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-logits))
    m = logits.max(axis=1, keepdims=True)
    e = np.exp(logits - np.where(np.isfinite(m), m, 0.0))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route(logits, bias, k, score, n_groups, topk_groups, group_top, renormalize, scale):
    """Ids and weights, token by token."""
    logits = logits.astype(np.float64)
    T, E = logits.shape
    s = scores(logits, score)
    c = s + (0.0 if bias is None else bias.astype(np.float64))
    c = np.where(np.isneginf(logits), -np.inf, c)
    per = E // n_groups
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        among = range(E)
        if n_groups > 1:
            total = [sum(sorted(c[t, g * per:(g + 1) * per], reverse=True)[:group_top])
                     for g in range(n_groups)]
            kept = sorted(range(n_groups), key=lambda g: (-total[g], g))[:topk_groups]
            among = [e for g in kept for e in range(g * per, (g + 1) * per)]
        ids = sorted(among, key=lambda e: (-c[t, e], e))[:k]
        v = s[t, ids]
        if renormalize:
            v = v / v.sum() if v.sum() > 0 else np.zeros(k)
        idx[t], w[t] = ids, v * scale
    return idx, w


def scored_grad(logits, idx, dw, add, score, renormalize, scale):
    """(dlogits, tolerance). One score carries e = (2 min(spread, 90) + 30) u (the exponent's rounding,
    exp, the quotient; as for the softmax of a row), a sum of n of them n u more; every term of dl
    has at most three scores, two differences and five products: 4 e + (k + 16) u of the sum of its
    magnitudes. Adding up to k terms and `add` is one u of the magnitudes each."""
    logits = logits.astype(np.float64)
    T, E = logits.shape
    k = idx.shape[1]
    d, tol = np.zeros((T, E)), np.zeros((T, E))
    s = scores(logits, score)
    for t in range(T):
        ok = [(j, idx[t, j]) for j in range(k) if 0 <= idx[t, j] < E]
        f = logits[t][np.isfinite(logits[t])]
        spread = 0.0 if not len(f) else max(f.max() - f.min(), np.abs(f).max())
        e = (2 * min(spread, 90.0) + 30) * U
        rel = 4 * e + (k + 16) * U
        if score == "softmax" and not renormalize:
            q = np.zeros(E)
            mag = np.zeros(E)
            for j, i in ok:
                q[i] += dw[t, j]
                mag[i] += abs(dw[t, j])
            d[t] = scale * s[t] * (q - (s[t] * q).sum())
            tol[t] = abs(scale) * s[t] * (mag + (s[t] * mag).sum()) * (rel + E / 16 * U)
        else:
            x = np.array([logits[t, i] for _, i in ok])
            g = np.array([dw[t, j] for j, _ in ok])
            if not len(x):
                continue
            if score == "softmax":
                m = x.max()
                v = np.exp(x - m) if np.isfinite(m) else np.zeros(len(x))
                slope = np.ones(len(x))
            else:
                top = min(x.max(), 0.0)
                with np.errstate(over="ignore", invalid="ignore"):
                    v = np.where(np.isneginf(x), 0.0, np.exp(np.minimum(x, 0.0) - top) / (1 + np.exp(-np.abs(x))))
                    slope = 1.0 / (1.0 + np.exp(x))
            if renormalize:
                v = v / v.sum() if v.sum() > 0 else np.zeros(len(x))
                term = scale * v * (g - (v * g).sum()) * slope
                size = abs(scale) * v * (np.abs(g) + (v * np.abs(g)).sum()) * slope
            else:
                v = np.array([s[t, i] for _, i in ok])
                term = scale * v * g * slope
                size = np.abs(term)
            for n, (_, i) in enumerate(ok):
                d[t, i] += term[n]
                tol[t, i] += size[n] * (rel + k * U)
    if add is not None:
        d = d + add
        tol += (np.abs(add) + np.abs(d)) * U
    return d, tol + TINY


# ----------------------------------------------------------------------------------- products --
def act(v, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.maximum(v, 0.0)
        if name == "silu":
            return v / (1.0 + np.exp(-v))
        if name == "gelu":
            return v / (1.0 + np.exp(-np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def act_slope(v, name):
    """(slope, bound of its fp32 error): s (1 + x (1 - s)) with s = sigmoid(t), x = v t': s carries
    (16 + 8 |t|) u, which enters twice (once times |x|), and the rest 8 u."""
    if name == "none":
        return np.ones_like(v), np.zeros_like(v)
    if name == "relu":
        return (v > 0).astype(np.float64), np.zeros_like(v)
    t = v if name == "silu" else np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3)
    dt = 1.0 if name == "silu" else np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * v * v)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-t))
        x = v * dt
        rest = 1.0 / (1.0 + np.exp(t))
        d = s * (1 + x * rest)
    at = np.minimum(np.abs(t), 100.0)
    ax = np.where(np.abs(t) < 100, np.abs(x), 0.0)
    return d, s * (1 + 2 * ax) * (24 + 8 * at) * U + TINY


def sums(size, n):
    """A sum of n exact products in fp32: a term goes through at most n / 16 matrix instructions, up to
    16 additions inside one, and the joins; each may truncate (2 u)."""
    return 2 * U * (n / 16 + 40) * size


def rows_of(offsets, e, R, src=None, A=None):
    lo = min(max(int(offsets[e]), 0), R)
    r = np.arange(lo, min(max(int(offsets[e + 1]), lo), R))
    return r if src is None else r[(src[r] >= 0) & (src[r] < A)]


def product(a, w, offsets, row_token, bias, name, residual, bf16):
    """(out, tolerance, pre, tolerance, rows written)."""
    R = a.shape[0] if row_token is None else len(row_token)
    n_w = w.shape[1]
    N = n_w // 2 if name == "swiglu" else n_w
    K = a.shape[1]
    src = np.arange(R) if row_token is None else row_token
    y, ty = np.zeros((R, n_w)), np.zeros((R, n_w))
    done = np.zeros(R, bool)
    for e in range(w.shape[0]):
        r = rows_of(offsets, e, R, src, a.shape[0])
        y[r] = a[src[r]] @ w[e].T + (0.0 if bias is None else bias[e])
        ty[r] = sums(np.abs(a[src[r]]) @ np.abs(w[e]).T, K) + 2 * U * np.abs(y[r])
        done[r] = True
    if name == "swiglu":
        g, u, tg, tu = y[:, :N], y[:, N:], ty[:, :N], ty[:, N:]
        s = act(g, "silu")
        out = s * u
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(s) * tu + np.abs(out) * (16 + 4 * np.minimum(np.abs(g), 100)) * U
    else:
        out = act(y, name)
        t = np.abs(y) if name == "silu" else np.sqrt(8 / np.pi) * np.abs(y + 0.044715 * y ** 3)
        rel = 0.0 if name in ("none", "relu") else (16 + 8 * np.minimum(t, 100)) * U
        tol = 1.2 * ty + np.abs(out) * rel
    if residual is not None:
        out = out + residual
        tol = tol + 2 * U * np.abs(out)
    return (out, tol + np.abs(out) * half(bf16) + TINY, y, ty + np.abs(y) * BF16_HALF + TINY, done)


def product_grad(dy, a, w, offsets, row_token, name, pre, da_bf16, dw_bf16):
    """{name: (value, tolerance)}, rows of da that are written."""
    R, N = dy.shape
    E, _, K = w.shape
    src = np.arange(R) if row_token is None else row_token
    dh, th, done = np.zeros((R, K)), np.zeros((R, K)), np.zeros(R, bool)
    dw, tw = np.zeros((E, N, K)), np.zeros((E, N, K))
    db, tb = np.zeros((E, N)), np.zeros((E, N))
    for e in range(E):
        r = rows_of(offsets, e, R, src, a.shape[0])
        dh[r] = dy[r] @ w[e]
        th[r] = sums(np.abs(dy[r]) @ np.abs(w[e]), N)
        dw[e] = dy[r].T @ a[src[r]]
        tw[e] = sums(np.abs(dy[r]).T @ np.abs(a[src[r]]), len(r))
        db[e] = dy[r].sum(axis=0)
        tb[e] = (len(r) + 32) * U * np.abs(dy[r]).sum(axis=0)
        done[r] = True
    if name == "swiglu":
        g, u = pre[:, :K], pre[:, K:]
        s, (d, td) = act(g, "silu"), act_slope(g, "silu")
        rel = (16 + 4 * np.minimum(np.abs(g), 100)) * U
        da = np.concatenate([dh * u * d, dh * s], 1)
        ta = np.concatenate([th * np.abs(u * d) + (np.abs(dh) + th) * np.abs(u) * (td + 4 * U * np.abs(d)),
                             th * np.abs(s) + (np.abs(dh) + th) * np.abs(s) * (rel + 4 * U)], 1)
    else:
        d, td = act_slope(pre if name != "none" else dh, name)
        da, ta = dh * d, th * np.abs(d) + (np.abs(dh) + th) * (td + 2 * U * np.abs(d))
    return {"da": (da, ta + np.abs(da) * half(da_bf16) + TINY),
            "dw": (dw, tw + np.abs(dw) * half(dw_bf16) + TINY), "dbias": (db, tb + TINY)}, done
