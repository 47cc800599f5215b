"""Plain 64-bit forms of the operators of include/moe_layer.h, and the error bounds of the fp32
arithmetic that computes them. u = 2^-24 is the largest relative error of one fp32 rounding."""
import numpy as np
import torch

U = 2.0 ** -24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def quant(x):
    """Codes and scales of float64 rows: 127 * x / a needs 31 bits before its division, so the
    fp64 quotient falls on a half only where the exact one does."""
    a = np.abs(x).max(axis=1)
    bad = ~np.isfinite(x).all(axis=1)
    safe = np.where(bad | (a == 0), 1.0, a)
    q = np.rint(127.0 * np.where(bad[:, None], 0.0, x) / safe[:, None])
    scale = np.where(a == 0, 1.0, safe / 127.0).astype(np.float32)
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def matmul(a, a_scale, w, w_scale, offsets, row_token, act, bf16):
    """(out, tolerance, rows written): out[r] in float64 and what the fp32 epilogue may be off by.
    y = fl(fl(fl(acc) sa) sw) is within 3u. With SwiGLU the gate's own 3u move silu by
    |1 + g (1 - sigmoid(g))| 3u <= (1 + |g|) 3u; exp (1 ulp = 2u), 1 + e, the quotient, the product
    and the up channel's 3u add 8u: (12 + 3 |g|) u, taken as (16 + 4 |g|) u for the second order.
    A result in bf16 is off by half a step more, one below 2^-126 by what may be flushed."""
    R = a.shape[0] if row_token is None else len(row_token)
    n_w = w.shape[1]
    N = n_w // 2 if act == "swiglu" else n_w
    out, tol = np.zeros((R, N)), np.zeros((R, N))
    done = np.zeros(R, bool)
    src = np.arange(R) if row_token is None else row_token
    for e in range(w.shape[0]):
        r = np.arange(offsets[e], offsets[e + 1])
        r = r[(src[r] >= 0) & (src[r] < a.shape[0])]
        if not len(r):
            continue
        acc = a[src[r]].astype(np.float64) @ w[e].astype(np.float64).T     # exact: below 2^53
        y = acc * a_scale[src[r]].astype(np.float64)[:, None] * w_scale[e].astype(np.float64)
        rel = 4 * U * np.ones_like(y)
        if act == "swiglu":
            g = y[:, :N]
            y = silu(g) * y[:, N:]
            rel = (16 + 4 * np.abs(g)) * U
        out[r], done[r] = y, True
        tol[r] = np.abs(y) * (rel + (BF16_HALF if bf16 else 0.0)) + 2.0 ** -120
    return out, tol, done


def probs(logits):
    m = logits.max(axis=1, keepdims=True)
    e = np.exp(logits - np.where(np.isfinite(m), m, 0.0))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def prob_error(logits):
    """Relative error of one fp32 probability: l - m is rounded (|l - m| u in the exponent), exp by
    two parts 4u, at most 16 + 6 additions of the row's sum, reciprocal and product 2u."""
    f = np.where(np.isfinite(logits), logits, np.nan)
    spread = np.nan_to_num(np.nanmax(f) - np.nanmin(f)) if np.isfinite(f).any() else 0.0
    return (2 * min(spread, 90.0) + 30) * U


def balance(logits, idx, mask, S, alpha):
    """loss, counts, prob sums, tokens of each sequence."""
    T, E = logits.shape
    k = idx.shape[1]
    keep = np.ones(T, bool) if mask is None else mask.astype(bool)
    p = probs(logits)
    counts, sums, tokens = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    loss = 0.0
    for s in range(S):
        rows = np.arange(s * (T // S), (s + 1) * (T // S))
        rows = rows[keep[rows]]
        ids = idx[rows].reshape(-1)
        counts[s] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        sums[s] = p[rows].sum(axis=0)
        n = tokens[s] = len(rows)
        if n:
            loss += alpha / S * E / (k * float(n) ** 2) * (counts[s] * sums[s]).sum()
    return loss, counts, sums, tokens


def route_grad(logits, idx, w, dw, mask, counts, tokens, g, S, alpha):
    """(dlogits, tolerance). p (c - dot) with centred counts c: p carries dp, dot = sum c p at most
    sum |c| p (dp + 32u), the difference and the products 4u; the weights' term w (dw - all): 4u,
    and k + 8 additions in all; adding them up one u a term."""
    T, E = logits.shape
    k = idx.shape[1]
    d, tol = np.zeros((T, E)), np.zeros((T, E))
    if counts is not None:
        p, dp = probs(logits), prob_error(logits)
        keep = np.ones(T, bool) if mask is None else mask.astype(bool)
        for t in range(T):
            s = t // (T // S)
            n = int(tokens[s])
            if not keep[t] or not n:
                continue
            f = g * alpha / S * E / (k * float(n) ** 2)
            c = counts[s] - float(round(k * n / E))
            dot, size = (c * p[t]).sum(), (np.abs(c) * p[t]).sum()
            d[t] = f * p[t] * (c - dot)
            tol[t] = abs(f) * p[t] * (np.abs(c - dot) * (dp + 4 * U) + size * (dp + 33 * U))
    if w is not None:
        for t in range(T):
            all_ = (w[t] * dw[t]).sum()
            size = np.abs(w[t] * dw[t]).sum()
            for j in range(k):
                e = idx[t, j]
                if 0 <= e < E:
                    d[t, e] += w[t, j] * (dw[t, j] - all_)
                    tol[t, e] += abs(w[t, j]) * (abs(dw[t, j] - all_) * 4 * U + size * (k + 8) * U)
                    tol[t, e] += abs(d[t, e]) * U
    return d, tol + 2.0 ** -120
