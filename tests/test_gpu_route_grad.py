"""GPU tests of the gradient of scored routing's logits: tokens that are sure of an expert, and more tokens
than a launch has places for, against plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from combine_moe_route_03_amd import _lib as moe
from test_gpu_block import _announce, dev, f64, off

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def sharp_grad(logits, idx, dw, score, renormalize, scale):
    """(dlogits, tolerance) without differences of nearly equal numbers: with shares v that add up to 1 and any
    c, dw_j - sum v dw = (dw_j - c) - sum v (dw - c), and c is the dw of the largest share where that is over
    half. A share is good to e = (2 min(distance from the largest, 90) + 30) u of itself; a term is a share, a
    difference of dw's and a sum of such products, the slope of a sigmoid, and some products: 4 e + (n + 16) u
    of the magnitudes that are left, n the terms of the sum that a lane adds up."""
    logits, dw = logits.astype(np.float64), dw.astype(np.float64)
    T, E = logits.shape
    k = idx.shape[1]
    d, tol = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if score == "softmax" and not renormalize:
            x, at = logits[t], np.arange(E)
            q, mag, n = np.zeros(E), np.zeros(E), E / 16 + k
            np.add.at(q, idx[t], dw[t])
            np.add.at(mag, idx[t], np.abs(dw[t]))
            mag = mag if len(set(idx[t])) < k else 0.0 * mag  # q of one slot is exact
        else:
            x, at, q, mag, n = logits[t, idx[t]], idx[t], dw[t], np.zeros(k), k
        v, slope = np.exp(x - x.max()), np.ones(len(x))
        if score == "sigmoid":
            v = np.exp(np.minimum(x, 0) - min(x.max(), 0)) / (1 + np.exp(-np.abs(x)))
            slope = 1 / (1 + np.exp(x))
        v = v / v.sum()
        m = np.argmax(v)
        diff = q - (q[m] if v[m] > 0.5 else 0.0)
        e = (2 * np.minimum(np.maximum(x.max() - x, np.abs(x) if score == "sigmoid" else 0), 90) + 30) * ref.U
        size = np.abs(diff) + (v * np.abs(diff)).sum()
        np.add.at(d[t], at, scale * v * slope * (diff - (v * diff).sum()))
        rel = 4 * max(e.max(), 0.0) + (n + 16) * ref.U
        near = np.where(np.arange(len(x)) == m, 0.0, mag + mag[m]) * k * ref.U
        np.add.at(tol[t], at, abs(scale) * v * slope * (size * rel + near + (v * near).sum()))
    return d, tol + 2.0 ** -120


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k", [(40, 8, 1), (40, 8, 4), (37, 7, 3), (33, 60, 6), (40, 64, 1), (35, 160, 8), (40, 256, 8),
                                   (9, 513, 17), (5, 1024, 64), (12, 4, 9)])
def test_gradient_of_a_token_that_is_sure(T, E, k, score, renormalize):
    """One logit leads by 2 to 40: what is left of the differences is small, and has to be right by itself.
    The leading expert is chosen in most tokens. With k > E ids repeat, among others that of the leading one."""
    _announce(f"gradient of sure tokens T={T} E={E} k={k} {score} {renormalize}")
    rng = np.random.default_rng(T + E + k)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.stack([rng.choice(E, k, replace=k > E) for _ in range(T)]).astype(np.int32)
    lead = idx[np.arange(T), rng.integers(0, k, T)]
    if not renormalize and score == "softmax":
        lead = np.where(np.arange(T) % 4 == 3, (idx[:, 0] + 1) % E, lead)
    base = 0.0 if score == "softmax" else -22.0
    logits += np.float32(base)
    logits[np.arange(T), lead] = base + 3 + 40.0 * np.arange(T) / T
    dw = (3 + rng.standard_normal((T, k))).astype(np.float32)
    got = moe.moe_route_scored_grad(dev(logits), dev(idx), dev(dw), score=score, renormalize=renormalize, scale=2.5)
    off(f64(got), *sharp_grad(logits, idx, dw, score, renormalize, 2.5), "dlogits")


def plain_grad(x, idx, dw, add, score, renormalize, scale):
    """(dlogits, tolerance) of many tokens, on the GPU in 64 bits; ids out of range take no part. The tolerance is
    that of block_ref.scored_grad with the spread of normal logits, 2 * 6 at the most."""
    T, E = x.shape
    k = idx.shape[1]
    ok = (idx >= 0) & (idx < E)
    at, g = idx.clamp(0, E - 1).long(), torch.where(ok, dw.double(), 0.0)
    s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
    rel = (4 * (2 * 24 + 30) + k + 16) * ref.U
    if score == "softmax" and not renormalize:
        q = torch.zeros_like(s).scatter_add_(1, at, g)
        d = scale * s * (q - (s * q).sum(1, keepdim=True))
        size = s * (q.abs() + (s * q.abs()).sum(1, keepdim=True)) * (rel + E / 16 * ref.U)
        mag = torch.zeros_like(s).scatter_add_(1, at, g.abs())
        size = torch.maximum(size, s * (mag + (s * mag).sum(1, keepdim=True)) * (rel + E / 16 * ref.U))
    else:
        v = torch.where(ok, s.gather(1, at), 0.0)
        slope = 1.0 if score == "softmax" else torch.sigmoid(-x.double().gather(1, at))
        if renormalize:
            total = v.sum(1, keepdim=True)
            v = torch.where(total > 0, v / total, 0.0)
            term = v * (g - (v * g).sum(1, keepdim=True)) * slope
            size = v * (g.abs() + (v * g.abs()).sum(1, keepdim=True)) * slope
        else:
            term = v * g * slope
            size = term.abs()
        d = torch.zeros_like(s).scatter_add_(1, at, scale * term)
        size = torch.zeros_like(s).scatter_add_(1, at, size) * (rel + k * ref.U)
    tol = abs(scale) * size + ref.TINY
    if add is not None:
        d = d + add
        tol += (add.abs() + d.abs()) * ref.U
    return d, tol


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", [(4096 * 128 + 5003, 8, 2), (4096 * 16 + 4099, 64, 8), (4096 * 4 + 1001, 256, 8),
                                   (2 * 4096 * 4 + 3, 33, 4), (4096 * 4 + 517, 320, 6)])
def test_gradient_of_more_tokens_than_workgroups(T, E, k, renormalize, score):
    """4096 workgroups take what there is in turns: every token against the plain form, some ids out of range."""
    _announce(f"gradient of many tokens T={T} E={E} k={k} {score} {renormalize}")
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.topk(torch.rand((T, E), generator=g, device="cuda"), k, dim=1)[1].to(torch.int32)
    spoil = torch.rand((T, k), generator=g, device="cuda") < 0.02
    idx = torch.where(spoil, torch.where(idx % 2 == 0, -1, E + 7), idx).to(torch.int32)
    dw = torch.randn((T, k), generator=g, device="cuda")
    for add in (None, torch.randn((T, E), generator=g, device="cuda")):
        got = moe.moe_route_scored_grad(x, idx, dw, score=score, renormalize=renormalize, scale=2.5, add=add)
        want, tol = plain_grad(x, idx, dw, add, score, renormalize, 2.5)
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), (bad.sum().item(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())
