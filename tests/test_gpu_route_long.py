"""GPU tests of scored routing from a few thousand tokens on, where 16 lanes take a token, against a plain
form in 64 bits that works on all tokens at once."""
import numpy as np
import pytest
import torch

import block_ref as ref
from combine_moe_route_03_amd import _lib as moe
from gpu_util import to_host
from test_gpu_block import _announce, dev, f64, off

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def largest(c, n):
    """Places of the n largest of each row, largest first, equal ones by their place."""
    return np.argsort(-c, axis=1, kind="stable")[:, :n]


def route(logits, bias, k, score, groups, kept, top, renormalize, scale):
    """Ids and weights, and the rows that they are sure in. An expert out of a kept group is behind all of a kept
    one, masked ones too. Groups may go either way where their sums differ by less than 2^-48 of the larger of |s|
    and |bias|: with s and bias as the test's ties have them, sums of different scores and biases come out equal
    but for their last bits. A row is not sure if there is such a group of other values than the last kept one."""
    T, E = logits.shape
    s = ref.scores(logits.astype(np.float64), score)
    c = s + (0.0 if bias is None else bias.astype(np.float64))
    c[np.isneginf(logits)] = -1e300                           # behind every other, and summed without infinities
    sure = np.ones(T, bool)
    if groups > 1:
        per = E // groups
        best = -np.sort(-c.reshape(T, groups, per), axis=2)[:, :, :top]
        total = np.zeros((T, groups))
        for j in range(top):
            total = total + best[:, :, j]
        total = np.where(total < -1e299, -np.inf, total)
        last = largest(total, kept)[:, -1:]
        with np.errstate(invalid="ignore"):                   # masked groups are equal, and no sums
            it = np.take_along_axis(total, last, axis=1)
            near = np.abs(total - it) < (np.abs(it) + (0.0 if bias is None else np.abs(bias).max())) * 2.0 ** -48
        other = (best != np.take_along_axis(best, last[:, :, None], axis=1)).any(axis=2)
        sure = ~(near & other).any(axis=1)
        closed = np.ones((T, groups), bool)
        np.put_along_axis(closed, largest(total, kept), False, axis=1)
        c[np.repeat(closed, per, axis=1)] = -np.inf
    idx = largest(c, k)
    w = np.take_along_axis(s, idx, axis=1)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return idx.astype(np.int32), w * scale, sure


def check(logits, bias, k, score, groups, kept, top, renormalize, scale, times=1):
    """Ids and weights of the rows, laid end to end `times` times."""
    idx, w = moe.moe_route_scored(dev(np.tile(logits, (times, 1))), k, score=score,
                                  bias=None if bias is None else dev(bias), n_groups=groups, topk_groups=kept,
                                  group_top=top, renormalize=renormalize, scale=scale)
    want, ww, sure = route(logits, bias, k, score, groups, kept, top, renormalize, scale)
    assert sure.mean() > 0.75
    idx, w = to_host(idx).reshape(times, -1, k)[:, sure], f64(w).reshape(times, -1, k)[:, sure]
    want, ww = np.tile(want[sure], (times, 1, 1)), np.tile(ww[sure], (times, 1, 1))
    assert np.array_equal(idx, want), np.argwhere(idx != want)[0]
    off(w, ww, np.abs(ww) * (ref.U * 1.001) + 2.0 ** -149, "weights")   # one rounding


# Below and from the lengths where 16 lanes take a token on, every number of experts that a lane holds, and
# the most choices and groups that 16 lanes take.
LONG = [
    # T, E, k, groups, kept, top
    (4095, 33, 4, 3, 1, 2), (4096, 64, 8, 8, 4, 2), (4097, 1, 1, 1, 1, 1), (4097, 7, 3, 1, 1, 1),
    (4097, 7, 7, 7, 7, 1), (4097, 32, 16, 16, 9, 2), (4099, 33, 4, 3, 2, 3), (4111, 64, 1, 1, 1, 1),
    (4097, 100, 16, 4, 2, 25), (4100, 128, 16, 16, 8, 3), (4097, 129, 8, 3, 2, 2), (4097, 160, 6, 8, 3, 1),
    (4109, 160, 16, 16, 10, 3), (8191, 161, 8, 7, 3, 2), (8193, 161, 8, 7, 3, 2), (8193, 256, 8, 8, 4, 2),
    (8193, 256, 16, 1, 1, 1), (8200, 256, 16, 16, 1, 3), (4097, 64, 17, 1, 1, 1), (4097, 64, 8, 32, 8, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,renormalize,scale", [(False, True, 1.0), (True, False, 2.5)])
@pytest.mark.parametrize("T,E,k,groups,kept,top", LONG)
def test_route_scored_long(T, E, k, groups, kept, top, biased, renormalize, scale, score):
    _announce(f"route_scored long T={T} E={E} k={k} groups={groups},{kept},{top} {score} {biased}")
    rng = np.random.default_rng(T * E + k)
    logits = (2 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    check(logits, bias, k, score, groups, kept, top, renormalize, scale)


SHAPES = [(7, 3, 1, 1, 1), (32, 8, 4, 2, 2), (60, 6, 4, 2, 2), (64, 8, 1, 1, 1), (128, 16, 16, 8, 3), (160, 6, 8, 3, 1),
          (256, 8, 8, 4, 2), (256, 16, 1, 1, 1)]


def mixed(rng, *kinds):
    """Rows of all kinds side by side, so that a wavefront has several."""
    rows = np.concatenate([np.atleast_2d(k) for k in kinds]).astype(np.float32)
    return rows[rng.permutation(len(rows))]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept,top", SHAPES)
def test_route_scored_long_ties(E, k, groups, kept, top, score):
    """Equal logits and biases, logits in bf16, values one step apart, choices that all lie with one lane, and
    biases that make up for the scores' differences, among rows that have nothing of it."""
    _announce(f"route_scored long, ties E={E} k={k} groups={groups} {score}")
    rng = np.random.default_rng(E + k)
    one_lane = rng.standard_normal((30, E))
    one_lane[:, 3 % E::16] += 8.0
    rows = mixed(rng, rng.integers(0, 3, (40, E)), torch.from_numpy(rng.standard_normal((40, E))).bfloat16().float(),
                 np.float32(0.3) + (rng.integers(0, 4, (40, E)) * 2.0 ** -24).astype(np.float32), np.zeros((2, E)),
                 one_lane, 2 * rng.standard_normal((41, E)))
    times = -(-8200 // len(rows))
    for bias in (None, (rng.integers(0, 3, E) * 0.25).astype(np.float32),
                 (rng.integers(0, 4, E) * 2.0 ** -26).astype(np.float32)):
        check(rows, bias, k, score, groups, kept, top, True, 1.0, times)
    l = rng.standard_normal((1, E)).astype(np.float32)
    bias = (0.75 - ref.scores(l.astype(np.float64), score)[0]).astype(np.float32)
    check(l, bias, k, score, groups, kept, top, False, 1.0, 8201)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept,top", SHAPES)
def test_route_scored_long_masks_and_extremes(E, k, groups, kept, top, score):
    _announce(f"route_scored long, masks E={E} k={k} groups={groups} {score}")
    rng = np.random.default_rng(E + 1)
    inf, low = np.inf, np.finfo(np.float32).min
    one, some, lowest, tail = np.full(E, -inf), rng.standard_normal((9, E)), rng.standard_normal(E), np.full(E, -inf)
    one[E // 2], tail[-1], lowest[::3] = -3.0, 5.0, low
    some[rng.random(some.shape) < 0.6] = -inf
    rows = mixed(rng, np.full(E, -inf), np.full(E, low), np.zeros(E), one, some, rng.standard_normal((5, E)) * 60,
                 lowest, tail, rng.standard_normal((20, E)))
    times = -(-8200 // len(rows))
    for bias in (None, (rng.random(E) - 0.5).astype(np.float32)):
        check(rows, bias, k, score, groups, kept, top, True, 1.0, times)
        check(rows, bias, k, score, groups, kept, top, False, -2.0, times)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_long_ids_are_valid_whatever_the_logits(score):
    """NaN and infinities: ids are distinct, there and of kept groups; rows without any have the ids that they
    have alone."""
    _announce(f"route_scored long, NaN and infinity {score}")
    rng = np.random.default_rng(2)
    for E, k, groups, kept in ((60, 7, 1, 1), (60, 7, 4, 2), (160, 6, 8, 3), (256, 16, 16, 2)):
        l = rng.standard_normal((8200, E)).astype(np.float32)
        clean = rng.random(len(l)) < 0.5
        spoiled = l[~clean]
        spoiled[rng.random(spoiled.shape) < 0.3] = np.nan
        spoiled[rng.random(spoiled.shape) < 0.2] = np.inf
        spoiled[rng.random(spoiled.shape) < 0.2] = -np.inf
        spoiled[0] = np.nan
        l[~clean] = spoiled
        idx = to_host(moe.moe_route_scored(dev(l), k, score=score, n_groups=groups, topk_groups=kept, group_top=2)[0])
        assert ((idx >= 0) & (idx < E)).all()
        each = np.sort(idx, axis=1)
        assert (each[:, 1:] != each[:, :-1]).all()
        of = np.sort(idx // (E // groups), axis=1)
        assert (1 + (of[:, 1:] != of[:, :-1]).sum(axis=1)).max() <= kept
        want = route(l[clean], None, k, score, groups, kept, 2, True, 1.0)[0]
        assert np.array_equal(idx[clean], want)


@pytest.mark.parametrize("T,E,k", [(2 ** 28 + 5, 1, 1), (2 ** 26 + 5, 17, 17)])
def test_route_scored_of_more_tokens_than_a_launch_takes(T, E, k):
    """2^32 threads and more, by 16 lanes a token and by 64: tokens at the ends, and around every border where a
    launch of 2^31 threads can end, have what they have alone."""
    _announce(f"route_scored of {T} tokens, E={E} k={k}")
    logits = torch.empty((T, E), device="cuda").normal_()
    idx, w = moe.moe_route_scored(logits, k, score="sigmoid", renormalize=False)
    lanes = 16 if k <= 16 else 64
    for at in (0, 2 ** 31 // lanes, 2 ** 32 // lanes, T - 1):
        rows = slice(max(0, at - 40), min(T, at + 40))
        ti, tw = moe.moe_route_scored(logits[rows].contiguous(), k, score="sigmoid", renormalize=False)
        assert torch.equal(idx[rows], ti) and torch.equal(w[rows], tw), at
    assert int(idx.min()) == 0 and int(idx.max()) == E - 1
    del logits, idx, w
    torch.cuda.empty_cache()
