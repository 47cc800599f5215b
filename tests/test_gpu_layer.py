"""GPU tests of the operators of include/moe_layer.h against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from combine_moe_route_03_amd import _lib as moe
from gpu_util import to_host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def _announce(msg):
    print(f"[gpu] {msg}", flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------------------ 8-bit rows --
def check_quant(x):
    q, scale = moe.moe_quant_rows(x)
    want_q, want_s = ref.quant(f64(x))
    assert np.array_equal(to_host(q), want_q)
    assert np.array_equal(to_host(scale), want_s, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,H", [(1, 16), (3, 64), (17, 512), (5, 528), (130, 1040), (33, 2048),
                                 (2, 2064), (128, 7168), (7, 8192), (4, 8208), (2, 40960)])
def test_quant_rows(R, H, dtype):
    _announce(f"quant_rows R={R} H={H} {dtype}")
    g = torch.Generator().manual_seed(R * H)
    x = torch.randn((R, H), generator=g) * torch.exp(2 * torch.randn((R, 1), generator=g))
    check_quant(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_rows_at_rounding_borders(dtype):
    """Quotients on and next to halves: small integers over every maximum up to 254, their
    neighbours one step away, and magnitudes from subnormal to the largest."""
    _announce(f"quant_rows borders {dtype}")
    rows = []
    for a in range(1, 255):
        v = np.arange(0, 255, dtype=np.float64) * (a / 254.0)
        rows.append(np.concatenate([[a], v]))
    x = torch.tensor(np.array(rows)).to(dtype)
    x = torch.cat([x, torch.nextafter(x, torch.full_like(x, np.inf)),
                   torch.nextafter(x, torch.full_like(x, -np.inf))])
    x[:, 0] = torch.arange(1, 255).repeat(3).to(dtype)
    check_quant((x * torch.where(torch.arange(256) % 2 == 0, 1, -1).to(dtype)).cuda())
    for e in (-149, -140, -133, -126, -100, -65, -64, -63, 60, 119):
        check_quant((x.double() * 2.0 ** e).to(dtype).cuda())


def test_quant_rows_special_rows():
    _announce("quant_rows special rows")
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn((9, 96)).to(dtype)
        x[0] = 0
        x[1, 5] = float("nan")
        x[2, 95] = float("inf")
        x[3, 0] = -float("inf")
        x[4] = float("nan")
        x[5] = torch.finfo(dtype).max
        x[6] = -0.0
        x[7, 1:] = 0
        check_quant(x.cuda())


@pytest.mark.parametrize("H", [64, 2048, 4096, 8224])
@pytest.mark.parametrize("n", [0, 1, 5, 13, 14, 99, -3])
def test_quant_rows_leaves_rows_behind_n_rows(n, H):
    _announce(f"quant_rows n_rows={n} H={H}")
    x = torch.randn((13, H)).cuda()
    q = torch.full((13, H), 77, dtype=torch.int8, device="cuda")
    s = torch.full((13,), -5.0, device="cuda")
    moe.moe_quant_rows(x, q=q, scale=s, n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
    m = min(max(n, 0), 13)
    want_q, want_s = ref.quant(f64(x))
    assert np.array_equal(to_host(q)[:m], want_q[:m]) and (to_host(q)[m:] == 77).all()
    assert np.array_equal(to_host(s)[:m], want_s[:m]) and (to_host(s)[m:] == -5.0).all()


# ------------------------------------------------------------------------ experts' product --
def counts_of(kind, E, R, rng):
    """Rows of each expert, R in all."""
    if kind == "even":
        c = np.full(E, R // E)
        c[: R % E] += 1
    elif kind == "one":                                  # all rows with one expert
        c = np.zeros(E, np.int64)
        c[E // 2] = R
    else:                                                # uneven, some experts without rows
        p = rng.random(E) ** 4
        p[rng.random(E) < 0.3] = 0
        p[E - 1] += 1e-3
        c = rng.multinomial(R, p / p.sum())
    return c


def make_matmul(T, k, E, N, K, act, gather, kind, seed=0, extreme=False):
    rng = np.random.default_rng(seed)
    R = T * k
    c = counts_of(kind, E, R, rng)
    offsets = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    A = T if gather else R
    n_w = 2 * N if act == "swiglu" else N
    lim = 128 if extreme else 127
    a = rng.integers(-lim, 128, (A, K)).astype(np.int8)
    w = rng.integers(-lim, 128, (E, n_w, K)).astype(np.int8)
    if extreme:
        a[0], w[:, 0] = -128, -128
    sa = (rng.random(A) + 0.5).astype(np.float32) / 64
    sw = ((rng.random((E, n_w)) + 0.5) / (64 * np.sqrt(K))).astype(np.float32)
    rt = rng.permutation(np.repeat(np.arange(T), k)).astype(np.int32) if gather else None
    return a, sa, w, sw, offsets, rt


def run_matmul(m, act, dtype, out=None, plain=False):
    a, sa, w, sw, off, rt = m
    return moe.moe_expert_matmul_i8(dev(a), dev(sa), dev(w), dev(sw), None if plain else dev(off),
                                    row_token=None if rt is None else dev(rt), act=act, out=out,
                                    out_dtype=dtype)


def check_matmul(m, act, dtype, plain=False):
    R = len(m[5]) if m[5] is not None else m[0].shape[0]
    N = m[2].shape[1] // (2 if act == "swiglu" else 1)
    out = torch.full((R, N), 12345.0, dtype=dtype, device="cuda")
    got = f64(run_matmul(m, act, dtype, out, plain))
    want, tol, done = ref.matmul(*m, act, dtype == torch.bfloat16)
    bad = np.abs(got - want)[done] > tol[done]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}"
    left = f64(torch.tensor(12345.0, dtype=dtype))
    assert (got[~done] == left).all()


SHAPES = [
    # T, k, E, N, K, kind: one token to many, tiles that end inside, odd channels
    (1, 1, 1, 16, 16, "even"), (1, 1, 1, 1, 64, "even"), (1, 2, 4, 40, 80, "uneven"),
    (3, 2, 8, 33, 128, "uneven"), (16, 1, 1, 64, 144, "even"), (17, 1, 1, 130, 272, "even"),
    (40, 4, 8, 7, 1040, "uneven"), (64, 2, 60, 96, 512, "uneven"), (65, 1, 2, 200, 400, "one"),
    (128, 8, 256, 48, 256, "uneven"), (100, 3, 5, 264, 2064, "uneven"),
    (300, 2, 3, 520, 208, "uneven"), (700, 1, 1, 300, 640, "even"), (513, 2, 2, 257, 128, "even"),
    (1100, 1, 4, 640, 160, "one"), (40, 8, 1024, 20, 48, "uneven"),
]


@pytest.mark.parametrize("act,dtype", [("none", torch.float32), ("none", torch.bfloat16),
                                       ("swiglu", torch.float32), ("swiglu", torch.bfloat16)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,k,E,N,K,kind", SHAPES)
def test_expert_matmul(T, k, E, N, K, kind, gather, act, dtype):
    _announce(f"matmul T={T} k={k} E={E} N={N} K={K} {kind} gather={gather} {act} {dtype}")
    check_matmul(make_matmul(T, k, E, N, K, act, gather, kind, seed=T + N), act, dtype)


# Enough tiles for every tile shape, persistent workgroups that take several tiles, K of one step,
# two, three and more, whole and ragged, channels that fill no block and rows of out off 16 bytes.
TILE_SHAPES = [
    (1100, 4, 1100, 48, "uneven", "none"), (350, 64, 520, 80, "uneven", "swiglu"),
    (1024, 1, 2056, 2064, "even", "none"),
    (2000, 40, 1000, 208, "uneven", "none"), (2000, 40, 996, 336, "uneven", "swiglu"),
    (1024, 1, 4096, 1024, "even", "none"),
    (1700, 20, 1100, 912, "uneven", "swiglu"), (2600, 40, 1100, 912, "uneven", "none"),
    (1024, 1, 4096, 1024, "even", "swiglu"),
    (4096, 2, 2048, 64, "uneven", "none"), (3000, 1, 2049, 144, "even", "swiglu"),
    (9000, 2, 1536, 128, "uneven", "none"), (3000, 3, 1028, 272, "one", "swiglu"),
    (6000, 2, 2056, 400, "uneven", "none"), (6000, 2, 1028, 400, "uneven", "swiglu"),
    (12000, 3, 1000, 384, "uneven", "none"), (8000, 4, 602, 528, "uneven", "swiglu"),
    (4000, 1, 2056, 272, "even", "swiglu"), (6000, 2, 4100, 400, "uneven", "none"),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,N,K,kind,act", TILE_SHAPES)
def test_expert_matmul_tiles(T, E, N, K, kind, act, gather, dtype):
    _announce(f"matmul tiles T={T} E={E} N={N} K={K} {kind} {act} gather={gather} {dtype}")
    check_matmul(make_matmul(T, 1, E, N, K, act, gather, kind, seed=T + N + K), act, dtype)


@pytest.mark.parametrize("T,E,N,K", [(1100, 4, 1100, 48), (2000, 40, 1000, 208),
                                     (2600, 40, 1100, 912), (3000, 2, 2056, 144),
                                     (12000, 3, 1000, 384)])
def test_expert_matmul_tiles_leave_rows_they_do_not_own(T, E, N, K):
    """Every tile shape: rows behind the last expert's, rows whose row_token is out of range, and
    memory on both sides of out."""
    _announce(f"matmul tiles, rows left alone T={T} E={E} N={N} K={K}")
    m = list(make_matmul(T, 1, E, N, K, "none", True, "uneven", seed=N))
    m[4] = np.minimum(m[4], T - T // 3).astype(np.int32)
    m[5][[0, 3, T // 4, T - 1]] = [-1, T, 2 ** 31 - 1, -2 ** 31]
    check_matmul(m, "none", torch.bfloat16)
    room = torch.full((T * N + 16,), 12345.0, dtype=torch.bfloat16, device="cuda")
    for at in (8, 1):                                    # 16-byte aligned, and 2
        room.fill_(12345.0)
        out = room[at:at + T * N].view(T, N)
        a, sa, w, sw, off, rt = m
        moe.moe_expert_matmul_i8(dev(a), dev(sa), dev(w), dev(sw), dev(off), row_token=dev(rt),
                                 out=out)
        want, tol, done = ref.matmul(*m, "none", True)
        got = f64(out)
        left = f64(torch.tensor(12345.0, dtype=torch.bfloat16))
        assert (np.abs(got - want)[done] <= tol[done]).all() and (got[~done] == left).all()
        assert (f64(room[:at]) == left).all() and (f64(room[at + T * N:]) == left).all()


def test_expert_matmul_tiles_of_one_expert_without_rows_between():
    """Experts without rows before, between and behind the ones that have them."""
    _announce("matmul tiles, empty experts")
    rng = np.random.default_rng(8)
    c = np.zeros(200, np.int64)
    c[[3, 4, 70, 131, 199]] = [500, 1, 129, 900, 257]
    m = list(make_matmul(int(c.sum()), 1, 200, 136, 160, "none", True, "even", seed=8))
    m[4] = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    m[5] = rng.permutation(int(c.sum())).astype(np.int32)
    check_matmul(m, "none", torch.float32)


@pytest.mark.parametrize("T,N,K", [(1, 4096, 7168), (5, 70, 96), (260, 300, 336)])
def test_plain_product(T, N, K):
    _announce(f"matmul without offsets T={T} N={N} K={K}")
    check_matmul(make_matmul(T, 1, 1, N, K, "none", False, "even", seed=9), "none",
                 torch.float32, plain=True)


@pytest.mark.parametrize("T", [1, 300])
def test_expert_matmul_largest_sums(T):
    """-128 * -128 over the longest K: 2147221504 of the int32's 2147483647."""
    _announce(f"matmul largest sums T={T}")
    m = make_matmul(T, 1, 1, 17, moe.MOE_MATMUL_MAX_K, "none", False, "even", extreme=True)
    m[0][-1] = -128
    m[2][0, -1] = -128
    check_matmul(m, "none", torch.float32)


@pytest.mark.parametrize("T,E", [(24, 8), (900, 3)])
def test_expert_matmul_leaves_rows_it_does_not_own(T, E):
    """Rows behind the last expert's, and rows whose row_token lies outside the rows of a."""
    _announce(f"matmul rows left alone T={T} E={E}")
    m = list(make_matmul(T, 1, E, 72, 192, "none", False, "uneven", seed=4))
    m[4] = np.minimum(m[4], T - T // 3).astype(np.int32)
    check_matmul(m, "none", torch.bfloat16)
    m = list(make_matmul(T, 1, E, 72, 192, "swiglu", True, "uneven", seed=5))
    m[5][[0, 3, T - 1]] = [-1, T, 2 ** 31 - 1]
    check_matmul(m, "swiglu", torch.float32)


def test_expert_matmul_nan_scale_reaches_its_rows_only():
    _announce("matmul NaN scale")
    m = list(make_matmul(50, 1, 4, 64, 128, "swiglu", True, "uneven", seed=6))
    m[1][7] = np.nan
    got = f64(run_matmul(m, "swiglu", torch.float32))
    rows = m[5] == 7
    assert np.isnan(got[rows]).all() and np.isfinite(got[~rows]).all()


GATES = [0.5, 20.0, 43.0, 64.1, 87.5, 88.5, 90.0, 133.0, 1e3, 1e30, 2.3e38, 2.36e38, 2.4e38, 3.4e38,
         np.inf, -0.5, -20.0, -43.0, -1e3, -1e30, -2.3e38, -2.36e38, -2.4e38, -3.4e38, -np.inf,
         -44.0, -45.0, -50.0, -63.9, -64.1, -66.0, -67.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0,
         -92.0, -95.0, -100.0, -110.0, -133.0, -178.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,N,E,K", [(60, 40, 8, 16), (60, 40, 1, 160), (104, 264, 30, 144),
                                     (2000, 996, 40, 336), (3000, 2049, 1, 16),
                                     (9000, 1032, 4, 1424), (6000, 1028, 2, 400),
                                     (4000, 2056, 1, 272)])
def test_expert_matmul_swiglu_over_the_range_of_gates(R, N, E, K, dtype):
    """silu(gate) * up for gates of both signs from 0.5 to infinity, by few rows and by tiles. A row
    has |gate| as its scale and the gate's sign in its first code, so that y is exactly the fp32
    product of scales: the gate is row scale times 1 or 2, up is row scale times 2^-130 to 1e30.
    Off by exp 3u, 1 + exp u, reciprocal 2u (far below zero two reciprocals of sqrt(exp), 5u each)
    and two or three products: 13u at most, taken as 16u for the second order; by what silu loses
    below 2^-126, four halves of its last place 2^-149, times up; by a result below 2^-126, which
    may be flushed; and by the last rounding."""
    _announce(f"matmul gates R={R} N={N} E={E} K={K} {dtype}")
    gates = np.array(GATES)[np.arange(R) * 7 % len(GATES)]
    a = np.zeros((R, K), np.int8)
    a[:, 0], a[:, 1] = np.sign(gates), 1
    w = np.zeros((E, 2 * N, K), np.int8)
    w[:, :N, 0], w[:, N:, 1] = 1, 1
    sa = np.abs(gates).astype(np.float32)
    sw = np.empty((E, 2 * N), np.float32)
    sw[:, :N] = np.array([1.0, 2.0], np.float32)[np.arange(N) // 4 % 2]
    sw[:, N:] = np.array([1.0, 1e-3, 1e30, 2.0 ** -130], np.float32)[np.arange(N) % 4]
    off = (np.arange(E + 1) * R // E).astype(np.int32)
    got = f64(run_matmul((a, sa, w, sw, off, None), "swiglu", dtype))
    u, half = ref.U, torch.finfo(dtype).eps / 2
    with np.errstate(all="ignore"):
        gate = ((a[:, :1] * sa[:, None]) * sw[0, :N]).astype(np.float64)
        up = (sa[:, None] * sw[0, N:]).astype(np.float64)
        want = ref.silu(gate) * up
        tol = np.abs(want) * (16 * u + half) + np.abs(up) * 4 * 2.0 ** -150 + 2.0 ** -126
        top = f64(torch.from_numpy(want).to(dtype))              # what the type cannot hold
        assert np.array_equal(np.isnan(got), np.isnan(want))
        inf = np.isinf(top)
        assert np.array_equal(got[inf], top[inf])
        rest = np.isfinite(top)
        bad = np.abs(got - want)[rest] > tol[rest]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, gates {np.unique(gate[rest][bad])}"


def test_expert_matmul_swiglu_of_a_row_does_not_depend_on_its_neighbours():
    """Rows whose gates take the plain form of silu, beside rows that take the one of any gate."""
    _announce("matmul gates beside each other")
    for T, N, K in ((24, 40, 64), (1040, 264, 64)):
        m = list(make_matmul(T, 1, 1, N, K, "swiglu", False, "even", seed=T))
        m[3] *= 8.0                                          # gates to some tens
        plain = run_matmul(m, "swiglu", torch.float32)
        m[1][::3] *= 1e3
        mixed = run_matmul(m, "swiglu", torch.float32)
        same = torch.arange(T) % 3 != 0
        assert torch.equal(plain[same], mixed[same]) and torch.isfinite(plain).all()


def test_expert_matmul_empty():
    _announce("matmul empty")
    m = make_matmul(4, 1, 4, 64, 128, "none", False, "one")
    out = moe.moe_expert_matmul_i8(dev(m[0])[:0], dev(m[1])[:0], dev(m[2]), dev(m[3]),
                                   dev(np.zeros(5, np.int32)))
    assert out.shape == (0, 64)


# ---------------------------------------------------------------------- loss and gradient --
def make_balance(T, S, E, k, masked, seed=0, spread=2.0):
    rng = np.random.default_rng(seed)
    logits = (spread * rng.standard_normal((T, E))).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = None
    if masked:
        mask = (np.arange(T // S)[None, :] < rng.integers(0, T // S + 1, S)[:, None]).reshape(-1)
        mask[:T // S] = rng.random(T // S) < 0.5         # holes in the first sequence
        if S > 1:
            mask[T - T // S:] = False                    # nothing left in the last of several
    kept = np.take_along_axis(logits, idx, 1).astype(np.float64)
    w = np.exp(kept - kept.max(axis=1, keepdims=True))
    w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
    dw = (rng.standard_normal((T, k)) / T).astype(np.float32)
    return logits, idx, mask, w, dw


def check_balance(logits, idx, mask, w, dw, S, alpha, stream=None):
    T, E = logits.shape
    dm = None if mask is None else dev(mask)
    out = moe.moe_balance_loss(dev(logits), dev(idx), alpha, n_seqs=S, token_mask=dm)
    loss, counts, sums, tokens = [to_host(t) for t in out]
    l64 = logits.astype(np.float64)
    r_loss, r_counts, r_sums, r_tokens = ref.balance(l64, idx, mask, S, alpha)
    assert np.array_equal(counts, r_counts) and np.array_equal(tokens, r_tokens)
    # all terms are positive: a probability's error, and the additions of a workgroup's chain
    rel = ref.prob_error(l64) + 100 * ref.U
    assert (np.abs(sums - r_sums) <= rel * r_sums + 2.0 ** -120).all()
    assert abs(loss[0] - r_loss) <= rel * r_loss
    g = torch.tensor([0.75], device="cuda")
    for parts in ("both", "loss", "weights"):
        kw = {}
        if parts != "weights":
            kw |= dict(expert_counts=out[1], seq_tokens=out[3], token_mask=dm, dloss=g)
        if parts != "loss":
            kw |= dict(topk_w=dev(w), dtopk_w=dev(dw))
        d = f64(moe.moe_route_grad(dev(logits), dev(idx), alpha=alpha, n_seqs=S, **kw))
        want, tol = ref.route_grad(l64, idx, None if parts == "loss" else w.astype(np.float64),
                                   dw.astype(np.float64), mask,
                                   None if parts == "weights" else r_counts, r_tokens, 0.75, S,
                                   alpha)
        bad = np.abs(d - want) > tol
        assert not bad.any(), (parts, int(bad.sum()), np.argwhere(bad)[0])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,S,E,k", [
    (1, 1, 1, 1), (1, 1, 8, 2), (2, 2, 4, 4), (7, 7, 8, 8), (33, 1, 16, 2), (128, 1, 256, 8),
    (96, 3, 60, 4), (50, 2, 7, 3), (130, 1, 130, 5), (257, 1, 384, 8), (40, 4, 513, 6),
    (24, 2, 1024, 64), (600, 1, 1000, 8), (300, 3, 24, 24), (4099, 1, 64, 6), (2050, 2, 160, 4),
    (640, 640, 12, 2), (65, 5, 33, 33)])
def test_balance_loss_and_gradient(T, S, E, k, masked):
    _announce(f"balance T={T} S={S} E={E} k={k} masked={masked}")
    check_balance(*make_balance(T, S, E, k, masked, seed=T + E), S, 0.01)


def test_balance_minus_infinity_and_large_logits():
    """Experts masked by -infinity, rows with one finite logit, rows with none, the type's lowest
    value as a mask, and a spread beyond exp's range."""
    _announce("balance masked experts")
    logits, idx, mask, w, dw = make_balance(90, 2, 32, 4, True, seed=1)
    logits[:, 20:] = -np.inf
    logits[3, 1:] = -np.inf
    logits[4] = -np.inf
    logits[5, 2:] = np.finfo(np.float32).min
    logits[6] = np.finfo(np.float32).min
    logits[7, 3] = 80.0
    logits[8, 3] = 1e30
    check_balance(logits, idx, mask, w, dw, 2, 0.3)


def test_balance_nan_and_infinity_reach_the_loss():
    _announce("balance NaN")
    for bad in (np.nan, np.inf):
        logits, idx, _, _, _ = make_balance(70, 1, 16, 2, False, seed=2)
        logits[11, 5] = bad
        loss, counts, sums, tokens = moe.moe_balance_loss(dev(logits), dev(idx), 0.1)
        assert torch.isnan(loss).all() and torch.isnan(sums).all()
        d = to_host(moe.moe_route_grad(dev(logits), dev(idx), expert_counts=counts,
                                       seq_tokens=tokens, alpha=0.1))
        assert np.isnan(d[11]).all() and np.isfinite(np.delete(d, 11, 0)).all()


def test_balance_ids_out_of_range_and_repeated():
    _announce("balance odd ids")
    logits, idx, mask, w, dw = make_balance(200, 2, 20, 4, True, seed=3)
    idx[5, 1], idx[6, 2], idx[7, 0], idx[8] = -1, 20, 2 ** 31 - 1, 9
    idx[9, 1:3] = idx[9, 0]
    check_balance(logits, idx, mask, w, dw, 2, 0.05)


def test_balance_even_routing_costs_alpha():
    _announce("balance even routing")
    T, E, k = 64, 16, 2
    idx = np.stack([np.arange(T) % E, (np.arange(T) + E // 2) % E], 1).astype(np.int32)
    loss, counts, _, _ = moe.moe_balance_loss(dev(np.zeros((T, E), np.float32)), dev(idx), 0.25)
    assert (to_host(counts) == T * k // E).all()
    assert abs(float(loss) - 0.25) <= 0.25 * 130 * ref.U


def test_balance_misaligned_rows():
    """A batch that does not start on 16 bytes takes the scalar rows."""
    _announce("balance misaligned")
    logits, idx, _, w, dw = make_balance(50, 1, 16, 2, False, seed=8)
    room = torch.empty(50 * 16 + 1, device="cuda")
    view = room[1:].view(50, 16)
    view.copy_(dev(logits))
    a = moe.moe_balance_loss(view, dev(idx), 0.1)
    b = moe.moe_balance_loss(dev(logits), dev(idx), 0.1)
    assert torch.equal(a[1], b[1])
    r = ref.balance(logits.astype(np.float64), idx, None, 1, 0.1)
    rel = ref.prob_error(logits.astype(np.float64)) + 100 * ref.U
    assert (np.abs(to_host(a[2]) - r[2]) <= rel * r[2]).all()


def test_balance_empty_batch():
    _announce("balance empty")
    out = moe.moe_balance_loss(torch.empty((0, 16), device="cuda"),
                               torch.empty((0, 2), dtype=torch.int32, device="cuda"), 0.1, n_seqs=3)
    assert all((to_host(t) == 0).all() for t in out) and out[1].shape == (3, 16)


def test_balance_same_bits_twice():
    _announce("balance determinism")
    logits, idx, mask, _, _ = make_balance(5000, 4, 96, 4, True, seed=12)
    args = (dev(logits), dev(idx), 0.1)
    kw = dict(n_seqs=4, token_mask=dev(mask))
    first = moe.moe_balance_loss(*args, **kw)
    ws = moe.alloc_balance_workspace(5000, 96, 4)
    for _ in range(5):
        ws.fill_(0xFF)
        again = moe.moe_balance_loss(*args, workspace=ws, **kw)
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(first, again))


# ------------------------------------------------------------- together, as they are used --
def make_layer(T, k, E, H, inner, seed):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w1 = rng.integers(-127, 128, (E, 2 * inner, H)).astype(np.int8)
    w2 = rng.integers(-127, 128, (E, H, inner)).astype(np.int8)
    s1 = ((rng.random((E, 2 * inner)) + 0.5) / (74 * np.sqrt(H))).astype(np.float32)
    s2 = ((rng.random((E, H)) + 0.5) / (74 * np.sqrt(inner))).astype(np.float32)
    return logits, x, w1, s1, w2, s2


@pytest.mark.parametrize("T,k,E,H,inner", [(1, 2, 8, 256, 64), (37, 4, 16, 400, 176),
                                           (512, 2, 4, 512, 320)])
def test_expert_layer(T, k, E, H, inner):
    """Routing, layout, 8-bit rows, both products and combine, each stage against its plain form
    on what the stage before wrote."""
    _announce(f"expert layer T={T} k={k} E={E} H={H} inner={inner}")
    logits, x, w1, s1, w2, s2 = make_layer(T, k, E, H, inner, seed=T)
    lay = moe.alloc_dispatch_out(T, H, E, k, 1, None)
    idx, wt = moe.moe_route_topk(dev(logits), k)
    moe.moe_dispatch_layout(idx, E, 1, lay, moe.alloc_workspace(T, E, k))
    q, sx = moe.moe_quant_rows(x.cuda())
    h = moe.moe_expert_matmul_i8(q, sx, dev(w1), dev(s1), lay.expert_offsets,
                                 row_token=lay.row_token, act="swiglu")
    hq, sh = moe.moe_quant_rows(h)
    y = moe.moe_expert_matmul_i8(hq, sh, dev(w2), dev(s2), lay.expert_offsets)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_combine(y, lay.token_row, wt, out)
    off, rt = to_host(lay.expert_offsets), to_host(lay.row_token)
    for stage, src in ((x, (q, sx)), (h, (hq, sh))):
        want_q, want_s = ref.quant(f64(stage))
        assert np.array_equal(to_host(src[0]), want_q) and np.array_equal(to_host(src[1]), want_s)
    want, tol, done = ref.matmul(to_host(q), to_host(sx), w1, s1, off, rt, "swiglu", True)
    assert done.all() and (np.abs(f64(h) - want) <= tol).all()
    want, tol, done = ref.matmul(to_host(hq), to_host(sh), w2, s2, off, None, "none", True)
    assert done.all() and (np.abs(f64(y) - want) <= tol).all()
    rows = f64(y)[to_host(lay.token_row)].reshape(T, k, H) * f64(wt)[:, :, None]
    tol = np.abs(rows).sum(1) * (k + 1) * ref.U + np.abs(rows.sum(1)) * ref.BF16_HALF
    assert (np.abs(f64(out) - rows.sum(1)) <= tol + 2.0 ** -120).all()


def test_router_training_step():
    """Top-k, the loss over padded sequences, and the gradient of loss and weights together."""
    _announce("router training step")
    logits, _, mask, _, dw = make_balance(240, 3, 48, 4, True, seed=21)
    idx, wt = moe.moe_route_topk(dev(logits), 4)
    check_balance(logits, to_host(idx), mask, to_host(wt), dw, 3, 0.02)


def test_expert_layer_of_one_rank_after_receive():
    """The rows that a rank received from two sources: 8-bit rows and both products up to the rows
    received (expert_offsets of moe_ep_recv), nothing behind them."""
    _announce("expert layer after moe_ep_recv")
    S, T, E, k, N, H, inner = 2, 160, 16, 4, 2, 256, 128
    L, cap = E // N, T * 4
    rng = np.random.default_rng(5)
    regions = torch.zeros((N * S * cap, H), dtype=torch.bfloat16, device="cuda")
    counts = torch.zeros((N, S, L), dtype=torch.int32, device="cuda")
    for s in range(S):
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
        idx, _ = moe.moe_route_topk(dev(rng.standard_normal((T, E)).astype(np.float32)), k)
        moe.moe_ep_send(x.cuda(), idx, E, N, s, S, cap, regions, counts,
                        torch.empty(T * k, dtype=torch.int32, device="cuda"),
                        moe.alloc_workspace(T, E, k))
    i32 = dict(dtype=torch.int32, device="cuda")
    grouped = torch.zeros((S * cap, H), dtype=torch.bfloat16, device="cuda")
    off, src = torch.empty(L + 1, **i32), torch.empty(S * cap, **i32)
    moe.moe_ep_recv(regions, E, N, 1, S, cap, counts, grouped, torch.empty(L, **i32), off, src)
    _, _, w1, s1, w2, s2 = make_layer(1, 1, L, H, inner, seed=9)
    n = int(off[L])
    assert 0 < n < S * cap
    q = torch.full((S * cap, H), 9, dtype=torch.int8, device="cuda")
    sx = torch.full((S * cap,), -1.0, device="cuda")
    moe.moe_quant_rows(grouped, q=q, scale=sx, n_rows=off[L:])
    h = torch.full((S * cap, inner), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_matmul_i8(q, sx, dev(w1), dev(s1), off, act="swiglu", out=h)
    assert (to_host(q)[n:] == 9).all() and (f64(sx)[n:] == -1.0).all() and (f64(h)[n:] == 7.0).all()
    want_q, want_s = ref.quant(f64(grouped)[:n])
    assert np.array_equal(to_host(q)[:n], want_q) and np.array_equal(to_host(sx)[:n], want_s)
    want, tol, done = ref.matmul(to_host(q), to_host(sx), w1, s1, to_host(off), None, "swiglu", True)
    assert done[:n].all() and not done[n:].any() and (np.abs(f64(h) - want)[:n] <= tol[:n]).all()


@pytest.mark.parametrize("T,E,N,K", [(2000, 40, 1000, 208), (2600, 40, 1100, 912),
                                     (12000, 3, 1000, 384)])
def test_tiles_in_a_graph(T, E, N, K):
    """The tile shapes that take more LDS than a launch has by default, first used in a capture."""
    _announce(f"tiles in a graph T={T} E={E} N={N} K={K}")
    m = make_matmul(T, 1, E, N, K, "none", False, "uneven", seed=3)
    a, sa, w, sw, off = [dev(v) for v in m[:5]]
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_expert_matmul_i8(a, sa, w, sw, off, out=out)
    want = moe.moe_expert_matmul_i8(a, sa, w, sw, off)
    for rep in range(4):
        out.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


def test_expert_layer_and_router_step_in_a_graph():
    """Captured once, replayed several times with eager work between: bit for bit the eager run."""
    _announce("layer graph")
    T, k, E, H, inner = 48, 4, 16, 256, 128
    logits, x, w1, s1, w2, s2 = make_layer(T, k, E, H, inner, seed=77)
    logits, x, w1, s1, w2, s2 = dev(logits), x.cuda(), dev(w1), dev(s1), dev(w2), dev(s2)
    lay = moe.alloc_dispatch_out(T, H, E, k, 1, None)
    ws, bws = moe.alloc_workspace(T, E, k), moe.alloc_balance_workspace(T, E, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(idx=torch.empty((T, k), **i32), wt=torch.empty((T, k), device="cuda"),
             q=torch.empty((T, H), dtype=torch.int8, device="cuda"), sx=torch.empty(T, device="cuda"),
             h=torch.empty((T * k, inner), dtype=torch.bfloat16, device="cuda"),
             hq=torch.empty((T * k, inner), dtype=torch.int8, device="cuda"),
             sh=torch.empty(T * k, device="cuda"),
             y=torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda"),
             out=torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
             loss=torch.empty(1, device="cuda"), counts=torch.empty((2, E), **i32),
             sums=torch.empty((2, E), device="cuda"), tokens=torch.empty(2, **i32),
             d=torch.empty((T, E), device="cuda"))

    def step():
        moe.moe_route_topk(logits, k, topk_idx=o["idx"], topk_w=o["wt"])
        moe.moe_dispatch_layout(o["idx"], E, 1, lay, ws)
        moe.moe_quant_rows(x, q=o["q"], scale=o["sx"])
        moe.moe_expert_matmul_i8(o["q"], o["sx"], w1, s1, lay.expert_offsets,
                                 row_token=lay.row_token, act="swiglu", out=o["h"])
        moe.moe_quant_rows(o["h"], q=o["hq"], scale=o["sh"])
        moe.moe_expert_matmul_i8(o["hq"], o["sh"], w2, s2, lay.expert_offsets, out=o["y"])
        moe.moe_combine(o["y"], lay.token_row, o["wt"], o["out"])
        moe.moe_balance_loss(logits, o["idx"], 0.1, n_seqs=2, loss=o["loss"],
                             expert_counts=o["counts"], prob_sums=o["sums"],
                             seq_tokens=o["tokens"], workspace=bws)
        moe.moe_route_grad(logits, o["idx"], topk_w=o["wt"], dtopk_w=o["wt"],
                           expert_counts=o["counts"], seq_tokens=o["tokens"], alpha=0.1, n_seqs=2,
                           dlogits=o["d"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in o.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        for t in o.values():
            t.view(torch.uint8).fill_(0xA5)
        bws.fill_(0x5A)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in o.items():
            assert torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)), (n, rep)


def test_two_streams_at_once():
    """Calls that run at the same time on streams of their own, each with its own workspace."""
    _announce("two streams")
    sets = []
    for i in range(2):
        logits, idx, mask, _, _ = make_balance(4000, 2, 64, 4, True, seed=30 + i)
        m = [dev(v) for v in make_matmul(200, 2, 8, 128, 512, "swiglu", True, "uneven", seed=i)]
        sets.append((dev(logits), dev(idx), dev(mask), m))

    def work(s, stream=None):
        a = moe.moe_balance_loss(s[0], s[1], 0.1, n_seqs=2, token_mask=s[2], stream=stream)
        m = s[3]
        b = moe.moe_expert_matmul_i8(m[0], m[1], m[2], m[3], m[4], row_token=m[5], act="swiglu",
                                     stream=stream)
        return [*a, b]

    want = [work(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [work(s, stream) for s, stream in zip(sets, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


# --------------------------------------------------------------- offsets beyond 32 bits --
def big(*shape):
    """Random 8-bit values, without a copy of them in a wider type."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    g = torch.Generator(device="cuda").manual_seed(len(flat) % 1000)
    for i in range(0, flat.numel(), 1 << 28):
        flat[i:i + (1 << 28)].random_(-127, 128, generator=g)
    return out


def test_quant_rows_beyond_2_31_elements():
    _announce("quant_rows beyond 2^31 elements")
    R, H = 300000, 8192
    x = torch.empty((R, H), dtype=torch.bfloat16, device="cuda").normal_()
    q, s = moe.moe_quant_rows(x)
    rows = [0, 1, R // 2, 2 ** 31 // H - 1, 2 ** 31 // H, R - 2, R - 1]
    want_q, want_s = ref.quant(f64(x[rows]))
    assert np.array_equal(to_host(q[rows]), want_q) and np.array_equal(to_host(s[rows]), want_s)


@pytest.mark.parametrize("R", [40, 700])
def test_expert_matmul_rows_and_weights_beyond_2_31_bytes(R):
    """Rows gathered from 2.5 GB, and an expert's weights of 2.5 GB, by few rows and by tiles."""
    _announce(f"matmul beyond 2^31 bytes R={R}")
    K, big_n = 8192, 300000
    rng = np.random.default_rng(1)
    a = big(big_n, K)
    rt = rng.integers(0, big_n, R).astype(np.int32)
    rt[:4] = [0, big_n - 1, 2 ** 31 // K, 2 ** 31 // K - 1]
    w = big(2, 264, K)
    sa, sw = torch.rand(big_n, device="cuda"), torch.rand((2, 264), device="cuda") / 1e5
    off = np.array([0, R // 3, R], np.int32)
    got = f64(moe.moe_expert_matmul_i8(a, sa, w, sw, dev(off), row_token=dev(rt),
                                       out_dtype=torch.float32))
    small = a[dev(rt).long()]
    want, tol, _ = ref.matmul(to_host(small), to_host(sa[dev(rt).long()]), to_host(w), to_host(sw),
                              off, None, "none", False)
    assert (np.abs(got - want) <= tol).all()
    del a
    w = big(2, big_n, K)
    sw = torch.rand((2, big_n), device="cuda") / 1e5
    x, sx = small, torch.rand(R, device="cuda")
    got = moe.moe_expert_matmul_i8(x, sx, w, sw, dev(off), out_dtype=torch.float32)
    cols = [0, 1, 2 ** 31 // K - 1, 2 ** 31 // K, big_n - 2, big_n - 1]
    want, tol, _ = ref.matmul(to_host(x), to_host(sx), to_host(w[:, cols].contiguous()),
                              to_host(sw[:, cols].contiguous()), off, None, "none", False)
    assert (np.abs(f64(got[:, cols]) - want) <= tol).all()


@pytest.mark.parametrize("N", [40000, 40001])
def test_expert_matmul_results_beyond_2_31_elements(N):
    _announce(f"matmul results beyond 2^31 elements N={N}")
    R, K = 60000, 32
    a, w = big(R, K), big(3, N, K)
    sa, sw = torch.rand(R, device="cuda"), torch.rand((3, N), device="cuda")
    off = np.array([0, 100, 50000, R], np.int32)
    got = moe.moe_expert_matmul_i8(a, sa, w, sw, dev(off))
    rows = np.array([0, 99, 100, 49999, 50000, 2 ** 31 // N - 1, 2 ** 31 // N, 2 ** 31 // N + 1,
                     R - 1])
    for e in range(3):
        r = rows[(rows >= off[e]) & (rows < off[e + 1])]
        d = dev(r)
        want, tol, _ = ref.matmul(to_host(a[d]), to_host(sa[d]), to_host(w[e:e + 1]),
                                  to_host(sw[e:e + 1]), [0, len(r)], None, "none", True)
        assert (np.abs(f64(got[d]) - want) <= tol).all()


def test_balance_beyond_2_31_logits():
    _announce("balance beyond 2^31 logits")
    T, E, k, S = 2200000, 1024, 2, 2
    logits = torch.empty((T, E), device="cuda").normal_()
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    loss, counts, sums, tokens = moe.moe_balance_loss(logits, idx, 0.01, n_seqs=S)
    assert to_host(tokens).tolist() == [T // S] * S
    for s in range(S):
        part = slice(s * (T // S), (s + 1) * (T // S))
        assert torch.equal(counts[s].long(), torch.bincount(idx[part].reshape(-1).long(), minlength=E))
        want = torch.zeros(E, dtype=torch.float64, device="cuda")
        for c in logits[part].split(1 << 17):
            want += torch.softmax(c.double(), 1).sum(0)
        # the additions of a workgroup's chain: its share of the tokens, and the probabilities' 50u
        assert ((sums[s] - want).abs() <= (T / S / 256 / 16 + 150) * ref.U * want).all()
    d = moe.moe_route_grad(logits, idx, expert_counts=counts, seq_tokens=tokens, alpha=0.01,
                           n_seqs=S)
    rows = [0, T // S - 1, T // S, 2 ** 31 // E - 1, 2 ** 31 // E, T - 1]
    l64, c64 = f64(logits[rows]), f64(counts)
    p = ref.probs(l64)
    for i, t in enumerate(rows):
        s = t // (T // S)
        c = c64[s] - float(round(k * (T // S) / E))
        f = 0.01 / S * E / (k * float(T // S) ** 2)
        want = f * p[i] * (c - (c * p[i]).sum())
        tol = f * p[i] * (np.abs(c - (c * p[i]).sum()) + (np.abs(c) * p[i]).sum()) * 80 * ref.U
        assert (np.abs(f64(d[t]) - want) <= tol + 2.0 ** -120).all()


def test_binding_refusals_on_the_gpu():
    _announce("binding refusals")
    x = torch.zeros((4, 32), device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="topk_idx: dtype"):
        moe.moe_balance_loss(x, idx.long(), 0.1)
    with pytest.raises(ValueError, match="n_seqs"):
        moe.moe_balance_loss(x, idx, 0.1, n_seqs=3)
    with pytest.raises(ValueError, match="topk_idx: shape"):
        moe.moe_balance_loss(x, idx[:3], 0.1)
    with pytest.raises(ValueError, match="token_mask: on cpu"):
        moe.moe_balance_loss(x, idx, 0.1, token_mask=torch.ones(4, dtype=torch.bool))
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_balance_loss(x, idx, 0.1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError, match="INVALID"):
        moe.moe_route_grad(x, idx)
    with pytest.raises(ValueError, match="x: not contiguous"):
        moe.moe_quant_rows(torch.zeros((32, 64), device="cuda").t())
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        moe.moe_quant_rows(torch.zeros((4, 24), device="cuda"))
    a, sa, w, sw, off, _ = [dev(v) if v is not None else None for v in
                            make_matmul(8, 1, 4, 32, 64, "none", False, "even")]
    with pytest.raises(ValueError, match="w: shape"):
        moe.moe_expert_matmul_i8(a, sa, w[:, :, :48].contiguous(), sw, off)
    with pytest.raises(ValueError, match="expert_offsets: shape"):
        moe.moe_expert_matmul_i8(a, sa, w, sw, off[:-1])
    with pytest.raises(moe.MoeError, match="INVALID"):
        moe.moe_expert_matmul_i8(a, sa, w, sw)
    with pytest.raises(ValueError, match="act"):
        moe.moe_expert_matmul_i8(a, sa, w, sw, off, act="relu")
    with pytest.raises(TypeError, match="out: dtype"):
        moe.moe_expert_matmul_i8(a, sa, w, sw, off, out_dtype=torch.float16)


def test_binding_refuses_sizes_beyond_int32():
    """Of every tensor that a size is taken from (tensors of one value, expanded: no memory)."""
    _announce("binding sizes beyond int32")
    def wide(dtype, *shape):
        return torch.zeros(1, dtype=dtype, device="cuda").expand(shape)
    over = 2 ** 32 + 16
    x = torch.zeros((4, 16), device="cuda")
    a, sa = torch.zeros((4, 16), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    w, sw = torch.zeros((1, 8, 16), dtype=torch.int8, device="cuda"), torch.zeros((1, 8), device="cuda")
    for name, call in (
            ("logits", lambda: moe.moe_balance_loss(wide(torch.float32, over, 16), None, 0.1)),
            ("topk_idx", lambda: moe.moe_balance_loss(x, wide(torch.int32, 4, over), 0.1)),
            ("topk_idx", lambda: moe.moe_route_grad(x, wide(torch.int32, 4, over))),
            ("n_seqs", lambda: moe.moe_balance_loss(x[:0], torch.zeros((0, 2), dtype=torch.int32,
                                                                       device="cuda"), 0.1, over)),
            ("n_seqs", lambda: moe.moe_route_grad(x, torch.zeros((4, 2), dtype=torch.int32,
                                                                 device="cuda"), n_seqs=over)),
            ("x", lambda: moe.moe_quant_rows(wide(torch.bfloat16, over, 16))),
            ("w", lambda: moe.moe_expert_matmul_i8(a, sa, wide(torch.int8, 1, over, 16), sw)),
            ("w", lambda: moe.moe_expert_matmul_i8(a, sa, wide(torch.int8, over, 8, 16), sw)),
            ("row_token", lambda: moe.moe_expert_matmul_i8(a, sa, w, sw,
                                                           row_token=wide(torch.int32, over)))):
        with pytest.raises(ValueError, match=f"{name}: .*2147483647"):
            call()
