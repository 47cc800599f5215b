"""GPU tests of the activations of the experts' product in bf16 over the whole range of fp32: large, lowest
and infinite sums, forwards and backwards, in every way that a product is made."""
import numpy as np
import pytest
import torch

import block_ref as ref
from combine_moe_route_03_amd import _lib as moe
from test_gpu_block import BF16, F32, _announce, dev, f64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

SIZES = [0.25, 1.0, 3.0, 6.0, 9.0, 9.9375, 10.0, 10.5, 11.0, 12.0, 14.0, 30.0, 50.0, 63.5, 64.0, 64.5, 66.0, 66.5,
         67.0, 86.5, 87.0, 87.5, 88.0, 89.0, 91.0, 92.0, 96.0, 100.0, 104.0, 128.0, 133.0, 134.0, 1e3, 1e4, 6e7,
         1e9, 1e13, 2e19, 1e20, 1e30, 2e38, float(torch.finfo(torch.bfloat16).max)]
VALUES = torch.tensor([0.0, -0.0] + [s for v in SIZES for s in (v, -v)]).bfloat16().double().numpy()
FAR = np.concatenate([VALUES, [np.inf, -np.inf, np.nan]])
FLUSHED = 2.0 ** -125                  # results below 2^-126 may be flushed, in two factors

# rows, experts, channels, terms of the sum: few rows, tiles, sums in parts
WAYS = [(8, 1, 24, 72), (FAR.size, 4, 40, 136), (2000, 2, 264, 136), (4096, 1, 1024, 64), (200, 1, 384, 7168)]


def rows_of_one(values, R, K):
    """Rows of R values each in one place, so that sums with ones are exactly these; others are 0."""
    a = np.zeros((R, K))
    a[np.arange(R), np.arange(R) % K] = values
    return torch.from_numpy(a).bfloat16()


def close(got, want, rel, floor, what, at):
    """got within rel |want| + floor of want as fp32 holds it; infinities and NaN the same."""
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(np.isfinite(want) & (np.abs(want) > np.finfo(np.float32).max),
                        np.sign(want) * np.inf, want)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        ok = same | (np.isfinite(got) & np.isfinite(want) & (np.abs(got - want) <= np.abs(want) * rel + floor))
    assert ok.all(), (what, at[~ok][:4], got[~ok][:4], want[~ok][:4])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("R,E,N,K", WAYS)
def test_activations_over_the_whole_range(R, E, N, K, act, dtype):
    """Sums that are exactly a value, in every channel. An activation that goes by a logistic function of t
    is off by (16 + 8 |t|) u at most, of which none is left where it vanishes. Up channels are 1/4 of the gates."""
    _announce(f"{act} over the range R={R} E={E} N={N} K={K} {dtype}")
    v = np.resize(FAR, R) if R >= FAR.size else None
    for part in [v] if v is not None else [np.resize(FAR[i:i + R], R) for i in range(0, FAR.size, R)]:
        off = np.linspace(0, R, E + 1).astype(np.int32)
        w = torch.ones((E, 2 * N if act == "swiglu" else N, K), dtype=BF16)
        if act == "swiglu":
            w[:, N:] = 0.25
        pre = torch.empty((R, w.shape[1]), dtype=BF16, device="cuda")
        out = moe.moe_expert_matmul(rows_of_one(part, R, K).cuda(), w.cuda(), dev(off), act=act, pre=pre,
                                    out_dtype=dtype)
        with np.errstate(invalid="ignore", over="ignore"):
            want = ref.act(part, "silu") * part * 0.25 if act == "swiglu" else ref.act(part, act)
            t = np.abs(np.sqrt(8 / np.pi) * (part + 0.044715 * part ** 3) if act == "gelu" else part)
            rel = 0.0 if act in ("none", "relu") else (16 + 8 * np.minimum(t, 100)) * ref.U
            rel = np.nan_to_num(rel) + ref.half(dtype == BF16)
        for c in (0, N // 2, N - 1):
            close(f64(out[:, c]), want, rel, FLUSHED, f"out, channel {c}", part)
        # one rounding of nothing: the sum is a bf16 value
        g = f64(pre[:, 0])
        assert ((g == part) | (np.isnan(g) & np.isnan(part))).all()


# rows, experts, terms of the sum (channels of dy), columns of da: tiles of several shapes, sums in parts
SLOPE_WAYS = [(VALUES.size, 1, 16, 24), (VALUES.size, 4, 40, 136), (2000, 2, 264, 136), (4096, 1, 64, 1024),
              (100, 1, 4096, 64)]


def slope_of(v, act):
    """(slope, bound of its fp32 error) of s (1 + x (1 - s)), s the logistic function of t, x = v t': s is good
    to e = (24 + 8 |t|) u of itself, and 1 - s to e s + u."""
    if act == "relu":
        return (v > 0).astype(np.float64), np.zeros_like(v)
    near = np.clip(v, -1e4, 1e4)                              # both slopes are 0 and 1 long before
    gelu = act == "gelu"
    t = np.sqrt(8 / np.pi) * (near + 0.044715 * near ** 3) if gelu else near
    x = near * (np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * near * near) if gelu else 1.0)
    with np.errstate(over="ignore"):
        s, rest = 1.0 / (1.0 + np.exp(-t)), 1.0 / (1.0 + np.exp(t))
    e = (24 + 8 * np.minimum(np.abs(t), 100)) * ref.U
    ax = np.where(t < 100, np.abs(x), 0.0)                    # 1 - s is 0 beyond
    d = s * (1 + x * rest)
    return d, np.abs(d) * e + s * ax * (e * s + 3 * ref.U)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("R,E,N,K", SLOPE_WAYS)
def test_activation_slopes_over_the_whole_range(R, E, N, K, act, dtype):
    """Gradients that are exactly a value, small and large, times the slope at every value. Where the logistic
    function is below exp(-87) a slope is at most (1 + |v t'|) exp(-87) < 2^-117 and may be 0; from -100 on it
    is 0 in fp32, and so is whatever it is multiplied with. SwiGLU's up channels are moderate and large."""
    _announce(f"slope of {act} over the range R={R} E={E} N={N} K={K} {dtype}")
    for d, up in ((1.0, 2.0), (-2.0 ** 100, -3.0), (2.0, 2.0 ** 120)):
        v = np.resize(VALUES, R)
        off = np.linspace(0, R, E + 1).astype(np.int32)
        dy = rows_of_one(np.full(R, d), R, N).cuda()
        w = torch.ones((E, N, K), dtype=BF16, device="cuda")
        pre = torch.from_numpy(v).bfloat16()[:, None].expand(R, K)
        if act == "swiglu":
            pre = torch.cat([pre, torch.full((R, K), up, dtype=BF16)], 1)
        da, = moe.moe_expert_matmul_grad(dy, None, w, dev(off), want="da", act=act, pre=pre.contiguous().cuda(),
                                         da_dtype=dtype)
        slope, err = slope_of(v, act)
        scale = d * up if act == "swiglu" else d
        tol = np.abs(scale) * (err + 4 * ref.U * np.abs(slope) + (0.0 if act == "relu" else 2.0 ** -117))
        tol = tol + np.abs(scale * slope) * ref.half(dtype == BF16) + FLUSHED
        zero = v <= -100.0
        for c in (0, K // 2, K - 1):
            got = f64(da[:, c])
            bad = np.where(zero, got != 0.0, ~(np.abs(got - scale * slope) <= tol))
            assert not bad.any(), (d, c, v[bad][:4], got[bad][:4], (scale * slope)[bad][:4])
            if act == "swiglu":                               # up: dh silu(gate)
                with np.errstate(over="ignore", invalid="ignore"):
                    want = d * ref.act(v, "silu")
                close(f64(da[:, K + c]), want, (20 + 8 * np.minimum(np.abs(v), 100)) * ref.U + ref.half(dtype == BF16),
                      FLUSHED * max(1.0, abs(d)), f"up, column {c}", v)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("R,E,N,K", [(5, 1, 16, 24), (300, 3, 40, 136), (2000, 2, 264, 72), (100, 1, 4096, 64)])
def test_gradients_through_a_pre_off_16_bytes(R, E, N, K, act):
    """pre and dbias that begin between 16-byte borders, with plain products among them: the bits of aligned ones."""
    _announce(f"gradient of {act}, pre off 16 bytes R={R} E={E} N={N} K={K}")
    g = torch.Generator().manual_seed(R + K)
    n = R * (2 * K if act == "swiglu" else K)
    pre = torch.randn(n + 8, generator=g).to(BF16).cuda()
    dy, a = torch.randn((R, N), generator=g).to(BF16).cuda(), torch.randn((R, K), generator=g).to(BF16).cuda()
    w = torch.randn((E, N, K), generator=g).to(BF16).cuda()
    off = None if E == 1 else dev(np.linspace(0, R, E + 1).astype(np.int32))
    want = ("da", "dw", "dbias")
    even = moe.moe_expert_matmul_grad(dy, a, w, off, want=want, act=act, pre=pre[1:n + 1].clone().view(R, -1))
    odd = moe.moe_expert_matmul_grad(dy, a, w, off, want=want, act=act, pre=pre[1:n + 1].view(R, -1),
                                     dbias=torch.empty(E * N + 4, device="cuda")[1:E * N + 1].view(E, N))
    assert all(torch.equal(u, v) for u, v in zip(even, odd))
