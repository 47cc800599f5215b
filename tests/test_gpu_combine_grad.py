"""GPU tests of the combine's gradient where a workgroup takes several slots of a token, all of them, or an
uneven share, and where rows go past the caches, against a plain form in 64 bits."""
import pytest
import torch

import block_ref as ref
from combine_moe_route_03_amd import _lib as moe
from test_gpu_block import BF16, F32, _announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def made(T, k, H, y_dtype, o_dtype):
    """Inputs with one slot in fifty out of range, and their rows in no order."""
    g = torch.Generator(device="cuda").manual_seed(T * H + k)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    row = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    out = torch.rand(T * k, generator=g, device="cuda") < 0.02
    row = torch.where(out, torch.where(row % 2 == 0, -1 - row, T * k + row), row).to(torch.int32)
    return normal(T, H).to(o_dtype), normal(T * k, H).to(y_dtype), row, normal(T, k)


def check(T, k, H, y_dtype, o_dtype):
    d, y, row, w = made(T, k, H, y_dtype, o_dtype)
    dy = torch.full((T * k, H), 77.0, dtype=y_dtype, device="cuda")
    got, dw = moe.moe_combine_grad(d, y, row, w, dy=dy)
    assert got is dy
    left = torch.ones(T * k, dtype=torch.bool, device="cuda")
    for j in range(k):
        r = row.view(T, k)[:, j].long()
        ok = (r >= 0) & (r < T * k)
        r = r[ok]
        left[r] = False
        want = w[ok, j:j + 1].double() * d[ok].double()
        bad = ~((dy[r].double() - want).abs() <= want.abs() * (ref.U + ref.half(y_dtype == BF16)) + ref.TINY)
        assert not bad.any(), ("dy", j, bad.nonzero()[0].tolist())
        prod = y[r].double() * d[ok].double()
        # a lane's chain of products, then 6 joins in a wavefront and 8 over wavefronts
        tol = prod.abs().sum(1) * (H / 64 + 32) * ref.U + ref.TINY
        bad = ~((dw[ok, j].double() - prod.sum(1)).abs() <= tol)
        assert not bad.any(), ("dtopk_w", j, bad.nonzero()[0].tolist())
        assert (dw[~ok, j] == 0).all()
    assert (dy[left] == 77.0).all()
    return d, y, row, w, dy, dw


# What a workgroup takes of a token's slots: the halves, rounded up, until there are 1024 workgroups, with one
# wavefront a token up to 1024 elements, four up to 2048, and eight.
SHARES = [
    # T, k, H: slots of a share
    (1100, 8, 520),    # 2
    (1500, 5, 520),    # 2, 2, 1
    (5000, 3, 520),    # 3
    (300, 8, 1032),    # 2
    (600, 5, 1032),    # 3, 2
    (600, 3, 2048),    # 2, 1
    (1100, 3, 2048),   # 3
    (300, 8, 2056),    # 2
    (600, 5, 2056),    # 3, 2
    (1100, 8, 2056),   # 8
    (1030, 64, 264),   # 16
]


@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,H", SHARES)
def test_combine_grad_shares(T, k, H, o_dtype, y_dtype):
    _announce(f"combine_grad shares T={T} k={k} H={H} {o_dtype} {y_dtype}")
    check(T, k, H, y_dtype, o_dtype)


@pytest.mark.parametrize("T,k,H,y_dtype,o_dtype", [(8400, 8, 1024, BF16, BF16), (4300, 8, 1000, F32, BF16),
                                                   (5600, 8, 1536, BF16, F32), (2900, 8, 1480, F32, F32),
                                                   (1100, 8, 8200, BF16, F32), (2100, 8, 2056, F32, BF16)])
def test_combine_grad_past_the_caches(T, k, H, y_dtype, o_dtype):
    """y and dy of more than 256 MB."""
    _announce(f"combine_grad of more than the caches hold T={T} k={k} H={H} {y_dtype} {o_dtype}")
    check(T, k, H, y_dtype, o_dtype)


@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,H", [(5, 3, 264), (1100, 8, 520), (600, 5, 1032), (300, 8, 2056)])
def test_combine_grad_of_one_kind(T, k, H, y_dtype):
    """Each gradient alone has the bits that both have; nothing else is needed, and nothing else made."""
    _announce(f"combine_grad, one of two T={T} k={k} H={H} {y_dtype}")
    d, y, row, w, dy, dw = check(T, k, H, y_dtype, BF16)
    none, only = moe.moe_combine_grad(d, y, row, w, want="dtopk_w")
    assert none is None and torch.equal(only, dw)
    kept = torch.full_like(dw, 5.0)
    assert moe.moe_combine_grad(d, y, row, w, want=("dtopk_w",), dtopk_w=kept)[1] is kept and torch.equal(kept, dw)
    again = torch.full_like(dy, 77.0)
    only, none = moe.moe_combine_grad(d, y, row, w, want="dy", dy=again)
    assert none is None and only is again and torch.equal(again, dy)
    both = moe.moe_combine_grad(d, y, row, w, want=("dtopk_w", "dy"), dy=again.fill_(77.0))
    assert torch.equal(both[0], dy) and torch.equal(both[1], dw)
    for bad, error in ((dict(want=()), ValueError), (dict(want="dx"), ValueError), (dict(want=("dy", "dy")), ValueError),
                       (dict(want="dtopk_w", dy=again), ValueError), (dict(want="dy", dtopk_w=kept), ValueError)):
        with pytest.raises(error, match="want|dy|dtopk_w"):
            moe.moe_combine_grad(d, y, row, w, **bad)
    with pytest.raises(ValueError, match="y"):
        moe.moe_combine_grad(d, None, row, w, want="dtopk_w")


def test_combine_grad_arguments_by_place():
    """dy, dtopk_w and the stream by their places."""
    _announce("combine_grad, arguments by place")
    d, y, row, w = made(40, 4, 264, BF16, BF16)
    row = torch.where(row < 0, -1, row)
    want = moe.moe_combine_grad(d, y, row, w, dy=torch.zeros_like(y))
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = moe.moe_combine_grad(d, y, row, w, dy, dw, stream)
    stream.synchronize()
    assert got[0] is dy and got[1] is dw and torch.equal(dy, want[0]) and torch.equal(dw, want[1])
