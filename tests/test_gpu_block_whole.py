"""GPU test of a whole MoE block with everything that it learns: the experts, the shared expert and the gate,
forwards and backwards, against autograd in 64 bits, and captured."""
import math

import pytest
import torch

from combine_moe_route_03_amd import _lib as moe
from test_gpu_block import BF16, F32, _announce
from test_gpu_block_run import SIZES, Block

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


class Whole(Block):
    """Block with the gradients of the shared expert and of the gate, and all of the hidden states'."""

    def __init__(self, T, H, inner, E, k, groups, seed=0):
        super().__init__(T, H, inner, E, k, groups, seed)
        need = max(moe.moe_matmul_grad_workspace_bytes(T, 1, n, k2) for n, k2 in ((H, inner), (inner, H), (E, H)))
        self.one_ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.spre, self.dspre, self.dl16 = e(T, inner), e(T, inner), e(T, E)
        self.dxs, self.dxg = e(T, H, dtype=F32), e(T, H, dtype=F32)
        self.ds1, self.ds2, self.dgate = (e(*t.shape, dtype=F32) for t in (self.s1, self.s2, self.gate))

    def forward(self):
        super().forward()
        moe.moe_expert_matmul(self.x, self.s1, act="gelu", pre=self.spre, out=self.sh)

    def backward(self):
        super().backward()
        moe.moe_expert_matmul_grad(self.dout, self.sh, self.s2, act="gelu", pre=self.spre, da=self.dspre,
                                   dw=self.ds2, workspace=self.one_ws)
        moe.moe_expert_matmul_grad(self.dspre, self.x, self.s1, da=self.dxs, dw=self.ds1, workspace=self.one_ws)
        self.dl16.copy_(self.dlogits)
        moe.moe_expert_matmul_grad(self.dl16, self.x, self.gate, da=self.dxg, dw=self.dgate, workspace=self.one_ws)

    def results(self):
        return dict(super().results(), **{n: getattr(self, n) for n in ("spre", "dspre", "dxs", "ds1", "ds2", "dl16",
                                                                        "dxg", "dgate")})

    def reference(self):
        d = lambda t: t.double()  # noqa: E731
        x, w1, b1, w2, s1, s2, gate = (d(t).requires_grad_() for t in (
            self.x, self.w1, self.b1, self.w2, self.s1, self.s2, self.gate))
        s = torch.sigmoid(x @ gate[0].t()).gather(1, self.idx.long())
        wt = 2.5 * s / s.sum(1, keepdim=True)
        v = x @ s1[0].t()
        out = (v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))) @ s2[0].t()
        for j in range(self.k):
            e = self.idx[:, j].long()
            u = (w1[e] * x[:, None, :]).sum(2) + b1[e]
            g, up = u.chunk(2, 1)
            h = g * torch.sigmoid(g) * up
            out = out + wt[:, j:j + 1] * (w2[e] * h[:, None, :]).sum(2)
        names = ("x", "w1", "b1", "w2", "s1", "s2", "gate")
        return out, dict(zip(names, torch.autograd.grad((out * d(self.dout)).sum(), (x, w1, b1, w2, s1, s2, gate))))


@pytest.mark.parametrize("T,H,inner,E,k,groups", [SIZES[0], SIZES[1], (160, 128, 72, 16, 2, 1)])
def test_everything_that_a_block_learns(T, H, inner, E, k, groups):
    """As for the block without these: at most ten tensors on a path are rounded to bf16, each off by 2^-8 of
    itself, and passed on no more than about twice: 10 * 2 * 2^-8 of a result's norm, below 1/12."""
    _announce(f"whole block T={T} H={H} inner={inner} E={E} k={k}")
    b = Whole(T, H, inner, E, k, groups, seed=3)
    b.forward()
    b.backward()
    out, want = b.reference()
    got = {"x": b.dx.double() + b.dxs.double() + b.dxg.double(), "w1": b.dw1, "b1": b.db1, "w2": b.dw2, "s1": b.ds1,
           "s2": b.ds2, "gate": b.dgate}
    assert (b.out.double() - out).norm() < out.norm() / 12
    for name, v in want.items():
        err = ((got[name].double() - v).norm() / v.norm()).item()
        assert err < 1 / 12, (name, err)


def test_everything_that_a_block_learns_captured():
    """Bit for bit the eager results, on changed inputs, replayed with eager work between the replays."""
    _announce("whole block in a graph")
    sizes = SIZES[1]
    b, e = Whole(*sizes), Whole(*sizes)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.forward()
            b.backward()
    torch.cuda.synchronize()
    for rep in range(3):
        x = torch.randn((sizes[0], sizes[1]), generator=torch.Generator().manual_seed(rep)).cuda().to(BF16)
        b.x.copy_(x)
        e.x.copy_(x)
        for t in b.results().values():
            t.fill_(3)
        graph.replay()
        e.forward()
        e.backward()
        torch.cuda.synchronize()
        for name, v in e.results().items():
            assert torch.equal(b.results()[name], v), (rep, name)
