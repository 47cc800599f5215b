"""GPU tests of persistent workgroups that take several tiles, in every tile shape: what runs on from
one tile into the next (stages, scales, the ring of tiles, stores) against the plain form in 64 bits."""
import pytest
import torch

from layer_tiles import MANY, SEVERAL
from test_gpu_layer import _announce, check_matmul, make_matmul

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tile,T,E,N,K,kind,act", SEVERAL)
def test_several_tiles_of_a_workgroup(tile, T, E, N, K, kind, act, gather, dtype):
    _announce(f"several tiles {tile} T={T} E={E} N={N} K={K} {kind} {act} gather={gather} {dtype}")
    check_matmul(make_matmul(T, 1, E, N, K, act, gather, kind, seed=T + N + K), act, dtype)


@pytest.mark.parametrize("tile,T,E,N,K,kind,act,gather", MANY)
def test_more_tiles_of_a_workgroup_than_the_ring_holds(tile, T, E, N, K, kind, act, gather):
    _announce(f"many tiles {tile} T={T} E={E} N={N} K={K} {kind} {act} gather={gather}")
    check_matmul(make_matmul(T, 1, E, N, K, act, gather, kind, seed=T + N + K), act, torch.bfloat16)
