"""Workspace sizes of the products of include/moe_block.h on the CPU: nothing for sizes that a product refuses."""
import pytest

from combine_moe_route_03_amd import _lib as moe
from test_abi import A16, A16b, S0


@pytest.mark.parametrize("R,channels,K", [(64, 384, 7168), (64, 384, 7164), (64, 384, 7161), (4096, 384, 4), (64, 1, 8),
                                          (4096, 1024, 2 ** 21), (4096, 2047, 2 ** 20), (4096, 2048, 2 ** 20),
                                          (64, 2 ** 22, 512), (64, 2 ** 22, 504)])
def test_refused_products_need_no_workspace(R, channels, K):
    """A product of these sizes, with no workspace: refused for its sizes, or for the workspace if it needs one."""
    need = moe.moe_expert_matmul_workspace_bytes(R, 1, channels, K)
    if K % 8 == 0 and 2 * channels * K < 2 ** 32 and need == 0:
        return                                                # would be launched
    status = moe.load().moe_expert_matmul(A16, R, None, A16b, None, None, R, 1, channels, K, 0, None, None, A16,
                                          moe.MOE_BF16, None, 0, S0)
    assert status == (moe.MOE_ERR_WORKSPACE if need else moe.MOE_ERR_UNSUPPORTED)
    assert (need == 0) == (K % 8 != 0 or 2 * channels * K >= 2 ** 32)
