"""The 4-bit linear's workspace: what the query returns for a number of rows is enough for every smaller one."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, ops
from nvfp4_block_scaled_quant_gb300 import build as B

NO_DEVICE = (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)
SIZES = [(12288, 4096, 32), (1137, 2000, 32), (7168, 7168, 128), (512, 512, 128), (64, 256, 32), (128, 8192, 32), (256, 7168, 64), (1, 8, 64)]


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


@pytest.mark.parametrize("N,K,group", SIZES)
def test_query_grows_with_the_rows(L, N, K, group):
    last = 0
    for M in [*range(0, 1200), *range(1200, 20000, 61), 10 ** 5, 10 ** 6]:
        n = L.nvfp4_w4_linear_workspace_bytes(M, N, K, group)
        assert n >= last, M
        assert n in (0, last) or last == 0
        last = n


@pytest.mark.parametrize("N,K,group", SIZES)
def test_one_workspace_for_every_smaller_number_of_rows(L, N, K, group):
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real: the calls have to end at the device")
    for most in (16, 300, 2048, 20000):
        n = L.nvfp4_w4_linear_workspace_bytes(most, N, K, group)
        for M in {1, 17, most, *range(129, min(most, 2049), 128)}:
            st = L.nvfp4_w4_linear(1 << 20, _lib.DT_BF16, M, K, K, N, 1 << 34, group, 0, 1 << 36, 1 << 40 if n else None, n, None)
            assert st in NO_DEVICE, (most, M, L.nvfp4_last_error_string())


def test_workspace_of_a_weight(L):
    w = ops.W4Weight(torch.zeros(0, dtype=torch.uint8), 1, 1137, 2000, 32, torch.bfloat16, False, False)
    for M in (1, 1500, 4096):
        assert ops.w4_linear_workspace(M, w).numel() == L.nvfp4_w4_linear_workspace_bytes(M, 1137, 2000, 32)
