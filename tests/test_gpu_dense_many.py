"""The dense operators where a CTA or a pair of CTAs takes several rows or output tiles, against the
definitions in 64 bits (on smaller shapes each takes at most one): rings that wrap, accumulators and barriers that
are used again, tiles stored while the next one runs, last rounds that are not full."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from tests import test_gpu_fp8_linear as fp8
from tests import test_gpu_gated_linear as gated
from tests import test_gpu_residual_norm as norm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("M,K", [(1000, 7168), (1000, 8192), (700, 8200), (700, 16384), (1001, 1544), (5000, 256)])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("dtype,rtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float32)])
def test_norm_of_many_rows(M, K, gate, dtype, rtype):
    norm.check(*norm.case(M, K, dtype, rtype, gate, seed=M + K))


@pytest.mark.parametrize("M,K,groups", [(1000, 7168, 8), (1000, 8192, 250), (700, 16384, 7), (704, 8200, 352), (2000, 1544, 1000)])
@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
def test_norm_of_many_rows_in_groups(M, K, groups, rtype):
    norm.check(*norm.case(M, K, torch.bfloat16, rtype, "groups", seed=groups, groups=groups))


@pytest.mark.parametrize("M", [1000, 700])
@pytest.mark.parametrize("which", ["dr_out", "dy"])
def test_norm_of_many_rows_with_a_gradient_absent(M, which):
    c, dr_out, dy = norm.case(M, 16384 if M == 700 else 7168, torch.bfloat16, torch.float32, "channel", seed=M)
    norm.check(c, None if which == "dr_out" else dr_out, None if which == "dy" else dy)


# 256 x 256 tiles: 121 and 132; 256 x 128: 231 and 242, on at most 76 pairs
@pytest.mark.parametrize("M,N", [(2600, 2600), (2817, 2579)])
@pytest.mark.parametrize("K", [128, 256, 384, 1152])
@pytest.mark.parametrize("dtype", TYPES)
def test_fp8_of_many_tiles(M, K, N, dtype):
    fp8.test_gemm_exact_integers(M, K, N, dtype)


@pytest.mark.parametrize("T,H,I", [(2600, 64, 2600), (2600, 136, 2600), (2817, 200, 1704), (5000, 72, 2600)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_forward_of_many_tiles(T, H, I, dtype):
    gated.test_forward_exact_integers(T, H, I, dtype)


@pytest.mark.parametrize("T,H,I", [(2600, 2600, 72), (2600, 2600, 264), (2600, 2600, 1000), (2817, 1704, 520), (300, 2600, 2600), (5000, 2600, 136)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_gradients_of_many_tiles(T, H, I, dtype):
    gated.test_backward_exact_integers(T, H, I, dtype)
