"""Residual norm and its gradients on rows far from an rms of 1, against the formulas in 64 bits.

The formulas use f and r' only normalised, so relative errors do not depend on the rows' size: the
bounds are those of the other tests.  The statistics need the sum of the squares of a thread's 16
columns within fp32's range, which the sizes here keep (an rms from 1e-18 to 4e17)."""

import pytest
import torch

from tests import test_gpu_residual_norm as base

pytestmark = pytest.mark.gpu


def sized(c, dr_out, dy, f_size, r_size):
    return {**c, "f": (c["f"].double() * f_size).to(c["f"].dtype), "r": (c["r"].double() * r_size).to(c["r"].dtype)}, dr_out, dy


@pytest.mark.parametrize("M,K", [(5, 1544), (700, 512), (3, 8200)])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("which", ["both", "dy", "dr_out"])
@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("f_size,r_size", [(1.0, 1e14), (1e14, 1e14), (1e15, 1.0), (1.0, 1e17), (1e17, 1e17)])
def test_large_rows(M, K, gate, which, rtype, f_size, r_size):
    c, dr_out, dy = sized(*base.case(M, K, torch.bfloat16, rtype, gate, seed=M + K), f_size, r_size)
    base.check(c, dr_out if which != "dy" else None, dy if which != "dr_out" else None)


@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("which", ["both", "dy"])
@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e-13, 0.0), (1e-15, 0.0), (1e-18, 0.0), (1e-15, 1e-5), (1e-15, 1e-30)])
def test_tiny_rows(monkeypatch, gate, which, rtype, size, eps):
    monkeypatch.setattr(base, "EPS", eps)
    c, dr_out, dy = sized(*base.case(40, 1544, torch.bfloat16, rtype, gate, seed=3), size, size)
    base.check(c, dr_out if which == "both" else None, dy)


@pytest.mark.parametrize("r_size", [1e14, 1e17])
def test_large_fp32_residual_of_fp16_blocks(r_size):
    c, dr_out, dy = sized(*base.case(40, 1544, torch.float16, torch.float32, "channel", seed=4), 1.0, r_size)
    base.check(c, None, dy)


@pytest.mark.parametrize("after,before", [(True, False), (False, True), (False, False)])
def test_large_rows_with_a_norm_absent(after, before):
    c, dr_out, dy = sized(*base.case(40, 1544, torch.bfloat16, torch.float32, "channel", seed=5, after=after, before=before), 1e15, 1e15)
    base.check(c, dr_out, dy)
