"""Calls of the fused MXFP4 operators that their documentation allows and that lie at an edge:
layers of experts that no token goes to, and as many tokens as there may be."""
import pytest
import torch

import dequant_gemv_nf4_amd as nf4
from test_gpu_fused import BF, DEV, F32, matrix, rand, run_moe

pytestmark = pytest.mark.gpu


# 16 columns a workgroup of the second product, 64, 64 by H; shared out over workgroups and not
@pytest.mark.parametrize("t,k,e,h,i", [(1, 1, 1, 64, 96), (4, 2, 8, 4096, 14336), (1, 2, 8, 4128, 64),
                                       (3, 2, 8, 8192, 544), (16, 8, 512, 256, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_moe_without_any_expert(t, k, e, h, i, dtype):
    """Every token gets its residual, or zero."""
    none = torch.full((t, k), -1, device=DEV)
    none[t - 1, k - 1] = e
    for residual in (False, True):
        m1, m2, x, experts, weights, out = run_moe(t, k, e, h, i, experts=none, residual=residual, dtype=dtype, seed=h)
        assert torch.equal(out, rand((t, h), h + 6, dtype) if residual else torch.zeros_like(out))
