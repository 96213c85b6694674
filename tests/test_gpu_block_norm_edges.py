"""Norms around a block at their edges (GPU): constants that change, magnitudes, masked places, rows walked one behind the other."""
from __future__ import annotations

import pytest
import torch

import fp8_ref as R
from test_gpu_block_norm import BF, DEV, F32, M, REL, check_backward, d64, half, make, on, rnd  # noqa: F401  (M: the fixture)

pytestmark = pytest.mark.gpu


def test_constants_that_change_between_calls(M):
    """residual_scale held in one tensor: forward and backward take its value at the call."""
    T, d = 4, 64
    z, res, dy = (rnd(i, T, d).to(DEV) for i in range(3))
    for s in (torch.tensor(1.0), torch.tensor(1.0, device=DEV)):
        for v in (1.0, 0.25):
            s.fill_(v)
            y = M.moe_block_norm(z, residual=res, residual_scale=s, y_dtype=F32)[0]
            assert torch.equal(y, M.moe_block_norm(z, residual=res, residual_scale=v, y_dtype=F32)[0])
            dr = M.moe_block_norm_backward(z, dy=dy, residual_scale=s, y_dtype=F32, want=("dresidual",))[1]
            assert torch.equal(dr, v * dy)
