"""Block-128 FP8 operators at their edges (GPU): what autograd sees, workspaces, tiles of every size, windows of scales."""
from __future__ import annotations

import warnings

import pytest
import torch

from test_gpu_fp8 import BF, DEV, F32, M, U8, codes_of, hidden, scales_of  # noqa: F401  (M: the fixture)

pytestmark = pytest.mark.gpu


def test_operands_that_require_grad_are_warned_of(M):
    T, n, k = 4, 32, 64
    w, x, r = (hidden(n, k, 1) * 0.1).to(DEV), hidden(T, k, 2).to(DEV), hidden(T, n, 3).to(DEV)
    layer = M.FP8Linear(w, T)
    grad = lambda t: t.clone().requires_grad_()
    for call, who in ((lambda: layer.forward(grad(x)), "moe_fp8_quantize"), (lambda: layer.forward(x, grad(r)), "moe_fp8_linear"),
                      (lambda: layer.set_weight(torch.nn.Parameter(w)), "moe_fp8_quantize_weight"), (lambda: M.FP8Linear(torch.nn.Parameter(w), T), "moe_fp8_quantize_weight"),
                      (lambda: M.moe_fp8_quantize(grad(x), cols=True), "moe_fp8_quantize")):
        with pytest.warns(UserWarning, match=f"{who}: an operand requires grad.*FP8Linear.backward"):
            call()
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                call()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        layer.forward(x, r)
        layer.backward(r)
