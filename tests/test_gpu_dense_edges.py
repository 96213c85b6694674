"""Dense bf16 layers where a bound relative to the largest value says little: tails of the activations, values that
are not finite, sums that cancel, gradients along themselves (GPU)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_ref as R

pytestmark = pytest.mark.gpu

bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import mxfp4_routed_expert_amd as m
    return m


def rnd(seed, *shape, std=1.0, dtype=bf16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


# The activations' values relative to themselves.  The product is exact (one 1 in each row of x), so z is the weight.
#   gelu       Phi(z) = E q, E = exp(-z^2 / 2): three roundings of z^2 / 2 and one of the exponential; q's fit (1.3e-7 = 2.2 of
#              2^-24) and its evaluation, nine fused steps whose terms add up to at most 6 times q: 64 of 2^-24 hold all
#   silu, gelu_tanh   z / (1 + exp(-t)): t's roundings (at most 8, relative) scale the exponential by 8 |t| 2^-24; 16 for
#              the exponential, the sum, the reciprocal and the product
# Ranges: as far out as the value and its factors are normal numbers.
TAILS = {"gelu": (12.5, lambda z: 2 * z * z + 64), "silu": (80.0, lambda z: 8 * z.abs() + 16),
         "gelu_tanh": (9.5, lambda z: 8 * (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs() + 16)}


@pytest.mark.parametrize("T", [2, 12, 80])
@pytest.mark.parametrize("fn", sorted(TAILS))
def test_activations_keep_their_relative_accuracy(M, fn, T):
    end, steps = TAILS[fn]
    v = torch.cat([torch.linspace(-end, end, 504), torch.tensor([-5.5, -5.59375, -6.0, -7.0, -8.0, -10.0, 0.0, 2.0 ** -60])]).to(bf16)
    x = torch.zeros(T, 8, dtype=bf16, device="cuda")
    x[:, 0] = 1
    w, wu = torch.zeros(512, 8, dtype=bf16, device="cuda"), torch.zeros(512, 8, dtype=bf16, device="cuda")
    w[:, 0] = v
    wu[:, 0] = torch.where(torch.arange(512) % 2 == 0, 64.0, -0.25).to(bf16)
    z, u = v.double(), wu[:, 0].double().cpu()
    s = torch.sigmoid(z if fn == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    f = z * torch.special.erfc(z * -math.sqrt(0.5)) / 2 if fn == "gelu" else z * s
    rel = steps(z) * R.EPS32
    for dt in (bf16, f32):
        half = R.BF16 if dt == bf16 else R.EPS32
        tol = rel + half * (1 + rel)
        y = M.moe_dense_linear(x, w, None, fn, out_dtype=dt).double().cpu()
        h, pre = M.moe_dense_gateup(x, w, wu, act_fn=fn, out_dtype=dt, want_pre=True)
        for name, got, ref in (("linear", y, f), ("gated", h.double().cpu(), f * u)):
            err = ((got - ref).abs() - tol * ref.abs()).amax(0)
            bad = err > 0
            assert not bad.any(), (fn, T, dt, name, v[bad].tolist()[:8], got[0][bad].tolist()[:8], ref[bad].tolist()[:8])
        # h again, from the input and from the pre-activations, is the forward result
        for p in (None, pre):
            again = M.moe_dense_gateup_backward(torch.ones_like(h), x, w, wu, act_fn=fn, pre=p, want=(), want_h=True, h_dtype=dt)[5]
            assert torch.equal(again, h), (fn, T, dt, p is None)
