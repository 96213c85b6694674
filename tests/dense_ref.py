"""float64 definitions of the dense layers and error bounds for their float32 / bf16 kernels.

Bounds, per element, from the rounding steps of the kernels (bf16 products are exact in float32):
  a sum of K float32 products in any order is within (K + 8) 2^-24 of the sum of magnitudes S;
  an activation or its derivative moves by at most 1.2 times what its argument moves (the second
  derivatives of silu, gelu and its tanh form are below 1.2 in magnitude) and is itself computed
  within 32 float32 roundings of (1 + |z|);
  a value rounded to bf16 is within 2^-8 of itself (2^-133 below the normal range);
  relu's derivative is either value where z lies within its own error of 0.
The intermediate dz (dg, du) is rounded to bf16 before the gradient products, when there are more than 64
tokens, and nowhere else; up to there two bf16 terms stand for it, within 2^-16.
"""
from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 2.0 ** -126


def act(name, z):
    """f(z), f'(z) in float64."""
    if name == "none":
        return z.clone(), torch.ones_like(z)
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z), (z > 0).double()
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def product(x, w, bias=None):
    """(x w^T + bias, bound of its float32 evaluation)"""
    x, w = x.double(), w.double()
    z = x @ w.t()
    s = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        s = s + bias.double().abs()
    return z, (x.shape[1] + 8) * EPS32 * s


def act_bound(name, z, dz):
    """Bounds of f(z) and f'(z) evaluated in float32 at a z that is off by up to dz."""
    if name == "none":
        return dz, torch.zeros_like(z)
    own = 32 * EPS32 * (1 + z.abs())
    f1 = 1.2 * dz + own
    f2 = 1.2 * dz + own
    if name == "relu":
        f1, f2 = dz, (z.abs() <= dz).double()
    return f1, f2


def rounded(v, tol, dtype):
    """The bound after rounding to dtype."""
    return tol + (BF16 if dtype == torch.bfloat16 else EPS32) * (v.abs() + tol) + TINY


def linear(x, w, bias, fn, residual, dtype):
    z, ez = product(x, w, bias)
    y = act(fn, z)[0]
    ey = act_bound(fn, z, ez)[0] + EPS32 * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + EPS32 * y.abs()
    return y, rounded(y, ey, dtype)


def gateup(x, wg, wu, bg, bu, fn, dtype):
    g, eg = product(x, wg, bg)
    u, eu = product(x, wu, bu)
    return gated(g, eg, u, eu, fn, dtype)


def gated(g, eg, u, eu, fn, dtype):
    a = act(fn, g)[0]
    ea = act_bound(fn, g, eg)[0]
    h = a * u
    return h, rounded(h, ea * (u.abs() + eu) + a.abs() * eu + 2 * EPS32 * h.abs(), dtype)


def grads(dz, edz, x, w, dx_dtype=torch.bfloat16, exact_dz=False):
    """From dz (exact) and the bound of its unrounded float32 value: dx, dw, dbias with their bounds.  exact_dz: dz is
    bf16 as it stands.  A float32 x enters dw as two bf16 terms, within 2^-15 (two truncations)."""
    xs = 2.0 ** -15 if x.dtype == torch.float32 else 0.0
    x, w = x.double(), w.double()
    n, k, T = w.shape[0], w.shape[1], x.shape[0]
    if exact_dz:
        er = edz
    elif T <= 64:
        er = edz + 2.0 ** -16 * (dz.abs() + edz) + TINY
    else:
        er = rounded(dz, edz, torch.bfloat16)
    m = dz.abs() + er
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    ex = er @ w.abs() + (n + 8) * EPS32 * (m @ w.abs())
    # (dz's low term, within 2^-8 of it, meets x's first term alone: 2^-8 times x's truncation of 2^-7 more)
    ew = er.t() @ x.abs() + ((3 * T + 8) * EPS32 + xs * 2) * (m.t() @ x.abs())
    eb = edz.sum(0) + (T + 8) * EPS32 * (dz.abs() + edz).sum(0) + TINY
    return (dx, rounded(dx, ex, dx_dtype)), (dw, rounded(dw, ew, torch.bfloat16)), (db, eb)


def linear_backward(dy, x, w, bias, fn, dx_dtype=torch.bfloat16):
    dy = dy.double()
    if fn == "none":
        return grads(dy, torch.zeros_like(dy), x, w, dx_dtype, exact_dz=True)
    z, ez = product(x, w, bias)
    d = act(fn, z)[1]
    ed = act_bound(fn, z, ez)[1]
    dz = dy * d
    return grads(dz, dy.abs() * ed + 2 * EPS32 * dz.abs(), x, w, dx_dtype)


def gateup_backward(dh, x, wg, wu, bg, bu, fn, pre=None, h_dtype=torch.bfloat16):
    """((dx, dw_gate, dw_up, db_gate, db_up, h), each with its bound)"""
    dh = dh.double()
    if pre is None:
        g, eg = product(x, wg, bg)
        u, eu = product(x, wu, bu)
    else:
        g, u = pre[0].double(), pre[1].double()
        eg = eu = torch.zeros_like(g)
    a, d = act(fn, g)
    ea, ed = act_bound(fn, g, eg)
    dg, du = dh * u * d, dh * a
    edg = dh.abs() * (eu * (d.abs() + ed) + u.abs() * ed) + 4 * EPS32 * dg.abs()
    edu = dh.abs() * ea + 2 * EPS32 * du.abs()
    (xg, exg), (wgd, ewg), (bgd, ebg) = grads(dg, edg, x, wg)
    (xu, exu), (wud, ewu), (bud, ebu) = grads(du, edu, x, wu)
    return (xg + xu, exg + exu + BF16 * (xg + xu).abs()), (wgd, ewg), (wud, ewu), (bgd, ebg), (bud, ebu), \
        gated(g, eg, u, eu, fn, h_dtype)


def check(got, ref, what):
    v, tol = ref
    assert tuple(got.shape) == tuple(v.shape), (what, got.shape, v.shape)
    err = (got.double().to(v.device) - v).abs()
    bad = ~(err <= tol)
    worst = (err / tol).max().item() if err.numel() else 0.0
    print(f"  {what}: worst error / bound {worst:.3f}", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {worst:.3f}"


def mxfp8(x):
    """(codes, scales) of OCP MXFP8 with exact arithmetic: x (bf16 or float32, on the CPU) in float64."""
    v = x.double().reshape(x.shape[0], -1, 32)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2)
    safe = torch.where((amax > 0) & ~bad, amax, torch.ones_like(amax))
    X = (torch.frexp(safe)[1] - 1 - 8).clamp(-127, 127)
    X = torch.where(amax > 0, X, torch.full_like(X, -127))
    q = (torch.where(bad[..., None], torch.zeros_like(v), v) * torch.exp2(-X.double())[..., None]).clamp(-448, 448)
    # nearest of the 127 magnitudes; a tie goes to the even code
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.searchsorted(mid, q.abs().contiguous(), right=False)       # mid[lo-1] < |q| <= mid[lo]
    tie = (lo < 126) & (q.abs() == mid[lo.clamp(max=125)])
    code = torch.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = code + 128 * torch.signbit(q).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code).to(torch.uint8).reshape(x.shape)
    return code, torch.where(bad, torch.full_like(X, 255), X + 127).to(torch.uint8)


def mxfp8_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().reshape(codes.shape[0], -1, 32)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (v * s[..., None]).reshape(codes.shape)
