"""Norms around a block at their edges (GPU): constants that change, magnitudes, masked places, rows walked one behind the other."""
from __future__ import annotations

import numpy as np
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


# ------------------------------------------------------------------ gradients of given rows

NAMES = ("dz", "dresidual", "dw_after", "dgate", "dw_before")


def gradients(M, z, w_after=None, gate=None, y=None, w_before=None, du=None, dy=None, rs=1.0, eps=1e-6, p=0.0, rng=None):
    yt = next(t.dtype for t in (dy, y) if t is not None)
    got = M.moe_block_norm_backward(on(z), w_after=on(w_after), gate=on(gate), y=on(y), w_before=on(w_before), du=on(du), dy=on(dy),
                                    residual_scale=rs, dropout=p, rng=on(rng), eps=eps, y_dtype=yt)
    return dict(zip(NAMES, (d64(t) for t in got)))


def expected(z, w_after, gate, y, w_before, du, dy, rs, eps, m, zt, yt):
    """(reference, tolerance) of dz and dresidual in 64 bits: each of a value's terms within 4 REL (two means, two roots and
    products), a float32 product that leaves its normal range off by 2^-149 more, and the result's rounding."""
    one = torch.ones(1, 1, dtype=torch.float64)
    t, tm = torch.zeros_like(z), torch.zeros_like(z)
    if dy is not None:
        t, tm = dy.clone(), dy.abs()
    if w_before is not None:
        ry, v = R.rms(y, eps), du * w_before
        t = t + ry * (v - y * ry * ry * (v * y).mean(1, keepdim=True))
        tm = tm + ry * (v.abs() + y.abs() * ry * ry * (v * y).abs().mean(1, keepdim=True))
    a, am = (one if gate is None else gate) * m * t, (one if gate is None else gate.abs()) * m * tm
    if w_after is not None:
        rz, v, vm = R.rms(z, eps), a * w_after, am * w_after.abs()
        dz, dzm = rz * (v - z * rz * rz * (v * z).mean(1, keepdim=True)), rz * (vm + z.abs() * rz * rz * (vm * z.abs()).mean(1, keepdim=True))
    else:
        dz, dzm = a, am
    tol = lambda ref, mag, dt: (4 * REL * mag + half(dt) * ref.abs()) * (1 + 2.0 ** -8) + 2.0 ** -140
    return dict(dz=(dz, tol(dz, dzm, zt)), dresidual=(rs * t, tol(rs * t, rs * tm, yt)))


def close(got, want):
    for name, (ref, tol) in want.items():
        err = (got[name] - ref).abs()
        assert (err <= tol).all(), f"{name}: {(err / tol).max():.3g} of the tolerance"


@pytest.mark.parametrize("zt,yt", [(F32, F32), (BF, BF)])
@pytest.mark.parametrize("d", [64, 520, 1040, 8208])
def test_gradients_of_large_and_small_rows(M, d, zt, yt):
    """Rows of 2^-60 to 2^56: the sum of squares stays in float32, r^3 does not.  The part along the row is as large as the one that
    it is taken from: a gradient along the row itself cancels."""
    T = 10
    scale = torch.tensor([2.0 ** e for e in (0, 42, 46, 48, 50, 52, 56, -20, -45, -60)])[:, None]
    z, y = (rnd(1, T, d) * scale).to(zt), (rnd(2, T, d) * scale.flip(0)).to(yt)
    wa, wb, g = rnd(3, d).abs() + 0.3, rnd(4, d).abs() + 0.3, rnd(5, T, 1)
    dy, du = rnd(6, T, d, dt=yt), rnd(7, T, d, dt=BF)
    eps = 1e-6
    args = dict(w_after=wa, gate=g, y=y, w_before=wb, du=du, dy=dy)
    want = expected(d64(z), d64(wa), d64(g), d64(y), d64(wb), d64(du), d64(dy), 0.5, eps, 1.0, zt, yt)
    close(gradients(M, z, rs=0.5, eps=eps, **args), want)
    along = (z.float() / scale / wa).to(yt)                    # w_a dy is the row itself
    want = expected(d64(z), d64(wa), None, None, None, None, d64(along), 1.0, eps, 1.0, zt, yt)
    close(gradients(M, z, w_after=wa, dy=along, eps=eps), want)


@pytest.mark.parametrize("eps", [1e-12, 1e-26, 1e-30, 1e-37])
def test_gradients_of_zero_rows_with_small_eps(M, eps):
    """r is 1 / sqrt(eps) there and its cube leaves float32; the mean that it multiplies is 0."""
    T, d = 3, 264
    z, y = torch.zeros(T, d), torch.zeros(T, d)
    z[1], y[2] = rnd(1, d), rnd(2, d)
    wa, wb, dy, du = rnd(3, d), rnd(4, d), rnd(5, T, d), rnd(6, T, d, dt=BF)
    dy, du = dy * 2.0 ** -20, du * 2.0 ** -20
    want = expected(d64(z), d64(wa), None, d64(y), d64(wb), d64(du), d64(dy), 1.0, eps, 1.0, F32, F32)
    assert all(torch.isfinite(ref).all() for ref, _ in want.values())
    close(gradients(M, z, w_after=wa, y=y, w_before=wb, du=du, dy=dy, eps=eps), want)


# ------------------------------------------------------------------ values that take no part

@pytest.mark.parametrize("zt", [F32, BF])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_without_a_norm_after_dz_does_not_depend_on_z(M, zt, gate):
    """dz = gate m t: infinite and NaN z change nothing, nor does a z that is not given."""
    T, d, p = 6, 520, 0.25
    s = make(T, d, zt, F32, False, True, gate, p, seed=3)
    z = s["z"].clone()
    z[1, 5], z[2, 7], z[3, 300], z[4] = float("inf"), float("nan"), float("-inf"), 3.0e38
    y, du, dy = rnd(11, T, d), rnd(12, T, d, dt=BF), rnd(13, T, d)
    kw = dict(gate=on(s["gate"]), y=on(y), w_before=on(s["w_before"]), du=on(du), dy=on(dy), dropout=p, rng=on(s["rng"]), want=("dz", "dresidual"))
    ref = M.moe_block_norm_backward(on(s["z"]), **kw)
    for got in (M.moe_block_norm_backward(on(z), **kw), M.moe_block_norm_backward(None, z_dtype=zt, **kw)):
        assert torch.isfinite(ref[0]).all() and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("after,bad", [(False, float("nan")), (False, float("inf")), (True, float("inf"))])
@pytest.mark.parametrize("d", [64, 520, 1040, 8208])
def test_dropped_elements_take_no_part_in_the_gates_and_weights_gradients(M, d, after, bad):
    """m n is 0 there whatever n is (an infinite z makes n NaN: inf * 0): dgate and dw_after are those of a 0 in its place."""
    T, p = 5, 0.5
    s = make(T, d, F32, F32, after, False, "token", p, seed=9)
    z, zero = s["z"].clone(), s["z"].clone()
    hit = []
    for t in (1, 3):
        c = int((s["m"][t] == 0).nonzero()[t])
        z[t, c], zero[t, c] = bad, 0.0
        hit.append((t, c))
    dy, ch = rnd(14, T, d), rnd(15, 1, d)
    for gate in (s["gate"], ch):
        kw = dict(w_after=on(s["w_after"]), gate=on(gate), dy=on(dy), dropout=p, rng=on(s["rng"]), y_dtype=F32, want=("dw_after", "dgate") if after else ("dgate",))
        got, plain = M.moe_block_norm_backward(on(z), **kw), M.moe_block_norm_backward(on(zero), **kw)
        for i in (2, 3):
            if got[i] is None:
                continue
            assert torch.isfinite(got[i]).all()
            if not after:                                     # (with a norm an infinite z makes r and its row's other n 0)
                assert torch.equal(got[i], plain[i])
        if after:
            # rows with an infinity: r = 0, so n is 0 but where z is infinite, and m n is 0 there too
            keep = torch.ones(T, 1, dtype=torch.float64)
            keep[[t for t, _ in hit]] = 0.0
            zr, wa, a = d64(zero), d64(s["w_after"]), s["m"] * d64(dy)
            n0 = keep * zr * R.rms(zr, 1e-6)
            col = 4 * REL + (T + 16) * 2.0 ** -24
            g = d64(gate)
            want_w, mag_w = (a * g * n0).sum(0), (a * g * n0).abs().sum(0)
            assert ((d64(got[2]) - want_w).abs() <= col * mag_w + 1e-30).all()
            n1, dim = a * n0 * wa, 1 if gate is s["gate"] else 0
            assert ((d64(got[3]) - n1.sum(dim, keepdim=True)).abs() <= (col + d * 2.0 ** -24) * n1.abs().sum(dim, keepdim=True) + 1e-30).all()


# ------------------------------------------------------------------ rows walked one behind the other

# More rows than a forward launch has workgroups (512) or, up to 1024 values a row, waves (2048): the next row is in flight while one is
# worked on, and the two buffers of its sums take turns.
@pytest.mark.parametrize("T,d", [(2049, 64), (4100, 8), (2500, 1000), (513, 1032), (1100, 7168), (1025, 8208), (520, 16384)])
@pytest.mark.parametrize("zt,yt,after,before,gate,p", [(BF, BF, True, True, "channel", 0.25), (F32, F32, True, True, "token", 0.0),
                                                      (BF, F32, False, True, "none", 0.1), (F32, BF, True, False, "token", 0.0)])
def test_forward_many_rows(M, T, d, zt, yt, after, before, gate, p):
    s = make(T, d, zt, yt, after, before, gate, p, seed=60)
    rs, eps = 0.75, 1e-5
    io = on(s["residual"]).clone()                             # the residual is the result
    y, u, c, sc = M.moe_block_norm(on(s["z"]), w_after=on(s["w_after"]), gate=on(s["gate"]), residual=io, w_before=on(s["w_before"]),
                                   residual_scale=rs, dropout=p, rng=on(s["rng"]), eps=eps, want_codes=before, out=(io, None, None, None))
    assert y is io
    branch = R.block_norm(d64(s["z"]), d64(s["w_after"]), d64(s["gate"]), None, 1.0, s["m"], eps)
    ref = rs * d64(s["residual"]) + branch
    tol = REL * branch.abs() + 2.0 ** -23 * (ref.abs() + (rs * d64(s["residual"])).abs())
    tol = tol * (1 + half(yt)) + half(yt) * ref.abs() + 1e-30
    err = (d64(y) - ref).abs()
    assert (err <= tol).all(), f"row {int((err > tol).any(1).nonzero()[0])}"
    apart = M.moe_block_norm(on(s["z"]), w_after=on(s["w_after"]), gate=on(s["gate"]), residual=on(s["residual"]), w_before=on(s["w_before"]),
                             residual_scale=rs, dropout=p, rng=on(s["rng"]), eps=eps)
    assert torch.equal(apart[0], y)
    if not before:
        return
    assert torch.equal(apart[1], u)
    yk = d64(y)
    uref = yk * R.rms(yk, eps) * d64(s["w_before"])
    assert ((d64(u) - uref).abs() <= (REL + 2.0 ** -8) * uref.abs() + 1e-30).all()
    qc, qs = M.moe_fp8_quantize(u)[:2]
    assert torch.equal(c, qc) and torch.equal(sc, qs)


@pytest.mark.parametrize("T,d", [(1025, 64), (1025, 1000), (257, 1032), (300, 8208)])
def test_backward_first_rows_that_are_walked(M, T, d):
    """A row more than a backward launch has waves (1024) or workgroups (256)."""
    check_backward(M, T, d, BF, F32, True, True, "token", 0.1, True)
    check_backward(M, T, d, F32, BF, True, False, "channel", 0.0, True)


def test_random_numbers_that_are_no_tensor_are_refused(M):
    z = torch.zeros(4, 64, device=DEV)
    for rng, err in (([1, 2], TypeError), (torch.tensor([1, 2], dtype=torch.int32, device=DEV), TypeError), (torch.tensor([1, 2]), ValueError),
                     (torch.tensor([1, 2, 3], device=DEV), ValueError)):
        with pytest.raises(err, match="rng"):
            M.moe_block_norm(z, dropout=0.5, rng=rng)
        with pytest.raises(err, match="rng"):
            M.moe_block_norm_backward(z, dy=z, dropout=0.5, rng=rng, y_dtype=F32)
    one = torch.tensor([1, 2], device=DEV)
    a, b = (M.moe_block_norm(z + 1, dropout=0.5, rng=r)[0] for r in (one, one.view(torch.uint64)))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ the largest sizes

def test_largest_rows(M):
    """Just under 2^31 values: the last rows as those rows by themselves, and the counter's bits there."""
    T, d, at, p = 262143, 8184, 262140, 0.25
    seed, off = 5, 6
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, dtype=BF, device=DEV, generator=g)
    z, res, wa, wb, ch = r(T, d), r(T, d), rnd(2, d).abs().to(DEV) + 0.3, rnd(3, d).abs().to(DEV) + 0.3, rnd(4, 1, d).to(DEV)
    end = lambda t: t[at:].clone()
    kw = dict(w_after=wa, gate=ch, w_before=wb)
    got = M.moe_block_norm(z, residual=res, want_codes=True, **kw)
    few = M.moe_block_norm(end(z), residual=end(res), want_codes=True, **kw)
    for a, b in zip(got, few):
        assert torch.equal(a[at:], b)
    y = got[0]
    del got
    # dropout: which elements stay in the last rows, from the counter
    b = np.arange(at * d // 8, T * d // 8, dtype=np.uint64)
    ctr = np.stack([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, off), np.zeros_like(b)], -1)
    words = R.philox4x32_10(ctr, (seed, 0))
    kept = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(T - at, d) >= int(p * 65536)
    rng = torch.tensor([seed, off], device=DEV)
    one = M.moe_block_norm(z.fill_(1.0), dropout=p, rng=rng)[0]
    assert torch.equal(one[at:].cpu() != 0, torch.from_numpy(kept))
    del one
    z.copy_(res)
    du, dy = r(T, d), r(T, d)
    got = M.moe_block_norm_backward(z, y=y, du=du, dy=dy, want=("dz", "dresidual", "dw_before"), **kw)
    few = M.moe_block_norm_backward(end(z), y=end(y), du=end(du), dy=end(dy), want=("dz", "dresidual", "dw_before"), **kw)
    assert torch.equal(got[0][at:], few[0]) and torch.equal(got[1][at:], few[1])
    # dw_before: a sum over all rows, each partial row (1024 and fewer terms) and their sum within T + 16 roundings of the magnitudes
    want, mag = torch.zeros(d, dtype=torch.float64, device=DEV), torch.zeros(d, dtype=torch.float64, device=DEV)
    for t in range(0, T, 8192):
        yb, db = y[t:t + 8192].double(), du[t:t + 8192].double()
        term = db * yb * torch.rsqrt((yb * yb).mean(1, keepdim=True) + 1e-6)
        want, mag = want + term.sum(0), mag + term.abs().sum(0)
    assert ((got[4].double() - want).abs() <= (4 * REL + (T + 16) * 2.0 ** -24) * mag).all()
