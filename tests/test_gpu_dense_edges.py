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


def _spread(got, clean, where, what):
    """NaN (or an infinity) exactly at `where` (a mask, or True / False for all / none); elsewhere the clean call's bits."""
    m = where if isinstance(where, torch.Tensor) else torch.full_like(clean, where, dtype=torch.bool)
    assert not torch.isfinite(got[m].float()).any(), f"{what}: {int(torch.isfinite(got[m].float()).sum())} of {int(m.sum())} values lost it"
    assert torch.equal(got[~m], clean[~m]), f"{what}: it reached other values"


def _at(t, *idx):
    m = torch.zeros_like(t, dtype=torch.bool)
    m[idx] = True
    return m


@pytest.mark.parametrize("T", [6, 20, 80, 300])
@pytest.mark.parametrize("fn", ["none", "silu", "gelu", "gelu_tanh", "relu"])
def test_nonfinite_values_in_linear_gradients(M, fn, T):
    n, k, all_ = 72, 136, slice(None)
    x, w, b, dy = rnd(1, T, k), rnd(2, n, k, std=k ** -0.5), rnd(3, n, dtype=f32), rnd(4, T, n)
    run = lambda x=x, w=w, b=b, dy=dy: M.moe_dense_linear_backward(dy, x, w, b, fn)
    cx, cw, cb = run()
    put = lambda t, i, v=math.nan: t.clone().index_put_(tuple(torch.tensor(j) for j in i), torch.tensor(v, dtype=t.dtype, device="cuda"))
    act = fn != "none"
    # row 2 of x enters z's row 2, hence every sum over tokens; without an activation only dw's own column
    dx, dw, db = run(x=put(x, (2, 5)))
    _spread(dx, cx, _at(cx, 2) if act else False, "dx of x")
    _spread(dw, cw, True if act else _at(cw, all_, 5), "dw of x")
    _spread(db, cb, act, "dbias of x")
    dx, dw, db = run(w=put(w, (70, 4)))
    _spread(dx, cx, True if act else _at(cx, all_, 4), "dx of w")
    _spread(dw, cw, _at(cw, 70) if act else False, "dw of w")
    _spread(db, cb, _at(cb, 70) if act else False, "dbias of w")
    dx, dw, db = run(b=put(b, (7,)))
    for g, c, m in ((dx, cx, True), (dw, cw, _at(cw, 7)), (db, cb, _at(cb, 7))):
        _spread(g, c, m if act else False, "bias")
    for v in (math.nan, math.inf):
        dx, dw, db = run(dy=put(dy, (2, 71), v))
        for g, c, m in ((dx, cx, _at(cx, 2)), (dw, cw, _at(cw, 71)), (db, cb, _at(cb, 71))):
            _spread(g, c, m, f"dy {v}")


@pytest.mark.parametrize("T", [6, 80, 300])
@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh", "relu"])
def test_nonfinite_values_in_gated_gradients(M, fn, T):
    d, f = 136, 72
    x, wg, wu, dh = rnd(1, T, d), rnd(2, f, d, std=d ** -0.5), rnd(3, f, d, std=d ** -0.5), rnd(4, T, f)
    run = lambda wg=wg, wu=wu, pre=None: M.moe_dense_gateup_backward(dh, x, wg, wu, act_fn=fn, pre=pre, want_h=True)
    put = lambda t, i: t.clone().index_put_(tuple(torch.tensor(j) for j in i), torch.tensor(math.nan, dtype=t.dtype, device="cuda"))
    clean = run()
    cx, cg, cu, cbg, cbu, ch = clean
    col, names = slice(None), ("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h")
    # a gate weight: g's column, so dg, du and h there; an up weight: dg and h, while du = dh f(g) knows nothing of u
    for got, masks, what in ((run(wg=put(wg, (70, 4))), (True, _at(cg, 70), _at(cu, 70), _at(cbg, 70), _at(cbu, 70), _at(ch, col, 70)), "w_gate"),
                             (run(wu=put(wu, (70, 4))), (True, _at(cg, 70), False, _at(cbg, 70), False, _at(ch, col, 70)), "w_up")):
        for g, c, m, name in zip(got, clean, masks, names):
            _spread(g, c, m, f"{name} of {what}")
    pre = M.moe_dense_gateup(x, wg, wu, act_fn=fn, want_pre=True)[1]
    clean = run(pre=pre)
    row = _at(clean[0], 2)
    for i, up in ((0, _at(cu, 70)), (1, False)):
        got = run(pre=put(pre, (i, 2, 70)))
        masks = (row, _at(cg, 70), up, _at(cbg, 70), _at(cbu, 70) if i == 0 else False, _at(ch, 2, 70))
        for g, c, m, name in zip(got, clean, masks, names):
            _spread(g, c, m, f"{name} of saved {'gu'[i]}")


@pytest.mark.parametrize("T", [2, 9, 64, 100])
def test_float32_rows_in_a_weight_gradient_are_within_two_terms(M, T):
    # dw = x0 - x1 with x1 the value of x0's top 16 bits (two bf16 terms, exactly): what is left is x0's low byte, and x0's
    # two leading terms are within 2^-16 of it; the bf16 rounding of the small difference and the sum's (two products a
    # token and term, of which four are not zero) add little
    k = 512
    bits = torch.randint(0, 2 ** 23, (k,), generator=torch.Generator().manual_seed(1), dtype=torch.int32) + 0x3f800000
    bits[:4] = torch.tensor([0x3f80ffff, 0x3f8000ff, 0x3fffffff, 0x3f800080], dtype=torch.int32)
    x0 = bits.view(f32)
    x = torch.zeros(T, k, dtype=f32)
    x[0], x[1] = x0, (bits & -256).view(f32)
    dy = torch.zeros(T, 8, dtype=bf16)
    dy[0], dy[1] = 1, -1
    w = rnd(2, 8, k)
    dw = M.moe_dense_linear_backward(dy.cuda(), x.cuda(), w, want=("dw",))[1].double().cpu()
    ref = x0.double() - x[1].double()
    tol = 2.0 ** -16 * x0.double() + R.BF16 * (ref + 2.0 ** -16 * x0.double()) + 8 * R.EPS32 * 2 * x0.double()
    worst = ((dw - ref).abs() / tol).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("T", [2, 12, 100])
@pytest.mark.parametrize("xt", [bf16, f32])
def test_small_rows_are_not_lost(M, T, xt):
    # rows down to the smallest numbers against weights of 2^100: a bf16 value is one term, subnormal or not, and float32's
    # terms end at 2^-133
    k = 64
    x, w = rnd(1, T, k, dtype=f32) * torch.exp2(-torch.arange(100, 100 + k, dtype=f32) * 0.5 - 60).cuda(), rnd(2, 24, k, std=0.1) * 2.0 ** 100
    x = (x * 2.0 ** -6).to(xt)
    y = M.moe_dense_linear(x, w, out_dtype=f32)
    ref, tol = R.linear(x, w, None, "none", None, f32)
    tol = tol + 2.0 ** -133 * w.double().abs().sum(1)
    worst = ((y.double() - ref).abs() / tol).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("n,k", [(40, 64), (2375, 2056), (8200, 7176)])
@pytest.mark.parametrize("xt", [bf16, f32])
def test_weight_gradients_of_no_tokens_are_zeros(M, n, k, xt):
    x, w, dy = torch.empty(0, k, dtype=xt, device="cuda"), rnd(1, n, k), torch.empty(0, n, dtype=bf16, device="cuda")
    for fn in ("none", "gelu"):
        dw, db = torch.full((n, k), math.nan, dtype=bf16, device="cuda"), torch.full((n,), math.nan, device="cuda")
        M.moe_dense_linear_backward(dy, x, w, None, fn, want=("dw", "dbias"), out=(None, dw, db))
        assert not dw.any() and not db.any()
    f = n // 8 * 8
    out = [torch.full(s, math.nan, dtype=t, device="cuda") for s, t in (((f, k), bf16), ((f, k), bf16), ((f,), f32), ((f,), f32))]
    M.moe_dense_gateup_backward(dy[:, :f].contiguous(), x.to(bf16), w[:f], w[:f], want=("dw", "db"), out=(None, *out, None))
    assert all(not t.any() for t in out)


def test_grids_of_more_threads_than_a_launch_holds(M):
    # 2^26 columns at four a workgroup of 256 threads, and 2^25 rows at two: whole numbers, so results are exact
    def ints(seed, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.int8).to(bf16)
    n = 2 ** 26 + 24
    w, wu, x = ints(1, -3, 3, n, 8), ints(2, -3, 3, n, 8), ints(3, 1, 2, 1, 8)
    y = M.moe_dense_linear(x, w, out_dtype=f32)
    z = (w * x).float().sum(1)
    assert torch.equal(y[0], z)
    del y
    h = M.moe_dense_gateup(x, w, wu, act_fn="relu", out_dtype=f32)[0]
    assert torch.equal(h[0], z.clamp(min=0) * (wu * x).float().sum(1))
    del w, wu, h, z
    T = 2 ** 25 + 6
    pre, dh, wg, wu = ints(4, -1, 1, 2, T, 8), ints(5, -2, 2, T, 8), ints(6, -1, 1, 8, 8), ints(7, -1, 1, 8, 8)
    dx, _, _, dbg, dbu, _ = M.moe_dense_gateup_backward(dh, None, wg, wu, act_fn="relu", pre=pre, want=("dx", "db"))
    dg, du = dh.float() * pre[1].float() * (pre[0] > 0), dh.float() * pre[0].float().clamp(min=0)
    assert torch.equal(dx.float(), dg @ wg.float() + du @ wu.float())
    # (sums of 2^25 whole numbers of both signs stay below 2^24: exact in float32)
    assert torch.equal(dbg.double(), dg.double().sum(0)) and torch.equal(dbu.double(), du.double().sum(0))


def test_short_workspaces_are_refused(M):
    T, n, k = 64, 264, 136
    x, w, dy = rnd(1, T, k, dtype=f32), rnd(2, n, k), rnd(3, T, n)
    xb = x.to(bf16)
    B = M.binding
    calls = [(B.moe_dense_linear_workspace(T, n, k, x_dtype=f32, out_dtype=f32), lambda ws: (M.moe_dense_linear(x, w, ws=ws),)),
             (B.moe_dense_linear_backward_workspace(T, n, k, "silu"), lambda ws: M.moe_dense_linear_backward(dy, xb, w, None, "silu", ws=ws)),
             (B.moe_dense_gateup_workspace(T, 2376, 72), lambda ws: M.moe_dense_gateup(rnd(4, T, 2376), rnd(5, 72, 2376), rnd(6, 72, 2376), ws=ws)[:1]),
             (B.moe_dense_gateup_backward_workspace(T, k, n), lambda ws: M.moe_dense_gateup_backward(dy, xb, w, w, ws=ws, want_h=True))]
    for i, (need, call) in enumerate(calls):
        assert need > 256, i
        for have in (8, need - 1):
            with pytest.raises(M.MoeError, match=f"workspace of {need} bytes needed, got {have}") as e:
                call(torch.empty(have, dtype=torch.uint8, device="cuda"))
            assert e.value.status == B.MOE_ERR_WORKSPACE
        with pytest.raises(TypeError, match="ws"):
            call(torch.empty(need, dtype=f32, device="cuda"))
        with pytest.raises(ValueError, match="ws"):
            call(torch.empty(need, dtype=torch.uint8))
        for a, b in zip(call(torch.empty(need, dtype=torch.uint8, device="cuda")), call(None)):
            assert torch.equal(a, b), i


# Sizes at which a product takes a tile shape in a form that those of test_gpu_dense.py do not reach (test_dense_host.py
# asserts that the two together reach every one): (tokens, d_ff, d_model) of the gated block, (tokens, n, k) of a linear
# layer with an activation and bf16 or float32 rows
MORE_GATED = [(4725, 400, 3456), (73, 5672, 4072), (257, 6816, 5416), (564, 4688, 7904), (1298, 1608, 5432), (7873, 5992, 136),
              (132, 7448, 808), (454, 64, 64), (7798, 5648, 272)]
MORE_LINEAR = [(11, 64, 64, f32), (569, 7888, 3616, f32), (3511, 5704, 432, f32), (6035, 368, 5464, f32), (554, 6104, 7496, bf16)]


def rnd_gpu(seed, *shape, std=1.0, dtype=bf16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("T,f,d", MORE_GATED)
def test_more_gated_tiles(M, T, f, d):
    x, wg, wu = rnd_gpu(1, T, d), rnd_gpu(2, f, d, std=d ** -0.5), rnd_gpu(3, f, d, std=d ** -0.5)
    bg, bu, dh = rnd_gpu(4, f, dtype=f32), rnd_gpu(5, f, dtype=f32), rnd_gpu(6, T, f)
    R.check(M.moe_dense_gateup(x, wg, wu, bg, bu, "silu")[0], R.gateup(x, wg, wu, bg, bu, "silu", bf16), "h")
    got = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, "silu", want_h=True)
    for name, g, r in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h"), got, R.gateup_backward(dh, x, wg, wu, bg, bu, "silu")):
        R.check(g, r, name)


@pytest.mark.parametrize("T,n,k,xt", MORE_LINEAR)
def test_more_linear_tiles(M, T, n, k, xt):
    x, w, b, dy = rnd_gpu(1, T, k, dtype=xt), rnd_gpu(2, n, k, std=k ** -0.5), rnd_gpu(3, n, dtype=f32), rnd_gpu(4, T, n)
    R.check(M.moe_dense_linear(x, w, b, "silu", out_dtype=f32), R.linear(x, w, b, "silu", None, f32), "y")
    for name, g, r in zip(("dx", "dw", "dbias"), M.moe_dense_linear_backward(dy, x, w, b, "silu"), R.linear_backward(dy, x, w, b, "silu")):
        R.check(g, r, name)


def _slope(loss, args, i, v):
    """d loss / d args[i] along v by central differences in float64, extrapolated from two steps."""
    def d(eps):
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + eps * v, args[i] - eps * v
        return ((loss(up) - loss(dn)) / (2 * eps)).item()
    step = 1e-3 / v.abs().max().item()
    a, b = d(step), d(step / 2)
    s = (4 * b - a) / 3
    assert abs(b - a) <= 1e-4 * abs(s), "the step is too long"
    return s


@pytest.mark.parametrize("T", [7, 24, 90])
@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
def test_gradients_along_themselves_against_differences(M, fn, T):
    # along a gradient g the loss rises by |g|^2: no signs cancel, so a factor in a derivative shows in full.  The error is at
    # most the sum of the elements' bounds times |g|, 2^-8 of |g|^2 and less for bf16 results; the extrapolated
    # differences leave 1e-4 squared
    d, f = 64, 40
    x, wg, wu = rnd(1, T, d), rnd(2, f, d, std=d ** -0.5), rnd(3, f, d, std=d ** -0.5)
    bg, bu, dh = rnd(4, f, dtype=f32), rnd(5, f, dtype=f32), rnd(6, T, f)
    args = [t.double() for t in (x, wg, wu, bg, bu)]
    loss = lambda a: ((R.act(fn, a[0] @ a[1].t() + a[3])[0] * (a[0] @ a[2].t() + a[4])) * dh.double()).sum()
    got = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, fn)
    for i, (g, (_, tol)) in enumerate(zip(got[:5], R.gateup_backward(dh, x, wg, wu, bg, bu, fn)[:5])):
        v = g.double()
        num, ana = _slope(loss, args, i, v), (v * v).sum().item()
        assert abs(num - ana) <= (tol * v.abs()).sum().item() + 1e-7 * ana, ("gated", i, num, ana)
    args, loss = [t.double() for t in (x, wg, bg)], lambda a: (R.act(fn, a[0] @ a[1].t() + a[2])[0] * dh.double()).sum()
    for xt in (bf16, f32):
        got = M.moe_dense_linear_backward(dh, x.to(xt), wg, bg, fn, dx_dtype=f32)
        for i, (g, (_, tol)) in enumerate(zip(got, R.linear_backward(dh, x.to(xt), wg, bg, fn, f32))):
            v = g.double()
            num, ana = _slope(loss, args, i, v), (v * v).sum().item()
            assert abs(num - ana) <= (tol * v.abs()).sum().item() + 1e-7 * ana, ("linear", xt, i, num, ana)


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T", [24, 100])
def test_block_called_on_its_own_results(M, checkpoint, T):
    # one block several times: its output is its next input, and its input's gradient the next pass's dy
    d, f = 96, 136
    w = rnd(1, f, d, std=d ** -0.5), rnd(2, f, d, std=d ** -0.5), rnd(3, d, f, std=f ** -0.5)
    a, b = (M.DenseFFN(*w, T, checkpoint=checkpoint) for _ in range(2))
    y, ref, dy = rnd(4, T, d), rnd(4, T, d), rnd(5, T, d)
    for step in range(3):
        y, ref = a.forward(y, y, train=True), b.forward(ref.clone(), ref.clone(), train=True)
        assert torch.equal(y, ref), step
        want = b.backward(dy.clone())
        for i, (g, r) in enumerate(zip(a.backward(dy), want)):
            assert torch.equal(g, r), (step, i)
        # (the gradient with respect to the input, in the block's own buffer, is what comes next)
        dy = a.dx
    assert a.forward(y, train=True) is y
    keep = rnd(4, T, d)
    first = b.forward(keep, train=True).clone()
    want = [t.clone() for t in b.backward(first)]
    assert all(torch.equal(g, r) for g, r in zip((a.forward(keep, train=True), a.backward(a.y))[1], want))


def test_offsets_past_two_gib_within_a_tile(M):
    # operands near the size limit: a tile's rows, or the rows of one step, lie up to 4 GiB apart.  One value a sum, so
    # results are exact
    def pattern(rows, cols):
        t = torch.empty(rows, cols, dtype=bf16, device="cuda")
        a = torch.arange(cols, device="cuda", dtype=torch.int32)
        for r in range(rows):
            t[r] = (a + 5 * r) % 251 - 125
        return t
    k = 2 ** 23
    x, w = torch.zeros(250, k, dtype=bf16, device="cuda"), pattern(40, k)
    at = [(0, 3), (127, k - 1), (128, 2 ** 22), (200, 0), (249, k - 1)]
    for r, c in at:
        x[r, c] = 2
    y = M.moe_dense_linear(x, w, out_dtype=f32)
    for r, c in at:
        assert torch.equal(y[r], 2 * w[:, c].float()), (r, c)
        y[r] = 0
    assert not y.any()
    del x, y, w
    n, k = 64, 2 ** 25 - 8
    w, dy = pattern(n, k), torch.zeros(3, n, dtype=bf16, device="cuda")
    dy[0, 63], dy[1, 0], dy[2, 40] = 1, 2, -1
    dx = M.moe_dense_linear_backward(dy, None, w, want=("dx",))[0]
    assert torch.equal(dx[0], w[63]) and torch.equal(dx[1], 2 * w[0]) and torch.equal(dx[2], -w[40])
    del w, dy, dx
    for T, n in ((72, 29826000), (64, 2 ** 25 - 16)):
        dy, x = pattern(T, n), torch.zeros(T, 8, dtype=bf16, device="cuda")
        for j in range(8):
            x[7 * j, j] = 1
        dw = M.moe_dense_linear_backward(dy, x, torch.empty(n, 8, dtype=bf16, device="cuda"), want=("dw",))[1]
        for j in range(8):
            assert torch.equal(dw[:, j], dy[7 * j]), (T, j)
        del dy, x, dw
