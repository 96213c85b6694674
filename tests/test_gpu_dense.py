"""Dense bf16 layers (linear, gated projections, gradients, MXFP8 checkpoints) against float64 (GPU)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_ref as R

pytestmark = pytest.mark.gpu

bf16, f32 = torch.bfloat16, torch.float32
FNS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import mxfp4_routed_expert_amd as m
    return m


def rnd(seed, *shape, std=1.0, dtype=bf16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def lin_inputs(T, n, k, bias, residual, xt=bf16, yt=bf16, seed=0):
    return (rnd(seed, T, k, dtype=xt), rnd(seed + 1, n, k, std=k ** -0.5), rnd(seed + 2, n, std=0.5, dtype=f32) if bias else None,
            rnd(seed + 3, T, n, dtype=yt) if residual else None)


# sizes: one token to several tiles; sums of a single chunk, with tails and of whole steps; odd widths
LIN = [(1, 1, 8), (1, 2048, 520), (2, 33, 72), (3, 130, 512), (5, 64, 1032), (8, 257, 200), (9, 31, 8), (16, 128, 64),
       (17, 100, 72), (63, 129, 264), (64, 256, 1024), (65, 77, 136), (129, 300, 2368), (300, 515, 200), (513, 1000, 520)]


@pytest.mark.parametrize("T,n,k", LIN)
@pytest.mark.parametrize("xt,yt", [(bf16, bf16), (bf16, f32), (f32, f32), (f32, bf16)])
def test_linear(M, T, n, k, xt, yt):
    i = LIN.index((T, n, k))
    fn = FNS[i % 5]
    x, w, b, r = lin_inputs(T, n, k, i % 2 == 0, i % 3 != 0, xt, yt, seed=10 * i)
    print(f"linear T={T} n={n} k={k} {fn} {xt} -> {yt}", flush=True)
    y = M.moe_dense_linear(x, w, b, fn, r, out_dtype=yt)
    R.check(y, R.linear(x, w, b, fn, r, yt), "y")
    assert torch.equal(y, M.moe_dense_linear(x, w, b, fn, r, out_dtype=yt)), "two runs differ"


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("T", [4, 40, 200])
def test_linear_activations(M, fn, T):
    x, w, b, r = lin_inputs(T, 96, 128, True, True, bf16, f32, seed=7)
    w = w * 6                                    # arguments of both signs out to the tails
    R.check(M.moe_dense_linear(x, w, b, fn, r, out_dtype=f32), R.linear(x, w, b, fn, r, f32), f"{fn} T={T}")


@pytest.mark.parametrize("T,n,k", [(2048, 2048, 520), (1500, 7168, 72), (700, 2376, 1032), (260, 7168, 2368)])
def test_linear_large_tiles(M, T, n, k):
    for fn, xt in (("gelu", bf16), ("none", f32)):
        x, w, b, r = lin_inputs(T, n, k, True, True, xt, f32, seed=3)
        R.check(M.moe_dense_linear(x, w, b, fn, r, out_dtype=f32), R.linear(x, w, b, fn, r, f32), f"T={T} n={n} k={k} {fn}")


def test_linear_residual_in_place(M):
    for T in (3, 70):
        x, w, b, r = lin_inputs(T, 136, 264, True, True, seed=5)
        ref = R.linear(x, w, b, "silu", r, bf16)
        y = M.moe_dense_linear(x, w, b, "silu", r, out=r)
        assert y is r
        R.check(y, ref, f"in place T={T}")


def test_linear_f32_terms(M):
    # float32 rows of every magnitude up to the largest, subnormals, infinities and NaN: finite rows keep
    # float32's accuracy, the others reach their own rows only
    k = 64
    x = rnd(1, 40, k, dtype=f32)
    x[3] *= 2.0 ** 120
    x[4] *= 2.0 ** -130
    x[5, 7] = math.inf
    x[6, 9] = math.nan
    x[7, 0] = torch.finfo(f32).max
    w = rnd(2, 24, k, std=0.01)
    y = M.moe_dense_linear(x, w, out_dtype=f32)
    ref, tol = R.linear(x, w, None, "none", None, f32)
    rows = [i for i in range(40) if i not in (5, 6)]
    R.check(y[rows], (ref[rows], tol[rows]), "finite rows")
    assert torch.isinf(y[5]).all() and torch.isnan(y[6]).all()
    assert torch.equal(torch.sign(y[5]), torch.sign(w[:, 7].float()))


@pytest.mark.parametrize("T", [6, 20, 300])
def test_nonfinite_values_stay_in_their_rows(M, T):
    x, w, b, _ = lin_inputs(T, 72, 136, True, False, seed=11)
    clean = M.moe_dense_linear(x, w, b, "silu")
    x2, w2 = x.clone(), w.clone()
    x2[2, 130] = math.nan
    w2[70, 3] = math.inf
    y = M.moe_dense_linear(x2, w2, b, "silu")
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[2] = False
    keep[:, 70] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[:, 70].float()).all()


@pytest.mark.parametrize("T", [2, 12, 80])
@pytest.mark.parametrize("fn", FNS[1:])
def test_activations_of_huge_arguments(M, fn, T):
    # f is z or 0 and f' 1 or 0 for every finite argument this far out, also where its powers overflow
    v = torch.tensor([s * m for m in (1e3, 1e5, 1e13, 1e20, 3e38) for s in (1, -1)] + [0.0] * 6).to(bf16).cuda()
    x = torch.zeros(T, 8, dtype=bf16, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(16, 8, dtype=bf16, device="cuda")
    w[:, 0] = v
    one = torch.ones(T, 16, dtype=bf16, device="cuda")
    f, on = v.float().clamp(min=0).expand(T, 16), (v[:10] > 0).float()
    assert torch.equal(M.moe_dense_linear(x, w, None, fn, out_dtype=f32), f)
    _, dw, db = M.moe_dense_linear_backward(one, x, w, None, fn, want=("dw", "dbias"))
    assert torch.equal(db[:10], T * on) and torch.equal(dw[:10, 0].float(), T * on)
    wu = torch.zeros_like(w)
    wu[:, 0] = 1
    h, pre = M.moe_dense_gateup(x, w, wu, act_fn=fn, out_dtype=f32, want_pre=True)
    assert torch.equal(h, f)
    for p in (None, pre):
        got = M.moe_dense_gateup_backward(one, x, w, wu, act_fn=fn, pre=p, want=("dw", "db"), want_h=True, h_dtype=f32)
        assert torch.equal(got[3][:10], T * on) and torch.equal(got[1][:10, 0].float(), T * on)
        assert torch.equal(got[5], f) and (got[4][v <= 0] == 0).all()


GATE = [(1, 8, 8), (1, 2048, 200), (2, 72, 40), (4, 520, 136), (7, 512, 64), (9, 136, 8), (33, 64, 264), (64, 264, 72),
        (100, 200, 136), (257, 72, 520), (520, 520, 328), (1100, 264, 2368)]


@pytest.mark.parametrize("T,d,f", GATE)
@pytest.mark.parametrize("ht", [bf16, f32])
def test_gateup(M, T, d, f, ht):
    i = GATE.index((T, d, f))
    fn = FNS[1 + i % 4]
    x, wg, wu = rnd(i, T, d), rnd(i + 1, f, d, std=d ** -0.5), rnd(i + 2, f, d, std=d ** -0.5)
    bg, bu = (rnd(i + 3, f, dtype=f32), rnd(i + 4, f, dtype=f32)) if i % 2 else (None, None)
    print(f"gateup T={T} d={d} f={f} {fn} -> {ht}", flush=True)
    h, pre = M.moe_dense_gateup(x, wg, wu, bg, bu, fn, out_dtype=ht, want_pre=True)
    R.check(h, R.gateup(x, wg, wu, bg, bu, fn, ht), "h")
    for j, (w, b) in enumerate(((wg, bg), (wu, bu))):
        z, ez = R.product(x, w, b)
        R.check(pre[j], (z, R.rounded(z, ez, bf16)), "pre")
    h2, none = M.moe_dense_gateup(x, wg, wu, bg, bu, fn, out_dtype=ht)
    assert none is None and torch.equal(h, h2), "keeping the pre-activations changes h"


BWD = [(1, 8, 8), (1, 520, 264), (5, 33, 72), (16, 130, 64), (63, 257, 96), (64, 64, 128), (65, 100, 520), (200, 515, 264),
       (333, 136, 1032), (1030, 520, 264)]


@pytest.mark.parametrize("T,n,k", BWD)
@pytest.mark.parametrize("fn", ["none", "gelu"])
def test_linear_backward(M, T, n, k, fn):
    i = BWD.index((T, n, k))
    x, w, b, _ = lin_inputs(T, n, k, i % 2 == 0, False, seed=20 * i)
    dy = rnd(20 * i + 9, T, n)
    print(f"linear backward T={T} n={n} k={k} {fn}", flush=True)
    got = M.moe_dense_linear_backward(dy, x, w, b, fn)
    for name, g, r in zip(("dx", "dw", "dbias"), got, R.linear_backward(dy, x, w, b, fn)):
        R.check(g, r, name)
    # each gradient alone is the same
    for j, name in enumerate(("dx", "dw", "dbias")):
        one = M.moe_dense_linear_backward(dy, x, w, b, fn, want=(name,))
        assert torch.equal(one[j], got[j]) and all(o is None for o in one[:j] + one[j + 1:])


@pytest.mark.parametrize("T,n,k", [(1, 40, 64), (9, 33, 72), (64, 136, 264), (65, 100, 136), (300, 264, 200)])
@pytest.mark.parametrize("fn", ["none", "silu"])
def test_linear_backward_float32(M, T, n, k, fn):
    x, w, b, _ = lin_inputs(T, n, k, True, False, xt=f32, seed=T)
    dy = rnd(T + 9, T, n)
    got = M.moe_dense_linear_backward(dy, x, w, b, fn, dx_dtype=f32)
    assert got[0].dtype == f32 and got[1].dtype == bf16
    for name, g, r in zip(("dx", "dw", "dbias"), got, R.linear_backward(dy, x, w, b, fn, f32)):
        R.check(g, r, name)


@pytest.mark.parametrize("fn", FNS)
def test_linear_backward_activations(M, fn):
    x, w, b, _ = lin_inputs(50, 96, 128, True, False, seed=7)
    w = w * 4
    dy = rnd(8, 50, 96)
    for g, r in zip(M.moe_dense_linear_backward(dy, x, w, b, fn), R.linear_backward(dy, x, w, b, fn)):
        R.check(g, r, fn)


GBWD = [(1, 8, 8), (1, 264, 72), (6, 64, 136), (17, 200, 40), (64, 96, 64), (65, 520, 328), (250, 72, 264), (333, 264, 520),
        (1030, 520, 136)]


@pytest.mark.parametrize("T,d,f", GBWD)
@pytest.mark.parametrize("saved", [False, True])
def test_gateup_backward(M, T, d, f, saved):
    i = GBWD.index((T, d, f))
    fn = FNS[1 + i % 4]
    x, wg, wu = rnd(i, T, d), rnd(i + 1, f, d, std=d ** -0.5), rnd(i + 2, f, d, std=d ** -0.5)
    bg, bu = (rnd(i + 3, f, dtype=f32), rnd(i + 4, f, dtype=f32)) if i % 2 == 0 else (None, None)
    dh = rnd(i + 5, T, f)
    pre = M.moe_dense_gateup(x, wg, wu, bg, bu, fn, want_pre=True)[1] if saved else None
    print(f"gateup backward T={T} d={d} f={f} {fn} saved={saved}", flush=True)
    got = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, fn, pre=pre, want_h=True)
    ref = R.gateup_backward(dh, x, wg, wu, bg, bu, fn, pre)
    for name, g, r in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h"), got, ref):
        R.check(g, r, name)
    for want, idx in ((("dx",), (0,)), (("dw",), (1, 2)), (("db",), (3, 4))):
        part = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, fn, pre=pre, want=want)
        for j in range(6):
            assert (torch.equal(part[j], got[j]) if j in idx else part[j] is None), (want, j)
    if saved:      # neither the products' input nor its weight gradient is needed for dx
        part = M.moe_dense_gateup_backward(dh, None, wg, wu, bg, bu, fn, pre=pre, want=("dx",))
        assert torch.equal(part[0], got[0])


@pytest.mark.parametrize("T", [1, 40, 64, 65, 200])
def test_gateup_backward_float32_dh(M, T):
    d, f = 136, 264
    x, wg, wu, dh = rnd(1, T, d), rnd(2, f, d, std=d ** -0.5), rnd(3, f, d, std=d ** -0.5), rnd(5, T, f, dtype=f32)
    for pre in (None, M.moe_dense_gateup(x, wg, wu, want_pre=True)[1]):
        got = M.moe_dense_gateup_backward(dh, x, wg, wu, pre=pre, want_h=True, h_dtype=f32)
        assert got[5].dtype == f32
        ref = R.gateup_backward(dh, x, wg, wu, None, None, "silu", pre, f32)
        for name, g, r in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h"), got, ref):
            R.check(g, r, name)


@pytest.mark.parametrize("rows,cols,dt", [(1, 32, bf16), (3, 64, f32), (77, 96, bf16), (130, 416, f32), (64, 7168, bf16)])
def test_mxfp8(M, rows, cols, dt):
    x = rnd(rows, rows, cols, dtype=f32) * torch.exp2(torch.randint(-30, 30, (rows, 1)).float()).cuda()
    x[:, ::7] *= 0.01
    x = x.to(dt)
    flat = x.view(-1, 32)
    flat[0] = 0
    if flat.shape[0] > 4:
        flat[1, 3] = math.inf
        flat[2, 31] = math.nan
        flat[3] *= 2.0 ** -126                       # down into the subnormals
        flat[4] = torch.tensor([(-1) ** i * (1 + i / 16) * 2.0 ** (i % 9) for i in range(32)]).to(dt)   # ties
    codes, scales = M.moe_mxfp8_quantize(x)
    rc, rs = R.mxfp8(x.cpu())
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)
    vals = R.mxfp8_values(rc, rs)
    for odt in (bf16, f32):
        got = M.moe_mxfp8_dequant(codes, scales, out_dtype=odt).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(vals))
        ok = ~torch.isnan(vals)
        assert torch.equal(got[ok], vals[ok].to(odt)), odt


def test_mxfp8_every_code(M):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8).cuda()
    vals = R.mxfp8_values(codes.cpu(), scales.cpu())
    got = M.moe_mxfp8_dequant(codes, scales, out_dtype=f32).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(vals))
    ok = ~torch.isnan(vals)
    assert torch.equal(got[ok], vals[ok].float())


@pytest.mark.parametrize("T,d,f", [(1, 64, 72), (40, 96, 136), (300, 288, 200)])
def test_backward_from_mxfp8(M, T, d, f):
    x, wg, wu = rnd(1, T, d), rnd(2, f, d, std=d ** -0.5), rnd(3, f, d, std=d ** -0.5)
    dh = rnd(4, T, f)
    codes, scales = M.moe_mxfp8_quantize(x)
    xv = M.moe_mxfp8_dequant(codes, scales)           # exact in bf16 at these magnitudes
    assert torch.equal(xv.double().cpu(), R.mxfp8_values(*R.mxfp8(x.cpu())))
    got = M.moe_dense_gateup_backward(dh, codes, wg, wu, x_scales=scales, want_h=True)
    for a, b in zip(got, M.moe_dense_gateup_backward(dh, xv, wg, wu, want_h=True)):
        assert torch.equal(a, b)
    for g, r in zip(got, R.gateup_backward(dh, xv, wg, wu, None, None, "silu")):
        R.check(g, r, "gateup from the checkpoint")
    got = M.moe_dense_linear_backward(dh, codes, wg, None, "silu", x_scales=scales)
    for g, r in zip(got, R.linear_backward(dh, xv, wg, None, "silu")):
        R.check(g, r, "linear from the checkpoint")


def test_gradients_against_differences(M):
    # central differences of the float64 definition along a random direction
    T, d, f, eps = 24, 64, 40, 1e-5
    x, wg, wu = rnd(1, T, d), rnd(2, f, d, std=d ** -0.5), rnd(3, f, d, std=d ** -0.5)
    bg, bu, dh = rnd(4, f, dtype=f32), rnd(5, f, dtype=f32), rnd(6, T, f)
    for fn in ("silu", "gelu", "gelu_tanh"):
        got = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, fn)
        args = [t.double() for t in (x, wg, wu, bg, bu)]
        loss = lambda a: ((R.act(fn, a[0] @ a[1].t() + a[3])[0] * (a[0] @ a[2].t() + a[4])) * dh.double()).sum()
        for i in range(5):
            v = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).cuda()
            up, dn = list(args), list(args)
            up[i], dn[i] = args[i] + eps * v, args[i] - eps * v
            num = ((loss(up) - loss(dn)) / (2 * eps)).item()
            ana = (got[i].double() * v).sum().item()
            # each gradient element is within about 2^-7 of the sums of magnitudes that form it; their random
            # signs leave the directional sum within 2^-7 of the root of its squares, tenfold for certainty
            scale = (got[i].double() * v).square().sum().sqrt().item() + 1e-6
            assert abs(num - ana) <= 10 * 2 ** -7 * scale * math.sqrt(f / 8), (fn, i, num, ana, scale)


def test_no_tokens(M):
    x, w, b, _ = lin_inputs(0, 40, 64, True, False)
    assert M.moe_dense_linear(x, w, b, "relu").shape == (0, 40)
    dx, dw, db = M.moe_dense_linear_backward(torch.empty(0, 40, dtype=bf16, device="cuda"), x, w, b, "relu")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    r = M.moe_dense_gateup_backward(torch.empty(0, 40, dtype=bf16, device="cuda"), x, w, w, want_h=True)
    assert r[0].shape == (0, 64) and all(not t.any() for t in r[1:5])
    assert M.moe_mxfp8_quantize(x)[0].shape == (0, 64)


# sizes at which a gradient's column sums and the sum of a split input gradient run beside the other product, and not
@pytest.mark.parametrize("T,n,k", [(61, 2376, 1032), (333, 2368, 2056), (70, 264, 2056), (1030, 1032, 520), (2060, 2056, 1032)])
@pytest.mark.parametrize("fn", ["none", "gelu"])
def test_gradients_do_not_depend_on_what_else_is_asked(M, T, n, k, fn):
    x, w, b, dy = rnd_gpu(1, T, k), rnd_gpu(2, n, k, std=k ** -0.5), rnd_gpu(3, n, dtype=f32), rnd_gpu(4, T, n)
    every = M.moe_dense_linear_backward(dy, x, w, b, fn)
    for want in (("dx",), ("dw",), ("dbias",), ("dx", "dw"), ("dx", "dbias"), ("dw", "dbias")):
        for name, g, e in zip(("dx", "dw", "dbias"), M.moe_dense_linear_backward(dy, x, w, b, fn, want=want), every):
            assert (g is None) == (name not in want) and (g is None or torch.equal(g, e)), (want, name)
    wu, dh = rnd_gpu(5, n, k, std=k ** -0.5)[:n // 8 * 8], rnd_gpu(6, T, n // 8 * 8)
    wg = w[:n // 8 * 8]
    every = M.moe_dense_gateup_backward(dh, x, wg, wu, act_fn="silu")
    for want in (("dx",), ("dw",), ("db",), ("dx", "dw"), ("dx", "db"), ("dw", "db")):
        got = M.moe_dense_gateup_backward(dh, x, wg, wu, act_fn="silu", want=want)
        for name, g, e in zip(("dx", "dw", "dw", "db", "db"), got, every):
            assert (g is None) == (name not in want) and (g is None or torch.equal(g, e)), (want, name)


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
def test_block_of_no_tokens(M, checkpoint):
    ffn = M.DenseFFN(rnd(1, 40, 64), rnd(2, 40, 64), rnd(3, 64, 40), 0, checkpoint=checkpoint)
    x = torch.empty(0, 64, dtype=bf16, device="cuda")
    assert ffn.forward(x, x, train=True).shape == (0, 64)
    dx, *dws = ffn.backward(x)
    assert dx.shape == (0, 64) and all((g == 0).all() for g in dws)


# (rows, columns, sum) at which the forward and input-gradient products take each tile shape (256 x 256, 256 x 128,
# 128 x 128 in its two forms, 64 x 128) with the sum whole, split for the tiles of a last partial round, and split everywhere
TILES = [(9, 264, 136), (260, 7176, 136), (260, 7176, 328), (1030, 7176, 136), (9, 264, 1160), (70, 2056, 2376), (130, 7176, 4104),
         (4100, 264, 7176), (520, 7176, 2376), (1030, 4104, 2376), (2060, 7176, 1160), (1100, 7176, 2376),
         (130, 4104, 2056), (1100, 7176, 2056), (520, 7176, 136), (520, 7176, 7176), (520, 4104, 7176)]
# the gated products' (tokens, d_ff, d_model)
PAIR_TILES = [(9, 264, 136), (130, 7176, 136), (130, 7176, 328), (520, 7176, 136), (9, 264, 1160), (70, 1032, 2376), (130, 4104, 4104),
              (700, 1032, 7176), (260, 7176, 2376), (1030, 2056, 2376), (2060, 7176, 520), (4100, 1032, 4104),
              (130, 2056, 2056), (4100, 1032, 2056), (260, 7176, 136), (130, 4104, 7176), (4100, 2056, 1160)]
# input gradients of the gated products (tokens, d_model, d_ff): a sum of two parts
TWO_PART_TILES = [(70, 264, 136), (260, 7176, 136), (1030, 7176, 136), (70, 264, 520), (70, 2056, 1160), (130, 7176, 2376),
                  (520, 7176, 1160), (1030, 4104, 1160), (4100, 4104, 328), (130, 4104, 1160), (1030, 7176, 1160), (520, 7176, 136),
                  (520, 7176, 2376), (130, 7176, 7176), (520, 4104, 2376), (2060, 7176, 136)]
# weight gradients (tokens, n, k)
GRAD_TILES = [(9, 1032, 7176), (70, 4104, 7176), (520, 264, 136), (1030, 1032, 7176), (5200, 264, 7176), (5200, 2376, 1160),
              (1030, 4104, 4104), (2600, 4104, 4104), (1030, 7176, 520), (4100, 7176, 1160), (4100, 2056, 7176), (9, 264, 136), (2056, 6152, 2056)]


def rnd_gpu(seed, *shape, std=1.0, dtype=bf16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("T,n,k", TILES)
def test_linear_tiles(M, T, n, k):
    n -= 3                                   # rows of odd length
    x, w, b, r = rnd_gpu(1, T, k), rnd_gpu(2, n, k, std=k ** -0.5), rnd_gpu(3, n, dtype=f32), rnd_gpu(4, T, n)
    R.check(M.moe_dense_linear(x, w, b, "gelu", r), R.linear(x, w, b, "gelu", r, bf16), "y")
    x = x.float() + rnd_gpu(5, T, k, std=2 ** -12, dtype=f32)
    R.check(M.moe_dense_linear(x, w, None, "none"), R.linear(x, w, None, "none", None, f32), "y of float32 rows")


def _linear_backward(M, T, n, k, fn):
    x, w, b, dy = rnd_gpu(1, T, k), rnd_gpu(2, n, k, std=k ** -0.5), rnd_gpu(3, n, dtype=f32), rnd_gpu(4, T, n)
    got = M.moe_dense_linear_backward(dy, x, w, b, fn)
    for name, g, r in zip(("dx", "dw", "dbias"), got, R.linear_backward(dy, x, w, b, fn)):
        R.check(g, r, name)


@pytest.mark.parametrize("T,n,k", TILES)
def test_linear_backward_tiles(M, T, n, k):
    _linear_backward(M, T, n, k, "silu")


@pytest.mark.parametrize("T,k,n", TILES[1:])
def test_input_gradient_tiles(M, T, k, n):
    _linear_backward(M, T, n - 1, k, "none")  # an odd n: dz is dy with padded rows


@pytest.mark.parametrize("T,n,k", GRAD_TILES)
def test_weight_gradient_tiles(M, T, n, k):
    _linear_backward(M, T, n, k, "none")


def _gateup(M, T, d, f, bias):
    x, wg, wu = rnd_gpu(1, T, d), rnd_gpu(2, f, d, std=d ** -0.5), rnd_gpu(3, f, d, std=d ** -0.5)
    bg, bu = (rnd_gpu(4, f, dtype=f32), rnd_gpu(5, f, dtype=f32)) if bias else (None, None)
    dh = rnd_gpu(6, T, f)
    h, pre = M.moe_dense_gateup(x, wg, wu, bg, bu, "gelu_tanh", want_pre=True)
    R.check(h, R.gateup(x, wg, wu, bg, bu, "gelu_tanh", bf16), "h")
    for p in (None, pre):
        got = M.moe_dense_gateup_backward(dh, x, wg, wu, bg, bu, "gelu_tanh", pre=p, want_h=True)
        ref = R.gateup_backward(dh, x, wg, wu, bg, bu, "gelu_tanh", p)
        for name, g, r in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h"), got, ref):
            R.check(g, r, name)


@pytest.mark.parametrize("T,f,d", PAIR_TILES)
def test_gateup_tiles(M, T, f, d):
    _gateup(M, T, d, f, True)


@pytest.mark.parametrize("T,d,f", TWO_PART_TILES)
def test_gateup_input_gradient_tiles(M, T, d, f):
    _gateup(M, T, d, f, False)


def _block_ref(x, xb, wg, wu, wd, res, dy):
    """float64 block and gradients; h is rounded to bf16 between the products beyond 64 tokens, its gradient never."""
    T = x.shape[0]
    few = T <= 64
    ht = f32 if few else bf16
    g, eg = R.product(x, wg)
    u, eu = R.product(x, wu)
    h, eh = R.gated(g, eg, u, eu, "silu", ht)
    wa = wd.double().abs()
    y = h @ wd.double().t() + res.double()
    ey = eh @ wa.t() + (h.shape[1] + 8) * R.EPS32 * (h.abs() + eh) @ wa.t()
    dh, edh = R.product(dy, wd.t())
    out = R.gateup_backward(dh, xb, wg, wu, None, None, "silu", h_dtype=ht)
    (dx, ex), (dwg, ewg), (dwu, ewu), _, _, (h2, eh2) = out
    # dh's own error passes through the gradients linearly (their bounds leave 2% for its square)
    g, _ = R.product(xb, wg)
    u, _ = R.product(xb, wu)
    a, d = R.act("silu", g)
    pg, pu = edh * (u * d).abs() * 1.02, edh * a.abs() * 1.02
    ex = ex + pg @ wg.double().abs() + pu @ wu.double().abs()
    ewg = ewg + pg.t() @ xb.double().abs()
    ewu = ewu + pu.t() @ xb.double().abs()
    da = dy.double().abs().t()
    dwd = dy.double().t() @ h2
    ewd = da @ eh2 + ((2 * T + 8) * R.EPS32 + (2.0 ** -14 if few else 0.0)) * (da @ (h2.abs() + eh2))
    return (y, R.rounded(y, ey, bf16)), (dx, ex), (dwg, ewg), (dwu, ewu), (dwd, R.rounded(dwd, ewd, bf16))


@pytest.mark.parametrize("T,d,f", [(1, 64, 72), (24, 96, 136), (260, 288, 520)])
@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
def test_block_step(M, T, d, f, checkpoint):
    wg, wu, wd = rnd(1, f, d, std=d ** -0.5), rnd(2, f, d, std=d ** -0.5), rnd(3, d, f, std=f ** -0.5)
    ffn = M.DenseFFN(wg, wu, wd, T, checkpoint=checkpoint)
    with pytest.raises(M.MoeError):
        ffn.backward(rnd(0, T, d))
    for step in range(2):
        x, res, dy = rnd(10 + step, T, d), rnd(20 + step, T, d), rnd(30 + step, T, d)
        xb = x if checkpoint == "bf16" else M.moe_mxfp8_dequant(*M.moe_mxfp8_quantize(x))
        y = ffn.forward(x, res, train=True).clone()
        got = (y,) + tuple(ffn.backward(dy))
        for name, g, r in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), got, _block_ref(x, xb, wg, wu, wd, res, dy)):
            R.check(g, r, name)


@pytest.mark.parametrize("T", [4, 48, 520])
def test_block_step_captured(M, T):
    d, f = 288, 520
    wg, wu, wd = rnd(1, f, d, std=d ** -0.5), rnd(2, f, d, std=d ** -0.5), rnd(3, d, f, std=f ** -0.5)
    ffn, eager = (M.DenseFFN(wg, wu, wd, T, checkpoint="mxfp8") for _ in range(2))
    x, res, dy = rnd(4, T, d), rnd(5, T, d), rnd(6, T, d)
    ffn.forward(x, res, train=True)
    ffn.backward(dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ffn.forward(x, res, train=True)
        grads = ffn.backward(dy)
    for it in range(4):
        x.copy_(rnd(40 + it, T, d))
        dy.copy_(rnd(50 + it, T, d))
        g.replay()
        torch.cuda.synchronize()
        ref = (eager.forward(x, res, train=True),) + tuple(eager.backward(dy))
        torch.cuda.synchronize()
        for a, b in zip((y,) + tuple(grads), ref):
            assert torch.equal(a, b), f"replay {it} differs from the eager step"


def test_two_streams(M):
    # two calls in flight at once, each with its own workspace and stream
    ins = [lin_inputs(200, 264, 520, True, True, seed=100 * i) for i in range(2)]
    want = [M.moe_dense_linear(x, w, b, "gelu", r) for x, w, b, r in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i, (x, w, b, r) in enumerate(ins):
            with torch.cuda.stream(streams[i]):
                outs[i].append(M.moe_dense_linear(x, w, b, "gelu", r))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_rows_do_not_depend_on_their_batch_mates(M):
    x, w, b, _ = lin_inputs(300, 264, 520, True, False)
    y = M.moe_dense_linear(x, w, b, "silu")
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(M.moe_dense_linear(x[perm].contiguous(), w, b, "silu"), y[perm])


def test_outputs_beside_are_left_alone(M):
    # results land inside a larger buffer: the rows before and after keep their values
    for T, n in ((5, 40), (70, 40), (300, 264)):
        x, w, b, _ = lin_inputs(T, n, 64, True, False)
        buf = torch.full((T + 16, n), 7.0, dtype=bf16, device="cuda")
        M.moe_dense_linear(x, w, b, out=buf[8:8 + T])
        assert (buf[:8] == 7).all() and (buf[8 + T:] == 7).all()


def test_binding_refusals(M):
    x, w, b, r = lin_inputs(4, 40, 64, True, True)
    bad = [
        (ValueError, lambda: M.moe_dense_linear(x.cpu(), w)),
        (ValueError, lambda: M.moe_dense_linear(x[:, ::2], w[:, :32].contiguous())),
        (ValueError, lambda: M.moe_dense_linear(x, w[:, :56].contiguous())),
        (ValueError, lambda: M.moe_dense_linear(x, w, act_fn="tanh")),
        (TypeError, lambda: M.moe_dense_linear(x.half(), w)),
        (TypeError, lambda: M.moe_dense_linear(x, w.float())),
        (TypeError, lambda: M.moe_dense_linear(x, w, residual=r, out_dtype=f32)),
        (ValueError, lambda: M.moe_dense_linear(x[0], w)),
        (M.MoeError, lambda: M.moe_dense_linear(torch.zeros(4, 60, dtype=bf16, device="cuda"), w[:, :60].contiguous())),
        (M.MoeError, lambda: M.moe_dense_linear(torch.zeros(4 * 64 + 1, dtype=bf16, device="cuda")[1:].view(4, 64), w)),
        (M.MoeError, lambda: M.moe_dense_linear(rnd(0, 64, 64), rnd(0, 40, 64), ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
         if M.binding.moe_dense_linear_workspace(64, 40, 64) > 8 else M.binding.check(3)),
        (ValueError, lambda: M.moe_dense_linear_backward(r, x, w, want=())),
        (ValueError, lambda: M.moe_dense_linear_backward(r, x, w, want=("dy",))),
        (TypeError, lambda: M.moe_dense_linear_backward(r, x.half(), w)),
        (TypeError, lambda: M.moe_dense_linear_backward(r, x, w, dx_dtype=torch.half)),
        (TypeError, lambda: M.moe_dense_gateup_backward(r, x.float(), w, w)),
        (M.MoeError, lambda: M.moe_dense_linear_backward(r, None, w, want=("dw",))),
        (ValueError, lambda: M.moe_dense_gateup(x, w, w[:8].contiguous())),
        (ValueError, lambda: M.moe_mxfp8_dequant(x.view(torch.uint8)[:, :64].contiguous(), torch.zeros(4, 3, dtype=torch.uint8, device="cuda"))),
        (M.MoeError, lambda: M.moe_mxfp8_quantize(x[:, :40].contiguous())),
    ]
    for i, (exc, call) in enumerate(bad):
        with pytest.raises(exc):
            call()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("T", [1, 3, 40, 130])
@pytest.mark.parametrize("gated", [False, True])
def test_layer_with_bf16_shared_expert(M, T, gated):
    import dataclasses

    import numpy as np

    import gpu_common as G
    import synth
    from oracle import layer as OL
    cfg = dataclasses.replace(synth.get("tiny"), T=T)
    dev = torch.device("cuda:0")
    t, inp = G.build(cfg, dev)
    w = G.layer_weights(cfg, t)
    f = 136
    w.shared = M.DenseWeights(rnd(1, f, cfg.H, std=0.06), rnd(2, f, cfg.H, std=0.06), rnd(3, cfg.H, f, std=0.08))
    w.w_shared_gate = rnd(4, cfg.H, std=0.05) if gated else None
    layer = M.MoELayer(w, T, dev)
    assert not layer.fused
    out = layer.forward(t["x"])
    x = t["x"].double()
    g, u = x @ w.shared.gate.double().t(), x @ w.shared.up.double().t()
    y = (R.act("silu", g)[0] * u) @ w.shared.down.double().t()
    if gated:
        y = y * torch.sigmoid(x @ w.w_shared_gate.double())[:, None]
    ge, _ = G.host_expert_getter(cfg)
    routed = OL.layer(cfg, inp, ge, None)
    G.assert_close(G.to_np(out), routed.out + y.cpu().numpy(), f"layer T={T} gated={gated}")
    out = out.clone()
    # the same step in a graph, replayed over other tokens between eager steps
    x2 = torch.empty_like(t["x"])
    x2.copy_(t["x"])
    layer.forward(x2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = layer.forward(x2)
    eager = M.MoELayer(w, T, dev)
    for it in range(3):
        x2.copy_(rnd(60 + it, T, cfg.H) if it else t["x"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager.forward(x2))
        if it == 0:
            assert torch.equal(o, out)
        torch.cuda.synchronize()
