"""Block-128 FP8 operators at their edges (GPU): what autograd sees, workspaces, tiles of every size, windows of scales."""
from __future__ import annotations

import ctypes
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


# ------------------------------------------------------------------ tiles of every size

class Plan(ctypes.Structure):
    _fields_ = [("bt", ctypes.c_int), ("split", ctypes.c_int)]


def plan(T, n, k, kind=0):
    """(rows of a tile, 0 where the weights are streamed; parts of the sum) of moe_fp8_linear."""
    import mxfp4_routed_expert_amd.binding as B
    f = B.lib._ZN3moe15fp8_linear_planEPK19moe_fp8_linear_desc
    f.restype = Plan
    p = f(ctypes.byref(B.Fp8LinearDesc(T, n, k, B.DT_FP8, 0, kind)))
    return p.bt, p.split


def forms(tiles, NT, bt, split, Kb, window, cus=256, order=None):
    """What the tile kernel runs: a set of (16 x 16 tiles a wave has along the rows (1 to 4: up to 64, 128, 192, 256 rows), what
    happens there): "one" or "split" sum, "window": scales of a second window of blocks within the sum, "again": not a workgroup's
    first unit.  tiles: rows of each tile of bt.  order: the rows item by item (experts), else as one matrix goes."""
    items = len(order) if order else len(tiles) * NT * split
    G = min(cus, 4 * items)
    full = items // G * G
    tail, most = items - full, bt // 64
    f = min(4, most) if 0 < 4 * tail <= G else min(2, most) if 0 < 2 * tail <= G else 1
    got = set()

    def unit(item, part, parts, again):
        s = 0
        if order:
            rows = order[item]
        else:
            s, r = divmod(item, NT * len(tiles))
            g, i = divmod(r, 4 * len(tiles))
            rows = tiles[i // min(4, NT - 4 * g)]
        live = min(rows - part * (bt // parts), bt // parts)
        if live <= 0:
            return
        tt = (live + 63) // 64
        a, b = Kb * s // split, Kb * (s + 1) // split
        got.add((tt, "split" if split > 1 else "one"))
        if any(a < w < b for w in range(window, Kb, window)):
            got.add((tt, "window"))
        if again:
            got.add((tt, "again"))
    for it in range(full):
        unit(it, 0, 1, it >= G)
    for u in range(f * tail):
        unit(full + u // f, u % f, f, full > 0)
    return got


def linear_forms(T, n, k, kind, cus=256):
    bt, split = plan(T, n, k)
    if bt == 0:
        return set()
    return forms([min(bt, T - t) for t in range(0, T, bt)], (n + 255) // 256, bt, split, (k + 127) // 128, 32 if kind == "row" else 64, cus)


# (T, n, k, forms that are to be among those that run; kinds of weight scales)
EVERY = ("f32", "e8m0", "row")
TILES = [
    (1029, 2056, 6160, {(2, "split")}, EVERY),                                         # 128 rows, 3 parts
    (1021, 6146, 528, {(2, "one")}, EVERY),
    (591, 22710, 144, {(1, "again"), (2, "again"), (3, "one")}, EVERY),                # 192 rows; a second unit, cut in thirds
    (553, 33461, 144, {(3, "again")}, EVERY),                                          # 192 rows, tile and tail
    (7168, 2368, 272, {(3, "one"), (2, "again")}, ("f32", "row")),
    (603, 39878, 144, {(2, "again"), (4, "again")}, EVERY),                            # 256 rows
    (412, 16661, 992, {(3, "one"), (4, "one")}, ("f32", "e8m0")),
    (75, 109, 4304, {(1, "split"), (1, "window")}, ("row",)),                          # windows: 32 blocks of a row's scales, 64 of a block's
    (68, 108, 8592, {(1, "split"), (1, "window")}, ("f32", "e8m0")),
    (66, 5338, 7872, {(2, "split"), (2, "window")}, ("row",)),
    (1606, 259, 8944, {(2, "split"), (2, "window")}, EVERY),
    (140, 11589, 5776, {(3, "split"), (3, "window")}, ("row",)),
    (146, 7678, 8896, {(3, "split"), (3, "window")}, EVERY),
    (457, 8358, 10080, {(4, "split"), (4, "window")}, EVERY),
    (1541, 7492, 4240, {(4, "one"), (4, "window")}, ("row",)),
    (589, 6507, 8480, {(2, "one"), (2, "window")}, ("f32",)),
]


def e4m3():
    return torch.arange(256, dtype=U8).view(torch.float8_e4m3fn).double().to(DEV)


def device_codes(n, k, seed, lead=()):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randint(0, 256, (*lead, n, k), generator=g, dtype=torch.uint8, device=DEV)
    return torch.where((c & 127) == 127, torch.zeros_like(c), c)


def values(c, s, rows):
    """float64 values of codes [r][c] with one scale (float32 or E8M0) per rows x 128 block."""
    s = s.double() if s.dtype is F32 else torch.exp2(s.double() - 127)
    return e4m3()[c.long()] * s.repeat_interleave(rows, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]]


def sum_tol(x, w):
    """test_gpu_fp8.sum_tol, on the device."""
    top = lambda v: torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8)).reshape(v.shape[0], -1, 8).amax(2)
    return 7 * 2.0 ** -13 * (top(x) @ top(w).T) + (x.shape[1] / 8 + 8) * 2.0 ** -23 * (x.abs() @ w.abs().T)


def check(y, ref, tol, res, what):
    """test_gpu_fp8.check_product's tolerance, every value of y."""
    if res is not None:
        ref = ref + res.double()
        tol = tol + 2.0 ** -24 * (ref.abs() + res.double().abs())
    if y.dtype is BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    over = (y.double() - ref).abs() > tol + 1e-30
    assert not over.any(), f"{what}: {int(over.sum())} values, first {over.nonzero()[0].tolist()}"


@pytest.mark.parametrize("T,n,k,want,kind", [(*c[:4], kind) for c in TILES for kind in c[4]],
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-{kind}" for c in TILES for kind in c[4]])
def test_tiles(M, T, n, k, want, kind):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert want <= linear_forms(T, n, k, kind, cus)
    x = hidden(T, k, T + n)
    c, s, _, _ = M.moe_fp8_quantize(x.to(DEV))
    w = device_codes(n, k, n + k)
    ws = scales_of(kind, n, k, n).to(DEV)
    xv, wv = values(c, s, 1), values(w, ws, 1 if kind == "row" else 128)
    ref, tol = xv @ wv.T, sum_tol(xv, wv)
    del wv
    res = torch.randn(T, n, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV) * float(ref.abs().mean())
    for dt in (BF, F32):
        y = M.moe_fp8_linear(c, w, ws, x_scales=s, out_dtype=dt)
        check(y, ref, tol, None, f"{kind} {dt}")
        # results in a buffer with a guard around them, added to what is there
        buf = torch.full((64 + T * n + 64,), 7.0, dtype=dt, device=DEV)
        acc = buf[64:64 + T * n].view(T, n)
        acc.copy_(res)
        r = acc.clone()
        M.moe_fp8_linear(c, w, ws, x_scales=s, residual=acc, out=acc)
        assert (buf[:64] == 7).all() and (buf[64 + T * n:] == 7).all()
        check(acc, ref, tol, r, f"{kind} {dt} with residual")
        assert torch.equal(M.moe_fp8_linear(c, w, ws, x_scales=s, out_dtype=dt), y), "the same bits again"


@pytest.mark.parametrize("T,n,k", [(1021, 2048, 6144), (2045, 7168, 2368)])
def test_layer_gradients_in_tiles(M, T, n, k):
    """A training step's three products, each in tiles above 64 rows, five column tiles and more."""
    for a in ((T, n, k), (T, k, n), (n, k, (T + 15) // 16 * 16)):
        assert plan(*a)[0] > 64
    w, x, dy = (hidden(n, k, 1) * 0.1).to(DEV), hidden(T, k, 2).to(DEV), hidden(T, n, 3).to(DEV)
    layer = M.FP8Linear(w, T, dw_dtype=F32)
    y = layer.forward(x)
    wc, wsc, wct, wst = layer.w_q
    xq, dyq = M.moe_fp8_quantize(x, cols=True), M.moe_fp8_quantize(dy, cols=True)
    wv = values(wc, wsc, 128)
    a = values(*xq[:2], 1)
    check(y, a @ wv.T, sum_tol(a, wv), None, "y")
    dx, dw = layer.backward(dy)
    g, wt = values(*dyq[:2], 1), values(wct, wst, 128)
    assert torch.equal(wt, wv.T)
    check(dx, g @ wv, sum_tol(g, wt), None, "dx")
    gt, xt = values(*dyq[2:], 1), values(*xq[2:], 1)
    check(dw, gt @ xt.T, sum_tol(gt, xt), None, "dw")


@pytest.mark.parametrize("T,n,k,tt", [(4500, 2048, 1040, 1), (8300, 1024, 1040, 2), (4500, 2304, 5120, 3), (4500, 4096, 4096, 4)])
def test_weight_gradient_of_many_tokens(M, T, n, k, tt):
    """More than 4096 tokens: a second window of scales along the sum, whole and in parts, in tiles of 64 to 256 rows."""
    assert (tt, "window") in linear_forms(n, k, (T + 15) // 16 * 16, "row", torch.cuda.get_device_properties(0).multi_processor_count)
    x, dy = hidden(T, k, 5).to(DEV), hidden(T, n, 6).to(DEV)
    layer = M.FP8Linear((hidden(n, k, 7) * 0.1).to(DEV), T)
    layer.forward(x)
    dw = layer.backward(dy)[1]
    gt, xt = values(*M.moe_fp8_quantize(dy, rows=False, cols=True)[2:], 1), values(*M.moe_fp8_quantize(x, rows=False, cols=True)[2:], 1)
    check(dw, gt @ xt.T, sum_tol(gt, xt), None, "dw")


# ------------------------------------------------------------------ experts in tiles of every size

def device_experts(M, E, H, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    m, s = {}, {}
    for i, (name, n, k) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
        m[name] = device_codes(n, k, seed + 7 * i, (E,))
        s[name] = (torch.rand(E, n // 128, k // 128, generator=g, device=DEV) + 0.5) * (0.01 * k ** -0.5)
    w = M.ExpertWeights("fp8b128", H, I, m["gate"], s["gate"], m["up"], s["up"], m["down"], s["down"])
    return w, lambda name, e: values(m[name][e], s[name][e], 128)


def check_expert_rows(M, w, value, x, k, offs, sp, o):
    """h, its codes and y of every row against 64 bits; o: the offsets on the host (one expert: [0, T])."""
    T = x.shape[0]
    h, hq, hs = M.moe_expert_gateup(w, x, "fp8", k, offs, sp)
    y = M.moe_expert_down(w, T, "fp8", k, offs, None, hq, hs)
    xv = values(*M.moe_fp8_quantize(x)[:2], 1)
    hv = values(hq, hs, 1)
    for e in range(len(o) - 1):
        if o[e] == o[e + 1]:
            continue
        r = slice(o[e], o[e + 1])
        a = xv if sp is None else xv[sp[r].long() // k]
        wg, wu = value("gate", e), value("up", e)
        g, u, eg, eu = a @ wg.T, a @ wu.T, sum_tol(a, wg), sum_tol(a, wu)
        ref = g / (1 + torch.exp(-g)) * u
        # |silu'| <= 1.1, |silu(g)| <= |g|; exp2, reciprocal and three products: 8 roundings
        tol = 1.1 * eg * u.abs() + g.abs() * eu + eg * eu + 2.0 ** -20 * ref.abs()
        assert ((h[r].double() - ref).abs() <= tol + 1e-30).all(), f"h of expert {e}"
        wd = value("down", e)
        check(y[r], hv[r] @ wd.T, sum_tol(hv[r], wd), None, f"y of expert {e}")
    live = slice(0, o[-1])
    c, s, _, _ = M.moe_fp8_quantize(h)
    assert torch.equal(c[live], hq[live]) and torch.equal(s[live], hs[live])
    assert torch.equal(M.moe_expert_ffn(w, x, "fp8", k, offs, sp)[live], y[live])


def expert_forms(counts, N, pair, Kb):
    cols = 128 if pair else 256
    order = [min(256, c - t) for c in counts for _ in range((N + cols - 1) // cols) for t in range(0, c, 256)]
    return forms(None, None, 256, 1, Kb, 64, torch.cuda.get_device_properties(0).multi_processor_count, order)


# rows of an expert, in turn
COUNTS = [256, 250, 193, 192, 130, 128, 65, 64, 1, 0, 300, 449, 17, 201, 100, 129]


@pytest.mark.parametrize("E,H,I,want_pair,want_down", [
    (32, 1280, 640, {(1, "one"), (2, "one"), (3, "one"), (4, "one")}, {(1, "one"), (2, "one"), (3, "one"), (4, "one")}),
    (64, 1280, 768, {(4, "one"), (3, "one"), (1, "again")}, {(4, "one"), (1, "again")}),
    (16, 8320, 1280, {(4, "window"), (3, "window"), (2, "window"), (1, "window")}, {(4, "again"), (2, "again")}),
    (16, 2560, 8320, {(4, "again"), (3, "again"), (2, "again")}, {(4, "window"), (3, "window"), (2, "window"), (1, "window")})])
def test_experts_in_tiles(M, E, H, I, want_pair, want_down):
    k = 2
    counts = [COUNTS[(e + e // 16) % 16] for e in range(E)]
    if sum(counts) % k:
        counts[0] -= 1
    # the pairs' experts in an order in which no token has one twice
    flat = torch.tensor([e for e in range(E) for _ in range(counts[e])], dtype=torch.int32)
    T = len(flat) // k
    ids = torch.stack([flat[:T], flat[T:]], 1)
    assert (ids[:, 0] != ids[:, 1]).all()
    assert want_pair <= expert_forms(counts, I, True, H // 128), expert_forms(counts, I, True, H // 128)
    assert want_down <= expert_forms(counts, H, False, I // 128), expert_forms(counts, H, False, I // 128)
    w, value = device_experts(M, E, H, I, 3)
    offs, sp, _ = M.moe_permute(ids[torch.randperm(T, generator=torch.Generator().manual_seed(1))].contiguous().to(DEV), E)
    o = offs.tolist()
    assert [b - a for a, b in zip(o, o[1:])] == counts
    check_expert_rows(M, w, value, hidden(T, H, 9).to(DEV), k, offs, sp, o)


@pytest.mark.parametrize("T,H,I,want", [(1930, 256, 2560, {(3, "one"), (4, "one")}), (100, 256, 16640, {(2, "one")}), (200, 128, 33280, {(4, "one"), (1, "again")})])
def test_shared_expert_in_tiles(M, T, H, I, want):
    """gate and up of one matrix (the identity form) above 64 rows."""
    bt = 256 if T > 128 else 128
    assert want <= forms([min(bt, T - t) for t in range(0, T, bt)], I // 128, bt, 1, H // 128, 64, torch.cuda.get_device_properties(0).multi_processor_count)
    w, value = device_experts(M, 1, H, I, 5)
    check_expert_rows(M, w, value, hidden(T, H, 10).to(DEV), 1, None, None, [0, T])


# ------------------------------------------------------------------ a layer's step in a graph

@pytest.mark.parametrize("T", [1, 4, 70, 300])
def test_captured_layer_with_fp8_activations(M, T):
    """MoELayer(act="fp8") and the norms around it in one graph, with eager steps of the same layer in between."""
    E, k, H, I = 8, 2, 256, 128
    w, _ = device_experts(M, E, H, I, 5)
    sh, _ = device_experts(M, 1, H, 256, 6)
    g = torch.Generator().manual_seed(9)
    wr, wsg = (torch.randn(E, H, generator=g) * 0.1).to(BF).to(DEV), (torch.randn(H, generator=g) * 0.1).to(BF).to(DEV)
    wb, wa = torch.rand(H, generator=g).to(DEV) + 0.5, torch.rand(H, generator=g).to(DEV) + 0.5
    layer = M.MoELayer(M.LayerWeights("sigmoid", k, True, 1.0, "fp8", wr, w, shared=sh, w_shared_gate=wsg), T, DEV)
    res = hidden(T, H, 10).to(DEV)

    def step():
        u = M.moe_block_norm(res, w_before=wb, want_y=False)[1]
        return M.moe_block_norm(layer.forward(u), w_after=wa, residual=res, w_before=wb, want_codes=True)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        res.copy_(hidden(T, H, 20 + i))
        graph.replay()
        got = [t.clone() for t in (*out, layer.ids, layer.out)]
        torch.cuda.synchronize()
        for a, b in zip(got, (*step(), layer.ids, layer.out)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ the largest sizes

def test_largest_rows(M):
    """Just under 2^31 values: both quantised forms, their values, and a product, at the last rows as those rows by themselves."""
    T, d, at = 131071, 16368, 130944                           # (the last block of 128 rows is a row short)
    x = torch.randn(T, d, dtype=BF, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    end = x[at:].clone()
    c, s, ct, st = M.moe_fp8_quantize(x, cols=True)
    rc, rs, rct, rst = M.moe_fp8_quantize(end, cols=True)
    assert torch.equal(c[at:], rc) and torch.equal(s[at:], rs) and torch.equal(ct[:, at:], rct) and torch.equal(st[:, -1:], rst)
    del ct, st
    c2, s2, _, _ = M.moe_fp8_quantize(x)
    assert torch.equal(c2, c) and torch.equal(s2, s)
    del c2, s2
    v = M.moe_fp8_dequant(c, s)
    assert torch.equal(v[at:], M.moe_fp8_dequant(rc, rs))
    del v
    n = 272
    w, ws = device_codes(n, d, 2), scales_of("f32", n, d, 3).to(DEV)
    xv, wv = values(rc, rs, 1), values(w, ws, 128)
    ref, tol = xv @ wv.T, sum_tol(xv, wv)
    check(M.moe_fp8_linear(c, w, ws, x_scales=s)[at:], ref, tol, None, "codes")
    check(M.moe_fp8_linear(x, w, ws, out_dtype=F32)[at:], ref, tol, None, "values")


@pytest.mark.parametrize("kind", EVERY)
def test_largest_weight(M, kind):
    """Just under 2^31 codes: streamed and in tiles, the last columns."""
    n, k, at = 131071, 16368, 130816
    w = device_codes(n, k, 4)
    ws = scales_of(kind, n, k, 5).to(DEV)
    for T in (3, 70):
        assert (plan(T, n, k)[0] > 0) == (T == 70)
        c, s, _, _ = M.moe_fp8_quantize(hidden(T, k, T).to(DEV))
        xv, wv = values(c, s, 1), values(w[at:], ws[at:] if kind == "row" else ws[at // 128:], 1 if kind == "row" else 128)
        y = M.moe_fp8_linear(c, w, ws, x_scales=s, out_dtype=F32)
        check(y[:, at:], xv @ wv.T, sum_tol(xv, wv), None, f"{T} rows")


def test_largest_weight_quantised(M):
    n, k, at = 131071, 16368, 130944
    w = torch.randn(n, k, dtype=BF, device=DEV, generator=torch.Generator(device=DEV).manual_seed(6))
    c, s, ct, st = M.moe_fp8_quantize_weight(w, U8, transpose=True)
    rc, rs, rct, rst = M.moe_fp8_quantize_weight(w[at:].clone(), U8, transpose=True)
    assert torch.equal(c[at:], rc) and torch.equal(s[-1:], rs) and torch.equal(ct[:, at:], rct) and torch.equal(st[:, -1:], rst)


@pytest.mark.parametrize("dt", [BF, F32])
def test_largest_result(M, dt):
    T, n, k, at = 32767, 65528, 16, 32700
    x, w, ws = hidden(T, k, 7).to(DEV), device_codes(n, k, 8), scales_of("f32", n, k, 9).to(DEV)
    c, s, _, _ = M.moe_fp8_quantize(x)
    xv, wv = values(c[at:], s[at:], 1), values(w, ws, 128)
    y = torch.ones(T, n, dtype=dt, device=DEV)
    M.moe_fp8_linear(c, w, ws, x_scales=s, residual=y, out=y)
    check(y[at:], xv @ wv.T, sum_tol(xv, wv), torch.ones(T - at, n, dtype=dt, device=DEV), "y")


def test_most_rows(M):
    """Rows of 8 values, as many as 2^31 values allow: the grid has nearly 2^32 threads."""
    T, at = 2 ** 28 - 16, 2 ** 28 - 80
    x = torch.randn(T, 8, dtype=BF, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    c, s, _, _ = M.moe_fp8_quantize(x)
    rc, rs, _, _ = M.moe_fp8_quantize(x[at:].clone())
    assert torch.equal(c[at:], rc) and torch.equal(s[at:], rs)
    mid = slice(2 ** 27 - 64, 2 ** 27 + 64)
    assert torch.equal(c[mid], M.moe_fp8_quantize(x[mid].clone())[0])
    assert torch.equal(M.moe_fp8_dequant(c, s)[at:], M.moe_fp8_dequant(rc, rs))
    with pytest.raises(M.MoeError, match="65535 blocks"):
        M.moe_fp8_quantize(x[:65535 * 128 + 1], cols=True)
    w = torch.ones(8, device=DEV)
    y = M.moe_block_norm(x, w_after=w)[0]
    assert torch.equal(y[at:], M.moe_block_norm(x[at:].clone(), w_after=w)[0])
    dz = M.moe_block_norm_backward(x, w_after=w, dy=y, want=("dz",))[0]
    assert torch.equal(dz[at:], M.moe_block_norm_backward(x[at:].clone(), w_after=w, dy=y[at:].clone(), want=("dz",))[0])


# ------------------------------------------------------------------ two calls at once

@pytest.mark.parametrize("T", [3, 40, 300])
def test_experts_and_norm_gradients_on_two_streams(M, T):
    """The same weights on two streams, a workspace and results for each: the bits of either alone."""
    E, k, H, I = 8, 2, 1280, 256
    w, _ = device_experts(M, E, H, I, 11)
    wa = torch.rand(H, device=DEV) + 0.5
    sides = []
    for i in range(2):
        x = hidden(T, H, 30 + i).to(DEV)
        ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(40 * i + t))[:k] for t in range(T)]).to(torch.int32).to(DEV)
        offs, sp, _ = M.moe_permute(ids, E)
        y, ws = torch.empty(T * k, H, device=DEV), torch.empty(M.binding.moe_expert_ffn_workspace(w, "fp8", T, k), dtype=U8, device=DEV)
        out = (torch.empty_like(x), torch.empty_like(x), torch.empty(H, device=DEV), None, None)
        ws2 = torch.empty(M.binding.moe_block_norm_backward_workspace(T, H), dtype=U8, device=DEV)

        def run(x=x, offs=offs, sp=sp, y=y, ws=ws, out=out, ws2=ws2):
            M.moe_expert_ffn(w, x, "fp8", k, offs, sp, out=y, ws=ws)
            M.moe_block_norm_backward(x, w_after=wa, dy=x, want=("dz", "dresidual", "dw_after"), out=out, ws=ws2)
            return y, *out[:3]
        sides.append((run, [t.clone() for t in run()], (y, *out[:3])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, (run, _, _) in zip(streams, sides):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for _, ref, got in sides:
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("E,T", [(8, 3), (256, 60), (8, 40), (4, 700)])
def test_non_finite_values_stay_in_their_rows(M, E, T):
    """Few rows, streamed experts, tiles of 64 and of more rows: a NaN or infinite x spoils its token's rows, a NaN code of gate its column of its expert's
    h (and so those rows of y), one of down its column of y; every other value keeps its bits."""
    k, H, I = 1, 512, 4480 if T == 700 else 256
    w, _ = device_experts(M, E, H, I, 13)
    x = hidden(T, H, 14).to(DEV)
    ids = (torch.arange(T, dtype=torch.int32)[:, None] % E).to(DEV)
    offs, sp, p2r = M.moe_permute(ids, E)
    run = lambda x: (*M.moe_expert_gateup(w, x, "fp8", k, offs, sp), M.moe_expert_ffn(w, x, "fp8", k, offs, sp))
    if T == 700:
        assert (3, "one") in expert_forms([175] * 4, I, True, H // 128)
    clean = run(x)
    assert all(torch.isfinite(t).all() for t in (clean[0], clean[3]))
    row, e = p2r.view(-1).long(), sp.long() % E                # (a token's row; a row's expert)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[1, 130] = bad
        h, hq, hs, y = run(z)
        hit = torch.zeros(T, dtype=torch.bool, device=DEV)
        hit[row[1]] = True
        assert torch.isnan(h[hit]).all() and ((hq[hit] & 127) == 127).all() and torch.isnan(y[hit]).all()
        for a, b in zip((h, hq, hs, y), clean):
            assert torch.equal(a[~hit], b[~hit])
    hit = e == 2
    w.gate[2, 100, 7] = 0x7F
    h, hq, hs, y = run(x)
    col = torch.arange(I, device=DEV) == 100
    assert torch.isnan(h[hit][:, col]).all() and torch.isnan(y[hit]).all() and torch.equal(h[hit][:, ~col], clean[0][hit][:, ~col])
    for a, b in zip((h, hq, hs, y), clean):
        assert torch.equal(a[~hit], b[~hit])
    w.gate[2, 100, 7] = 0
    base = run(x)
    w.down[2, 300, 9] = 0x7F
    y = run(x)[3]
    col = torch.arange(H, device=DEV) == 300
    assert torch.isnan(y[hit][:, col]).all() and torch.equal(y[hit][:, ~col], base[3][hit][:, ~col]) and torch.equal(y[~hit], base[3][~hit])
