"""Dense layers without a GPU: refusals of the C entry points, workspace queries, and the float64
definitions that the GPU tests compare with (against torch's autograd and float8 type)."""
import ctypes
import math

import pytest
import torch

import dense_ref as R

B = pytest.importorskip("mxfp4_routed_expert_amd.binding",
                        reason="libmoe.so not built (python mxfp4_routed_expert_amd/build.py)")
lib = B.lib
P = ctypes.c_void_p(0x1000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)        # not 16-byte aligned
BIG = 1 << 40


def lin(**kw):
    d = dict(T=64, n=96, kdim=64, fn=0, x_dtype=0, y_dtype=0)
    d.update(kw)
    return ctypes.byref(B.LinearDesc(**d))


def gate(**kw):
    d = dict(T=64, d_model=64, d_ff=96, fn=1, x_dtype=0, h_dtype=0)
    d.update(kw)
    return ctypes.byref(B.GateupDesc(**d))


def refused(status, code, text):
    assert status == code, (status, B.last_error())
    assert text in B.last_error(), B.last_error()


@pytest.mark.parametrize("kw,text", [(dict(T=-1), "T=-1"), (dict(n=0), "n=0"), (dict(kdim=60), "kdim=60"), (dict(kdim=0), "kdim=0"),
                                     (dict(fn=9), "activation 9"), (dict(fn=-1), "activation -1"), (dict(x_dtype=2), "x_dtype 2"),
                                     (dict(y_dtype=5), "y_dtype 5"), (dict(T=1 << 20, n=1 << 12), "overflow"),
                                     (dict(T=1 << 24, kdim=1 << 10), "overflow"), (dict(n=1 << 20, kdim=1 << 12), "overflow"),
                                     (dict(n=2 ** 31 - 1, kdim=8), "overflow")])
def test_linear_rejects_bad_descriptor(kw, text):
    refused(lib.moe_dense_linear(lin(**kw), P, P, None, None, P, P, BIG, None), B.MOE_ERR_INVALID_ARG, text)
    assert lib.moe_dense_linear_workspace(lin(**kw)) == 0


def test_linear_rejects_pointers_and_workspaces():
    call = lambda x=P, w=P, b=None, r=None, y=P, ws=P, n=BIG, d=lin(): lib.moe_dense_linear(d, x, w, b, r, y, ws, n, None)
    refused(lib.moe_dense_linear(None, P, P, None, None, P, P, BIG, None), B.MOE_ERR_INVALID_ARG, "NULL descriptor")
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        refused(call(**kw), B.MOE_ERR_INVALID_ARG, "NULL")
    for kw in (dict(x=ODD), dict(w=ODD), dict(b=ODD), dict(r=ODD), dict(y=ODD)):
        refused(call(**kw), B.MOE_ERR_INVALID_ARG, "aligned")
    f32 = lin(x_dtype=1)
    need = lib.moe_dense_linear_workspace(f32)
    assert need >= 3 * 64 * 64 * 2                       # the three bf16 planes of float32 x
    refused(call(d=f32, n=need - 1), B.MOE_ERR_WORKSPACE, f"{need} bytes")
    refused(call(d=f32, ws=None), B.MOE_ERR_WORKSPACE, f"{need} bytes")
    refused(call(d=f32, ws=ODD, n=need), B.MOE_ERR_INVALID_ARG, "aligned")
    assert lib.moe_dense_linear_workspace(lin(T=8, x_dtype=1)) == 0          # few tokens need none
    assert call(d=lin(T=0), x=None, w=None, y=None, ws=None, n=0) == B.MOE_OK


def test_linear_backward_refusals():
    def call(dy=P, x=P, xs=None, w=P, b=None, dx=P, dw=P, db=P, ws=P, n=BIG, d=lin()):
        return lib.moe_dense_linear_backward(d, dy, x, xs, w, b, dx, dw, db, ws, n, None)
    bad = B.MOE_ERR_INVALID_ARG
    refused(call(dx=None, dw=None, db=None), bad, "no gradient")
    refused(call(d=lin(x_dtype=3)), bad, "x_dtype 3")
    refused(call(d=lin(dx_dtype=2)), bad, "dx_dtype 2")
    refused(call(d=lin(x_dtype=2, kdim=40), xs=P), bad, "kdim = 40")
    refused(call(d=lin(x_dtype=2)), bad, "x_scales")
    refused(call(dy=None), bad, "NULL")
    refused(call(x=None), bad, "NULL")
    refused(call(x=None, dw=None, d=lin(fn=2)), bad, "NULL")     # the activation needs x again
    refused(call(w=None), bad, "NULL")
    refused(call(dw=ODD), bad, "aligned")
    need = lib.moe_dense_linear_backward_workspace(lin(fn=2))
    assert need >= 64 * 96 * 2
    refused(call(d=lin(fn=2), n=need - 1), B.MOE_ERR_WORKSPACE, f"{need} bytes")


@pytest.mark.parametrize("kw,text", [(dict(T=-3), "T=-3"), (dict(d_model=12), "d_model=12"), (dict(d_ff=4), "d_ff=4"),
                                     (dict(d_ff=0), "d_ff=0"), (dict(fn=5), "activation 5"), (dict(x_dtype=1), "x_dtype 1"),
                                     (dict(h_dtype=2), "h_dtype 2"), (dict(T=1 << 20, d_ff=1 << 11), "overflow"),
                                     (dict(d_ff=2 ** 30 - 8, d_model=8), "overflow")])
def test_gateup_rejects_bad_descriptor(kw, text):
    refused(lib.moe_dense_gateup(gate(**kw), P, P, P, None, None, P, None, P, BIG, None), B.MOE_ERR_INVALID_ARG, text)
    assert lib.moe_dense_gateup_workspace(gate(**kw)) == 0


def test_gateup_refusals():
    for i in range(4):
        a = [P] * 4
        a[i] = None
        refused(lib.moe_dense_gateup(gate(), a[0], a[1], a[2], None, None, a[3], None, P, BIG, None), B.MOE_ERR_INVALID_ARG, "NULL")
    refused(lib.moe_dense_gateup(gate(), P, P, P, None, None, P, ODD, P, BIG, None), B.MOE_ERR_INVALID_ARG, "aligned")

    def call(dh=P, x=P, xs=None, wg=P, wu=P, pre=None, dx=P, dwg=P, dwu=P, dbg=P, dbu=P, h=P, ws=P, n=BIG, d=gate()):
        return lib.moe_dense_gateup_backward(d, dh, x, xs, wg, wu, None, None, pre, dx, dwg, dwu, dbg, dbu, h, ws, n, None)
    bad = B.MOE_ERR_INVALID_ARG
    refused(call(d=gate(dh_dtype=2)), bad, "dh_dtype 2")
    refused(call(dwg=None), bad, "together")
    refused(call(dbu=None), bad, "together")
    refused(call(dx=None, dwg=None, dwu=None, dbg=None, dbu=None, h=None), bad, "no result")
    refused(call(dh=None), bad, "NULL")
    refused(call(x=None), bad, "NULL")
    refused(call(x=None, pre=P), bad, "NULL")                    # the weight gradient still reads x
    refused(call(d=gate(x_dtype=2)), bad, "x_scales")
    refused(call(d=gate(x_dtype=2, d_model=40), xs=P), bad, "d_model = 40")
    refused(call(h=ODD), bad, "aligned")
    need = lib.moe_dense_gateup_backward_workspace(gate())
    assert need >= 64 * 2 * 96 * 2
    refused(call(n=need - 1), B.MOE_ERR_WORKSPACE, f"{need} bytes")
    refused(call(ws=None), B.MOE_ERR_WORKSPACE, f"{need} bytes")


def test_mxfp8_refusals():
    bad = B.MOE_ERR_INVALID_ARG
    refused(lib.moe_mxfp8_quantize(4, 40, P, 0, P, P, None), bad, "cols=40")
    refused(lib.moe_mxfp8_quantize(-1, 64, P, 0, P, P, None), bad, "rows=-1")
    refused(lib.moe_mxfp8_quantize(4, 64, P, 2, P, P, None), bad, "dtype 2")
    refused(lib.moe_mxfp8_quantize(1 << 20, 1 << 12, P, 0, P, P, None), bad, "overflow")
    refused(lib.moe_mxfp8_quantize(4, 64, None, 0, P, P, None), bad, "NULL")
    refused(lib.moe_mxfp8_quantize(4, 64, ODD, 0, P, P, None), bad, "aligned")
    refused(lib.moe_mxfp8_dequant(4, 64, P, None, P, 0, None), bad, "NULL")
    refused(lib.moe_mxfp8_dequant(4, 64, P, P, P, 7, None), bad, "dtype 7")
    assert lib.moe_mxfp8_quantize(0, 64, None, 0, None, None, None) == B.MOE_OK


def test_no_tokens_and_nothing_to_write():
    # an empty dx has no address: with no tokens that is no refusal
    e = (None,) * 3
    assert lib.moe_dense_linear_backward(lin(T=0, fn=1), None, None, None, None, None, None, None, None, P, BIG, None) == B.MOE_OK
    assert lib.moe_dense_gateup_backward(gate(T=0), None, None, None, None, None, None, None, None, *e, None, None, None, P, BIG,
                                         None) == B.MOE_OK


@pytest.mark.parametrize("T", [16, 64])
def test_kept_terms_count_in_the_size_limit(T):
    # up to 64 tokens dz, dg and du are kept as two terms and a float32 x as three, in one operand each
    fits, over = (2 ** 31 - 1) // (2 * T) - 15, 2 ** 31 // (2 * T)
    n = fits - fits % 8
    assert lib.moe_dense_linear_backward_workspace(lin(T=T, n=n, kdim=8, fn=1)) > 0
    refused(lib.moe_dense_linear_backward(lin(T=T, n=over, kdim=8, fn=1), P, P, None, P, None, P, P, P, P, BIG, None),
            B.MOE_ERR_INVALID_ARG, "overflow")
    k = 2 ** 31 // (3 * T) // 8 * 8 + 8
    refused(lib.moe_dense_linear(lin(T=T, n=1, kdim=k, x_dtype=1), P, P, None, None, P, P, BIG, None), B.MOE_ERR_INVALID_ARG, "overflow")
    f = 2 ** 31 // (4 * T)
    refused(lib.moe_dense_gateup_backward(gate(T=T, d_model=8, d_ff=f), P, P, None, P, P, None, None, None, P, P, P, P, P, P, P, BIG, None),
            B.MOE_ERR_INVALID_ARG, "overflow")


def test_workspaces_do_not_depend_on_a_gpu():
    # a pure function of the sizes: the same on every query, and finite for the largest call
    d = dict(T=4096, d_model=7168, d_ff=2368)
    a = [lib.moe_dense_gateup_backward_workspace(gate(**d, x_dtype=x)) for x in (0, 2, 0)]
    assert a[0] == a[2] and a[1] - a[0] == 4096 * 7168 * 2


def test_definitions_against_autograd():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    for fn, f in (("none", lambda z: z), ("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                  ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh")), ("relu", torch.relu)):
        x, wg, wu, bg, bu, dh = (t.requires_grad_() for t in (r(7, 24), r(10, 24), r(10, 24), r(10), r(10), r(7, 10)))
        h = f(x @ wg.t() + bg) * (x @ wu.t() + bu)
        want = torch.autograd.grad(h, (x, wg, wu, bg, bu), dh.detach())
        with torch.no_grad():
            got = R.gateup_backward(dh, x, wg, wu, bg, bu, fn)
            assert torch.allclose(R.gateup(x, wg, wu, bg, bu, fn, torch.float32)[0], h)
            for a, b in zip(want, got):
                assert torch.allclose(a, b[0], rtol=1e-10, atol=1e-10), fn
        y = f(x @ wg.t() + bg)
        want = torch.autograd.grad(y, (x, wg, bg), dh.detach())
        with torch.no_grad():
            for a, b in zip(want, R.linear_backward(dh, x, wg, bg, fn)):
                assert torch.allclose(a, b[0], rtol=1e-10, atol=1e-10), fn


def test_mxfp8_definition_against_float8():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(64, 96, generator=g) * torch.exp2(torch.randint(-20, 20, (64, 1), generator=g).float())).to(torch.bfloat16)
    codes, scales = R.mxfp8(x)
    v = x.float().view(64, 3, 32)
    e = torch.frexp(v.abs().amax(2))[1] - 9
    assert torch.equal(scales.int(), (e + 127).int())
    ref = torch.ldexp(v, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(codes.view(torch.float8_e4m3fn).float(), ref.float().view(64, 96))
    err = (R.mxfp8_values(codes, scales) - x.double()).abs()
    # half a step of the element's own binade (2^-4), the subnormal step at the bottom, and what saturation
    # cuts off: values up to 512 / 448 of the largest code
    lim = torch.maximum(x.double().abs() * 2 ** -4, torch.exp2(scales.double() - 127 - 10).repeat_interleave(32, 1))
    lim = torch.maximum(lim, (x.double().abs() - 448 * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)))
    assert (err <= lim).all()
    assert math.isnan(R.mxfp8_values(torch.zeros(1, 32, dtype=torch.uint8), torch.tensor([[255]], dtype=torch.uint8))[0, 0])


def test_binding_refuses_host_tensors():
    x, w, c = torch.zeros(4, 64).bfloat16(), torch.zeros(32, 64).bfloat16(), torch.zeros(4, 64, dtype=torch.uint8)
    h = torch.zeros(4, 32).bfloat16()
    for call in (lambda: B.moe_dense_linear(x, w), lambda: B.moe_dense_linear_backward(h, x, w), lambda: B.moe_dense_gateup(x, w, w),
                 lambda: B.moe_dense_gateup_backward(h, x, w, w), lambda: B.moe_mxfp8_quantize(x),
                 lambda: B.moe_mxfp8_dequant(c, c[:, :2].contiguous())):
        with pytest.raises(ValueError, match="device memory"):
            call()


class Plan(ctypes.Structure):
    """DensePlan of csrc/dense.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("cfg", "tr", "tc", "full", "split", "steps", "cs_rows")] + [("part_bytes", ctypes.c_size_t)]


FORWARD, INPUT_GRAD, WEIGHT_GRAD = range(3)


def plan(form, rows, cols, k, nseg=1, terms=1, pair=False):
    f = lib._ZN3moe10dense_planEibiiiii
    f.restype, f.argtypes = Plan, [ctypes.c_int, ctypes.c_bool] + [ctypes.c_int] * 5
    return f(form, pair, rows, cols, k, nseg, terms)


@pytest.mark.parametrize("nseg", [1, 2, 3])
def test_a_sum_of_no_tokens_has_a_step_in_every_segment(nseg):
    # the product kernel finds a step's segment by dividing by the steps of one
    for rows, cols in ((8, 8), (4096, 7168), (264, 136)):
        assert plan(WEIGHT_GRAD, rows, cols, 0, nseg).steps == nseg
        assert plan(WEIGHT_GRAD, rows, cols, 65, nseg).steps == 2 * nseg


def test_sizes_past_int32_are_refused(monkeypatch):
    # ctypes cuts an int off at 32 bits: 2^32 + 64 tokens would run as 64
    big, bf, u8 = 2 ** 32 + 64, torch.bfloat16, torch.uint8
    e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device="meta")
    monkeypatch.setattr(B, "_operands", lambda *a: None)
    monkeypatch.setattr(B, "_launch", lambda *a: pytest.fail("launched with sizes past int32"))
    w = e(64, 64)
    for call in (lambda: B.moe_dense_linear_workspace(big, 64, 64, x_dtype=torch.float32), lambda: B.moe_dense_linear_workspace(64, 64, big),
                 lambda: B.moe_dense_linear_backward_workspace(64, big, 64), lambda: B.moe_dense_gateup_workspace(big, 64, 64),
                 lambda: B.moe_dense_gateup_backward_workspace(64, 64, big),
                 lambda: B.moe_dense_linear(e(big, 64), w), lambda: B.moe_dense_linear_backward(e(big, 64), e(big, 64), w),
                 lambda: B.moe_dense_gateup(e(64, big), e(64, big), e(64, big)),
                 lambda: B.moe_dense_gateup_backward(e(big, 64), e(big, 64), w, w),
                 lambda: B.moe_mxfp8_quantize(e(big, 64)), lambda: B.moe_mxfp8_quantize(e(64, big)),
                 lambda: B.moe_mxfp8_dequant(e(big, 64, dt=u8), e(big, 2, dt=u8))):
        with pytest.raises(B.MoeError, match="int32"):
            call()


def _forms(T, *sizes, gated=False, act=True, f32=False):
    """(product, tile shape, how its sum is split) of a forward and a backward call, as csrc/dense.hip asks for them."""
    def form(name, p):
        tiles = p.tr * p.tc
        return name, "LMSDWB"[p.cfg], "whole" if p.full == tiles else ("all tiles" if p.full == 0 else "tail")
    few = T <= 64
    if gated:
        f, d = sizes
        t = 2 if few else 1
        return [form("gated", plan(FORWARD, T, f, d, pair=True)), form("gated dx", plan(INPUT_GRAD, T * t, d, f, 2, t)),
                form("gated dw", plan(WEIGHT_GRAD, 2 * f, d, T, t))]
    n, k = sizes
    xs = 3 if f32 else 1                 # float32 rows: three terms, as rows or as segments
    z = form("linear", plan(FORWARD, T * (xs if few else 1), n, k, 1 if few else xs, xs if few else 1))
    t = 2 if act and few else 1          # terms of dz
    return [z, form("linear dx", plan(INPUT_GRAD, T * t, k, n, 1, t)), form("linear dw", plan(WEIGHT_GRAD, n, k, T, (2 if f32 else 1) + t - 1))]


def test_gpu_tests_reach_every_tile_shape_and_split():
    import test_gpu_dense as G
    import test_gpu_dense_edges as E
    got = set()
    for T, n, k in G.TILES:
        got.update(_forms(T, n - 3, k)[:1] + _forms(T, n, k))
    for T, k, n in G.TILES[1:]:
        got.update(_forms(T, n - 1, k, act=False)[1:])
    for T, n, k in G.GRAD_TILES:
        got.update(_forms(T, n, k, act=False)[1:])
    for T, n, k, xt in E.MORE_LINEAR:
        got.update(_forms(T, n, k, f32=xt == torch.float32))
    for T, f, d in G.PAIR_TILES + [(T, f, d) for T, d, f in G.TWO_PART_TILES] + E.MORE_GATED:
        got.update(_forms(T, f, d, gated=True))
    # forward products and input gradients take every shape but W, weight gradients L, B, M and W; the first two split no M
    # tail tiles alone (none of 60000 drawn sizes did)
    want = set()
    for name in ("linear", "gated"):
        for suffix, tiles in (("", "LBDMS"), (" dx", "LBDMS"), (" dw", "LBMW")):
            want.update((name + suffix, t, s) for t in tiles for s in ("whole", "tail", "all tiles")
                        if not (t == "M" and s == "tail" and suffix != " dw"))
    assert want <= got, sorted(want - got)


def test_operands_that_require_grad_are_warned_of(monkeypatch):
    import warnings
    monkeypatch.setattr(B, "_operands", lambda *a: None)
    monkeypatch.setattr(B, "_launch", lambda *a: None)
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")
    linear = lambda x, w, b, r: B.moe_dense_linear(x, w, b, "silu", r)
    gated = lambda x, w, b, r: B.moe_dense_gateup(x, w, w, b, b)
    for call, who, n in ((linear, "moe_dense_linear_backward", 4), (gated, "moe_dense_gateup_backward", 3)):
        for i in range(n):
            t = [e(9, 64), e(32, 64), e(32, dt=torch.float32), e(9, 32)]
            with warnings.catch_warnings():
                warnings.simplefilter("error")
                call(*t)
                t[i].requires_grad_()
                with torch.no_grad():
                    call(*t)
            with pytest.warns(UserWarning, match=who):
                call(*t)


def test_size_limit_counts_terms_only_where_they_are_kept():
    # without an activation dz is dy itself, one term, and x enters dw as segments; up to 8 tokens a forward pass multiplies float32
    T, n, k = 64, (2 ** 31 - 1) // 64 // 8 * 8 - 16, (2 ** 31 - 1) // 64 // 8 * 8
    assert lib.moe_dense_linear_backward_workspace(lin(T=T, n=n, kdim=8)) > 0
    assert lib.moe_dense_linear_backward_workspace(lin(T=T, n=8, kdim=k, x_dtype=1)) > 0
    few = lin(T=8, n=1, kdim=(2 ** 31 - 1) // 8 // 8 * 8, x_dtype=1)
    refused(lib.moe_dense_linear(few, P, P, None, None, ODD, None, 0, None), B.MOE_ERR_INVALID_ARG, "aligned")
    for kw in (dict(T=T, n=n, kdim=8, fn=1), dict(T=T, n=8, kdim=k, x_dtype=1, fn=1)):
        assert lib.moe_dense_linear_backward_workspace(lin(**kw)) == 0
        assert "overflow" in B.last_error()
    assert lib.moe_dense_linear_workspace(lin(T=T, n=8, kdim=k, x_dtype=1)) == 0 and "overflow" in B.last_error()
