"""Block-128 FP8 operators and block norms on the host: constants, buffers, workspaces and plans at their edges."""
import ctypes

import pytest
import torch

B = pytest.importorskip("mxfp4_routed_expert_amd.binding", reason="libmoe.so not built (python mxfp4_routed_expert_amd/build.py)")
lib = B.lib


# ------------------------------------------------------------------ constants of the norms

@pytest.mark.parametrize("name", ["eps", "residual_scale", "dropout"])
def test_norm_constants_are_read_at_each_call(name):
    """A tensor (or parameter) may change between calls: its value counts, not the object."""
    for value in (torch.tensor(0.5), torch.nn.Parameter(torch.tensor(0.5)), torch.tensor([0.5], dtype=torch.float64)):
        kw = dict(eps=1e-6, residual_scale=1.0, dropout=0.0)
        kw[name] = value
        got = []
        for v in (0.5, 0.125):
            with torch.no_grad():
                value.fill_(v)
            got.append(getattr(B._norm_desc(4, 64, 0, 0, 0, **kw)[0]._obj, name))
        assert got == [0.5, 0.125]


def test_norm_constants_of_every_kind():
    d = B._norm_desc(4, 64, 0, 0, 0, 1e-6, -0.0, 0.0)[0]._obj
    assert str(d.residual_scale) == "0.0" and d.eps == ctypes.c_float(1e-6).value
    assert B._norm_desc(4, 64, 0, 0, 0, 1, True, 0)[0]._obj.residual_scale == 1.0
    for bad in ("0.5", None, torch.tensor([1.0, 2.0])):
        with pytest.raises((TypeError, ValueError)):
            B._norm_desc(4, 64, 0, 0, 0, 1e-6, bad, 0.0)


# ------------------------------------------------------------------ the experts' buffers

def _experts(fmt, E=2, H=256, I=128):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    if fmt == "fp8b128":
        s = lambda *n: torch.ones(n)
        return B.ExpertWeights(fmt, H, I, u8(E, I, H), s(E, 1, 2), u8(E, I, H), s(E, 1, 2), u8(E, H, I), s(E, 2, 1))
    return B.ExpertWeights(fmt, H, I, u8(E, I, H // 2), u8(E, I, H // 32), u8(E, I, H // 2), u8(E, I, H // 32), u8(E, H, I // 2), u8(E, H, I // 32))


class Reached(Exception):
    """A call got past its checks to the library."""


@pytest.fixture
def host(monkeypatch):
    """The binding with host tensors: all but the place of a tensor is checked, and the library is not called."""
    class Lib:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return lambda *a: 16
            raise Reached(name)
    need = B._need

    def anywhere(t, dtype, name, shape=None):
        try:
            need(t, dtype, name, shape)
        except ValueError as e:
            if "device memory" not in str(e):
                raise
            if dtype is not None and t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}")
    monkeypatch.setattr(B, "lib", Lib())
    monkeypatch.setattr(B, "_need", anywhere)


@pytest.mark.parametrize("act,fmt,codes,scales", [("fp8", "fp8b128", 128, 1), ("mxfp4", "mxfp4", 64, 4), ("float", "mxfp4", 64, 4)])
def test_experts_refuse_short_buffers(host, act, fmt, codes, scales):
    """Buffers of another mode, or a row short, are refused before a kernel could run past their end."""
    w, T, k = _experts(fmt), 3, 2
    R, H, I = T * k, w.d_model, w.d_ff
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    offs, sp = torch.zeros(3, dtype=torch.int32), torch.zeros(R, dtype=torch.int32)
    h, hq, hs, y = torch.zeros(R, I), u8(R, codes), u8(R, scales), torch.zeros(R, H)
    gateup = lambda h=h, hq=hq, hs=hs, offs=offs, sp=sp: B.moe_expert_gateup(w, x, act, k, offs, sp, out=(h, hq, hs))
    down = lambda h=h, hq=hq, hs=hs, offs=offs, y=y: B.moe_expert_down(w, T, act, k, offs, h, hq, hs, out=y)
    for call in (gateup, down):
        with pytest.raises(Reached):
            call()
        with pytest.raises(ValueError, match="expert_offsets"):
            call(offs=offs[:2])
        with pytest.raises(TypeError, match="expert_offsets"):
            call(offs=offs.long())
    if act == "float":
        for call in (gateup, down):
            with pytest.raises(ValueError, match="h has shape"):
                call(h=h[:R - 1])
    else:
        for call in (gateup, down):
            for short in (dict(hq=hq[:R - 1]), dict(hs=hs[:R - 1]), dict(hq=u8(R, codes // 2))):
                with pytest.raises(ValueError, match="h_codes has shape|h_scales has shape"):
                    call(**short)
            with pytest.raises(TypeError, match="h_codes"):
                call(hq=hq.float())
        with pytest.raises(Reached):
            gateup(h=None)
    with pytest.raises(ValueError, match="h has shape"):
        gateup(h=h[:R - 1])
    with pytest.raises(ValueError, match="sorted_pairs"):
        gateup(sp=sp[:R - 1])
    with pytest.raises(ValueError, match="y_rows"):
        down(y=y[:R - 1])
    with pytest.raises(TypeError, match="y_rows"):
        down(y=y.bfloat16())
    ffn = lambda sp=sp, ws=None: B.moe_expert_ffn(w, x, act, k, offs, sp, ws=ws)
    with pytest.raises(ValueError, match="sorted_pairs"):
        ffn(sp=sp[:R - 1])
    with pytest.raises(Reached):
        ffn()
    # buffers of more rows are taken, as before
    with pytest.raises(Reached):
        gateup(h=torch.zeros(R + 1, I), hq=u8(R + 1, codes), hs=u8(R + 1, scales))


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("query", ["moe_expert_gateup_workspace", "moe_expert_ffn_workspace"])
@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("E,H,I", [(1, 256, 128), (1, 128, 1024), (64, 1024, 512)])
def test_expert_workspaces_grow_with_tokens_and_k(query, act, E, H, I):
    """A workspace for T tokens and top k serves fewer of either (the identity form ignores k: any k's serves it)."""
    P = 0x10000
    w = B.ExpertWeightsC(1 if act == 2 else 0, E, H, I, P, P, P, P, P, P)
    f = lambda T, k: getattr(lib, query)(ctypes.byref(w), act, T, k)
    for k in (1, 2, 8):
        sizes = [f(T, k) for T in (1, 2, 4, 5, 15, 16, 17, 31, 32, 33, 64, 100, 1000)]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for T in (1, 3, 5, 16, 32, 33):
        sizes = [f(T, k) for k in (1, 2, 3, 8, 32)]
        assert sizes == sorted(sizes)


def test_identity_form_takes_a_workspace_of_any_k():
    P = ctypes.c_void_p(0x10000)
    w = B.ExpertWeightsC(1, 1, 128, 1024, *[P.value] * 6)
    T, k = 8, 8
    need = lib.moe_expert_gateup_workspace(ctypes.byref(w), 2, T, k)
    # (the alignment of x is checked first and the workspace last: neither reaches the device)
    call = lambda n: lib.moe_expert_gateup(ctypes.byref(w), 2, T, k, P, 0, None, None, None, P, P, P, n, None)
    assert need >= lib.moe_expert_gateup_workspace(ctypes.byref(w), 2, T, 1)
    assert call(lib.moe_expert_gateup_workspace(ctypes.byref(w), 2, T, 1) - 1) == B.MOE_ERR_WORKSPACE


# ------------------------------------------------------------------ the GPU tests' sizes

def test_tiles_cover_the_forms():
    """Every size of tile with whole and split sums, a second window of each kind of scale, and a second unit."""
    from test_gpu_fp8_edges import EVERY, TILES, linear_forms, plan
    seen = {}
    for T, n, k, want, kinds in TILES:
        for kind in kinds:
            got = linear_forms(T, n, k, kind)
            assert want <= got, (T, n, k, kind, plan(T, n, k), want - got)
            seen.setdefault(kind, set()).update(got)
    for kind in EVERY:
        for tt in (1, 2, 3, 4):
            assert {(tt, w) for w in ("one", "split", "window", "again")} <= seen[kind] | {(1, "split")}, (kind, tt, seen[kind])
