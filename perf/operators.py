"""Workloads of the dense feed-forward operators: the linear layer with its epilogue, the gated
projections, their backward passes, and the 8-bit checkpoint of a block's input.

Widths are those of this repository's layers (hidden 7168 with d_ff 2368 and latent 2048; hidden
6144 with d_ff 2048) and generic ones; token counts run from one decoded token to a training
batch of a few thousand.
"""
import math

import torch

own = False


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through a latent down projection (bf16 in, float32 out)
        dict(name="linear_decode_1", op="linear", T=1, n=2048, k=7168, act="none", bias=False, residual=False,
             xt="bf16", yt="f32"),
        # four decoded tokens through the latent up projection: float32 rows, float32 residual
        dict(name="linear_decode_4_f32", op="linear", T=4, n=7168, k=2048, act="none", bias=False, residual=True,
             xt="f32", yt="f32"),
        # a prompt's chunk through a down projection with its residual
        dict(name="linear_prefill_512", op="linear", T=512, n=7168, k=2368, act="none", bias=False, residual=True,
             xt="bf16", yt="bf16"),
        # a ragged training batch through a biased GELU layer
        dict(name="linear_gelu_4093", op="linear", T=4093, n=7168, k=2048, act="gelu", bias=True, residual=False,
             xt="bf16", yt="bf16"),
        # the gradients of a biased GELU layer on a short ragged batch (activation recomputed)
        dict(name="linear_bwd_gelu_333", op="linear_bwd", T=333, n=2368, k=7168, act="gelu", bias=True, ckpt=False),
        # the gradients of a down projection in a training step
        dict(name="linear_bwd_2048", op="linear_bwd", T=2048, n=7168, k=2368, act="none", bias=False, ckpt=False),
        # one decoded token through a shared expert's gate and up projections
        dict(name="gateup_decode_1", op="gateup", T=1, d=7168, f=2368, act="silu", bias=False, ht="f32"),
        # a prompt's chunk through them
        dict(name="gateup_prefill_512", op="gateup", T=512, d=7168, f=2368, act="silu", bias=False, ht="bf16"),
        # a short odd batch with saved pre-activations and biases, the GELU form
        dict(name="gateup_bwd_saved_61", op="gateup_bwd", T=61, d=6144, f=2048, act="gelu_tanh", bias=True, ckpt=False,
             saved=True),
        # the training step of the gated projections whose input was kept in 8 bits
        dict(name="gateup_bwd_ckpt_4096", op="gateup_bwd", T=4096, d=7168, f=2368, act="silu", bias=False, ckpt=True,
             saved=False),
        # a layer's input kept in 8 bits and read back
        dict(name="mxfp8_8192", op="mxfp8", T=8192, d=7168),
        # a whole block's training step: forward with an 8-bit checkpoint, then every gradient
        dict(name="block_step_1024", op="block", T=1024, d=6144, f=2048, act="silu", ckpt=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(lo, _logint(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "gateup", "gateup", "gateup_bwd", "gateup_bwd",
                     "mxfp8", "block"])
    if op == "mxfp8":
        return dict(op=op, T=_logint(rng, 1, 8192), d=_mult(rng, 32, 7168, 32))
    acts = ["silu", "gelu", "gelu_tanh", "relu"]
    flag = lambda p=0.5: rng.random() < p
    if op == "linear":
        xt = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, T=_logint(rng, 1, 4096), n=_logint(rng, 64, 7168), k=_mult(rng, 64, 7168, 8),
                    act=rng.choice(["none"] + acts), bias=flag(), residual=flag(), xt=xt,
                    yt="f32" if xt == "f32" else rng.choice(["bf16", "bf16", "f32"]))
    if op == "linear_bwd":
        ckpt = flag(0.3)
        return dict(op=op, T=_logint(rng, 1, 4096), n=_logint(rng, 64, 7168),
                    k=_mult(rng, 64, 7168, 32 if ckpt else 8), act=rng.choice(["none"] + acts), bias=flag(), ckpt=ckpt)
    if op == "gateup":
        return dict(op=op, T=_logint(rng, 1, 4096), d=_mult(rng, 64, 7168, 8), f=_mult(rng, 64, 2368, 8),
                    act=rng.choice(acts), bias=flag(), ht=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gateup_bwd":
        ckpt = flag(0.4)
        return dict(op=op, T=_logint(rng, 1, 4096), d=_mult(rng, 64, 7168, 32 if ckpt else 8),
                    f=_mult(rng, 64, 2368, 8), act=rng.choice(acts), bias=flag(), ckpt=ckpt, saved=flag(0.4))
    return dict(op=op, T=_logint(rng, 1, 2048), d=_mult(rng, 64, 7168, 32), f=_mult(rng, 64, 2368, 8), act="silu",
                ckpt=flag(0.7))


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    c, T = case, case["T"]
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "mxfp8":
        e = T * c["d"]
        return {"bytes": 2 * (2 * e + e + e // 32), "flops": 4 * e}
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        b = T * k * size[c["xt"]] + 2 * n * k + T * n * size[c["yt"]] * (2 if c["residual"] else 1)
        return {"bytes": b + (4 * n if c["bias"] else 0), "flops": 2 * T * n * k}
    if c["op"] == "linear_bwd":
        n, k = c["n"], c["k"]
        # dy, x, W in; dx, dW, dbias out; the recomputed product counts where the activation needs it
        b = 2 * T * n + 2 * T * k + 2 * n * k + 2 * T * k + 2 * n * k + 4 * n
        b += T * k + T * k // 32 if c["ckpt"] else 0
        return {"bytes": b, "flops": (4 if c["act"] == "none" else 6) * T * n * k}
    d, f = c["d"], c["f"]
    if c["op"] == "gateup":
        return {"bytes": 2 * T * d + 4 * d * f + T * f * size[c["ht"]], "flops": 4 * T * d * f}
    if c["op"] == "gateup_bwd":
        b = 2 * T * f + 2 * T * d + 4 * d * f + 2 * T * d + 4 * d * f + 2 * T * f
        b += 4 * T * f if c["saved"] else 0
        b += T * d + T * d // 32 if c["ckpt"] else 0
        return {"bytes": b, "flops": (8 if c["saved"] else 12) * T * d * f}
    # block: x, three weights, dy, residual in; y, dx and three weight gradients out; forward 6, backward 12 products,
    # and gate and up recomputed
    b = 2 * (5 * T * d + 6 * d * f)
    return {"bytes": b, "flops": (6 + 12 + 4) * T * d * f}


# ----------------------------------------------------------------------------- inputs

class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)


def _activations(gen, T, d, dtype=torch.bfloat16):
    # a normalised hidden state: unit variance, every 64th channel an order larger
    x = torch.randn(T, d, generator=gen.g, device="cuda")
    x[:, 7::64] *= 8.0
    return x.to(dtype)


def _inputs(case, seed):
    c, T = case, case["T"]
    g = _Gen(seed * 7919 + 17)
    if c["op"] == "mxfp8":
        return dict(x=_activations(g, T, c["d"]))
    if c["op"] in ("linear", "linear_bwd"):
        n, k = c["n"], c["k"]
        xt = torch.float32 if c.get("xt") == "f32" else torch.bfloat16
        s = dict(x=_activations(g, T, k, xt), w=g.normal(n, k, std=k ** -0.5),
                 bias=g.normal(n, std=0.5, dtype=torch.float32) if c["bias"] else None)
        if c["op"] == "linear":
            yt = torch.float32 if c["yt"] == "f32" else torch.bfloat16
            s["residual"] = g.normal(T, n, dtype=yt) if c["residual"] else None
        else:
            s["dy"] = g.normal(T, n, std=0.25)
        return s
    d, f = c["d"], c["f"]
    s = dict(x=_activations(g, T, d), wg=g.normal(f, d, std=d ** -0.5), wu=g.normal(f, d, std=d ** -0.5))
    if c["op"] == "block":
        s["wd"] = g.normal(d, f, std=f ** -0.5)
        s["residual"] = g.normal(T, d)
        s["dy"] = g.normal(T, d, std=0.25)
        return s
    s["bg"] = g.normal(f, std=0.5, dtype=torch.float32) if c["bias"] else None
    s["bu"] = g.normal(f, std=0.5, dtype=torch.float32) if c["bias"] else None
    if c["op"] == "gateup_bwd":
        s["dh"] = g.normal(T, f, std=0.25)
        # what a forward pass left behind: gate and up products, [2][T][f]
        s["pre"] = g.normal(2, T, f, std=1.2) if c["saved"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] == "block":
        import mxfp4_routed_expert_amd as M
        s["ffn"] = M.DenseFFN(s["wg"], s["wu"], s["wd"], case["T"], act_fn=case["act"],
                              checkpoint="mxfp8" if case["ckpt"] else "bf16")
    return s


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(s):
    import mxfp4_routed_expert_amd as M
    c = s["case"]
    op = c["op"]
    if op == "linear":
        return M.moe_dense_linear(s["x"], s["w"], s["bias"], c["act"], s["residual"],
                                  out_dtype=torch.float32 if c["yt"] == "f32" else torch.bfloat16)
    if op == "gateup":
        return M.moe_dense_gateup(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], c["act"],
                                  out_dtype=torch.float32 if c["ht"] == "f32" else torch.bfloat16)[0]
    if op == "mxfp8":
        codes, scales = M.moe_mxfp8_quantize(s["x"])
        return M.moe_mxfp8_dequant(codes, scales)
    if op == "block":
        y = s["ffn"].forward(s["x"], s["residual"], train=True)
        dx, dwg, dwu, dwd = s["ffn"].backward(s["dy"])
        return y, dx, dwg, dwu, dwd
    x, xs = M.moe_mxfp8_quantize(s["x"]) if c["ckpt"] else (s["x"], None)
    if op == "linear_bwd":
        return M.moe_dense_linear_backward(s["dy"], x, s["w"], s["bias"], c["act"], x_scales=xs)
    dx, dwg, dwu, dbg, dbu, h = M.moe_dense_gateup_backward(s["dh"], x, s["wg"], s["wu"], s["bg"], s["bu"], c["act"],
                                                            x_scales=xs, pre=s["pre"], want_h=True)
    return dx, dwg, dwu, dbg, dbu, h


# ----------------------------------------------------------------------------- plain form

def _act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
    return torch.clamp(z, min=0.0)


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(a * (z + 0.044715 * z * z * z))
        return s + z * s * (1.0 - s) * a * (1.0 + 3.0 * 0.044715 * z * z)
    return (z > 0).to(z.dtype)


def _mxfp8_round_trip(x):
    """float32 values of the OCP MXFP8 (E4M3) encoding of x, 32-value blocks along the row."""
    b = x.float().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    e = torch.frexp(amax)[1] - 1 - 8
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    v = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return torch.ldexp(v, e).reshape(x.shape)


def _affine(x, w, bias):
    z = x @ w.float().t()
    return z if bias is None else z + bias


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    bf = torch.bfloat16
    if op == "mxfp8":
        return _mxfp8_round_trip(s["x"]).to(bf)
    if op == "linear":
        y = _act(c["act"], _affine(s["x"].float(), s["w"], s["bias"]))
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(torch.float32 if c["yt"] == "f32" else bf)
    if op == "gateup":
        x = s["x"].float()
        h = _act(c["act"], _affine(x, s["wg"], s["bg"])) * _affine(x, s["wu"], s["bu"])
        return h.to(torch.float32 if c["ht"] == "f32" else bf)
    x = _mxfp8_round_trip(s["x"]) if c["ckpt"] else s["x"].float()
    if op == "linear_bwd":
        dy = s["dy"].float()
        dz = dy if c["act"] == "none" else dy * _act_grad(c["act"], _affine(x, s["w"], s["bias"]))
        return (dz @ s["w"].float()).to(bf), (dz.t() @ x).to(bf), dz.sum(0)
    if op == "gateup_bwd":
        dh = s["dh"].float()
        if s["pre"] is not None:
            g, u = s["pre"][0].float(), s["pre"][1].float()
        else:
            g, u = _affine(x, s["wg"], s["bg"]), _affine(x, s["wu"], s["bu"])
        a = _act(c["act"], g)
        dg, du = dh * u * _act_grad(c["act"], g), dh * a
        dx = dg @ s["wg"].float() + du @ s["wu"].float()
        return dx.to(bf), (dg.t() @ x).to(bf), (du.t() @ x).to(bf), dg.sum(0), du.sum(0), (a * u).to(bf)
    # block: the forward pass sees x itself, the backward pass the checkpoint
    x0 = s["x"].float()
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    h0 = _act(c["act"], x0 @ wg.t()) * (x0 @ wu.t())
    y = h0 @ wd.t() + s["residual"].float()
    dy = s["dy"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a = _act(c["act"], g)
    dh = dy @ wd
    dg, du = dh * u * _act_grad(c["act"], g), dh * a
    return (y.to(bf), (dg @ wg + du @ wu).to(bf), (dg.t() @ x).to(bf), (du.t() @ x).to(bf),
            (dy.t() @ (a * u)).to(bf))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- 64 bits

def _f64_act_pair(name, z):
    """The activation and its derivative at z, in 64 bits, from their definitions."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).double()
        return z * on, on
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s + z * s * (1.0 - s)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2.0) * (2.0 * math.pi) ** -0.5
    r = (2.0 / math.pi) ** 0.5
    t = torch.tanh(r * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * r * (1.0 + 0.134145 * z * z)


def _f64_mxfp8(x):
    v = x.double()
    T, d = v.shape
    v = v.view(T, d // 32, 32)
    top = v.abs().max(dim=2, keepdim=True).values
    scale = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - 8.0, -127.0, 127.0))
    q = v / scale
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(q.abs())), min=-6.0) - 3.0)
    q = torch.clamp(torch.round(q / step) * step, -448.0, 448.0)      # round() takes halves to even
    return torch.where(top > 0, q * scale, torch.zeros_like(q)).view(T, d)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "mxfp8":
        return _f64_mxfp8(s["x"])
    lin = lambda x, w, b: torch.matmul(x, w.double().transpose(0, 1)) + (0.0 if b is None else b.double())
    if op == "linear":
        y = _f64_act_pair(case["act"], lin(s["x"].double(), s["w"], s["bias"]))[0]
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "gateup":
        x = s["x"].double()
        return _f64_act_pair(case["act"], lin(x, s["wg"], s["bg"]))[0] * lin(x, s["wu"], s["bu"])
    x = _f64_mxfp8(s["x"]) if case["ckpt"] else s["x"].double()
    if op == "linear_bwd":
        dz = s["dy"].double()
        if case["act"] != "none":
            dz = dz * _f64_act_pair(case["act"], lin(x, s["w"], s["bias"]))[1]
        return torch.matmul(dz, s["w"].double()), torch.matmul(dz.transpose(0, 1), x), dz.sum(dim=0)

    def gated(dh, g, u):
        a, da = _f64_act_pair(case["act"], g)
        dg, du = dh * u * da, dh * a
        dx = torch.matmul(dg, s["wg"].double()) + torch.matmul(du, s["wu"].double())
        return dx, torch.matmul(dg.transpose(0, 1), x), torch.matmul(du.transpose(0, 1), x), dg, du, a * u

    if op == "gateup_bwd":
        g, u = (s["pre"][0].double(), s["pre"][1].double()) if case["saved"] else (lin(x, s["wg"], s["bg"]),
                                                                                  lin(x, s["wu"], s["bu"]))
        dx, dwg, dwu, dg, du, h = gated(s["dh"].double(), g, u)
        return dx, dwg, dwu, dg.sum(dim=0), du.sum(dim=0), h
    x0, dy = s["x"].double(), s["dy"].double()
    y = lin(_f64_act_pair(case["act"], lin(x0, s["wg"], None))[0] * lin(x0, s["wu"], None), s["wd"], None)
    dx, dwg, dwu, _, _, h = gated(torch.matmul(dy, s["wd"].double()), lin(x, s["wg"], None), lin(x, s["wu"], None))
    return y + s["residual"].double(), dx, dwg, dwu, torch.matmul(dy.transpose(0, 1), h)
