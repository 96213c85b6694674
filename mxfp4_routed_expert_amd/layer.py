"""One routed MoE layer step composed from the C-ABI calls.

route -> permute -> routed experts (moe_expert_ffn) -> shared expert (moe_expert_ffn,
identity form) -> combine; LatentMoE layers add moe_dense_bf16 before the routed experts
and after the combine (Kimi K3 article, architecture section); a gated shared expert's
output is scaled by its gate before it is added after the up projection.  A shared expert
with bf16 weights (DenseWeights) runs as moe_dense_gateup and moe_dense_linear.  Decode-sized
LatentMoE steps run the routed down product and the combine into z as one down-combine
launch.  Decode-sized
batches use the fused calls instead, three kernels a step -- the router's logits; the
selection with the routed and shared gate/up in one launch (moe_topk_gateup_shared); down
and combine in one launch -- or, on request, the whole step as one launch
(moe_decode_step).
With act "fp8" the experts (FP8 block-128 weights) multiply 8-bit activations on the matrix cores.
Every step runs in the HIP library; this module only wires buffers.  All buffers for a token count are allocated once, so a step enqueues kernels and
allocates nothing.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


@dataclass
class LayerWeights:
    """Device tensors of one layer (see moe.h for layouts)."""
    score: str
    k: int
    renormalize: bool
    routed_scaling: float
    act: str
    w_router: torch.Tensor                 # bf16 [E][H]
    experts: B.ExpertWeights
    logit_bias: torch.Tensor | None = None
    select_bias: torch.Tensor | None = None
    shared: B.ExpertWeights | B.DenseWeights | None = None   # DenseWeights: a bf16 shared expert
    w_shared_gate: torch.Tensor | None = None  # bf16 [H]
    p_down: torch.Tensor | None = None     # bf16 [L][H]
    p_up: torch.Tensor | None = None       # bf16 [H][L]
    n_group: int = 1                       # group-limited selection (1: none)
    topk_group: int = 1

    @property
    def H(self):
        return self.w_router.shape[1]

    @property
    def E(self):
        return self.w_router.shape[0]


# LDS a down-combine workgroup may hold: per slot (k, +1 with a shared expert) the h row
# in 4 * roundup(d_ff, 512) bytes and a table of 128 floats (the library's own rule)
FUSED_LDS_LIMIT = 150 * 1024


def down_combine_lds(k: int, shared: bool, d_ff: int) -> int:
    s = k + (1 if shared else 0)
    return s * 4 * ((d_ff + 511) // 512 * 512) + s * 128 * 4


def fuses(w: LayerWeights, T: int) -> bool:
    """Whether a step of T tokens takes the fused decode calls: decode-sized batches
    (T <= 4) with FLOAT activations and no latent projections, a shared expert (if any)
    of the routed format and widths (a bf16 one runs as its own calls), and k + 1 rows of d_ff within the LDS limit."""
    ex, sh = w.experts, w.shared
    return (w.act == "float" and w.p_down is None and w.p_up is None and 1 <= T <= 4
            and (sh is None or (not isinstance(sh, B.DenseWeights) and sh.fmt == ex.fmt and sh.d_model == ex.d_model
                                and sh.d_ff == ex.d_ff))
            and down_combine_lds(w.k, sh is not None, ex.d_ff) <= FUSED_LDS_LIMIT)


class MoELayer:
    def __init__(self, w: LayerWeights, T: int, device, single_launch: bool = False):
        """single_launch: fused decode steps run as one moe_decode_step launch instead of its
        three calls (moe_router_logits, moe_topk_gateup_shared, moe_expert_down_combine); the
        results are the same bits.  The three calls are the default: on MI355X they measure a
        few per cent faster per step than the single launch."""
        self.w, self.T, self.dev = w, T, device
        E, H, k = w.E, w.H, w.k
        L, I = w.experts.d_model, w.experts.d_ff
        f32, i32 = torch.float32, torch.int32
        e = lambda *s, dt=f32: torch.empty(s, dtype=dt, device=device)
        # Decode-sized batches: the shared expert joins the routed gate/up launch and the
        # down product writes the combined output directly (moe_expert_gateup_shared,
        # moe_expert_down_combine), so y_rows and y_shared never exist.
        self.fused = fuses(w, T)
        # decode-sized LatentMoE steps: the routed down product and the combine into z run as
        # one down-combine launch with no shared slot (the shared expert's output is added after
        # the up projection), so y_rows never exists
        self.latent_down_combine = (w.act == "float" and w.p_up is not None and 1 <= T <= 8
                                    and down_combine_lds(w.k, False, w.experts.d_ff) <= FUSED_LDS_LIMIT)
        self.down_combined = self.fused or self.latent_down_combine
        sh = w.shared
        self.ids, self.topk_w = e(T, k, dt=i32), e(T, k)
        self.sg = e(T) if w.w_shared_gate is not None else None
        self.offs, self.sp, self.p2r = e(E + 1, dt=i32), e(T * k, dt=i32), e(T * k, dt=i32)
        self.x_lat = e(T, L) if w.p_down is not None else None
        self.y_rows = None if self.down_combined else e(T * k, L)
        self.y_s = e(T, H) if (sh is not None and not self.fused) else None
        self.z = e(T, L) if w.p_up is not None else None
        # LatentMoE with a gated shared expert: g * y_s is formed by moe_combine with no
        # routed slots (k = 0) before it becomes the residual of the up projection
        self.latent_gate = w.p_up is not None and sh is not None and w.w_shared_gate is not None
        self.y_sg = e(T, H) if self.latent_gate else None
        self.no_rows = e(0, dt=i32)
        self.no_w = e(T, 0)
        self.out = e(T, H)
        self.ws_route = B._workspace(B.moe_route_workspace(T, H, E, k, w.score), device)
        self.logits = e(T, E + (1 if w.w_shared_gate is not None else 0)) if self.fused else None
        self.single = self.fused and single_launch
        self.sync = B.decode_step_sync(device) if self.single else None
        # h rows: the staged form runs gate/up and down as separate calls on these buffers
        # (float32 h in FLOAT mode, codes and scales in MXFP4 and FP8 mode), as does the fused form
        quant, fp8 = w.act != "float", w.act == "fp8"
        code_width = lambda d: d if fp8 else d // 2
        scale_width = lambda d: d // 128 if fp8 else d // 32
        self.h = e(T * k, I) if not fp8 else None
        self.hq = e(T * k, code_width(I), dt=torch.uint8) if quant else None
        self.hs = e(T * k, scale_width(I), dt=torch.uint8) if quant else None
        self.ws_gu = B._workspace(B.moe_expert_gateup_workspace(w.experts, w.act, T, k), device)
        # a bf16 shared expert: dense products from x itself, h in float32 as the routed experts'
        self.dense_sh = isinstance(sh, B.DenseWeights)
        staged_sh = sh is not None and not self.fused and not self.dense_sh
        Is = sh.d_ff if sh is not None else 0
        self.h_sh = e(T, Is) if sh is not None else None
        self.hq_sh = e(T, code_width(Is), dt=torch.uint8) if (staged_sh and quant) else None
        self.hs_sh = e(T, scale_width(Is), dt=torch.uint8) if (staged_sh and quant) else None
        self.ws_gu_sh = B._workspace(B.moe_expert_gateup_workspace(sh, w.act, T, 1), device) if staged_sh else None
        if self.dense_sh:
            need = max(B.moe_dense_gateup_workspace(T, H, Is, "silu", f32), B.moe_dense_linear_workspace(T, H, Is, x_dtype=f32, out_dtype=f32))
            self.ws_gu_sh = B._workspace(need, device)
        # otherwise the shared expert does not depend on routing: it runs on a second stream,
        # joined before the combine, so it overlaps router, permutation and routed experts;
        # so does the latent down-projection, which the routed gate/up waits for
        side = w.shared is not None or w.p_down is not None
        self.side = torch.cuda.Stream(device=device) if (side and not self.fused) else None
        self.lat_ready = torch.cuda.Event() if (w.p_down is not None and not self.fused) else None

    def forward(self, x, mark=None):
        """One layer step on tokens x (bf16 [T][H]); returns the float32 output buffer.

        With `mark`, mark(name) is called on the step's stream before and after the routed
        gate/up call ("gateup_begin", "gateup_end") and the down call ("down_begin",
        "down_end"; the down product with the combine in the fused form), or around the
        single-launch step ("step_begin", "step_end"), so a caller can record events around
        those kernels."""
        w = self.w
        if self.single:
            # the whole step in one launch (the three calls below, same results)
            if mark is not None:
                mark("step_begin")
            B.moe_decode_step(x, w.w_router, w.k, w.experts, w.shared, w.score, w.renormalize, w.routed_scaling,
                              w.logit_bias, w.select_bias, w.w_shared_gate, sync=self.sync,
                              out=(self.logits, self.ids, self.topk_w, self.sg, self.offs, self.sp, self.p2r, self.h,
                                   self.h_sh, self.out), n_group=w.n_group, topk_group=w.topk_group)
            if mark is not None:
                mark("step_end")
            return self.out
        if self.fused:
            # three kernels: the router's logits, one gate/up launch that routes in its
            # prologue (the routing results land in the same buffers as moe_route_permute's),
            # and the down product with the combine
            B.moe_router_logits(x, w.w_router, w.k, w.score, w.w_shared_gate, out=self.logits, ws=self.ws_route,
                                n_group=w.n_group, topk_group=w.topk_group)
            if mark is not None:
                mark("gateup_begin")
            B.moe_topk_gateup_shared(self.logits, x, w.k, w.experts, w.shared, w.score, w.renormalize,
                                     w.routed_scaling, w.logit_bias, w.select_bias, w.w_shared_gate is not None,
                                     out=(self.ids, self.topk_w, self.sg, self.offs, self.sp, self.p2r, self.h,
                                          self.h_sh), n_group=w.n_group, topk_group=w.topk_group)
            if mark is not None:
                mark("gateup_end")
            if mark is not None:
                mark("down_begin")
            B.moe_expert_down_combine(w.experts, w.shared, self.h, self.h_sh, self.ids, self.topk_w, self.p2r,
                                      self.sg, out=self.out)
            if mark is not None:
                mark("down_end")
            return self.out
        quant = w.act != "float"
        cur = torch.cuda.current_stream()
        xe = x
        if self.side is not None:
            self.side.wait_stream(cur)
            with torch.cuda.stream(self.side):
                if w.p_down is not None:
                    xe = B.moe_dense_bf16(x, w.p_down, out=self.x_lat)
                    self.lat_ready.record(self.side)
                if self.dense_sh:
                    B.moe_dense_gateup(x, w.shared.gate, w.shared.up, out=self.h_sh, ws=self.ws_gu_sh)
                    B.moe_dense_linear(self.h_sh, w.shared.down, out=self.y_s, ws=self.ws_gu_sh)
                elif w.shared is not None:
                    B.moe_expert_gateup(w.shared, x, w.act, 1, None, None,
                                        out=(None if quant else self.h_sh, self.hq_sh, self.hs_sh), ws=self.ws_gu_sh)
                    B.moe_expert_down(w.shared, self.T, w.act, 1, None, self.h_sh, self.hq_sh, self.hs_sh,
                                      out=self.y_s)
        B.moe_route_permute(x, w.w_router, w.k, w.score, w.renormalize, w.routed_scaling, w.logit_bias,
                            w.select_bias, w.w_shared_gate,
                            out=(self.ids, self.topk_w, self.sg, self.offs, self.sp, self.p2r), ws=self.ws_route,
                            n_group=w.n_group, topk_group=w.topk_group)
        if w.p_down is not None:
            cur.wait_event(self.lat_ready)
        if mark is not None:
            mark("gateup_begin")
        B.moe_expert_gateup(w.experts, xe, w.act, w.k, self.offs, self.sp,
                            out=(None if quant else self.h, self.hq, self.hs), ws=self.ws_gu)
        if mark is not None:
            mark("gateup_end")
        if mark is not None:
            mark("down_begin")
        if self.latent_down_combine:
            B.moe_expert_down_combine(w.experts, None, self.h, None, self.ids, self.topk_w, self.p2r, out=self.z)
        else:
            B.moe_expert_down(w.experts, self.T, w.act, w.k, self.offs, self.h, self.hq, self.hs, out=self.y_rows)
        if mark is not None:
            mark("down_end")
        if self.side is not None:
            cur.wait_stream(self.side)
        if w.p_up is not None:
            if not self.latent_down_combine:
                B.moe_combine(self.y_rows, self.p2r, self.topk_w, out=self.z)
            res = self.y_s
            if self.latent_gate:
                res = B.moe_combine(None, self.no_rows, self.no_w, self.y_s, self.sg, out=self.y_sg)
            B.moe_dense_bf16(self.z, w.p_up, residual=res, out=self.out)
        else:
            B.moe_combine(self.y_rows, self.p2r, self.topk_w, self.y_s, self.sg, out=self.out)
        return self.out


# Token counts up to which DenseFFN keeps h in float32 (where the library keeps low terms too)
FFN_F32_TOKENS = 64


class DenseFFN:
    """A dense gated feed-forward block (bf16 weights): y = (act_fn(x Wg^T) * (x Wu^T)) Wd^T + residual, and its
    training step.

    forward(x, residual, train=True) keeps what backward(dy) needs: the input as it is (checkpoint="bf16": a reference,
    so it must not change until backward has run) or in 8 bits (checkpoint="mxfp8": a copy of 33/64 of its bytes, which
    stands for x in every gradient; the workspace has room for its bf16 form).  The backward pass recomputes the gate and up
    products from it.  Buffers for T tokens and one workspace are allocated once: results of a call are overwritten by the
    next, and calls must run in order (on one stream, or on streams that wait for each other); x, residual and dy may be
    the block's own last results.  Autograd does not see the calls."""

    def __init__(self, w_gate, w_up, w_down, T: int, act_fn: str = "silu", checkpoint: str = "bf16"):
        if checkpoint not in ("bf16", "mxfp8"):
            raise ValueError(f"checkpoint must be 'bf16' or 'mxfp8' (got {checkpoint!r})")
        f, d = w_gate.shape
        if tuple(w_up.shape) != (f, d) or tuple(w_down.shape) != (d, f):
            raise ValueError("w_gate and w_up are [d_ff][d_model], w_down is [d_model][d_ff]")
        self.wg, self.wu, self.wd, self.T, self.act_fn = w_gate, w_up, w_down, T, act_fn
        dev, mx = w_gate.device, checkpoint == "mxfp8"
        if mx and d % 32 != 0:
            raise ValueError(f"an MXFP8 checkpoint needs d_model a multiple of 32 (got {d})")
        bf, u8 = torch.bfloat16, torch.uint8
        e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=dev)
        # h between the products: float32 while the weights' bytes bound them (it costs nothing), else bf16;
        # its gradient float32 always (read once by an epilogue)
        ht = torch.float32 if T <= FFN_F32_TOKENS else bf
        self.h, self.y = e(T, f, dt=ht), e(T, d)
        self.x_saved = (e(T, d, dt=u8), e(T, d // 32, dt=u8)) if mx else None
        self.saved = None                      # (x or codes, scales or None) of the last training forward
        self.dh, self.dx = e(T, f, dt=torch.float32), e(T, d)
        self.dwg, self.dwu, self.dwd = e(f, d), e(f, d), e(d, f)
        need = max(B.moe_dense_gateup_workspace(T, d, f, act_fn, ht), B.moe_dense_linear_workspace(T, d, f, x_dtype=ht),
                   B.moe_dense_linear_backward_workspace(T, d, f, x_dtype=ht),
                   B.moe_dense_gateup_backward_workspace(T, d, f, act_fn, mx))
        self.ws = B._workspace(need, dev)

    @staticmethod
    def _within(t, *buffers):
        return isinstance(t, torch.Tensor) and any(t.untyped_storage().data_ptr() == b.untyped_storage().data_ptr() for b in buffers)

    def forward(self, x, residual=None, train: bool = False):
        # the input is kept before anything is written: it may be this block's own last result
        saved = self.saved
        if train:
            self.saved = None                  # (its buffers are written now)
            saved = B.moe_mxfp8_quantize(x, out=self.x_saved) if self.x_saved is not None else (x.clone() if self._within(x, self.y, self.dx) else x, None)
        B.moe_dense_gateup(x, self.wg, self.wu, act_fn=self.act_fn, out=self.h, ws=self.ws)
        B.moe_dense_linear(self.h, self.wd, residual=residual, out=self.y, ws=self.ws)
        self.saved = saved
        return self.y

    def backward(self, dy):
        """(dx, dw_gate, dw_up, dw_down) at dy; the residual's gradient is dy itself."""
        if self.saved is None:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, "DenseFFN.backward: no forward(..., train=True) before it")
        x, xs = self.saved
        if self._within(dy, self.dx):          # dx is written before dw_down reads dy
            dy = dy.clone()
        B.moe_dense_linear_backward(dy, None, self.wd, want=("dx",), out=(self.dh, None, None), ws=self.ws)
        B.moe_dense_gateup_backward(self.dh, x, self.wg, self.wu, act_fn=self.act_fn, x_scales=xs, want=("dx", "dw"),
                                    want_h=True, out=(self.dx, self.dwg, self.dwu, None, None, self.h), ws=self.ws)
        B.moe_dense_linear_backward(dy, self.h, self.wd, want=("dw",), out=(None, self.dwd, None), ws=self.ws)
        self.saved = None
        return self.dx, self.dwg, self.dwu, self.dwd


class FP8Linear:
    """A linear layer whose products run on block-128 FP8 operands: y = x W^T + residual, and its training step.

    set_weight(w) quantises a bf16 or float32 weight [n][kdim] (both multiples of 16) to 128 x 128 blocks, with its
    transpose for the input gradient; a training step calls it after each update of w.  forward(x, residual) keeps x's 8-bit
    transpose for the weight gradient (train=False: keeps nothing); backward(dy) gives dx and dw, bf16 (dw float32 with
    dw_dtype; dw_accumulate adds to the last dw, zeros at first, for a batch in pieces).  x and dy are bf16 or float32 [T][.].
    Buffers for T tokens and one workspace are allocated once: results of a call are overwritten by the next, and calls must
    run in order (on one stream, or on streams that wait for each other).  Autograd does not see the calls (they warn of a weight,
    x or residual that requires grad)."""

    def __init__(self, w, T: int, dw_dtype=torch.bfloat16):
        n, k = w.shape
        if n % 16 != 0 or k % 16 != 0:
            raise ValueError(f"FP8Linear needs n and kdim multiples of 16 (got {n} x {k})")
        self.n, self.k, self.T = n, k, T
        dev, u8 = w.device, torch.uint8
        e = lambda *s, dt=u8: torch.empty(s, dtype=dt, device=dev)
        nb, kb, tb, ld = (n + 127) // 128, (k + 127) // 128, (T + 127) // 128, (T + 15) // 16 * 16
        self.w_q = (e(n, k), e(nb, kb), e(k, n), e(kb, nb))
        self.x_q = (e(T, k), e(T, kb), e(k, ld), e(k, tb))
        self.dy_q = (e(T, n), e(T, nb), e(n, ld), e(n, tb))
        self.y, self.dx, self.dw = e(T, n, dt=torch.bfloat16), e(T, k, dt=torch.bfloat16), e(n, k, dt=dw_dtype)
        need = max(B.moe_fp8_linear_workspace(T, n, k, u8, w_scale=B.FP8_SCALE_E8M0),
                   B.moe_fp8_linear_workspace(T, k, n, u8, w_scale=B.FP8_SCALE_E8M0),
                   B.moe_fp8_linear_workspace(n, k, ld, u8, dw_dtype, B.FP8_SCALE_E8M0_ROW) if T else 0)
        self.ws = B._workspace(need, dev)
        self.dw.zero_()                                     # (what a first dw_accumulate adds to)
        self.saved = False
        self.set_weight(w)

    def set_weight(self, w):
        B.moe_fp8_quantize_weight(w, torch.uint8, transpose=True, out=self.w_q)

    def forward(self, x, residual=None, train: bool = True):
        q = self.x_q if train else (*self.x_q[:2], None, None)
        self.saved = False
        B.moe_fp8_quantize(x, cols=train, out=q)
        B.moe_fp8_linear(self.x_q[0], *self.w_q[:2], x_scales=self.x_q[1], residual=residual, out=self.y, ws=self.ws)
        self.saved = train
        return self.y

    def backward(self, dy, dw_accumulate: bool = False):
        """(dx, dw) at dy; the residual's gradient is dy itself."""
        if not self.saved:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, "FP8Linear.backward: no forward(..., train=True) before it")
        B.moe_fp8_quantize(dy, cols=True, out=self.dy_q)
        B.moe_fp8_linear(self.dy_q[0], *self.w_q[2:], x_scales=self.dy_q[1], out=self.dx, ws=self.ws)
        if self.T:
            B.moe_fp8_linear(self.dy_q[2], *self.x_q[2:], x_scales=self.dy_q[3], residual=self.dw if dw_accumulate else None,
                             out=self.dw, ws=self.ws)
        elif not dw_accumulate:
            self.dw.zero_()
        self.saved = False
        return self.dx, self.dw
