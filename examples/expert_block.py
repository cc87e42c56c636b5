"""A feed-forward block of experts in FP8, forward and backward.

    y   = N(x)                                      pre norm, codes per token
    xs  = rows of y sorted by expert                codes and factors
    h   = silu(xs Wg^T) * (xs Wu^T)                 one gated product per expert, codes
    o   = h Wd^T                                    one product per expert
    b   = sum over a token's experts of w o
    x'  = alpha x + gate * N_post(b)                residual scale, learned gate
    z   = N(x')                                     the next block's input

Everything between the tensors is a call of this package, on the device: the
experts' row counts never come to the host in the forward pass.  The backward
pass runs the same chain back.  ExpertBlock casts per tensor and per token; its
weight gradients are one GEMM per expert, so it reads the row counts once.
BlockScaledExperts casts in blocks of 128, keeps nothing but 8-bit codes of the
experts' activations for the backward pass, and never reads the row counts.

    python examples/expert_block.py [--recipe block] [--tokens 4096] [--experts 16] ...
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_fp8_linear_gb300 as F   # noqa: E402


def scale_for(top, x):
    """The scale that takes x's largest magnitude to `top`; finite for a
    tensor of zeros."""
    return top / F.fp8_amax(x).clamp_min(1e-20)


def weight_codes(w):
    """E4M3 codes of w [E, N, K] with one factor per expert, and transposed."""
    E, N, K = w.shape
    q, q_t = torch.empty(E, N, K, dtype=torch.uint8, device=w.device), \
        torch.empty(E, K, N, dtype=torch.uint8, device=w.device)
    inv = torch.empty(E, device=w.device)
    for e in range(E):
        scale = scale_for(448.0, w[e])
        F.fp8_quantize(w[e], F.E4M3, scale=scale, q=q[e], q_t=q_t[e])
        inv[e] = 1.0 / scale[0]
    return q, q_t, inv


class ExpertBlock:
    """The block's weights (bf16 masters, FP8 codes) and its delayed scales."""

    def __init__(self, width, hidden, experts, slots, alpha=1.0, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: (torch.randn(*s, generator=g, device=device) * std)
        self.experts, self.slots, self.alpha = experts, slots, alpha
        self.w_pre, self.w_post = 1 + r(width, std=0.1), 1 + r(width, std=0.1)
        self.w_next = 1 + r(width, std=0.1)
        self.gate = r(1, width, std=0.3).to(torch.bfloat16)
        self.router = r(experts, width, std=width ** -0.5).to(torch.bfloat16)
        self.w_in = r(experts, 2 * hidden, width, std=width ** -0.5).to(torch.bfloat16)
        self.w_out = r(experts, width, hidden, std=hidden ** -0.5).to(torch.bfloat16)
        self.in_q, self.in_qt, self.in_inv = weight_codes(self.w_in)
        self.out_q, self.out_qt, self.out_inv = weight_codes(self.w_out)
        # delayed scales of the hidden codes and of the gradients' codes
        self.h_scale = torch.full((1,), 32.0, device=device)

    def forward(self, x):
        s = {"x": x}
        s["pre"] = F.fp8_norm_fwd(x, w_pre=self.w_pre, q_fmt=F.E4M3, q_gran=F.GRAN_ROW,
                                  want_stats=True, want_x_out=False)
        p = torch.softmax((s["pre"].y @ self.router.t()).float(), dim=1)
        w, ids = p.topk(self.slots, dim=1)
        s["w"], s["ids"] = (w / w.sum(1, keepdim=True)).contiguous(), ids.int()
        s["plan"] = F.fp8_moe_plan(s["ids"], self.experts, align=32)
        s["xs"], s["xs_inv"] = F.fp8_moe_permute(s["pre"].q, s["plan"].row_of, s["plan"].src,
                                                 scale=s["pre"].q_scale_inv)
        s["up"] = F.fp8_gemm_act(s["xs"], F.E4M3, self.in_q, F.E4M3, s["xs_inv"],
                                 self.in_inv[:, None].expand(-1, self.in_q.shape[1]).contiguous(),
                                 ga=F.GRAN_ROW, gb=F.GRAN_ROW, act=F.ACT_SILU, gated=True, want_z=True,
                                 want_d=False, q_fmt=F.E4M3, q_scale=self.h_scale, want_amax=True,
                                 offsets=s["plan"].offsets)
        s["o"] = F.fp8_gemm_act(s["up"].q, F.E4M3, self.out_q, F.E4M3, 1.0 / self.h_scale, self.out_inv,
                                offsets=s["plan"].offsets).d
        s["b"] = F.fp8_moe_unpermute(s["o"], s["plan"].row_of, weights=s["w"])
        s["post"] = F.fp8_norm_fwd(x, s["b"], alpha=self.alpha, gate=self.gate, post_norm=True,
                                   w_post=self.w_post, w_pre=self.w_next, want_stats=True)
        return s["post"].x_out, s["post"].y, s

    def backward(self, dx_out, dz, s):
        """Gradients of the inputs and weights from those of x' and z (the
        router's own gradient through the softmax is left to the caller, who
        gets dw, the gradient of the experts' weights)."""
        plan, off = s["plan"], s["plan"].offsets.tolist()
        g = {}
        n = F.fp8_norm_bwd(dz, s["post"].x_out, s["post"].stats, dx_out=dx_out, h=s["b"],
                           alpha=self.alpha, gate=self.gate, post_norm=True, w_post=self.w_post,
                           w_pre=self.w_next)
        g.update(w_next=n.dw_pre, w_post=n.dw_post, gate=n.dgate)
        do, g["w"] = F.fp8_moe_unpermute_bwd(n.dh, s["o"], plan.row_of, plan.src, s["w"])
        # the second product: codes of its gradient, dgrad per expert, wgrad per expert
        do_scale = scale_for(57344.0, do)
        do_q = F.fp8_quantize(do, F.E5M2, scale=do_scale)[0]
        do_inv = 1.0 / do_scale
        dh = F.fp8_gemm_act(do_q, F.E5M2, self.out_qt, F.E4M3, do_inv, self.out_inv,
                            offsets=plan.offsets).d
        g["w_out"] = self._wgrad(do_q, do_inv, s["up"].q, 1.0 / self.h_scale, off)
        # the epilogue's gradient, as codes
        dz_scale = scale_for(2048.0, dh[:off[-1]])
        a = F.fp8_act_bwd(dh, s["up"].z, F.ACT_SILU, gated=True, want_dz=False, q_fmt=F.E5M2,
                          q_scale=dz_scale, offsets=plan.offsets)
        dxs = F.fp8_gemm_act(a.q, F.E5M2, self.in_qt, F.E4M3, 1.0 / dz_scale, self.in_inv,
                             offsets=plan.offsets).d
        ys = s["pre"].y   # the wgrad reads the tokens' rows with one factor
        y_scale = scale_for(448.0, ys)
        y_q = F.fp8_moe_permute(F.fp8_quantize(ys, F.E4M3, scale=y_scale)[0], plan.row_of, plan.src)[0]
        g["w_in"] = self._wgrad(a.q, 1.0 / dz_scale, y_q, 1.0 / y_scale, off)
        dy = F.fp8_moe_unpermute(dxs, plan.row_of)
        m = F.fp8_norm_bwd(dy, s["x"], s["pre"].stats, dx_out=n.dx, w_pre=self.w_pre)
        g.update(x=m.dx, w_pre=m.dw_pre)
        return g

    def _wgrad(self, d_q, d_inv, x_q, x_inv, off):
        """dW [E, N, K] = d^T x over each expert's rows (zeros without any)."""
        out = torch.zeros(len(off) - 1, d_q.shape[1], x_q.shape[1], device=d_q.device)
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if b > a:
                F.fp8_gemm(d_q[a:b], F.E5M2, x_q[a:b], F.E4M3, d_inv, x_inv, out=F.OUT_F32, D=out[e],
                           layout=F.LAYOUT_KM_KN)
        return out


def block_codes(w, pow2):
    """E4M3 codes of w [E, N, K] in 128x128 blocks with their factors, and transposed."""
    parts = [F.fp8_quantize_blocks(w[e], F.E4M3, F.GRAN_128x128, pow2=pow2, transpose=True) for e in range(w.shape[0])]
    return [torch.stack(p) for p in zip(*parts)]


class BlockScaledExperts(ExpertBlock):
    """The same block under the block recipe: weights in 128x128 blocks,
    activations and gradients in 1x128 blocks.  Of the experts' activations the
    backward pass gets the codes of the sorted inputs and of the pre-activations."""

    def __init__(self, width, hidden, experts, slots, alpha=1.0, seed=0, device="cuda", pow2=False):
        super().__init__(width, hidden, experts, slots, alpha, seed, device)
        self.pow2 = pow2
        self.in_q, self.in_inv, self.in_qt, self.in_inv_t = block_codes(self.w_in, pow2)
        self.out_q, self.out_inv, self.out_qt, self.out_inv_t = block_codes(self.w_out, pow2)

    def forward(self, x):
        p2 = dict(pow2=self.pow2)
        s = {"x": x}
        s["pre"] = F.fp8_norm_fwd(x, w_pre=self.w_pre, want_stats=True, want_x_out=False)
        p = torch.softmax((s["pre"].y @ self.router.t()).float(), dim=1)
        w, ids = p.topk(self.slots, dim=1)
        s["w"], s["ids"] = (w / w.sum(1, keepdim=True)).contiguous(), ids.int()
        # whole blocks of 128 tokens an expert, for the weight gradients
        rows = -(-F.fp8_moe_rows(x.shape[0], self.slots, self.experts, 128) // 128) * 128
        s["plan"] = plan = F.fp8_moe_plan(s["ids"], self.experts, align=128, rows=rows)
        q, inv = F.fp8_quantize_blocks(s["pre"].y, F.E4M3, F.GRAN_1x128, **p2)[:2]
        s["xs"] = F.fp8_moe_permute(q, plan.row_of, plan.src)[0]
        s["xs_inv"] = F.fp8_moe_permute(inv, plan.row_of, plan.src)[0]
        z = F.fp8_gemm_experts(s["xs"], F.E4M3, self.in_q, F.E4M3, s["xs_inv"], self.in_inv, plan.offsets, **p2)
        s["up"] = F.fp8_act_block(z, F.ACT_SILU, gated=True, keep=True, offsets=plan.offsets, **p2)
        s["o"] = F.fp8_gemm_experts(s["up"].q, F.E4M3, self.out_q, F.E4M3, s["up"].scale_inv, self.out_inv,
                                    plan.offsets, **p2)
        s["b"] = F.fp8_moe_unpermute(s["o"], plan.row_of, weights=s["w"])
        s["post"] = F.fp8_norm_fwd(x, s["b"], alpha=self.alpha, gate=self.gate, post_norm=True,
                                   w_post=self.w_post, w_pre=self.w_next, want_stats=True)
        return s["post"].x_out, s["post"].y, s

    def backward(self, dx_out, dz, s):
        p2 = dict(pow2=self.pow2)
        plan, up, g = s["plan"], s["up"], {}
        n = F.fp8_norm_bwd(dz, s["post"].x_out, s["post"].stats, dx_out=dx_out, h=s["b"],
                           alpha=self.alpha, gate=self.gate, post_norm=True, w_post=self.w_post,
                           w_pre=self.w_next)
        g.update(w_next=n.dw_pre, w_post=n.dw_post, gate=n.dgate)
        do, g["w"] = F.fp8_moe_unpermute_bwd(n.dh, s["o"], plan.row_of, plan.src, s["w"])
        do_q, do_inv, do_t, do_inv_t = F.fp8_quantize_blocks(do, F.E5M2, F.GRAN_1x128, transpose=True, **p2)
        dh = F.fp8_gemm_experts(do_q, F.E5M2, self.out_qt, F.E4M3, do_inv, self.out_inv_t, plan.offsets, **p2)
        a = F.fp8_act_block_bwd(dh, up.z_q, up.z_scale_inv, F.ACT_SILU, gated=True, want_t=True, want_h_t=True,
                                offsets=plan.offsets, **p2)
        g["w_out"] = F.fp8_wgrad_experts(do_t, F.E5M2, a.h_t, F.E4M3, do_inv_t, a.h_scale_inv_t, plan.offsets, **p2)
        dxs = F.fp8_gemm_experts(a.q, F.E5M2, self.in_qt, F.E4M3, a.scale_inv, self.in_inv_t, plan.offsets, **p2)
        xs_t, xs_inv_t = F.fp8_block_transpose(s["xs"], F.E4M3, s["xs_inv"], **p2)
        g["w_in"] = F.fp8_wgrad_experts(a.q_t, F.E5M2, xs_t, F.E4M3, a.scale_inv_t, xs_inv_t, plan.offsets, **p2)
        dy = F.fp8_moe_unpermute(dxs, plan.row_of)
        m = F.fp8_norm_bwd(dy, s["x"], s["pre"].stats, dx_out=n.dx, w_pre=self.w_pre)
        g.update(x=m.dx, w_pre=m.dw_pre)
        return g


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--slots", type=int, default=2)
    ap.add_argument("--recipe", choices=["tensor", "block", "block_pow2"], default="tensor")
    a = ap.parse_args()
    if a.recipe == "tensor":
        block = ExpertBlock(a.width, a.hidden, a.experts, a.slots)
    else:
        block = BlockScaledExperts(a.width, a.hidden, a.experts, a.slots, pow2=a.recipe == "block_pow2")
    x = torch.randn(a.tokens, a.width, device="cuda").to(torch.bfloat16)
    d = (torch.randn(a.tokens, a.width, device="cuda") * 1e-3).to(torch.bfloat16)

    def timed(f, n=10):
        for _ in range(3):
            f()
        b, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        b.record()
        for _ in range(n):
            f()
        e.record()
        e.synchronize()
        return b.elapsed_time(e) / n

    fwd = timed(lambda: block.forward(x))
    _, _, s = block.forward(x)
    bwd = timed(lambda: block.backward(d, d, s))
    flop = 2 * a.tokens * a.slots * 3 * a.hidden * a.width
    F.check_device_status()
    print(f"{a.tokens} tokens to {a.slots} of {a.experts} experts, {a.width} x {a.hidden}: forward "
          f"{fwd:.3f} ms, backward {bwd:.3f} ms, {3 * flop / (fwd + bwd) / 1e9:.0f} TFLOP/s over both")
    assert math.isfinite(fwd)


if __name__ == "__main__":
    main()
