"""The MoE half of a decoder block on one GPU, forward and backward.

    x, residual -> residual add + norm -> router -> layout -> FP8 dispatch
      -> experts' gate and up product -> gated activation -> down product
      -> weighted combine

The experts are frozen FP8 weights (e4m3, one scale per 128x128 block); the
norm's gain, the router and everything before the block train.  What the
backward pass needs of the experts' inputs is kept in 8 bits.

    python examples/moe_layer.py [--tokens T] [--hidden H] [--ffn F]
                                 [--experts E] [--topk K]

prints how far the outputs and gradients are from a plain fp32 evaluation and
the time of a forward and of a forward and backward pass.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_topk_idx_gb300 as ep  # noqa: E402

FP8 = torch.float8_e4m3fn


def quantise_weights(w: torch.Tensor):
    """e4m3 bytes of w [E, n, k] and fp32 scales [E, ceil(n / 128), k / 128]."""
    E, n, k = w.shape
    nb = -(-n // 128)
    full = torch.zeros(E, nb * 128, k, device=w.device)
    full[:, :n] = w
    b = full.view(E, nb, 128, k // 128, 128)
    sf = (b.abs().amax(dim=(2, 4)) / 448.0).clamp_min(1e-30)
    q = (b / sf[:, :, None, :, None]).view(E, nb * 128, k)[:, :n].clamp(-448, 448)
    return q.to(FP8).view(torch.uint8).contiguous(), sf.contiguous()


def dequantise_weights(q: torch.Tensor, sf: torch.Tensor) -> torch.Tensor:
    n = q.shape[1]
    s = sf.repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)
    return q.view(FP8).float() * s


class MoeHalf:
    """Weights and one forward's saved state.  All sizes fixed at construction;
    hidden and ffn are multiples of 128."""

    def __init__(self, hidden, ffn, experts, topk, ranks=1, eps=1e-6, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.hidden, self.ffn, self.experts, self.topk = hidden, ffn, experts, topk
        self.ranks, self.eps = ranks, eps
        self.gamma = 1 + normal(hidden, std=0.1)
        self.router = normal(experts, hidden, std=hidden ** -0.5).bfloat16()
        self.w_in, self.w_in_sf = quantise_weights(
            normal(experts, 2 * ffn, hidden, std=hidden ** -0.5))
        self.w_out, self.w_out_sf = quantise_weights(normal(experts, hidden, ffn, std=ffn ** -0.5))
        # the gradient's products take the transposed bytes and block scales, laid out once
        self.w_in_t = self.w_in.transpose(1, 2).contiguous()
        self.w_in_t_sf = self.w_in_sf.transpose(1, 2).contiguous()
        self.w_out_t = self.w_out.transpose(1, 2).contiguous()
        self.w_out_t_sf = self.w_out_sf.transpose(1, 2).contiguous()

    def forward(self, x, residual, keep=False):
        """(block output, residual stream); with ``keep`` what backward needs is saved."""
        T = x.shape[0]
        n = ep.alloc_rmsnorm(x, residual=True, bf16=True, fp8=True, col_major_sf=True, rstd=keep)
        ep.ep_rmsnorm(x, self.gamma, self.eps, residual, **n)
        probs = torch.softmax(n["y"] @ self.router.t(), dim=1, dtype=torch.float32)
        w, idx = probs.topk(self.topk, dim=1)
        cfg = ep.make_config(T, self.topk, self.experts, self.ranks, self.hidden,
                             max(1, -(-T // self.ranks)), 16, do_expand=True,
                             do_zero_padding=True, do_cpu_sync=False, use_fp8=True,
                             use_tma_aligned_col_major_sf=True)
        h = ep.ep_layout(cfg, idx)
        recv = ep.alloc_recv(h)
        ep.ep_dispatch_fp8(h, n["y_fp8"], n["y_sf"], None, **recv)
        gate_up = ep.ep_expert_gemm(h, recv["recv_x"], recv["recv_sf"], self.w_in, self.w_in_sf)
        act, act_sf = ep.alloc_fp8(h, self.ffn)
        ckpt = ckpt_sf = None
        if keep:
            rows = h.rows_alloc
            ckpt = torch.empty(rows, 2 * self.ffn, dtype=torch.uint8, device="cuda")
            ckpt_sf = torch.empty(rows, 2 * self.ffn // 128, device="cuda")
        ep.ep_swiglu(h, gate_up, act_fp8=act, act_sf=act_sf, ckpt=ckpt, ckpt_sf=ckpt_sf)
        y = ep.ep_expert_gemm(h, act, act_sf, self.w_out, self.w_out_sf)
        out = ep.ep_combine(h, y, w)
        if keep:
            self.saved = (h, n, probs, w, idx, ckpt, ckpt_sf, y)
        return out, n["residual_out"]

    def backward(self, grad_out, grad_residual):
        """(gradient of x and of the residual, of gamma, of the router)."""
        h, n, probs, w, idx, ckpt, ckpt_sf, y = self.saved
        gw = torch.empty_like(w)
        gy, gy_sf = ep.alloc_fp8(h, self.hidden)
        ep.ep_combine_weighted_backward(h, grad_out, y, w, grad_y_fp8=gy, grad_y_sf=gy_sf,
                                        grad_topk_weights=gw)
        grad_act = ep.ep_expert_gemm(h, gy, gy_sf, self.w_out_t, self.w_out_t_sf)
        gh, gh_sf = ep.alloc_fp8(h, 2 * self.ffn)
        ep.ep_swiglu_backward(h, grad_act, ckpt, ckpt_sf, grad_fp8=gh, grad_sf=gh_sf)
        grad_rows = ep.ep_expert_gemm(h, gh, gh_sf, self.w_in_t, self.w_in_t_sf)
        grad_norm, _ = ep.ep_dispatch_backward(h, grad_rows)
        # the router: weights = probs at the chosen experts
        gp = torch.zeros_like(probs).scatter_(1, idx, gw)
        gl = (probs * (gp - (gp * probs).sum(1, keepdim=True))).bfloat16()
        grad_norm = grad_norm + gl @ self.router
        grad_x, grad_gamma = ep.ep_rmsnorm_backward(grad_norm, n["residual_out"], self.gamma,
                                                    n["rstd"], grad_residual)
        return grad_x, grad_gamma, gl.t() @ n["y"]


def rounded(v: torch.Tensor) -> torch.Tensor:
    """v with every 1x128 block rounded to e4m3; gradients pass through."""
    b = v.detach().view(v.shape[0], v.shape[1] // 128, 128)
    sf = (b.abs().amax(2, keepdim=True) / 448.0).clamp_min(1e-30)
    q = (b / sf).clamp(-448, 448).to(FP8).float() * sf
    return v + (q.view(v.shape) - v.detach())


def plain(m: MoeHalf, x, residual, grad_out, grad_residual, idx, eight_bit=False):
    """The same block in fp32 with autograd, on the experts' dequantised weights
    and the routing `idx`; with ``eight_bit`` the experts' inputs are rounded
    where the block holds them in 8 bits."""
    hold = rounded if eight_bit else (lambda v: v)
    xs = x.float().requires_grad_()
    gamma = m.gamma.clone().requires_grad_()
    router = m.router.float().requires_grad_()
    s = xs + residual.float()
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + m.eps) * gamma
    w = torch.softmax(y @ router.t(), dim=1).gather(1, idx)
    w_in, w_out = (dequantise_weights(*a) for a in
                   ((m.w_in, m.w_in_sf), (m.w_out, m.w_out_sf)))
    out = torch.zeros_like(s)
    for e in range(m.experts):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        g, u = (hold(y[t]) @ w_in[e].t()).chunk(2, dim=1)
        rows = hold(torch.nn.functional.silu(g) * u) @ w_out[e].t()
        out = out.index_add(0, t, rows * w[t, k, None])
    torch.autograd.backward([out, s], [grad_out.float(), grad_residual.float()])
    return {"out": out.detach(), "residual": s.detach(), "grad x": xs.grad,
            "grad gamma": gamma.grad, "grad router": router.grad}


def compare(m: MoeHalf, tokens: int, seed=1, eight_bit=False) -> dict:
    """Relative 2-norm distance of every output and gradient from the plain form."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, res, go, gr = (torch.randn((tokens, m.hidden), generator=g, device="cuda").bfloat16()
                      for _ in range(4))
    out, stream = m.forward(x, res, keep=True)
    gx, gg, gt = m.backward(go, gr)
    want = plain(m, x, res, go, gr, m.saved[4], eight_bit)
    got = {"out": out, "residual": stream, "grad x": gx, "grad gamma": gg, "grad router": gt}
    return {k: float((got[k].float() - v).norm() / v.norm()) for k, v in want.items()}


def main():
    a = argparse.ArgumentParser()
    for name, value in (("tokens", 1024), ("hidden", 1024), ("ffn", 512), ("experts", 32),
                        ("topk", 4)):
        a.add_argument("--" + name, type=int, default=value)
    a = a.parse_args()
    m = MoeHalf(a.hidden, a.ffn, a.experts, a.topk)
    for k, v in compare(m, a.tokens).items():
        print(f"{k:12s} relative error {v:.4f}")
    x, res, go, gr = (torch.randn(a.tokens, a.hidden, device="cuda").bfloat16() for _ in range(4))
    for name, step in (("forward", lambda: m.forward(x, res)),
                       ("forward and backward",
                        lambda: (m.forward(x, res, keep=True), m.backward(go, gr)))):
        for _ in range(3):
            step()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            step()
        torch.cuda.synchronize()
        print(f"{name:20s} {(time.perf_counter() - t) / 20 * 1e6:.0f} us")


if __name__ == "__main__":
    main()
