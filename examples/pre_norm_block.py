"""A normed expert layer, served and trained: the norm, the layer and the
4-bit products as a program uses them together.

    python examples/pre_norm_block.py            # needs an MI355X and the built library

DecodeStep: one step of a few sequences (or drafted tokens).  The attention's
output x joins the residual stream, the norm of the stream goes through the
expert layer with 4-bit experts, which adds its result to the stream, and the
final norm through a 4-bit output head:
    r = r + x,  r = r + MoE(norm(r) w1),  logits = Head(norm(r) w2)

TrainStep: the E4M3 training step of one layer behind its norm.  The norm
writes u and u's E4M3 tiles in one pass, the expert products take the tiles
as they are, and the layer's input gradient goes on through the norm:
    u = norm(r + x) w,  h' = u + MoE(u)
"""
from __future__ import annotations

import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_expert_routing_sigmoid_amd as M  # noqa: E402
import workloads as W  # noqa: E402

EPS = 1e-6


class DecodeStep:
    """Weights and buffers of one decode step of T tokens; forward() returns the logits [T, vocab] (fp32)."""

    def __init__(self, T, cfg: W.LayerConfig, experts: M.ExpertWeights, centroids, bias, w1, w2, head_q, head_scale):
        dev = centroids.device
        self.centroids, self.bias, self.w1, self.w2 = centroids, bias, w1, w2
        self.head_q, self.head_scale = head_q, head_scale
        self.layer = M.FewTokenLayer(T, cfg.d, cfg.Nr, cfg.Ns, cfg.I, cfg.K, torch.bfloat16, experts,
                                     out_dtype=torch.float32, device=dev)
        self.u = torch.empty((T, cfg.d), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((T, head_q.shape[0]), dtype=torch.float32, device=dev)
        self.ws = torch.empty((max(M.fp4_matvec_workspace_bytes(T, head_q.shape[0], cfg.d), 1),), dtype=torch.uint8,
                              device=dev)

    def forward(self, x, stream):
        """x [T, d] bf16, the residual stream [T, d] fp32 (updated in place)."""
        M.moe_rmsnorm(x, self.w1, EPS, residual=stream, r_out=stream, u=self.u)
        stream.copy_(self.layer.forward(self.u, self.centroids, self.bias, residual=stream))
        M.moe_rmsnorm(stream, self.w2, EPS, u=self.u)
        M.fp4_matvec(self.u, self.head_q, self.head_scale, self.logits, self.ws)
        return self.logits


class TrainStep:
    """One E4M3 training step of a layer behind its norm."""

    def __init__(self, cfg: W.LayerConfig, experts: M.ExpertWeights, centroids, bias, w, tile_m=32):
        T, d, dev = cfg.T, cfg.d, centroids.device
        self.centroids, self.bias, self.w = centroids, bias, w
        self.layer = M.MoeLayer(T, d, cfg.Nr, cfg.Ns, cfg.I, cfg.K, torch.bfloat16, experts, x_fp8=True, tile_m=tile_m,
                                device=dev, train=True)
        self.r = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
        self.u = torch.empty_like(self.r)
        self.dx = torch.empty_like(self.r)
        self.rstd = torch.empty((T,), dtype=torch.float32, device=dev)
        self.dw = torch.empty((d,), dtype=torch.float32, device=dev)
        self.ws = torch.empty((max(M.moe_rmsnorm_backward_workspace_bytes(T, d), 1),), dtype=torch.uint8, device=dev)

    def forward(self, x, stream):
        M.moe_rmsnorm(x, self.w, EPS, residual=stream, r_out=self.r, u=self.u, q=self.layer.xq, q_scale=self.layer.xs,
                      rstd=self.rstd)
        return self.layer.forward(self.u, self.centroids, self.bias, tiles_ready=True)

    def backward(self, grad_out):
        """(dx, dw of the norm, de, dW13, dW2) for dL/dh' = grad_out; dx is the gradient of x and of the stream."""
        du, de, dw13, dw2 = self.layer.backward(grad_out, self.u, self.centroids)
        M.moe_rmsnorm_backward(du, self.r, self.w, self.rstd, None, self.dx, self.dw, self.ws)
        return self.dx, self.dw, de, dw13, dw2


def make_decode(cfg: W.LayerConfig, T, vocab, device="cuda"):
    w13, w2 = W.make_expert_weights(cfg.with_(weights="f32"), device)
    experts = M.quantize_weights_fp4(w13, w2)
    head = W.make_free((vocab, cfg.d), cfg.d ** -0.5, 1, device)
    q = torch.empty((vocab, cfg.d // 2), dtype=torch.uint8, device=device)
    s = torch.empty((vocab, cfg.d // 32), dtype=torch.uint8, device=device)
    M.fp4_quantize_groups(head, q, s)
    norm = [1 + W.make_free((cfg.d,), 0.1, 2 + i, device) for i in range(2)]
    return DecodeStep(T, cfg, experts, W.make_centroids(cfg, device), W.make_bias(cfg, device), *norm, q, s)


def make_train(cfg: W.LayerConfig, device="cuda"):
    w13, w2 = W.make_expert_weights(cfg.with_(weights="f32"), device)
    return TrainStep(cfg, M.quantize_weights(w13, w2), W.make_centroids(cfg, device), W.make_bias(cfg, device),
                     1 + W.make_free((cfg.d,), 0.1, 2, device))


def main():
    cfg = W.CONFIGS["mid_bf16"].with_(I=1280)            # the middle layer, at a multiple of the E4M3 step's 256
    for T in (1, 8, 32):
        step = make_decode(cfg, T, vocab=32768)
        x = W.make_free((T, cfg.d), 1.0, 10, "cuda", torch.bfloat16)
        stream = W.make_free((T, cfg.d), 1.0, 11, "cuda")
        step.forward(x, stream)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(50):
            step.forward(x, stream)
        torch.cuda.synchronize()
        print(f"decode, {T} tokens: {(time.perf_counter() - t) / 50 * 1e6:.0f} us a step, "
              f"greedy tokens {step.logits.argmax(dim=1).tolist()[:8]}", flush=True)
    step = make_train(cfg)
    x, stream, grad = (W.make_free((cfg.T, cfg.d), 1.0, 12 + i, "cuda", torch.bfloat16) for i in range(3))
    for i in range(3):
        t = time.perf_counter()
        out = step.forward(x, stream)
        dx = step.backward(grad)[0]
        torch.cuda.synchronize()
        print(f"training step of {cfg.T} tokens: {(time.perf_counter() - t) * 1e3:.2f} ms, |h'| {out.float().norm():.4e}, "
              f"|dx| {dx.float().norm():.4e}", flush=True)


if __name__ == "__main__":
    main()
