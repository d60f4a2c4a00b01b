"""The example's decode step and training step against the oracles, step by
step: each call's result is compared with the fp64 formulas on what the step
before it left on the GPU, so every tolerance is that of one operator."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
import workloads as W
from examples import pre_norm_block as X
from moe_testutil import f64_of, np_of, rel_l2
from oracle import fp4 as F
from oracle import moe as O
from oracle import norm as N

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 3, 20])
def test_decode_step(T):
    cfg = W.CONFIGS["mid_bf16"].with_(d=512, Nr=16, Ns=1, I=256, K=4)
    step = X.make_decode(cfg, T, vocab=1000)
    x, stream = W.make_free((T, cfg.d), 1.0, 10, "cuda", torch.bfloat16), W.make_free((T, cfg.d), 2.0, 11, "cuda")
    r0, x0 = f64_of(stream), f64_of(x)
    logits = step.forward(x, stream)
    w = step.layer.w
    v13, v2 = (np.stack([F.dequantize_groups(np_of(q[i]), np_of(s[i])) for i in range(cfg.E)])
               for q, s in ((w.w13, w.w13_scale), (w.w2, w.w2_scale)))
    r1, _, u1 = N.rmsnorm(x0, r0, f64_of(step.w1), X.EPS)
    u1 = torch.from_numpy(u1).float().bfloat16()                       # u is handed on in bf16
    o = O.layer_forward(f64_of(u1), f64_of(step.centroids), f64_of(step.bias), v13, v2, cfg.Nr, cfg.Ns, cfg.K)
    assert o.routing.boundary_gap.min() > 1e-3                         # the roundings of u cannot change the selection
    assert np.array_equal(np.sort(np_of(step.layer.topk_idx), 1), np.sort(o.routing.idx, 1))
    want = r1 + o.out - f64_of(u1)
    # u and h are each rounded to bf16, 2^-8 of a value at most, independently: below 2 x 2^-8 of the experts' part
    assert np.linalg.norm(f64_of(stream) - want) < 2 * 2.0 ** -8 * np.linalg.norm(want - r1)
    _, _, u2 = N.rmsnorm(f64_of(stream), None, f64_of(step.w2), X.EPS)
    head = F.dequantize_groups(np_of(step.head_q), np_of(step.head_scale))
    assert rel_l2(f64_of(logits), u2 @ head.T) < 2.0 ** -8             # u in bf16, the product exact to fp32


def test_training_step():
    cfg = W.CONFIGS["mid_bf16"].with_(T=96, d=512, Nr=16, Ns=1, I=256, K=4)
    step = X.make_train(cfg)
    x, stream, G = (W.make_free((cfg.T, cfg.d), 1.0, 12 + i, "cuda", torch.bfloat16) for i in range(3))
    out = step.forward(x, stream).clone()
    r64, c64, u64 = N.rmsnorm(f64_of(x), f64_of(stream), f64_of(step.w), X.EPS)
    assert rel_l2(f64_of(step.u), u64) < 2.0 ** -8
    # the layer on the norm's own u and tiles: exactly the layer that quantises those tiles' values again
    ref = M.MoeLayer(cfg.T, cfg.d, cfg.Nr, cfg.Ns, cfg.I, cfg.K, torch.bfloat16, step.layer.w, x_fp8=True, train=True)
    ref.route(step.u, step.centroids, step.bias)
    ref.permute()
    ref.xq.copy_(step.layer.xq)
    ref.xs.copy_(step.layer.xs)
    ref.experts(step.u, tiles_ready=True)
    assert torch.equal(ref.combine(step.u), out)
    dx, dw, de, dw13, dw2 = step.backward(G)
    du = ref.backward(G, step.u, step.centroids)[0]
    assert torch.equal(step.layer.du, du)
    want_dx, want_dw = N.rmsnorm_backward(f64_of(du), f64_of(step.r), f64_of(step.w), f64_of(step.rstd))
    assert rel_l2(f64_of(dx), want_dx) < 2.0 ** -8                     # one bf16 rounding
    assert rel_l2(f64_of(dw), want_dw) < 1e-5                          # fp32 sums over 96 rows
    assert np.isfinite(f64_of(dw13)).all() and np.isfinite(f64_of(dw2)).all() and np.isfinite(f64_of(de)).all()


def test_tiles_ready_needs_tiles():
    cfg = W.CONFIGS["tiny_fp32"]
    w13, w2 = W.make_expert_weights(cfg, "cuda")
    layer = M.MoeLayer(cfg.T, cfg.d, cfg.Nr, cfg.Ns, cfg.I, cfg.K, torch.float32, M.ExpertWeights(M.MOE_F32, w13, w2))
    with pytest.raises(ValueError):
        layer.forward(W.make_tokens(cfg, 0, "cuda"), W.make_centroids(cfg, "cuda"), W.make_bias(cfg, "cuda"),
                      tiles_ready=True)
