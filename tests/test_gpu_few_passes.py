"""moe_layer_few where an expert has more tokens than one tile holds (8 of
E4M3 weights and 4 of E2M1 weights in the packed form, which runs for T K <=
2 Nr; else 16): the turns of a tile against the layer's fp64 oracle, by the
tolerances of test_gpu_few."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
import workloads as W
from moe_testutil import check_routing, f64_of, np_of
from oracle import moe as O
from test_gpu_few import check_out, inputs, weights

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def run(wt, T, d, Nr, Ns, I, K, b_add=None, seed=0):
    w, v13, v2 = weights(wt, Nr + Ns, d, I, 300 + seed)
    u, e, b = inputs(wt, T, d, Nr, 400 + seed)
    if b_add is not None:
        b += b_add
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, u.dtype, w, out_dtype=F32)
    layer.ws.fill_(0xFF)
    out = layer.forward(u, e, b)
    o = O.layer_forward(f64_of(u), f64_of(e), f64_of(b), v13, v2, Nr, Ns, K)
    ok, tied = check_routing(np_of(layer.topk_idx), f64_of(layer.topk_gate), np_of(layer.expert_load), o.routing, Nr)
    assert not tied, "a near-tie: choose another seed"
    check_out(out, o, f64_of(u), wt != "f32")
    first = out.clone()
    assert torch.equal(layer.forward(u, e, b), first)
    return layer, (u, e, b), first


@pytest.mark.parametrize("wt,T,d,Nr,Ns,I,K", [("e4m3", 32, 256, 128, 1, 128, 8), ("e4m3", 9, 128, 64, 2, 256, 4),
                                              ("e4m3", 17, 384, 130, 1, 128, 5), ("e2m1", 32, 256, 128, 1, 128, 8),
                                              ("e2m1", 5, 128, 64, 2, 256, 4), ("e2m1", 13, 384, 130, 3, 128, 5),
                                              ("e2m1", 32, 96, 128, 1, 160, 8), ("e2m1", 8, 128, 16, 1, 128, 2),
                                              ("bf16", 32, 128, 64, 2, 72, 4), ("f32", 31, 72, 64, 1, 40, 4)])
def test_shared_experts_of_several_turns(wt, T, d, Nr, Ns, I, K):
    run(wt, T, d, Nr, Ns, I, K, seed=T)


@pytest.mark.parametrize("wt", ["e4m3", "e2m1", "bf16", "f32"])
@pytest.mark.parametrize("T,Nr,K", [(32, 32, 2), (20, 64, 3), (9, 40, 4), (8, 16, 2), (5, 16, 2), (31, 300, 16)])
def test_routed_experts_of_several_turns(wt, T, Nr, K):
    """A bias takes every token to the same K experts, the first, the last and those between."""
    add = torch.zeros((Nr,), device="cuda")
    add[[i * (Nr - 1) // (K - 1) for i in range(K)]] = 10.0
    layer, _, _ = run(wt, T, 256, Nr, 1, 128, K, add, seed=T + K)
    assert sorted(set(layer.expert_load.tolist())) == [0, T]


@pytest.mark.parametrize("wt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("bad", [0, 3, 4, 8, 30])
def test_a_nan_token_of_another_turn_stays_alone(wt, bad):
    T, d, Nr, Ns, I, K = 31, 256, 128, 1, 128, 8
    layer, (u, e, b), a = run(wt, T, d, Nr, Ns, I, K, seed=7)
    idx = layer.topk_idx.clone()
    u2 = u.clone()
    u2[bad, 5] = float("nan")
    c = layer.forward(u2, e, b)
    live = [t for t in range(T) if t != bad]
    assert torch.equal(layer.topk_idx[live], idx[live])
    assert torch.equal(c[live], a[live]) and torch.isnan(c[bad]).all()
