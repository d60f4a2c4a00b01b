"""GPU parity of moe_layer_few / FewTokenLayer with the layer's fp64 oracle.

Tolerances.  Routing: the layer's rule (near-ties below 1e-6 aside, equal
selections; gates within 1e-5).  Output, per token, against the oracle on the
stored weights.  fp32 layers: relative L2 1e-5, the layer's fp32 contract.
bf16 tokens: each h is rounded to bf16, at most 2^-8 of it and independently,
so y is off by less than 2^-8 of its norm; sums, y and the gates are fp32.  A
bf16 result adds at most 2^-8 of the result."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
import workloads as W
from moe_testutil import check_routing, f64_of, np_of, rel_l2
from oracle import e4m3 as E
from oracle import fp4 as F
from oracle import moe as O

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
CODE = {"f32": M.MOE_F32, "bf16": M.MOE_BF16, "e4m3": M.MOE_E4M3, "e2m1": M.MOE_E2M1}


def weights(wt, E_, d, I, seed):
    """(ExpertWeights, the fp64 values of w13 and w2)."""
    dt = BF16 if wt == "bf16" else F32
    w13 = W.make_free((E_, 2 * I, d), d ** -0.5, seed, "cuda", dt)
    w2 = W.make_free((E_, d, I), d ** -0.5, seed + 1, "cuda", dt)
    if wt in ("f32", "bf16"):
        return M.ExpertWeights(CODE[wt], w13, w2), f64_of(w13), f64_of(w2)
    w = M.quantize_weights(w13, w2) if wt == "e4m3" else M.quantize_weights_fp4(w13, w2)
    value = (lambda q, s: E.dequantize_tiles(q, s, 128, 128)) if wt == "e4m3" else F.dequantize_groups
    v = [np.stack([value(np_of(q[i]), np_of(s[i])) for i in range(E_)])
         for q, s in ((w.w13, w.w13_scale), (w.w2, w.w2_scale))]
    return w, v[0], v[1]


def inputs(wt, T, d, Nr, seed):
    u = W.make_free((T, d), 1.0, seed + 2, "cuda", F32 if wt == "f32" else BF16)
    e = W.make_free((Nr, d), d ** -0.5, seed + 3, "cuda")
    b = W.make_free((Nr,), 0.01, seed + 4, "cuda")
    return u, e, b


def check_out(out, o, resid64, bf16_tokens):
    """Each token's row: the experts' part by its own norm, plus the rounding of out."""
    ffn = o.y_shared.sum(axis=0) + np.einsum("tk,tkd->td", o.routing.gate, o.y_routed)
    want = ffn if resid64 is None else ffn + resid64
    err = np.linalg.norm(f64_of(out) - want, axis=1)
    tol = (2.0 ** -8 if bf16_tokens else 1e-5) * np.linalg.norm(ffn, axis=1) + 1e-6 * np.linalg.norm(want, axis=1)
    if out.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.linalg.norm(want, axis=1)
    assert np.all(err <= tol), (err / tol).max()


CASES = [("f32", 1, 256, 16, 1, 128, 4), ("f32", 7, 264, 20, 2, 136, 3), ("f32", 32, 64, 5, 0, 40, 5),
         ("f32", 17, 72, 65, 1, 24, 2), ("bf16", 1, 512, 16, 1, 256, 4), ("bf16", 16, 264, 33, 2, 88, 6),
         ("bf16", 32, 520, 300, 1, 72, 8), ("bf16", 3, 2048, 64, 2, 1408, 6), ("bf16", 4, 64, 1023, 1, 32, 16),
         ("bf16", 2, 8, 1, 0, 8, 1), ("e4m3", 1, 256, 16, 1, 128, 4), ("e4m3", 19, 384, 40, 1, 256, 8),
         ("e4m3", 32, 128, 8, 3, 128, 8), ("e2m1", 1, 256, 16, 1, 128, 4), ("e2m1", 5, 288, 24, 1, 160, 4),
         ("e2m1", 32, 96, 8, 2, 32, 8), ("e2m1", 20, 1024, 257, 0, 64, 7), ("e2m1", 2, 32, 3, 1, 32, 1),
         ("e4m3", 6, 256, 12, 2, 128, 5), ("bf16", 8, 512, 64, 1, 256, 6), ("bf16", 2, 64, 300, 1, 2080, 16),
         ("e2m1", 8, 128, 200, 1, 64, 8)]


@pytest.mark.parametrize("wt,T,d,Nr,Ns,I,K", CASES)
@pytest.mark.parametrize("out_t", [F32, BF16])
def test_layer(wt, T, d, Nr, Ns, I, K, out_t):
    w, v13, v2 = weights(wt, Nr + Ns, d, I, 100 + d)
    u, e, b = inputs(wt, T, d, Nr, 200 + T)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, u.dtype, w, out_dtype=out_t)
    need = layer.ws.numel()
    layer.ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")    # nothing may rest on its contents
    for t in (layer.topk_idx, layer.topk_gate, layer.topk_score, layer.expert_load, layer.out):
        t.fill_(77)
    o = O.layer_forward(f64_of(u), f64_of(e), f64_of(b), v13, v2, Nr, Ns, K)
    for flags, resid in ((0, None), (M.MOE_COMBINE_NO_RESIDUAL, None), (0, W.make_free((T, d), 1.0, 9, "cuda", BF16))):
        out = layer.forward(u, e, b, residual=resid, flags=flags)
        ok, tied = check_routing(np_of(layer.topk_idx), f64_of(layer.topk_gate), np_of(layer.expert_load), o.routing, Nr)
        assert not tied, "a near-tie: choose another seed"
        np.testing.assert_allclose(f64_of(layer.topk_score), o.routing.score, rtol=0, atol=1e-5)
        r64 = None if flags else f64_of(u if resid is None else resid)
        check_out(out, o, r64, wt != "f32")
        first = out.clone()
        assert torch.equal(layer.forward(u, e, b, residual=resid, flags=flags), first)
    assert bool((layer.ws[need:] == 0xFF).all())


def test_equal_to_the_layer_of_many_tokens():
    """The same layer through MoeLayer: the same routing, outputs within both sides' bf16 roundings."""
    T, d, Nr, Ns, I, K = 24, 1024, 32, 1, 256, 4
    w, _, _ = weights("bf16", Nr + Ns, d, I, 7)
    u, e, b = inputs("bf16", T, d, Nr, 8)
    few = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w, out_dtype=F32)
    many = M.MoeLayer(T, d, Nr, Ns, I, K, BF16, w, out_dtype=F32)
    a, c = few.forward(u, e, b), many.forward(u, e, b)
    assert torch.equal(few.topk_idx, many.topk_idx) and torch.equal(few.expert_load, many.expert_load)
    assert rel_l2(f64_of(a - u.float()), f64_of(c - u.float())) < 2 * 2.0 ** -8


@pytest.mark.parametrize("n", [0, 1, 5, 17, 20])
def test_fewer_tokens_than_the_layer_holds(n):
    T, d, Nr, Ns, I, K = 20, 256, 16, 1, 64, 3
    w, v13, v2 = weights("bf16", Nr + Ns, d, I, 17)
    u, e, b = inputs("bf16", T, d, Nr, 18)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w, out_dtype=F32)
    layer.out.fill_(77)
    layer.expert_load.fill_(77)
    out = layer.forward(u[:n], e, b)
    assert out.shape == (n, d) and bool((layer.out[n:] == 77).all())
    assert int(layer.expert_load.sum()) == n * K
    if n:
        o = O.layer_forward(f64_of(u[:n]), f64_of(e), f64_of(b), v13, v2, Nr, Ns, K)
        check_routing(np_of(layer.topk_idx[:n]), f64_of(layer.topk_gate[:n]), np_of(layer.expert_load), o.routing, Nr)
        check_out(out, o, f64_of(u[:n]), True)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_exponent_bytes_at_any_address(off):
    T, d, Nr, Ns, I, K = 3, 512, 12, 1, 256, 4
    w, _, _ = weights("e2m1", Nr + Ns, d, I, 17)
    u, e, b = inputs("e2m1", T, d, Nr, 18)
    want = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w, out_dtype=F32).forward(u, e, b).clone()
    for name in ("w13_scale", "w2_scale"):
        s = getattr(w, name)
        held = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
        held[off:off + s.numel()] = s.flatten()
        moved = M.ExpertWeights(w.w_t, w.w13, w.w2, w.w13_scale, w.w2_scale)
        setattr(moved, name, held[off:off + s.numel()].view(s.shape))
        got = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, moved, out_dtype=F32).forward(u, e, b)
        assert torch.equal(got, want)                           # the same sums in the same order


def test_ties_go_to_the_lower_index():
    for Nr in (40, 130, 700):
        d, I, K, T = 64, 32, 6, 5
        w, _, _ = weights("bf16", Nr, d, I, 27)
        u = W.make_free((T, d), 1.0, 28, "cuda", BF16)
        layer = M.FewTokenLayer(T, d, Nr, 0, I, K, BF16, w)
        e = W.make_free((1, d), d ** -0.5, 29, "cuda").expand(Nr, d).contiguous()
        b = torch.zeros((Nr,), device="cuda")
        layer.forward(u, e, b)
        assert torch.equal(layer.topk_idx.cpu(), torch.arange(K, dtype=torch.int32).expand(T, K))
        b[Nr - 3:] = 1.0                                         # the last three, then the first ones
        layer.forward(u, e, b)
        assert torch.equal(layer.topk_idx.cpu(), torch.tensor([Nr - 3, Nr - 2, Nr - 1, 0, 1, 2], dtype=torch.int32).expand(T, K))
        b[:] = float("-inf")
        b[7] = 0
        layer.forward(u, e, b)
        assert torch.equal(layer.topk_idx.cpu(), torch.tensor([7, 0, 1, 2, 3, 4], dtype=torch.int32).expand(T, K))


@pytest.mark.parametrize("wt", ["f32", "bf16", "e4m3", "e2m1"])
def test_nan_stays_with_its_token_and_expert(wt):
    T, d, Nr, Ns, I, K = 18, 256, 24, 1, 128, 3
    w, _, _ = weights(wt, Nr + Ns, d, I, 37)
    u, e, b = inputs(wt, T, d, Nr, 38)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, u.dtype, w, out_dtype=F32)
    a = layer.forward(u, e, b).clone()
    idx = layer.topk_idx.clone()
    bad_t, bad_e = 4, int(idx[9, 0])
    u2 = u.clone()
    u2[bad_t, 250] = float("nan")
    if wt in ("f32", "bf16"):
        w.w2[bad_e, 17, 3] = float("nan")
    elif wt == "e4m3":
        w.w2[bad_e, 17, 3] = 0x7F                                # E4M3's NaN
    else:
        w.w2_scale[bad_e, 17, 0] = 255
    c = layer.forward(u2, e, b)
    live = [t for t in range(T) if t != bad_t]
    assert torch.equal(layer.topk_idx[live], idx[live])          # other tokens' routing
    for row in layer.topk_idx.tolist():                          # and any routing is one of existing, distinct experts
        assert len(set(row)) == K and min(row) >= 0 and max(row) < Nr
    clean = [t for t in live if bad_e not in idx[t].tolist()]
    hit = [t for t in live if bad_e in idx[t].tolist()]
    assert clean and hit
    assert torch.equal(a[clean], c[clean])
    assert torch.isnan(c[hit, 17]).all() and torch.equal(a[hit, :17], c[hit, :17]) and torch.equal(a[hit, 18:], c[hit, 18:])
    assert torch.isnan(c[bad_t]).all()


def test_result_on_its_residual_and_on_u():
    T, d, Nr, Ns, I, K = 6, 264, 12, 1, 72, 2
    w, _, _ = weights("bf16", Nr + Ns, d, I, 47)
    u, e, b = inputs("bf16", T, d, Nr, 48)
    r = W.make_free((T, d), 1.0, 49, "cuda", F32)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w, out_dtype=F32)
    want = layer.forward(u, e, b, residual=r).clone()
    args = (layer.topk_idx, layer.topk_gate, layer.topk_score, layer.expert_load, layer.ws)
    r2 = r.clone()
    M.moe_layer_few(u, e, b, w, Ns, I, K, r2, *args, r2)
    assert torch.equal(r2, want)
    want = layer.forward(u, e, b).bfloat16()
    u2 = u.clone()
    M.moe_layer_few(u2, e, b, w, Ns, I, K, u2, *args, u2)
    assert torch.equal(u2, want)


@pytest.mark.parametrize("wt", ["e2m1", "e4m3"])
def test_graph_replays(wt):
    """One captured call, replayed with new tokens and with eager work between, against eager calls."""
    T, d, Nr, Ns, I, K = 4, 512, 32, 1, 128, 4
    w, _, _ = weights(wt, Nr + Ns, d, I, 57)
    u, e, b = inputs(wt, T, d, Nr, 58)
    layer, eager = (M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w) for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        layer.forward(u, e, b)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(u, e, b)
    for i in range(6):
        u.copy_(W.make_free((T, d), 1.0, 60 + i, "cuda", BF16))
        want = eager.forward(u, e, b).clone()
        if i % 2:
            torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want) and torch.equal(layer.topk_idx, eager.topk_idx)
        assert torch.equal(layer.expert_load, eager.expert_load)


def test_on_another_stream():
    T, d, Nr, Ns, I, K = 3, 256, 16, 1, 64, 4
    w, _, _ = weights("bf16", Nr + Ns, d, I, 67)
    u, e, b = inputs("bf16", T, d, Nr, 68)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, BF16, w)
    want = layer.forward(u, e, b).clone()
    st = torch.cuda.Stream()
    u2 = torch.zeros_like(u)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        u2.copy_(u)
        out = layer.forward(u2, e, b)
    st.synchronize()
    assert torch.equal(out, want)


def test_experts_past_32_bit_offsets():
    """W13 of 3.8e9 bytes: the last experts' results against the oracle."""
    T, d, Nr, I, K = 2, 7168, 256, 2048, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    w = M.ExpertWeights(M.MOE_E2M1, rnd(Nr, 2 * I, d // 2), rnd(Nr, d, I // 2),
                        torch.full((Nr, 2 * I, d // 32), 119, dtype=torch.uint8, device="cuda"),
                        torch.full((Nr, d, I // 32), 119, dtype=torch.uint8, device="cuda"))
    u, e, b = inputs("e2m1", T, d, Nr, 78)
    b[-2:] = 10.0
    layer = M.FewTokenLayer(T, d, Nr, 0, I, K, BF16, w, out_dtype=F32)
    out = layer.forward(u, e, b, flags=M.MOE_COMBINE_NO_RESIDUAL)
    assert sorted(layer.topk_idx[0].tolist()) == [254, 255]
    v13 = [F.dequantize_groups(np_of(w.w13[i]), np_of(w.w13_scale[i])) for i in (254, 255)]
    v2 = [F.dequantize_groups(np_of(w.w2[i]), np_of(w.w2_scale[i])) for i in (254, 255)]
    r = O.route(f64_of(u), f64_of(e), f64_of(b), K)
    for t in range(T):
        want = sum(r.gate[t, k] * O.swiglu_ffn(f64_of(u[t:t + 1]), v13[r.idx[t, k] - 254], v2[r.idx[t, k] - 254])[0][0]
                   for k in range(K))
        assert rel_l2(f64_of(out[t]), want) < 2.0 ** -8


def test_bias_step():
    T, d, Nr, Ns, I, K = 8, 64, 16, 0, 32, 4
    w, _, _ = weights("f32", Nr, d, I, 87)
    u, e, b = inputs("f32", T, d, Nr, 88)
    layer = M.FewTokenLayer(T, d, Nr, Ns, I, K, F32, w)
    layer.forward(u[:6], e, b)
    want = O.bias_update(np_of(b), np_of(layer.expert_load), 6, K)
    layer.update_bias(b, tokens=6)
    assert np.array_equal(np_of(b).view(np.uint32), want.view(np.uint32))
