"""GPU parity of moe_rmsnorm and moe_rmsnorm_backward with the fp64 oracle.

Tolerances.  eps32 = 2^-24 is the relative error of one fp32 operation.  A
row's sum of squares is a chain of at most 32 fused adds, a 6-step and a
16-step tree: 54 roundings; the division, the root, the reciprocal and the
products add fewer than 10: every fp32 result is within 64 eps32 of the sum
of its terms' magnitudes.  A bf16 result is off by another half unit in the
last place: bf16 has 8 significant bits, so that is 2^-9 of the power of two
just above its magnitude."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
import workloads as W
from moe_testutil import f64_of
from oracle import e4m3 as E
from oracle import norm as N

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SLOP = 64 * 2.0 ** -24
EPS = 1e-6


def out_tol(dtype, mag, value):
    tol = SLOP * mag
    if dtype == BF16:
        tol = tol + np.ldexp(2.0 ** -9, np.frexp(np.abs(value) + tol)[1])
    return tol


def make(T, d, xt, rt, wt, seed):
    x = W.make_free((T, d), 1.0, seed, "cuda", xt)
    resid = None if rt is None else W.make_free((T, d), 2.0, seed + 1, "cuda", rt)
    w = (1 + W.make_free((d,), 0.2, seed + 2, "cuda")).to(wt)
    return x, resid, w


def check_tiles(q, scale, u64):
    """Codes and power-of-two scales of u in 1x128 tiles: the rule of fp8_quantize_tiles up to fp32 rounding of u."""
    T, d = u64.shape
    sc = f64_of(scale)
    amax = np.abs(u64).reshape(T, d // 128, 128).max(axis=2)
    m, _ = np.frexp(sc)
    assert np.all(m == 0.5)
    nz = amax > 0
    assert np.all(amax[nz] * (1 - SLOP) <= 448 * sc[nz]) and np.all(amax[nz] * (1 + SLOP) > 224 * sc[nz])
    assert np.all(sc[~nz] == 1.0)
    full = np.repeat(sc, 128, axis=1)
    got = E.e4m3_decode(q.cpu().numpy()) * full
    # half a code step: 2^-4 of the value, or 2^-10 of the scale among the subnormal codes
    assert np.all(np.abs(got - u64) <= np.maximum(2.0 ** -4 * np.abs(u64), 2.0 ** -10 * full) * (1 + SLOP) + SLOP * np.abs(u64))


@pytest.mark.parametrize("T,d", [(1, 8), (3, 24), (1, 7168), (5, 512), (5, 520), (7, 1016), (130, 2048), (9, 2056),
                                 (3, 8192), (2, 8200), (1, 32768), (2, 30000), (5003, 264)])
@pytest.mark.parametrize("xt,rt,wt,ut", [(BF16, BF16, F32, BF16), (F32, None, BF16, F32), (BF16, F32, BF16, F32),
                                         (F32, BF16, F32, BF16), (BF16, None, F32, BF16), (F32, F32, F32, F32)])
def test_forward(T, d, xt, rt, wt, ut):
    x, resid, w = make(T, d, xt, rt, wt, 3 * d + T)
    u = torch.full((T, d), 7.0, dtype=ut, device="cuda")
    r_out = None if rt is None else torch.full((T, d), 7.0, dtype=rt, device="cuda")
    rstd = torch.full((T,), 7.0, device="cuda")
    M.moe_rmsnorm(x, w, EPS, resid, r_out, u, rstd=rstd)
    r64, c64, u64 = N.rmsnorm(f64_of(x), None if resid is None else f64_of(resid), f64_of(w), EPS)
    assert np.all(np.abs(f64_of(u) - u64) <= out_tol(ut, np.abs(u64), u64))
    assert np.all(np.abs(f64_of(rstd) - c64) <= SLOP * c64)
    if rt is not None:
        assert np.all(np.abs(f64_of(r_out) - r64) <= out_tol(rt, np.abs(r64), r64))


@pytest.mark.parametrize("T,d", [(1, 128), (3, 640), (33, 2048), (2, 7168), (17, 7168), (3, 8320), (1, 32768)])
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (F32, F32), (BF16, None)])
@pytest.mark.parametrize("with_u", [True, False])
def test_forward_tiles(T, d, xt, rt, with_u):
    x, resid, w = make(T, d, xt, rt, F32, d + T)
    if T > 2:
        x[1] = 0                                                # a row of zeros: codes 0, scale 1
        if resid is not None:
            resid[1] = 0
    x[0, :128] *= 2.0 ** -20                                    # a tile far below the others
    u = torch.empty((T, d), dtype=BF16, device="cuda") if with_u else None
    q = torch.full((T, d), 0x55, dtype=torch.uint8, device="cuda")
    qs = torch.full((T, d // 128), 7.0, device="cuda")
    M.moe_rmsnorm(x, w, EPS, resid, u=u, q=q, q_scale=qs)
    _, _, u64 = N.rmsnorm(f64_of(x), None if resid is None else f64_of(resid), f64_of(w), EPS)
    check_tiles(q, qs, u64)
    if with_u:
        assert np.all(np.abs(f64_of(u) - u64) <= out_tol(BF16, np.abs(u64), u64))


def test_fp32_tiles_are_those_of_the_quantiser():
    """With u kept in fp32, its tiles are fp8_quantize_tiles' of it, bit for bit."""
    T, d = 37, 1152
    x, resid, w = make(T, d, F32, F32, F32, 5)
    u = torch.empty((T, d), device="cuda")
    q, qs = torch.empty((T, d), dtype=torch.uint8, device="cuda"), torch.empty((T, d // 128), device="cuda")
    M.moe_rmsnorm(x, w, EPS, resid, u=u, q=q, q_scale=qs)
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    M.fp8_quantize_tiles(u, 1, q2, qs2)
    assert torch.equal(q, q2) and torch.equal(qs, qs2)


def test_rows_do_not_touch_each_other():
    """Infinities, NaN and overflowing squares stay in their row, and follow the formula there."""
    T, d = 9, 2056
    x, resid, w = make(T, d, F32, F32, F32, 11)
    u0, u1 = (torch.empty((T, d), device="cuda") for _ in range(2))
    M.moe_rmsnorm(x, w, EPS, resid, u=u0)
    x[1, 5], x[3, 7], x[4], x[6] = float("inf"), float("nan"), 1e30, 0
    resid[6] = 0
    M.moe_rmsnorm(x, w, EPS, resid, u=u1)
    same = [0, 2, 5, 7, 8]
    assert torch.equal(u0[same], u1[same])
    assert torch.isnan(u1[1, 5]) and not u1[1, :5].any()        # inf * (1 / inf), and finite / inf
    assert torch.isnan(u1[3]).all()
    assert not u1[4].any()                                      # the sum of squares is infinite
    assert not u1[6].any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_results_on_their_operands(dt):
    T, d = 600, 1032
    x, resid, w = make(T, d, dt, dt, F32, 21)
    u, r = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty((T,), device="cuda")
    M.moe_rmsnorm(x, w, EPS, resid, r, u, rstd=rstd)
    x1, resid1 = x.clone(), resid.clone()
    M.moe_rmsnorm(x1, w, EPS, resid1, resid1, x1)
    assert torch.equal(x1, u) and torch.equal(resid1, r)
    ws = torch.empty((M.moe_rmsnorm_backward_workspace_bytes(T, d),), dtype=torch.uint8, device="cuda")
    du, dr = W.make_free((T, d), 1.0, 22, "cuda", dt), W.make_free((T, d), 1.0, 23, "cuda", dt)
    dx, dw, dw1 = torch.empty_like(r), torch.empty((d,), device="cuda"), torch.empty((d,), device="cuda")
    M.moe_rmsnorm_backward(du, r, w, rstd, dr, dx, dw, ws)
    dr1, du1 = dr.clone(), du.clone()
    M.moe_rmsnorm_backward(du, r, w, rstd, dr1, dr1, dw1, ws)
    assert torch.equal(dr1, dx) and torch.equal(dw1, dw)
    M.moe_rmsnorm_backward(du1, r, w, rstd, dr, du1, dw1, ws)
    assert torch.equal(du1, dx) and torch.equal(dw1, dw)


@pytest.mark.parametrize("T,d", [(1, 8), (1, 7168), (2, 512), (70, 520), (2500, 256), (530, 2048), (9, 2056), (600, 7168),
                                 (3, 8200), (700, 16384), (2, 32768)])
@pytest.mark.parametrize("gt,rt,wt,with_dr", [(BF16, F32, F32, True), (BF16, BF16, BF16, True), (F32, BF16, F32, False),
                                              (F32, F32, BF16, False)])
def test_backward(T, d, gt, rt, wt, with_dr):
    r, _, w = make(T, d, rt, None, wt, 7 * d + T)
    du = W.make_free((T, d), 1.0, d + 1, "cuda", gt)
    dr = W.make_free((T, d), 1.0, d + 2, "cuda", rt) if with_dr else None
    rstd = torch.rsqrt(r.float().square().mean(dim=1) + EPS)
    need = M.moe_rmsnorm_backward_workspace_bytes(T, d)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN, and a guard behind it
    dx = torch.full((T, d), 7.0, dtype=rt, device="cuda")
    dw, dw2 = torch.full((d,), 7.0, device="cuda"), torch.empty((d,), device="cuda")
    M.moe_rmsnorm_backward(du, r, w, rstd, dr, dx, dw, ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    r64, w64, c, g64 = f64_of(r), f64_of(w), f64_of(rstd), f64_of(du)
    dx64, dw64 = N.rmsnorm_backward(g64, r64, w64, c, None if dr is None else f64_of(dr))
    gx = np.abs(g64 * w64 * r64 * c[:, None])
    mag = c[:, None] * (np.abs(g64 * w64) + np.abs(r64) * c[:, None] * gx.mean(axis=1, keepdims=True))
    mag = mag + (0 if dr is None else np.abs(f64_of(dr)))
    assert np.all(np.abs(f64_of(dx) - dx64) <= out_tol(rt, mag, dx64))
    # dw_j: three roundings a term, and a chain over rows and row groups no longer than T + 16
    tol = (T + 20) * 2.0 ** -24 * np.abs(g64 * r64 * c[:, None]).sum(axis=0)
    assert np.all(np.abs(f64_of(dw) - dw64) <= tol)
    M.moe_rmsnorm_backward(du, r, w, rstd, dr, dx, dw2, ws[:need])
    assert torch.equal(dw, dw2)


def test_forward_and_backward_against_differences():
    """The GPU gradient of sum(G u) against differences of the fp64 formula at the same fp32 inputs."""
    T, d = 3, 40
    x, resid, w = make(T, d, F32, F32, F32, 31)
    G = W.make_free((T, d), 1.0, 32, "cuda")
    u, r, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty((T,), device="cuda")
    M.moe_rmsnorm(x, w, 1e-3, resid, r, u, rstd=rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty((M.moe_rmsnorm_backward_workspace_bytes(T, d),), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(G, r, w, rstd, None, dx, dw, ws)
    x64, r64, w64, g64 = (f64_of(t) for t in (x, resid, w, G))
    loss = lambda x, w: np.sum(g64 * N.rmsnorm(x, r64, w, 1e-3)[2])  # noqa: E731
    h = 1e-5
    for t, j in [(0, 0), (1, 17), (2, 39)]:
        e = np.zeros((T, d))
        e[t, j] = h
        # fp32 rounding of r, c and the terms (each below 10): 64 eps32 x 30; the quotient: 1e-7
        assert abs((loss(x64 + e, w64) - loss(x64 - e, w64)) / (2 * h) - f64_of(dx)[t, j]) < 64 * 2.0 ** -24 * 30 + 1e-7
    e = np.zeros(d)
    e[5] = h
    assert abs((loss(x64, w64 + e) - loss(x64, w64 - e)) / (2 * h) - f64_of(dw)[5]) < 64 * 2.0 ** -24 * 30 + 1e-7


def test_no_rows():
    w, e = torch.ones((256,), device="cuda"), torch.empty((0, 256), device="cuda")
    M.moe_rmsnorm(e, w, EPS, u=torch.empty((0, 256), device="cuda"))
    dw = torch.full((256,), 7.0, device="cuda")
    M.moe_rmsnorm_backward(e, e, w, torch.empty((0,), device="cuda"), None, e, dw, None)
    assert not dw.any()


def test_past_32_bit_offsets():
    T, d = 300_000, 7168                                        # 2.15e9 elements
    x = torch.empty((T, d), dtype=BF16, device="cuda")
    tail = W.make_free((3, d), 1.0, 41, "cuda", BF16)
    x[-3:] = tail
    x[:-3] = 1.0
    w = torch.ones((d,), device="cuda")
    M.moe_rmsnorm(x, w, EPS, u=x)
    want = N.rmsnorm(f64_of(tail), None, np.ones(d), EPS)[2]
    assert np.all(np.abs(f64_of(x[-3:]) - want) <= out_tol(BF16, np.abs(want), want))
    assert bool((x[:2] == 1.0).all()) and bool((x[150_000] == 1.0).all())


def test_more_rows_than_one_launch_has_threads_for():
    T, d = (1 << 26) + 1003, 8                                  # 64 threads to a row: past 2^32 of them
    x = torch.ones((T, d), dtype=BF16, device="cuda")
    tail = W.make_free((1100, d), 1.0, 61, "cuda", BF16)
    x[-1100:] = tail
    w = torch.ones((d,), device="cuda")
    u, rstd = torch.zeros_like(x), torch.zeros((T,), device="cuda")
    M.moe_rmsnorm(x, w, EPS, u=u, rstd=rstd)
    want = N.rmsnorm(f64_of(tail), None, np.ones(d), EPS)[2]
    assert np.all(np.abs(f64_of(u[-1100:]) - want) <= out_tol(BF16, np.abs(want), want))
    assert bool((u[:-1100] == 1.0).all()) and bool((rstd > 0).all())


def test_on_another_stream():
    T, d = 64, 1024
    st = torch.cuda.Stream()
    x, resid, w = make(T, d, BF16, BF16, F32, 51)
    want, got = torch.empty_like(x), torch.empty_like(x)
    M.moe_rmsnorm(x, w, EPS, resid, u=want)
    x2 = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        x2.copy_(x)                                             # the call must follow this on st
        M.moe_rmsnorm(x2, w, EPS, resid, u=got)
    st.synchronize()
    assert torch.equal(got, want)
