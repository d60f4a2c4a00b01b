"""GPU parity of the 4-bit calls with the fp64 oracle: codes and values bit
for bit, products within a derived bound.

Products: every term x w is exact in fp32 (8 by 2 significant bits).  A wave
adds the terms of every 8th step of 128 columns, the 8 waves' sums are added
at the end, so no chain of additions is longer than
ceil(K / 1024) 128 + 8; each may lose one unit in the last place of a partial
sum, 2^-23 of the sum of the terms' magnitudes.  bf16 results: another half
unit in the last place (2^-9 of the power of two above the magnitude)."""
import numpy as np
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
import workloads as W
from moe_testutil import f64_of
from oracle import fp4 as F

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def codes(rows, cols, seed, lo=120, hi=130):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(lo, hi, (rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
    return q, s


def quantized(x):
    q = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0x55, dtype=torch.uint8, device="cuda")
    M.fp4_quantize_groups(x, q, s)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (37, 2048), (1, 7168)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_quantize(rows, cols, dt):
    x = W.make_free((rows, cols), 1.0, rows + cols, "cuda", dt)
    x[:, ::32] *= torch.exp2(torch.randint(-8, 8, x[:, ::32].shape, device="cuda").float()).to(dt)
    x[-1, -32:] = 0
    x[-1, -1] = -0.0
    q, s = quantized(x)
    q64, s64 = F.quantize_groups(f64_of(x))
    assert np.array_equal(s.cpu().numpy(), s64) and np.array_equal(q.cpu().numpy(), q64)


def test_quantize_ties_and_extremes():
    rows = []
    for base in (1.0, 2.0 ** -126, 2.0 ** -100, 2.0 ** 120):
        r = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6,
                          0.2500001, 0.7499999, 5.0000005, 4.9999995] + [0.0] * 12, dtype=torch.float64) * base
        rows.append(r)
    rows.append(torch.full((32,), 2.0 ** -149, dtype=torch.float64))       # the smallest fp32
    rows.append(torch.full((32,), -3.4028234663852886e38, dtype=torch.float64))
    x = torch.stack(rows).float().cuda()
    q, s = quantized(x)
    q64, s64 = F.quantize_groups(f64_of(x))
    assert np.array_equal(s.cpu().numpy(), s64) and np.array_equal(q.cpu().numpy(), q64)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_quantize_infinities_and_nan(dt, bad):
    x = W.make_free((3, 256), 1.0, 5, "cuda", dt)
    for r, c in ((0, 0), (1, 77), (2, 255)):
        x[r, c] = bad
    q, s = quantized(x)
    q64, s64 = F.quantize_groups(f64_of(x))
    assert np.array_equal(s.cpu().numpy(), s64) and np.array_equal(q.cpu().numpy(), q64)
    back = torch.empty_like(x)
    M.fp4_dequantize_groups(q, s, back)
    nan = torch.isnan(back).reshape(3, 8, 32)
    assert torch.equal(nan.all(dim=2), nan.any(dim=2)) and nan.any(dim=2).sum() == 3
    assert bool(nan[0, 0].all() and nan[1, 2].all() and nan[2, 7].all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_dequantize_every_code_and_scale(dt):
    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)         # [256, 512 columns]
    s = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 16).contiguous()
    out = torch.empty((256, 512), dtype=dt, device="cuda")
    M.fp4_dequantize_groups(q, s, out)
    want = F.dequantize_groups(q.cpu().numpy(), s.cpu().numpy())
    got = f64_of(out)
    assert np.array_equal(got[:253], want[:253])            # 6 * 2^125 is the last that fits
    assert np.isnan(got[255]).all()


def check(x, q, s, y):
    x64, w = f64_of(x), F.dequantize_groups(q.cpu().numpy(), s.cpu().numpy())
    K = x64.shape[1]
    want = x64 @ w.T
    tol = (-(-K // 1024) * 128 + 8) * 2.0 ** -23 * (np.abs(x64) @ np.abs(w).T)
    if y.dtype == BF16:
        tol = tol + np.ldexp(2.0 ** -9, np.frexp(np.abs(want) + tol)[1])
    assert np.all(np.abs(f64_of(y) - want) <= tol)


@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("N,K", [(1, 32), (15, 64), (16, 128), (17, 160), (1409, 1408), (250, 7168), (4099, 1056)])
@pytest.mark.parametrize("yt", [F32, BF16])
def test_matvec(T, N, K, yt):
    x = W.make_free((T, K), 1.0, T + N, "cuda", BF16)
    q, s = codes(N, K, T * N + K)
    need = M.fp4_matvec_workspace_bytes(T, N, K)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    guard = torch.full((T * N + 64,), 7.0, dtype=yt, device="cuda")
    y = guard[: T * N].view(T, N)
    M.fp4_matvec(x, q, s, y, ws[:need] if need else None)
    check(x, q, s, y)
    assert bool((guard[T * N:] == 7.0).all()) and bool((ws[need:] == 0xFF).all())
    y2 = torch.empty_like(y)
    M.fp4_matvec(x, q, s, y2, ws[:need] if need else None)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T", [1, 16, 31])
@pytest.mark.parametrize("N,K", [(8200, 384), (16390, 288), (16390, 640), (24580, 1152), (30001, 1056), (65540, 288),
                                 (65537, 2176), (45060, 288), (45060, 1152), (65530, 2176), (29000, 640)])
def test_matvec_many_rows(T, N, K):
    x = W.make_free((T, K), 1.0, T, "cuda", BF16)
    q, s = codes(N, K, T)
    y = torch.empty((T, N), device="cuda")
    ws = torch.empty((M.fp4_matvec_workspace_bytes(T, N, K),), dtype=torch.uint8, device="cuda")
    M.fp4_matvec(x, q, s, y, ws)
    check(x, q, s, y)


def test_matvec_of_quantized_weights():
    N, K, T = 96, 512, 3
    w = W.make_free((N, K), K ** -0.5, 5, "cuda", BF16)
    q, s = quantized(w)
    x = W.make_free((T, K), 1.0, 6, "cuda", BF16)
    y = torch.empty((T, N), device="cuda")
    ws = torch.empty((M.fp4_matvec_workspace_bytes(T, N, K),), dtype=torch.uint8, device="cuda")
    M.fp4_matvec(x, q, s, y, ws)
    check(x, q, s, y)
    wd = torch.empty((N, K), device="cuda")
    M.fp4_dequantize_groups(q, s, wd)
    assert np.array_equal(f64_of(wd), F.dequantize_groups(q.cpu().numpy(), s.cpu().numpy()))


def test_nan_stays_in_its_row_and_token():
    T, N, K = 20, 100, 416
    x = W.make_free((T, K), 1.0, 8, "cuda", BF16)
    q, s = codes(N, K, 9)
    ws = torch.empty((M.fp4_matvec_workspace_bytes(T, N, K),), dtype=torch.uint8, device="cuda")
    y0, y1 = (torch.empty((T, N), device="cuda") for _ in range(2))
    M.fp4_matvec(x, q, s, y0, ws)
    x[4, 411], x[17, 3], s[33, 12] = float("nan"), float("inf"), 255
    M.fp4_matvec(x, q, s, y1, ws)
    t = [i for i in range(T) if i not in (4, 17)]
    n = [i for i in range(N) if i != 33]
    assert torch.equal(y0[t][:, n], y1[t][:, n])
    assert torch.isnan(y1[4]).all() and torch.isnan(y1[:, 33]).all() and not torch.isfinite(y1[17]).any()


@pytest.mark.parametrize("N", [100, 24576, 65600, 65500])
@pytest.mark.parametrize("K", [1152, 1056, 128])
def test_nan_scales_of_the_next_row(N, K):
    """A row whose first groups are NaN, behind a row that ends inside a block's turn of K."""
    T = 3
    x = W.make_free((T, K), 1.0, 18, "cuda", BF16)
    q, s = codes(N, K, 19)
    y0, y1 = (torch.empty((T, N), device="cuda") for _ in range(2))
    M.fp4_matvec(x, q, s, y0)
    s[34], s[N - 1] = 255, 255
    M.fp4_matvec(x, q, s, y1)
    keep = [i for i in range(N) if i not in (34, N - 1)]
    assert torch.equal(y0[:, keep], y1[:, keep]) and torch.isnan(y1[:, 34]).all() and torch.isnan(y1[:, N - 1]).all()


@pytest.mark.parametrize("off", [1, 2, 3, 4])
@pytest.mark.parametrize("T,N,K", [(1, 40, 1152), (20, 24600, 256), (3, 65600, 128), (17, 65540, 640),
                                   (2, 65530, 640)])
def test_exponent_bytes_at_any_address(T, N, K, off):
    x = W.make_free((T, K), 1.0, 81, "cuda", BF16)
    q, s = codes(N, K, 82)
    held = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
    at = held[off:off + s.numel()].view(s.shape)
    at.copy_(s)
    y = torch.full((T, N), 7.0, device="cuda")
    M.fp4_matvec(x, q, at, y)
    check(x, q, s, y)


def test_past_32_bit_offsets():
    N, K = 1_250_000, 7168                                      # 4.5e9 bytes of codes
    q = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    q[-40:], s[-40:] = codes(40, K, 3)
    x = W.make_free((2, K), 1.0, 4, "cuda", BF16)
    y = torch.full((2, N), 7.0, device="cuda")
    M.fp4_matvec(x, q, s, y, torch.empty((M.fp4_matvec_workspace_bytes(2, N, K),), dtype=torch.uint8, device="cuda"))
    check(x, q[-40:], s[-40:], y[:, -40:].contiguous())
    assert not y[:, :-40].any()


def test_more_values_than_one_launch_has_threads_for():
    rows, cols = (1 << 21) + 5, 1 << 14                         # 2^35 values and more, eight to a thread
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GiB")
    tail = W.make_free((6, cols), 1.0, 71, "cuda", BF16)
    x = torch.ones((rows, cols), dtype=BF16, device="cuda")
    x[-6:] = tail
    q = torch.zeros((rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((rows, cols // 32), dtype=torch.uint8, device="cuda")
    M.fp4_quantize_groups(x, q, s)
    q64, s64 = F.quantize_groups(f64_of(tail))
    assert np.array_equal(s[-6:].cpu().numpy(), s64) and np.array_equal(q[-6:].cpu().numpy(), q64)
    assert bool((s[:-6] == int(s[0, 0])).all()) and bool((q[1 << 20] == 0x66).all())   # ones: code 6 (4) at 2^-2
    x.zero_()
    M.fp4_dequantize_groups(q, s, x)
    assert bool((x[:2] == 1.0).all()) and bool((x[1 << 20] == 1.0).all())
    assert np.array_equal(f64_of(x[-6:]), F.dequantize_groups(q64, s64))
    del x, q, s
    torch.cuda.empty_cache()


def test_no_rows_and_no_tokens():
    q, s = codes(8, 64, 1)
    M.fp4_matvec(torch.empty((0, 64), dtype=BF16, device="cuda"), q, s, torch.empty((0, 8), device="cuda"))
    M.fp4_matvec(torch.zeros((2, 64), dtype=BF16, device="cuda"), q[:0], s[:0], torch.empty((2, 0), device="cuda"))
