"""fp4_matvec at whole sizes of every form, and at the ends of the scale range,
against exact products.

Tokens are whole numbers of magnitude 8 at most (times a power of two) and
scales 2^-1, 1 or 2 (times another), so every product and every partial sum
is a multiple of a quarter below 8 * 12 * K < 2^20 (K <= 7168): a whole number
of quarters below 2^22, exact in fp32 in any order of the additions.  fp32
results are therefore equal to the fp64 ones, and bf16 results to these
rounded once to nearest even."""
import pytest
import torch

import sparse_expert_routing_sigmoid_amd as M
from oracle import fp4 as F

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def exact_product(x, q, s):
    """fp64 x W^T, 4096 rows of W at a time."""
    table = torch.from_numpy(F.VALUES).cuda()
    parts = []
    for i in range(0, q.shape[0], 4096):
        c = torch.stack([q[i:i + 4096] & 15, q[i:i + 4096] >> 4], dim=2).flatten(1).long()
        w = table[c] * torch.exp2(s[i:i + 4096].double() - 127).repeat_interleave(F.GROUP, dim=1)
        parts.append(x.double() @ w.t().contiguous())
    return torch.cat(parts, dim=1)


def operands(T, N, K, byte, x_exp, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").double() * 2.0 ** x_exp
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(byte - 1, byte + 2, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return x.to(BF16), q, s


def check(T, N, K, yt, byte=127, x_exp=0):
    x, q, s = operands(T, N, K, byte, x_exp, T + N + K)
    y = torch.full((T, N), 7.0, dtype=yt, device="cuda")
    M.fp4_matvec(x, q, s, y)
    want = exact_product(x, q, s)
    assert torch.equal(want.float().double(), want)              # the inputs are what the opening comment says
    assert torch.equal(y, want.float().to(yt))


@pytest.mark.parametrize("T", [1, 4, 5, 16, 17, 32, 40])
@pytest.mark.parametrize("N,K", [(40, 7168), (4096, 7168), (6150, 7168), (12300, 7168), (24580, 7168), (29000, 7168),
                                 (45060, 7168), (65536, 7168), (65536, 1408), (65530, 1056), (100003, 2176)])
def test_whole_sizes(T, N, K):
    check(T, N, K, F32)


@pytest.mark.parametrize("T,N,K", [(3, 4096, 7168), (16, 65536, 7168), (20, 24580, 1056)])
def test_bf16_results(T, N, K):
    check(T, N, K, BF16)


@pytest.mark.parametrize("T,N,K", [(1, 40, 288), (3, 4096, 256), (20, 12300, 256), (16, 32768, 384), (17, 65536, 256)])
@pytest.mark.parametrize("byte,x_exp", [(1, 100), (60, 40), (200, -70), (251, -120)])
def test_ends_of_the_scale_range(T, N, K, byte, x_exp):
    """Scales down to 2^-127, whose codes 0.5 and 1 are subnormal in bf16, and up to 2^125, whose code 6 is the largest."""
    check(T, N, K, F32, byte, x_exp)
