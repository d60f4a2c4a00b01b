"""Latent attention held to norm bounds (mla_testutil), which shrink with the
outputs: long requests, the batches that k_out's larger blocks are for, requests
split into more pieces than a wave joins at once, calls of few blocks in bf16,
gradients over many tiles."""
import numpy as np
import pytest
import torch

import mla_testutil as U
import sparse_expert_routing_sigmoid_amd as M
import test_gpu_mla_attention as T
import test_gpu_mla_decode as D
from moe_testutil import f64_of
from oracle import attention as A

pytestmark = pytest.mark.gpu


def exact_queries(q, dn, seed):
    """q^n picks one row of W^K, times 16: q~ is exact in bf16, and its rounding takes no part."""
    g = torch.Generator().manual_seed(seed)
    at = torch.randint(dn, q.shape[:2], generator=g)
    q[:, :, :dn] = 0
    q[:, :, :dn].scatter_(2, at[:, :, None].cuda(), 16.0)


def decode(lens, S, H, dims, page, max_len=None, seed=0, exact=True):
    """Both types of output; half_p by the rule of the division."""
    dn, dr, dv, dc = dims
    q, w, cache, table, n, rows = D.make(lens, S, H, dims, page, seed=seed)
    if exact:
        exact_queries(q, dn, seed)
    most = table.shape[1] * page if max_len is None else max_len
    half_p = S * H > 32 and len(lens) * -(-most // 64) * -(-S * H // 64) >= 256
    for t in (torch.float32, torch.bfloat16):
        out = D.run(q, w, cache, table, n, S, dims, t, max_len=max_len)
        U.check_decode(f64_of(out), f64_of(q), f64_of(w), rows, S, dn, dc, (dn + dr) ** -0.5, half_p,
                       t == torch.bfloat16, rounded_q=not exact)
    return half_p


@pytest.mark.parametrize("H,dims,page", [(16, D.WIDE, 64), (128, D.WIDE, 64), (16, D.NARROW, 16), (40, D.ODD, 100)])
def test_a_long_request(H, dims, page):
    assert decode([9000], 1, H, dims, page, seed=H) == (H == 128)


@pytest.mark.parametrize("B,S,dims", [(17, 1, D.WIDE), (33, 1, D.WIDE), (70, 1, D.WIDE), (23, 3, D.WIDE),
                                      (40, 1, D.NARROW), (33, 1, D.ODD)])
def test_batches_of_many_heads(B, S, dims):
    """128 heads: from 33 tokens on k_out takes 32 of them a block (here 32 and 1; 32, 32 and 6; 32, 32 and 5), below 16."""
    decode([(37 * b + 11 * B) % 150 for b in range(B)], S, 128, dims, 16, seed=B)


@pytest.mark.parametrize("B,S,H,dims", [(9, 1, 8, D.WIDE), (31, 1, 8, D.WIDE), (31, 2, 8, D.NARROW), (31, 1, 128, D.WIDE)])
def test_one_long_request_among_short_ones(B, S, H, dims):
    """The long one's 110 to 250 pieces of a row are joined by one or two waves, more than 64 to each."""
    decode([40 + b for b in range(B // 2)] + [16000] + [5 + b for b in range(B - B // 2 - 1)], S, H, dims, 64, seed=B + H)


@pytest.mark.parametrize("H", [8, 70])
def test_the_rounding_of_absorbed_queries(H):
    """Against exact q~: its rounding's own bound, in both sizes of blocks."""
    assert decode([700, 90, 1], 1, H, D.WIDE, 16, max_len=60000, seed=90 + H, exact=False) == (H > 32)


# -------------------------------------------------------------- attention --
def attention(lq, lk, H, dims, causal, seed):
    q, kv, r, cu_q, cu_k = T.make(lq, lk, H, dims, seed=seed, lead=2, tail=3)
    for t in (torch.float32, torch.bfloat16):
        out, lse = T.forward(q, kv, r, cu_q, cu_k, causal, dims, t)
        T.check_forward(q, kv, r, cu_q, cu_k, causal, dims, out, lse)
        assert all(torch.all(x[:2] == 7) and torch.all(x[2 + sum(lq):] == 7) for x in (out, lse))
        q64, kv64, r64, o64 = map(f64_of, (q, kv, r, out))
        for i, j in T.sequences(cu_q, cu_k):
            want, _, P = A.attention(q64[i], kv64[j], r64[j], dims[0], causal, (dims[0] + dims[1]) ** -0.5)
            U.check_attention(o64[i], want, P, kv64[j], dims[0], t == torch.bfloat16)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dims", [T.WIDE, T.NARROW, T.ODD, T.MIXED])
@pytest.mark.parametrize("H,lq,lk", [(3, [1], [600]), (3, [40, 3], [500, 900]), (2, [600], [300]),
                                     (5, [31, 0, 32, 33], [257, 900, 128, 129]), (2, [130], [4100])])
def test_calls_of_few_blocks(H, lq, lk, dims, causal):
    """32 rows a block and the keys shared out: (Tq / 32 + B) H is at most the keys of a sequence, and those 256 or more."""
    Tq, Tk, B = sum(lq) + 5, sum(lk) + 5, len(lq)
    assert Tk // B >= 256 and (Tq // 32 + B) * H <= min(Tk // B, 512)
    attention(lq, lk, H, dims, causal, seed=H + len(lq))


@pytest.mark.parametrize("dims", [T.WIDE, T.NARROW])
def test_many_blocks(dims):
    attention([900, 65], [900, 700], 24, dims, True, seed=5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dims", [T.WIDE, T.NARROW, T.ODD, T.MIXED])
@pytest.mark.parametrize("lq,lk", [([700], [700]), ([1, 300, 5], [600, 400, 300])])
def test_gradients_over_many_tiles(lq, lk, dims, causal):
    H, scale = 3, (dims[0] + dims[1]) ** -0.5
    x = T.make(lq, lk, H, dims, seed=len(lq), lead=2, tail=3)
    for t in (torch.float32, torch.bfloat16):
        out, lse, dout, *grads = T.gradient(x, causal, dims, t, t)
        assert all(torch.all(g[:2] == 7) and torch.all(g[-3:] == 7) for g in grads)
        q64, kv64, r64, o64, l64, g64, a64, b64, c64 = map(f64_of, (*x[:3], out, lse, dout, *grads))
        for i, j in T.sequences(*x[3:]):
            want = A.attention_backward(g64[i], q64[i], kv64[j], r64[j], o64[i], l64[i], dims[0], causal, scale)
            P = A.attention(q64[i], kv64[j], r64[j], dims[0], causal, scale)[2]
            U.check_gradient(a64[i], b64[j], c64[j], want, P, q64[i], kv64[j], r64[j], g64[i], o64[i], dims[0], scale,
                             t == torch.bfloat16)
