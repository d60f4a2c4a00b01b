"""The norm bounds (mla_testutil) hold for right results with the kernels'
roundings, and fail for what the bounds by element let through: a missing tile,
a missing rotary term, a mask off by one, a scale, operands rounded once where
they should be in two halves."""
import numpy as np
import pytest
import torch

import mla_testutil as U
from oracle import attention as A

DN, DR, DV, DC, H = 32, 16, 128, 64, 4
SCALE = 48 ** -0.5


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def inputs(n, S, seed=0):
    """q^n picks one row of W^K, times a power of two: q~ is exact in bf16."""
    r = np.random.default_rng(seed)
    q = bf16(r.standard_normal((S, H, DN + DR)))
    q[:, :, :DN] = 0
    for i in range(S):
        for h in range(H):
            q[i, h, r.integers(DN)] = 8.0
    return q, bf16(r.standard_normal((H, DN + DV, DC)) * DC ** -0.5), bf16(r.standard_normal((n, DC + DR)))


def answer(q, w, x, S, rope=True, drop=None, shift=0, p_round=lambda p: p, o_round=lambda o: o):
    out = np.zeros((S, H, DV))
    for i in range(S):
        see = max(0, len(x) - (S - 1 - i) + shift)
        for h in range(H):
            s = x[:see, :DC] @ (q[i, h, :DN] @ w[h, :DN]) + (x[:see, DC:] @ q[i, h, DN:] if rope else 0)
            if drop is not None:
                s[drop] = -np.inf
            e = np.exp(SCALE * (s - s.max()))
            out[i, h] = w[h, DN:] @ o_round(p_round(e) @ x[:see, :DC] / e.sum())
    return out


def check(got, q, w, x, S, half_p=False, bf16_out=False, **kw):
    U.check_decode(got, q, w, [x], S, DN, DC, SCALE, half_p, bf16_out, **kw)


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("n", [5, 150, 700, 3000, 9000])
def test_decode_bounds(n, S):
    q, w, x = inputs(n, S)
    right = answer(q, w, x, S)
    want = A.absorbed(q, w, x, DN, DC, S, SCALE)[0]
    assert np.allclose(right, want, rtol=0, atol=1e-12)
    check(right.astype(np.float32), q, w, x, S)
    check(bf16(right), q, w, x, S, bf16_out=True)
    rounded = answer(q, w, x, S, p_round=bf16)
    check(rounded, q, w, x, S, half_p=True)
    check(bf16(rounded), q, w, x, S, half_p=True, bf16_out=True)
    wrong = [answer(q, w, x, S, rope=False), right * 1.05, answer(q, w, x, S, drop=slice(n - 1, n)),
             answer(q, w, x, S, shift=-1)]
    if n > 64:
        wrong += [answer(q, w, x, S, drop=slice(n - 64, n)), answer(q, w, x, S, drop=slice(0, 64))]
    for bad in wrong:                                              # also where the weights come in two halves
        with pytest.raises(AssertionError):
            check(bad, q, w, x, S)
    for bad in wrong[:2] + wrong[4:]:                              # weights rounded once hide a single token
        for out in (bad, bf16(bad)):
            with pytest.raises(AssertionError):
                check(out, q, w, x, S, half_p=True, bf16_out=out is not bad)
    # a second half that is lost (the weights' own roundings average out over many tokens)
    for bad in [answer(q, w, x, S, o_round=bf16)] + ([rounded] if n <= 3000 else []):
        with pytest.raises(AssertionError):
            check(bad, q, w, x, S)


def test_decode_bound_of_rounded_queries():
    q, w, x = inputs(700, 1, seed=1)
    q[:, :, :DN] = bf16(np.random.default_rng(2).standard_normal((1, H, DN)) * 2)
    got = A.absorbed(q, w, x, DN, DC, 1, SCALE, bf16)[0]
    check(got, q, w, x, 1, rounded_q=True)
    with pytest.raises(AssertionError):
        check(got, q, w, x, 1)
    with pytest.raises(AssertionError):
        check(answer(q, w, x, 1, drop=slice(0, 64)), q, w, x, 1, rounded_q=True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [(40, 40), (3, 900), (200, 700)])
def test_attention_and_gradient_bounds(lq, lk, causal):
    r = np.random.default_rng(lq)
    q, kv, kr = (bf16(r.standard_normal(s)) for s in ((lq, H, DN + DR), (lk, H, DN + DV), (lk, DR)))
    dout = bf16(r.standard_normal((lq, H, DV)))
    out, lse, P = A.attention(q, kv, kr, DN, causal, SCALE)
    low = np.einsum("hij,jhd->ihd", bf16(P), kv[:, :, DN:])
    U.check_attention(out, out, P, kv, DN, False)
    U.check_attention(bf16(low), out, P, kv, DN, True)
    tile = P.copy()
    tile[:, :, :16] = 0
    for bad in (out * 1.05, np.einsum("hij,jhd->ihd", tile, kv[:, :, DN:]),
                A.attention(q, kv, kr * 0, DN, causal, SCALE)[0]):
        with pytest.raises(AssertionError):
            U.check_attention(bad, out, P, kv, DN, False)
    want = A.attention_backward(dout, q, kv, kr, out, lse, DN, causal, SCALE)

    def grads(dS, P):
        k = np.concatenate([kv[:, :, :DN], np.repeat(kr[:, None], H, 1)], axis=2)
        dk = SCALE * np.einsum("hij,ihd->jhd", dS, q)
        dv = np.einsum("hij,ihd->jhd", P, dout)
        return SCALE * np.einsum("hij,jhd->ihd", dS, k), np.concatenate([dk[:, :, :DN], dv], axis=2), dk[:, :, DN:].sum(1)

    def check(g, bf16_out):
        U.check_gradient(*g, want, P, q, kv, kr, dout, out, DN, SCALE, bf16_out)

    check(grads(want[3], P), False)
    check([bf16(t) for t in grads(bf16(want[3]), bf16(P))], True)
    cut, cut_p = want[3].copy(), P.copy()
    cut[:, -2:, :32], cut_p[:, -2:, :32] = 0, 0                    # a piece of the last queries' tiles
    for dS, p in ((want[3] * 1.05, P), (want[3], P * 1.05), (cut, P), (want[3], cut_p)):
        with pytest.raises(AssertionError):
            check(grads(dS, p), False)
    one_head = list(want[:3])
    one_head[2] = one_head[2] - SCALE * want[3][0].T @ q[:, 0, DN:]
    with pytest.raises(AssertionError):
        check(one_head, False)
