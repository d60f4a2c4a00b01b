"""Norm bounds for latent attention's outputs, beside the bounds by element.

A bound by element adds up magnitudes, so it stays where it is while outputs
shrink as 1 / sqrt(length), and a long request could lack whole tiles under it.
Here the error of a row of dv outputs is held against the root of the sum of
squares of its roundings.  Where a sum's terms a_j are each rounded, by 2^-8 of
a_j at most and with signs that have nothing to do with each other, the
variance of the error is at most 2^-16 sum |a_j|^2 / 3 (an error spread evenly
up to its bound), and 3.5 times 2^-8 sqrt(sum |a_j|^2) is six deviations.  (Of a
row of up to 12 terms it is more than all of them together.)

The fp32 sums: K roundings of 2^-24 of partial sums no larger than the sum of
the terms' magnitudes, of any sign, so sqrt(K) of them.  A score has 576
products at most, and scale times the sum of their magnitudes is below 32 here:
24 x 2^-24 x 32 = 2^-14.4 of a weight, and the exponential and its argument add
2^-22 of it: FP = 2^-12 of the size of the weights' roundings covers them.  Sums
over up to 16384 tokens are off by sqrt(16384) x 2^-24 = 2^-17, and what comes in
two bf16 halves by 2^-16 (3.5 deviations: 2^-14.2): LOW = 2^-14.
"""
import numpy as np

R8, FP, LOW, DEV = 2.0 ** -8, 2.0 ** -12, 2.0 ** -14, 3.5


def softmax(s):
    e = np.exp(s - s.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def decode_row(q, w, rows, dn, dc, see, scale, rounded_q=False):
    """One head of one token: q [dn + dr], w [dn + dv, dc], rows [n, dc + dr].  Returns the output [dv], o~ [dc], the
    size of the weights' roundings, that of o~'s, and with rounded_q that of q~'s (all before 2^-8)."""
    dv = w.shape[0] - dn
    if see <= 0:
        return np.zeros(dv), np.zeros(dc), 0.0, 0.0, 0.0
    x = rows[:see]
    c = x[:, :dc]
    qa = q[:dn] @ w[:dn]
    p = softmax(scale * (c @ qa + x[:, dc:] @ q[dn:]))
    v = c @ w[dn:].T
    mid = p @ c
    size_q = 0.0
    if rounded_q:                       # d out / d q~_c = scale sum_j p_j (c_jc - mid_c) v_j
        g = scale * ((p[:, None] * c).T @ v - np.outer(mid, p @ v))
        size_q = np.sqrt((qa ** 2 * (g ** 2).sum(axis=1)).sum())
    return (w[dn:] @ mid, mid, np.sqrt((p ** 2 * (v ** 2).sum(axis=1)).sum()),
            np.sqrt((mid ** 2 * (w[dn:] ** 2).sum(axis=0)).sum()), size_q)


def check_decode(got, q, w, requests, S, dn, dc, scale, half_p, bf16_out, rounded_q=False):
    """got, q [B S, H, ..], w [H, dn + dv, dc], requests a list of rows [n, dc + dr]; all fp64.  half_p: the weights are
    rounded to bf16 (64 rows a block); otherwise in two halves, as o~ always is.  Without rounded_q q~
    has to be exact in bf16.  Returns the largest error over its bound."""
    worst = 0.0
    for b, x in enumerate(requests):
        for i in range(S):
            for h in range(w.shape[0]):
                want, _, sp, so, sq = decode_row(q[b * S + i, h], w[h], x, dn, dc, len(x) - (S - 1 - i), scale, rounded_q)
                size = np.linalg.norm(want)
                tol = LOW * (size + so) + FP * sp + (DEV * R8 * sp if half_p else 0.0) + DEV * R8 * sq
                tol += R8 * (size + tol) if bf16_out else 0.0
                off = np.linalg.norm(got[b * S + i, h] - want)
                assert off <= tol, (b, i, h, off / tol, off / max(size, 1e-300))
                worst = max(worst, off / tol if tol else 0.0)
    return worst


def _norm(x, axis=-1):
    return np.sqrt((x ** 2).sum(axis=axis))


def _near(got, want, tol, bf16_out):
    """Rows (the last axis) of got and want, tol one number a row."""
    size = _norm(want)
    tol = tol + LOW * size
    tol = tol + (R8 * (size + tol) if bf16_out else 0.0)
    off = _norm(got - want)
    assert np.all(off <= tol), (np.max((off / np.maximum(tol, 1e-300))), np.unravel_index(np.argmax(off - tol), off.shape))


def check_attention(got, want, P, kv, dn, bf16_out):
    """got, want [lq, H, dv], the exact weights P [H, lq, lk], kv [lk, H, dn + dv]."""
    size = np.sqrt(np.einsum("hij,jh->ih", P ** 2, (kv[:, :, dn:] ** 2).sum(axis=2)))
    _near(got, want, (DEV * R8 + FP) * size, bf16_out)


def check_gradient(dq, dkv, dr, want, P, q, kv, k_rope, dout, out, dn, scale, bf16_out):
    """want: dq, dkv, dk_rope and dS of the oracle for the same out and lse.  P and dS are rounded to bf16; dS's fp32
    terms P dP and P D may cancel, so their sizes count."""
    wq, wkv, wr, dS = want
    k = np.concatenate([kv[:, :, :dn], np.repeat(k_rope[:, None], kv.shape[1], 1)], axis=2)
    terms = P * (np.einsum("ihd,jhd->hij", np.abs(dout), np.abs(kv[:, :, dn:])) +
                 (np.abs(dout) * np.abs(out)).sum(axis=2).T[:, :, None])
    e2 = (DEV * R8 * dS) ** 2 + (FP * terms) ** 2
    k2, q2, g2 = (k ** 2).sum(axis=2), (q ** 2).sum(axis=2), (dout ** 2).sum(axis=2)
    _near(dq, wq, scale * np.sqrt(np.einsum("hij,jh->ih", e2, k2)), bf16_out)
    to_k = scale * np.sqrt(np.einsum("hij,ih->jh", e2, q2))
    _near(dkv[:, :, :dn], wkv[:, :, :dn], to_k, bf16_out)
    _near(dkv[:, :, dn:], wkv[:, :, dn:], (DEV * R8 + FP) * np.sqrt(np.einsum("hij,ih->jh", P ** 2, g2)), bf16_out)
    # the heads' parts are roundings of their own; their fp32 sums stay below FP of the parts
    _near(dr, wr, np.sqrt((to_k ** 2).sum(axis=1)) + FP * _norm(to_k), bf16_out)
