"""fp64 oracle of latent attention ("DeepSeek-V3 Technical Report" reading
guide, Method section 1): keys and values of a token's heads from one latent c
and one rotary key r, k = [W^K c ; r], v = W^V c; the paged cache that holds
them; expanded attention and its gradient."""
from __future__ import annotations

import numpy as np


def softmax_rows(s):
    """Weights and log-sum-exp of the rows of s [.., n]; a row without a finite score has weights 0 and lse -inf."""
    top = s.max(axis=-1, keepdims=True, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - safe)
    z = e.sum(axis=-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (safe + np.log(z))[..., 0]
    return e / np.where(z > 0, z, 1.0), lse


def hidden(lq, lk, causal):
    """[lq, lk]: key j is hidden from query i (causal: j > i + lk - lq)."""
    if not causal:
        return np.zeros((lq, lk), bool)
    return np.arange(lk)[None, :] > np.arange(lq)[:, None] + (lk - lq)


def attention(q, kv, k_rope, dn, causal, scale):
    """One sequence: q [lq, H, dn + dr], kv [lk, H, dn + dv], k_rope [lk, dr].
    Returns out [lq, H, dv], lse [lq, H] and the weights [H, lq, lk]."""
    lq, H, _ = q.shape
    lk, dv = kv.shape[0], kv.shape[2] - dn
    out, lse, P = np.zeros((lq, H, dv)), np.full((lq, H), -np.inf), np.zeros((H, lq, lk))
    mask = hidden(lq, lk, causal)
    for h in range(H):
        s = scale * (q[:, h, :dn] @ kv[:, h, :dn].T + q[:, h, dn:] @ k_rope.T)
        s[mask] = -np.inf
        P[h], lse[:, h] = softmax_rows(s)
        out[:, h] = P[h] @ kv[:, h, dn:]
    return out, lse, P


def attention_backward(dout, q, kv, k_rope, out, lse, dn, causal, scale):
    """Gradients (dq, dkv, dk_rope) of one sequence, from the given out and lse, and dS [H, lq, lk] (before scale)."""
    lq, H, _ = q.shape
    lk = kv.shape[0]
    dq, dkv, dr = np.zeros_like(q), np.zeros_like(kv), np.zeros_like(k_rope)
    dS = np.zeros((H, lq, lk))
    mask = hidden(lq, lk, causal)
    for h in range(H):
        k = np.concatenate([kv[:, h, :dn], k_rope], axis=1)
        s = scale * (q[:, h] @ k.T)
        with np.errstate(over="ignore", invalid="ignore"):
            p = np.where(mask, 0.0, np.exp(s - lse[:, h, None]))
        dS[h] = p * (dout[:, h] @ kv[:, h, dn:].T - (dout[:, h] * out[:, h]).sum(axis=1)[:, None])
        dq[:, h] = scale * dS[h] @ k
        dk = scale * dS[h].T @ q[:, h]
        dkv[:, h, :dn], dkv[:, h, dn:] = dk[:, :dn], p.T @ dout[:, h]
        dr += dk[:, dn:]
    return dq, dkv, dr, dS


def absorbed(q, w, rows, dn, dc, S, scale, round_q=lambda x: x):
    """The newest S tokens of one request: q [S, H, dn + dr], w [H, dn + dv, dc], rows [n, dc + dr] the cached tokens.
    round_q: the rounding of q~.  Returns out [S, H, dv] and the weights [S, H, n]."""
    H, n = w.shape[0], rows.shape[0]
    out, P = np.zeros((S, H, w.shape[1] - dn)), np.zeros((S, H, n))
    for i in range(S):
        see = max(0, n - (S - 1 - i))
        for h in range(H):
            qa = round_q(q[i, h, :dn] @ w[h, :dn])
            s = scale * (rows[:, :dc] @ qa + rows[:, dc:] @ q[i, h, dn:])
            s[see:] = -np.inf
            P[i, h] = softmax_rows(s)[0]
            out[i, h] = w[h, dn:] @ (P[i, h] @ rows[:, :dc])
    return out, P


def pages_extend(seq_len, new_len, page, table, free, n_free, N):
    """The paging step in plain integers; table is a list of lists.  Returns
    (table, seq_len, n_free, failed, cu, slot, position)."""
    table = [list(r) for r in table]
    W = len(table[0]) if table else 0
    out_len, cu, slot, position = [], [0], [], []
    taken = given = failed = 0
    n_free = max(0, min(n_free, len(free)))
    for b, (old, add) in enumerate(zip(seq_len, new_len)):
        old, add = max(0, old), max(0, add)
        have, want = -(-old // page), -(-(old + add) // page)
        need = want - have
        room = add == 0 or (want <= W and cu[-1] + add <= N)
        ok = room and (need == 0 or taken + need <= n_free)
        if ok:
            for i in range(need):
                table[b][have + i] = free[n_free - 1 - taken - i]
            given += need
        else:
            failed += 1
        if room:
            taken += need
        for j in range(old, old + add):
            slot.append(table[b][j // page] * page + j % page if ok else -1)
            position.append(j)
        cu.append(cu[-1] + add)
        out_len.append(old + add if ok else old)
    slot = (slot + [-1] * N)[:N]
    position = (position + [-1] * N)[:N]
    return table, out_len, n_free - given, failed, cu, slot, position


def pages_release(done, seq_len, page, table, free, n_free):
    free, seq_len = list(free), list(seq_len)
    for b, d in enumerate(done):
        if d:
            for i in range(min(-(-max(0, seq_len[b]) // page), len(table[b]))):
                if n_free < len(free):
                    free[n_free] = table[b][i]
                    n_free += 1
            seq_len[b] = 0
    return seq_len, free, n_free
