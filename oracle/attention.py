"""Attention over packed prompts and over a paged cache, and the cache's bookkeeping
(oracle; test infrastructure only).

For one head and one sequence with query rows Q [Lq][d] and key rows K, V [Lk][d],
query i seeing key j iff not causal or j <= i + Lk - Lq:
  s_ij = scale Q_i . K_j,  lse_i = log sum_j exp(s_ij),  P = exp(s - lse),  O = P V
(no key seen: O_i = 0, lse_i = -inf), and for dL/dO = G, with O and lse as given,
  dL/dV = P^T G,  dS = P * (G V^T - rowsum(G O)),  dL/dQ = scale dS K,
  dL/dK = scale dS^T Q,  a key head's gradients summed over the heads that read it.
"""
from __future__ import annotations

import numpy as np


def scores(q, k, scale, causal):
    """(s, seen) of one head."""
    lq, lk = len(q), len(k)
    seen = np.ones((lq, lk), bool)
    if causal:
        seen = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq
    return scale * (q @ k.T), seen


def head_forward(q, k, v, scale, causal):
    """(o, lse, p) of one head."""
    s, seen = scores(q, k, scale, causal)
    o, lse, p = np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf), np.zeros(s.shape)
    for i in range(len(q)):
        if seen[i].any():
            row = s[i, seen[i]]
            lse[i] = row.max() + np.log(np.sum(np.exp(row - row.max())))
            p[i, seen[i]] = np.exp(row - lse[i])
            o[i] = p[i, seen[i]] @ v[seen[i]]
    return o, lse, p


def head_backward(g, q, k, v, o, lse, scale, causal):
    """(dq, dk, dv, p, ds) of one head."""
    s, seen = scores(q, k, scale, causal)
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.where(seen, np.exp(s - lse[:, None]), 0.0)
    ds = p * (g @ v.T - np.sum(g * o, axis=1)[:, None])
    return scale * ds @ k, scale * ds.T @ q, p.T @ g, p, ds


def sequences(cu_q, cu_k):
    for b in range(len(cu_q) - 1):
        yield slice(int(cu_q[b]), int(cu_q[b + 1])), slice(int(cu_k[b]), int(cu_k[b + 1]))


def attention_forward(q, k, v, cu_q, cu_k, scale, causal=True):
    """q [n][heads][d], k, v [m][kv heads][d] -> o like q, lse [heads][n]."""
    o, lse = np.zeros(q.shape), np.full(q.shape[1::-1], -np.inf)
    group = q.shape[1] // k.shape[1]
    for a, b in sequences(cu_q, cu_k):
        for h in range(q.shape[1]):
            o[a, h], lse[h, a], _ = head_forward(q[a, h], k[b, h // group], v[b, h // group], scale, causal)
    return o, lse


def attention_backward(g, q, k, v, o, lse, cu_q, cu_k, scale, causal=True):
    """(dq, dk, dv)."""
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    group = q.shape[1] // k.shape[1]
    for a, b in sequences(cu_q, cu_k):
        for h in range(q.shape[1]):
            c = h // group
            x, y, z, _, _ = head_backward(g[a, h], q[a, h], k[b, c], v[b, c], o[a, h], lse[h, a], scale, causal)
            dq[a, h] = x
            dk[b, c] += y
            dv[b, c] += z
    return dq, dk, dv


def cache_rows(cache, table, length):
    """Rows 0 .. length - 1 of a request from the pages [n_pages][kv heads][page][d]: [length][kv heads][d]."""
    page = cache.shape[2]
    return np.array([cache[table[p // page], :, p % page] for p in range(length)]).reshape(length, *cache.shape[1::2])


def kv_tables(cached, new, table, ring, state, page, n_slots):
    """One step of the page allocator, request by request, for lengths that are valid.
    table [n][max_pages], ring [n_pages] are changed in place.  Returns seq_lens, cu_new,
    slots, positions, token_seqs, state, and whether a request went without pages."""
    head, tail = state
    free, asked, end, short = tail - head, 0, head, False
    seq_lens, cu, slots, pos, seqs, put = [], [0], [], [], [], []
    for b, (c, r) in enumerate(zip(cached, new)):
        held = -(-c // page)
        if r < 0:
            put += [table[b][j] for j in range(held)]
            seq_lens.append(0)
            cu.append(cu[-1])
            continue
        need = -(-(c + r) // page) - held
        served = need == 0 or asked + need <= free
        if served:
            for j in range(need):
                table[b][held + j] = ring[(head + asked + j) % len(ring)]
            if need:
                end = head + asked + need
        else:
            short = True
        asked += need
        for p in range(c, c + r):
            slots.append(table[b][p // page] * page + p % page if served else -1)
            pos.append(p)
            seqs.append(b)
        seq_lens.append(c + r if served else c)
        cu.append(cu[-1] + r)
    for i, p in enumerate(put):
        ring[(tail + i) % len(ring)] = p
    pad = [-1] * (n_slots - len(slots))
    return seq_lens, cu, slots + pad, pos + pad, seqs + pad, (end, tail + len(put)), short
