"""Per-adapter gradient norms over many tensors and clipping (oracle; test
infrastructure only).

norm_a = sqrt(sum over adapter a's tensors of g^2); the clipped gradient is
min(1, max_norm / (norm_a + 1e-6)) g.  A group with a non-finite gradient is not
clipped, and not stepped by the AdamW that follows (its counter stays).
"""
from __future__ import annotations

import numpy as np

from .adam import adam_step


def norms(tensors, n_groups, g):
    """tensors: (offset, count, group) triples; g flat."""
    s = np.zeros(n_groups)
    for off, cnt, a in tensors:
        s[a] += np.sum(np.asarray(g[off:off + cnt], np.float64) ** 2)
    return np.sqrt(s)


def clip(tensors, n_groups, g, max_norm, out=None):
    """(clipped gradient, norms); elements outside every tensor are out's (zeros if None)."""
    g = np.asarray(g, np.float64)
    res = np.zeros_like(g) if out is None else np.array(out, np.float64)
    n = norms(tensors, n_groups, g)
    for off, cnt, a in tensors:
        c = min(1.0, max_norm / (n[a] + 1e-6)) if np.isfinite(n[a]) else 1.0
        res[off:off + cnt] = g[off:off + cnt] * c
    return res, n


def adam_clipped(tensors, n_groups, steps, p, g, m, v, max_norm, lr, beta1=0.9, beta2=0.999,
                 eps=1e-8, weight_decay=0.0):
    """(p, m, v, steps, norms) after one call; inputs are not modified."""
    p, m, v = (np.array(a, np.float64) for a in (p, m, v))
    steps = np.array(steps, np.int64)
    cg, n = clip(tensors, n_groups, g, max_norm)
    steps[np.isfinite(n)] += 1
    for off, cnt, a in tensors:
        if not np.isfinite(n[a]):
            continue
        at = slice(off, off + cnt)
        p[at], m[at], v[at] = adam_step(p[at], cg[at], m[at], v[at], int(steps[a]), lr, beta1, beta2,
                                        eps, weight_decay)
    return p, m, v, steps, n
