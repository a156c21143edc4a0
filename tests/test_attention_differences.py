"""The gradients of attention against central differences of the float64 forward.

The loss is sum(dout o).  Its differences know nothing of how a backward goes about it, so what
the backward is given and rounds on its way counts in full (u = 2^-8, half a step of bf16,
relative; e = 2^-24 of fp32; each term element by element, no maxima):
  * o as given is off by eo = u |o| + (u + 2 w + n e) sum p|v| (p as operand, then o itself; w: what
    fp32 scores of d products leave of a weight, n keys), so delta by ed = sum |g| eo, ds by p ed;
  * lse as given is off by el = w + n e + 4 e |lse|, so p and ds by that share of themselves;
  * p and ds are rounded to bf16 as operands (u), dp and delta are sums of d products in fp32:
    eds = (u + w + el) |ds| + p (ed + (d + 4) e (sum |g v| + sum |g o|)), ep = (u + w + el) p;
  * dq: u |dq| + scale sum eds |k|, dk likewise over the queries, dv: u |dv| + sum ep |g|, with the
    sums' own rounding, rows times e, and all times 1 + 2 u for the products of roundings.
Differences with a step of 1e-4 are off by about 1e-8 of the loss' third derivative: 1e-6.
"""
import numpy as np
import pytest

import oracle.attention as OA
import workloads.bf16 as B

U, E = 2.0 ** -8, 2.0 ** -24
STEP = 1e-4


class Problem:
    """Packed sequences of bf16 values in float64, and what each gradient may be off by."""

    def __init__(self, lens_q, lens_k=None, heads=4, kv=2, d=64, causal=True, seed=0):
        rng = np.random.default_rng(seed)
        lens_k = lens_q if lens_k is None else lens_k
        self.cu_q, self.cu_k = ([int(x) for x in np.concatenate([[0], np.cumsum(a)])] for a in (lens_q, lens_k))
        self.heads, self.kv, self.d, self.causal = heads, kv, d, causal
        self.scale = float(np.float32(d ** -0.5))
        bf = lambda *s: B.round_bf16(rng.standard_normal(s))  # noqa: E731
        n, m = self.cu_q[-1], self.cu_k[-1]
        self.q, self.k, self.v, self.g = bf(n, heads, d), bf(m, kv, d), bf(m, kv, d), bf(n, heads, d)
        self.rng = rng

    def forward(self):
        return OA.attention_forward(self.q, self.k, self.v, self.cu_q, self.cu_k, self.scale, self.causal)

    def difference(self, x, i):
        loss = lambda: np.sum(self.forward()[0] * self.g)  # noqa: E731
        keep = x[i]
        x[i] = keep + STEP
        up = loss()
        x[i] = keep - STEP
        down = loss()
        x[i] = keep
        return (up - down) / (2 * STEP)

    def bounds(self):
        tol = [np.zeros(a.shape) for a in (self.q, self.k, self.v)]
        o, lse = self.forward()
        exact = OA.attention_backward(self.g, self.q, self.k, self.v, o, lse, self.cu_q, self.cu_k, self.scale, self.causal)
        group, size, d = self.heads // self.kv, abs(self.scale), self.d
        for a, b in OA.sequences(self.cu_q, self.cu_k):
            for h in range(self.heads):
                c = h // group
                q, g, k, v = self.q[a, h], self.g[a, h], self.k[b, c], self.v[b, c]
                if len(q) == 0 or len(k) == 0:
                    continue
                _, _, _, p, ds = OA.head_backward(g, q, k, v, o[a, h], lse[h, a], self.scale, self.causal)
                big = (np.abs(q) @ np.abs(k).T * size).max()
                w = 2 * (d + 4) * E * big + 8 * E * (big + 4)
                n, rows = len(k) * E, group * len(q) * E
                eo = U * np.abs(o[a, h]) + (U + 2 * w + n) * (p @ np.abs(v))
                ed = np.sum(np.abs(g) * eo, 1)[:, None]
                el = (w + n + 4 * E * np.abs(np.where(np.isinf(lse[h, a]), 0, lse[h, a])))[:, None]
                sums = (d + 4) * E * (np.abs(g) @ np.abs(v).T + np.sum(np.abs(g * o[a, h]), 1)[:, None])
                eds = (U + w + el) * np.abs(ds) + p * (ed + sums)
                tol[0][a, h] = (U * np.abs(exact[0][a, h]) + size * (eds + n * np.abs(ds)) @ np.abs(k)) * (1 + 2 * U)
                tol[1][b, c] += size * (eds + rows * np.abs(ds)).T @ np.abs(q) * (1 + 2 * U)
                tol[2][b, c] += ((U + w + el + rows) * p).T @ np.abs(g) * (1 + 2 * U)
        tol[1] += U * np.abs(exact[1]) * (1 + 2 * U)
        tol[2] += U * np.abs(exact[2]) * (1 + 2 * U)
        return [t + 1e-6 for t in tol]

    def sampled(self, count=30):
        """[(which, index, difference, bound)]: `count` elements of each of dq, dk and dv."""
        tol = self.bounds()
        for n, x in enumerate((self.q, self.k, self.v)):
            for _ in range(count):
                i = tuple(int(self.rng.integers(s)) for s in x.shape)
                yield n, i, self.difference(x, i), tol[n][i]


CASES = [dict(lens_q=[9, 40], heads=2, kv=1, seed=17), dict(lens_q=[12, 20], lens_k=[30, 20], heads=4, kv=2, d=128, seed=18),
         dict(lens_q=[25, 8], lens_k=[14, 33], heads=3, kv=3, causal=False, seed=19)]


def _rounded(p):
    """A backward as the kernels go about it: o in bf16, p and ds in bf16 as operands, gradients in bf16."""
    o, lse = p.forward()
    o16, r = B.round_bf16(o), B.round_bf16
    out = [np.zeros(a.shape) for a in (p.q, p.k, p.v)]
    for a, b in OA.sequences(p.cu_q, p.cu_k):
        for h in range(p.heads):
            c = h * p.kv // p.heads
            _, _, _, w, ds = OA.head_backward(p.g[a, h], p.q[a, h], p.k[b, c], p.v[b, c], o16[a, h], lse[h, a], p.scale, p.causal)
            out[0][a, h] = p.scale * r(ds) @ p.k[b, c]
            out[1][b, c] += p.scale * r(ds).T @ p.q[a, h]
            out[2][b, c] += r(w).T @ p.g[a, h]
    return [r(x) for x in out]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_bounds_take_roundings_and_no_mistake(case):
    """The bounds against gradients made on the host: rounded ones pass; zeros, turned signs, and
    those of a backward without delta, without the scale, or of one head of a group do not."""
    p = Problem(**case)
    o, lse = p.forward()
    right = _rounded(p)
    args = (p.cu_q, p.cu_k, p.scale, p.causal)
    no_delta = OA.attention_backward(p.g, p.q, p.k, p.v, np.zeros_like(o), lse, *args)
    first = p.g.copy()
    first[:, 1:] = 0
    one_head = OA.attention_backward(first, p.q, p.k, p.v, o, lse, *args)
    twice = [2 * x for x in right]
    wrong = {"zero": [0 * x for x in right], "turned": [-x for x in right], "no delta": no_delta, "twice": twice, "one head": one_head,
             "no scale": [right[0] / p.scale, right[1] / p.scale, right[2]]}
    caught = {k: [0, 0, 0] for k in wrong}
    for n, i, num, tol in p.sampled():
        assert abs(right[n][i] - num) <= tol, (n, i, right[n][i], num, tol)
        for k, x in wrong.items():
            caught[k][n] += abs(x[n][i] - num) > tol
    for k, hits in caught.items():      # of 30 samples each
        for n in range(3):
            if (k, n) not in (("no delta", 2), ("no scale", 2), ("one head", 0)):
                assert hits[n] >= 5, (k, n, caught)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_kernels_against_differences(case):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_util import dev_bf16, dev_i32, f64_of
    import rl_lora_linear_amd.lib as L
    p = Problem(**case)
    q, k, v, g = (dev_bf16(B.to_bf16_bits(a)) for a in (p.q, p.k, p.v, p.g))
    cq, ck = dev_i32(np.array(p.cu_q)), dev_i32(np.array(p.cu_k))
    shape = L.make_attention_shape(len(p.q), len(p.k), len(p.cu_q) - 1, p.heads, p.kv, p.d, p.scale, causal=p.causal)
    ws = L.empty_workspace(L.attention_workspace_bytes(shape))
    o, lse = torch.empty_like(q), torch.empty(p.heads, len(p.q), device="cuda")
    L.attention_forward(shape, q, k, v, cq, ck, o, lse, ws)
    grads = tuple(torch.empty_like(t) for t in (q, k, v))
    L.attention_backward(shape, g, q, k, v, o, lse, cq, ck, *grads, ws)
    got = [f64_of(t) for t in grads]
    assert L.lora_device_status(ws) == 0
    for n, i, num, tol in p.sampled():
        assert abs(got[n][i] - num) <= tol, (("dq", "dk", "dv")[n], i, got[n][i], num, tol)
