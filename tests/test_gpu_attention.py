"""Attention over packed prompts against the float64 oracle.

Tolerances.  With u = 2^-8 (half a step of bf16, relative) and e = 2^-24 (of fp32):
  * a score is an fp32 sum of d products, times the scale in powers of two:
    |error| <= es = (d + 4) e sum|q k| scale, largest over the case's scores; the exponent's
    argument and lse add 4 e (|s| + |lse|) and the exponential itself 4 e;
    so a weight is off by the factor w = 2 es + 8 e (max|s| + 4) at most, its sum likewise;
  * o = sum p v rounds p and o once: |error| <= u |o| + (u + 2 w) sum p|v|  (p's sum is made of
    the unrounded weights), all times 1 + 2 u for the roundings' products;
  * ds = p (dp - delta), dp and delta fp32 sums of d products: off by
    eds = (u + w) |ds| + p (d + 4) e (sum|g v| + sum|g o|);
    dq = scale sum ds k: |error| <= u |dq| + scale sum eds |k|, dk likewise; dv as o;
  * fp32 accumulation over n rows adds n e times the sum of magnitudes.
"""
import numpy as np
import pytest

import oracle.attention as OA
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import dev_bf16, dev_i32, f64_of  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402
from test_gpu_graph import _replay_check  # noqa: E402

U, E = 2.0 ** -8, 2.0 ** -24
NAN = float("nan")


def bf(rng, *shape):
    return B.round_bf16(rng.standard_normal(shape))


class Case:
    """q, k, v (and dout) of packed sequences on the host in float64 (bf16 values) and on the device."""

    def __init__(self, lens_q, lens_k=None, heads=4, kv=2, d=64, causal=True, scale=None, seed=0, fused=False, front=0, behind=0):
        rng = np.random.default_rng(seed)
        lens_k = lens_q if lens_k is None else lens_k
        self.cu_q, self.cu_k = (front + np.concatenate([[0], np.cumsum(a)]).astype(int) for a in (lens_q, lens_k))
        self.n, self.m = int(self.cu_q[-1]) + behind, int(self.cu_k[-1]) + behind
        self.heads, self.kv, self.d, self.causal = heads, kv, d, causal
        self.scale = float(np.float32(d ** -0.5 if scale is None else scale))
        self.q, self.g = bf(rng, self.n, heads, d), bf(rng, self.n, heads, d)
        self.k, self.v = bf(rng, self.m, kv, d), bf(rng, self.m, kv, d)
        self.fused = fused
        self.upload()

    def put(self, a):
        return dev_bf16(B.to_bf16_bits(a))

    def upload(self):
        if self.fused:   # one projection's output; the last head's columns belong to nobody
            self.buf = torch.full((self.n, self.heads + 2 * self.kv + 1, self.d), NAN, dtype=torch.bfloat16, device="cuda")
            self.grad = torch.full_like(self.buf, NAN)
            cut = lambda t: (t[:, :self.heads], t[:, self.heads:self.heads + self.kv], t[:, self.heads + self.kv:-1])  # noqa: E731
            self.dev, self.dgrad = cut(self.buf), cut(self.grad)
            for t, a in zip(self.dev, (self.q, self.k, self.v)):
                t.copy_(self.put(a))
        else:
            self.dev = tuple(self.put(a) for a in (self.q, self.k, self.v))
            self.dgrad = tuple(torch.full_like(t, NAN) for t in self.dev)
        self.o = torch.full((self.n, self.heads, self.d), NAN, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.heads, self.n), NAN, device="cuda")
        st = [t.stride(0) if t.shape[0] > 1 else t.shape[1] * self.d for t in self.dev]
        self.shape = L.make_attention_shape(self.n, self.m, len(self.cu_q) - 1, self.heads, self.kv, self.d, self.scale, causal=self.causal,
                                            q_stride=st[0], k_stride=st[1], v_stride=st[2])
        self.cq, self.ck = dev_i32(self.cu_q), dev_i32(self.cu_k)
        self.ws = L.empty_workspace(L.attention_workspace_bytes(self.shape))

    def forward(self):
        L.attention_forward(self.shape, *self.dev, self.cq, self.ck, self.o, self.lse, self.ws)
        return f64_of(self.o), f64_of(self.lse)

    def backward(self, dout=None):
        self.dout = self.put(self.g) if dout is None else dout
        L.attention_backward(self.shape, self.dout, *self.dev, self.o, self.lse, self.cq, self.ck, *self.dgrad, self.ws)
        return tuple(f64_of(t) for t in self.dgrad)

    def bounds(self, o, lse):
        """The oracle's (o, lse, dq, dk, dv) and how far each may be off; gradients for the given o, lse."""
        res = [np.zeros(self.q.shape), np.full((self.heads, self.n), -np.inf), np.zeros(self.q.shape), np.zeros(self.k.shape), np.zeros(self.v.shape)]
        tol = [np.zeros(r.shape) for r in res]
        group = self.heads // self.kv
        for a, b in OA.sequences(self.cu_q, self.cu_k):
            for h in range(self.heads):
                c = h // group
                q, g, k, v = self.q[a, h], self.g[a, h], self.k[b, c], self.v[b, c]
                if len(q) == 0:
                    continue
                ro, rl, p = OA.head_forward(q, k, v, self.scale, self.causal)
                res[0][a, h], res[1][h, a] = ro, rl
                if len(k) == 0:
                    continue
                size = abs(self.scale)
                absq = np.abs(q) @ np.abs(k).T * size
                big = absq.max() if absq.size else 0.0
                w = 2 * (self.d + 4) * E * big + 8 * E * (big + 4)
                n = len(k) * E
                tol[0][a, h] = (U * np.abs(ro) + (U + 2 * w + n) * (p @ np.abs(v))) * (1 + 2 * U)
                tol[1][h, a] = w + n + 4 * E * np.abs(np.where(np.isinf(rl), 0, rl))
                dq, dk, dv, p, ds = OA.head_backward(g, q, k, v, o[a, h], lse[h, a], self.scale, self.causal)
                eds = (U + w) * np.abs(ds) + p * (self.d + 4) * E * (np.abs(g) @ np.abs(v).T + np.sum(np.abs(g * o[a, h]), 1)[:, None])
                ads = np.abs(ds)
                res[2][a, h] = dq
                res[3][b, c] += dk
                res[4][b, c] += dv
                tol[2][a, h] = (U * np.abs(dq) + size * (eds + n * ads) @ np.abs(k)) * (1 + 2 * U)
                m = group * len(q) * E
                tol[3][b, c] += size * (eds + m * ads).T @ np.abs(q) * (1 + 2 * U)
                tol[4][b, c] += ((U + w + m) * p).T @ np.abs(g) * (1 + 2 * U)
        tol[3] += U * np.abs(res[3]) * (1 + 2 * U)
        tol[4] += U * np.abs(res[4]) * (1 + 2 * U)
        return res, tol

    def inside(self):
        """Rows that belong to a sequence, of q and of k."""
        q, k = np.zeros(self.n, bool), np.zeros(self.m, bool)
        q[self.cu_q[0]:self.cu_q[-1]], k[self.cu_k[0]:self.cu_k[-1]] = True, True
        return q, k

    def check(self, backward=True):
        o, lse = self.forward()
        inq, ink = self.inside()
        assert np.isnan(o[~inq]).all() and np.isnan(lse[:, ~inq]).all()
        grads = self.backward() if backward else ()
        res, tol = self.bounds(np.where(inq[:, None, None], o, 0), np.where(inq, lse, 0))
        got = [o, lse, *grads]
        rows = [inq, None, inq, ink, ink]
        for x, r, t, keep, name in zip(got, res, tol, rows, ("o", "lse", "dq", "dk", "dv")):
            if name == "lse":
                x, r, t = x[:, inq], r[:, inq], t[:, inq]
                assert np.array_equal(np.isinf(x), np.isinf(r)), name
                x, r = np.where(np.isinf(r), 0, x), np.where(np.isinf(r), 0, r)
            else:
                assert np.isnan(x[~keep]).all(), name
                x, r, t = x[keep], r[keep], t[keep]
            worst = np.max(np.abs(x - r) / np.maximum(t, 1e-30)) if x.size else 0.0
            fine = not np.isnan(x).any() and bool(np.all(np.abs(x - r) <= t + 1e-30))
            assert fine, (name, worst)
        assert L.lora_device_status(self.ws) == 0
        return got


LENS = [[1], [1, 1, 1], [31, 32, 33], [0, 5, 0, 0, 37, 0], [64, 65, 63], [127, 128, 129], [300, 1, 70], [257]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_causal_packed(lens, d):
    Case(lens, d=d, seed=sum(lens)).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (5, 1), (8, 2), (7, 7), (12, 4)])
def test_head_groups(heads, kv, d):
    Case([70, 3, 130], heads=heads, kv=kv, d=d, seed=heads).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([5, 1, 40], [9, 200, 40]), ([40, 3, 150, 2], [10, 0, 149, 1]), ([0, 4, 0], [7, 0, 130]), ([1, 1], [300, 129]),
                                   ([200], [72]), ([130, 260], [1, 3])], ids=str)
def test_keys_other_than_queries(lq, lk, causal, d):
    Case(lq, lk, d=d, causal=causal, seed=len(lq)).check()


@pytest.mark.parametrize("d", [64, 128])
def test_every_key_seen(d):
    Case([33, 1, 190, 64], d=d, causal=False, seed=3).check()


@pytest.mark.parametrize("d", [64, 128])
def test_fused_projection_strides(d):
    c = Case([40, 100, 1], heads=6, kv=2, d=d, fused=True, seed=8)
    c.check()
    assert torch.isnan(c.grad[:, -1].float()).all()   # the columns between the rows


@pytest.mark.parametrize("d", [64, 128])
def test_rows_outside_every_sequence_stay(d):
    Case([30, 140], d=d, front=13, behind=150, seed=9).check()


def test_rows_far_apart():
    """The longest strides: rows of k, v and their gradients over more than 4 GiB, the bits of dense ones."""
    c = Case([100, 41], heads=2, kv=1, d=64, seed=21)
    o, lse = c.forward()
    dq, dk, dv = c.backward()
    stride = (1 << 24) - 8
    far = [torch.empty(c.m * stride, dtype=torch.bfloat16, device="cuda").as_strided((c.m, 2, 64), (stride, 64, 1)) for _ in range(2)]
    (k, v), (fk, fv) = ((t[:, :1], t[:, 1:]) for t in far)
    k.copy_(c.dev[1])
    v.copy_(c.dev[2])
    shape = L.make_attention_shape(c.n, c.m, 2, 2, 1, 64, c.scale, k_stride=stride, v_stride=stride)
    o2, lse2, fq = torch.full_like(c.o, NAN), torch.full_like(c.lse, NAN), torch.full_like(c.o, NAN)
    L.attention_forward(shape, c.dev[0], k, v, c.cq, c.ck, o2, lse2, c.ws)
    assert np.array_equal(f64_of(o2), o) and np.array_equal(f64_of(lse2), lse)
    L.attention_backward(shape, c.dout, c.dev[0], k, v, o2, lse2, c.cq, c.ck, fq, fk, fv, c.ws)
    for a, b in ((fq, dq), (fk, dk), (fv, dv)):
        assert np.array_equal(f64_of(a.contiguous()), b)
    assert L.lora_device_status(c.ws) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_has_no_gradient_through_its_score(d):
    """Where a query sees one key, o is v, and dq and dk are 0, not what rounding leaves of dout.v - dout.o."""
    c = Case([1, 1, 1, 1], heads=6, kv=2, d=d, seed=19)
    _, _, dq, dk, dv = c.check()
    assert not dq.any() and not dk.any() and dv.any()
    c = Case([3, 1], [1, 1], heads=2, kv=2, d=d, causal=False, seed=20)
    _, _, dq, dk, _ = c.check()
    assert not dq.any() and not dk.any()


def test_many_short_sequences():
    rng = np.random.default_rng(1)
    Case(rng.integers(0, 9, 300).tolist(), heads=2, kv=1, d=64, seed=10).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,heads,kv,d", [(24, 4, 1, 64), (25, 2, 2, 128), (40, 8, 2, 64), (150, 8, 2, 64), (150, 4, 1, 128)])
def test_many_sequences_behind_earlier_keys(n, heads, kv, d, causal):
    """More and fewer sequences than are sorted, blocks of 32 rows of four heads among them, with keys in front of the
    queries, fewer keys than queries, none of either, and rows of neither side's sequences at both ends."""
    rng = np.random.default_rng(n + heads)
    lq = rng.integers(1, 20, n)
    lk = lq + rng.integers(-6, 30, n).clip(-lq)
    lq[3], lk[5], lq[n - 2] = 0, 0, 90
    lq[7], lk[7] = 75, 200
    c = Case(lq.tolist(), lk.tolist(), heads=heads, kv=kv, d=d, causal=causal, seed=n, front=9, behind=70)
    got = c.check()
    again = c.backward()
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got[2:], again))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 28])
def test_scores_of_any_documented_size(size, d):
    """Scores up to 2^28, those of a row 2^-7 of it apart and growing: the last key that a query sees has all the
    weight, so o is its value but for the roundings of p and o (2 u), and lse its score."""
    c = Case([120, 1], heads=2, kv=1, d=d, scale=1.0, seed=31)
    c.q[:], c.k[:] = 0, 0
    c.q[:, :, 3], c.k[:, 0, 3] = size, np.arange(c.m) / 128.0
    c.upload()
    o, lse = c.forward()
    last = np.arange(c.m)
    assert np.all(np.abs(o - c.v[last]) <= 2 * U * (1 + U) * np.abs(c.v[last]))
    assert np.all(np.abs(lse - size * last / 128.0) <= 8 * E * size * last / 128.0 + 8 * E)
    assert L.lora_device_status(c.ws) == 0


@pytest.mark.parametrize("scale", [0.0, 4.0, -1.0])
def test_scales(scale):
    """All weights alike; one weight of nearly 1 (scores of +-100 and more); a negative scale."""
    c = Case([150, 20], d=64, scale=scale, seed=11)
    c.check()


def test_long_sequence_rows_sampled():
    """2500 tokens: tiles that no mask touches, several key tiles a block."""
    Case([2500, 37], heads=2, kv=1, d=128, seed=12).check()


def test_weights_of_zero_against_far_maximum():
    """Keys in order of growing score: the running maximum rises with every tile."""
    c = Case([400], heads=2, kv=1, d=64, causal=False, seed=13)
    c.q[:] = B.round_bf16(np.abs(c.q))
    c.k[:] = B.round_bf16(np.linspace(-3, 3, c.m)[:, None, None] * np.ones(c.k.shape))
    c.upload()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_later_keys_never_reach_a_query(value, d):
    c = Case([200, 130], heads=2, kv=1, d=d, seed=14)
    o, lse = c.forward()
    for at in (37, 100, 150):      # in the first sequence; 37 in the diagonal tile of earlier rows
        k, v = c.dev[1].clone(), c.dev[2].clone()
        k[at], v[at, 0, ::3] = value, value
        o2, lse2 = torch.full_like(c.o, NAN), torch.full_like(c.lse, NAN)
        L.attention_forward(c.shape, c.dev[0], k, v, c.cq, c.ck, o2, lse2, c.ws)
        o2, lse2 = f64_of(o2), f64_of(lse2)
        assert np.array_equal(o2[:at], o[:at]) and np.array_equal(lse2[:, :at], lse[:, :at]), at
        assert np.array_equal(o2[200:], o[200:]) and np.array_equal(lse2[:, 200:], lse[:, 200:]), at
        # a query that sees it: an infinite value with a finite key stays where it is
        v = c.dev[2].clone()
        v[at, 0, 5] = value
        L.attention_forward(c.shape, c.dev[0], c.dev[1], v, c.cq, c.ck, c.o, c.lse, c.ws)
        got = f64_of(c.o)
        assert not np.isfinite(got[at:200, :, 5]).any() and np.array_equal(np.delete(got, 5, 2), np.delete(o, 5, 2))
        assert np.array_equal(got[:at], o[:at])
        if np.isinf(value):
            assert np.all(got[at:200, :, 5] == value)


@pytest.mark.parametrize("d,heads,kv", [(64, 2, 1), (128, 4, 2), (128, 3, 3)])
def test_later_keys_never_show_in_a_query_s_bits(d, heads, kv):
    """Finite keys of any size behind a query: they raise the running maxima of the rows next to it."""
    c = Case([300, 130], heads=heads, kv=kv, d=d, seed=18)
    o, lse = c.forward()
    for at in (1, 40, 100, 131, 260):
        k, v = c.dev[1].clone(), c.dev[2].clone()
        k[at:300] *= 30
        v[at:300] *= -7
        o2, lse2 = torch.full_like(c.o, NAN), torch.full_like(c.lse, NAN)
        L.attention_forward(c.shape, c.dev[0], k, v, c.cq, c.ck, o2, lse2, c.ws)
        o2, lse2 = f64_of(o2), f64_of(lse2)
        assert np.array_equal(o2[:at], o[:at]) and np.array_equal(lse2[:, :at], lse[:, :at]), at
        assert not np.array_equal(o2[at:300], o[at:300])
        assert np.array_equal(o2[300:], o[300:]) and np.array_equal(lse2[:, 300:], lse[:, 300:]), at


def test_a_sequence_s_nan_stays_its_own():
    c = Case([100, 90, 130], heads=4, kv=2, d=128, seed=15)
    c.forward()
    ref = c.backward()
    for t in (*c.dev, c.dout):
        t[100:190] = NAN
    L.attention_forward(c.shape, *c.dev, c.cq, c.ck, c.o, c.lse, c.ws)
    got = c.backward(c.dout)
    for a, b in zip(got, ref):
        assert np.array_equal(a[:100], b[:100]) and np.array_equal(a[190:], b[190:]) and np.isnan(a[100:190]).all()


def test_same_bits_in_every_batch_and_call():
    lens = [190, 64, 301]
    c = Case(lens, heads=4, kv=2, d=128, seed=16)
    o, lse = c.forward()
    ref = c.backward()
    again = c.backward()
    assert all(np.array_equal(a, b) for a, b in zip(ref, again))
    for b in range(3):
        s = slice(c.cu_q[b], c.cu_q[b + 1])
        one = Case([lens[b]], heads=4, kv=2, d=128)
        one.q, one.k, one.v, one.g = c.q[s], c.k[s], c.v[s], c.g[s]
        one.upload()
        o1, lse1 = one.forward()
        assert np.array_equal(o1, o[s]) and np.array_equal(lse1, lse[:, s])
        assert np.array_equal(one.backward()[0], ref[0][s])


@pytest.mark.parametrize("d,heads,kv", [(128, 8, 4), (64, 9, 3), (128, 5, 5), (64, 8, 4), (128, 6, 1), (128, 8, 2), (64, 4, 1)])
def test_large_grids(d, heads, kv):
    """Blocks of one, two and four heads of a group, of 128 and of 64 keys, sequences found by the offsets' order: many sequences of two tiles and some of several, sampled against the oracle."""
    rng = np.random.default_rng(d + heads)
    lens = rng.integers(100, 260, 140)
    lens[5], lens[77], lens[90:95] = 700, 0, [1, 128, 256, 129, 257]
    c = Case(lens.tolist(), heads=heads, kv=kv, d=d, seed=26)
    o, lse = c.forward()
    grads = c.backward()
    assert L.lora_device_status(c.ws) == 0
    again = c.backward()
    assert all(np.array_equal(a, b) for a, b in zip(grads, again))
    for b in (0, 5, 90, 91, 92, 93, 94, 139):
        s = slice(c.cu_q[b], c.cu_q[b + 1])
        one = Case([int(lens[b])], heads=heads, kv=kv, d=d)
        one.q, one.k, one.v, one.g = c.q[s], c.k[s], c.v[s], c.g[s]
        res, tol = one.bounds(o[s], lse[:, s])
        for x, r, t in zip((o[s], lse[:, s], *(g[s] for g in grads)), res, tol):
            assert np.all(np.abs(x - r) <= t + 1e-30), b


@pytest.mark.parametrize("lq,lk,d,heads,kv,causal", [([2100], [2100], 128, 64, 32, True), ([2077], [2077], 64, 66, 22, True),
                                                     ([2100], [2100], 64, 64, 64, True), ([4100, 50], [4200, 30], 128, 64, 16, True),
                                                     ([2100], [2300], 128, 64, 32, False)], ids=str)
def test_long_sequences_of_many_heads(lq, lk, d, heads, kv, causal):
    """The kernels of eight waves (two heads of a group by 128 rows, or 256 rows of one): two key heads against the
    oracle, and the bits of a call with these alone, which blocks of four waves make."""
    c = Case(lq, lk, heads=heads, kv=kv, d=d, causal=causal, seed=27)
    o, lse = c.forward()
    grads = c.backward()
    assert L.lora_device_status(c.ws) == 0
    group = heads // kv
    for kvh in (1, kv - 1):
        hs, ks = slice(kvh * group, (kvh + 1) * group), slice(kvh, kvh + 1)
        one = Case(lq, lk, heads=group, kv=1, d=d, causal=causal)
        one.q, one.g, one.k, one.v = c.q[:, hs], c.g[:, hs], c.k[:, ks], c.v[:, ks]
        one.upload()
        o1, lse1 = one.forward()
        assert np.array_equal(o1, o[:, hs]) and np.array_equal(lse1, lse[hs])
        assert np.array_equal(one.backward()[0], grads[0][:, hs])
        res, tol = one.bounds(o1, lse1)
        for x, r, t in zip((o1, lse1, grads[0][:, hs], grads[1][:, ks], grads[2][:, ks]), res, tol):
            both = np.isinf(x) & np.isinf(r)
            assert np.all(np.abs(np.where(both, 0, x) - np.where(both, 0, r)) <= t + 1e-30), kvh
    if causal:
        at = lk[0] - 700
        k, v = c.dev[1].clone(), c.dev[2].clone()
        k[at], v[at] = NAN, NAN
        L.attention_forward(c.shape, c.dev[0], k, v, c.cq, c.ck, c.o, c.lse, c.ws)
        first = at - (lk[0] - lq[0])     # the first query that sees it
        assert np.array_equal(f64_of(c.o)[:first], o[:first]) and np.array_equal(f64_of(c.lse)[:, :first], lse[:, :first])
        assert np.isnan(f64_of(c.o)[first:lq[0]]).all()


def test_gradients_against_differences():
    """The gradients of sum(dout o) against central differences of the float64 forward."""
    c = Case([9, 40], heads=2, kv=1, d=64, seed=17)
    c.forward()
    grads = c.backward()
    rng = np.random.default_rng(18)
    loss = lambda: np.sum(OA.attention_forward(c.q, c.k, c.v, c.cu_q, c.cu_k, c.scale)[0] * c.g)  # noqa: E731
    o, lse = OA.attention_forward(c.q, c.k, c.v, c.cu_q, c.cu_k, c.scale)
    _, tol = c.bounds(o, lse)
    for x, dx, t in zip((c.q, c.k, c.v), grads, tol[2:]):
        for _ in range(12):
            i = tuple(int(rng.integers(n)) for n in x.shape)
            keep = x[i]
            x[i] = keep + 1e-4
            up = loss()
            x[i] = keep - 1e-4
            num = (up - loss()) / 2e-4
            x[i] = keep
            # delta from the bf16 o: off by u sum|g o|, times p, over the keys
            extra = U * np.abs(c.g).max() * np.abs(o).max() * c.d * c.scale * np.abs(c.k).max()
            assert abs(dx[i] - num) <= t[i] + extra + 1e-6


def test_bad_offsets_are_flagged_and_left_out():
    c = Case([40, 50, 60], heads=2, kv=1, d=64, seed=19)
    o, _ = c.forward()
    for bad in ([0, 40, 30, 150], [-5, 40, 90, 150], [0, 40, 90, 151], [0, 2 ** 31 - 1, 90, 150], [-2 ** 31, 40, 90, 150]):
        cu = dev_i32(np.array(bad, np.int64).astype(np.int32))
        c.o.fill_(NAN)
        L.attention_forward(c.shape, *c.dev, cu, cu, c.o, c.lse, c.ws)
        assert L.lora_device_status(c.ws) == L.FLAG_BAD_LENGTH, bad
        got = f64_of(c.o)
        for b in range(3):
            s0, s1 = bad[b], bad[b + 1]
            if 0 <= s0 <= s1 <= c.n and (s0, s1) == (c.cu_q[b], c.cu_q[b + 1]) and all(x >= s1 or x <= s0 for x in bad):
                assert np.array_equal(got[s0:s1], o[s0:s1]), (bad, b)
        c.dout = c.put(c.g)
        L.attention_backward(c.shape, c.dout, *c.dev, c.o, c.lse, cu, cu, *c.dgrad, c.ws)
        assert L.lora_device_status(c.ws) == L.FLAG_BAD_LENGTH, bad


def test_empty_calls():
    c = Case([], heads=2, kv=1, d=64, seed=20)
    c.forward()
    c.backward()
    c = Case([0, 0], [3, 4], heads=2, kv=1, d=64, seed=21)   # keys without queries
    c.check()
    c = Case([3, 4], [0, 0], heads=2, kv=1, d=64, seed=22)
    c.check()


def test_graph_and_streams():
    c = Case([150, 1, 260], heads=4, kv=2, d=128, seed=23)
    c.dout = c.put(c.g)
    other = Case([77], heads=2, kv=1, d=64, seed=24)

    def run():
        L.attention_forward(c.shape, *c.dev, c.cq, c.ck, c.o, c.lse, c.ws)
        L.attention_backward(c.shape, c.dout, *c.dev, c.o, c.lse, c.cq, c.ck, *c.dgrad, c.ws)

    def elsewhere():
        other.forward()
        other.backward()

    _replay_check(run, [c.o, c.lse, *c.dgrad], elsewhere)
    run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (c.o, c.lse, *c.dgrad)]
    side = torch.cuda.Stream()
    for t in (c.o, c.lse, *c.dgrad):
        t.fill_(NAN)
    torch.cuda.synchronize()
    with torch.cuda.stream(other_stream := torch.cuda.Stream()):
        elsewhere()
    L.attention_forward(c.shape, *c.dev, c.cq, c.ck, c.o, c.lse, c.ws, stream=side)
    L.attention_backward(c.shape, c.dout, *c.dev, c.o, c.lse, c.cq, c.ck, *c.dgrad, c.ws, stream=side)
    side.synchronize()
    other_stream.synchronize()
    for a, b in zip(ref, (c.o, c.lse, *c.dgrad)):
        assert torch.equal(a, b)


def test_binding_refuses():
    c = Case([8], heads=2, kv=1, d=64, seed=25)
    fwd = lambda **kw: L.attention_forward(c.shape, *(kw.get(n, t) for n, t in zip(("q", "k", "v", "cq", "ck", "o", "lse", "ws"), (*c.dev, c.cq, c.ck, c.o, c.lse, c.ws))))  # noqa: E731
    for kw in ({"q": c.dev[0].float()}, {"k": c.dev[1][:4]}, {"q": c.dev[0].transpose(1, 2)}, {"cq": c.cq.long()}, {"o": c.o.cpu()},
               {"lse": c.lse.half()}, {"v": torch.empty(8, 1, 128, dtype=torch.bfloat16, device="cuda")[:, :, :64]}, {"ws": c.ws[:64]}, {"o": c.dev[0]}):
        with pytest.raises(L.LoraError):
            fwd(**kw)
