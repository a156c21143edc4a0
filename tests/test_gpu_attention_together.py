"""Attention and the key-value cache as they are used together with the layer calls.

* A training step of one attention block on a packed mixed-adapter batch: norm -> fused
  q/k/v projection (lora_forward) -> attention -> output projection, and the backward of
  all of it, against the float64 chain that starts from the inputs alone (bf16 activations
  between the stages: 2e-2 of max(|value|, rms), as the other chains).
* A rollout: prompts prefilled (kv_tables, attention_forward, kv_write), then decoding
  steps on a 4-bit base (norm to 8 bits, lora_forward_w4, kv_write, attention_decode), with
  requests that end, start anew and share the pages, in bf16 and in 8 bits.  Each decoded
  row is checked against the float64 attention over all of its request's keys and values
  so far, as they were written.
* A decoding step captured once and replayed: it walks on by itself.
"""
import numpy as np
import pytest

import oracle.attention as OA
import oracle.lora as OL
import oracle.norm as ON
import workloads as W
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import TOL_BF16, TOL_F32, DevLayer, dev_bf16, dev_i32, f64_of, rel_err  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402

EPS = 1e-6


def _bf(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def test_training_step():
    heads, kv, d, hidden = 4, 2, 64, 256
    lens = [70, 1, 130, 33]
    n = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    ids = np.repeat([0, 1, 1, 2], lens).astype(np.int32)
    ranks = [8, 16, 32]
    qkv_l = W.lora_layer(51, n, hidden, (heads + 2 * kv) * d, ranks, [32.0] * 3, ids=ids, w_std=0.08)
    out_l = W.lora_layer(52, n, heads * d, hidden, ranks, [32.0] * 3, ids=ids, w_std=0.08)
    dq_l, do_l = DevLayer(qkv_l), DevLayer(out_l)
    rng = np.random.default_rng(53)
    wb = B.to_bf16_bits(1 + 0.2 * rng.standard_normal(hidden))
    scale = d ** -0.5
    x, Wq, Aq, Bq, sq, _ = dq_l.oracle_args()
    _, Wo, Ao, Bo, so, _ = do_l.oracle_args()
    split = lambda t: (t.reshape(n, -1, d)[:, :heads], t.reshape(n, -1, d)[:, heads:heads + kv], t.reshape(n, -1, d)[:, heads + kv:])  # noqa: E731

    # ---- the float64 chain
    w = B.bf16_bits_to_f64(wb)
    y1, r1 = ON.rmsnorm_forward(x, w, EPS)
    qkv, _ = OL.lora_forward(y1, Wq, Aq, Bq, sq, ids)
    o, lse = OA.attention_forward(*split(qkv), cu, cu, scale)
    y, _ = OL.lora_forward(o.reshape(n, -1), Wo, Ao, Bo, so, ids)
    g = out_l.dy()
    do, dAo, dBo, _ = OL.lora_backward(g, o.reshape(n, -1), Wo, Ao, Bo, so, ids)
    grads = OA.attention_backward(do.reshape(n, heads, d), *split(qkv), o, lse, cu, cu, scale)
    dqkv = np.concatenate(grads, 1).reshape(n, -1)
    dy1, dAq, dBq, _ = OL.lora_backward(dqkv, y1, Wq, Aq, Bq, sq, ids)
    dx, dw = ON.rmsnorm_backward(dy1, x, w, r1)

    # ---- the library's
    Wn, rstd, n1 = dev_bf16(wb), torch.empty(n, device="cuda"), _bf(n, hidden)
    L.rmsnorm_forward(dq_l.x, Wn, EPS, n1, rstd=rstd)
    qkv_g, u1 = dq_l.forward(x=n1)
    q, k, v = split(qkv_g)
    stride = (heads + 2 * kv) * d
    shape = L.make_attention_shape(n, n, len(lens), heads, kv, d, scale, q_stride=stride, k_stride=stride, v_stride=stride)
    ws = L.empty_workspace(L.attention_workspace_bytes(shape))
    cu_g, o_g, lse_g = dev_i32(cu), _bf(n, heads, d), torch.empty(heads, n, device="cuda")
    L.attention_forward(shape, q, k, v, cu_g, cu_g, o_g, lse_g, ws)
    y_g, u2 = do_l.forward(x=o_g.view(n, -1))
    do_g, gpack_o = do_l.backward(u2, x=o_g.view(n, -1))
    dqkv_g = _bf(n, stride)
    L.attention_backward(shape, do_g.view(n, heads, d), q, k, v, o_g, lse_g, cu_g, cu_g, *split(dqkv_g), ws)
    dy1_g, gpack_q = dq_l.backward(u1, dy=dqkv_g, x=n1)
    dx_g, dw_g = _bf(n, hidden), torch.empty(hidden, device="cuda")
    L.rmsnorm_backward(dy1_g, dq_l.x, Wn, rstd, dx_g, dweight=dw_g, ws=L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, hidden)))
    for got, want, what in ((qkv_g, qkv, "qkv"), (o_g, o, "o"), (y_g, y, "y"), (do_g, do, "do"), (dqkv_g, dqkv, "dqkv"), (dx_g, dx, "dx"), (dw_g, dw, "dw")):
        e, l2 = rel_err(f64_of(got), want), np.linalg.norm(f64_of(got).reshape(-1) - want.reshape(-1)) / np.linalg.norm(want)
        print(f"[together] {what}: max {e:.3g} l2 {l2:.3g}", flush=True)
        # a chain of roundings: the norm-wise error within the tolerance, no element far out
        assert l2 < TOL_BF16 and e < 4 * TOL_BF16, what
    for dl, pack, dA, dB in ((do_l, gpack_o, dAo, dBo), (dq_l, gpack_q, dAq, dBq)):
        for got, want in zip(dl.split_grad(f64_of(pack)), (dA, dB)):
            for a, b in zip(got, want):
                assert np.linalg.norm(a - b) < 2 * TOL_BF16 * np.linalg.norm(b)
        assert dl.status() == 0
    assert L.lora_device_status(ws) == 0


class Rollout:
    """A layer's attention part for a batch of requests, on a cache of few pages."""

    def __init__(self, n, x8, seed=0, heads=4, kv=2, d=64, page=16, n_pages=40, width=8, slots=256):
        rng = np.random.default_rng(seed)
        self.n, self.heads, self.kv, self.d, self.page, self.x8, self.width = n, heads, kv, d, page, x8, width
        self.hidden, self.cols = 256, (heads + 2 * kv) * d
        self.shape = L.make_kv_shape(n, kv, d, page, n_pages, width)
        full = (n_pages, kv, page)
        if x8:
            self.c = [torch.full((*full, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
                     [torch.full((*full, d // 32), 254, dtype=torch.uint8, device="cuda") for _ in range(2)]
        else:
            self.c = [_bf(*full, d) for _ in range(2)] + [None, None]
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.table = torch.full((n, width), -5, dtype=torch.int32, device="cuda")
        self.ring = dev_i32(rng.permutation(n_pages))
        self.state = torch.tensor([0, n_pages], device="cuda")
        self.cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        self.slots, self.pos, self.seq = (torch.zeros(slots, dtype=torch.int32, device="cuda") for _ in range(3))
        self.max_len = width * page
        self.ws = torch.zeros(max(1024, L.attention_decode_workspace_bytes(self.shape, heads, self.max_len)), dtype=torch.uint8, device="cuda")
        ranks = [16, 8]
        sizes = np.array(ranks) * (self.hidden + self.cols)
        a_off = np.concatenate([[0], np.cumsum(sizes)[:-1]])
        self.pack = dev_bf16(B.to_bf16_bits(0.05 * rng.standard_normal(int(sizes.sum()))))
        self.desc = L.make_desc(a_off, a_off + np.array(ranks) * self.hidden, ranks, np.array([2.0, 4.0], np.float32))
        self.adapter = dev_i32(rng.integers(0, 2, n))
        Wb = dev_bf16(B.to_bf16_bits(0.08 * rng.standard_normal((self.cols, self.hidden))))
        self.Wd, self.pack_n = Wb, self.pack.numel()
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.codes, self.scales = u8(self.cols, self.hidden // 2), u8(self.cols, self.hidden // 32)
        L.w4_quantize(Wb, self.codes, self.scales)
        self.norm_w = dev_bf16(B.to_bf16_bits(1 + 0.1 * rng.standard_normal(self.hidden)))
        self.scale = d ** -0.5
        self.lshape = L.make_shape(n, self.hidden, self.cols, self.pack_n, self.pack_n, 2, 16, L.IDS_INTERLEAVED)
        self.lws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(self.lshape))
        self.q8, self.q8s, self.qkv, self.o = u8(n, self.hidden), u8(n, self.hidden // 32), _bf(n, self.cols), _bf(n, heads, d)
        self.x = torch.zeros(n, self.hidden, dtype=torch.bfloat16, device="cuda")
        self.one = torch.ones(n, dtype=torch.int32, device="cuda")
        self.rows = [[np.zeros((0, kv, d)) for _ in range(n)] for _ in range(2)]   # keys and values of each request, as written

    def tables(self, new):
        L.kv_tables(self.shape, self.lens, new, self.lens, self.table, self.ring, self.state, self.state, self.cu, self.slots, self.ws,
                    positions=self.pos, token_seqs=self.seq)

    def write(self, k, v, m):
        L.kv_write(self.shape, k, v, self.slots[:m], self.c[0], self.c[1], self.ws, k_scales=self.c[2], v_scales=self.c[3])

    def heads_of(self, t):
        t = t.view(t.shape[0], -1, self.d)
        return t[:, :self.heads], t[:, self.heads:self.heads + self.kv], t[:, self.heads + self.kv:]

    def stored(self, t):
        """What the cache holds for rows t."""
        t = f64_of(t)
        if self.x8 and len(t):
            q, e = ON.quantize8(t.reshape(-1, self.d))
            t = (q * np.repeat(np.exp2(e.astype(float)), 32, -1)).reshape(t.shape)
        return t

    def decode_step(self):
        """One new token of every request: norm to 8 bits, projection with adapters, cache, attention."""
        self.tables(self.one)
        L.rmsnorm_forward_q8(self.x, self.norm_w, EPS, self.q8, self.q8s)
        L.lora_forward_w4(self.lshape, self.q8, self.codes, self.scales, self.pack, self.pack, self.desc, self.adapter, self.qkv, self.lws,
                          x_scales=self.q8s)
        q, k, v = self.heads_of(self.qkv)
        self.write(k, v, self.n)
        L.attention_decode(self.shape, q, self.c[0], self.c[1], self.table, self.lens, self.max_len, self.scale, self.o, self.ws,
                           k_scales=self.c[2], v_scales=self.c[3])

    def note(self, k, v, lens_before, lens_after):
        k, v = self.stored(k), self.stored(v)
        at = 0
        for b in range(self.n):
            m = lens_after[b] - lens_before[b]
            for rows, t in zip(self.rows, (k, v)):
                rows[b] = np.concatenate([rows[b], t[at:at + m]])
            at += m

    def check_decoded(self):
        q, o = f64_of(self.heads_of(self.qkv)[0]), f64_of(self.o)
        for b in range(self.n):
            for h in range(self.heads):
                c = h * self.kv // self.heads
                want, _, p = OA.head_forward(q[b, h][None], self.rows[0][b][:, c], self.rows[1][b][:, c], self.scale, False)
                # the weights and o rounded to bf16, and fp32 scores: see test_gpu_kvcache
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1e-4) * (p @ np.abs(self.rows[1][b][:, c]))
                assert np.all(np.abs(o[b, h] - want[0]) <= tol[0] * (1 + 2.0 ** -7)), (b, h)


@pytest.mark.parametrize("x8", [False, True])
def test_rollout(x8):
    r = Rollout(5, x8, seed=60)
    rng = np.random.default_rng(61)

    def prefill(new):
        """Prompts of the requests that have some (rows appended; 0: none, -1: the request ends),
        projected and attended, each among its own rows, in one packed batch."""
        before = r.lens.tolist()
        r.tables(dev_i32(new))
        after, n = r.lens.tolist(), int(sum(max(v, 0) for v in new))
        assert L.lora_device_status(r.ws) == 0 and r.cu.tolist()[-1] == n
        for b in range(r.n):
            if after[b] < before[b]:
                for rows in r.rows:
                    rows[b] = rows[b][:0]
        x = dev_bf16(B.to_bf16_bits(rng.standard_normal((n, r.hidden))))
        shape = L.make_shape(n, r.hidden, r.cols, r.pack_n, r.pack_n, 2, 16, L.IDS_INTERLEAVED)
        ids = r.adapter[r.seq[:n].long()].contiguous()        # each row's adapter by its request
        y, u = _bf(n, r.cols), _bf(2, n, 16)
        L.lora_forward(shape, x, r.Wd, r.pack, r.pack, r.desc, ids, y, u, L.empty_workspace(L.lora_workspace_bytes(shape)))
        q, k, v = r.heads_of(y)
        sh = L.make_attention_shape(n, n, r.n, r.heads, r.kv, r.d, r.scale, q_stride=r.cols, k_stride=r.cols, v_stride=r.cols)
        o, lse = _bf(n, r.heads, r.d), torch.empty(r.heads, n, device="cuda")
        ws = L.empty_workspace(L.attention_workspace_bytes(sh))
        L.attention_forward(sh, q, k, v, r.cu, r.cu, o, lse, ws)
        r.write(k, v, n)
        assert L.lora_device_status(ws) == 0 and L.lora_device_status(r.ws) == 0
        want, want_lse = OA.attention_forward(*(f64_of(t) for t in (q, k, v)), r.cu.tolist(), r.cu.tolist(), r.scale)
        assert rel_err(f64_of(o), want) < TOL_BF16 and rel_err(f64_of(lse), want_lse) < TOL_F32
        r.note(k, v, [0 if m < 0 else b for m, b in zip(new, before)], after)

    prefill([40, 15, 0, 1, 63])
    for step in range(24):
        if step == 8:
            prefill([-1, 0, 16, 0, 0])      # a request ends (another starts in its place), one gets more rows
        if step == 15:
            prefill([30, 0, -1, 0, -1])
        before = r.lens.tolist()
        r.x.copy_(dev_bf16(B.to_bf16_bits(rng.standard_normal((r.n, r.hidden)))))
        r.decode_step()
        assert L.lora_device_status(r.ws) == 0 and L.lora_device_status(r.lws) == 0
        _, k, v = r.heads_of(r.qkv)
        r.note(k, v, before, r.lens.tolist())
        r.check_decoded()
    held = [r.table[b, :-(-ln // r.page)].tolist() for b, ln in enumerate(r.lens.tolist())]
    free = [r.ring[i % r.ring.numel()].item() for i in range(*r.state.tolist())]
    assert sorted(sum(held, []) + free) == list(range(r.ring.numel()))


@pytest.mark.parametrize("x8", [False, True])
def test_captured_step_walks_on(x8):
    r, other = Rollout(3, x8, seed=62), Rollout(2, not x8, seed=63)
    rng = np.random.default_rng(64)
    other.decode_step()
    r.decode_step()
    torch.cuda.synchronize()
    r.lens.zero_()
    r.ring.copy_(torch.arange(r.ring.numel(), device="cuda", dtype=torch.int32))
    r.state.copy_(torch.tensor([0, r.ring.numel()]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.decode_step()
    for step in range(40):                      # across page ends
        r.x.copy_(dev_bf16(B.to_bf16_bits(rng.standard_normal((r.n, r.hidden)))))
        g.replay()
        torch.cuda.synchronize()
        _, k, v = r.heads_of(r.qkv)
        r.note(k, v, [step] * r.n, [step + 1] * r.n)
        assert r.lens.tolist() == [step + 1] * r.n
        if step % 5 == 4 or step < 2:
            r.check_decoded()
        other.decode_step() if step < 30 else None
    assert L.lora_device_status(r.ws) == 0


def test_two_graphs_share_a_workspace():
    """Two captured steps on one workspace, replayed one after the other on one stream."""
    a, b = Rollout(3, False, seed=65), Rollout(3, False, seed=65)
    b.ws = a.ws
    for r in (a, b):
        r.x.copy_(torch.randn(r.n, r.hidden, generator=torch.Generator("cuda").manual_seed(5), device="cuda"))
        r.decode_step()
    torch.cuda.synchronize()
    graphs = []
    for r in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            r.decode_step()
    for _ in range(20):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o, b.o) and torch.equal(a.lens, b.lens) and torch.equal(a.table, b.table) and a.lens.tolist() == [21] * 3
    assert L.lora_device_status(a.ws) == 0
