"""The norm, the 4-bit products and the clipped optimizer as they are used together
with the library's other calls, and replayed from captured graphs.

* A training step of one block and the lm_head on a mixed-adapter batch: norm with
  the residual's addition -> lora_forward -> final norm -> token_logprobs ->
  loss_grad -> token_logprobs_backward -> rmsnorm_backward -> lora_backward ->
  rmsnorm_backward -> adam_step_clipped, every stage against the float64 chain
  that starts from the inputs alone.  The chain carries bf16 activations: the
  tolerance is the one of the other chains (2e-2 of max(|value|, rms)).
* A decoding step: norm to 8 bits -> 4-bit mixed-adapter projection -> norm -> 4-bit
  lm_head, each call against float64 on the bits it was given.
* Every call captured into a graph and replayed, with eager work between the
  replays; two graphs that share one workspace; the step counters count on.
"""
import numpy as np
import pytest

import oracle.clip as OC
import oracle.logprob as OP
import oracle.lora as OL
import oracle.loss as OLs
import oracle.norm as ON
import oracle.w4 as OQ
import workloads as W
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import TOL_BF16, DevLayer, bits_of, dev_bf16, dev_f32, dev_i32, f64_of, rel_err  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402
from test_gpu_graph import _replay_check  # noqa: E402

EPS = 1e-6


def _bf(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _tables(c):
    """Each adapter's A and B of the pack as tensors of a group."""
    out = []
    for i in range(c.n_adapters):
        r = int(c.ranks[i])
        out += [(int(c.a_off[i]), r * c.d_in, i), (int(c.b_off[i]), r * c.d_out, i)]
    return out


def test_training_step():
    c = W.tiny_chain(1)
    lay, targets, weights = c.layer, c.targets, c.weights
    dl = DevLayer(lay)
    n, d, V = lay.n_tokens, lay.d_out, c.U_bits.shape[0]
    assert lay.d_in == lay.d_out
    rng = np.random.default_rng(12)
    rb = B.to_bf16_bits(rng.standard_normal((n, d)))
    w1, w2 = (B.to_bf16_bits(1 + 0.2 * rng.standard_normal(d)) for _ in range(2))
    x, Wb, A, Bm, s, ids = dl.oracle_args()
    U64 = c.U()

    # ---- the float64 chain
    h_o = B.round_bf16(x + B.bf16_bits_to_f64(rb))
    y1_o, r1_o = ON.rmsnorm_forward(h_o, B.bf16_bits_to_f64(w1), EPS)
    y_o, _ = OL.lora_forward(y1_o, Wb, A, Bm, s, ids)
    h2_o = y_o + h_o
    y2_o, r2_o = ON.rmsnorm_forward(h2_o, B.bf16_bits_to_f64(w2), EPS)
    lp_o, _ = OP.token_logprobs(y2_o, U64, targets)
    _, dlp_o = OLs.loss_grad(OLs.CROSS_ENTROPY, lp_o, weights)
    dy2_o = OP.token_logprobs_backward(y2_o, U64, targets, dlp_o)
    dh2_o, dw2_o = ON.rmsnorm_backward(dy2_o, h2_o, B.bf16_bits_to_f64(w2), r2_o)
    dy1_o, dA_o, dB_o, _ = OL.lora_backward(dh2_o, y1_o, Wb, A, Bm, s, ids)
    dx_o, dw1_o = ON.rmsnorm_backward(dy1_o, h_o, B.bf16_bits_to_f64(w1), r1_o, dh2_o)
    g_o = np.zeros(lay.pack_elems)
    for i in range(lay.n_adapters):
        a, b, r = int(lay.a_off[i]), int(lay.b_off[i]), int(lay.ranks[i])
        g_o[a:a + r * lay.d_in], g_o[b:b + r * d] = dA_o[i].reshape(-1), dB_o[i].reshape(-1)
    tensors = _tables(lay)
    max_norm = 0.5 * float(np.median(OC.norms(tensors, lay.n_adapters, g_o)))

    # ---- the library's chain
    W1, W2 = dev_bf16(w1), dev_bf16(w2)
    h, y1, h2, y2 = (_bf(n, d) for _ in range(4))
    r1, r2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    L.rmsnorm_forward(dl.x, W1, EPS, y1, rstd=r1, residual=dev_bf16(rb), h=h)
    y, u = dl.forward(x=y1)
    L.rmsnorm_forward(y, W2, EPS, y2, rstd=r2, residual=h, h=h2)
    U = dev_bf16(c.U_bits)
    Ut = _bf(d, V)
    L.lora_transpose_bf16(U, Ut)
    tgt, lp, lse = dev_i32(targets), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    L.token_logprobs(y2, U, tgt, lp, lse, L.empty_workspace(L.token_logprobs_workspace_bytes(n, V)))
    loss, dlp = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
    L.loss_grad(L.LOSS_CROSS_ENTROPY, lp, dev_f32(weights), None, None, None, None, loss, dlp,
                L.empty_workspace(L.loss_grad_workspace_bytes(n)))
    dy2, dh2, dx = (_bf(n, d) for _ in range(3))
    L.token_logprobs_backward(y2, U, Ut, tgt, lse, dlp, dy2, L.empty_workspace(L.token_logprobs_backward_workspace_bytes(n, V, 256)))
    dw1, dw2 = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, d))
    L.rmsnorm_backward(dy2, h2, W2, r2, dh2, dweight=dw2, ws=ws)
    dy1, grad = dl.backward(u, dy=dh2, x=y1)
    L.rmsnorm_backward(dy1, h, W1, r1, dx, dh=dh2, dweight=dw1, ws=ws)
    for got, want, what in ((y1, y1_o, "norm"), (y, y_o, "layer"), (y2, y2_o, "final norm"), (lp, lp_o, "logprob"),
                            (dy2, dy2_o, "d final norm"), (dh2, dh2_o, "d layer"), (dx, dx_o, "dx"), (dw1, dw1_o, "dw1"), (dw2, dw2_o, "dw2")):
        assert rel_err(f64_of(got), want) < TOL_BF16, what

    shape, table = L.make_grad_table(tensors, lay.n_adapters, lay.pack_elems)
    p0 = W.bf16_bits_to_f32(lay.pack_bits).astype(np.float32)
    m0, v0 = np.zeros(lay.pack_elems, np.float32), np.zeros(lay.pack_elems, np.float32)
    for o, k, _ in tensors:     # moments of the gradient's size: the update is then smooth in it
        rms = np.sqrt(np.mean(g_o[o:o + k] ** 2))
        m0[o:o + k], v0[o:o + k] = 0.5 * rms * rng.standard_normal(k), rms * rms * rng.uniform(0.5, 1.5, k)
    p, m, v, pb = dev_f32(p0), dev_f32(m0), dev_f32(v0), dl.pack.clone()
    steps = torch.full((lay.n_adapters,), 2, dtype=torch.int64, device="cuda")
    norms = torch.empty(lay.n_adapters, device="cuda")
    ws_g = L.adam_step_clipped(shape, table, steps, p, grad, m, v, max_norm, 1e-4, p_bf16=pb, norms=norms)
    p_o, m_o, v_o, _, n_o = OC.adam_clipped(tensors, lay.n_adapters, [2] * lay.n_adapters, p0, g_o, m0, v0, max_norm, 1e-4)
    assert rel_err(f64_of(norms), n_o) < TOL_BF16
    dp, dp_o = f64_of(p) - p0, p_o - p0
    for o, k, _ in tensors:
        at = slice(o, o + k)
        assert rel_err(f64_of(m)[at], m_o[at]) < TOL_BF16
        scale = np.maximum(np.abs(dp_o[at]), np.sqrt(np.mean(dp_o[at] ** 2)))
        # the stored fp32 parameter resolves the step only to one ulp of p
        assert np.all(np.abs(dp[at] - dp_o[at]) <= TOL_BF16 * scale + np.spacing(np.abs(p_o[at]).astype(np.float32)))
    # the next forward reads the updated bf16 pack
    assert not np.array_equal(bits_of(pb), lay.pack_bits) and dl.status() == 0 and L.lora_device_status(ws_g) == 0


def _decode_inputs(n=9, H=512, V=1024, seed=13):
    rng = np.random.default_rng(seed)
    ranks = [16, 8, 32]
    sizes = np.array(ranks) * 2 * H
    a_off = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int64)
    b_off = a_off + np.array(ranks) * H
    pack = B.to_bf16_bits(0.1 * rng.standard_normal(int(sizes.sum())))
    d = {"n": n, "H": H, "V": V, "ranks": ranks, "a_off": a_off, "b_off": b_off, "pack": pack, "scale": np.array([2.0, 4.0, 1.0], np.float32),
         "x": B.to_bf16_bits(rng.standard_normal((n, H))), "res": B.to_bf16_bits(rng.standard_normal((n, H))),
         "w1": B.to_bf16_bits(1 + 0.1 * rng.standard_normal(H)), "w2": B.to_bf16_bits(1 + 0.1 * rng.standard_normal(H)),
         "W": B.to_bf16_bits(0.05 * rng.standard_normal((H, H))), "U": B.to_bf16_bits(0.05 * rng.standard_normal((V, H))),
         "ids": rng.integers(0, 3, n).astype(np.int32)}
    return d


class _Decode:
    """One decoding step's buffers; run() makes its calls."""

    def __init__(self, d):
        self.d = d
        n, H, V = d["n"], d["H"], d["V"]
        up = lambda k: dev_bf16(d[k])  # noqa: E731
        self.x, self.res, self.w1, self.w2, self.pack = (up(k) for k in ("x", "res", "w1", "w2", "pack"))
        self.desc, self.ids = L.make_desc(d["a_off"], d["b_off"], d["ranks"], d["scale"]), dev_i32(d["ids"])
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.Wc, self.Ws, self.Uc, self.Us = u8(H, H // 2), u8(H, H // 32), u8(V, H // 2), u8(V, H // 32)
        L.w4_quantize(up("W"), self.Wc, self.Ws)
        L.w4_quantize(up("U"), self.Uc, self.Us)
        self.h, self.h2, self.y, self.z, self.logits = _bf(n, H), _bf(n, H), _bf(n, H), _bf(n, H), _bf(n, V)
        self.q, self.qs = u8(n, H), u8(n, H // 32)
        self.shape = L.make_shape(n, H, H, len(d["pack"]), len(d["pack"]), 3, 32, L.IDS_INTERLEAVED)
        self.ws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(self.shape))

    def run(self):
        L.rmsnorm_forward_q8(self.x, self.w1, EPS, self.q, self.qs, residual=self.res, h=self.h)
        L.lora_forward_w4(self.shape, self.q, self.Wc, self.Ws, self.pack, self.pack, self.desc, self.ids, self.y, self.ws, x_scales=self.qs)
        L.rmsnorm_forward(self.y, self.w2, EPS, self.z, residual=self.h, h=self.h2)
        L.w4_linear(self.z, self.Uc, self.Us, self.logits)

    def outs(self):
        return [self.q, self.qs, self.h, self.y, self.h2, self.z, self.logits]


def test_decoding_step():
    d = _decode_inputs()
    s = _Decode(d)
    s.run()
    f64, H = B.bf16_bits_to_f64, d["H"]
    h = B.to_bf16_bits_f32(B.bf16_bits_to_f32(d["x"]) + B.bf16_bits_to_f32(d["res"])).reshape(d["n"], H)
    assert np.array_equal(bits_of(s.h), h)
    v, _ = ON.rmsnorm_forward(f64(h), f64(d["w1"]), EPS)
    q = s.q.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64) * np.repeat(np.exp2(s.qs.cpu().numpy().astype(float) - 127), 32, axis=1)
    assert np.linalg.norm(q - v) < 2.0 ** -4 * np.linalg.norm(v)
    Wv, Uv = (OQ.values(*OQ.quantize(f64(d[k]))) for k in ("W", "U"))
    p = f64(d["pack"])
    A = [p[a:a + r * H].reshape(r, H) for a, r in zip(d["a_off"], d["ranks"])]
    Bm = [p[b:b + r * H].reshape(H, r) for b, r in zip(d["b_off"], d["ranks"])]
    y, _ = OL.lora_forward(q, Wv, A, Bm, d["scale"].astype(np.float64), d["ids"])
    assert rel_err(f64_of(s.y), y) < TOL_BF16
    h2 = B.to_bf16_bits_f32(B.bf16_bits_to_f32(bits_of(s.y)) + B.bf16_bits_to_f32(h)).reshape(d["n"], H)
    assert np.array_equal(bits_of(s.h2), h2)
    z, _ = ON.rmsnorm_forward(f64(h2), f64(d["w2"]), EPS)
    assert rel_err(f64_of(s.z), z) < TOL_BF16
    assert rel_err(f64_of(s.logits), f64_of(s.z) @ Uv.T) < TOL_BF16
    assert L.lora_device_status(s.ws) == 0


@pytest.mark.parametrize("n", [1, 9, 40])
def test_decoding_step_graph(n):
    s, other = _Decode(_decode_inputs(n)), _Decode(_decode_inputs(5, seed=14))
    _replay_check(s.run, [t for t in s.outs() if t.dtype == torch.bfloat16], other.run)
    assert L.lora_device_status(s.ws) == 0


def test_norm_backward_graph():
    n, H = 3000, 1024
    x, dy, dh = (torch.randn(n, H, device="cuda").to(torch.bfloat16) for _ in range(3))
    w, rstd = torch.randn(H, device="cuda").to(torch.bfloat16), torch.rand(n, device="cuda") + 0.5
    dx, dw = _bf(n, H), torch.empty(H, device="cuda")
    ws = L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, H))
    scratch = torch.empty(1 << 20, device="cuda")
    _replay_check(lambda: L.rmsnorm_backward(dy, x, w, rstd, dx, dh=dh, dweight=dw, ws=ws), [dx, dw], lambda: scratch.normal_())


def _capture(run):
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            run()
    torch.cuda.current_stream().wait_stream(side)
    return g


def test_two_graphs_share_a_workspace_and_count_steps():
    n = 50000
    tensors = [(0, 20000, 0), (20000, 9000, 1), (30000, 19999, 1)]
    shape, table = L.make_grad_table(tensors, 2, n)
    ws = L.empty_workspace(L.grad_workspace_bytes(shape))
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, device="cuda", generator=gen) for _ in range(2)]

    def state():
        z = torch.zeros(n, device="cuda")
        return [torch.ones(n, device="cuda"), z, z.clone(), torch.zeros(2, dtype=torch.int64, device="cuda")]

    def step(st, g):
        L.adam_step_clipped(shape, table, st[3], st[0], g, st[1], st[2], 1.0, 1e-3, ws=ws)

    eager, played = [state(), state()], [state(), state()]
    order = [0, 1, 1, 0, 1, 0, 0]
    for k in order:
        step(eager[k], grads[k])
    graphs = [_capture(lambda k=k: step(played[k], grads[k])) for k in range(2)]
    scratch = torch.empty(1 << 20, device="cuda")
    for k in order:
        graphs[k].replay()
        scratch.normal_()
        torch.cuda.synchronize()
    for k in range(2):
        assert played[k][3].tolist() == eager[k][3].tolist() == [order.count(k)] * 2
        for a, b in zip(played[k], eager[k]):
            assert torch.equal(a, b)
    assert L.lora_device_status(ws) == 0


def test_grad_clip_graph():
    n = 300000
    shape, table = L.make_grad_table([(0, 100000, 0), (100003, 150000, 1)], 2, n)
    ws, norms, out = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(2, device="cuda"), torch.zeros(n, device="cuda")
    g = torch.randn(n, device="cuda")
    scratch = torch.empty(1 << 20, device="cuda")
    got = [torch.empty(250000, device="cuda"), norms]

    def run():
        L.grad_clip(shape, table, g, 3.0, out, norms, ws)
        got[0].copy_(torch.cat((out[:100000], out[100003:250003])))

    _replay_check(run, got, lambda: scratch.normal_())
    assert L.lora_device_status(ws) == 0


def test_neighbouring_parts_of_one_buffer():
    """Operands that lie one behind the other in one allocation share no byte and are taken."""
    n, H = 4, 64
    rng = np.random.default_rng(14)
    part = torch.empty(5, n, H, dtype=torch.bfloat16, device="cuda")
    part[:] = torch.randn(5, n, H, device="cuda").to(torch.bfloat16)
    w, rstd = dev_bf16(B.to_bf16_bits(rng.standard_normal(H))), torch.rand(n, device="cuda")
    apart = [t.clone() for t in part]
    out = [_bf(n, H) for _ in range(3)]
    L.rmsnorm_backward(apart[0], apart[2], w, rstd, out[0])
    L.rmsnorm_backward(part[0], part[2], w, rstd, part[1])     # dx in front of h
    L.rmsnorm_backward(part[0], part[2], w, rstd, part[3])     # and behind it
    assert np.array_equal(bits_of(part[1]), bits_of(out[0])) and np.array_equal(bits_of(part[3]), bits_of(out[0]))
    codes = torch.randint(0, 256, (H, H // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((H, H // 32), 127, dtype=torch.uint8, device="cuda")
    L.w4_linear(apart[2], codes, scales, out[1])
    L.w4_linear(part[2], codes, scales, part[1])
    L.w4_linear(part[2], codes, scales, part[3])
    assert np.array_equal(bits_of(part[1]), bits_of(out[1])) and np.array_equal(bits_of(part[3]), bits_of(out[1]))
    raw = torch.empty(3 * n * H + n * H // 32, dtype=torch.uint8, device="cuda")     # q, x, q_scales
    x = raw[n * H:3 * n * H].view(torch.bfloat16).view(n, H)
    x.copy_(apart[0])
    q, s = torch.empty(n, H, dtype=torch.uint8, device="cuda"), torch.empty(n, H // 32, dtype=torch.uint8, device="cuda")
    L.rmsnorm_forward_q8(apart[0], w, EPS, q, s)
    L.rmsnorm_forward_q8(x, w, EPS, raw[:n * H].view(n, H), raw[3 * n * H:].view(n, H // 32))
    assert torch.equal(raw[:n * H].view(n, H), q) and torch.equal(raw[3 * n * H:].view(n, H // 32), s)
