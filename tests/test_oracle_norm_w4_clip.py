"""Pins for oracle.norm, oracle.w4 and oracle.clip (CPU only): the norm and its
gradients against torch autograd in float64, the 8-bit rounding against torch's
e4m3 conversion, the 4-bit rounding by brute force, clipping against
torch.nn.utils.clip_grad_norm_ and AdamW on top against torch.optim.AdamW."""
import numpy as np
import pytest
import torch

import oracle.clip as OC
import oracle.norm as ON
import oracle.w4 as OQ


def test_norm_and_its_gradients_match_autograd():
    rng = np.random.default_rng(0)
    h, w, dv, dh = rng.standard_normal((5, 37)), rng.standard_normal(37), rng.standard_normal((5, 37)), rng.standard_normal((5, 37))
    ht, wt = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    v = torch.nn.functional.rms_norm(ht, (37,), wt, 1e-6)
    (v * torch.tensor(dv)).sum().backward()
    got, rstd = ON.rmsnorm_forward(h, w, 1e-6)
    np.testing.assert_allclose(got, v.detach().numpy(), rtol=1e-12)
    d, dw = ON.rmsnorm_backward(dv, h, w, rstd, dh)
    np.testing.assert_allclose(d, ht.grad.numpy() + dh, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_eight_bit_rounding():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-40, 40, (40, 1)))
    v[3, :32] = 0.0
    v[4, :32] = 448.0 * 2.0 ** -3       # the largest value without a larger scale
    v[5, :32] = 448.0 * 2.0 ** -3 * (1 + 2 ** -20)
    q, e = ON.quantize8(v)
    assert e[4, 0] == -3 and e[5, 0] == -2 and e[3, 0] == -126
    top = np.abs(v).reshape(40, 2, 32).max(axis=2)
    live = top > 0
    assert np.all(top <= 448 * np.exp2(e.astype(float))) and np.all(top[live] > 448 * np.exp2(e[live] - 1.0))
    s = (v.reshape(40, 2, 32) * np.exp2(-e.astype(float))[..., None]).reshape(40, 64)
    # exact in fp32 is not given: compare on values that are
    s32 = s.astype(np.float32)
    ref = torch.from_numpy(s32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ON.round_to_grid(s32.astype(np.float64), 3, -6), ref)


def test_four_bit_rounding_by_brute_force():
    rng = np.random.default_rng(2)
    W = rng.standard_normal((6, 64)) * np.exp2(rng.integers(-30, 30, (6, 1)))
    W[0, :32] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.tile([1, -1], 16)  # ties
    W[1, :32] = 0.0
    codes, scales = OQ.quantize(W)
    v = OQ.values(codes, scales)
    want = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert np.array_equal(np.abs(v[0, :8]), want) and np.all(v[1, :32] == 0)
    for i in range(6):
        for b in range(2):
            w = W[i, 32 * b:32 * b + 32]
            s = 2.0 ** (int(scales[i, b]) - 127)
            assert np.max(np.abs(w)) <= 6 * s and (not w.any() or np.max(np.abs(w)) > 3 * s)
            grid = np.concatenate([OQ.MAGNITUDES, -OQ.MAGNITUDES]) * s
            best = np.min(np.abs(w[:, None] - grid), axis=1)
            assert np.array_equal(np.abs(w - v[i, 32 * b:32 * b + 32]), best)


@pytest.mark.parametrize("max_norm", [0.3, 1e3, 0.0])
def test_clip_and_adam_match_torch(max_norm):
    rng = np.random.default_rng(3)
    tensors = [(2, 30, 0), (40, 17, 0), (60, 25, 1), (90, 0, 1)]
    g, p = rng.standard_normal(100), rng.standard_normal(100)
    got, n = OC.clip(tensors, 3, g, max_norm)
    assert n[2] == 0
    pa, ma, va, st, _ = OC.adam_clipped(tensors, 3, [0, 0, 7], p, g, np.zeros(100), np.zeros(100), max_norm, 1e-2, weight_decay=0.1)
    assert list(st) == [1, 1, 8]
    for a in (0, 1):
        prm = [torch.nn.Parameter(torch.tensor(p[o:o + c])) for o, c, b in tensors if b == a]
        for q, (o, c, b) in zip(prm, [t for t in tensors if t[2] == a]):
            q.grad = torch.tensor(g[o:o + c])
        total = torch.nn.utils.clip_grad_norm_(prm, max_norm, foreach=False)
        assert abs(float(total) - n[a]) < 1e-12
        opt = torch.optim.AdamW(prm, lr=1e-2, eps=1e-8, weight_decay=0.1, foreach=False)
        for q, (o, c, b) in zip(prm, [t for t in tensors if t[2] == a]):
            np.testing.assert_allclose(got[o:o + c], q.grad.numpy(), rtol=1e-12)
        opt.step()
        for q, (o, c, b) in zip(prm, [t for t in tensors if t[2] == a]):
            np.testing.assert_allclose(pa[o:o + c], q.detach().numpy(), rtol=1e-11, atol=1e-13)
    outside = np.ones(100, bool)
    for o, c, _ in tensors:
        outside[o:o + c] = False
    assert np.array_equal(pa[outside], p[outside]) and not got[outside].any()


def test_clip_leaves_a_non_finite_group():
    g = np.array([1.0, np.inf, 2.0, 3.0])
    out, n = OC.clip([(0, 2, 0), (2, 2, 1)], 2, g, 0.1)
    assert np.array_equal(out[:2], g[:2]) and np.isinf(n[0]) and np.all(out[2:] < 0.1)
    p, m, v, st, _ = OC.adam_clipped([(0, 2, 0), (2, 2, 1)], 2, [4, 4], np.ones(4), g, np.zeros(4), np.zeros(4), 0.1, 1e-2)
    assert list(st) == [4, 5] and np.all(p[:2] == 1) and np.all(p[2:] < 1)
