"""rmsnorm_forward, rmsnorm_forward_q8 and rmsnorm_backward against oracle.norm.

Tolerances, from the arithmetic: a bf16 rounding is off by at most 2^-8 of the
value; rstd is an fp32 sum of H squares held as at most 32 terms a lane, 6
shuffle steps and 16 waves, each step off by 2^-24 of the partial sum, so by
at most 54 * 2^-24 of the sum and half of that after the root, with two roundings
more: 2^-19 bounds it.  Products of three fp32 factors add 2^-22.
"""
import numpy as np
import pytest

import oracle.norm as ON
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import bits_of, dev_bf16, dev_f32, f64_of  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402

EPS = 1e-6
U16 = 2.0 ** -8
U32 = 2.0 ** -19

SHAPES = [(1, 1), (3, 7), (5, 8), (1, 32), (9, 33), (70, 64), (257, 128), (3, 136), (5, 250), (33, 512), (4, 513),
          (2, 520), (7, 1000), (5, 1024), (3, 1032), (1, 2048), (300, 2048), (2, 4096), (1, 4099), (3, 12288),
          (2, 16384), (2, 16400), (2, 20001), (1, 32768)]


def _rows(rng, n, H):
    """Rows of different sizes, a few columns much larger, one row zero where there are several."""
    x = rng.standard_normal((n, H)) * np.exp2(rng.integers(-8, 8, (n, 1)))
    x[:, rng.random(H) < 0.02] *= 30
    if n > 2:
        x[n // 2] = 0
    return B.to_bf16_bits(x)


def _bits_to_f32(b):
    return B.bf16_bits_to_f32(b)


def _empty(n, H):
    return torch.full((n, H), float("nan"), dtype=torch.bfloat16, device="cuda")


def _close(got, want, rel, extra=0.0):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= rel * np.abs(want) + extra)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,H", SHAPES)
def test_forward(n, H, residual):
    rng = np.random.default_rng(n * 100003 + H)
    xb, rb, wb = _rows(rng, n, H), _rows(rng, n, H), B.to_bf16_bits(1 + 0.3 * rng.standard_normal(H))
    h32 = _bits_to_f32(xb) + (_bits_to_f32(rb) if residual else np.float32(0))   # one fp32 sum, then one rounding
    hb = B.to_bf16_bits_f32(h32).reshape(n, H) if residual else xb
    x, w, y = dev_bf16(xb), dev_bf16(wb), _empty(n, H)
    h, rstd = (_empty(n, H) if residual else None), torch.full((n,), float("nan"), device="cuda")
    L.rmsnorm_forward(x, w, EPS, y, rstd=rstd, residual=dev_bf16(rb) if residual else None, h=h)
    v, r = ON.rmsnorm_forward(B.bf16_bits_to_f64(hb), B.bf16_bits_to_f64(wb), EPS)
    if residual:
        assert np.array_equal(bits_of(h), hb)
    _close(f64_of(rstd), r, U32)
    _close(f64_of(y), v, U16 + 2 * U32)
    # without rstd the same bits, and in place
    y2 = x.clone()
    L.rmsnorm_forward(y2, w, EPS, y2, residual=dev_bf16(rb) if residual else None, h=h)
    assert np.array_equal(bits_of(y2), bits_of(y))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,H", [s for s in SHAPES if s[1] % 32 == 0] + [(5, 96), (4097, 64), (3, 544), (2, 16416)])
def test_forward_eight_bits(n, H, residual):
    rng = np.random.default_rng(n * 7 + H)
    xb, rb, wb = _rows(rng, n, H), _rows(rng, n, H), B.to_bf16_bits(1 + 0.3 * rng.standard_normal(H))
    wb[:32] = 0                                              # a block of zeros
    h32 = _bits_to_f32(xb) + (_bits_to_f32(rb) if residual else np.float32(0))
    hb = B.to_bf16_bits_f32(h32).reshape(n, H)
    h, rstd = (_empty(n, H) if residual else None), torch.empty(n, device="cuda")
    q = torch.full((n, H), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((n, H // 32), 255, dtype=torch.uint8, device="cuda")
    L.rmsnorm_forward_q8(dev_bf16(xb), dev_bf16(wb), EPS, q, s, rstd=rstd, residual=dev_bf16(rb) if residual else None, h=h)
    v, r = ON.rmsnorm_forward(B.bf16_bits_to_f64(hb), B.bf16_bits_to_f64(wb), EPS)
    _, e = ON.quantize8(v)
    if residual:
        assert np.array_equal(bits_of(h), hb)
    _close(f64_of(rstd), r, U32)
    got_e = s.cpu().numpy().astype(int) - 127
    top = np.abs(v).reshape(n, -1, 32).max(axis=2) / (448 * np.exp2(e.astype(float)))
    border = (top > 1 - 2 * U32) | (top < 0.5 * (1 + 2 * U32))   # either exponent, as fp32 falls
    assert np.all((got_e == e) | (border & (e > -126) & (np.abs(got_e - e) == 1)))
    scale = np.repeat(np.exp2(got_e.astype(float)), 32, axis=1)
    val = q.view(torch.float8_e4m3fn).to(torch.float32).cpu().numpy().astype(np.float64) * scale
    # half a step: 2^-4 of the value, 2^-10 of the scale among the subnormals
    bad = ~(np.abs(val - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * scale) * (1 + U32) + 2 * U32 * np.abs(v))
    assert not bad.any()


@pytest.mark.parametrize("n,H", SHAPES)
@pytest.mark.parametrize("dh,dw,accumulate", [(False, False, False), (True, True, False), (True, False, False), (False, True, True)])
def test_backward(n, H, dh, dw, accumulate):
    rng = np.random.default_rng(n * 17 + H)
    hb, db, ub = _rows(rng, n, H), _rows(rng, n, H), _rows(rng, n, H)
    wb = B.to_bf16_bits(1 + 0.3 * rng.standard_normal(H))
    h64, d64, u64, w64 = (B.bf16_bits_to_f64(a) for a in (hb, db, ub, wb))
    r32 = (1 / np.sqrt((h64 ** 2).mean(axis=1) + EPS)).astype(np.float32)
    before = rng.standard_normal(H).astype(np.float32)
    g_w = dev_f32(before) if dw else None
    ws = L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, H)) if dw else None
    dx = _empty(n, H)
    args = (dev_bf16(db), dev_bf16(hb), dev_bf16(wb), dev_f32(r32), dx)
    L.rmsnorm_backward(*args, dh=dev_bf16(ub) if dh else None, dweight=g_w, accumulate=accumulate, ws=ws)
    want, want_w = ON.rmsnorm_backward(d64, h64, w64, r32, u64 if dh else None)
    # fp32 parts: the mean of g xh within 54 * 2^-24 of the mean of |g xh|, times rstd |xh|; the other terms 2^-21 each
    r = r32.astype(np.float64)[:, None]
    g, xh = d64 * w64, h64 * r
    slack = r * np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True) * 2.0 ** -18 + r * np.abs(g) * 2.0 ** -21
    if dh:
        slack += np.abs(u64) * 2.0 ** -23
    _close(f64_of(dx), want, U16, extra=slack * (1 + U16))
    if dw:
        # at most 5 rows a team, 64 teams, 64 blocks of a column group and 16 groups in sequence here: 256 * 2^-24
        base = before.astype(np.float64) if accumulate else 0.0
        _close(f64_of(g_w), want_w + base, 2.0 ** -22, extra=2.0 ** -16 * np.abs(d64 * xh).sum(axis=0))
        again = dev_f32(before)
        L.rmsnorm_backward(*args, dh=dev_bf16(ub) if dh else None, dweight=again, accumulate=accumulate, ws=ws)
        assert np.array_equal(again.cpu().numpy(), g_w.cpu().numpy())
    # dx in the place of dy
    inplace = args[0].clone()
    L.rmsnorm_backward(inplace, *args[1:4], inplace, dh=dev_bf16(ub) if dh else None)
    assert np.array_equal(bits_of(inplace), bits_of(dx))


def test_backward_many_rows_sum_the_weight_gradient():
    # every block takes several rows, H that ends inside a wave's columns
    n, H = 20011, 200
    rng = np.random.default_rng(5)
    hb, db = B.to_bf16_bits(rng.standard_normal((n, H))), B.to_bf16_bits(rng.standard_normal((n, H)))
    h64, d64 = B.bf16_bits_to_f64(hb), B.bf16_bits_to_f64(db)
    r32 = (1 / np.sqrt((h64 ** 2).mean(axis=1) + EPS)).astype(np.float32)
    w = np.ones(H)
    g_w, dx = torch.empty(H, device="cuda"), _empty(n, H)
    ws = L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, H))
    L.rmsnorm_backward(dev_bf16(db), dev_bf16(hb), dev_bf16(B.to_bf16_bits(w)), dev_f32(r32), dx, dweight=g_w, ws=ws)
    want, want_w = ON.rmsnorm_backward(d64, h64, w, r32)
    _close(f64_of(g_w), want_w, 2.0 ** -22, extra=2.0 ** -16 * np.abs(d64 * h64 * r32[:, None]).sum(axis=0))
    _close(f64_of(dx), want, U16, extra=2.0 ** -16)   # values of order 1


def test_gradient_against_differences():
    """<dx, d> of the forward's own y against central differences in float64 of the oracle."""
    n, H = 3, 96
    rng = np.random.default_rng(6)
    h = B.round_bf16(rng.standard_normal((n, H)))
    w, dv = B.round_bf16(1 + 0.2 * rng.standard_normal(H)), B.round_bf16(rng.standard_normal((n, H)))
    f = lambda a: float((ON.rmsnorm_forward(a, w, EPS)[0] * dv).sum())  # noqa: E731
    x, y, rstd, dx = dev_bf16(B.to_bf16_bits(h)), _empty(n, H), torch.empty(n, device="cuda"), _empty(n, H)
    wd = dev_bf16(B.to_bf16_bits(w))
    L.rmsnorm_forward(x, wd, EPS, y, rstd=rstd)
    L.rmsnorm_backward(dev_bf16(B.to_bf16_bits(dv)), x, wd, rstd, dx)
    got = f64_of(dx)
    for _ in range(5):
        d = rng.standard_normal((n, H))
        want = (f(h + 1e-6 * d) - f(h - 1e-6 * d)) / 2e-6
        # bf16 dx: each element off by 2^-8 of itself; differences to 1e-6
        assert abs((got * d).sum() - want) <= U16 * np.abs(got * d).sum() + 1e-5


def test_weight_gradient_against_differences():
    """dweight against central differences of the oracle in float64 (y is linear in the weight)."""
    n, H = 37, 200
    rng = np.random.default_rng(8)
    h = B.round_bf16(rng.standard_normal((n, H)))
    w, dv = B.round_bf16(1 + 0.2 * rng.standard_normal(H)), B.round_bf16(rng.standard_normal((n, H)))
    f = lambda a: float((ON.rmsnorm_forward(h, a, EPS)[0] * dv).sum())  # noqa: E731
    x, wd, y, rstd = dev_bf16(B.to_bf16_bits(h)), dev_bf16(B.to_bf16_bits(w)), _empty(n, H), torch.empty(n, device="cuda")
    L.rmsnorm_forward(x, wd, EPS, y, rstd=rstd)
    dx, dw = _empty(n, H), torch.empty(H, device="cuda")
    ws = torch.empty(L.rmsnorm_backward_workspace_bytes(n, H), dtype=torch.uint8, device="cuda")
    L.rmsnorm_backward(dev_bf16(B.to_bf16_bits(dv)), x, wd, rstd, dx, dweight=dw, ws=ws)
    got = f64_of(dw)
    mag = np.abs(dv * h / np.sqrt((h * h).mean(1, keepdims=True) + EPS)).sum(0)
    for _ in range(5):
        d = rng.standard_normal(H)
        want = (f(w + 1e-3 * d) - f(w - 1e-3 * d)) / 2e-3
        # rstd to 2^-19, two more roundings a term and n - 1 additions of 2^-24 each: below
        # 2^-17 of the terms; the difference is exact but for float64's ~1e-10
        assert abs((got * d).sum() - want) <= 2.0 ** -17 * (mag * np.abs(d)).sum() + 1e-8


def test_no_rows_and_zero_gradient():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    L.rmsnorm_forward(x, w, EPS, x)
    dw = torch.full((64,), 3.0, device="cuda")
    ws = L.empty_workspace(L.rmsnorm_backward_workspace_bytes(0, 64))
    L.rmsnorm_backward(x, x, w, torch.empty(0, device="cuda"), x, dweight=dw, accumulate=True, ws=ws)
    assert bool((dw == 3).all())
    L.rmsnorm_backward(x, x, w, torch.empty(0, device="cuda"), x, dweight=dw, ws=ws)
    assert bool((dw == 0).all())


def test_rows_do_not_depend_on_the_batch():
    rng = np.random.default_rng(8)
    for H in (128, 520, 4096):
        xb, wb = _rows(rng, 700, H), B.to_bf16_bits(1 + 0.3 * rng.standard_normal(H))
        x, w = dev_bf16(xb), dev_bf16(wb)
        y = _empty(700, H)
        L.rmsnorm_forward(x, w, EPS, y)
        for rows in (slice(0, 1), slice(13, 20), slice(699, 700)):
            part = x[rows].clone()
            L.rmsnorm_forward(part, w, EPS, part)
            assert np.array_equal(bits_of(part), bits_of(y[rows]))


def test_non_finite_rows():
    H = 64
    x = torch.ones(4, H, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[1, 5], x[2, :] = float("inf"), float("nan"), 3e38   # the last row's squares overflow fp32
    w, y = torch.ones(H, dtype=torch.bfloat16, device="cuda"), _empty(4, H)
    L.rmsnorm_forward(x, w, EPS, y)
    got = f64_of(y)
    assert np.isnan(got[0, 3]) and np.all(np.delete(got[0], 3) == 0)
    assert np.all(np.isnan(got[1])) and np.all(got[2] == 0) and np.all(np.abs(got[3] - 1) <= U16)
    q = torch.empty(4, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(4, 2, dtype=torch.uint8, device="cuda")
    L.rmsnorm_forward_q8(x, w, EPS, q, s)
    v = q.view(torch.float8_e4m3fn).float().cpu().numpy()
    assert np.isnan(v[0, 3]) and np.all(np.delete(v[0], 3) == 0) and np.all(np.isnan(v[1])) and np.all(v[2] == 0)
    assert np.all(v[3] != 0) and np.all(s[3].cpu().numpy() == 127 - 8)


def test_on_another_stream():
    x = torch.randn(64, 2048, device="cuda").to(torch.bfloat16)
    w, ref, y = torch.ones(2048, dtype=torch.bfloat16, device="cuda"), _empty(64, 2048), _empty(64, 2048)
    L.rmsnorm_forward(x, w, EPS, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.rmsnorm_forward(x, w, EPS, y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert np.array_equal(bits_of(y), bits_of(ref))


def _device_rows(seed, n, H):
    """_rows' kind of rows, made on the device (for batches of hundreds of megabytes)."""
    g = torch.Generator("cuda").manual_seed(seed)
    size = torch.randint(-8, 8, (n, 1), generator=g, device="cuda").float().exp2()
    wide = torch.where(torch.rand(H, generator=g, device="cuda") < 0.02, 30.0, 1.0)
    return (torch.randn(n, H, generator=g, device="cuda") * size * wide).to(torch.bfloat16)


# calls of more than 96 MB (non-temporal accesses), several rounds of every block: rows of one wave's team, of
# several waves, past 16384 columns, and element by element
LARGE = [(8193, 4096), (131075, 128), (2051, 20480), (5003, 4099)]


def _sample(n):
    return np.unique(np.concatenate(([0, 1, n // 2, n - 2, n - 1], np.random.default_rng(n).integers(0, n, 60))))


@pytest.mark.parametrize("n,H", LARGE)
def test_forward_large(n, H):
    x, r, w = _device_rows(1, n, H), _device_rows(2, n, H), dev_bf16(B.to_bf16_bits(1 + 0.3 * np.random.default_rng(H).standard_normal(H)))
    h, y, rstd = _empty(n, H), _empty(n, H), torch.full((n,), float("nan"), device="cuda")
    L.rmsnorm_forward(x, w, EPS, y, rstd=rstd, residual=r, h=h)
    assert bool((h == (x.float() + r.float()).to(torch.bfloat16)).all()) and bool(torch.isfinite(rstd).all()) and bool(torch.isfinite(y).all())
    at = torch.from_numpy(_sample(n)).to("cuda")
    v, rs = ON.rmsnorm_forward(f64_of(h[at]), f64_of(w), EPS)
    _close(f64_of(rstd[at]), rs, U32)
    _close(f64_of(y[at]), v, U16 + 2 * U32)
    # the same rows in a small batch: the same bits
    h2, y2, rstd2 = _empty(len(at), H), _empty(len(at), H), torch.empty(len(at), device="cuda")
    L.rmsnorm_forward(x[at], w, EPS, y2, rstd=rstd2, residual=r[at], h=h2)
    assert np.array_equal(bits_of(y2), bits_of(y[at])) and np.array_equal(bits_of(h2), bits_of(h[at])) and torch.equal(rstd2, rstd[at])
    if H % 32 == 0:
        q, s = torch.full((n, H), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((n, H // 32), 255, dtype=torch.uint8, device="cuda")
        L.rmsnorm_forward_q8(x, w, EPS, q, s, rstd=rstd, residual=r, h=h)
        q2, s2 = torch.empty(len(at), H, dtype=torch.uint8, device="cuda"), torch.empty(len(at), H // 32, dtype=torch.uint8, device="cuda")
        L.rmsnorm_forward_q8(x[at], w, EPS, q2, s2, residual=r[at], h=h2)
        assert torch.equal(q2, q[at]) and torch.equal(s2, s[at]) and torch.equal(rstd[at], rstd2)
        e = s[at].cpu().numpy().astype(int) - 127
        scale = np.repeat(np.exp2(e.astype(float)), 32, axis=1)
        val = q[at].view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64) * scale
        bad = ~(np.abs(val - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * scale) * (1 + U32) + 2 * U32 * np.abs(v))
        assert not bad.any()
        # no value saturates, and none could do with half the scale
        top = np.abs(v).reshape(len(at), -1, 32).max(axis=2) / np.exp2(e.astype(float))
        assert np.all(top <= 448 * (1 + 2 * U32)) and np.all((top >= 224 * (1 - 2 * U32)) | (e == -126))
        assert bool((q & 127 != 127).all()) and bool((s != 255).all())


@pytest.mark.parametrize("dh,dw", [(True, True), (False, False)])
@pytest.mark.parametrize("n,H", LARGE)
def test_backward_large(n, H, dh, dw):
    h, dy, u = _device_rows(3, n, H), _device_rows(4, n, H), _device_rows(5, n, H) if dh else None
    w = dev_bf16(B.to_bf16_bits(1 + 0.3 * np.random.default_rng(H).standard_normal(H)))
    rstd = torch.cat([1 / (p.double().square().mean(1) + EPS).sqrt() for p in h.split(1024)]).float()
    g_w, ws = None, None
    if dw:
        g_w, ws = torch.full((H,), float("nan"), device="cuda"), L.empty_workspace(L.rmsnorm_backward_workspace_bytes(n, H))
    dx = _empty(n, H)
    L.rmsnorm_backward(dy, h, w, rstd, dx, dh=u, dweight=g_w, ws=ws)
    assert bool(torch.isfinite(dx).all())
    at = torch.from_numpy(_sample(n)).to("cuda")
    d64, h64, w64, r64 = (f64_of(t) for t in (dy[at], h[at], w, rstd[at]))
    want, _ = ON.rmsnorm_backward(d64, h64, w64, r64, f64_of(u[at]) if dh else None)
    # as in test_backward: the mean of g xh, the other terms
    r = r64[:, None]
    g, xh = d64 * w64, h64 * r
    slack = r * np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True) * 2.0 ** -18 + r * np.abs(g) * 2.0 ** -21
    if dh:
        slack += np.abs(f64_of(u[at])) * 2.0 ** -23
    _close(f64_of(dx[at]), want, U16, extra=slack * (1 + U16))
    small = _empty(len(at), H)
    L.rmsnorm_backward(dy[at], h[at], w, rstd[at], small, dh=u[at] if dh else None)
    assert np.array_equal(bits_of(small), bits_of(dx[at]))
    if dw:
        term = [(p.double() * q.double() * s.double()[:, None]) for p, q, s in zip(dy.split(1024), h.split(1024), rstd.split(1024))]
        want_w, mag = sum(t.sum(0) for t in term), sum(t.abs().sum(0) for t in term)
        # additions behind one another: a team's rows, the block's teams, every 128th of its blocks, then 4 and 32 sums of
        # these; each off by 2^-24 of the magnitudes, and two products before them
        blocks = (L.rmsnorm_backward_workspace_bytes(n, H) - 256) // (4 * H)
        teams = 16 if H == 128 else 1
        steps = -(-n // (blocks * teams)) + teams + -(-blocks // 128) + 4 + 32 + 2
        _close(f64_of(g_w), f64_of(want_w), 2.0 ** -24, extra=steps * 2.0 ** -24 * f64_of(mag))
        again = torch.zeros(H, device="cuda")
        L.rmsnorm_backward(dy, h, w, rstd, dx, dh=u, dweight=again, accumulate=True, ws=ws)
        assert torch.equal(again, g_w)


@pytest.mark.parametrize("n,H", [(5, 64), (9, 33), (300, 2048), (3, 4099), (2, 20480)])
def test_outputs_in_the_place_of_inputs(n, H):
    """h in the place of x or of residual, y then in the other's; dx in the place of dh."""
    rng = np.random.default_rng(n + H)
    x, r, w = dev_bf16(_rows(rng, n, H)), dev_bf16(_rows(rng, n, H)), dev_bf16(B.to_bf16_bits(1 + 0.3 * rng.standard_normal(H)))
    h, y = _empty(n, H), _empty(n, H)
    L.rmsnorm_forward(x, w, EPS, y, residual=r, h=h)
    for place in ("x", "residual"):
        a, b, out = x.clone(), r.clone(), _empty(n, H)
        L.rmsnorm_forward(a, w, EPS, out, residual=b, h=a if place == "x" else b)
        assert np.array_equal(bits_of(out), bits_of(y)) and np.array_equal(bits_of(a if place == "x" else b), bits_of(h))
    a, b = x.clone(), r.clone()
    L.rmsnorm_forward(a, w, EPS, a, residual=b, h=b)
    assert np.array_equal(bits_of(a), bits_of(y)) and np.array_equal(bits_of(b), bits_of(h))
    if H % 32 == 0:
        q, s = torch.empty(n, H, dtype=torch.uint8, device="cuda"), torch.empty(n, H // 32, dtype=torch.uint8, device="cuda")
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        L.rmsnorm_forward_q8(x, w, EPS, q, s, residual=r, h=h)
        a = x.clone()
        L.rmsnorm_forward_q8(a, w, EPS, q2, s2, residual=r, h=a)
        assert torch.equal(q, q2) and torch.equal(s, s2) and np.array_equal(bits_of(a), bits_of(h))
    rstd, dx, u = torch.rand(n, device="cuda"), _empty(n, H), dev_bf16(_rows(rng, n, H))
    L.rmsnorm_backward(y, h, w, rstd, dx, dh=u)
    L.rmsnorm_backward(y, h, w, rstd, u, dh=u)
    assert np.array_equal(bits_of(u), bits_of(dx))
