"""w4_quantize, w4_linear and lora_forward_w4 against oracle.w4 and oracle.lora.

Tolerance of y, from the arithmetic: its rounding to bf16 is off by at most 2^-8
of the value; the fp32 sum of d_in products runs over at most d_in/8 terms in
sequence in a wave (all 32 of one matrix instruction counted), 16 wave sums and 64
rank terms behind them, each step off by 2^-24 of the sum of magnitudes; u adds
d_in/64 + 6 steps of its own to the delta's part of that sum.
"""
import numpy as np
import pytest

import oracle.lora as OL
import oracle.norm as ON
import oracle.w4 as OQ
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import bits_of, dev_bf16, dev_i32, f64_of  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def _weights(rng, d_out, d_in):
    """Random codes (every one of the 16) and scales over some binades."""
    return rng.integers(0, 256, (d_out, d_in // 2), dtype=np.uint8), rng.integers(110, 130, (d_out, d_in // 32)).astype(np.uint8)


def _x(rng, n, d_in, x8):
    """(device x, device scales or None, float64 values)."""
    v = rng.standard_normal((n, d_in)) * np.exp2(rng.integers(-6, 6, (n, 1)))
    v[:, rng.random(d_in) < 0.02] *= 30
    if not x8:
        b = B.to_bf16_bits(v)
        return dev_bf16(b), None, B.bf16_bits_to_f64(b)
    codes = rng.integers(0, 256, (n, d_in), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0x38
    s = rng.integers(115, 135, (n, d_in // 32)).astype(np.uint8)
    val = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy() * np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    return _dev(codes), _dev(s), val


def _check(y, want, mag, d_in):
    got = f64_of(y)
    tol = 2.0 ** -8 * np.abs(want) + (d_in / 8 + 80) * 2.0 ** -24 * (1 + 2.0 ** -8) * mag
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


SIZES = [(1, 64, 64), (1, 4096, 64), (2, 192, 128), (7, 320, 192), (15, 1024, 320), (16, 1088, 64), (17, 512, 128),
         (31, 2112, 64), (33, 640, 192), (64, 1024, 256), (65, 256, 64), (100, 1600, 128), (129, 192, 320), (255, 576, 64), (256, 1024, 192),
         (1, 12288, 128), (5, 16448, 64),
         # every number of pairs of 256 columns that a wave holds, a token past a tile
         (3, 4352, 64), (20, 4416, 128), (2, 8192, 64), (33, 8192, 64), (5, 8256, 64), (17, 10240, 64), (4, 10304, 128), (40, 12288, 64),
         (40, 13056, 64), (256, 12352, 64),
         # more row tiles than CUs, of few columns: two teams of waves a block
         (1, 64, 4224), (16, 320, 4160), (3, 2048, 4288), (5, 1984, 8256),
         # four teams, and two with two token tiles
         (3, 1024, 8256), (40, 320, 4160), (90, 1984, 4160)]


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_linear(n, d_in, d_out, x8):
    rng = np.random.default_rng(n * 31 + d_in + d_out)
    codes, scales = _weights(rng, d_out, d_in)
    x, xs, xv = _x(rng, n, d_in, x8)
    W = OQ.values(codes, scales)
    y = torch.full((n + 1, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, _dev(codes), _dev(scales), y[:n], x_scales=xs)
    _check(y[:n], xv @ W.T, np.abs(xv) @ np.abs(W).T, d_in)
    assert bool(torch.isnan(y[n]).all())      # the row behind the last token


def _adapters(rng, ranks, d_in, d_out):
    sizes = np.array(ranks) * (d_in + d_out)
    a_off = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int64)
    b_off = a_off + np.array(ranks) * d_in
    pack = B.to_bf16_bits(rng.standard_normal(int(sizes.sum())) * 0.1)
    v = B.bf16_bits_to_f64(pack)
    A = [v[a:a + r * d_in].reshape(r, d_in) for a, r in zip(a_off, ranks)]
    Bm = [v[b:b + r * d_out].reshape(d_out, r) for b, r in zip(b_off, ranks)]
    scale = (32.0 / np.maximum(1, np.array(ranks))).astype(np.float32)
    return pack, a_off, b_off, A, Bm, scale


def _magnitude(xv, W, A, Bm, s, ids):
    """Sum of magnitudes behind each y (the delta's with its inner sums' magnitudes)."""
    mag = np.abs(xv) @ np.abs(W).T
    for t, a in enumerate(ids):
        if 0 <= a < len(A) and A[a].size:
            # u's own error (d_in/64 + 6 steps) is smaller than the d_in/8 + 80 allowed below
            mag[t] += s[a] * (np.abs(Bm[a]) @ (np.abs(A[a]) @ np.abs(xv[t])))
    return mag


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_lora_forward(n, d_in, d_out, x8):
    rng = np.random.default_rng(n * 37 + d_in + d_out)
    codes, scales = _weights(rng, d_out, d_in)
    scales = np.minimum(scales, 122).astype(np.uint8)
    x, xs, xv = _x(rng, n, d_in, x8)
    ranks = [8, 16, 24, 32, 40, 48, 56, 64, 8]
    pack, a_off, b_off, A, Bm, s = _adapters(rng, ranks, d_in, d_out)
    desc = L.make_desc(a_off, b_off, ranks, s)
    ids = rng.integers(-1, len(ranks) + 1, n).astype(np.int32)
    ids[0] = len(ranks) - 1 if n == 1 else -1
    shape = L.make_shape(n, d_in, d_out, len(pack), len(pack), len(ranks), 64, L.IDS_INTERLEAVED)
    ws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape))
    y = torch.full((n, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    p = dev_bf16(pack)
    args = (_dev(codes), _dev(scales), p, p, desc, dev_i32(ids))
    L.lora_forward_w4(shape, x, *args, y, ws, x_scales=xs)
    W = OQ.values(codes, scales)
    want, _ = OL.lora_forward(xv, W, A, Bm, s.astype(np.float64), ids)
    _check(y, want, _magnitude(xv, W, A, Bm, s, ids), d_in)
    flags = L.lora_device_status(ws)
    assert flags == (L.FLAG_ID_RANGE if ((ids < 0) | (ids >= len(ranks))).any() else 0)
    y2 = torch.empty_like(y)
    L.lora_forward_w4(shape, x, *args, y2, ws, x_scales=xs)
    assert np.array_equal(bits_of(y), bits_of(y2))
    # a token without an adapter: the base product's bits
    base = torch.empty_like(y)
    L.w4_linear(x, args[0], args[1], base, x_scales=xs)
    out = (ids < 0) | (ids >= len(ranks))
    assert np.array_equal(bits_of(y)[out], bits_of(base)[out])


@pytest.mark.parametrize("n,d_in,d_out", [(1, 12416, 4224), (6, 14336, 8256), (18, 12352, 4224), (16, 20480, 64)])
@pytest.mark.parametrize("x8", [False, True])
def test_long_rows(n, d_in, d_out, x8):
    """Rows whose x does not fit the registers, several tiles a block; scales of x that
    begin at an odd multiple of two bytes; sampled rows."""
    rng = np.random.default_rng(n + d_in + d_out)
    codes, scales = _weights(rng, d_out, d_in)
    x, xs, xv = _x(rng, n + 1, d_in, x8)
    x, xs, xv = x[1:], xs[1:] if x8 else None, xv[1:]
    ranks = [16, 64, 8]
    pack, a_off, b_off, A, Bm, s = _adapters(rng, ranks, d_in, d_out)
    ids = rng.integers(0, 3, n).astype(np.int32)
    rows = np.unique(np.concatenate((rng.integers(0, d_out, 100), [0, d_out - 1])))
    W = OQ.values(codes[rows], scales[rows])
    y = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, _dev(codes), _dev(scales), y, x_scales=xs)
    _check(y[:, _dev(rows)], xv @ W.T, np.abs(xv) @ np.abs(W).T, d_in)
    shape = L.make_shape(n, d_in, d_out, len(pack), len(pack), 3, 64, L.IDS_INTERLEAVED)
    ws, desc = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape)), L.make_desc(a_off, b_off, ranks, s)
    dp = dev_bf16(pack)
    L.lora_forward_w4(shape, x, _dev(codes), _dev(scales), dp, dp, desc, _dev(ids), y, ws, x_scales=xs)
    Br = [b[rows] for b in Bm]
    want = xv @ W.T + np.stack([float(s[a]) * (Br[a] @ (A[a] @ xv[t])) for t, a in enumerate(ids)])
    _check(y[:, _dev(rows)], want, _magnitude(xv, W, A, Br, s, ids), d_in)
    assert L.lora_device_status(ws) == 0


@pytest.mark.parametrize("d_in,d_out", [(64, 4224), (1024, 8256), (2048, 4288), (4032, 50048), (4096, 64), (8192, 128), (8192, 24640),
                                        (9216, 64), (12288, 64), (12352, 4224)])
@pytest.mark.parametrize("x8", [False, True])
def test_batch_invariance(d_in, d_out, x8):
    """A token's bits are the same alone and in every larger batch, with adapters and without."""
    rng = np.random.default_rng(d_in + d_out)
    dev = torch.Generator("cuda").manual_seed(d_in)
    codes = torch.randint(0, 256, (d_out, d_in // 2), dtype=torch.uint8, device="cuda", generator=dev)
    scales = torch.randint(115, 125, (d_out, d_in // 32), dtype=torch.uint8, device="cuda", generator=dev)
    n = 256
    x, xs, _ = _x(rng, n, d_in, x8)
    ranks = [16, 64, 8, 32]
    pack, a_off, b_off, _, _, s = _adapters(rng, ranks, d_in, d_out)
    ids, desc, p = dev_i32(rng.integers(0, 4, n).astype(np.int32)), L.make_desc(a_off, b_off, ranks, s), dev_bf16(pack)

    def run(n, adapters):
        y = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
        if not adapters:
            L.w4_linear(x[:n], codes, scales, y, x_scales=xs[:n] if x8 else None)
            return bits_of(y)
        shape = L.make_shape(n, d_in, d_out, len(pack), len(pack), 4, 64, L.IDS_INTERLEAVED)
        ws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape))
        L.lora_forward_w4(shape, x[:n], codes, scales, p, p, desc, ids[:n], y, ws, x_scales=xs[:n] if x8 else None)
        return bits_of(y)

    for adapters in (False, True):
        whole = run(n, adapters)
        for k in (1, 4, 5, 16, 17, 80, 81):
            assert np.array_equal(run(k, adapters), whole[:k]), (adapters, k)


def test_bad_descriptors_and_order():
    rng = np.random.default_rng(3)
    d_in, d_out, ranks = 128, 64, [16, 16, 16, 16, 16]
    codes, scales = _weights(rng, d_out, d_in)
    pack, a_off, b_off, A, Bm, s = _adapters(rng, ranks, d_in, d_out)
    n = 6
    x, _, xv = _x(rng, n, d_in, False)
    W = OQ.values(codes, scales)
    p = dev_bf16(pack)
    ids = np.array([0, 1, 2, 3, 4, 0], np.int32)
    base = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, _dev(codes), _dev(scales), base)

    def call(a=a_off, b=b_off, r=ranks, order=L.IDS_INTERLEAVED, who=ids, elems=len(pack), max_rank=16):
        shape = L.make_shape(n, d_in, d_out, elems, elems, 5, max_rank, order)
        ws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape))
        y = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
        L.lora_forward_w4(shape, x, _dev(codes), _dev(scales), p, p, L.make_desc(a, b, r, s), dev_i32(who), y, ws)
        return y, L.lora_device_status(ws)

    good, flags = call()
    assert flags == 0
    for what in ("past the pack", "negative", "unaligned", "rank", "rank above max_rank"):
        a, b, r = a_off.copy(), b_off.copy(), list(ranks)
        if what == "past the pack":
            b[2] = len(pack) - 8
        elif what == "negative":
            a[2] = -8
        elif what == "unaligned":
            a[2] += 4
        elif what == "rank":
            r[2] = 12
        else:
            r[2] = 24
        y, flags = call(a, b, r)
        assert flags == L.FLAG_BAD_DESC, what
        assert np.array_equal(bits_of(y)[2], bits_of(base)[2]), what
        keep = [0, 1, 3, 4, 5]
        assert np.array_equal(bits_of(y)[keep], bits_of(good)[keep]), what
    y, flags = call(r=[16, 16, 0, 16, 16])      # rank 0: an unused slot, no flag
    assert flags == 0 and np.array_equal(bits_of(y)[2], bits_of(base)[2])
    y, flags = call(order=L.IDS_SORTED)
    assert flags == L.FLAG_UNSORTED and np.array_equal(bits_of(y), bits_of(good))
    y, flags = call(order=L.IDS_SORTED, who=np.sort(ids))
    assert flags == 0


@pytest.mark.parametrize("rows,cols", [(64, 64), (128, 1600), (320, 4096)])
def test_quantize(rows, cols):
    rng = np.random.default_rng(rows)
    W = B.round_bf16(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1))))
    W[0, :32] = 0
    W[1, :32] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.tile([1, -1], 16)   # ties
    codes = torch.full((rows, cols // 2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 255, dtype=torch.uint8, device="cuda")
    L.w4_quantize(dev_bf16(B.to_bf16_bits(W)), codes, scales)
    want_c, want_s = OQ.quantize(W)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(OQ.values(codes.cpu().numpy(), want_s), OQ.values(want_c, want_s))


def test_largest_and_smallest_scales():
    """Scale bytes 1 and 250: exact products far from one."""
    d_in = 64
    codes = np.full((64, d_in // 2), 0x22, np.uint8)           # ones
    x = torch.ones(1, d_in, dtype=torch.bfloat16, device="cuda")
    for byte in (10, 127, 240):
        scales = np.full((64, 2), byte, np.uint8)
        y = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
        L.w4_linear(x, _dev(codes), _dev(scales), y)
        assert np.all(f64_of(y) == 64 * 2.0 ** (byte - 127))
    for byte in (10, 127, 240):
        xs = np.full((1, 2), byte, np.uint8)
        xq = np.full((1, d_in), 0x38, np.uint8)                # ones in e4m3
        y = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
        L.w4_linear(_dev(xq), _dev(codes), _dev(np.full((64, 2), 127, np.uint8)), y, x_scales=_dev(xs))
        assert np.all(f64_of(y) == 64 * 2.0 ** (byte - 127))


def test_non_finite_x_and_scales():
    """A non-finite x reaches its own token alone; the NaN scale its own row."""
    rng = np.random.default_rng(9)
    codes, scales = _weights(rng, 64, 256)
    codes[:, 50] = 0x22                                        # ones at columns 100 and 101
    x = torch.ones(3, 256, dtype=torch.bfloat16, device="cuda")
    x[1, 100] = float("inf")
    y = torch.empty(3, 64, dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, _dev(codes), _dev(scales), y)
    got = f64_of(y)
    assert np.all(np.isinf(got[1])) and np.all(np.isfinite(got[[0, 2]]))
    scales[5, 1] = 255
    L.w4_linear(x, _dev(codes), _dev(scales), y)
    got = f64_of(y)
    assert np.all(np.isnan(got[:, 5])) and np.all(np.isfinite(np.delete(got[[0, 2]], 5, axis=1)))


def test_host_operands_are_refused():
    """Every operand of the adapter call left on the host, or too short, raises before any launch."""
    d_in, d_out, n = 64, 64, 2
    dev = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    good = {"x": dev(n, d_in, dtype=bf), "codes": dev(d_out, 32), "scales": dev(d_out, 2), "A_pack": dev(4096, dtype=bf), "B_pack": dev(4096, dtype=bf),
            "desc": dev(48), "ids": dev(n, dtype=torch.int32), "y": dev(n, d_out, dtype=bf)}
    shape = L.make_shape(n, d_in, d_out, 4096, 4096, 2, 16)
    good["ws"] = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape))
    L.lora_forward_w4(shape, *good.values())
    for name in good:
        with pytest.raises(L.LoraError, match=name):
            L.lora_forward_w4(shape, *{**good, name: good[name].cpu()}.values())
    for name in ("A_pack", "B_pack", "desc"):
        with pytest.raises(L.LoraError, match=name):
            L.lora_forward_w4(shape, *{**good, name: good[name][:-1]}.values())
    with pytest.raises(L.LoraError):
        L.lora_forward_w4(shape, *{**good, "ws": good["ws"][:32]}.values())
    assert L.lora_device_status(good["ws"]) == 0


def test_eight_bit_norm_feeds_the_product():
    """rmsnorm_forward_q8's own output as x, through lora_forward_w4."""
    rng = np.random.default_rng(10)
    n, H, d_out, ranks = 9, 512, 256, [16, 8]
    hb, wb = B.to_bf16_bits(rng.standard_normal((n, H))), B.to_bf16_bits(1 + 0.1 * rng.standard_normal(H))
    q = torch.empty(n, H, dtype=torch.float8_e4m3fn, device="cuda")
    qs = torch.empty(n, H // 32, dtype=torch.float8_e8m0fnu, device="cuda")
    L.rmsnorm_forward_q8(dev_bf16(hb), dev_bf16(wb), 1e-6, q, qs)
    val = q.float().cpu().numpy().astype(np.float64) * np.repeat(qs.float().cpu().numpy().astype(np.float64), 32, axis=1)
    v, _ = ON.rmsnorm_forward(B.bf16_bits_to_f64(hb), B.bf16_bits_to_f64(wb), 1e-6)
    assert np.linalg.norm(val - v) < 2.0 ** -4 * np.linalg.norm(v)
    codes, scales = OQ.quantize(B.round_bf16(0.05 * rng.standard_normal((d_out, H))))
    pack, a_off, b_off, A, Bm, s = _adapters(rng, ranks, H, d_out)
    ids = rng.integers(0, 2, n).astype(np.int32)
    shape = L.make_shape(n, H, d_out, len(pack), len(pack), 2, 16, L.IDS_INTERLEAVED)
    ws, p = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape)), dev_bf16(pack)
    y = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
    L.lora_forward_w4(shape, q, _dev(codes), _dev(scales), p, p, L.make_desc(a_off, b_off, ranks, s), dev_i32(ids), y, ws, x_scales=qs)
    W = OQ.values(codes, scales)
    want, _ = OL.lora_forward(val, W, A, Bm, s.astype(np.float64), ids)
    _check(y, want, _magnitude(val, W, A, Bm, s, ids), H)
    assert L.lora_device_status(ws) == 0


@pytest.mark.parametrize("n,d_in,d_out", [(1, 4096, 49216), (16, 4096, 49216), (3, 8192, 24640), (17, 4096, 49216), (2, 1024, 196672), (9, 2048, 98368)])
def test_codes_larger_than_the_caches(n, d_in, d_out):
    """Codes of a little over 96 MB (read once, non-temporally, by one token tile); sampled rows."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(0, 256, (d_out, d_in // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(110, 130, (d_out, d_in // 32), dtype=torch.uint8, device="cuda", generator=gen)
    assert codes.numel() > 96 << 20
    rng = np.random.default_rng(n)
    rows = np.unique(np.concatenate([[0, 15, 16, d_out - 1], rng.integers(0, d_out, 40)]))
    for x8 in (False, True):
        x, xs, xv = _x(rng, n, d_in, x8)
        y = torch.full((n, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
        L.w4_linear(x, codes, scales, y, x_scales=xs)
        at = torch.from_numpy(rows).to("cuda")
        W = OQ.values(codes[at].cpu().numpy(), scales[at].cpu().numpy())
        _check(y[:, at].contiguous(), xv @ W.T, np.abs(xv) @ np.abs(W).T, d_in)
        assert bool(torch.isfinite(y).all())


def test_codes_past_four_gigabytes():
    """Row offsets beyond 32 bits: 2^17 rows of 2^16 + 64 columns; sampled outputs."""
    d_in, d_out = (1 << 16) + 64, 1 << 17
    codes = torch.zeros(d_out, d_in // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((d_out, d_in // 32), 127, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    rows = np.array([0, 1, 65535, 65536, d_out - 64, d_out - 1])
    part = rng.integers(0, 256, (len(rows), d_in // 2), dtype=np.uint8)
    codes[torch.from_numpy(rows).to("cuda")] = _dev(part)
    x, _, xv = _x(rng, 2, d_in, False)
    y = torch.empty(2, d_out, dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, codes, scales, y)
    W = OQ.values(part, np.full((len(rows), d_in // 32), 127, np.uint8))
    _check(y[:, torch.from_numpy(rows).to("cuda")].contiguous(), xv @ W.T, np.abs(xv) @ np.abs(W).T, d_in)
    rest = torch.ones(d_out, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(rows).to("cuda")] = False
    assert bool((y[:, rest] == 0).all())


@pytest.mark.parametrize("which", ["A", "B"])
@pytest.mark.parametrize("offset", [(1 << 63) - 8, (1 << 63) - 16 * 128 - 8, 1 << 62])
def test_offsets_near_the_largest_integer(which, offset):
    """A descriptor whose end lies past 64 bits: flagged, its token gets the base output, the others their own."""
    rng = np.random.default_rng(12)
    d_in, d_out, ranks, n = 128, 64, [16, 8, 16], 3
    codes, scales = _weights(rng, d_out, d_in)
    pack, a_off, b_off, _, _, s = _adapters(rng, ranks, d_in, d_out)
    x, _, _ = _x(rng, n, d_in, False)
    p, ids = dev_bf16(pack), dev_i32(np.arange(n))
    shape = L.make_shape(n, d_in, d_out, len(pack), len(pack), 3, 16, L.IDS_INTERLEAVED)
    ws = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape))
    good, y, base = (torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    L.w4_linear(x, _dev(codes), _dev(scales), base)
    L.lora_forward_w4(shape, x, _dev(codes), _dev(scales), p, p, L.make_desc(a_off, b_off, ranks, s), ids, good, ws)
    assert L.lora_device_status(ws) == 0
    (a_off if which == "A" else b_off)[1] = offset
    L.lora_forward_w4(shape, x, _dev(codes), _dev(scales), p, p, L.make_desc(a_off, b_off, ranks, s), ids, y, ws)
    assert L.lora_device_status(ws) == L.FLAG_BAD_DESC
    assert np.array_equal(bits_of(y)[[0, 2]], bits_of(good)[[0, 2]]) and np.array_equal(bits_of(y)[1], bits_of(base)[1])


# every size class of x in registers with several row tiles a block: one pair of columns a wave (two token
# tiles and one), two, five and six
@pytest.mark.parametrize("n,d_in,d_out", [(256, 4096, 4224), (33, 4032, 8256), (5, 4352, 8256), (20, 8192, 4224), (33, 8256, 4224),
                                          (40, 10240, 4160), (256, 9216, 1088), (1, 12288, 8256), (64, 12288, 4096)])
@pytest.mark.parametrize("x8", [False, True])
def test_several_tiles_a_block(n, d_in, d_out, x8):
    """Rings that stay full from tile to tile, the join's buffers in turn, deltas of several
    tokens a wave, tokens without an adapter between them; sampled rows of every block's tiles."""
    rng = np.random.default_rng(n + d_in + d_out)
    codes, scales = _weights(rng, d_out, d_in)
    scales = np.minimum(scales, 122).astype(np.uint8)
    x, xs, xv = _x(rng, n, d_in, x8)
    ranks = [16, 64, 8, 40]
    pack, a_off, b_off, A, Bm, s = _adapters(rng, ranks, d_in, d_out)
    ids = rng.integers(-1, 4, n).astype(np.int32)
    ids[0] = 1
    rows = np.unique(np.concatenate((rng.integers(0, d_out, 150), [0, d_out - 1], np.arange(7, d_out, 1031))))
    W = OQ.values(codes[rows], scales[rows])
    dc, ds, at = _dev(codes), _dev(scales), _dev(rows)
    want, mag = xv @ W.T, np.abs(xv) @ np.abs(W).T
    y = torch.full((n, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.w4_linear(x, dc, ds, y, x_scales=xs)
    _check(y[:, at], want, mag, d_in)
    assert bool(torch.isfinite(y).all())
    shape = L.make_shape(n, d_in, d_out, len(pack), len(pack), 4, 64, L.IDS_INTERLEAVED)
    ws, desc, p = L.empty_workspace(L.lora_forward_w4_workspace_bytes(shape)), L.make_desc(a_off, b_off, ranks, s), dev_bf16(pack)
    z = torch.full((n, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.lora_forward_w4(shape, x, dc, ds, p, p, desc, _dev(ids), z, ws, x_scales=xs)
    Br = [b[rows] for b in Bm]
    want = want + np.stack([float(s[a]) * (Br[a] @ (A[a] @ xv[t])) if a >= 0 else np.zeros(len(rows)) for t, a in enumerate(ids)])
    _check(z[:, at], want, _magnitude(xv, W, A, Br, s, ids), d_in)
    assert bool(torch.isfinite(z).all()) and np.array_equal(bits_of(z)[ids < 0], bits_of(y)[ids < 0])
    assert L.lora_device_status(ws) == (L.FLAG_ID_RANGE if (ids < 0).any() else 0)


@pytest.mark.parametrize("d_in,d_out", [(9216, 4224), (12288, 4160)])
@pytest.mark.parametrize("x8", [False, True])
def test_batch_invariance_over_several_tiles(d_in, d_out, x8):
    test_batch_invariance(d_in, d_out, x8)


def test_quantize_non_finite_weights():
    """NaN becomes 0, +-Inf the largest code of the finite weights' scale; blocks without a finite weight too."""
    rng = np.random.default_rng(13)
    W = B.round_bf16(rng.standard_normal((64, 128)))
    clean = W.copy()
    W[0, [3, 40, 41]], clean[0, [3, 40, 41]] = [np.nan, np.inf, -np.inf], 0
    W[1, 32:64], clean[1, 32:64] = np.nan, 0
    W[2, 0:32], clean[2, 0:32] = np.inf, 0
    W[3, 64:96], clean[3, 64:96] = -np.inf, 0
    with np.errstate(invalid="ignore"):
        bits = B.to_bf16_bits(W)
    codes, scales = torch.empty(64, 64, dtype=torch.uint8, device="cuda"), torch.empty(64, 4, dtype=torch.uint8, device="cuda")
    L.w4_quantize(dev_bf16(bits), codes, scales)
    want_c, want_s = OQ.quantize(clean)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    want = OQ.values(want_c, want_s)
    top = 6 * np.repeat(np.exp2(want_s.astype(float) - 127), 32, axis=1)
    want = np.where(np.isinf(W), np.sign(W) * top, want)
    assert np.array_equal(OQ.values(codes.cpu().numpy(), want_s), want)


def test_every_scale_byte():
    """Weights of scale bytes 0 to 252 are exact bf16, below the normal numbers too; 8-bit x from byte 3 to 246.  Under
    byte 3 x is rounded to a multiple of 2^-133; 255 is NaN.  One row of weights a byte, one code a column; the
    other operand brings the product back to the middle of fp32's range."""
    mag = np.array([0.5, 1, 1.5, 2, 3, 4, 6])
    codes = np.zeros((256, 32), np.uint8)       # 64 columns: 7 codes and zeros
    for c in range(1, 8):
        codes[:, c // 2] |= c << 4 * (c % 2)
    for bytes_, k in ((range(0, 120), 100), (range(120, 253), -90)):
        scales = np.full((256, 2), 127, np.uint8)
        scales[list(bytes_), 0] = list(bytes_)
        x = np.zeros((7, 64))
        x[np.arange(7), np.arange(1, 8)] = 2.0 ** k
        y = torch.empty(7, 256, dtype=torch.bfloat16, device="cuda")
        L.w4_linear(dev_bf16(B.to_bf16_bits(x)), _dev(codes), _dev(scales), y)
        got = f64_of(y)
        for b in bytes_:
            assert np.array_equal(got[:, b], mag * 2.0 ** (b - 127 + k)), b
    every = np.concatenate((np.arange(0, 127), np.arange(128, 255))).astype(np.uint8)    # e4m3 without its NaNs
    val = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    eye = np.zeros((256, 128), np.uint8)        # row i takes column i: 256 columns, code 1.0
    eye[np.arange(256), np.arange(256) // 2] = np.where(np.arange(256) % 2, 0x20, 0x02)
    q = np.full((1, 256), 0x00, np.uint8)
    q[0, :254] = every
    for b in (0, 1, 2, 3, 4, 9, 10, 60, 126, 127, 190, 240, 245, 246):
        k = 100 if b < 120 else -100
        y = torch.empty(1, 256, dtype=torch.bfloat16, device="cuda")
        L.w4_linear(_dev(q), _dev(eye), _dev(np.full((256, 8), 127 + k, np.uint8)), y, x_scales=_dev(np.full((1, 8), b, np.uint8)))
        want, got = val * 2.0 ** (b - 127), f64_of(y)[0, :254] / 2.0 ** k
        if b >= 3:
            assert np.array_equal(got, want), b
        else:
            assert np.all(np.abs(got - want) <= 2.0 ** -134), b
    L.w4_linear(_dev(q), _dev(eye), _dev(np.full((256, 8), 127, np.uint8)), y, x_scales=_dev(np.full((1, 8), 255, np.uint8)))
    assert bool(torch.isnan(y).all())


def test_values_beyond_bf16():
    """A code times its scale of 2^128 or more is infinite: y of that row (or token) is not finite, the others' are."""
    for d_in in (64, 256, 12352):
        codes, scales = np.full((64, d_in // 2), 0x22, np.uint8), np.full((64, d_in // 32), 127, np.uint8)
        codes[[3, 5], 0], scales[[3, 5], 0], codes[9, 0], scales[9, 0] = 0x26, (253, 254), 0x25, 253       # 4.0; 3.0
        x = torch.ones(2, d_in, dtype=torch.bfloat16, device="cuda") * 2.0 ** -20
        y = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
        L.w4_linear(x, _dev(codes), _dev(scales), y)
        finite = np.isfinite(f64_of(y))
        assert not finite[:, [3, 5]].any() and np.delete(finite, [3, 5], axis=1).all()
        q, qs = np.full((2, d_in), 0x38, np.uint8), np.full((2, d_in // 32), 127, np.uint8)
        q[1, 0], qs[1, 0] = 0x7E, 247                                                                      # 448 2^120
        L.w4_linear(_dev(q), _dev(np.full((64, d_in // 2), 0x22, np.uint8)), _dev(np.full((64, d_in // 32), 107, np.uint8)), y, x_scales=_dev(qs))
        assert not np.isfinite(f64_of(y)[1]).any() and np.isfinite(f64_of(y)[0]).all()
