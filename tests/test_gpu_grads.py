"""grad_norm, grad_clip and adam_step_clipped against oracle.clip.

Tolerances, from the arithmetic: the sums are 64-bit, so a norm is off by its
rounding to fp32, 2^-24; the factor c adds 2^-24 and its product with g another,
2^-22 with room.  AdamW's m and v are sums of two products with fp32 constants, g
scaled before (and squared): at most 8 roundings, 2^-21 of the two terms'
magnitudes.  p has three roundings of its own (2^-22), the error of m carried
through the quotient, and that of the denominator and the quotient, within 2^-20
of the step.
"""
import numpy as np
import pytest

import oracle.clip as OC
import workloads.bf16 as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpu_util import bits_of, dev_bf16, dev_f32, f64_of  # noqa: E402
import rl_lora_linear_amd.lib as L  # noqa: E402

LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8


def _tensors(kind):
    """(tensors, n_groups, n_elems)"""
    if kind == "one element":
        return [(0, 1, 0)], 1, 1
    if kind == "one tensor":
        return [(0, 100003, 0)], 1, 100003
    if kind == "empty groups":      # groups 0, 2 and 4 have no tensor, group 3 an empty one
        return [(8, 40, 1), (64, 0, 3)], 5, 80
    if kind == "chunk borders":
        out, at = [], 0
        for i, c in enumerate((8191, 8192, 8193, 16384, 1, 4, 5)):
            out.append((at, c, i % 2))
            at += c + 4 - c % 4 + 4
        return out, 2, at
    if kind == "unaligned":         # offsets at every residue of 4, layers listed before adapters
        out, at = [], 3
        for layer in range(6):
            for a in range(4):
                c = 701 * (a + 1) + 13 * layer
                out.append((at, c, a))
                at += c + layer % 3
        return out, 4, at + 5
    rng = np.random.default_rng(1)  # many: 3000 tensors over 50 groups
    out, at = [], 0
    for i in range(3000):
        c = int(rng.integers(0, 2000))
        out.append((at, c, int(rng.integers(0, 50))))
        at += c + int(rng.integers(0, 3)) * 4
    return out, 50, at + 1


KINDS = ["one element", "one tensor", "empty groups", "chunk borders", "unaligned", "many"]


def _inside(tensors, n):
    m = np.zeros(n, bool)
    for o, c, _ in tensors:
        m[o:o + c] = True
    return m


def _close(got, want, rel, extra=0.0):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= rel * np.abs(want) + extra)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def _setup(kind, seed=0):
    tensors, G, n = _tensors(kind)
    rng = np.random.default_rng(seed)
    g = (rng.standard_normal(n) * np.exp2(rng.integers(-20, 4, n))).astype(np.float32)
    shape, table = L.make_grad_table(tensors, G, n)
    return tensors, G, n, rng, g, shape, table, L.empty_workspace(L.grad_workspace_bytes(shape))


@pytest.mark.parametrize("kind", KINDS)
def test_norm_and_clip(kind):
    tensors, G, n, rng, g, shape, table, ws = _setup(kind)
    dg, norms = dev_f32(g), torch.full((G,), -1.0, device="cuda")
    L.grad_norm(shape, table, dg, norms, ws)
    want = OC.norms(tensors, G, g)
    _close(f64_of(norms), want, 2.0 ** -23)
    live = want[want > 0]
    for max_norm in (float(live.min()) * 0.5, float(np.median(live)), float("inf"), 0.0):
        out, norms2 = torch.full((n,), 7.0, device="cuda"), torch.empty(G, device="cuda")
        L.grad_clip(shape, table, dg, max_norm, out, norms2, ws)
        res, _ = OC.clip(tensors, G, g, max_norm, out=np.full(n, 7.0))
        got, inside = f64_of(out), _inside(tensors, n)
        assert np.array_equal(got[~inside], np.full((~inside).sum(), 7.0))
        _close(got[inside], res[inside], 2.0 ** -22, extra=2.0 ** -149)
        assert np.array_equal(norms2.cpu().numpy(), norms.cpu().numpy())
        # in place: the same bits
        same = dg.clone()
        L.grad_clip(shape, table, same, max_norm, same, None, ws)
        assert np.array_equal(same.cpu().numpy()[inside], out.cpu().numpy()[inside])
        if max_norm == float("inf"):
            assert np.array_equal(same.cpu().numpy(), g)
    assert np.array_equal(dg.cpu().numpy(), g) and L.lora_device_status(ws) == 0


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
@pytest.mark.parametrize("wd", [0.0, 0.1])
@pytest.mark.parametrize("kind", KINDS)
def test_adam(kind, wd, max_norm):
    tensors, G, n, rng, g, shape, table, ws = _setup(kind)
    p, m = rng.standard_normal(n).astype(np.float32), (rng.standard_normal(n) * 0.1).astype(np.float32)
    v = (rng.random(n) * 0.01 + 1e-4).astype(np.float32)
    steps = rng.integers(0, 50, G)
    dp, dm, dv, st = dev_f32(p), dev_f32(m), dev_f32(v), torch.from_numpy(steps).to("cuda")
    pb, norms = dev_bf16(np.zeros(n, np.uint16)), torch.empty(G, device="cuda")
    want = (p, m, v, steps)
    inside = _inside(tensors, n)
    for it in range(2):      # the second call from the first's state: the counters go on
        before = [f64_of(a) for a in (dp, dm, dv)]
        L.adam_step_clipped(shape, table, st, dp, dev_f32(g), dm, dv, max_norm, LR, B1, B2, EPS, wd, p_bf16=pb, norms=norms, ws=ws)
        want = OC.adam_clipped(tensors, G, steps + it, *before[:1], g, *before[1:], max_norm, LR, B1, B2, EPS, wd)
        _close(f64_of(norms), want[4], 2.0 ** -23)
        cg, _ = OC.clip(tensors, G, g, max_norm)
        gp, gm, gv = (f64_of(a) for a in (dp, dm, dv))
        slack = 2.0 ** -21 * (np.abs(B1 * before[1]) + np.abs((1 - B1) * cg))
        _close(gm, want[1], 0, extra=slack)
        _close(gv, want[2], 2.0 ** -21)
        t = np.zeros(n)
        for o, c, a in tensors:
            t[o:o + c] = steps[a] + it + 1
        t[~inside] = 1
        per_m = LR / (1 - B1 ** t) / (np.sqrt(want[2] / (1 - B2 ** t)) + EPS)
        _close(gp, want[0], 0, extra=2.0 ** -22 * np.abs(before[0]) + per_m * (slack + 2.0 ** -20 * np.abs(want[1])))
        assert np.array_equal(st.cpu().numpy(), steps + it + 1)
        for got, old in zip((gp, gm, gv), before):
            assert np.array_equal(got[~inside], old[~inside])
        assert np.array_equal(bits_of(pb)[inside], B.to_bf16_bits_f32(dp.cpu().numpy())[inside])
        assert not bits_of(pb)[~inside].any()
    assert L.lora_device_status(ws) == 0


def test_adam_without_clipping_is_near_adam_step_multi():
    tensors, G, n, rng, g, shape, table, ws = _setup("one tensor")
    p = rng.standard_normal(n).astype(np.float32)
    a = [dev_f32(p), dev_f32(np.zeros(n)), dev_f32(np.zeros(n))]
    b = [t.clone() for t in a]
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    for t in range(3):
        L.adam_step_clipped(shape, table, st, a[0], dev_f32(g), a[1], a[2], float("inf"), LR, ws=ws)
        L.adam_step_multi([(0, n, t + 1)], b[0], dev_f32(g), b[1], b[2], LR)
    # adam_step_multi's 1 - beta2 is that of an fp32 0.999: v differs by 1.3e-5, sqrt(v) with its
    # correction cancels it but for some 1e-6 of the three steps
    _close(f64_of(a[2]), f64_of(b[2]), 2e-5)
    _close(f64_of(a[0]), f64_of(b[0]), 2.0 ** -22, extra=3 * LR * 1e-4)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["first", "last", "aligned tail"])
def test_non_finite_group_is_left_alone(bad, where):
    tensors, G, n, rng, g, shape, table, ws = _setup("unaligned")
    mine = sorted(t for t in tensors if t[2] == 2)
    at = {"first": mine[0][0], "last": mine[-1][0] + mine[-1][1] - 1, "aligned tail": mine[2][0] + mine[2][1] - 1}[where]
    g[at] = bad
    other = np.zeros(n, bool)
    for o, c, a in tensors:
        other[o:o + c] = a != 2
    inside = _inside(tensors, n)
    dg, out, norms = dev_f32(g), torch.zeros(n, device="cuda"), torch.empty(G, device="cuda")
    L.grad_clip(shape, table, dg, 0.1, out, norms, ws)
    assert L.lora_device_status(ws) == L.FLAG_NONFINITE_GRAD
    nn = f64_of(norms)
    assert not np.isfinite(nn[2]) and np.all(np.isfinite(np.delete(nn, 2)))
    mask = inside & ~other
    assert np.array_equal(out.cpu().numpy()[mask].view(np.uint32), g[mask].view(np.uint32))
    assert np.all(np.isfinite(out.cpu().numpy()[other]))
    p = rng.standard_normal(n).astype(np.float32)
    dp, dm, dv = dev_f32(p), dev_f32(np.zeros(n)), dev_f32(np.zeros(n))
    st = torch.full((G,), 4, dtype=torch.int64, device="cuda")
    pb = dev_bf16(np.zeros(n, np.uint16))
    L.adam_step_clipped(shape, table, st, dp, dg, dm, dv, 0.1, LR, p_bf16=pb, ws=ws)
    assert L.lora_device_status(ws) == L.FLAG_NONFINITE_GRAD
    assert list(st.cpu().numpy()) == [5, 5, 4, 5]
    got = dp.cpu().numpy()
    assert np.array_equal(got[mask], p[mask]) and not bits_of(pb)[mask].any() and not dm.cpu().numpy()[mask].any()
    # the others step: their m is a share of their g (p itself may move by less than its last bit)
    assert np.array_equal(dm.cpu().numpy()[other] != 0, g[other] != 0) and np.any(got[other] != p[other])


def test_fresh_workspace_on_another_stream():
    """A workspace that the call makes itself is cleared on the call's stream, not on a busy current one."""
    n = 5000
    g = torch.ones(n, device="cuda")
    g[7] = float("nan")
    shape, table = L.make_grad_table([(0, n, 0)], 1, n)
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    steps, side = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = torch.ones(4096, 4096, device="cuda")
    for _ in range(50):      # some milliseconds of work on the current stream
        a = a @ a * 2.0 ** -12
    ws = L.adam_step_clipped(shape, table, steps, p, g, m, v, 1.0, LR, stream=side)
    torch.cuda.synchronize()
    assert L.lora_device_status(ws) == L.FLAG_NONFINITE_GRAD and int(steps) == 0 and not bool(m.any())


def test_large_finite_gradients_do_not_overflow():
    n = 5000
    g = np.full(n, 3e38, np.float32)
    shape, table = L.make_grad_table([(0, n, 0)], 1, n)
    ws, out, norms = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(n, device="cuda"), torch.empty(1, device="cuda")
    L.grad_clip(shape, table, dev_f32(g), 1.0, out, norms, ws)
    # the norm itself is beyond fp32, the clipped gradient is not
    assert np.isinf(f64_of(norms)[0]) and L.lora_device_status(ws) == 0
    _close(f64_of(out), np.full(n, 1 / np.sqrt(n)), 2.0 ** -21)


def test_subnormal_gradients_are_not_rounded():
    """A factor of 1 (no clipping, or a group that is skipped) leaves every element's bits."""
    tiny = np.arange(1, 1001, dtype=np.uint32).view(np.float32)      # 1 .. 1000 times 2^-149
    g = np.concatenate((tiny, -tiny, np.float32([np.inf]), tiny))
    for split in (2000, 1):     # the Inf in a group of its own tail, then with nearly everything
        shape, table = L.make_grad_table([(0, split, 0), (split, len(g) - split, 1)], 2, len(g))
        ws, out = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(len(g), device="cuda")
        L.grad_clip(shape, table, dev_f32(g), float("inf"), out, None, ws)
        assert np.array_equal(out.cpu().numpy().view(np.uint32), g.view(np.uint32))
        assert L.lora_device_status(ws) == L.FLAG_NONFINITE_GRAD


def test_broken_tables_stay_inside_the_buffer():
    """Entries that break the rules are flagged and touch nothing outside n_elems."""
    n = 20000
    guard = torch.full((3 * n,), 5.0, device="cuda")
    g, out = torch.ones(n, device="cuda"), guard[n:2 * n]
    for bad in ([(0, 8192, 0, 0), (15000, 8192, 0, 1)], [(-8, 100, 0, 0), (0, 8, 0, 1)], [(0, 100, 7, 0), (0, 8, 0, 1)],
                [(0, 100, 0, 5), (0, 8, 0, 6)], [(0, 100, 0, -1), (200, 100, 0, 1)], [(0, 1 << 62, 0, 0), (0, 8, 0, 1)]):
        d = np.array(bad, L.GRAD_DTYPE)
        table = torch.from_numpy(d.view(np.uint8).copy()).to("cuda")
        shape = L.GradShape(n, 2, 2, 1)
        ws, norms = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(1, device="cuda")
        L.grad_clip(shape, table, g, 0.5, out, norms, ws)
        assert L.lora_device_status(ws) & L.FLAG_BAD_DESC
        assert bool((guard[:n] == 5).all()) and bool((guard[2 * n:] == 5).all())


@pytest.mark.parametrize("n_chunks, bad", [
    (2, [(0, 9000, 0, 0), (9000, 100, 0, 1)]),                        # the first tensor's second chunk is missing
    (2, [(0, 100, 0, 0), (200, 9000, 0, 1)]),                         # the last one's
    (1, [(0, 100, 0, 0), (200, 0, 1, 0)]),                            # an empty tensor before the last chunk's end
    (2, [(0, 100, 1, 0), (200, 100, 0, 1)]),                          # groups out of order
    (1, [(0, 0, 0, 0), (30000, 0, 0, 0), (0, 100, 0, 0)]),            # an empty tensor outside
    (2, [(0, 100, (1 << 31) - 1, 0), (200, 100, 0, 1)]),
])
def test_tables_that_leave_elements_out_are_flagged(n_chunks, bad):
    d = np.array(bad, L.GRAD_DTYPE)
    table = torch.from_numpy(d.view(np.uint8).copy()).to("cuda")
    shape = L.GradShape(20000, n_chunks, len(bad), 2)
    ws, norms, g = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(2, device="cuda"), torch.ones(20000, device="cuda")
    L.grad_norm(shape, table, g, norms, ws)
    assert L.lora_device_status(ws) & L.FLAG_BAD_DESC


def test_host_operands_are_refused():
    n = 100
    shape, table = L.make_grad_table([(0, n, 0)], 1, n)
    ws, g, norms = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.ones(n, device="cuda"), torch.empty(1, device="cuda")
    for name, args in (("table", (table.cpu(), g, norms, ws)), ("g", (table, g.cpu(), norms, ws)), ("norms", (table, g, norms.cpu(), ws)),
                       ("ws", (table, g, norms, ws.cpu()))):
        with pytest.raises(L.LoraError, match=name):
            L.grad_norm(shape, *args)
    with pytest.raises(L.LoraError, match="steps"):
        L.adam_step_clipped(shape, table, torch.zeros(1, dtype=torch.int64), g, g, g, g, 1.0, 1e-3, ws=ws)
    assert L.lora_device_status(ws) == 0


def test_no_tensors():
    shape, table = L.make_grad_table([], 3, 16)
    ws, norms = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.full((3,), -1.0, device="cuda")
    g = torch.ones(16, device="cuda")
    L.grad_clip(shape, table, g, 1.0, g, norms, ws)
    assert bool((norms == 0).all()) and bool((g == 1).all())


def test_elements_past_32_bits():
    """A tensor whose offset does not fit 32 bits."""
    n = (1 << 32) + 1000
    g = torch.zeros(n, device="cuda")
    g[n - 900:] = 2.0
    shape, table = L.make_grad_table([(n - 900, 900, 0), (0, 100, 1)], 2, n)
    ws, norms = L.empty_workspace(L.grad_workspace_bytes(shape)), torch.empty(2, device="cuda")
    L.grad_clip(shape, table, g, 6.0, g, norms, ws)
    assert list(f64_of(norms)) == [60.0, 0.0]
    _close(f64_of(g[n - 900:]), np.full(900, 0.2), 2.0 ** -21)
    assert not bool(g[:n - 900].any())


def _crowd(blocks_over):
    """20000 tensors of a few elements over 300 uneven groups, empty ones between them, and one group that spans many
    blocks: more chunks than blocks in every launch, groups that begin and end inside a block."""
    rng = np.random.default_rng(blocks_over)
    owner = np.sort((300 * rng.random(20000) ** 2).astype(int))
    counts = rng.integers(0, 6, 20000)
    counts[rng.integers(0, 20000, 40)] = rng.integers(8000, 9000, 40)
    counts[np.searchsorted(owner, 150)] = blocks_over * L.GRAD_CHUNK + 77
    gaps = rng.integers(0, 3, 20000)
    ends = np.cumsum(counts + gaps)
    tensors = [(int(e - g - c), int(c), int(a)) for e, g, c, a in zip(ends, gaps, counts, owner)]
    return tensors, 301, int(ends[-1]) + 3


@pytest.mark.parametrize("bad", [False, True])
def test_more_chunks_than_blocks(bad):
    tensors, G, n = _crowd(60)
    rng = np.random.default_rng(7)
    g = (rng.standard_normal(n) * np.exp2(rng.integers(-20, 4, n))).astype(np.float32)
    shape, table = L.make_grad_table(tensors, G, n)
    assert shape.n_chunks > 16384      # the most blocks of any launch
    ws = L.empty_workspace(L.grad_workspace_bytes(shape))
    owner = np.full(n, -1)
    for o, c, a in tensors:
        owner[o:o + c] = a
    inside = owner >= 0
    sick = 149 if bad else G     # (no group)
    if bad:
        g[np.flatnonzero(owner == sick)[-1]] = np.inf
    dg, norms = dev_f32(g), torch.full((G,), -1.0, device="cuda")
    flag = L.FLAG_NONFINITE_GRAD if bad else 0
    L.grad_norm(shape, table, dg, norms, ws)
    assert L.lora_device_status(ws) == flag
    want = OC.norms(tensors, G, g)
    _close(np.delete(f64_of(norms), sick) if bad else f64_of(norms), np.delete(want, sick) if bad else want, 2.0 ** -23)
    assert f64_of(norms)[G - 1] == 0 and (not bad or np.isinf(f64_of(norms)[sick]))
    max_norm = float(np.median(want[want > 0]))
    out, norms2 = torch.full((n,), 7.0, device="cuda"), torch.empty(G, device="cuda")
    L.grad_clip(shape, table, dg, max_norm, out, norms2, ws)
    assert L.lora_device_status(ws) == flag and torch.equal(norms, norms2)
    res, _ = OC.clip(tensors, G, g, max_norm, out=np.full(n, 7.0))
    fine = owner != sick
    _close(f64_of(out)[fine], res[fine], 2.0 ** -22, extra=2.0 ** -149)
    assert np.array_equal(f64_of(out)[~inside], np.full((~inside).sum(), 7.0))
    assert np.array_equal(out.cpu().numpy()[~fine], g[~fine])
    p, m = rng.standard_normal(n).astype(np.float32), (rng.standard_normal(n) * 0.1).astype(np.float32)
    v = (rng.random(n) * 0.01 + 1e-4).astype(np.float32)
    steps = rng.integers(0, 50, G)
    dp, dm, dv, st, pb = dev_f32(p), dev_f32(m), dev_f32(v), torch.from_numpy(steps).to("cuda"), dev_bf16(np.zeros(n, np.uint16))
    L.adam_step_clipped(shape, table, st, dp, dg, dm, dv, max_norm, LR, B1, B2, EPS, 0.1, p_bf16=pb, norms=norms2, ws=ws)
    assert L.lora_device_status(ws) == flag and torch.equal(norms, norms2)
    want_p, want_m, want_v, want_steps, _ = OC.adam_clipped(tensors, G, steps, p, g, m, v, max_norm, LR, B1, B2, EPS, 0.1)
    assert np.array_equal(st.cpu().numpy(), want_steps)
    cg = np.where(fine, OC.clip(tensors, G, g, max_norm)[0], 0.0)
    gp, gm, gv = (f64_of(a) for a in (dp, dm, dv))
    slack = 2.0 ** -21 * (np.abs(B1 * m.astype(np.float64)) + np.abs((1 - B1) * cg))
    _close(gm, want_m, 0, extra=slack)
    _close(gv, want_v, 2.0 ** -21)
    t = np.where(inside, want_steps[owner], 1)
    t = np.where(fine, t, 1)
    per_m = LR / (1 - B1 ** t) / (np.sqrt(want_v / (1 - B2 ** t)) + EPS)
    _close(gp, want_p, 0, extra=2.0 ** -22 * np.abs(p) + per_m * (slack + 2.0 ** -20 * np.abs(want_m)))
    still = ~inside | ~fine
    for got, old in ((gp, p), (gm, m), (gv, v)):
        assert np.array_equal(got[still], old[still])
    assert np.array_equal(bits_of(pb)[~still], B.to_bf16_bits_f32(dp.cpu().numpy())[~still]) and not bits_of(pb)[still].any()


def test_counters_that_count_no_steps():
    """A negative step counter (or one that cannot be counted up) has no step 1 or later: the group keeps its values
    and its counter and is flagged, as adam_step refuses steps below 1; the others step."""
    n, top = 5000, (1 << 63) - 1
    tensors = [(0, 1000, 0), (1000, 9, 1), (1009, 1500, 2), (2509, 500, 3)]      # group 4 has no tensor
    shape, table = L.make_grad_table(tensors, 6, n)
    ws = L.empty_workspace(L.grad_workspace_bytes(shape))
    rng = np.random.default_rng(3)
    p, g = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    steps = np.array([-1, 0, -7, top, -2, 4])
    dp, dm, dv, st, norms = dev_f32(p), dev_f32(np.zeros(n)), dev_f32(np.zeros(n)), torch.from_numpy(steps).to("cuda"), torch.empty(6, device="cuda")
    L.adam_step_clipped(shape, table, st, dp, dev_f32(g), dm, dv, 1.0, LR, norms=norms, ws=ws)
    assert L.lora_device_status(ws) == L.FLAG_BAD_DESC
    assert list(st.cpu().numpy()) == [-1, 1, -7, top, -2, 5]
    moved = np.zeros(n, bool)
    moved[1000:1009] = True
    assert np.array_equal(dp.cpu().numpy()[~moved], p[~moved]) and not dm.cpu().numpy()[~moved].any() and not dv.cpu().numpy()[~moved].any()
    assert np.all(dp.cpu().numpy()[moved] != p[moved]) and np.all(np.isfinite(dp.cpu().numpy()))
    _close(f64_of(norms), OC.norms(tensors, 6, g), 2.0 ** -23)
