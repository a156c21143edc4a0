"""The paged key-value cache against the float64 oracle: page tables and slots (exact),
rows written (bf16 bits; 8-bit codes exact), and the attention of one new token.

Tolerances of the attention as in test_gpu_attention: u = 2^-8, e = 2^-24, a weight off by
the factor w = 2 (d + 4) e max(sum|q k| scale) + 8 e (max|s| + 4);
|o error| <= (u |o| + (u + 2 w + n e) sum p|v|) (1 + 2 u); the joins of the splits scale by
fp32 factors: 8 e more of sum p|v|, within the factor's second 2 u.
"""
import numpy as np
import pytest

import oracle.attention as OA
import oracle.norm as ON
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


def put(a):
    return dev_bf16(B.to_bf16_bits(a))


# ---------------------------------------------------------------- tables

class Tables:
    def __init__(self, n, page, n_pages, width, n_slots, seed=0, head=0):
        rng = np.random.default_rng(seed)
        self.page, self.n_slots = page, n_slots
        self.shape = L.make_kv_shape(n, 1, 64, page, n_pages, width)
        self.lens, self.table = [0] * n, [[-7] * width for _ in range(n)]
        self.ring = np.roll(rng.permutation(n_pages), head % n_pages).tolist()
        self.state = (head, head + n_pages)
        i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
        self.d = {"lens": dev_i32(self.lens), "table": dev_i32(self.table), "ring": dev_i32(self.ring),
                  "state": torch.tensor(self.state, device="cuda"), "cu": i32(n + 1), "slots": i32(n_slots), "positions": i32(n_slots),
                  "token_seqs": i32(n_slots)}
        self.ws = L.empty_workspace(L.kv_tables_workspace_bytes(self.shape))

    def call(self, new):
        d = self.d
        L.kv_tables(self.shape, d["lens"], dev_i32(new), d["lens"], d["table"], d["ring"], d["state"], d["state"], d["cu"], d["slots"], self.ws,
                    positions=d["positions"], token_seqs=d["token_seqs"])

    def step(self, new):
        """One step in place, against the oracle's."""
        self.call(new)
        self.lens, cu, slots, pos, seqs, self.state, short = OA.kv_tables(self.lens, list(new), self.table, self.ring, self.state, self.page, self.n_slots)
        want = {"lens": self.lens, "table": self.table, "ring": self.ring, "state": self.state, "cu": cu, "slots": slots, "positions": pos, "token_seqs": seqs}
        for k, w in want.items():
            got = self.d[k].cpu().numpy()
            assert np.array_equal(got, np.array(w, got.dtype).reshape(got.shape)), k
        assert L.lora_device_status(self.ws) == (L.FLAG_NO_PAGES if short else 0)
        return short


@pytest.mark.parametrize("n,page,n_slots", [(1, 16, 40), (7, 16, 200), (64, 32, 4096), (65, 16, 5000), (1000, 16, 20000), (1500, 64, 4000)])
def test_tables_over_many_steps(n, page, n_slots):
    """Requests that start, grow, wait, end and start anew; few pages, so that some go without."""
    rng = np.random.default_rng(n)
    most = max(1, n_slots // n)
    t = Tables(n, page, max(3, n * 3), 8, n_slots, seed=n, head=5 * n)
    short = 0
    for _ in range(12):
        room = 8 * page - np.array(t.lens)
        new = np.minimum(rng.integers(0, most + 1, n), room)
        new = np.where((rng.random(n) < 0.15) | (room < most), -1, new)
        short += t.step(new.tolist())
    assert short or n < 60 or page == 64   # (some went without pages)


def test_tables_edges():
    t = Tables(3, 16, 6, 3, 64)
    t.step([16, 17, 0])       # a page filled to its end; one row over it
    t.step([1, -1, 0])
    t.step([-1, -1, 33])      # an ended request without rows ends again; a page freed in this step is not taken in it
    t.step([48, -1, -1])
    t.step([0, 48, -1])
    none = L.make_kv_shape(0, 1, 64, 16, 4, 1)
    st, i32 = torch.tensor([4, 8], device="cuda"), lambda *s: torch.full(s, 5, dtype=torch.int32, device="cuda")
    cu, slots, out = i32(1), i32(3), torch.zeros(2, dtype=torch.int64, device="cuda")
    L.kv_tables(none, i32(0), i32(0), i32(0), i32(0, 1), i32(4), st, out, cu, slots, t.ws)
    assert cu.item() == 0 and slots.tolist() == [-1] * 3 and out.tolist() == [4, 8]


def test_tables_separate_outputs_leave_inputs():
    t = Tables(40, 16, 100, 4, 300, seed=4)
    t.step([3] * 40)
    d = {k: v.clone() for k, v in t.d.items()}
    lens, state = torch.full_like(d["lens"], -3), torch.zeros_like(d["state"])
    new = dev_i32([5, -1] * 20)
    for _ in range(2):   # the same call twice gives the same
        L.kv_tables(t.shape, d["lens"], new, lens, d["table"], d["ring"], d["state"], state, None, d["slots"], t.ws)
    assert torch.equal(d["lens"], t.d["lens"]) and torch.equal(d["state"], t.d["state"])
    t.step([5, -1] * 20)
    assert lens.tolist() == t.lens and tuple(state.tolist()) == t.state and torch.equal(d["slots"], t.d["slots"])
    assert torch.equal(d["table"], t.d["table"]) and torch.equal(d["ring"], t.d["ring"])


@pytest.mark.parametrize("n_slots", [64, 6000])
def test_tables_refuse_bad_requests_alone(n_slots):
    t = Tables(6, 16, 50, 2, n_slots, seed=5)
    t.step([4, 4, 4, 4, 4, 4])
    before = {k: v.clone() for k, v in t.d.items()}
    # too long for its table; a negative length; a negative length that ends; int32's ends
    t.d["lens"][2] = -1
    t.d["lens"][3] = -5
    t.d["lens"][4] = 2 ** 31 - 1
    t.call([29, 1, 1, -1, 2 ** 31 - 1, 1])
    assert L.lora_device_status(t.ws) == L.FLAG_BAD_LENGTH
    lens = t.d["lens"].tolist()
    assert lens == [4, 5, -1, -5, 2 ** 31 - 1, 4]     # the last: its row lies behind n_slots, as request 4's do
    slots = t.d["slots"].tolist()
    assert slots[:29] == [-1] * 29 and slots[29] == t.d["table"][1, 0].item() * 16 + 4 and slots[30:] == [-1] * (n_slots - 30)
    assert t.d["cu"].tolist() == [0, 29, 30, 31, 31, n_slots, n_slots]
    assert torch.equal(t.d["table"], before["table"]) and torch.equal(t.d["ring"], before["ring"]) and torch.equal(t.d["state"], before["state"])


@pytest.mark.parametrize("n_slots", [64, 6000])
def test_tables_no_positions_where_lengths_break_the_rules(n_slots):
    """Rows of a request with a negative length, or of more rows than its table holds, have no position: -1, as behind the last row."""
    t = Tables(6, 16, 50, 2, n_slots, seed=5)
    t.step([4, 4, 4, 4, 4, 4])
    t.d["lens"][1], t.d["lens"][3], t.d["lens"][4] = -3, 30, 2 ** 31 - 1
    t.call([2, 3, 1, 3, 5, 2])      # request 3 would end at row 33 of 32
    assert L.lora_device_status(t.ws) == L.FLAG_BAD_LENGTH
    assert t.d["positions"].tolist()[:16] == [4, 5, -1, -1, -1, 4, -1, -1, -1, -1, -1, -1, -1, -1, 4, 5]
    assert t.d["token_seqs"].tolist()[:16] == [0, 0, 1, 1, 1, 2, 3, 3, 3, 4, 4, 4, 4, 4, 5, 5]
    page = [t.d["table"][b, 0].item() * 16 for b in range(6)]
    assert t.d["slots"].tolist()[:16] == [page[0] + 4, page[0] + 5, -1, -1, -1, page[2] + 4] + [-1] * 8 + [page[5] + 4, page[5] + 5]
    for k in ("slots", "positions", "token_seqs"):
        assert t.d[k].tolist()[16:] == [-1] * (n_slots - 16), k


def test_tables_bad_ring():
    for state in ([5, 4], [-1, 3], [0, 51], [2 ** 62, -2 ** 62]):
        t = Tables(2, 16, 50, 4, 64)
        t.d["lens"].copy_(torch.tensor([3, 16]))
        t.d["table"].copy_(torch.tensor([[1, 0, 0, 0], [2, 0, 0, 0]]))
        t.d["state"].copy_(torch.tensor(state))
        ring = t.d["ring"].clone()
        t.call([1, 1])      # one needs no page, the other one
        assert L.lora_device_status(t.ws) == L.FLAG_BAD_PAGE | L.FLAG_NO_PAGES
        assert t.d["lens"].tolist() == [4, 16] and t.d["slots"].tolist()[:2] == [19, -1] and t.d["state"].tolist() == state
        t.call([-1, 0])
        assert L.lora_device_status(t.ws) == L.FLAG_BAD_PAGE and torch.equal(t.d["ring"], ring)
    t = Tables(2, 16, 4, 4, 64)          # more pages put than the ring has room for
    t.d["lens"].copy_(torch.tensor([3, 16]))
    t.call([-1, 0])
    assert L.lora_device_status(t.ws) == L.FLAG_BAD_PAGE and t.d["state"].tolist() == [0, 4]
    t = Tables(2, 16, 4, 4, 64)          # page ids out of range, in the ring and in a table
    t.d["ring"].copy_(torch.tensor([9, -1, 2, 2 ** 31 - 1]))
    t.call([20, 3])
    assert L.lora_device_status(t.ws) == L.FLAG_BAD_PAGE
    assert t.d["slots"].tolist() == [-1] * 20 + [32, 33, 34] + [-1] * 41
    t.call([1, 1])
    assert L.lora_device_status(t.ws) == L.FLAG_BAD_PAGE and t.d["slots"].tolist()[:2] == [-1, 35]


def test_tables_graph_steps_on():
    """A captured step (in place) walks on with every replay, past pages' ends."""
    t = Tables(5, 16, 30, 4, 5, seed=6, head=29)
    t.step([1] * 5)
    new = dev_i32([1, 1, 0, 1, 1])
    d = t.d
    run = lambda: L.kv_tables(t.shape, d["lens"], new, d["lens"], d["table"], d["ring"], d["state"], d["state"], d["cu"], d["slots"], t.ws,  # noqa: E731
                              positions=d["positions"], token_seqs=d["token_seqs"])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    scratch = torch.empty(1 << 20, device="cuda")
    for _ in range(40):
        g.replay()
        scratch.normal_()
        torch.cuda.synchronize()
        t.lens, cu, slots, pos, seqs, t.state, _ = OA.kv_tables(t.lens, [1, 1, 0, 1, 1], t.table, t.ring, t.state, 16, 5)
        assert d["lens"].tolist() == t.lens and d["slots"].tolist() == slots and d["table"].tolist() == t.table
        assert tuple(d["state"].tolist()) == t.state


# ---------------------------------------------------------------- writes

def caches(n_pages, kv, page, d, x8, fill=3):
    if not x8:
        return [torch.full((n_pages, kv, page, d), float(fill), dtype=torch.bfloat16, device="cuda") for _ in range(2)] + [None, None]
    return [torch.full((n_pages, kv, page, d), fill, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
           [torch.full((n_pages, kv, page, d // 32), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]


def codes_of(rows):
    """(e4m3 codes, E8M0 bytes) of rows [n][kv][d] by the oracle's rounding."""
    n, kv, d = rows.shape
    q, e = ON.quantize8(rows.reshape(n * kv, d))
    code = torch.from_numpy(q).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return code.reshape(n, kv, d), (e + 127).astype(np.uint8).reshape(n, kv, d // 32)


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("n,kv,d,page", [(1, 1, 64, 16), (3, 8, 128, 16), (67, 5, 64, 32), (300, 3, 128, 256), (33, 1, 128, 64)])
def test_write(n, kv, d, page, x8):
    rng = np.random.default_rng(n)
    n_pages = -(-n // page) + 5
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 2:
        slots[1] = -1
    rows = [B.round_bf16(rng.standard_normal((n, kv, d)) * np.exp2(rng.integers(-30, 30, (n, kv, 1)))) for _ in range(2)]
    for r in rows:
        r[-1, 0, :32] = 0
    dev = [torch.cat((put(r), put(r[:, :1])), 1)[:, :kv] for r in rows]    # rows that lie apart
    c = caches(n_pages, kv, page, d, x8)
    ws = L.empty_workspace(256)
    shape = L.make_kv_shape(1, kv, d, page, n_pages, 1)
    L.kv_write(shape, *dev, dev_i32(slots), c[0], c[1], ws, k_scales=c[2], v_scales=c[3])
    assert L.lora_device_status(ws) == 0
    for i in range(2):
        want = [3.0 * np.ones(c[0].shape)] if not x8 else [np.full(c[0].shape, 3), np.full(c[2].shape, 3)]
        parts = [rows[i]] if not x8 else codes_of(rows[i])
        for t, s in enumerate(slots):
            if s >= 0:
                for w, p in zip(want, parts):
                    w[s // page, :, s % page] = p[t]
        for w, got in zip(want, c[i::2]):
            assert np.array_equal(f64_of(got), w)


def test_write_not_finite_and_bad_slots():
    kv, d, page = 2, 64, 16
    x = torch.zeros(5, kv, d, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0], x[0, 0, 1], x[1, 1, 40] = NAN, 2.0, float("inf")
    shape, ws = L.make_kv_shape(1, kv, d, page, 2, 1), L.empty_workspace(256)
    for bad in (32, 2 ** 31 - 1, -2, -2 ** 31):
        c = caches(2, kv, page, d, True)
        L.kv_write(shape, x, x, dev_i32([0, 31, -1, bad, 5]), c[0], c[1], ws, k_scales=c[2], v_scales=c[3])
        assert L.lora_device_status(ws) == L.FLAG_BAD_PAGE
        codes = c[0].view(torch.float8_e4m3fn).float()
        assert torch.isnan(codes[0, 0, 0, 0]) and codes[0, 0, 0, 1] * 2.0 ** (c[2][0, 0, 0, 0].item() - 127) == 2.0
        assert torch.isnan(codes[1, 1, 15, 40])
        untouched = torch.ones(2, page, dtype=torch.bool)
        untouched[0, 0] = untouched[0, 5] = untouched[1, 15] = False
        for t in c:
            assert (t.permute(0, 2, 1, 3)[untouched.cuda()] == 3).all()


# ---------------------------------------------------------------- decoding

class Decode:
    def __init__(self, lens, heads=4, kv=2, d=64, page=16, x8=False, scale=None, seed=0, n_pages=None, spare=2, gain=1.0, max_len=None):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv, self.d, self.page, self.x8 = list(lens), heads, kv, d, page, x8
        self.scale = float(np.float32(d ** -0.5 if scale is None else scale))
        need = [-(-n // page) for n in lens]
        self.n_pages = n_pages or sum(need) + spare
        width = max([1, *need]) + 1
        ids = rng.permutation(self.n_pages)[:sum(need)] if n_pages is None else self.n_pages - 1 - rng.permutation(sum(need))
        self.table = np.full((len(lens), width), 2 ** 31 - 1, np.int64)   # entries behind a request's pages: never read
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        self.q = B.round_bf16(gain * rng.standard_normal((len(lens), heads, d)))
        total = sum(lens)
        rows = [B.round_bf16(rng.standard_normal((total, kv, d))) for _ in range(2)]
        self.slots = np.array([self.table[b, p // page] * page + p % page for b, n in enumerate(lens) for p in range(n)], np.int64)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.max_len = max([0, *lens]) if max_len is None else max_len
        self.shape = L.make_kv_shape(len(lens), kv, d, page, self.n_pages, width)
        shape = (self.n_pages, kv, page)
        # whatever lies behind a request's last row: NaN, in codes and in scales too
        if x8:
            self.c = [torch.full((*shape, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
                     [torch.full((*shape, d // 32), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        else:
            self.c = [torch.full((*shape, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2)] + [None, None]
        page_at, row_at = (torch.from_numpy(a).cuda() for a in (self.slots // page, self.slots % page))
        self.rows = []
        for i, r in enumerate(rows):
            if x8:
                code, byte = codes_of(r) if total else (np.zeros((0, kv, d), np.uint8), np.zeros((0, kv, d // 32), np.uint8))
                self.c[i][page_at, :, row_at] = torch.from_numpy(code).cuda()
                self.c[2 + i][page_at, :, row_at] = torch.from_numpy(byte).cuda()
                val = torch.from_numpy(code).view(torch.float8_e4m3fn).double().numpy()
                r = val * np.repeat(np.exp2(byte.astype(float) - 127), 32, -1)
            else:
                self.c[i][page_at, :, row_at] = put(r)
            self.rows.append(r)
        self.dq = put(self.q)
        self.tab, self.dl = dev_i32(self.table), dev_i32(self.lens)
        self.o = torch.full((len(lens), heads, d), NAN, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((len(lens), heads), NAN, device="cuda")
        self.ws = torch.full((max(256, L.attention_decode_workspace_bytes(self.shape, heads, self.max_len)),), 0xFF, dtype=torch.uint8, device="cuda")
        L.lora_workspace_init(self.ws)

    def run(self, lse=True, stream=None):
        L.attention_decode(self.shape, self.dq, self.c[0], self.c[1], self.tab, self.dl, self.max_len, self.scale, self.o, self.ws,
                           k_scales=self.c[2], v_scales=self.c[3], lse=self.lse if lse else None, stream=stream)
        return f64_of(self.o), f64_of(self.lse)

    def check(self):
        o, lse = self.run()
        assert L.lora_device_status(self.ws) == 0
        group = self.heads // self.kv
        for b, n in enumerate(self.lens):
            s = slice(self.cu[b], self.cu[b + 1])
            for h in range(self.heads):
                q, k, v = self.q[b, h][None], self.rows[0][s, h // group], self.rows[1][s, h // group]
                ro, rl, p = OA.head_forward(q, k, v, self.scale, False)
                if n == 0:
                    assert np.all(o[b, h] == 0) and lse[b, h] == -np.inf
                    continue
                big = (np.abs(q) @ np.abs(k).T).max() * abs(self.scale)
                w = 2 * (self.d + 4) * E * big + 8 * E * (big + 4)
                tol = (U * np.abs(ro) + (U + 2 * w + n * E) * (p @ np.abs(v))) * (1 + 2 * U)
                assert np.all(np.abs(o[b, h] - ro[0]) <= tol[0]), (b, h, np.max(np.abs(o[b, h] - ro[0]) / tol[0]))
                assert abs(lse[b, h] - rl[0]) <= w + n * E + 4 * E * abs(rl[0]), (b, h)
        return o, lse


LENS = [[1], [0, 3, 0], [15, 16, 17], [127, 128, 129, 130], [31, 32, 33, 64, 65, 96], [256, 511], [255, 257, 513, 1025], [700, 5]]


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_decode_lengths(lens, d, x8):
    Decode(lens, d=d, x8=x8, seed=sum(lens)).check()


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 1), (24, 3), (14, 2)])
def test_decode_head_groups(heads, kv, x8):
    Decode([200, 37], heads=heads, kv=kv, d=128, x8=x8, seed=heads).check()


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(page, x8):
    Decode([1, 300, 255, 257], d=128, page=page, x8=x8, seed=page).check()


@pytest.mark.parametrize("n", [4096, 4097, 5000, 8193, 20000])
def test_decode_long(n):
    """Around the lengths where a split grows; more than one tile a wave."""
    Decode([n, 77], heads=2, kv=1, d=64, seed=n).check()


@pytest.mark.parametrize("x8", [False, True])
def test_decode_peaked_and_flat(x8):
    Decode([400, 90], d=128, x8=x8, gain=20.0, seed=1).check()
    Decode([400, 90], d=128, x8=x8, scale=0.0, seed=2).check()
    Decode([400, 90], d=128, x8=x8, scale=-0.5, seed=3).check()


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 28])
def test_decode_scores_of_any_documented_size(size):
    """As in attention over prompts: growing scores up to 2^28, so the last key has all the weight."""
    lens = [1, 40, 128, 77]
    c = Decode(lens, heads=2, kv=1, d=64, scale=1.0, seed=12)
    q = np.zeros(c.q.shape)
    q[:, :, 3] = size
    c.dq = put(q)
    k = np.zeros(c.rows[0].shape)
    k[:, 0, 3] = np.concatenate([np.arange(n) / 128.0 for n in lens])
    page_at, row_at = (torch.from_numpy(a).cuda() for a in (c.slots // c.page, c.slots % c.page))
    c.c[0][page_at, :, row_at] = put(k)
    o, lse = c.run()
    assert L.lora_device_status(c.ws) == 0
    for b, n in enumerate(lens):
        v, s = c.rows[1][c.cu[b + 1] - 1, 0], size * (n - 1) / 128.0
        assert np.all(np.abs(o[b] - v) <= 2 * U * (1 + U) * np.abs(v)), b
        assert np.all(np.abs(lse[b] - s) <= 8 * E * s + 8 * E), b


@pytest.mark.parametrize("x8", [False, True])
def test_decode_same_bits_in_every_batch(x8):
    lens = [300, 1, 2000, 129, 4500]
    c = Decode(lens, heads=4, kv=1, d=128, x8=x8, seed=4)
    o, lse = c.run()
    again, _ = c.run()
    assert np.array_equal(o, again)
    for b in range(len(lens)):
        c1 = Decode(lens, heads=4, kv=1, d=128, x8=x8, seed=4)
        w = c1.table.shape[1]
        c1.shape = L.make_kv_shape(1, 1, 128, 16, c1.n_pages, w)
        c1.dq, c1.tab, c1.dl, c1.o, c1.lse = c.dq[b:b + 1], c.tab[b:b + 1], c.dl[b:b + 1], c1.o[:1], c1.lse[:1]
        c1.max_len = min(lens[b] + 40 * b, w * 16)      # another bound, another launch
        o1, lse1 = c1.run()
        assert np.array_equal(o1[0], o[b]) and np.array_equal(lse1[0], lse[b]), b


@pytest.mark.parametrize("d,kv,group,x8", [(128, 8, 2, False), (64, 8, 4, True), (128, 4, 16, True), (128, 4, 9, False)])
def test_decode_large_batches_cut_elsewhere(d, kv, group, x8):
    """Batches large enough that a block takes 2, 4 and 8 units: the bits of requests alone."""
    rng = np.random.default_rng(d + group)
    for n, longest in ((256, 400), (300, 1100), (400, 4200)):
        lens = rng.integers(0, longest, n)
        lens[:4] = longest, longest - 127, longest // 2 + 1, 130
        pages = -(-lens // 16)
        ids = torch.randperm(int(pages.sum()), device="cuda", dtype=torch.int32)
        width = int(pages.max())
        table = torch.zeros(n, width, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < torch.from_numpy(pages).cuda()[:, None]] = ids
        shape = (len(ids), kv, 16, d)
        if x8:
            c = [torch.randint(0, 0x7E, shape, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
                [torch.randint(115, 122, (*shape[:3], d // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
        else:
            c = [torch.randn(shape, device="cuda").bfloat16() for _ in range(2)] + [None, None]
        q = torch.randn(n, kv * group, d, device="cuda").bfloat16()

        def run(rows, bound):
            m = len(rows)
            s = L.make_kv_shape(m, kv, d, 16, len(ids), width)
            o, lse = torch.full((m, kv * group, d), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((m, kv * group), NAN, device="cuda")
            ws = torch.full((L.attention_decode_workspace_bytes(s, kv * group, bound),), 0xFF, dtype=torch.uint8, device="cuda")
            L.lora_workspace_init(ws)
            L.attention_decode(s, q[rows].contiguous(), c[0], c[1], table[rows].contiguous(), dev_i32(lens[rows]), bound, 0.1, o, ws,
                               k_scales=c[2], v_scales=c[3], lse=lse)
            assert L.lora_device_status(ws) == 0
            return o, lse

        o, lse = run(np.arange(n), longest)
        assert not torch.isnan(o).any()
        for b in (0, 1, 2, 3, n - 1):
            o1, lse1 = run(np.array([b]), width * 16)
            assert torch.equal(o1[0], o[b]) and torch.equal(lse1[0], lse[b]), (n, b)


def test_decode_heads_leave_one_another_alone():
    """A head's bits do not follow the scores of its group's other heads."""
    c = Decode([300, 1, 777], heads=8, kv=2, d=128, seed=7)
    o, lse = c.run()
    keep = c.dq.clone()
    c.dq[:, 1::2] *= 40
    o2, lse2 = c.run()
    c.dq.copy_(keep)
    assert np.array_equal(o2[:, ::2], o[:, ::2]) and np.array_equal(lse2[:, ::2], lse[:, ::2])
    assert not np.array_equal(o2[2, 1::2], o[2, 1::2])


def test_decode_q_in_a_fused_row():
    c = Decode([40, 200, 3], heads=6, kv=2, d=64, seed=5)
    wide = torch.full((3, 10, 64), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, :6] = c.dq
    c.dq = wide[:, :6]
    c.check()
    o = c.o.clone()
    c.o.fill_(NAN)
    c.run(lse=False)
    assert torch.equal(o, c.o)


def test_decode_far_pages():
    """Pages whose elements lie past 2^31 and bytes past 2^32."""
    n_pages = (2 ** 31 + 2 ** 25) // (8 * 16 * 128)
    c = Decode([300, 20], heads=16, kv=8, d=128, n_pages=n_pages, seed=6)
    assert c.slots.max() * 8 * 128 > 2 ** 31
    c.check()
    # the same rows, written by the library
    for t in c.c[:2]:
        t.view(torch.int16)[n_pages - 40:] = -1
    ws = L.empty_workspace(256)
    L.kv_write(c.shape, put(c.rows[0]), put(c.rows[1]), dev_i32(c.slots), c.c[0], c.c[1], ws)
    c.check()


def test_decode_bad_pages_and_lengths():
    c = Decode([100, 60, 300], heads=4, kv=2, d=64, seed=7)
    o, _ = c.run()
    for bad in (c.n_pages, -1, 2 ** 31 - 1, -2 ** 31):
        tab = c.tab.clone()
        tab[1, 1] = bad                              # rows 16 .. 31 of the second request
        c.tab, keep = tab, c.tab
        got, _ = c.run()
        c.tab = keep
        assert L.lora_device_status(c.ws) == L.FLAG_BAD_PAGE
        assert np.array_equal(got[0], o[0]) and np.array_equal(got[2], o[2]) and np.isfinite(got[1]).all()
        s = c.cu[1]
        rows = [np.delete(r[s:s + 60], np.s_[16:32], 0) for r in c.rows]
        for h in range(4):
            ro, _, p = OA.head_forward(c.q[1, h][None], rows[0][:, h // 2], rows[1][:, h // 2], c.scale, False)
            assert np.all(np.abs(got[1, h] - ro[0]) <= 3 * U * (p @ np.abs(rows[1][:, h // 2]))[0])
    for bad in (301, -1, 2 ** 31 - 1, -2 ** 31):
        c.dl[2] = bad
        got, lse = c.run()
        assert L.lora_device_status(c.ws) == L.FLAG_BAD_LENGTH
        assert np.array_equal(got[:2], o[:2]) and np.all(got[2] == 0) and np.all(np.isneginf(lse[2]))


def test_decode_not_finite_rows():
    """A NaN of a request's own reaches that request's heads that read it, and nothing else."""
    c = Decode([50, 140], heads=4, kv=2, d=64, seed=8)
    o, _ = c.run()
    s = c.slots[c.cu[1] + 130]
    c.c[1][s // 16, 1, s % 16, 7] = NAN
    got, _ = c.run()
    assert np.isnan(got[1, 2:, 7]).all()
    got[1, 2:, 7] = o[1, 2:, 7]
    assert np.array_equal(got, o)
    c.c[0][s // 16, 0, s % 16, 3] = NAN
    got, lse = c.run()
    assert np.isnan(got[1, :2]).all() and np.isnan(lse[1, :2]).all() and np.array_equal(got[0], o[0])


def test_decode_empty():
    c = Decode([], seed=9)
    c.run()
    c = Decode([0, 0], seed=10)
    c.check()


def test_decode_graph_and_streams():
    c = Decode([500, 30, 0, 4200], heads=8, kv=2, d=128, seed=11)
    other = Decode([100], seed=12)
    call = lambda stream=None: L.attention_decode(c.shape, c.dq, c.c[0], c.c[1], c.tab, c.dl, c.max_len, c.scale, c.o, c.ws, lse=c.lse, stream=stream)  # noqa: E731
    _replay_check(call, [c.o, c.lse], lambda: other.run())
    call()
    torch.cuda.synchronize()
    ref = c.o.clone()
    c.o.fill_(NAN)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    assert torch.equal(ref, c.o)


def test_binding_refuses():
    c = Decode([20], x8=True, seed=13)
    kw = dict(k_scales=c.c[2], v_scales=c.c[3])
    call = lambda q=c.dq, kc=c.c[0], tab=c.tab, dl=c.dl, o=c.o, ws=c.ws, n=c.max_len, **k: L.attention_decode(c.shape, q, kc, c.c[1], tab, dl, n, c.scale, o, ws, **{**kw, **k})  # noqa: E731
    call()
    for bad in ({"q": c.dq.float()}, {"kc": c.c[0][:-1]}, {"tab": c.tab[:, :1]}, {"dl": c.dl.long()}, {"o": c.o.cpu()}, {"ws": c.ws[:100]},
                {"k_scales": None}, {"v_scales": None}, {"n": -1}, {"n": 10 ** 6}, {"o": c.dq}, {"kc": c.c[0].view(torch.bfloat16)}):
        with pytest.raises(L.LoraError):
            call(**bad)
