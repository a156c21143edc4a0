"""Host-side refusals of the attention and key-value cache calls (CPU only: every call here
fails before anything is enqueued, or has nothing to do, whatever its pointers hold)."""
import ctypes
import time

import pytest

from test_operator_refusals import BIG, L, ODD, P, _is  # noqa: F401


def at(n):
    return ctypes.c_void_p(n << 20)     # buffers 1 MiB apart, never dereferenced


def test_attention(L):  # noqa: F811
    lib, E = L.LIB, L.LORA_E_INVALID_ARG
    good = dict(n_q=100, n_k=120, n_seqs=3, n_heads=4, n_kv_heads=2, head_dim=64, scale=0.1)
    mk = lambda **kw: L.make_attention_shape(**{**good, **kw})  # noqa: E731
    need = L.attention_workspace_bytes(mk())
    assert 256 + 8 * 4 * 100 <= need

    def fwd(s=None, q=at(1), k=at(2), v=at(3), cq=P, ck=P, o=at(4), lse=at(10), ws=at(11), nb=BIG):
        return lib.attention_forward(ctypes.byref(s or mk()), q, k, v, cq, ck, o, lse, ws, nb, None)

    def bwd(s=None, do=at(1), q=at(2), k=at(3), v=at(4), o=at(5), lse=at(10), cq=P, ck=P, dq=at(6), dk=at(7), dv=at(8), ws=at(11), nb=BIG):
        return lib.attention_backward(ctypes.byref(s or mk()), do, q, k, v, o, lse, cq, ck, dq, dk, dv, ws, nb, None)

    shapes = [(dict(n_q=-1), E, b"n_q"), (dict(n_k=1 << 30), E, b"n_k"), (dict(n_seqs=-1), E, b"n_seqs"), (dict(n_seqs=65537), E, b"n_seqs"),
              (dict(n_heads=3), E, b"multiple"), (dict(n_heads=0), E, b"multiple"), (dict(n_kv_heads=0), E, b"multiple"),
              (dict(n_heads=1026), E, b"1024"), (dict(head_dim=80), L.LORA_E_UNSUPPORTED, b"64 or 128"), (dict(head_dim=256), L.LORA_E_UNSUPPORTED, b"64 or 128"),
              (dict(scale=float("nan")), E, b"scale"), (dict(scale=float("inf")), E, b"scale"), (dict(scale=-(2.0 ** 127)), E, b"scale"), (dict(causal=2), E, b"causal"),
              (dict(q_stride=255), E, b"multiple of 8"), (dict(q_stride=248), E, b"shorter"), (dict(k_stride=120), E, b"shorter"),
              (dict(v_stride=-8), E, b"shorter"), (dict(o_stride=1 << 24), E, b"2^24"),
              (dict(n_q=(1 << 30) - 1, n_heads=1024, n_kv_heads=2), L.LORA_E_UNSUPPORTED, b"one launch"),
              (dict(n_seqs=65536, n_heads=128, n_kv_heads=128, q_stride=128 * 64, k_stride=128 * 64, v_stride=128 * 64, o_stride=128 * 64), L.LORA_E_UNSUPPORTED, b"one launch")]
    for kw, kind, word in shapes:
        s = mk(**kw)
        assert lib.attention_workspace_bytes(ctypes.byref(s)) == 0
        _is(L, fwd(s=s), kind, word)
        _is(L, bwd(s=s), kind, word)
    _is(L, lib.attention_forward(None, P, P, P, P, P, P, P, P, BIG, None), E, b"NULL")
    for k in ("q", "k", "v", "cq", "ck", "o", "lse"):
        _is(L, fwd(**{k: None}), E, b"non-NULL")
    for k in ("do", "q", "k", "v", "o", "lse", "cq", "ck", "dq", "dk", "dv"):
        _is(L, bwd(**{k: None}), E, b"non-NULL")
    for k in ("q", "k", "v", "o", "ws"):
        _is(L, fwd(**{k: ODD}), E, b"aligned")
    for k in ("do", "q", "k", "v", "o", "dq", "dk", "dv", "ws"):
        _is(L, bwd(**{k: ODD}), E, b"aligned")
    odd4 = ctypes.c_void_p((12 << 20) + 2)
    for f in (fwd, bwd):
        for k in ("lse", "cq", "ck"):
            _is(L, f(**{k: odd4}), E, b"4-byte aligned")
        _is(L, f(ws=None), L.LORA_E_WORKSPACE)
        _is(L, f(nb=need - 1), L.LORA_E_WORKSPACE)
    for k in ("q", "k", "v"):
        _is(L, fwd(**{k: at(4)}), E, b"overlaps")
    for own, out in ((6, "dq"), (7, "dk"), (8, "dv")):
        for n in range(1, 9):
            if n != own:
                _is(L, bwd(**{out: at(n)}), E, b"overlap")
    for k in ("lse", "ws"):
        for n in (1, 2, 3, 4):
            _is(L, fwd(**{k: at(n)}), E, b"overlaps")
        _is(L, fwd(**{k: P}), E, b"overlaps")
    _is(L, fwd(lse=at(11)), E, b"overlaps")
    for n in range(1, 9):
        _is(L, bwd(ws=at(n)), E, b"overlaps")
        if n >= 6:
            _is(L, bwd(lse=at(n)), E, b"overlap")
            _is(L, bwd(cq=at(n)), E, b"overlap")
    # slices of one buffer lie between one another: taken; a slice too far: refused
    row = 8 * 64
    s = mk(n_k=100, q_stride=row, k_stride=row, v_stride=row)
    sl = lambda base, head: ctypes.c_void_p((base << 20) + 2 * 64 * head)  # noqa: E731
    ok = dict(q=sl(1, 0), k=sl(1, 4), v=sl(1, 6), dq=sl(3, 0), dk=sl(3, 4), dv=sl(3, 6))
    none = mk(n_k=100, q_stride=row, k_stride=row, v_stride=row, n_seqs=0)     # past every check, nothing to do
    assert bwd(s=none, do=at(8), o=at(9), **ok) == L.LORA_OK
    _is(L, bwd(s=s, do=at(8), o=at(9), **{**ok, "dk": sl(3, 3)}), E, b"overlap")
    _is(L, bwd(s=s, do=at(8), o=at(9), **{**ok, "dv": sl(3, 7)}), E, b"overlap")
    _is(L, bwd(s=s, do=at(8), o=at(9), **{**ok, "dv": sl(1, 6)}), E, b"overlaps an input")
    s = mk(n_q=0, n_k=0)
    assert fwd(s=s, q=None, k=None, v=None, o=None, lse=None) == L.LORA_OK
    assert bwd(s=s, do=None, q=None, k=None, v=None, o=None, lse=None, dq=None, dk=None, dv=None) == L.LORA_OK
    assert fwd(s=mk(n_seqs=0), cq=None, ck=None) == L.LORA_OK


def test_attention_output_on_the_offsets(L):  # noqa: F811
    """cu_q and cu_k are read by every block, so o may not be written over them."""
    s = L.make_attention_shape(100, 120, 3, 4, 2, 64, 0.1)
    for cq, ck in ((at(4), at(9)), (at(9), at(4)), (ctypes.c_void_p((4 << 20) + 2 * 100 * 4 * 64 - 4), at(9))):
        _is(L, L.LIB.attention_forward(ctypes.byref(s), at(1), at(2), at(3), cq, ck, at(4), at(10), at(11), BIG, None), L.LORA_E_INVALID_ARG, b"overlaps")


def _kv(L, **kw):
    return L.make_kv_shape(**{**dict(n_seqs=3, n_kv_heads=2, head_dim=64, page_size=16, n_pages=20, max_pages=4), **kw})


def _bad_kv(L):
    E, U = L.LORA_E_INVALID_ARG, L.LORA_E_UNSUPPORTED
    return [(dict(n_seqs=-1), E), (dict(n_seqs=4097), E), (dict(n_kv_heads=0), E), (dict(n_kv_heads=1025), E), (dict(n_pages=0), E),
            (dict(max_pages=0), E), (dict(head_dim=96), U), (dict(page_size=8), U), (dict(page_size=24), U), (dict(page_size=512), U),
            (dict(n_pages=1 << 27), U), (dict(max_pages=1 << 27), U)]


def test_tables(L):  # noqa: F811
    lib, E = L.LIB, L.LORA_E_INVALID_ARG

    def call(s=None, c=at(20), n=at(21), sl=at(1), t=at(2), r=at(3), st=at(22), so=at(4), cu=at(5), ns=10, slots=at(6), pos=at(7), seq=at(8),
             ws=at(9), nb=BIG):
        return lib.kv_tables(ctypes.byref(s or _kv(L)), c, n, sl, t, r, st, so, cu, ns, slots, pos, seq, ws, nb, None)

    for kw, kind in _bad_kv(L):
        assert lib.kv_tables_workspace_bytes(ctypes.byref(_kv(L, **kw))) == 0
        _is(L, call(s=_kv(L, **kw)), kind)
    for k in ("c", "n", "sl", "t", "r", "st", "so", "slots"):
        _is(L, call(**{k: None}), E, b"non-NULL")
    odd4 = ctypes.c_void_p(66)
    for k in ("c", "n", "sl", "t", "r", "cu", "slots", "pos", "seq"):
        _is(L, call(**{k: odd4}), E, b"aligned")
    for k in ("st", "so"):
        _is(L, call(**{k: ctypes.c_void_p(68)}), E, b"aligned")
    _is(L, call(ns=-1), E, b"n_slots")
    _is(L, call(ns=1 << 30), E, b"n_slots")
    for k in ("sl", "t", "r", "so", "cu", "slots", "pos", "seq", "ws"):
        for other in (*range(1, 10), 20, 21, 22):
            own = {"sl": (1, 20), "t": (2,), "r": (3,), "so": (4, 22), "cu": (5,), "slots": (6,), "pos": (7,), "seq": (8,), "ws": (9,)}[k]
            if other not in own:
                _is(L, call(**{k: at(other)}), E, b"overlaps")
    _is(L, call(sl=ctypes.c_void_p((20 << 20) + 4)), E, b"overlaps")       # over cached_lens, but not on it
    _is(L, call(so=ctypes.c_void_p((22 << 20) + 8)), E, b"overlaps")
    _is(L, call(ws=None), L.LORA_E_WORKSPACE)
    _is(L, call(nb=255), L.LORA_E_WORKSPACE)
    _is(L, call(ws=ODD), E, b"aligned")


def test_write(L):  # noqa: F811
    lib, E = L.LIB, L.LORA_E_INVALID_ARG

    def call(s=None, n=5, k=at(1), ks=128, v=at(2), vs=128, sl=at(9), kc=at(3), vc=at(4), sk=None, sv=None, ws=at(10), nb=256):
        return lib.kv_write(ctypes.byref(s or _kv(L)), n, k, ks, v, vs, sl, kc, vc, sk, sv, ws, nb, None)

    for kw, kind in _bad_kv(L):
        _is(L, call(s=_kv(L, **kw)), kind)
    for k in ("k", "v", "sl", "kc", "vc"):
        _is(L, call(**{k: None}), E)
    for k in ("k", "v", "kc", "vc", "ws"):
        _is(L, call(**{k: ODD}), E, b"aligned")
    for st in (120, 132, 1 << 31, -128):
        _is(L, call(ks=st), E, b"stride")
        _is(L, call(vs=st), E, b"stride")
    _is(L, call(n=-1), E, b"n ")
    _is(L, call(n=1 << 30), E, b"n ")
    _is(L, call(sk=at(5)), E, b"go together")
    _is(L, call(sk=at(5), sv=ctypes.c_void_p(66)), E, b"4-byte")
    _is(L, call(ws=None), L.LORA_E_WORKSPACE)
    _is(L, call(nb=255), L.LORA_E_WORKSPACE)
    for a, b in (("k", 3), ("k", 4), ("v", 3), ("v", 4)):
        _is(L, call(**{a: at(b)}), E, b"overlaps")
    _is(L, call(vc=at(3)), E, b"caches overlap")
    for n in (1, 2, 3, 4, 9, 10):
        _is(L, call(sk=at(n), sv=at(6)), E, b"overlap")
        _is(L, call(sk=at(6), sv=at(n)), E, b"overlap")
        if n != 10:
            _is(L, call(ws=at(n)), E, b"overlap")
    _is(L, call(sl=at(3)), E, b"overlaps slots")
    assert call(n=0, k=None, v=None, sl=None) == L.LORA_OK


def test_decode(L):  # noqa: F811
    lib, E = L.LIB, L.LORA_E_INVALID_ARG

    def call(s=None, h=4, q=at(1), qs=256, kc=at(2), vc=at(3), sk=None, sv=None, t=at(9), ln=at(10), m=50, sc=0.1, o=at(4), lse=None, ws=at(11), nb=BIG):
        return lib.attention_decode(ctypes.byref(s or _kv(L)), h, q, qs, kc, vc, sk, sv, t, ln, m, sc, o, lse, ws, nb, None)

    size = lambda s=None, h=4, m=50: lib.attention_decode_workspace_bytes(ctypes.byref(s or _kv(L)), h, m)  # noqa: E731
    for kw, kind in _bad_kv(L):
        assert size(s=_kv(L, **kw)) == 0
        _is(L, call(s=_kv(L, **kw)), kind)
    for h in (0, 3, 1026, -2):
        assert size(h=h) == 0
        _is(L, call(h=h), E, b"n_heads")
    for m in (-1, 65):
        assert size(m=m) == 0
        _is(L, call(m=m), E, b"max_len")
    assert size(s=_kv(L, n_seqs=4096, n_kv_heads=1024), h=1024) == 0 and b"one launch" in lib.lora_last_error()
    for k in ("q", "kc", "vc", "t", "ln", "o"):
        _is(L, call(**{k: None}), E)
    for k in ("q", "kc", "vc", "o", "ws"):
        _is(L, call(**{k: ODD}), E, b"aligned")
    for k in ("t", "ln", "lse"):
        _is(L, call(**{k: ctypes.c_void_p(66)}), E, b"aligned")
    for st in (248, 260, 1 << 31):
        _is(L, call(qs=st), E, b"q_stride")
    _is(L, call(sc=float("inf")), E, b"scale")
    _is(L, call(sc=-(2.0 ** 127)), E, b"scale")
    far = _kv(L, page_size=256, max_pages=(1 << 22) + 1)
    assert size(far, m=1 << 30) > 0 and size(far, m=(1 << 30) + 1) == 0
    _is(L, call(s=far, m=(1 << 30) + 1), L.LORA_E_UNSUPPORTED, b"2^30")
    _is(L, call(sk=at(6)), E, b"go together")
    long = _kv(L, max_pages=400)
    need = size(s=long, m=6400)
    # a maximum, a sum and a row of fp32 for each part of a request: two parts at least, where one block does not take it whole
    assert need >= 256 + 3 * 4 * 2 * (8 + 4 * 64) and size() == 256
    _is(L, call(s=long, m=6400, nb=need - 1), L.LORA_E_WORKSPACE)
    _is(L, call(ws=None), L.LORA_E_WORKSPACE)
    _is(L, call(o=at(1)), E, b"overlaps q")
    for k in ("o", "lse", "ws"):
        for n in (2, 3, 9, 10, 4, 11, 6, 7):
            if (k, n) not in (("o", 4), ("ws", 11)):
                _is(L, call(**{"sk": at(6), "sv": at(7), k: at(n)}), E, b"overlaps another")
    assert call(s=_kv(L, n_seqs=0), q=None, o=None, t=None, ln=None) == L.LORA_OK


@pytest.mark.parametrize("bound", [0, 1, 128, 129, 256, 257, 1000, 4096, 4097, 8193, 100000])
def test_decode_workspace_grows_with_the_bound(L, bound):  # noqa: F811
    s = _kv(L, max_pages=10000)
    n = L.attention_decode_workspace_bytes(s, 8, bound)
    parts = min(32, max(1, -(-bound // 256)))     # units of 256 keys, or 32 of them
    assert n == 256 if parts == 1 else n >= 256 + 3 * 8 * parts * (8 + 4 * 64)


@pytest.mark.parametrize("heads,kv", [(8, 8), (32, 8), (40, 1)])
def test_decode_workspace_of_a_large_batch_serves_smaller_ones(L, heads, kv):  # noqa: F811
    """Large batches are cut into fewer parts than small ones; a workspace sized for them serves all."""
    rng = __import__("random").Random(heads)
    mk = lambda n: _kv(L, n_seqs=n, n_kv_heads=kv, max_pages=1000)  # noqa: E731
    for _ in range(60):
        n, m = rng.randint(1, 700), rng.randint(1, 16000)
        have = L.attention_decode_workspace_bytes(mk(n), heads, m)
        assert have >= L.attention_decode_workspace_bytes(mk(rng.randint(1, n)), heads, rng.randint(0, m))


def _parts(L, n, heads, kv, m):
    """How many parts a call cuts a request of the bound's length into, from the workspace that it asks for."""
    s = _kv(L, n_seqs=n, n_kv_heads=kv, max_pages=2000)
    st = L.LIB.attention_decode(ctypes.byref(s), heads, at(1), heads * 64, at(2000), at(4000), None, None, at(6000), at(6500), m, 0.1, at(7000), None,
                                at(8000), 0, None)
    _is(L, st, L.LORA_E_WORKSPACE)
    need = int(L.LIB.lora_last_error().split(b"< ")[1].split()[0])
    if need <= 256:
        return 1
    rows = n * heads
    parts = (need - 256) // (rows * (8 + 4 * 64))
    assert need == 256 + -(-rows * parts * 8 // 256) * 256 + rows * parts * 4 * 64
    return parts


@pytest.mark.parametrize("n,kv,m", [(249, 4, 3000), (250, 4, 3000), (251, 4, 3000), (400, 4, 3000), (800, 2, 3000), (200, 8, 3000), (100, 8, 8000), (64, 8, 8000),
                                    (300, 1, 8000), (4096, 8, 31000)])
def test_decode_cuts_long_requests_of_large_batches_alike(L, n, kv, m):  # noqa: F811
    """A request too long for one block is cut into runs of at most four units of its length (runs of
    eight end a launch on long blocks), and into those wherever the batch is large."""
    assert _parts(L, n, 4 * kv, kv, m) == -(-min(32, -(-m // 256)) // 4)


def test_decode_cuts_follow_the_compute_units(L):  # noqa: F811
    """Longer runs where nine blocks a compute unit (256 of them) are left: on both sides of it."""
    for n, parts in ((191, 6), (192, 3)):      # four key heads, 12 units: 764 and 768 columns of three runs
        assert _parts(L, n, 16, 4, 3000) == parts
    for n, parts in ((63, 6), (64, 1)):        # whole requests of up to eight units from 256 blocks on
        assert _parts(L, n, 16, 4, 1500) == parts


@pytest.mark.parametrize("n,heads,kv,m", [(200, 16, 4, 4000), (77, 8, 8, 20000), (260, 32, 1, 1500), (40, 48, 2, 700), (3, 4, 2, 8192), (1, 4, 4, 257)])
def test_decode_workspace_is_the_most_that_any_smaller_call_asks_for(L, n, heads, kv, m):  # noqa: F811
    """No less than a call of fewer requests or a shorter bound uses, and no more than the largest of them."""
    bound = L.attention_decode_workspace_bytes(_kv(L, n_seqs=n, n_kv_heads=kv, max_pages=2000), heads, m)
    lengths = sorted({min(256 * u, m) for u in range(1, min(32, -(-m // 256)) + 1)} | {m})
    rows = max(b * p for b in range(1, n + 1) for x in lengths if (p := _parts(L, b, heads, kv, x)) > 1) * heads
    assert bound == 256 + -(-rows * 8 // 256) * 256 + rows * 4 * 64


def test_decode_workspace_is_a_quick_question(L):  # noqa: F811
    """A caller may ask at every step: microseconds, however many requests there are."""
    s = _kv(L, n_seqs=4096, n_kv_heads=8, max_pages=2000)
    began = time.perf_counter()
    for i in range(500):
        L.attention_decode_workspace_bytes(s, 32, 31000 + i)
    assert time.perf_counter() - began < 1.0
