"""Host-side refusals of the norm, 4-bit and gradient-norm calls (CPU only: every
call here fails before anything is enqueued, whatever its pointers hold)."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p(64)       # never dereferenced
ODD = ctypes.c_void_p(72)     # not 16-byte aligned
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    from test_abi_host import _ensure_built
    _ensure_built()
    import rl_lora_linear_amd.lib as lib
    return lib


def _is(L, st, kind, word=b""):
    assert st == kind and word in L.LIB.lora_last_error(), (st, L.LIB.lora_last_error())


def test_norm(L):
    lib, E = L.LIB, L.LORA_E_INVALID_ARG
    fwd = lambda n=4, H=64, x=P, r=P, w=P, eps=1e-6, h=ctypes.c_void_p(1 << 20), y=P: lib.rmsnorm_forward(n, H, x, r, w, eps, h, y, None, None)  # noqa: E731
    _is(L, fwd(n=-1), E)
    _is(L, fwd(n=1 << 30), E)
    _is(L, fwd(H=0), E)
    _is(L, fwd(H=32769), L.LORA_E_UNSUPPORTED, b"32768")
    _is(L, fwd(eps=-1.0), E, b"eps")
    _is(L, fwd(eps=float("nan")), E, b"eps")
    _is(L, fwd(x=None), E)
    _is(L, fwd(w=None), E)
    _is(L, fwd(y=None), E)
    _is(L, fwd(h=None), E, b"go together")
    _is(L, fwd(r=None), E, b"go together")
    for k in ("x", "r", "w", "h", "y"):
        _is(L, fwd(**{k: ODD}), E, b"aligned")
    _is(L, fwd(h=P, y=P), E, b"same buffer")
    assert fwd(n=0, x=None, y=None) == L.LORA_OK
    q8 = lambda H=64, q=P, s=P: lib.rmsnorm_forward_q8(4, H, P, None, P, 1e-6, None, q, s, None, None)  # noqa: E731
    _is(L, q8(H=40), L.LORA_E_UNSUPPORTED, b"multiple of 32")
    _is(L, q8(q=None), E)
    _is(L, q8(s=None), E)
    _is(L, q8(q=ODD), E, b"aligned")
    bwd = lambda n=4, H=64, dy=P, dh=P, h=P, w=P, r=P, dx=P, dw=P, ws=P, nb=BIG: lib.rmsnorm_backward(n, H, dy, dh, h, w, r, dx, dw, 0, ws, nb, None)  # noqa: E731
    _is(L, bwd(dy=None), E)
    _is(L, bwd(r=None), E)
    _is(L, bwd(dx=ODD), E, b"aligned")
    _is(L, bwd(H=40000), L.LORA_E_UNSUPPORTED)
    _is(L, bwd(ws=None), L.LORA_E_WORKSPACE)
    _is(L, bwd(ws=ODD), E, b"aligned")
    _is(L, bwd(nb=lib.rmsnorm_backward_workspace_bytes(4, 64) - 1), L.LORA_E_WORKSPACE)
    assert bwd(n=0, dy=None, dh=None, h=None, r=None, dx=None, dw=None, ws=None, nb=0) == L.LORA_OK
    assert lib.rmsnorm_backward_workspace_bytes(-1, 64) == 0 == lib.rmsnorm_backward_workspace_bytes(4, 32769)
    for H in (1, 8, 128, 4096, 32768):
        assert 256 + 4 * H <= lib.rmsnorm_backward_workspace_bytes(1 << 20, H) <= 256 + (1 << 25)


def test_four_bit(L):
    lib, E = L.LIB, L.LORA_E_INVALID_ARG
    lin = lambda n=2, i=128, o=64, x=P, xs=None, c=P, s=P, y=P: lib.w4_linear(n, i, o, x, xs, c, s, y, None)  # noqa: E731
    _is(L, lin(n=-1), E)
    _is(L, lin(n=L.W4_MAX_TOKENS + 1), L.LORA_E_UNSUPPORTED, b"at most 256")
    _is(L, lin(i=96), L.LORA_E_UNSUPPORTED)
    _is(L, lin(o=100), L.LORA_E_UNSUPPORTED)
    _is(L, lin(i=(1 << 20) + 64), L.LORA_E_UNSUPPORTED)
    _is(L, lin(o=0), E)
    for k in ("x", "c", "s", "y"):
        _is(L, lin(**{k: None}), E)
    for k in ("x", "c", "s", "y"):
        _is(L, lin(**{k: ODD}), E, b"aligned")
    assert lin(n=0, x=None, y=None) == L.LORA_OK
    _is(L, lib.w4_quantize(P, 64, 100, P, P, None), L.LORA_E_UNSUPPORTED)
    _is(L, lib.w4_quantize(P, 64, 128, None, P, None), E)
    _is(L, lib.w4_quantize(ODD, 64, 128, P, P, None), E)

    sh = L.make_shape(2, 128, 64, 4096, 4096, 4, 16, L.IDS_INTERLEAVED)
    need = L.lora_forward_w4_workspace_bytes(sh)
    call = lambda s=sh, x=P, c=P, sc=P, A=P, B=P, d=P, ids=P, y=P, ws=P, nb=need: lib.lora_forward_w4(ctypes.byref(s), x, None, c, sc, A, B, d, ids, y, ws, nb, None)  # noqa: E731
    for k in ("x", "c", "sc", "A", "B", "d", "ids", "y"):
        _is(L, call(**{k: None}), E)
    for k in ("x", "c", "sc", "A", "B", "y", "ws"):
        _is(L, call(**{k: ODD}), E, b"aligned")
    _is(L, call(ws=None), L.LORA_E_WORKSPACE)
    _is(L, call(nb=need - 1), L.LORA_E_WORKSPACE)
    many = L.make_shape(257, 128, 64, 4096, 4096, 4, 16)
    _is(L, call(s=many), L.LORA_E_UNSUPPORTED, b"at most")
    assert lib.lora_forward_w4_workspace_bytes(ctypes.byref(many)) == 0
    _is(L, call(s=L.make_shape(2, 128, 64, 4096, 4096, 4, 24)), E, b"max_rank")
    none = L.make_shape(0, 128, 64, 4096, 4096, 4, 16)
    assert call(s=none, x=None, ids=None, y=None) == L.LORA_OK


def test_gradients(L):
    lib, E = L.LIB, L.LORA_E_INVALID_ARG
    G = L.GradShape
    good = G(1000, 2, 2, 1)
    need = L.grad_workspace_bytes(good)
    for bad in (G(-1, 2, 2, 1), G(1000, -1, 2, 1), G(1000, 1 << 24, 2, 1), G(1000, 2, -1, 1), G(1000, 2, 0, 1),
                G(1000, 2, 2, 0), G(1000, 2, 2, 16385), G(1000, 2, 2, 1, 5), G((1 << 42) + 1, 2, 2, 1)):
        assert lib.grad_workspace_bytes(ctypes.byref(bad)) == 0
        _is(L, lib.grad_norm(ctypes.byref(bad), P, P, P, P, BIG, None), E)
        _is(L, lib.grad_clip(ctypes.byref(bad), P, P, 1.0, P, P, P, BIG, None), E)
        _is(L, lib.adam_step_clipped(ctypes.byref(bad), P, P, P, P, P, P, 1.0, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, P, P, BIG, None), E)
    norm = lambda t=P, g=P, n=P, ws=P, nb=need: lib.grad_norm(ctypes.byref(good), t, g, n, ws, nb, None)  # noqa: E731
    for k in ("t", "g", "n"):
        _is(L, norm(**{k: None}), E)
    _is(L, norm(ws=None), L.LORA_E_WORKSPACE)
    _is(L, norm(nb=need - 1), L.LORA_E_WORKSPACE)
    _is(L, norm(ws=ODD), E, b"aligned")
    clip = lambda m=1.0, o=P: lib.grad_clip(ctypes.byref(good), P, P, m, o, P, P, need, None)  # noqa: E731
    _is(L, clip(m=-1.0), E, b"max_norm")
    _is(L, clip(m=float("nan")), E, b"max_norm")
    _is(L, clip(o=None), E)
    adam = lambda st=P, p=P, m=P, v=P, b1=0.9, b2=0.99, mx=1.0: lib.adam_step_clipped(ctypes.byref(good), P, st, p, P, m, v, mx, 1e-3, b1, b2, 1e-8, 0.0, None, P, P, need, None)  # noqa: E731
    for k in ("st", "p", "m", "v"):
        _is(L, adam(**{k: None}), E)
    _is(L, adam(b1=1.0), E, b"betas")
    _is(L, adam(b2=-0.1), E, b"betas")
    _is(L, adam(mx=-0.5), E)


def test_table_builder(L):
    shape, table = L.make_grad_table([(20000, 9000, 1), (0, 8192, 0), (9000, 0, 1), (10000, 8193, 0)], 3, 30000, device="cpu")
    d = table.numpy().view(L.GRAD_DTYPE)
    assert list(d["group"]) == [0, 0, 1, 1] and list(d["offset"]) == [0, 10000, 20000, 9000]
    assert list(d["first_chunk"]) == [0, 1, 3, 5] and shape.n_chunks == 5 and shape.n_tensors == 4
    empty, t0 = L.make_grad_table([], 2, 10, device="cpu")
    assert empty.n_chunks == 0 and t0.numel() == 0
    for bad in ([(0, 11, 0)], [(-1, 3, 0)], [(0, 3, 2)], [(0, 3, -1)], [(0, 5, 0), (4, 2, 1)]):
        with pytest.raises(L.LoraError):
            L.make_grad_table(bad, 2, 10, device="cpu")


def test_binding_checks_tensors(L):
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for args, kw, word in (
            ((x.float(), w, 1e-6, x), {}, "x: needs"), ((x, w, 1e-6, x[:1]), {}, "x: needs a device"), ((torch.zeros(64, 2, dtype=torch.bfloat16).t(), w, 1e-6, x), {}, "x: needs"),
            ((x[0], w, 1e-6, x), {}, "x must be")):
        with pytest.raises(L.LoraError, match=word):
            L.rmsnorm_forward(*args, **kw)
    codes, sc = torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.uint8)
    y = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(L.LoraError, match="x: needs"):      # 8-bit x without its scales
        L.w4_linear(x.to(torch.uint8), codes, sc, y)
    with pytest.raises(L.LoraError, match="x: needs"):      # bf16 x with scales
        L.w4_linear(x, codes, sc, y, x_scales=torch.zeros(2, 2, dtype=torch.uint8))
    shape, table = L.make_grad_table([(0, 10, 0)], 1, 10, device="cpu")
    with pytest.raises(L.LoraError, match="g: needs"):
        L.grad_norm(shape, table, torch.zeros(9), torch.zeros(1), table)
    with pytest.raises(L.LoraError, match="shorter"):
        L.grad_norm(L.GradShape(10, 1, 2, 1), table, torch.zeros(10), torch.zeros(1), table)
    sh = L.make_shape(2, 64, 64, 100, 100, 4, 16)
    pack, desc, ids = torch.zeros(100, dtype=torch.bfloat16), torch.zeros(96, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(L.LoraError, match="x: needs a device"):
        L.lora_forward_w4(sh, x, codes, sc, pack, pack, desc, ids, y, codes)
    with pytest.raises(L.LoraError, match="table: needs|g: needs a device"):
        L.grad_norm(shape, table, torch.zeros(10), torch.zeros(1), table)
    assert np.array_equal(x.float().numpy(), np.zeros((2, 64)))


def test_operands_of_two_devices(L):
    """Checked on the host: stand-ins for tensors that say where they lie."""
    class On:
        def __init__(self, dev, dtype, *shape):
            self.dev, self.dtype, self.shape = dev, dtype, torch.Size(shape)
            self.nbytes = self.shape.numel() * dtype.itemsize

        def get_device(self):
            return self.dev

        def is_contiguous(self):
            return True

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.shape.numel()

        def data_ptr(self):
            assert self.dev == 0
            return 64

    b, f, u = torch.bfloat16, torch.float32, torch.uint8
    x, other = On(0, b, 2, 64), On(1, b, 2, 64)
    w = On(0, b, 64)
    for call in (lambda: L.rmsnorm_forward(x, On(1, b, 64), 1e-6, x), lambda: L.rmsnorm_forward(x, w, 1e-6, other),
                 lambda: L.rmsnorm_backward(x, x, w, On(1, f, 2), x),
                 lambda: L.w4_linear(x, On(1, u, 64, 32), On(1, u, 64, 2), x),
                 lambda: L.grad_norm(L.GradShape(4, 1, 1, 1), On(1, u, 24), On(0, f, 4), On(0, f, 1), On(0, u, 512))):
        with pytest.raises(L.LoraError, match="on device"):
            call()


def test_norm_gradient_in_the_place_of_h(L):
    """dx may be dy or dh; h is read only, also where only a part of it lies under dx."""
    n, H, E = 4, 64, L.LORA_E_INVALID_ARG
    at = lambda byte: ctypes.c_void_p((1 << 20) + byte)  # noqa: E731
    bwd = lambda h, dx: L.LIB.rmsnorm_backward(n, H, P, None, h, P, P, dx, None, 0, None, 0, None)  # noqa: E731
    size = n * H * 2
    for byte in (0, 16, size - 16):
        _is(L, bwd(at(0), at(byte)), E, b"dx overlaps h")
        _is(L, bwd(at(byte), at(0)), E, b"dx overlaps h")


def test_eight_bit_norm_in_the_place_of_its_input(L):
    """q's rows are shorter than x's: no place inside x, residual or h suits them."""
    n, H, E = 4, 64, L.LORA_E_INVALID_ARG
    at = lambda byte: ctypes.c_void_p((1 << 20) + byte)  # noqa: E731
    far = {"x": at(1 << 14), "r": at(2 << 14), "h": at(3 << 14), "q": at(4 << 14), "s": at(5 << 14)}

    def call(**kw):
        a = {**far, **kw}
        return L.LIB.rmsnorm_forward_q8(n, H, a["x"], a["r"], P, 1e-6, a["h"], a["q"], a["s"], None, None)

    for name in ("x", "r", "h"):
        for byte in (0, n * H, 2 * n * H - 16):
            place = ctypes.c_void_p(far[name].value + byte)
            _is(L, call(q=place), E, b"overlaps")
            _is(L, call(s=place), E, b"overlaps")


@pytest.mark.parametrize("byte", [65, 66, 68])
def test_tables_that_are_not_aligned(L, byte):
    """Descriptors and gradient tables cut out of a byte buffer at any place but a multiple of 8."""
    lib, E, at = L.LIB, L.LORA_E_INVALID_ARG, ctypes.c_void_p(byte)
    sh = L.make_shape(2, 128, 64, 4096, 4096, 4, 16, L.IDS_INTERLEAVED)
    _is(L, lib.lora_forward_w4(ctypes.byref(sh), P, None, P, P, P, P, at, P, P, P, BIG, None), E, b"desc must be 8-byte aligned")
    good = L.GradShape(1000, 2, 2, 1)
    _is(L, lib.grad_norm(ctypes.byref(good), at, P, P, P, BIG, None), E, b"table must be 8-byte aligned")
    _is(L, lib.grad_clip(ctypes.byref(good), at, P, 1.0, P, P, P, BIG, None), E, b"table must be 8-byte aligned")
    _is(L, lib.adam_step_clipped(ctypes.byref(good), at, P, P, P, P, P, 1.0, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, P, P, BIG, None), E, b"table must be 8-byte")


@pytest.mark.parametrize("bad", [(1 << 63) - 8, (1 << 62) + (1 << 61)])
def test_table_builder_offsets_near_the_largest_integer(L, bad):
    for entry in ((bad, 100, 0), (100, bad, 0), (bad, bad, 0)):
        with pytest.raises(L.LoraError, match="outside a buffer"):
            L.make_grad_table([entry], 1, 1000, device="cpu")
    with pytest.raises(L.LoraError, match="outside a buffer"):
        L.make_grad_table([(0, 10, 0), (bad, 8, 0)], 1, (1 << 42), device="cpu")


def test_four_bit_outputs_in_the_place_of_inputs(L):
    """Blocks read all of x, or of W, while others write: no output may lie there."""
    lib, E, n, d = L.LIB, L.LORA_E_INVALID_ARG, 2, 128
    at = lambda byte: ctypes.c_void_p((1 << 20) + byte)  # noqa: E731
    sh = L.make_shape(n, d, d, 4096, 4096, 4, 16, L.IDS_INTERLEAVED)
    layer = lambda x, xs, y: lib.lora_forward_w4(ctypes.byref(sh), x, xs, P, P, P, P, P, P, y, P, BIG, None)  # noqa: E731
    linear = lambda x, xs, y: lib.w4_linear(n, d, d, x, xs, P, P, y, None)  # noqa: E731
    far = at(1 << 16)
    for call in (layer, linear):
        for byte in (0, 16, n * d * 2 - 16):
            _is(L, call(at(0), None, at(byte)), E, b"overlaps x")
            _is(L, call(at(byte), None, at(0)), E, b"overlaps x")
        _is(L, call(at(0), far, at(n * d - 16)), E, b"overlaps x")
        _is(L, call(far, at(0), at(0)), E, b"overlaps x")
    for codes, scales in ((at(0), far), (at(d * d * 2 - 16), far), (far, at(d * d * 2 - 1))):
        _is(L, lib.w4_quantize(at(0), d, d, codes, scales, None), E, b"overlap W")
