"""ctypes binding of liblora_mi355x.so (include/lora_mi355x.h).

Argument marshalling only: every function below forwards torch tensors'
device pointers, sizes and the current HIP stream to the C entry point of the
same name and raises LoraError on a non-zero status.  All computation runs in
the library's gfx950 kernels; there is no fallback path.  If the library is
missing the import of this module raises, loudly.  LORA_MI355X_LIB, when set,
names another build of the same library to load instead (the host-sanitizer
build of `python -m rl_lora_linear_amd.build --host-asan`).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("LORA_MI355X_LIB") or os.path.join(_HERE, "liblora_mi355x.so")

# status codes and flags (include/lora_mi355x.h)
LORA_OK, LORA_E_INVALID_ARG, LORA_E_UNSUPPORTED, LORA_E_WORKSPACE, LORA_E_HIP, LORA_E_DEVICE_CHECK = range(6)
FLAG_ID_RANGE, FLAG_UNSORTED, FLAG_TARGET_RANGE, FLAG_BAD_DESC = 0x1, 0x2, 0x4, 0x8
FLAG_NONFINITE_GRAD, FLAG_NONFINITE_LOSS = 0x10, 0x20
IDS_SORTED, IDS_INTERLEAVED = 0, 1
LOSS_CROSS_ENTROPY, LOSS_IMPORTANCE_SAMPLING, LOSS_PPO, LOSS_CUSTOM = range(4)
TIMER_BASE_GEMM, TIMER_LOGPROB_FWD, TIMER_LOGPROB_BWD, TIMER_SHRINK, TIMER_EXPAND, TIMER_GRAD, TIMER_ADAM = range(7)

EXPORTS = [
    "lora_workspace_bytes", "lora_workspace_init", "lora_device_status", "lora_last_error",
    "lora_segments_workspace_bytes", "lora_segments", "lora_transpose_bf16", "lora_forward",
    "lora_backward", "token_logprobs_workspace_bytes", "token_logprobs",
    "token_logprobs_backward_workspace_bytes", "token_logprobs_backward",
    "loss_grad_workspace_bytes", "loss_grad", "adam_workspace_bytes", "adam_step",
    "adam_step_multi", "swiglu_forward",
    "swiglu_backward", "bf16_add", "moe_route", "moe_workspace_bytes", "moe_saved_bytes", "moe_forward",
    "moe_backward", "mlp_workspace_bytes", "mlp_saved_bytes", "mlp_forward", "mlp_backward",
    "lora_timing_enable", "lora_timing_reset", "lora_timing_read",
    "lora_forward_noalloc_scratch_bytes", "lora_forward_noalloc",
    "rmsnorm_forward", "rmsnorm_forward_q8", "rmsnorm_backward_workspace_bytes", "rmsnorm_backward",
    "w4_quantize", "w4_linear", "lora_forward_w4_workspace_bytes", "lora_forward_w4",
    "grad_workspace_bytes", "grad_norm", "grad_clip", "adam_step_clipped",
    "lora_probe_mfma_flops_per_iter", "lora_probe_mfma", "lora_probe_copy", "lora_probe_read",
]


class LoraError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


class LoraShape(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("a_pack_elems", ctypes.c_int64), ("b_pack_elems", ctypes.c_int64),
                ("n_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("order", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoeShape(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("d_ff", ctypes.c_int64),
                ("gate_pack_elems", ctypes.c_int64), ("up_pack_elems", ctypes.c_int64),
                ("down_pack_elems", ctypes.c_int64), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_adapters", ctypes.c_int32),
                ("max_rank", ctypes.c_int32)]


class MlpShape(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("d_ff", ctypes.c_int64),
                ("gate_pack_elems", ctypes.c_int64), ("up_pack_elems", ctypes.c_int64),
                ("down_pack_elems", ctypes.c_int64), ("n_adapters", ctypes.c_int32),
                ("max_rank", ctypes.c_int32)]


class AdamSegment(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("count", ctypes.c_int64), ("step", ctypes.c_int64)]


class LossConfig(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float)]


class GradShape(ctypes.Structure):
    _fields_ = [("n_elems", ctypes.c_int64), ("n_chunks", ctypes.c_int32),
                ("n_tensors", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


W4_MAX_TOKENS = 256
GRAD_CHUNK = 8192
GRAD_DTYPE = np.dtype([("offset", "<i8"), ("count", "<i8"), ("group", "<i4"), ("first_chunk", "<i4")])
DESC_DTYPE = np.dtype([("a_off", "<i8"), ("b_off", "<i8"), ("rank", "<i4"), ("scale", "<f4")])
DESC_BYTES = GRAD_TENSOR_BYTES = 24
assert DESC_DTYPE.itemsize == DESC_BYTES and GRAD_DTYPE.itemsize == GRAD_TENSOR_BYTES

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F = ctypes.c_float
_D = ctypes.c_double
_SZ = ctypes.c_size_t


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m rl_lora_linear_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "lora_workspace_bytes": (_SZ, [ctypes.POINTER(LoraShape)]),
        "lora_workspace_init": (_I32, [_P, _SZ, _P]),
        "lora_device_status": (_I32, [_P, ctypes.POINTER(_I32), _P]),
        "lora_last_error": (ctypes.c_char_p, []),
        "lora_segments_workspace_bytes": (_SZ, [_I64, _I32]),
        "lora_segments": (_I32, [_P, _I64, _I32, _I32, _P, _P, _P, _SZ, _P]),
        "lora_transpose_bf16": (_I32, [_P, _P, _I64, _I64, _P]),
        "lora_forward": (_I32, [ctypes.POINTER(LoraShape), _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "lora_backward": (_I32, [ctypes.POINTER(LoraShape), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _I32, _P, _SZ, _P]),
        "token_logprobs_workspace_bytes": (_SZ, [_I64, _I64]),
        "token_logprobs": (_I32, [_I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "token_logprobs_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
        "token_logprobs_backward": (_I32, [_I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "loss_grad_workspace_bytes": (_SZ, [_I64]),
        "loss_grad": (_I32, [_I32, _I64, _P, _P, _P, _P, _P, ctypes.POINTER(LossConfig), _P, _P, _P,
                             _SZ, _P]),
        "adam_workspace_bytes": (_SZ, [_I32]),
        "adam_step": (_I32, [_I64, _P, _P, _P, _P, _I64, _F, _F, _F, _F, _F, _P, _P, _SZ, _P]),
        "adam_step_multi": (_I32, [_I32, ctypes.POINTER(AdamSegment), _P, _P, _P, _P, _F, _F, _F, _F,
                                   _F, _P, _P, _SZ, _P]),
        "swiglu_forward": (_I32, [_I64, _P, _P, _P, _P]),
        "bf16_add": (_I32, [_I64, _P, _P, _P, _P]),
        "moe_route": (_I32, [_I64, _I32, _I32, _P, _P, _P, _P]),
        "moe_workspace_bytes": (_SZ, [ctypes.POINTER(MoeShape)]),
        "moe_saved_bytes": (_SZ, [ctypes.POINTER(MoeShape)]),
        "moe_forward": (_I32, [ctypes.POINTER(MoeShape)] + [_P] * 16 + [_SZ, _P]),
        "moe_backward": (_I32, [ctypes.POINTER(MoeShape)] + [_P] * 19 + [_I32, _P, _P, _SZ, _P]),
        "mlp_workspace_bytes": (_SZ, [ctypes.POINTER(MlpShape)]),
        "mlp_saved_bytes": (_SZ, [ctypes.POINTER(MlpShape)]),
        "mlp_forward": (_I32, [ctypes.POINTER(MlpShape)] + [_P] * 14 + [_SZ, _P]),
        "mlp_backward": (_I32, [ctypes.POINTER(MlpShape)] + [_P] * 17 + [_I32, _P, _P, _SZ, _P]),
        "swiglu_backward": (_I32, [_I64, _P, _P, _P, _P, _P, _P]),
        "lora_forward_noalloc_scratch_bytes": (_SZ, []),
        "lora_forward_noalloc": (_I32, [ctypes.POINTER(LoraShape), _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _P]),
        "rmsnorm_forward": (_I32, [_I64, _I64, _P, _P, _P, _F, _P, _P, _P, _P]),
        "rmsnorm_forward_q8": (_I32, [_I64, _I64, _P, _P, _P, _F, _P, _P, _P, _P, _P]),
        "rmsnorm_backward_workspace_bytes": (_SZ, [_I64, _I64]),
        "rmsnorm_backward": (_I32, [_I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _SZ, _P]),
        "w4_quantize": (_I32, [_P, _I64, _I64, _P, _P, _P]),
        "w4_linear": (_I32, [_I64, _I64, _I64, _P, _P, _P, _P, _P, _P]),
        "lora_forward_w4_workspace_bytes": (_SZ, [ctypes.POINTER(LoraShape)]),
        "lora_forward_w4": (_I32, [ctypes.POINTER(LoraShape)] + [_P] * 10 + [_SZ, _P]),
        "grad_workspace_bytes": (_SZ, [ctypes.POINTER(GradShape)]),
        "grad_norm": (_I32, [ctypes.POINTER(GradShape), _P, _P, _P, _P, _SZ, _P]),
        "grad_clip": (_I32, [ctypes.POINTER(GradShape), _P, _P, _F, _P, _P, _P, _SZ, _P]),
        "adam_step_clipped": (_I32, [ctypes.POINTER(GradShape), _P, _P, _P, _P, _P, _P, _F] + [_D] * 5 +
                              [_P, _P, _P, _SZ, _P]),
        "lora_probe_mfma_flops_per_iter": (_I64, [_I32]),
        "lora_probe_mfma": (_I32, [_I64, _I32, _P, _P]),
        "lora_probe_copy": (_I32, [_P, _P, _I64, _P]),
        "lora_probe_read": (_I32, [_P, _I64, _P, _P]),
        "lora_timing_enable": (None, [_I32]),
        "lora_timing_reset": (None, []),
        "lora_timing_read": (_I32, [_I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I64)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def _check(st: int):
    if st != LORA_OK:
        raise LoraError(st, LIB.lora_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------------ helpers
def make_shape(n_tokens, d_in, d_out, a_pack_elems, b_pack_elems, n_adapters, max_rank,
               order=IDS_SORTED) -> LoraShape:
    return LoraShape(n_tokens, d_in, d_out, a_pack_elems, b_pack_elems, n_adapters, max_rank, order, 0)


def make_desc(a_off, b_off, ranks, scales, device="cuda") -> torch.Tensor:
    """Device descriptor table (24-byte records) as a uint8 tensor."""
    d = np.zeros(len(ranks), DESC_DTYPE)
    d["a_off"], d["b_off"], d["rank"], d["scale"] = a_off, b_off, ranks, scales
    return torch.from_numpy(d.view(np.uint8).copy()).to(device)


def empty_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace (its status word starts cleared)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ C entry points
def lora_workspace_bytes(shape: LoraShape) -> int:
    n = LIB.lora_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def lora_workspace_init(ws: torch.Tensor, stream=None):
    _check(LIB.lora_workspace_init(_ptr(ws), _nbytes(ws), _stream(stream)))


def lora_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise, read and clear the workspace status word; returns the flags
    (does not raise on content errors)."""
    flags = _I32(0)
    st = LIB.lora_device_status(_ptr(ws), ctypes.byref(flags), _stream(stream))
    if st not in (LORA_OK, LORA_E_DEVICE_CHECK):
        _check(st)
    return flags.value


def lora_segments_workspace_bytes(n: int, n_keys: int) -> int:
    return LIB.lora_segments_workspace_bytes(n, n_keys)


def lora_segments(ids, n_keys, order, perm, offsets, ws, stream=None):
    _check(LIB.lora_segments(_ptr(ids), ids.numel(), n_keys, order, _ptr(perm), _ptr(offsets),
                             _ptr(ws), _nbytes(ws), _stream(stream)))


def lora_transpose_bf16(src, dst, stream=None):
    rows, cols = src.shape
    _check(LIB.lora_transpose_bf16(_ptr(src), _ptr(dst), rows, cols, _stream(stream)))


def lora_forward(shape, x, W, A_pack, B_pack, desc, ids, y, u_saved, ws, stream=None):
    _check(LIB.lora_forward(ctypes.byref(shape), _ptr(x), _ptr(W), _ptr(A_pack), _ptr(B_pack),
                            _ptr(desc), _ptr(ids), _ptr(y), _ptr(u_saved), _ptr(ws), _nbytes(ws),
                            _stream(stream)))


def lora_forward_noalloc_scratch_bytes() -> int:
    return LIB.lora_forward_noalloc_scratch_bytes()


def lora_forward_noalloc(shape, x, W, A_pack, B_pack, desc, ids, y, u_saved, status=None,
                         stream=None):
    """lora_forward on the library's fixed scratch array (no workspace); status:
    optional device int32 tensor the call's flags are OR-ed into."""
    _check(LIB.lora_forward_noalloc(ctypes.byref(shape), _ptr(x), _ptr(W), _ptr(A_pack),
                                    _ptr(B_pack), _ptr(desc), _ptr(ids), _ptr(y), _ptr(u_saved),
                                    _ptr(status), _stream(stream)))


def lora_backward(shape, dy, x, W_t, A_pack, B_pack, desc, ids, u_saved, dx, dA_pack, dB_pack,
                  accumulate, ws, stream=None):
    _check(LIB.lora_backward(ctypes.byref(shape), _ptr(dy), _ptr(x), _ptr(W_t), _ptr(A_pack),
                             _ptr(B_pack), _ptr(desc), _ptr(ids), _ptr(u_saved), _ptr(dx),
                             _ptr(dA_pack), _ptr(dB_pack), int(accumulate), _ptr(ws), _nbytes(ws),
                             _stream(stream)))


def token_logprobs_workspace_bytes(n, vocab) -> int:
    return LIB.token_logprobs_workspace_bytes(n, vocab)


def token_logprobs(h, lm_head, targets, logprobs, lse, ws, stream=None):
    n, hidden = h.shape
    vocab = lm_head.shape[0]
    _check(LIB.token_logprobs(n, hidden, vocab, _ptr(h), _ptr(lm_head), _ptr(targets),
                              _ptr(logprobs), _ptr(lse), _ptr(ws), _nbytes(ws), _stream(stream)))


def token_logprobs_backward_workspace_bytes(n, vocab, chunk_rows) -> int:
    return LIB.token_logprobs_backward_workspace_bytes(n, vocab, chunk_rows)


def token_logprobs_backward(h, lm_head, lm_head_t, targets, lse, dlogp, dh, ws, stream=None):
    n, hidden = h.shape
    vocab = lm_head.shape[0]
    _check(LIB.token_logprobs_backward(n, hidden, vocab, _ptr(h), _ptr(lm_head), _ptr(lm_head_t),
                                       _ptr(targets), _ptr(lse), _ptr(dlogp), _ptr(dh), _ptr(ws),
                                       _nbytes(ws), _stream(stream)))


def loss_grad_workspace_bytes(n) -> int:
    return LIB.loss_grad_workspace_bytes(n)


def loss_grad(kind, logprobs, weights, advantages, sampler_logprobs, custom_g, clip, loss_out,
              dlogp, ws, stream=None):
    cfg = LossConfig(*clip) if clip is not None else None
    _check(LIB.loss_grad(kind, logprobs.numel(), _ptr(logprobs), _ptr(weights), _ptr(advantages),
                         _ptr(sampler_logprobs), _ptr(custom_g),
                         ctypes.byref(cfg) if cfg is not None else None, _ptr(loss_out), _ptr(dlogp),
                         _ptr(ws), _nbytes(ws), _stream(stream)))


def adam_workspace_bytes(n_seg: int) -> int:
    return LIB.adam_workspace_bytes(n_seg)


def adam_skip_flags(ws: torch.Tensor, n_seg: int) -> np.ndarray:
    """Per-segment skip flags of the latest AdamW call on this workspace
    (int32 at byte 256 + 4 i: 1 = skipped, 0 = stepped); synchronises."""
    torch.cuda.synchronize()
    return ws[256:256 + 4 * n_seg].cpu().numpy().view(np.int32).copy()


def adam_step(p, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
              p_bf16=None, ws=None, stream=None):
    """ws: workspace of adam_workspace_bytes(1) (a fresh zeroed one if None).
    A gradient holding NaN or Inf skips the whole step and sets
    FLAG_NONFINITE_GRAD in the workspace status word."""
    if ws is None:
        ws = empty_workspace(adam_workspace_bytes(1), device=p.device)
    _check(LIB.adam_step(p.numel(), _ptr(p), _ptr(g), _ptr(m), _ptr(v), int(step), lr, beta1,
                         beta2, eps, weight_decay, _ptr(p_bf16), _ptr(ws), _nbytes(ws),
                         _stream(stream)))
    return ws


def adam_step_multi(segments, p, g, m, v, lr, beta1=0.9, beta2=0.999, eps=1e-8,
                    weight_decay=0.0, p_bf16=None, ws=None, stream=None):
    """segments: list of (offset, count, step) into the flat p/g/m/v buffers.
    ws: workspace of adam_workspace_bytes(len(segments)) (fresh if None)."""
    n = p.numel()
    for t in (g, m, v):
        if t.numel() != n:
            raise LoraError(LORA_E_INVALID_ARG, "p, g, m, v must have the same length")
    if p_bf16 is not None and p_bf16.numel() != n:
        raise LoraError(LORA_E_INVALID_ARG, "p_bf16 must have the length of p")
    for o, c, _ in segments:
        if o < 0 or c < 0 or o + c > n:
            raise LoraError(LORA_E_INVALID_ARG, f"segment ({o}, {c}) outside a buffer of {n}")
    if ws is None:
        ws = empty_workspace(adam_workspace_bytes(len(segments)), device=p.device)
    arr = (AdamSegment * max(1, len(segments)))(*[AdamSegment(int(o), int(c), int(t)) for o, c, t in segments])
    _check(LIB.adam_step_multi(len(segments), arr, _ptr(p), _ptr(g), _ptr(m), _ptr(v), lr, beta1,
                               beta2, eps, weight_decay, _ptr(p_bf16), _ptr(ws), _nbytes(ws),
                               _stream(stream)))
    return ws


def bf16_add(a, b, out, stream=None):
    _check(LIB.bf16_add(a.numel(), _ptr(a), _ptr(b), _ptr(out), _stream(stream)))


def moe_route(logits, top_k, experts, weights, stream=None):
    n, E = logits.shape
    _check(LIB.moe_route(n, E, top_k, _ptr(logits), _ptr(experts), _ptr(weights), _stream(stream)))


def moe_workspace_bytes(shape: MoeShape) -> int:
    n = LIB.moe_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def moe_saved_bytes(shape: MoeShape) -> int:
    n = LIB.moe_saved_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def moe_forward(shape, x, experts, weights, ids, W_gate, W_up, W_down, packs, descs, y, saved, ws,
                stream=None):
    """packs, descs: (gate, up, down) triples."""
    _check(LIB.moe_forward(ctypes.byref(shape), _ptr(x), _ptr(experts), _ptr(weights), _ptr(ids),
                           _ptr(W_gate), _ptr(W_up), _ptr(W_down), *[_ptr(p) for p in packs],
                           *[_ptr(d) for d in descs], _ptr(y), _ptr(saved), _ptr(ws), _nbytes(ws),
                           _stream(stream)))


def moe_backward(shape, dy, x, experts, weights, ids, W_gate_t, W_up_t, W_down_t, packs, descs,
                 saved, dx, grads, accumulate, ws, trace=None, stream=None):
    """packs, descs, grads: (gate, up, down) triples; trace: optional bf16 [3][N*K][F]."""
    _check(LIB.moe_backward(ctypes.byref(shape), _ptr(dy), _ptr(x), _ptr(experts), _ptr(weights),
                            _ptr(ids), _ptr(W_gate_t), _ptr(W_up_t), _ptr(W_down_t),
                            *[_ptr(p) for p in packs], *[_ptr(d) for d in descs], _ptr(saved),
                            _ptr(dx), *[_ptr(g) for g in grads], int(accumulate), _ptr(trace),
                            _ptr(ws), _nbytes(ws), _stream(stream)))


def mlp_workspace_bytes(shape: MlpShape) -> int:
    n = LIB.mlp_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def mlp_saved_bytes(shape: MlpShape) -> int:
    n = LIB.mlp_saved_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def mlp_forward(shape, x, ids, W_gate, W_up, W_down, packs, descs, y, saved, ws, stream=None):
    """packs, descs: (gate, up, down) triples."""
    _check(LIB.mlp_forward(ctypes.byref(shape), _ptr(x), _ptr(ids), _ptr(W_gate), _ptr(W_up),
                           _ptr(W_down), *[_ptr(p) for p in packs], *[_ptr(d) for d in descs],
                           _ptr(y), _ptr(saved), _ptr(ws), _nbytes(ws), _stream(stream)))


def mlp_backward(shape, dy, x, ids, W_gate_t, W_up_t, W_down_t, packs, descs, saved, dx, grads,
                 accumulate, ws, trace=None, stream=None):
    """packs, descs, grads: (gate, up, down) triples; trace: optional bf16 [3 * N * F]."""
    _check(LIB.mlp_backward(ctypes.byref(shape), _ptr(dy), _ptr(x), _ptr(ids), _ptr(W_gate_t),
                            _ptr(W_up_t), _ptr(W_down_t), *[_ptr(p) for p in packs],
                            *[_ptr(d) for d in descs], _ptr(saved), _ptr(dx),
                            *[_ptr(g) for g in grads], int(accumulate), _ptr(trace), _ptr(ws),
                            _nbytes(ws), _stream(stream)))


def swiglu_forward(gate, up, h, stream=None):
    _check(LIB.swiglu_forward(gate.numel(), _ptr(gate), _ptr(up), _ptr(h), _stream(stream)))


def swiglu_backward(dh, gate, up, dgate, dup, stream=None):
    _check(LIB.swiglu_backward(gate.numel(), _ptr(dh), _ptr(gate), _ptr(up), _ptr(dgate), _ptr(dup),
                               _stream(stream)))


def _arg(cond, msg):
    if not cond:
        raise LoraError(LORA_E_INVALID_ARG, msg)


def _on_device(t: torch.Tensor, name: str, dev: int):
    at = t.get_device()
    if at < 0:
        raise LoraError(LORA_E_INVALID_ARG, f"{name}: needs a device tensor")
    if at != dev and dev >= 0:   # (an operand of device -1 has its own refusal)
        raise LoraError(LORA_E_INVALID_ARG, f"{name}: on device {at}, the other operands on {dev}")


def _dense(t: Optional[torch.Tensor], dtypes, shape, name: str, dev: int):
    """Checks one operand of the calls below, which lie on device dev, and returns its
    pointer (None for None)."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise LoraError(LORA_E_INVALID_ARG, f"{name}: needs a contiguous {' or '.join(map(str, dtypes))} "
                        f"tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev or dev < 0:
        _on_device(t, name, dev)
    return t.data_ptr()


def _device_ptr(t: torch.Tensor, name: str, dev: int):
    """The pointer of an operand whose shape the library checks itself."""
    if t.get_device() != dev or dev < 0:
        _on_device(t, name, dev)
    if not t.is_contiguous():
        raise LoraError(LORA_E_INVALID_ARG, f"{name}: needs a contiguous device tensor")
    return t.data_ptr()


def _stream_for(t: torch.Tensor, stream=None):
    """The stream to enqueue on (the current one if None); t must lie on the current device,
    which is where the library launches."""
    dev = torch._C._cuda_getDevice()
    if t.get_device() != dev or (stream is not None and stream.device_index != dev):
        raise LoraError(LORA_E_INVALID_ARG, f"the tensors are on {t.device}, the stream on "
                        f"{dev if stream is None else stream.device}, the current device is {dev}")
    # the raw handle: building a torch.cuda.Stream costs 2.7 us, as much as a launch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_BF16, _F32, _I64T, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int64,), (torch.uint8,)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_E8M0 = (torch.uint8, torch.float8_e8m0fnu)


def _norm_args(x, weight, rstd, residual, h):
    _arg(x.dim() == 2, "x must be [n][hidden]")
    n, hidden = x.shape
    dev = x.get_device()
    return n, hidden, dev, (_dense(x, _BF16, x.shape, "x", dev),
                            _dense(residual, _BF16, x.shape, "residual", dev),
                            _dense(weight, _BF16, (hidden,), "weight", dev),
                            _dense(h, _BF16, x.shape, "h", dev), _dense(rstd, _F32, (n,), "rstd", dev))


def rmsnorm_forward(x, weight, eps, y, rstd=None, residual=None, h=None, stream=None):
    """y = norm(x + residual) weight; h receives x + residual (given exactly with residual)."""
    n, hidden, dev, (px, pr, pw, ph, ps) = _norm_args(x, weight, rstd, residual, h)
    _check(LIB.rmsnorm_forward(n, hidden, px, pr, pw, eps, ph, _dense(y, _BF16, x.shape, "y", dev), ps,
                               _stream_for(x, stream)))


def rmsnorm_forward_q8(x, weight, eps, q, q_scales, rstd=None, residual=None, h=None, stream=None):
    """q: e4m3 codes [n][hidden] (uint8 or float8_e4m3fn); q_scales: E8M0 [n][hidden/32]."""
    n, hidden, dev, (px, pr, pw, ph, ps) = _norm_args(x, weight, rstd, residual, h)
    _check(LIB.rmsnorm_forward_q8(n, hidden, px, pr, pw, eps, ph, _dense(q, _E4M3, x.shape, "q", dev),
                                  _dense(q_scales, _E8M0, (n, hidden // 32), "q_scales", dev), ps,
                                  _stream_for(x, stream)))


def rmsnorm_backward_workspace_bytes(n, hidden) -> int:
    return LIB.rmsnorm_backward_workspace_bytes(n, hidden)


def rmsnorm_backward(dy, h, weight, rstd, dx, dh=None, dweight=None, accumulate=False, ws=None,
                     stream=None):
    """dweight (with ws of rmsnorm_backward_workspace_bytes) is optional: a frozen weight has none."""
    _arg(dy.dim() == 2, "dy must be [n][hidden]")
    n, hidden = dy.shape
    dev = dy.get_device()
    _check(LIB.rmsnorm_backward(n, hidden, _dense(dy, _BF16, dy.shape, "dy", dev),
                                _dense(dh, _BF16, dy.shape, "dh", dev), _dense(h, _BF16, dy.shape, "h", dev),
                                _dense(weight, _BF16, (hidden,), "weight", dev),
                                _dense(rstd, _F32, (n,), "rstd", dev), _dense(dx, _BF16, dy.shape, "dx", dev),
                                _dense(dweight, _F32, (hidden,), "dweight", dev), int(accumulate),
                                None if ws is None else _device_ptr(ws, "ws", dev), 0 if ws is None else ws.nbytes,
                                _stream_for(dy, stream)))


def w4_quantize(W, codes, scales, stream=None):
    """W bf16 [d_out][d_in] -> codes uint8 [d_out][d_in/2], scales uint8 [d_out][d_in/32]."""
    _arg(W.dim() == 2, "W must be [d_out][d_in]")
    d_out, d_in = W.shape
    dev = W.get_device()
    _check(LIB.w4_quantize(_dense(W, _BF16, W.shape, "W", dev), d_out, d_in,
                           _dense(codes, _U8, (d_out, d_in // 2), "codes", dev),
                           _dense(scales, _E8M0, (d_out, d_in // 32), "scales", dev), _stream_for(W, stream)))


def _w4_args(n, d_in, d_out, x, x_scales, codes, scales, y):
    dev = codes.get_device()
    return (_dense(x, _BF16 if x_scales is None else _E4M3, (n, d_in), "x", dev),
            _dense(x_scales, _E8M0, (n, d_in // 32), "x_scales", dev),
            _dense(codes, _U8, (d_out, d_in // 2), "codes", dev),
            _dense(scales, _E8M0, (d_out, d_in // 32), "scales", dev), _dense(y, _BF16, (n, d_out), "y", dev))


def w4_linear(x, codes, scales, y, x_scales=None, stream=None):
    """y = x W^T with 4-bit W; x bf16, or e4m3 codes with their x_scales."""
    _arg(x.dim() == 2 and codes.dim() == 2, "x must be [n][d_in] and codes [d_out][d_in/2]")
    n, d_in = x.shape
    d_out = codes.shape[0]
    px, pxs, pc, ps, py = _w4_args(n, d_in, d_out, x, x_scales, codes, scales, y)
    _check(LIB.w4_linear(n, d_in, d_out, px, pxs, pc, ps, py, _stream_for(codes, stream)))


def lora_forward_w4_workspace_bytes(shape: LoraShape) -> int:
    n = LIB.lora_forward_w4_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def lora_forward_w4(shape, x, codes, scales, A_pack, B_pack, desc, ids, y, ws, x_scales=None,
                    stream=None):
    """lora_forward on a 4-bit base (see w4_linear for x, codes and the scales)."""
    px, pxs, pc, ps, py = _w4_args(shape.n_tokens, shape.d_in, shape.d_out, x, x_scales, codes, scales, y)
    if A_pack.dtype != torch.bfloat16 or A_pack.numel() < shape.a_pack_elems:
        raise LoraError(LORA_E_INVALID_ARG, f"A_pack: needs {shape.a_pack_elems} bfloat16 elements")
    if B_pack.dtype != torch.bfloat16 or B_pack.numel() < shape.b_pack_elems:
        raise LoraError(LORA_E_INVALID_ARG, f"B_pack: needs {shape.b_pack_elems} bfloat16 elements")
    dev = codes.get_device()
    _arg(desc.nbytes >= shape.n_adapters * DESC_BYTES, "desc is shorter than n_adapters entries")
    _check(LIB.lora_forward_w4(ctypes.byref(shape), px, pxs, pc, ps, _device_ptr(A_pack, "A_pack", dev),
                               _device_ptr(B_pack, "B_pack", dev), _device_ptr(desc, "desc", dev),
                               _dense(ids, (torch.int32,), (shape.n_tokens,), "ids", dev), py,
                               _device_ptr(ws, "ws", dev), ws.nbytes, _stream_for(codes, stream)))


def make_grad_table(tensors, n_groups, n_elems, device="cuda"):
    """tensors: (offset, count, group) triples of one flat buffer of n_elems, in any order.
    Returns the GradShape and the device table (sorted by group) of the calls below."""
    t = np.array([tuple(map(int, e)) for e in tensors], np.int64).reshape(-1, 3)
    _arg(np.all(t[:, :2] >= 0) and np.all(t[:, 0] <= n_elems - t[:, 1]),   # (a sum could wrap)
         f"a tensor lies outside a buffer of {n_elems}")
    _arg(np.all((t[:, 2] >= 0) & (t[:, 2] < n_groups)), f"a group outside [0, {n_groups})")
    by_place = t[np.argsort(t[:, 0], kind="stable")]
    by_place = by_place[by_place[:, 1] > 0]
    _arg(np.all(by_place[:-1, 0] + by_place[:-1, 1] <= by_place[1:, 0]), "tensors overlap")
    t = t[np.argsort(t[:, 2], kind="stable")]
    chunks = -(-t[:, 1] // GRAD_CHUNK)
    _arg(chunks.sum() < 1 << 24, "too many elements for one table")
    d = np.zeros(len(t), GRAD_DTYPE)
    d["offset"], d["count"], d["group"], d["first_chunk"] = t[:, 0], t[:, 1], t[:, 2], np.cumsum(chunks) - chunks
    table = torch.from_numpy(d.view(np.uint8).copy()).to(device)
    return GradShape(int(n_elems), int(chunks.sum()), len(t), int(n_groups), 0), table


def grad_workspace_bytes(shape: GradShape) -> int:
    n = LIB.grad_workspace_bytes(ctypes.byref(shape))
    if n == 0:
        raise LoraError(LORA_E_INVALID_ARG, LIB.lora_last_error().decode())
    return n


def _grad_args(shape, table, flat, norms):
    _arg(table.nbytes >= shape.n_tensors * GRAD_TENSOR_BYTES, "table is shorter than n_tensors entries")
    dev = flat[0][1].get_device()
    ptrs = [_dense(t, _F32, (shape.n_elems,), name, dev) for name, t in flat]
    return (_device_ptr(table, "table", dev), *ptrs, _dense(norms, _F32, (shape.n_groups,), "norms", dev))


def grad_norm(shape, table, g, norms, ws, stream=None):
    """norms[a] = the norm of group a's gradient (shape, table: make_grad_table)."""
    pt, pg, pn = _grad_args(shape, table, (("g", g),), norms)
    dev = g.get_device()
    _check(LIB.grad_norm(ctypes.byref(shape), pt, pg, pn, _device_ptr(ws, "ws", dev), ws.nbytes, _stream_for(g, stream)))


def grad_clip(shape, table, g, max_norm, out, norms, ws, stream=None):
    """out = g scaled to at most max_norm per group; out may be g, norms may be None."""
    pt, pg, po, pn = _grad_args(shape, table, (("g", g), ("out", out)), norms)
    dev = g.get_device()
    _check(LIB.grad_clip(ctypes.byref(shape), pt, pg, max_norm, po, pn, _device_ptr(ws, "ws", dev), ws.nbytes,
                         _stream_for(g, stream)))


def adam_step_clipped(shape, table, steps, p, g, m, v, max_norm, lr, beta1=0.9, beta2=0.999,
                      eps=1e-8, weight_decay=0.0, p_bf16=None, norms=None, ws=None, stream=None):
    """One AdamW step per group on its clipped gradient; steps: device int64 [n_groups], the
    steps made so far (>= 0), counted up by the call.  ws: workspace of grad_workspace_bytes(shape)
    (a fresh zeroed one if None)."""
    pt, pp, pg, pm, pv, pn = _grad_args(shape, table, (("p", p), ("g", g), ("m", m), ("v", v)), norms)
    dev = p.get_device()
    if ws is None:
        with torch.cuda.stream(stream):   # cleared, and later reused, in the call's own order
            ws = empty_workspace(grad_workspace_bytes(shape), device=p.device)
    _check(LIB.adam_step_clipped(ctypes.byref(shape), pt, _dense(steps, _I64T, (shape.n_groups,), "steps", dev),
                                 pp, pg, pm, pv, max_norm, lr, beta1, beta2, eps, weight_decay,
                                 _dense(p_bf16, _BF16, (shape.n_elems,), "p_bf16", dev), pn, _device_ptr(ws, "ws", dev),
                                 ws.nbytes, _stream_for(p, stream)))
    return ws


def lora_probe_mfma(iters, blocks, sink, stream=None):
    """Register-only bf16 MFMA loop; returns its flop count."""
    _check(LIB.lora_probe_mfma(int(iters), int(blocks), _ptr(sink), _stream(stream)))
    return LIB.lora_probe_mfma_flops_per_iter(int(blocks)) * int(iters)


def lora_probe_copy(src, dst, stream=None):
    """Streaming device copy of src's bytes into dst."""
    _check(LIB.lora_probe_copy(_ptr(src), _ptr(dst), _nbytes(src), _stream(stream)))


def lora_probe_read(src, sink, stream=None):
    """Read-only stream over src's bytes (sink: a device int32 tensor)."""
    _check(LIB.lora_probe_read(_ptr(src), _nbytes(src), _ptr(sink), _stream(stream)))


def lora_timing_enable(on: bool):
    LIB.lora_timing_enable(1 if on else 0)


def lora_timing_reset():
    LIB.lora_timing_reset()


def lora_timing_read(timer: int):
    ms = ctypes.c_double(0)
    n = _I64(0)
    _check(LIB.lora_timing_read(timer, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
