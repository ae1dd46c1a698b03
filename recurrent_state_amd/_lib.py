"""ctypes binding of libkda (the C ABI declared in include/kda.h).

Argument marshalling only: every function checks that the torch tensors it is
given have the sizes, types, device and contiguity the C ABI expects (the C
side only sees pointers), then passes their device pointers and the current
HIP stream.  All arithmetic happens in the library's HIP kernels.  There is no
fallback: if libkda.so is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import os
import warnings

import torch  # loads the HIP runtime that libkda then shares (same soname)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_BF16, KDA_F32, KDA_E4M3 = 0, 1, 2
VARIANTS = {0: "none", 1: "decode", 2: "verify", 3: "commit", 4: "snapshot", 5: "restore",
            6: "prefill_recurrent", 7: "prefill_chunked", 8: "commit_verify", 9: "verify_varlen",
            10: "commit_verify_varlen", 11: "decode_prep", 12: "verify_prep", 13: "commit_verify_prep",
            14: "decode_slots", 15: "slot_copy", 16: "prefill_chunked_prep", 17: "prefill_recurrent_prep",
            18: "verify_slots", 19: "commit_slots", 20: "commit_verify_slots", 21: "prefill_chunked_slots",
            22: "mixed", 23: "kv_append", 24: "attn_decode", 25: "kv_append_axes", 26: "kv_append_blocks",
            27: "attn_decode_blocks", 28: "attn_weights", 29: "kv_evict"}
GATE_EXP_NEG_SOFTPLUS, GATE_SIGMOID = 0, 1
DEV_ERR_ACCEPTED, DEV_ERR_CKPT_SLOT, DEV_ERR_DRAFT_LEN, DEV_ERR_SLOT_ID, DEV_ERR_MIXED = 1, 2, 4, 8, 16
DEV_ERR_PAGE, DEV_ERR_POS, DEV_ERR_TOKENS = 32, 64, 128
ROLE_IDLE, ROLE_DECODE, ROLE_SPEC, ROLE_PREFILL = 0, 1, 2, 3


class KdaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libkda status {status}: {msg}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Log(ctypes.Structure):
    _fields_ = [("dev", ctypes.c_void_p), ("bytes", ctypes.c_size_t), ("T_max", ctypes.c_int32),
                ("pending_T", ctypes.c_int32), ("pending_form", ctypes.c_int32)]


class _Slots(ctypes.Structure):
    _fields_ = [("states", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("n_slots", ctypes.c_int32)]


class KvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hkv", "dk", "dv", "in_dtype", "cache_dtype")]


class _Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class _Rotation(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32), ("start", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("pairs", ctypes.c_int32)]


class _Axes(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("stride", ctypes.c_int64), ("n_axes", ctypes.c_int32),
                ("axis_of", ctypes.c_char_p)]


class _BlockScales(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block", ctypes.c_int32)]


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_SIGS = {
    "kda_log_bytes": (ctypes.c_size_t, [ctypes.POINTER(Shape), _I]),
    "kda_slot_bytes": (ctypes.c_size_t, [ctypes.POINTER(Shape)]),
    "kda_decode_step": (_I, [ctypes.POINTER(Shape), _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "kda_decode_step_prep": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "kda_verify_prep": (_I, [ctypes.POINTER(Shape), _I, _I, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Log), _P]),
    "kda_commit_verify_prep": (_I, [ctypes.POINTER(Shape), _I, _I, _P, _P, _P, _P, _P, _P, _P, _P,
                                    ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_verify": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Log), _P]),
    "kda_commit": (_I, [ctypes.POINTER(Shape), _P, _P, ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_commit_verify": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Log), _P,
                               _P, _P]),
    "kda_verify_varlen": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Log), _P,
                               _P]),
    "kda_commit_verify_varlen": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_decode_step_slots": (_I, [ctypes.POINTER(Shape), _P, ctypes.POINTER(_Slots), _P, _P, _P, _P, _P, _P, _P,
                                   _P]),
    "kda_slot_copy": (_I, [ctypes.POINTER(Shape), _P, _P, _I, ctypes.POINTER(_Slots), _P]),
    "kda_prefill_chunked_slots": (_I, [ctypes.POINTER(Shape), _I, _I, _P, ctypes.POINTER(_Slots), _P, _P, _P, _P, _P,
                                       _P, _I, _P, _P, _P]),
    "kda_verify_slots": (_I, [ctypes.POINTER(Shape), _I, _P, ctypes.POINTER(_Slots), _P, _P, _P, _P, _P, _P,
                              ctypes.POINTER(_Log), _P, _P]),
    "kda_commit_slots": (_I, [ctypes.POINTER(Shape), _P, ctypes.POINTER(_Slots), ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_commit_verify_slots": (_I, [ctypes.POINTER(Shape), _I, _P, ctypes.POINTER(_Slots), _P, _P, _P, _P, _P, _P,
                                     ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_snapshot": (_I, [ctypes.POINTER(Shape), _P, _P, _P, _P, _I, ctypes.POINTER(_Slots), _P]),
    "kda_restore": (_I, [ctypes.POINTER(Shape), _P, _P, _P, _P, _I, ctypes.POINTER(_Slots), _P]),
    "kda_prefill_chunked": (_I, [ctypes.POINTER(Shape), _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P,
                                 ctypes.POINTER(_Slots), _P, _P]),
    "kda_prefill_recurrent": (_I, [ctypes.POINTER(Shape), _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P,
                                   ctypes.POINTER(_Slots), _P, _P]),
    "kda_prefill_chunked_prep": (_I, [ctypes.POINTER(Shape), _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P,
                                      ctypes.POINTER(_Slots), _P, _P]),
    "kda_prefill_recurrent_prep": (_I, [ctypes.POINTER(Shape), _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P,
                                        ctypes.POINTER(_Slots), _P, _P]),
    "kda_mixed_step": (_I, [ctypes.POINTER(Shape), _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P,
                            ctypes.POINTER(_Log), _P, _P, _P]),
    "kda_kv_append": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), _P, _I, _P, _I, _P, _P, _L, _P, _L, _P, _L,
                           _P, _L, ctypes.POINTER(_Rotation), _P, _P]),
    "kda_attn_decode": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), _P, _I, _P, _I, _P, _P, _L,
                             ctypes.c_float, _I, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "kda_kv_append_axes": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), _P, _I, _P, _I, _P, _P, _L, _P, _L, _P,
                                _L, _P, _L, ctypes.POINTER(_Rotation), ctypes.POINTER(_Axes), _P, _P]),
    "kda_kv_append_blocks": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), ctypes.POINTER(_BlockScales), _P, _I,
                                  _P, _I, _P, _P, _L, _P, _L, _P, _L, _P, _L, ctypes.POINTER(_Rotation),
                                  ctypes.POINTER(_Axes), _P, _P]),
    "kda_attn_decode_blocks": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), ctypes.POINTER(_BlockScales), _P,
                                    _I, _P, _I, _P, _P, _L, ctypes.c_float, _I, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "kda_attn_weights": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), ctypes.POINTER(_BlockScales), _P, _I, _P,
                              _I, _P, _P, _L, ctypes.c_float, _I, _P, _P, _L, _P, _P]),
    "kda_kv_evict": (_I, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), ctypes.POINTER(_BlockScales), _P, _I, _P, _P,
                          _L, _I, _I, _P, _I, _P, _P, _P, _P, _P]),
    "kda_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(KvShape), ctypes.POINTER(_Pages), _I]),
    "kda_status_str": (ctypes.c_char_p, [_I]),
    "kda_last_variant": (_I, []),
    "kda_abi_version": (_I, []),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m recurrent_state_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(status: int):
    if status != 0:
        raise KdaError(status, lib().kda_status_str(status).decode())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(state, in_dtype, scale):
    B, H, dk, dv = state.shape
    code = KDA_BF16 if in_dtype == torch.bfloat16 else KDA_F32 if in_dtype == torch.float32 else None
    if code is None:
        raise TypeError(f"q/k/v dtype must be bfloat16 or float32, not {in_dtype}")
    sc = float(dk) ** -0.5 if scale is None else float(scale)
    return Shape(B, H, dk, dv, code, sc)


def _check_tokens(state, T, q, k, v, alpha, beta, o):
    B, H, dk, dv = state.shape
    dev = state.device
    dt = q.dtype
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(alpha, "alpha", (B, T, H, dk), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    _need(o, "o", (B, T, H, dv), torch.float32, dev)


def log_bytes(shape: Shape, T_max: int) -> int:
    return int(lib().kda_log_bytes(ctypes.byref(shape), T_max))


def slot_bytes(shape: Shape) -> int:
    return int(lib().kda_slot_bytes(ctypes.byref(shape)))


def last_variant() -> str:
    return VARIANTS.get(int(lib().kda_last_variant()), "unknown")


class InputLog:
    """Device buffer for the verify input log plus its host-side bookkeeping."""

    def __init__(self, state: torch.Tensor, T_max: int, in_dtype=torch.bfloat16):
        self.shape = _shape(state, in_dtype, None)
        n = log_bytes(self.shape, T_max)
        if n == 0:
            raise ValueError("unsupported log shape")
        self.buf = torch.empty(n, dtype=torch.uint8, device=state.device)
        self.c = _Log(self.buf.data_ptr(), n, T_max, 0)

    @property
    def pending_T(self) -> int:
        return int(self.c.pending_T)


class SlotPool:
    """Caller-owned slot pool: states f32 [n_slots][H][dk][dv], pos i64 [n_slots]."""

    def __init__(self, n_slots: int, H: int, dk: int, dv: int, device):
        self.states = torch.zeros((n_slots, H, dk, dv), dtype=torch.float32, device=device)
        self.pos = torch.full((n_slots,), -1, dtype=torch.int64, device=device)
        self.c = _Slots(self.states.data_ptr(), self.pos.data_ptr(), n_slots)

    @property
    def n_slots(self) -> int:
        return int(self.c.n_slots)


def decode_step(state, pos, q, k, v, alpha, beta, o, scale=None):
    """One decode token for every (sequence, head); inputs [B][1][H][d] (or [B][H][d])."""
    B, H, dk, dv = state.shape
    if beta.dim() == 2:  # [B][H] form: add the token axis
        q, k, v, alpha, beta, o = (x.unsqueeze(1) for x in (q, k, v, alpha, beta, o))
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _check_tokens(state, 1, q, k, v, alpha, beta, o)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_decode_step(ctypes.byref(sh), _ptr(state), _ptr(pos), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(alpha), _ptr(beta), _ptr(o), _stream()))


def decode_step_prep(state, pos, q, k, v, alpha_logit, beta_logit, o, gate=GATE_EXP_NEG_SOFTPLUS, scale=None):
    """decode_step from raw projections: q, k un-normalised, the decay and beta as logits
    (decay = exp(-softplus(x)) for GATE_EXP_NEG_SOFTPLUS, sigmoid(x) for GATE_SIGMOID)."""
    B, H, dk, dv = state.shape
    if beta_logit.dim() == 2:
        q, k, v, alpha_logit, beta_logit, o = (x.unsqueeze(1) for x in (q, k, v, alpha_logit, beta_logit, o))
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _check_tokens(state, 1, q, k, v, alpha_logit, beta_logit, o)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_decode_step_prep(ctypes.byref(sh), int(gate), _ptr(state), _ptr(pos), _ptr(q), _ptr(k),
                                      _ptr(v), _ptr(alpha_logit), _ptr(beta_logit), _ptr(o), _stream()))


def _verify_args(state, q, k, v, alpha, beta, o, log: InputLog, scale):
    B, H, dk, dv = state.shape
    T = q.shape[1]
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _check_tokens(state, T, q, k, v, alpha, beta, o)
    sh = _shape(state, q.dtype, scale)
    if sh.in_dtype != log.shape.in_dtype or (B, H, dk, dv) != (log.shape.B, log.shape.H, log.shape.dk,
                                                               log.shape.dv):
        raise ValueError("log was sized for a different shape")
    return sh, T, tuple(_ptr(t) for t in (state, q, k, v, alpha, beta, o))


def verify(state, q, k, v, alpha, beta, o, log: InputLog, scale=None):
    """Verify T draft tokens (inputs [B][T][H][d]) from the committed state; fills the log."""
    sh, T, ptrs = _verify_args(state, q, k, v, alpha, beta, o, log, scale)
    _check(lib().kda_verify(ctypes.byref(sh), T, *ptrs, ctypes.byref(log.c), _stream()))


def verify_prep(state, q, k, v, alpha_logit, beta_logit, o, log: InputLog, gate=GATE_EXP_NEG_SOFTPLUS, scale=None):
    """verify from raw projections and logits (prepared in the kernel, logged raw)."""
    sh, T, ptrs = _verify_args(state, q, k, v, alpha_logit, beta_logit, o, log, scale)
    _check(lib().kda_verify_prep(ctypes.byref(sh), int(gate), T, *ptrs, ctypes.byref(log.c), _stream()))


def verify_varlen(state, q, k, v, alpha, beta, o, log: InputLog, draft_len, dev_err, scale=None):
    """verify where sequence b has only its first draft_len[b] tokens (device int32 [B], each in [0, T])."""
    sh, T, ptrs = _verify_args(state, q, k, v, alpha, beta, o, log, scale)
    _need(draft_len, "draft_len", (state.shape[0],), torch.int32, state.device)
    _need(dev_err, "dev_err", (1,), torch.int32, state.device)
    _check(lib().kda_verify_varlen(ctypes.byref(sh), T, _ptr(draft_len), *ptrs, ctypes.byref(log.c), _ptr(dev_err),
                                   _stream()))


def commit(state, pos, log: InputLog, accepted, dev_err):
    """Replay accepted[b] logged tokens onto the committed state (accepted: device int32 [B])."""
    B, H, dk, dv = state.shape
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _need(accepted, "accepted", (B,), torch.int32, state.device)
    _need(dev_err, "dev_err", (1,), torch.int32, state.device)
    if (B, H, dk, dv) != (log.shape.B, log.shape.H, log.shape.dk, log.shape.dv):
        raise ValueError("log was sized for a different shape")
    _check(lib().kda_commit(ctypes.byref(log.shape), _ptr(state), _ptr(pos), ctypes.byref(log.c),
                            _ptr(accepted), _ptr(dev_err), _stream()))


def _commit_verify_args(state, pos, q, k, v, alpha, beta, o, log: InputLog, accepted, dev_err, scale):
    B, H, dk, dv = state.shape
    T = q.shape[1]
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _check_tokens(state, T, q, k, v, alpha, beta, o)
    if accepted is not None:
        _need(accepted, "accepted", (B,), torch.int32, state.device)
    if dev_err is not None:
        _need(dev_err, "dev_err", (1,), torch.int32, state.device)
    sh = _shape(state, q.dtype, scale)
    if (B, H, dk, dv, sh.in_dtype) != (log.shape.B, log.shape.H, log.shape.dk, log.shape.dv, log.shape.in_dtype):
        raise ValueError("log was sized for a different shape")
    ptrs = tuple(_ptr(t) for t in (state, pos, q, k, v, alpha, beta, o))
    extra = (_ptr(accepted) if accepted is not None else None, _ptr(dev_err) if dev_err is not None else None)
    return sh, T, ptrs, extra


def commit_verify(state, pos, q, k, v, alpha, beta, o, log: InputLog, accepted=None, dev_err=None, scale=None):
    """Commit the pending verify's accepted prefix, then verify T new drafts, in one launch."""
    sh, T, ptrs, extra = _commit_verify_args(state, pos, q, k, v, alpha, beta, o, log, accepted, dev_err, scale)
    _check(lib().kda_commit_verify(ctypes.byref(sh), T, *ptrs, ctypes.byref(log.c), *extra, _stream()))


def commit_verify_prep(state, pos, q, k, v, alpha_logit, beta_logit, o, log: InputLog, accepted=None, dev_err=None,
                       gate=GATE_EXP_NEG_SOFTPLUS, scale=None):
    """commit_verify whose new drafts are raw projections and logits (as verify_prep)."""
    sh, T, ptrs, extra = _commit_verify_args(state, pos, q, k, v, alpha_logit, beta_logit, o, log, accepted, dev_err,
                                             scale)
    _check(lib().kda_commit_verify_prep(ctypes.byref(sh), int(gate), T, *ptrs, ctypes.byref(log.c), *extra,
                                        _stream()))


def commit_verify_varlen(state, pos, q, k, v, alpha, beta, o, log: InputLog, draft_len, accepted=None, dev_err=None,
                         scale=None):
    """commit_verify whose new drafts have a length per sequence (draft_len: device int32 [B])."""
    sh, T, ptrs, extra = _commit_verify_args(state, pos, q, k, v, alpha, beta, o, log, accepted, dev_err, scale)
    _need(draft_len, "draft_len", (state.shape[0],), torch.int32, state.device)
    _check(lib().kda_commit_verify_varlen(ctypes.byref(sh), T, _ptr(draft_len), *ptrs, ctypes.byref(log.c), *extra,
                                          _stream()))


def _pairs(seq_ids, slot_ids):
    s = (ctypes.c_int32 * len(seq_ids))(*[int(x) for x in seq_ids])
    t = (ctypes.c_int32 * len(slot_ids))(*[int(x) for x in slot_ids])
    if len(seq_ids) != len(slot_ids):
        raise ValueError("seq_ids and slot_ids differ in length")
    return s, t


class _Batch:
    """Stands in for a [B][H][dk][dv] state tensor where only its shape and device matter."""

    def __init__(self, B, pool: SlotPool):
        _, H, dk, dv = pool.states.shape
        self.shape = (B, H, dk, dv)
        self.device = pool.states.device


def _decode_slots_args(slot_ids, pool: SlotPool, q, k, v, alpha, beta, o, dev_err, scale):
    B = slot_ids.shape[0]
    _need(slot_ids, "slot_ids", (B,), torch.int32, pool.states.device)
    _need(dev_err, "dev_err", (1,), torch.int32, pool.states.device)
    if beta.dim() == 2:
        q, k, v, alpha, beta, o = (x.unsqueeze(1) for x in (q, k, v, alpha, beta, o))
    batch = _Batch(B, pool)
    _check_tokens(batch, 1, q, k, v, alpha, beta, o)
    sh = _shape(batch, q.dtype, scale)
    return sh, (slot_ids, q, k, v, alpha, beta, o, dev_err)


def decode_step_slots(slot_ids, pool: SlotPool, q, k, v, alpha, beta, o, dev_err, scale=None):
    """decode_step on states in a slot pool: sequence b updates pool slot slot_ids[b] (device int32 [B])."""
    sh, t = _decode_slots_args(slot_ids, pool, q, k, v, alpha, beta, o, dev_err, scale)
    slot_ids, q, k, v, alpha, beta, o, dev_err = t
    _check(lib().kda_decode_step_slots(ctypes.byref(sh), _ptr(slot_ids), ctypes.byref(pool.c), _ptr(q), _ptr(k),
                                       _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _ptr(dev_err), _stream()))


class DecodeSlotsPlan:
    """A decode_step_slots call validated once (see DecodePlan)."""

    def __init__(self, slot_ids, pool: SlotPool, q, k, v, alpha, beta, o, dev_err, scale=None):
        self._shape, t = _decode_slots_args(slot_ids, pool, q, k, v, alpha, beta, o, dev_err, scale)
        self._keep = (pool,) + t
        slot_ids, q, k, v, alpha, beta, o, dev_err = t
        self._args = (ctypes.byref(self._shape), _ptr(slot_ids), ctypes.byref(pool.c)) + tuple(
            _ptr(x) for x in (q, k, v, alpha, beta, o, dev_err))
        self._fn = lib().kda_decode_step_slots

    def __call__(self):
        _check(self._fn(*self._args, _stream()))


def _slots_batch(slot_ids, pool: SlotPool, log: InputLog, dev_err):
    B = slot_ids.shape[0]
    _need(slot_ids, "slot_ids", (B,), torch.int32, pool.states.device)
    _need(dev_err, "dev_err", (1,), torch.int32, pool.states.device)
    batch = _Batch(B, pool)
    if batch.shape != (log.shape.B, log.shape.H, log.shape.dk, log.shape.dv):
        raise ValueError("log was sized for a different shape")
    return batch


def verify_slots(slot_ids, pool: SlotPool, q, k, v, alpha, beta, o, log: InputLog, dev_err, scale=None):
    """verify on states in a slot pool (sequence b reads slot slot_ids[b]); log, inputs and o are the batch's."""
    batch = _slots_batch(slot_ids, pool, log, dev_err)
    T = q.shape[1]
    _check_tokens(batch, T, q, k, v, alpha, beta, o)
    sh = _shape(batch, q.dtype, scale)
    _check(lib().kda_verify_slots(ctypes.byref(sh), T, _ptr(slot_ids), ctypes.byref(pool.c),
                                  *(_ptr(x) for x in (q, k, v, alpha, beta, o)), ctypes.byref(log.c), _ptr(dev_err),
                                  _stream()))


def commit_slots(slot_ids, pool: SlotPool, log: InputLog, accepted, dev_err):
    """commit onto states and positions in a slot pool (sequence b updates slot slot_ids[b])."""
    batch = _slots_batch(slot_ids, pool, log, dev_err)
    _need(accepted, "accepted", (batch.shape[0],), torch.int32, pool.states.device)
    _check(lib().kda_commit_slots(ctypes.byref(log.shape), _ptr(slot_ids), ctypes.byref(pool.c), ctypes.byref(log.c),
                                  _ptr(accepted), _ptr(dev_err), _stream()))


def commit_verify_slots(slot_ids, pool: SlotPool, q, k, v, alpha, beta, o, log: InputLog, dev_err, accepted=None,
                        scale=None):
    """commit_verify on states and positions in a slot pool."""
    batch = _slots_batch(slot_ids, pool, log, dev_err)
    T = q.shape[1]
    _check_tokens(batch, T, q, k, v, alpha, beta, o)
    if accepted is not None:
        _need(accepted, "accepted", (batch.shape[0],), torch.int32, pool.states.device)
    sh = _shape(batch, q.dtype, scale)
    _check(lib().kda_commit_verify_slots(ctypes.byref(sh), T, _ptr(slot_ids), ctypes.byref(pool.c),
                                         *(_ptr(x) for x in (q, k, v, alpha, beta, o)), ctypes.byref(log.c),
                                         _ptr(accepted) if accepted is not None else None, _ptr(dev_err), _stream()))


def prefill_chunked_slots(state_slots, pool: SlotPool, q, k, v, alpha, beta, o, dev_err, *, chunk=64, ckpt_every=0,
                          ckpt_slots=None, scale=None):
    """prefill_chunked on states in a slot pool: sequence b starts from and ends in slot state_slots[b]."""
    B = state_slots.shape[0]
    _need(state_slots, "state_slots", (B,), torch.int32, pool.states.device)
    _need(dev_err, "dev_err", (1,), torch.int32, pool.states.device)
    batch = _Batch(B, pool)
    L = q.shape[1]
    _check_tokens(batch, L, q, k, v, alpha, beta, o)
    n_ckpt = L // ckpt_every if ckpt_every > 0 else 0
    if n_ckpt > 0:
        _need(ckpt_slots, "ckpt_slots", (B, n_ckpt), torch.int32, pool.states.device)
    sh = _shape(batch, q.dtype, scale)
    _check(lib().kda_prefill_chunked_slots(ctypes.byref(sh), L, chunk, _ptr(state_slots), ctypes.byref(pool.c),
                                           *(_ptr(x) for x in (q, k, v, alpha, beta, o)), ckpt_every,
                                           _ptr(ckpt_slots) if n_ckpt else None, _ptr(dev_err), _stream()))


def mixed_step(state, pos, roles, tok_start, counts, q, k, v, alpha, beta, o, dev_err, *, log: InputLog = None,
               accepted=None, slot_ids=None, scale=None):
    """One serving step over a mixed batch in one launch (kda_mixed_step).

    roles (device int32 [B], ROLE_*) and tok_start (device int32 [B + 1])
    describe the batch; counts = (n_decode, n_spec, n_prefill) are the host's
    role counts.  Tokens are packed: q, k [N][H][dk], v [N][H][dv], alpha
    [N][H][dk], beta [N][H], o [N][H][dv].  state / pos are the dense [B]
    states, or a slot pool's arrays when slot_ids (device int32 [B]) is given.
    """
    B = roles.shape[0]
    dev = state.device
    _need(roles, "roles", (B,), torch.int32, dev)
    _need(tok_start, "tok_start", (B + 1,), torch.int32, dev)
    _need(dev_err, "dev_err", (1,), torch.int32, dev)
    n_slots, H, dk, dv = state.shape
    _need(state, "state", (n_slots, H, dk, dv), torch.float32, dev)
    _need(pos, "pos", (n_slots,), torch.int64, dev)
    if slot_ids is None:
        if n_slots != B:
            raise ValueError("without slot_ids, state holds one entry per sequence")
    else:
        _need(slot_ids, "slot_ids", (B,), torch.int32, dev)
    N = q.shape[0]
    _need(q, "q", (N, H, dk), q.dtype, dev)
    _need(k, "k", (N, H, dk), q.dtype, dev)
    _need(v, "v", (N, H, dv), q.dtype, dev)
    _need(alpha, "alpha", (N, H, dk), torch.float32, dev)
    _need(beta, "beta", (N, H), torch.float32, dev)
    _need(o, "o", (N, H, dv), torch.float32, dev)
    if accepted is not None:
        _need(accepted, "accepted", (B,), torch.int32, dev)
    sh = _shape(torch.empty((B, H, dk, dv), device="meta"), q.dtype, scale)
    if log is not None and (B, H, dk, dv, sh.in_dtype) != (log.shape.B, log.shape.H, log.shape.dk, log.shape.dv,
                                                           log.shape.in_dtype):
        raise ValueError("log was sized for a different shape")
    n_dec, n_spec, n_pf = (int(c) for c in counts)
    _check(lib().kda_mixed_step(ctypes.byref(sh), _ptr(roles), _ptr(tok_start), N, n_dec, n_spec, n_pf, _ptr(state),
                                _ptr(pos), _ptr(slot_ids), n_slots if slot_ids is not None else 0,
                                *(_ptr(x) for x in (q, k, v, alpha, beta, o)),
                                ctypes.byref(log.c) if log is not None else None, _ptr(accepted), _ptr(dev_err),
                                _stream()))


def slot_copy(src_slots, dst_slots, pool: SlotPool):
    """Copy whole states and positions between pool slots: dst_slots[i] <- src_slots[i] (host ids)."""
    s, t = _pairs(src_slots, dst_slots)
    _, H, dk, dv = pool.states.shape
    sh = Shape(0, H, dk, dv, KDA_BF16, 1.0)
    _check(lib().kda_slot_copy(ctypes.byref(sh), s, t, len(src_slots), ctypes.byref(pool.c), _stream()))


def snapshot(state, pos, seq_ids, slot_ids, pool: SlotPool):
    B, H, dk, dv = state.shape
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _need(pool.states, "pool.states", (pool.n_slots, H, dk, dv), torch.float32, state.device)
    s, t = _pairs(seq_ids, slot_ids)
    sh = Shape(B, H, dk, dv, KDA_BF16, 1.0)
    _check(lib().kda_snapshot(ctypes.byref(sh), _ptr(state), _ptr(pos), s, t, len(seq_ids),
                              ctypes.byref(pool.c), _stream()))


def restore(state, pos, seq_ids, slot_ids, pool: SlotPool):
    B, H, dk, dv = state.shape
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _need(pool.states, "pool.states", (pool.n_slots, H, dk, dv), torch.float32, state.device)
    s, t = _pairs(seq_ids, slot_ids)
    sh = Shape(B, H, dk, dv, KDA_BF16, 1.0)
    _check(lib().kda_restore(ctypes.byref(sh), _ptr(state), _ptr(pos), s, t, len(seq_ids),
                             ctypes.byref(pool.c), _stream()))


def _prefill_args(state, pos, q, k, v, alpha, beta, o, ckpt_every, ckpt_slots, pool, dev_err):
    B, H, dk, dv = state.shape
    L = q.shape[1]
    _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
    _need(pos, "pos", (B,), torch.int64, state.device)
    _check_tokens(state, L, q, k, v, alpha, beta, o)
    n_ckpt = L // ckpt_every if ckpt_every > 0 else 0
    if n_ckpt > 0:
        if pool is None or ckpt_slots is None or dev_err is None:
            raise ValueError("checkpoints need ckpt_slots, a slot pool and dev_err")
        _need(ckpt_slots, "ckpt_slots", (B, n_ckpt), torch.int32, state.device)
        _need(dev_err, "dev_err", (1,), torch.int32, state.device)
        _need(pool.states, "pool.states", (pool.n_slots, H, dk, dv), torch.float32, state.device)
    return L, n_ckpt


def prefill_chunked(state, pos, q, k, v, alpha, beta, o, *, chunk=64, ckpt_every=0, ckpt_slots=None,
                    pool: SlotPool | None = None, dev_err=None, scale=None):
    """Chunked (WY/UT form) prompt processing of L tokens ([B][L][H][d]) into the state."""
    L, n_ckpt = _prefill_args(state, pos, q, k, v, alpha, beta, o, ckpt_every, ckpt_slots, pool, dev_err)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_prefill_chunked(ctypes.byref(sh), L, chunk, _ptr(state), _ptr(pos), _ptr(q), _ptr(k),
                                     _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), ckpt_every,
                                     _ptr(ckpt_slots) if n_ckpt else None,
                                     ctypes.byref(pool.c) if pool is not None else None,
                                     _ptr(dev_err), _stream()))


def prefill_recurrent(state, pos, q, k, v, alpha, beta, o, *, ckpt_every=0, ckpt_slots=None,
                      pool: SlotPool | None = None, dev_err=None, scale=None):
    """Token-by-token prompt processing (state in registers for the whole prompt)."""
    L, n_ckpt = _prefill_args(state, pos, q, k, v, alpha, beta, o, ckpt_every, ckpt_slots, pool, dev_err)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_prefill_recurrent(ctypes.byref(sh), L, _ptr(state), _ptr(pos), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(alpha), _ptr(beta), _ptr(o), ckpt_every,
                                       _ptr(ckpt_slots) if n_ckpt else None,
                                       ctypes.byref(pool.c) if pool is not None else None,
                                       _ptr(dev_err), _stream()))


def prefill_chunked_prep(state, pos, q, k, v, alpha_logit, beta_logit, o, *, gate=GATE_EXP_NEG_SOFTPLUS, chunk=64,
                         ckpt_every=0, ckpt_slots=None, pool: SlotPool | None = None, dev_err=None, scale=None):
    """prefill_chunked from raw projections and logits (prepared in the kernel)."""
    L, n_ckpt = _prefill_args(state, pos, q, k, v, alpha_logit, beta_logit, o, ckpt_every, ckpt_slots, pool, dev_err)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_prefill_chunked_prep(ctypes.byref(sh), int(gate), L, chunk, _ptr(state), _ptr(pos), _ptr(q),
                                          _ptr(k), _ptr(v), _ptr(alpha_logit), _ptr(beta_logit), _ptr(o), ckpt_every,
                                          _ptr(ckpt_slots) if n_ckpt else None,
                                          ctypes.byref(pool.c) if pool is not None else None,
                                          _ptr(dev_err), _stream()))


def prefill_recurrent_prep(state, pos, q, k, v, alpha_logit, beta_logit, o, *, gate=GATE_EXP_NEG_SOFTPLUS,
                           ckpt_every=0, ckpt_slots=None, pool: SlotPool | None = None, dev_err=None, scale=None):
    """prefill_recurrent from raw projections and logits (bit-identical to decode_step_prep token by token)."""
    L, n_ckpt = _prefill_args(state, pos, q, k, v, alpha_logit, beta_logit, o, ckpt_every, ckpt_slots, pool, dev_err)
    sh = _shape(state, q.dtype, scale)
    _check(lib().kda_prefill_recurrent_prep(ctypes.byref(sh), int(gate), L, _ptr(state), _ptr(pos), _ptr(q),
                                            _ptr(k), _ptr(v), _ptr(alpha_logit), _ptr(beta_logit), _ptr(o),
                                            ckpt_every, _ptr(ckpt_slots) if n_ckpt else None,
                                            ctypes.byref(pool.c) if pool is not None else None,
                                            _ptr(dev_err), _stream()))


class DecodePlan:
    """A decode_step call validated once, for launch-bound loops and HIP-graph
    capture: calling the plan only passes the stored pointers and the current
    stream to the library."""

    def __init__(self, state, pos, q, k, v, alpha, beta, o, scale=None, prep_gate=None):
        B, H, dk, dv = state.shape
        if beta.dim() == 2:
            q, k, v, alpha, beta, o = (x.unsqueeze(1) for x in (q, k, v, alpha, beta, o))
        _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
        _need(pos, "pos", (B,), torch.int64, state.device)
        _check_tokens(state, 1, q, k, v, alpha, beta, o)
        self._keep = (state, pos, q, k, v, alpha, beta, o)
        self._shape = _shape(state, q.dtype, scale)
        if prep_gate is None:      # prepared inputs
            self._args = (ctypes.byref(self._shape),) + tuple(_ptr(t) for t in self._keep)
            self._fn = lib().kda_decode_step
        else:                      # raw projections and logits (decode_step_prep)
            self._args = (ctypes.byref(self._shape), int(prep_gate)) + tuple(_ptr(t) for t in self._keep)
            self._fn = lib().kda_decode_step_prep

    def __call__(self):
        _check(self._fn(*self._args, _stream()))


class VerifyPlan:
    """A verify call validated once (see DecodePlan); with draft_len (and
    dev_err) it is a verify_varlen call."""

    def __init__(self, state, q, k, v, alpha, beta, o, log: InputLog, scale=None, draft_len=None, dev_err=None,
                 prep_gate=None):
        self._shape, T, ptrs = _verify_args(state, q, k, v, alpha, beta, o, log, scale)
        self._keep = (state, q, k, v, alpha, beta, o, log, draft_len, dev_err)
        if prep_gate is not None:
            if draft_len is not None:
                raise ValueError("draft lengths and raw projections do not combine")
            self._args = (ctypes.byref(self._shape), int(prep_gate), T) + ptrs + (ctypes.byref(log.c),)
            self._fn = lib().kda_verify_prep
        elif draft_len is None:
            self._args = (ctypes.byref(self._shape), T) + ptrs + (ctypes.byref(log.c),)
            self._fn = lib().kda_verify
        else:
            _need(draft_len, "draft_len", (state.shape[0],), torch.int32, state.device)
            _need(dev_err, "dev_err", (1,), torch.int32, state.device)
            self._args = (ctypes.byref(self._shape), T, _ptr(draft_len)) + ptrs + (ctypes.byref(log.c),
                                                                                   _ptr(dev_err))
            self._fn = lib().kda_verify_varlen

    def __call__(self):
        _check(self._fn(*self._args, _stream()))


class CommitPlan:
    """A commit call validated once (see DecodePlan)."""

    def __init__(self, state, pos, log: InputLog, accepted, dev_err):
        B, H, dk, dv = state.shape
        _need(state, "state", (B, H, dk, dv), torch.float32, state.device)
        _need(pos, "pos", (B,), torch.int64, state.device)
        _need(accepted, "accepted", (B,), torch.int32, state.device)
        _need(dev_err, "dev_err", (1,), torch.int32, state.device)
        if (B, H, dk, dv) != (log.shape.B, log.shape.H, log.shape.dk, log.shape.dv):
            raise ValueError("log was sized for a different shape")
        self._keep = (state, pos, log, accepted, dev_err)
        self._args = (ctypes.byref(log.shape), _ptr(state), _ptr(pos), ctypes.byref(log.c), _ptr(accepted),
                      _ptr(dev_err))
        self._fn = lib().kda_commit

    def __call__(self):
        _check(self._fn(*self._args, _stream()))


class CommitVerifyPlan:
    """A commit_verify call validated once (see DecodePlan).  The pending
    count of the log when the plan is called is the one committed."""

    def __init__(self, state, pos, q, k, v, alpha, beta, o, log: InputLog, accepted=None, dev_err=None, scale=None,
                 draft_len=None, prep_gate=None):
        self._shape, T, ptrs, extra = _commit_verify_args(state, pos, q, k, v, alpha, beta, o, log, accepted,
                                                          dev_err, scale)
        self._keep = (state, pos, q, k, v, alpha, beta, o, log, accepted, dev_err, draft_len)
        if prep_gate is not None:
            if draft_len is not None:
                raise ValueError("draft lengths and raw projections do not combine")
            self._args = (ctypes.byref(self._shape), int(prep_gate), T) + ptrs + (ctypes.byref(log.c),) + extra
            self._fn = lib().kda_commit_verify_prep
        elif draft_len is None:
            self._args = (ctypes.byref(self._shape), T) + ptrs + (ctypes.byref(log.c),) + extra
            self._fn = lib().kda_commit_verify
        else:
            _need(draft_len, "draft_len", (state.shape[0],), torch.int32, state.device)
            self._args = (ctypes.byref(self._shape), T, _ptr(draft_len)) + ptrs + (ctypes.byref(log.c),) + extra
            self._fn = lib().kda_commit_verify_varlen

    def __call__(self):
        _check(self._fn(*self._args, _stream()))


_DTYPE_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.float8_e4m3fn: KDA_E4M3}


class PagePool:
    """Caller-owned pages of the attention cache: k [n_pages][Hkv][page_size][dk], v [n_pages][Hkv][page_size][dv].

    `latent` pools have no v: a row's first dv values are its value.  An e4m3
    pool (dtype torch.float8_e4m3fn) holds value / scale, with one f32 scale
    per kv head in k_scale and v_scale, or, with `scale_block`, one for each
    scale_block tokens of a page and kv head, f32
    [n_pages][Hkv][page_size / scale_block], which the appends set.
    """

    c_scales = None  # scales by blocks, for the calls that take them apart from the pages

    def __init__(self, n_pages: int, page_size: int, Hkv: int, dk: int, dv: int, device, dtype=torch.bfloat16,
                 latent: bool = False, k_scale=None, v_scale=None, scale_block: int = 0):
        if scale_block:
            _check_scale_block(scale_block, page_size, dtype, latent)
            per = (n_pages, Hkv, page_size // scale_block)
            k_scale = torch.ones(per, dtype=torch.float32, device=device) if k_scale is None else k_scale
            v_scale = torch.ones(per, dtype=torch.float32, device=device) if v_scale is None else v_scale
        k = torch.zeros((n_pages, Hkv, page_size, dk), dtype=dtype, device=device)
        v = None if latent else torch.zeros((n_pages, Hkv, page_size, dv), dtype=dtype, device=device)
        self._hold(k, v, dv, k_scale, v_scale, scale_block)

    @classmethod
    def from_tensors(cls, k, v=None, *, dv=None, k_scale=None, v_scale=None, scale_block: int = 0) -> "PagePool":
        """A pool over existing tensors (v None: latent, dv its value width)."""
        pool = cls.__new__(cls)
        if v is None and dv is None:
            raise ValueError("a latent pool needs its value width dv")
        pool._hold(k, v, v.shape[-1] if v is not None else int(dv), k_scale, v_scale, scale_block)
        return pool

    def _hold(self, k, v, dv, k_scale, v_scale, scale_block=0):
        if k.dim() != 4:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [n_pages][Hkv][page_size][dk]")
        n_pages, Hkv, page_size, dk = k.shape
        if k.dtype not in _DTYPE_CODES:
            raise TypeError(f"page dtype must be bfloat16, float32 or float8_e4m3fn, not {k.dtype}")
        _need_gpu(k, "k")
        _need(k, "k", k.shape, k.dtype, k.device)
        if v is not None:
            _need(v, "v", (n_pages, Hkv, page_size, dv), k.dtype, k.device)
        if scale_block:
            _check_scale_block(scale_block, page_size, k.dtype, v is None)
        if k.dtype == torch.float8_e4m3fn:
            per = (n_pages, Hkv, page_size // scale_block) if scale_block else (Hkv,)
            _need(k_scale, "k_scale", per, torch.float32, k.device)
            _need(v_scale, "v_scale", per, torch.float32, k.device)
        elif k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to float8_e4m3fn pages only")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.Hkv, self.page_size, self.dk = n_pages, Hkv, page_size, dk
        self.dv, self.latent, self.device, self.scale_block = dv, v is None, k.device, int(scale_block)
        self.c = _Pages(*(None if x is None else x.data_ptr() for x in (k, v, k_scale, v_scale)), n_pages, page_size)
        if scale_block:
            self.c_scales = _BlockScales(k_scale.data_ptr(), v_scale.data_ptr(), scale_block)


def _scales(pool):
    """A call's kda_block_scales: None for a pool without scales by blocks."""
    c = getattr(pool, "c_scales", None)
    return None if c is None else ctypes.byref(c)


def _check_scale_block(block, page_size, dtype, latent):
    if dtype != torch.float8_e4m3fn or latent:
        raise ValueError("scales by blocks belong to float8_e4m3fn pages of keys and values")
    if block < 16 or block > min(page_size, 256) or block & (block - 1):
        raise ValueError(f"scale_block is {block}, expected a power of two from 16 to 256, at most the page size")


def _need_gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}: the library reads device memory")


# The current stream's handle without building a torch.cuda.Stream around it (0.1 against 2.7 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch_on(device, fn, args):
    """Calls fn on the current stream of the tensors' device."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch_on(device, fn, args)
    _check(fn(*args, _raw_stream(device.index)))


def _kv_shape(pool: PagePool, table, pos, Hq, T, in_dtype, tok_start):
    if in_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"token dtype must be bfloat16 or float32, not {in_dtype}")
    if table.dim() != 2:
        raise ValueError(f"table has shape {tuple(table.shape)}, expected [B][max_pages]")
    B, max_pages = table.shape
    _need(table, "table", (B, max_pages), torch.int32, pool.device)
    if pos is not None:
        _need(pos, "pos", (B,), torch.int64, pool.device)
    if tok_start is not None:
        _need(tok_start, "tok_start", (B + 1,), torch.int32, pool.device)
    return KvShape(B, T, Hq, pool.Hkv, pool.dk, pool.dv, _DTYPE_CODES[in_dtype], _DTYPE_CODES[pool.k.dtype])


def _rows(t, name, B, T, width, dtype, device, tok_start, heads=None):
    """Token rows [B][T][heads][width] (or [N][heads][width] with tok_start), each row dense and the rows evenly
    spaced: (heads, rows, stride in elements)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    lead = 1 if tok_start is not None else 2
    if t.dim() != lead + 2 or t.shape[-1] != width or (heads is not None and t.shape[-2] != heads) or \
            (lead == 2 and tuple(t.shape[:2]) != (B, T)):
        want = f"[N][{heads or 'heads'}][{width}]" if lead == 1 else f"[{B}][{T}][{heads or 'heads'}][{width}]"
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    H = t.shape[-2]
    rows = t.shape[0] if lead == 1 else B * T
    # The distance of neighbouring rows; a length-1 axis has no say.
    if rows <= 1:
        stride = H * width
    elif lead == 1 or T == 1:
        stride = t.stride(0)
    else:
        stride = t.stride(1)
        if B > 1 and t.stride(0) != T * stride:
            raise ValueError(f"{name}: the rows of one sequence must follow those of the one before")
    if (width > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != width) or (rows > 1 and stride < H * width):
        raise ValueError(f"{name}: the values of a row must be dense")
    return H, rows, stride


def _packed_T(t, tok_start, T, name):
    """T of a call: given for packed rows, the tensor's own otherwise."""
    if tok_start is None:
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B][T][heads][width] without tok_start")
        if T is not None and T != t.shape[1]:
            raise ValueError(f"T is {T}, but {name} brings {t.shape[1]} tokens to each sequence")
        return t.shape[1]
    if T is None:
        raise ValueError("packed rows need T, the most tokens of a sequence")
    return int(T)


def rotation_axes(sections, interleaved: bool = False):
    """The axis of each rotated pair, for kv_append's axis_of: sections[a] pairs turn by axis a, section after section,
    or, interleaved, dealt to the axes in turn while each one's section lasts."""
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 4 or any(n < 0 for n in sections):
        raise ValueError("sections are the pairs of one to four axes")
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]


def _axes(axis_pos, axis_of, rot, sh, N, device, tok_start):
    """kda_axes of an append: axis_pos int64 [axes][B][T] (packed rows: [axes][N])."""
    if rot is None:
        raise ValueError("positions on axes need cos_sin")
    if not isinstance(axis_pos, torch.Tensor):
        raise TypeError("axis_pos must be a torch.Tensor")
    A = axis_pos.shape[0] if axis_pos.dim() else 0
    _need(axis_pos, "axis_pos", (A, N) if tok_start is not None else (A, sh.B, sh.T), torch.int64, device)
    of = [0] * (rot.dim // 2) if axis_of is None and A == 1 else axis_of
    if of is None or len(of) != rot.dim // 2:
        raise ValueError(f"axis_of names the axis of each of the {rot.dim // 2} rotated pairs")
    if not 1 <= A <= 4 or any(not 0 <= int(a) < A for a in of):
        raise ValueError("one to four axes, and axis_of below their number")
    return _Axes(axis_pos.data_ptr(), N, A, bytes(int(a) for a in of))


class KvAppendPlan:
    """A kv_append call validated once (see DecodePlan)."""

    def __init__(self, pool: PagePool, table, pos, k, v, dev_err, *, q=None, q_out=None, cos_sin=None, rot_start=0,
                 rot_pairs=False, axis_pos=None, axis_of=None, tok_start=None, T=None):
        dev, dt = pool.device, k.dtype
        T = _packed_T(k, tok_start, T, "k")
        sh = _kv_shape(pool, table, pos, 1 if q is None else q.shape[-2], T, dt, tok_start)
        _need(dev_err, "dev_err", (1,), torch.int32, dev)
        if (v is None) != pool.latent:
            raise ValueError("values go with pools that have value pages, and only those")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out belong together")
        if q is not None and cos_sin is None:
            raise ValueError("queries are only rotated: q needs cos_sin")
        if q is None:
            sh.Hq = sh.Hkv
        _, N, ks = _rows(k, "k", sh.B, T, pool.dk, dt, dev, tok_start, pool.Hkv)
        vs = qs = qos = 0
        if v is not None:
            vs = _rows(v, "v", sh.B, T, pool.dv, dt, dev, tok_start, pool.Hkv)
        if q is not None:
            qs = _rows(q, "q", sh.B, T, pool.dk, dt, dev, tok_start)
            qos = _rows(q_out, "q_out", sh.B, T, pool.dk, dt, dev, tok_start, q.shape[-2])
        for name, r in (("v", vs), ("q", qs), ("q_out", qos)):
            if r and r[1] != N:
                raise ValueError(f"{name} has {r[1]} rows, k has {N}")
        vs, qs, qos = (r[2] if r else 0 for r in (vs, qs, qos))
        rot = None
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise ValueError(f"cos_sin has shape {tuple(cos_sin.shape)}, expected [max_pos][rotated values]")
            _need(cos_sin, "cos_sin", cos_sin.shape, torch.float32, dev)
            rot = _Rotation(cos_sin.data_ptr(), cos_sin.shape[0], int(rot_start), cos_sin.shape[1], int(rot_pairs))
        axes = None if axis_pos is None else _axes(axis_pos, axis_of, rot, sh, N, dev, tok_start)
        if axes is None and axis_of is not None:
            raise ValueError("axis_of needs axis_pos")
        self._keep = (pool, table, pos, k, v, q, q_out, cos_sin, axis_pos, tok_start, dev_err, sh, rot, axes)
        self._device = dev
        scales = _scales(pool)
        by_ref = [None if x is None else ctypes.byref(x) for x in (rot, axes)]
        self._args = (ctypes.byref(sh), ctypes.byref(pool.c), *(() if scales is None else (scales,)), _ptr(table),
                      table.shape[1], _ptr(tok_start), N, _ptr(pos), _ptr(k), ks, _ptr(v), vs, _ptr(q), qs,
                      _ptr(q_out), qos, *(by_ref[:1] if scales is None and axes is None else by_ref), _ptr(dev_err))
        self._fn = (lib().kda_kv_append_blocks if scales is not None else
                    lib().kda_kv_append if axes is None else lib().kda_kv_append_axes)

    def __call__(self):
        _launch_on(self._device, self._fn, self._args)


def kv_append(pool: PagePool, table, pos, k, v, dev_err, **kw):
    """Append new tokens' keys (rotated) and values to the paged cache, and rotate their queries into q_out.

    Rows are [B][T][heads][width], or packed [N][heads][width] with tok_start
    (device int32 [B + 1]) and T, the most tokens of a sequence; they may be
    slices of one projection.  cos_sin: f32 [max_pos][rotated values], cosines
    then sines, rotating the values from rot_start on (rot_pairs: neighbours
    form the pairs, else halves).  axis_pos: int64 [axes][B][T] ([axes][N]),
    positions for the rotation apart from the places in the cache, of which
    axis_of (see rotation_axes) names one for each pair; one axis needs no
    axis_of.  A pool with scale_block gets the scales that the values need.
    Keywords: q, q_out, cos_sin, rot_start, rot_pairs, axis_pos, axis_of,
    tok_start, T.
    """
    KvAppendPlan(pool, table, pos, k, v, dev_err, **kw)()


def attn_workspace(pool: PagePool, table, *, Hq: int, T: int = 1):
    """A workspace for attn_decode calls with this pool, table shape, query heads and up to T new tokens."""
    sh = _kv_shape(pool, table, None, Hq, T, torch.float32 if pool.k.dtype == torch.float32 else torch.bfloat16, None)
    n = int(lib().kda_attn_workspace_bytes(ctypes.byref(sh), ctypes.byref(pool.c), table.shape[1]))
    if n == 0:
        raise ValueError("unsupported attention shape")
    return torch.empty(n, dtype=torch.uint8, device=pool.device)


def _attn_scale(pool: PagePool, scale):
    """A call's scale: the keys' width ** -0.5 where none is given."""
    if scale is not None:
        return float(scale)
    if pool.latent:
        # Not an error: latent calls without a scale have always had this one.
        warnings.warn(f"a latent cache's keys are {pool.dk} wide, but its model's scale is that of the width before "
                      f"the up-projection was absorbed: pass scale ({pool.dk} ** -0.5 is used)", stacklevel=3)
    return float(pool.dk) ** -0.5


class AttnDecodePlan:
    """An attn_decode call validated once (see DecodePlan)."""

    def __init__(self, pool: PagePool, table, pos, q, o, workspace, dev_err, *, lse=None, scale=None, window=0,
                 tok_start=None, T=None):
        dev, dt = pool.device, q.dtype
        T = _packed_T(q, tok_start, T, "q")
        sh = _kv_shape(pool, table, pos, q.shape[-2], T, dt, tok_start)
        Hq, N, qs = _rows(q, "q", sh.B, T, pool.dk, dt, dev, tok_start)
        lead = (N,) if tok_start is not None else (sh.B, T)
        _need(o, "o", lead + (Hq, pool.dv), dt, dev)
        if lse is not None:
            _need(lse, "lse", lead + (Hq,), torch.float32, dev)
        _need(dev_err, "dev_err", (1,), torch.int32, dev)
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
        self._keep = (pool, table, pos, q, o, workspace, lse, tok_start, dev_err, sh)
        self._device = dev
        scales = _scales(pool)
        self._args = (ctypes.byref(sh), ctypes.byref(pool.c), *(() if scales is None else (scales,)), _ptr(table),
                      table.shape[1], _ptr(tok_start), N, _ptr(pos), _ptr(q), qs, _attn_scale(pool, scale),
                      int(window), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(dev_err))
        self._fn = lib().kda_attn_decode if scales is None else lib().kda_attn_decode_blocks

    def __call__(self):
        _launch_on(self._device, self._fn, self._args)


def attn_decode(pool: PagePool, table, pos, q, o, workspace, dev_err, **kw):
    """Attention of the new tokens' queries over the paged cache, up to and including their own positions.

    q, o: [B][T][Hq][width], or packed [N][Hq][width] with tok_start and T;
    lse (optional): f32, o's shape without the width.  window: the tokens that a
    query sees (0: all).  scale: of the scores, the pool's dk ** -0.5 if left
    out; a latent pool's should be given, since its keys are wider than those
    that the model trained with (a warning says so).  Keywords: lse, scale,
    window, tok_start, T.
    """
    AttnDecodePlan(pool, table, pos, q, o, workspace, dev_err, **kw)()


def _need_weights(weights, name, pool, table):
    """Sums of weights f32 [B][Hkv][places], at least the table's; the stride of a row in floats."""
    if not isinstance(weights, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    B, places = table.shape[0], table.shape[1] * pool.page_size
    if weights.dim() != 3 or tuple(weights.shape[:2]) != (B, pool.Hkv) or weights.shape[2] < places:
        raise ValueError(f"{name} has shape {tuple(weights.shape)}, expected [{B}][{pool.Hkv}][{places} or more]")
    _need(weights, name, weights.shape, torch.float32, pool.device)
    return weights.shape[2]


class AttnWeightsPlan:
    """An attn_weights call validated once (see DecodePlan)."""

    def __init__(self, pool: PagePool, table, pos, q, lse, weights, dev_err, *, scale=None, window=0, tok_start=None,
                 T=None):
        dev, dt = pool.device, q.dtype
        T = _packed_T(q, tok_start, T, "q")
        sh = _kv_shape(pool, table, pos, q.shape[-2], T, dt, tok_start)
        Hq, N, qs = _rows(q, "q", sh.B, T, pool.dk, dt, dev, tok_start)
        _need(lse, "lse", ((N,) if tok_start is not None else (sh.B, T)) + (Hq,), torch.float32, dev)
        stride = _need_weights(weights, "weights", pool, table)
        _need(dev_err, "dev_err", (1,), torch.int32, dev)
        self._keep = (pool, table, pos, q, lse, weights, tok_start, dev_err, sh)
        self._device = dev
        scales = _scales(pool)
        self._args = (ctypes.byref(sh), ctypes.byref(pool.c), scales, _ptr(table), table.shape[1], _ptr(tok_start), N,
                      _ptr(pos), _ptr(q), qs, _attn_scale(pool, scale), int(window), _ptr(lse), _ptr(weights), stride,
                      _ptr(dev_err))
        self._fn = lib().kda_attn_weights

    def __call__(self):
        _launch_on(self._device, self._fn, self._args)


def attn_weights(pool: PagePool, table, pos, q, lse, weights, dev_err, **kw):
    """Adds the attention weights of the new tokens' queries to each cached token's sum.

    q, scale and window as given to attn_decode, lse as it returned it; weights:
    f32 [B][Hkv][places], summed over the rows and the query heads of a kv head.
    A new token's own sum begins with this call.  Keywords: scale, window,
    tok_start, T.
    """
    AttnWeightsPlan(pool, table, pos, q, lse, weights, dev_err, **kw)()


class KvEvictPlan:
    """A kv_evict call validated once (see DecodePlan)."""

    def __init__(self, pool: PagePool, table, length, weights, dst_table, new_length, new_weights, kept, dev_err, *,
                 recent=0):
        dev = pool.device
        sh = _kv_shape(pool, table, length, pool.Hkv, 1,
                       torch.float32 if pool.k.dtype == torch.float32 else torch.bfloat16, None)
        if dst_table.dim() != 2:
            raise ValueError(f"dst_table has shape {tuple(dst_table.shape)}, expected [B][pages]")
        _need(dst_table, "dst_table", (sh.B, dst_table.shape[1]), torch.int32, dev)
        _need(new_length, "new_length", (sh.B,), torch.int64, dev)
        stride = _need_weights(weights, "weights", pool, table)
        _need(new_weights, "new_weights", weights.shape, torch.float32, dev)
        if kept.dim() != 3:
            raise ValueError(f"kept has shape {tuple(kept.shape)}, expected [B][Hkv][tokens to keep]")
        keep, room = kept.shape[2], dst_table.shape[1] * pool.page_size
        _need(kept, "kept", (sh.B, pool.Hkv, keep), torch.int32, dev)
        if not 1 <= keep <= room:
            raise ValueError(f"kept names {keep} tokens to keep, expected 1 to the {room} that a row of dst_table holds")
        if not 0 <= int(recent) <= keep:
            raise ValueError(f"recent is {recent}, expected 0 to the {keep} tokens to keep")
        _need(dev_err, "dev_err", (1,), torch.int32, dev)
        self._keep = (pool, table, length, weights, dst_table, new_length, new_weights, kept, dev_err, sh)
        self._device = dev
        scales = _scales(pool)
        self._args = (ctypes.byref(sh), ctypes.byref(pool.c), scales, _ptr(table), table.shape[1], _ptr(length),
                      _ptr(weights), stride, keep, int(recent), _ptr(dst_table), dst_table.shape[1],
                      _ptr(new_length), _ptr(new_weights), _ptr(kept), _ptr(dev_err))
        self._fn = lib().kda_kv_evict

    def __call__(self):
        _launch_on(self._device, self._fn, self._args)


def kv_evict(pool: PagePool, table, length, weights, dst_table, new_length, new_weights, kept, dev_err, **kw):
    """Cuts every sequence longer than kept.shape[2] tokens to that many.

    length: int64 [B], the cached tokens; weights: as attn_weights left them.
    Each kv head keeps the last `recent` tokens and those of the greatest sums;
    they go, in order, to the pages of dst_table (int32 [B][pages], pages that no
    sequence of the call has), their sums to new_weights, and their places to
    kept (int32 [B][Hkv][tokens to keep]).  Shorter sequences stay where they are
    (kept -1).  new_length: int64 [B], may be length itself; new_weights may not
    be weights (the call refuses it), and later attn_weights go on with it.
    Keyword: recent.
    """
    KvEvictPlan(pool, table, length, weights, dst_table, new_length, new_weights, kept, dev_err, **kw)()
