"""ctypes binding of ``libzeroshard.so`` (C ABI in ``include/zero_shard.h``).

Argument marshalling only: every function has the name of the C entry point it
wraps, turns torch tensors into device pointers and Python values into C
structs, and raises :class:`ZeroShardError` on a non-zero status.  Every step
of the computation runs in the library's CUDA kernels.  There is no fallback:
if the library has not been built, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Iterable, List, Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# ZS_CHECKED=1 in the environment selects the debug build (kernel index checks)
LIB_PATH = os.path.join(_PKG, "libzeroshard_checked.so" if os.environ.get("ZS_CHECKED") == "1"
                        else "libzeroshard.so")

ZS_OK, ZS_ERR_ARG, ZS_ERR_ALIGN, ZS_ERR_CUDA, ZS_ERR_TIMEOUT = 0, -1, -2, -3, -4
ZS_MAX_ND = 1024
ZS_MAX_SHARDS = 256
ZS_NOALLOC_MAX_SHARDS = 64
ZS_QWZ_BLOCK = 256
ZS_ADAM8_BLOCK = 2048
ZS_MATH_IEEE, ZS_MATH_FAST = 0, 1
ZS_F32, ZS_F16, ZS_BF16 = 0, 1, 2
ZS_STATE_F32, ZS_STATE_U8 = 0, 1
ZS_WORK_BYTES = 65536
ZS_MAX_TENSORS = 16384
ZS_POLICY_TOTALS = 5
ZS_PREFERENCE_TOTALS = 3
ZS_PREFERENCE_SIGMOID, ZS_PREFERENCE_HINGE, ZS_PREFERENCE_SQUARED = 0, 1, 2

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F64 = ctypes.c_double


class ZeroShardError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})" + (f": {detail}" if detail else ""))


class Fragment(ctypes.Structure):
    _fields_ = [("tensor", _I32), ("shard", _I32), ("tensor_offset", _I64),
                ("shard_offset", _I64), ("length", _I64)]


class Adam(ctypes.Structure):
    _fields_ = [("lr", _F64), ("beta1", _F64), ("beta2", _F64), ("eps", _F64), ("weight_decay", _F64),
                ("math", _I32), ("reserved", _I32)]


class Shard(ctypes.Structure):
    _fields_ = [("grads", ctypes.POINTER(_P)), ("master", _P * 2), ("m", _P * 2), ("v", _P * 2),
                ("params", _P), ("n", _I64), ("qcodes", _P), ("qscales", _P)]


class Adam8Shard(ctypes.Structure):
    _fields_ = [("grads", ctypes.POINTER(_P)), ("master", _P * 2), ("m_codes", _P * 2), ("v_codes", _P * 2),
                ("m_scale", _P * 2), ("v_scale", _P * 2), ("params", _P), ("n", _I64)]


class OffloadShard(ctypes.Structure):
    _fields_ = [("grads_dev", ctypes.POINTER(_P)), ("params_dev", _P), ("grads_host", ctypes.POINTER(_P)),
                ("params_host", _P), ("master", _P * 2), ("m", _P * 2), ("v", _P * 2), ("n", _I64)]


class Sgd(ctypes.Structure):
    _fields_ = [("lr", _F64), ("momentum", _F64), ("weight_decay", _F64)]


class Logits(ctypes.Structure):
    _fields_ = [("data", _P), ("rows", _I64), ("vocab", _I64), ("row_stride", _I64), ("type", _I32),
                ("reserved", _I32), ("inv_temperature", _F64)]


class Policy(ctypes.Structure):
    _fields_ = [("clip_low", _F64), ("clip_high", _F64), ("dual_clip", _F64), ("kl_coef", _F64),
                ("entropy_coef", _F64)]


class Preference(ctypes.Structure):
    _fields_ = [("beta", _F64), ("label_smoothing", _F64), ("margin", _F64), ("kind", _I32), ("average", _I32)]


class Tensor(ctypes.Structure):
    _fields_ = [("grad", _P), ("master", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P), ("param", _P),
                ("n", _I64), ("lr_mult", _F64), ("decay_mult", _F64), ("grad_type", _I32), ("param_type", _I32),
                ("state", _I32), ("reserved", _I32)]


class Head(ctypes.Structure):
    _fields_ = [("hidden", _P), ("weight", _P), ("rows", _I64), ("vocab", _I64), ("width", _I64),
                ("hidden_stride", _I64), ("weight_stride", _I64), ("type", _I32), ("reserved", _I32),
                ("inv_temperature", _F64)]


class Norm(ctypes.Structure):
    _fields_ = [("x", _P), ("gamma", _P), ("beta", _P), ("rows", _I64), ("width", _I64), ("x_stride", _I64),
                ("type", _I32), ("param_type", _I32), ("eps", _F64)]


class Embed(ctypes.Structure):
    _fields_ = [("table", _P), ("ids", _P), ("tokens", _I64), ("vocab", _I64), ("width", _I64),
                ("table_stride", _I64), ("type", _I32), ("reserved", _I32), ("scale", _F64)]


class Ctrl(ctypes.Structure):
    _fields_ = [("loss_scale", _F64), ("beta1_pow", _F64), ("beta2_pow", _F64), ("step", _I64),
                ("skipped", _I64), ("cur", _I32), ("overflow", _I32), ("last_overflow", _I32),
                ("arrivals", ctypes.c_uint32)]


FRAGMENT_DTYPE = np.dtype([("tensor", np.int32), ("shard", np.int32), ("tensor_offset", np.int64),
                           ("shard_offset", np.int64), ("length", np.int64)])
assert FRAGMENT_DTYPE.itemsize == ctypes.sizeof(Fragment) == 32
CTRL_BYTES = ctypes.sizeof(Ctrl)

_lock = threading.Lock()
_lib = None

_SIGNATURES = {
    "zero_partition_layout": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "zero_partition_layout_device": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _I64, _P]),
    "zero_state_bytes": (_F64, [_F64, _I32, _I32, _F64]),
    "zero_shard_step": (_I32, [_P, _I32, _I32, _P, _F64, _I64, _I32, _P, _P, _P]),
    "zero_shard_step_noalloc": (_I32, [_P, _I32, _I32, _P, _F64, _I64, _I32, _P, _P]),
    "zero_ctrl_init": (_I32, [_P, _F64, _P]),
    "zero_shard_step_async": (_I32, [_P, _I32, _I32, _P, _P, _P]),
    "zero_shard_step_host": (_I32, [_P, _I32, _P, _P, _P, _P]),
    "zero_shard_reduce_adam_async": (_I32, [_P, _I32, _P, _P, _P]),
    "zero_shard_reduce_adam_all_async": (_I32, [_P, _I32, _I32, _P, _P, _P]),
    "zero_shard_grad_sqnorm_async": (_I32, [_P, _I32, _P, _P, _P, _P]),
    "zero_shard_clipped_adam_async": (_I32, [_P, _I32, _P, _F64, _P, _P, _P, _P]),
    "zero_shard_step_clipped_async": (_I32, [_P, _I32, _I32, _P, _F64, _P, _P, _P, _P]),
    "zero_shard_grad_sqnorm_all_async": (_I32, [_P, _I32, _I32, _P, _P, _P, _P]),
    "zero_shard_clipped_adam_all_async": (_I32, [_P, _I32, _I32, _P, _F64, _P, _P, _P, _P]),
    "zero_step_commit_async": (_I32, [_P, _I32, _P, _P, _P]),
    "zero_params_from_master": (_I32, [_P, _P, _I64, _P]),
    "zero_shard_step_cpu": (_I32, [_P, _I32, _I32, _P, _F64, _I64, _I32, _I32, _P]),
    "zero_shard_step_offload": (_I32, [_P, _I32, _P, _F64, _I64, _I32, _I32, _I64, _P, _P, _P]),
    "zero_shard_step_sgd_async": (_I32, [_P, _I32, _I32, _P, _P, _P]),
    "zero_shard_step_adam8_async": (_I32, [_P, _I32, _I32, _P, _P, _P]),
    "zero_adam8_maps": (_I32, [_P, _P]),
    "zero_qwz_quantize": (_I32, [_P, _I64, _P, _P, _P]),
    "zero_qwz_dequantize": (_I32, [_P, _P, _I64, _P, _P]),
    "zero_token_logp_async": (_I32, [_P, _P, _P, _P, _P, _P]),
    "zero_token_logp_grad_async": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "zero_policy_loss_async": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P]),
    "zero_preference_loss_async": (_I32, [_P, _P, _P, _I64, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "zero_head_work_bytes": (_I64, [_I64, _I64, _I64, _I64, _I32]),
    "zero_head_logp_async": (_I32, [_P, _P, _P, _P, _P, _I64, _P]),
    "zero_head_logp_grad_async": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P]),
    "zero_layer_norm_async": (_I32, [_P, _P, _I64, _P, _P]),
    "zero_layer_norm_work_bytes": (_I64, [_I64, _I64]),
    "zero_layer_norm_grad_async": (_I32, [_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _I64, _P]),
    "zero_embed_async": (_I32, [_P, _P, _I64, _P]),
    "zero_embed_work_bytes": (_I64, [_I64, _I64]),
    "zero_embed_grad_async": (_I32, [_P, _P, _I64, _P, _I64, _I32, _I32, _P, _I64, _P]),
    "zero_tensors_sqnorm_async": (_I32, [_P, _I32, _P, _P, _P, _P]),
    "zero_tensors_adamw_async": (_I32, [_P, _I32, _P, _F64, _P, _P, _P]),
    "zero_adam8_dequantize": (_I32, [_P, _P, _I64, _I32, _P, _P]),
    "zero_status_string": (ctypes.c_char_p, [_I32]),
    "zero_last_error": (ctypes.c_char_p, []),
    "zero_kernel_launches": (_I64, []),
    "zero_debug_checks": (_I32, [_P]),
    "zero_debug_wait_limit": (_I32, [_I32]),
}
EXPORTED = tuple(_SIGNATURES)


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:      # (a call's common case: no lock)
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                                   "(there is no CPU fallback)")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def status_string(status: int) -> str:
    if _lib is None and not os.path.exists(LIB_PATH):
        return str(status)
    return lib().zero_status_string(int(status)).decode()


def zero_last_error() -> str:
    return lib().zero_last_error().decode()


def zero_kernel_launches() -> int:
    return int(lib().zero_kernel_launches())


def zero_debug_checks():
    """(built with index checks, first recorded failure or 0); clears the
    record and synchronises the device."""
    out = ctypes.c_uint64(0)
    rc = int(lib().zero_debug_checks(ctypes.byref(out)))
    if rc < 0:
        _check(rc, "zero_debug_checks")
    return rc == 1, int(out.value)


def _check(rc: int, what: str):
    if rc != ZS_OK:
        raise ZeroShardError(rc, what, zero_last_error() if rc == ZS_ERR_CUDA else "")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev_ptr(t: Optional[torch.Tensor], dtype, what: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


# ------------------------------------------------------------------ layout ---

def zero_partition_layout(numels: Sequence[int], n_d: int, align: int) -> dict:
    """Host partition; returns psi, psi_pad, shard_numel, tensor_offsets,
    shard_offsets (numpy int64) and fragments (numpy structured array)."""
    L = lib()
    arr = np.ascontiguousarray(np.asarray(numels, dtype=np.int64))
    t = arr.size
    psi, psi_pad, s, nf = _I64(), _I64(), _I64(), _I64()
    toff = np.empty(t, np.int64)
    soff = np.empty(max(int(n_d), 0) + 1, np.int64)
    rc = L.zero_partition_layout(arr.ctypes.data if t else None, t, int(n_d), int(align),
                                 ctypes.byref(psi), ctypes.byref(psi_pad), ctypes.byref(s),
                                 toff.ctypes.data if t else None, soff.ctypes.data, None, 0,
                                 ctypes.byref(nf))
    _check(rc, "zero_partition_layout")
    frags = np.zeros(nf.value, FRAGMENT_DTYPE)
    rc = L.zero_partition_layout(arr.ctypes.data if t else None, t, int(n_d), int(align),
                                 ctypes.byref(psi), ctypes.byref(psi_pad), ctypes.byref(s),
                                 toff.ctypes.data if t else None, soff.ctypes.data,
                                 frags.ctypes.data if nf.value else None, nf.value, ctypes.byref(nf))
    _check(rc, "zero_partition_layout")
    return {"psi": psi.value, "psi_pad": psi_pad.value, "shard_numel": s.value,
            "tensor_offsets": toff, "shard_offsets": soff, "fragments": frags}


def zero_partition_layout_device(numels_dev: torch.Tensor, n_d: int, align: int, scalars_dev: torch.Tensor,
                                 tensor_offsets_dev: torch.Tensor, shard_offsets_dev: torch.Tensor,
                                 frags_dev: Optional[torch.Tensor], frag_cap: int, stream=None):
    """Device partition (stream-ordered).  ``frags_dev`` is a byte or int64
    tensor of at least 32 * frag_cap bytes, or None."""
    fptr = None
    if frags_dev is not None:
        if frags_dev.numel() * frags_dev.element_size() < 32 * frag_cap:
            raise ValueError("frags_dev too small for frag_cap")
        fptr = _dev_ptr(frags_dev, frags_dev.dtype, "frags_dev")
    n = numels_dev.numel()
    rc = lib().zero_partition_layout_device(
        _dev_ptr(numels_dev, torch.int64, "numels_dev") if n else None, n, int(n_d), int(align),
        _dev_ptr(scalars_dev, torch.int64, "scalars_dev"),
        _dev_ptr(tensor_offsets_dev, torch.int64, "tensor_offsets_dev") if n else None,
        _dev_ptr(shard_offsets_dev, torch.int64, "shard_offsets_dev"), fptr, int(frag_cap), _stream(stream))
    _check(rc, "zero_partition_layout_device")


def fragments_from_bytes(raw: np.ndarray, count: int) -> np.ndarray:
    """View a host copy of a device fragment table as the structured dtype."""
    return np.frombuffer(np.ascontiguousarray(raw).tobytes(), dtype=FRAGMENT_DTYPE, count=count)


def zero_state_bytes(psi: float, n_d: int, stage: int, k: float = 12.0) -> float:
    return float(lib().zero_state_bytes(float(psi), int(n_d), int(stage), float(k)))


# ------------------------------------------------------------------ shards ---

class ShardView:
    """One shard's device buffers, and the C struct that describes them.

    grads: list of n_d fp16 CUDA tensors (each >= n elements);
    master, m, v: pairs (set 0, set 1) of fp32 CUDA tensors (the same tensor
    twice means in-place); params: fp16 CUDA tensor (the shard's slice of the
    full parameter buffer); n: elements stepped; qcodes / qscales: optional
    int8 / fp32 CUDA tensors for the qwZ copy of the fp16 slice."""

    def __init__(self, grads: Sequence[torch.Tensor], master, m, v, params: torch.Tensor, n: int,
                 qcodes: Optional[torch.Tensor] = None, qscales: Optional[torch.Tensor] = None):
        self.grads = list(grads)
        self.master, self.m, self.v = tuple(master), tuple(m), tuple(v)
        self.params = params
        self.n = int(n)
        self._table = (_P * max(len(self.grads), 1))(
            *[_dev_ptr(g, torch.float16, "grads") for g in self.grads])
        self.struct = Shard()
        self.struct.grads = ctypes.cast(self._table, ctypes.POINTER(_P))
        for i in range(2):
            self.struct.master[i] = _dev_ptr(self.master[i], torch.float32, "master")
            self.struct.m[i] = _dev_ptr(self.m[i], torch.float32, "m")
            self.struct.v[i] = _dev_ptr(self.v[i], torch.float32, "v")
        self.struct.params = _dev_ptr(params, torch.float16, "params")
        self.struct.n = self.n
        self.qcodes, self.qscales = qcodes, qscales
        if (qcodes is None) != (qscales is None):
            raise ValueError("qcodes and qscales go together")
        if qcodes is not None:
            if qcodes.numel() < self.n or qscales.numel() < (self.n + ZS_QWZ_BLOCK - 1) // ZS_QWZ_BLOCK:
                raise ValueError("qwZ buffers too small")
            self.struct.qcodes = _dev_ptr(qcodes, torch.int8, "qcodes")
            self.struct.qscales = _dev_ptr(qscales, torch.float32, "qscales")

    @property
    def n_d(self) -> int:
        return len(self.grads)


def _shard_array(shards: Sequence[ShardView]):
    arr = (Shard * len(shards))()
    for i, s in enumerate(shards):
        arr[i] = s.struct
    return arr


def adam(lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
         weight_decay: float = 0.0, math: int = None) -> Adam:
    """Adam hyper-parameters; math is ZS_MATH_IEEE (default) or ZS_MATH_FAST."""
    return Adam(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                ZS_MATH_IEEE if math is None else int(math), 0)


def sgd(lr: float, momentum: float = 0.9, weight_decay: float = 0.0) -> Sgd:
    return Sgd(float(lr), float(momentum), float(weight_decay))


def zero_shard_step_sgd_async(shards: Sequence[ShardView], n_d: int, hp: Sgd, ctrl_dev: torch.Tensor, stream=None):
    """Stream-ordered step with SGD with momentum (momentum in ShardView.m)."""
    arr = _shard_array(shards)
    rc = lib().zero_shard_step_sgd_async(arr, len(shards), int(n_d), ctypes.byref(hp),
                                         _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_step_sgd_async")


# -------------------------------------------------------------- 8-bit Adam ---

class Adam8View:
    """One shard of 8-bit Adam state and the C struct that describes it.

    grads, params, n as ShardView; master: pair of fp32 CUDA tensors; m_codes,
    v_codes: pairs of uint8 CUDA tensors (>= n); m_scale, v_scale: pairs of
    fp32 CUDA tensors (>= ceil(n / ZS_ADAM8_BLOCK))."""

    def __init__(self, grads: Sequence[torch.Tensor], master, m_codes, v_codes, m_scale, v_scale,
                 params: torch.Tensor, n: int):
        self.grads = list(grads)
        self.master, self.m_codes, self.v_codes = tuple(master), tuple(m_codes), tuple(v_codes)
        self.m_scale, self.v_scale = tuple(m_scale), tuple(v_scale)
        self.params = params
        self.n = int(n)
        blocks = (self.n + ZS_ADAM8_BLOCK - 1) // ZS_ADAM8_BLOCK
        for pair in (self.m_codes, self.v_codes):
            if any(t.numel() < self.n for t in pair):
                raise ValueError("code buffers too small")
        for pair in (self.m_scale, self.v_scale):
            if any(t.numel() < blocks for t in pair):
                raise ValueError("scale buffers too small")
        self._table = (_P * max(len(self.grads), 1))(
            *[_dev_ptr(g, torch.float16, "grads") for g in self.grads])
        self.struct = Adam8Shard()
        self.struct.grads = ctypes.cast(self._table, ctypes.POINTER(_P))
        for i in range(2):
            self.struct.master[i] = _dev_ptr(self.master[i], torch.float32, "master")
            self.struct.m_codes[i] = _dev_ptr(self.m_codes[i], torch.uint8, "m_codes")
            self.struct.v_codes[i] = _dev_ptr(self.v_codes[i], torch.uint8, "v_codes")
            self.struct.m_scale[i] = _dev_ptr(self.m_scale[i], torch.float32, "m_scale")
            self.struct.v_scale[i] = _dev_ptr(self.v_scale[i], torch.float32, "v_scale")
        self.struct.params = _dev_ptr(params, torch.float16, "params")
        self.struct.n = self.n


def zero_shard_step_adam8_async(shards: Sequence[Adam8View], n_d: int, hp: Adam, ctrl_dev: torch.Tensor,
                                stream=None):
    """Stream-ordered step with 8-bit Adam states."""
    arr = (Adam8Shard * len(shards))()
    for i, s in enumerate(shards):
        arr[i] = s.struct
    rc = lib().zero_shard_step_adam8_async(arr, len(shards), int(n_d), ctypes.byref(hp),
                                           _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_step_adam8_async")


def zero_adam8_maps():
    """The library's code maps: (mag7[128], mag8[256]) float32 numpy arrays."""
    mag7 = np.empty(128, np.float32)
    mag8 = np.empty(256, np.float32)
    _check(lib().zero_adam8_maps(mag7.ctypes.data, mag8.ctypes.data), "zero_adam8_maps")
    return mag7, mag8


def zero_shard_step(shards: Sequence[ShardView], n_d: int, hp: Adam, loss_scale: float, step: int, cur: int,
                    flag_dev: torch.Tensor, stream=None) -> int:
    """Synchronous step over ``shards``; returns the overflow flag (0/1)."""
    arr = _shard_array(shards)
    ovf = _I32(-1)
    rc = lib().zero_shard_step(arr, len(shards), int(n_d), ctypes.byref(hp), float(loss_scale), int(step),
                               int(cur), _dev_ptr(flag_dev, torch.int32, "flag_dev"), _stream(stream),
                               ctypes.byref(ovf))
    _check(rc, "zero_shard_step")
    return int(ovf.value)


def zero_shard_step_noalloc(shards: Sequence[ShardView], n_d: int, hp: Adam, loss_scale: float, step: int,
                            cur: int, stream=None) -> int:
    """zero_shard_step without the caller's flag buffer: for callers that may
    not allocate device memory, the overflow words live in a small array
    compiled into the library.  Returns the overflow flag (0/1)."""
    arr = _shard_array(shards)
    ovf = _I32(-1)
    rc = lib().zero_shard_step_noalloc(arr, len(shards), int(n_d), ctypes.byref(hp), float(loss_scale),
                                       int(step), int(cur), _stream(stream), ctypes.byref(ovf))
    if rc != ZS_OK:
        raise ZeroShardError(rc, "zero_shard_step_noalloc", zero_last_error())
    return int(ovf.value)


def new_ctrl(device="cuda") -> torch.Tensor:
    """Device memory for one zs_ctrl (int64-typed so it is 8-byte aligned)."""
    return torch.zeros((CTRL_BYTES + 7) // 8, dtype=torch.int64, device=device)


def zero_ctrl_init(ctrl_dev: torch.Tensor, loss_scale: float, stream=None):
    rc = lib().zero_ctrl_init(_dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), float(loss_scale), _stream(stream))
    _check(rc, "zero_ctrl_init")


def zero_shard_step_async(shards: Sequence[ShardView], n_d: int, hp: Adam, ctrl_dev: torch.Tensor, stream=None):
    arr = _shard_array(shards)
    rc = lib().zero_shard_step_async(arr, len(shards), int(n_d), ctypes.byref(hp),
                                     _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_step_async")


def zero_shard_reduce_adam_all_async(shards: Sequence[ShardView], n_d: int, hp: Adam, ctrl_dev: torch.Tensor,
                                     stream=None):
    arr = _shard_array(shards)
    rc = lib().zero_shard_reduce_adam_all_async(arr, len(shards), int(n_d), ctypes.byref(hp),
                                                _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_reduce_adam_all_async")


class HostShardView(ShardView):
    """A shard whose gradient contributions and fp16 slice (and optional qwZ
    copy) are page-locked HOST tensors (``tensor.pin_memory()``); master/m/v
    are CUDA tensors."""

    def __init__(self, grads, master, m, v, params, n, qcodes=None, qscales=None):
        for g in list(grads) + [params]:
            if g.is_cuda or not g.is_pinned() or g.dtype != torch.float16 or not g.is_contiguous():
                raise TypeError("host shard: grads and params must be contiguous pinned fp16 host tensors")
        self.grads = list(grads)
        self.master, self.m, self.v = tuple(master), tuple(m), tuple(v)
        self.params = params
        self.n = int(n)
        self._table = (_P * max(len(self.grads), 1))(*[g.data_ptr() for g in self.grads])
        self.struct = Shard()
        self.struct.grads = ctypes.cast(self._table, ctypes.POINTER(_P))
        for i in range(2):
            self.struct.master[i] = _dev_ptr(self.master[i], torch.float32, "master")
            self.struct.m[i] = _dev_ptr(self.m[i], torch.float32, "m")
            self.struct.v[i] = _dev_ptr(self.v[i], torch.float32, "v")
        self.struct.params = params.data_ptr()
        self.struct.n = self.n
        self.qcodes, self.qscales = qcodes, qscales
        if qcodes is not None:
            for t in (qcodes, qscales):
                if t.is_cuda or not t.is_pinned():
                    raise TypeError("host shard: qwZ buffers must be pinned host tensors")
            self.struct.qcodes = qcodes.data_ptr()
            self.struct.qscales = qscales.data_ptr()


class CpuShardView(ShardView):
    """A shard whose buffers all live in host memory (CPU torch tensors), for
    the step on the host cores."""

    def __init__(self, grads, master, m, v, params, n):
        def host(t, dtype, what):
            if t.is_cuda or t.dtype != dtype or not t.is_contiguous():
                raise TypeError(f"{what}: expected a contiguous host {dtype} tensor")
            return t.data_ptr()
        self.grads = list(grads)
        self.master, self.m, self.v = tuple(master), tuple(m), tuple(v)
        self.params = params
        self.n = int(n)
        self._table = (_P * max(len(self.grads), 1))(*[host(g, torch.float16, "grads") for g in self.grads])
        self.struct = Shard()
        self.struct.grads = ctypes.cast(self._table, ctypes.POINTER(_P))
        for i in range(2):
            self.struct.master[i] = host(self.master[i], torch.float32, "master")
            self.struct.m[i] = host(self.m[i], torch.float32, "m")
            self.struct.v[i] = host(self.v[i], torch.float32, "v")
        self.struct.params = host(params, torch.float16, "params")
        self.struct.n = self.n


def zero_shard_step_cpu(shards: Sequence[ShardView], n_d: int, hp: Adam, loss_scale: float, step: int, cur: int,
                        n_threads: int = 0) -> int:
    """The shard step on the host cores (every buffer in host memory); returns
    the overflow flag.  Same results as zero_shard_step, bit for bit."""
    arr = _shard_array(shards)
    ovf = _I32(-1)
    rc = lib().zero_shard_step_cpu(arr, len(shards), int(n_d), ctypes.byref(hp), float(loss_scale), int(step),
                                   int(cur), int(n_threads), ctypes.byref(ovf))
    _check(rc, "zero_shard_step_cpu")
    return int(ovf.value)


class OffloadShardView:
    """One rank's shard for the ZeRO-Offload step: the device contributions
    and fp16 slice, page-locked host staging buffers for both, and the host
    fp32 state (two sets each of master, m, v)."""

    def __init__(self, grads_dev, params_dev, grads_host, params_host, master, m, v, n):
        def host(t, dtype, what, pinned=False):
            if t.is_cuda or t.dtype != dtype or not t.is_contiguous():
                raise TypeError(f"{what}: expected a contiguous host {dtype} tensor")
            if pinned and not t.is_pinned():
                raise TypeError(f"{what}: expected page-locked host memory (pin_memory())")
            return t.data_ptr()
        self.n = int(n)
        self.grads_dev, self.grads_host = list(grads_dev), list(grads_host)
        self.params_dev, self.params_host = params_dev, params_host
        self.master, self.m, self.v = tuple(master), tuple(m), tuple(v)
        self._dev = (_P * max(len(self.grads_dev), 1))(*[_dev_ptr(g, torch.float16, "grads_dev")
                                                          for g in self.grads_dev])
        self._host = (_P * max(len(self.grads_host), 1))(*[host(g, torch.float16, "grads_host", True)
                                                           for g in self.grads_host])
        self.struct = OffloadShard()
        self.struct.grads_dev = ctypes.cast(self._dev, ctypes.POINTER(_P))
        self.struct.grads_host = ctypes.cast(self._host, ctypes.POINTER(_P))
        self.struct.params_dev = _dev_ptr(params_dev, torch.float16, "params_dev")
        self.struct.params_host = host(params_host, torch.float16, "params_host", True)
        for i in range(2):
            self.struct.master[i] = host(self.master[i], torch.float32, "master")
            self.struct.m[i] = host(self.m[i], torch.float32, "m")
            self.struct.v[i] = host(self.v[i], torch.float32, "v")
        self.struct.n = self.n


def zero_shard_step_offload(shard: OffloadShardView, n_d: int, hp: Adam, loss_scale: float, step: int, cur: int,
                            n_threads: int = 0, chunk: int = 0, d2h_stream=None, h2d_stream=None) -> int:
    """ZeRO-Offload step: contributions to the host, the step on the host
    cores, fp16 parameters back to the device, overlapped by chunks; returns
    the overflow flag (synchronous)."""
    ovf = _I32(-1)
    rc = lib().zero_shard_step_offload(ctypes.byref(shard.struct), int(n_d), ctypes.byref(hp), float(loss_scale),
                                       int(step), int(cur), int(n_threads), int(chunk), _stream(d2h_stream),
                                       _stream(h2d_stream), ctypes.byref(ovf))
    _check(rc, "zero_shard_step_offload")
    return int(ovf.value)


def zero_shard_step_host(shard: HostShardView, n_d: int, hp: Adam, ctrl_dev: torch.Tensor, stream=None) -> int:
    """Step with host-resident contributions and fp16 shard; returns the flag."""
    ovf = _I32(-1)
    rc = lib().zero_shard_step_host(ctypes.byref(shard.struct), int(n_d), ctypes.byref(hp),
                                    _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream),
                                    ctypes.byref(ovf))
    _check(rc, "zero_shard_step_host")
    return int(ovf.value)


def zero_shard_reduce_adam_async(shard: ShardView, n_d: int, hp: Adam, ctrl_dev: torch.Tensor, stream=None):
    rc = lib().zero_shard_reduce_adam_async(ctypes.byref(shard.struct), int(n_d), ctypes.byref(hp),
                                            _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_reduce_adam_async")


def zero_step_commit_async(shards: Sequence[ShardView], hp: Adam, ctrl_dev: torch.Tensor, stream=None):
    arr = _shard_array(shards)
    rc = lib().zero_step_commit_async(arr, len(shards), ctypes.byref(hp),
                                      _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_step_commit_async")


def new_sqnorm(device="cuda") -> torch.Tensor:
    """Device accumulator for the squared gradient norm (one float64)."""
    return torch.zeros(1, dtype=torch.float64, device=device)


def zero_shard_grad_sqnorm_async(shard: ShardView, n_d: int, sqnorm_dev: torch.Tensor, ctrl_dev: torch.Tensor,
                                 g_dev: Optional[torch.Tensor] = None, stream=None):
    """Clipping pass 1 for one shard: adds its sum of squares to sqnorm_dev."""
    rc = lib().zero_shard_grad_sqnorm_async(ctypes.byref(shard.struct), int(n_d),
                                            _dev_ptr(g_dev, torch.float32, "g_dev"),
                                            _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                            _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_grad_sqnorm_async")


def zero_shard_clipped_adam_async(shard: ShardView, n_d: int, hp: Adam, max_norm: float, sqnorm_dev: torch.Tensor,
                                  ctrl_dev: torch.Tensor, g_dev: Optional[torch.Tensor] = None, stream=None):
    """Clipping pass 2 for one shard: clipped update and fp16 cast."""
    rc = lib().zero_shard_clipped_adam_async(ctypes.byref(shard.struct), int(n_d), ctypes.byref(hp),
                                             float(max_norm), _dev_ptr(g_dev, torch.float32, "g_dev"),
                                             _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                             _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_clipped_adam_async")


def zero_shard_step_clipped_async(shards: Sequence[ShardView], n_d: int, hp: Adam, max_norm: float,
                                  sqnorm_dev: torch.Tensor, ctrl_dev: torch.Tensor,
                                  g_dev: Optional[Sequence[Optional[torch.Tensor]]] = None, stream=None):
    """Whole clipped step over shards that all live on this device."""
    arr = _shard_array(shards)
    table = None
    if g_dev is not None:
        table = (_P * len(shards))(*[_dev_ptr(g, torch.float32, "g_dev") for g in g_dev])
    rc = lib().zero_shard_step_clipped_async(arr, len(shards), int(n_d), ctypes.byref(hp), float(max_norm), table,
                                             _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                             _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_step_clipped_async")


def _g_table(shards, g_dev):
    if g_dev is None:
        return None
    return (_P * len(shards))(*[_dev_ptr(g, torch.float32, "g_dev") for g in g_dev])


def zero_shard_grad_sqnorm_all_async(shards: Sequence[ShardView], n_d: int, sqnorm_dev: torch.Tensor,
                                     ctrl_dev: torch.Tensor, g_dev=None, stream=None):
    """Clipping pass 1 for a list of shards (grouped launches)."""
    arr = _shard_array(shards)
    rc = lib().zero_shard_grad_sqnorm_all_async(arr, len(shards), int(n_d), _g_table(shards, g_dev),
                                                _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                                _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_grad_sqnorm_all_async")


def zero_shard_clipped_adam_all_async(shards: Sequence[ShardView], n_d: int, hp: Adam, max_norm: float,
                                      sqnorm_dev: torch.Tensor, ctrl_dev: torch.Tensor, g_dev=None, stream=None):
    """Clipping pass 2 for a list of shards (grouped launches)."""
    arr = _shard_array(shards)
    rc = lib().zero_shard_clipped_adam_all_async(arr, len(shards), int(n_d), ctypes.byref(hp), float(max_norm),
                                                 _g_table(shards, g_dev),
                                                 _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                                 _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream(stream))
    _check(rc, "zero_shard_clipped_adam_all_async")


def zero_params_from_master(master: torch.Tensor, params: torch.Tensor, n: int, stream=None):
    rc = lib().zero_params_from_master(_dev_ptr(master, torch.float32, "master"),
                                       _dev_ptr(params, torch.float16, "params"), int(n), _stream(stream))
    _check(rc, "zero_params_from_master")


def zero_qwz_quantize(params: torch.Tensor, n: int, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """int8 codes and per-256 fp32 scales of an fp16 slice (stream-ordered)."""
    rc = lib().zero_qwz_quantize(_dev_ptr(params, torch.float16, "params"), int(n),
                                 _dev_ptr(codes, torch.int8, "codes"), _dev_ptr(scales, torch.float32, "scales"),
                                 _stream(stream))
    _check(rc, "zero_qwz_quantize")


def zero_qwz_dequantize(codes: torch.Tensor, scales: torch.Tensor, n: int, params: torch.Tensor, stream=None):
    """fp16 slice rebuilt from int8 codes and scales (the all-gather receiver)."""
    rc = lib().zero_qwz_dequantize(_dev_ptr(codes, torch.int8, "codes"), _dev_ptr(scales, torch.float32, "scales"),
                                   int(n), _dev_ptr(params, torch.float16, "params"), _stream(stream))
    _check(rc, "zero_qwz_dequantize")


# ------------------------------------------------------------------ losses ---

_TYPES = {torch.float32: ZS_F32, torch.float16: ZS_F16, torch.bfloat16: ZS_BF16}


def _stream_of(stream, t: torch.Tensor) -> Optional[int]:
    """As _stream; None: the current stream of the tensor's device (read without
    making a Stream object, which costs a small call a third of its time)."""
    if stream is None and t.is_cuda:
        return torch._C._cuda_getCurrentRawStream(t.device.index)
    return _stream(stream)


def new_work(device="cuda") -> torch.Tensor:
    """Scratch of the calls that add up over a batch (cleared; one per stream)."""
    return torch.zeros(ZS_WORK_BYTES // 8, dtype=torch.int64, device=device)


def _vector(t: Optional[torch.Tensor], dtype, n: int, what: str) -> Optional[int]:
    """Device pointer of a contiguous tensor of at least n elements, or None."""
    if t is None:
        return None
    ptr = _dev_ptr(t, dtype, what)
    if t.numel() < n:
        raise ValueError(f"{what}: {t.numel()} elements, {n} needed")
    return ptr


def _work_ptr(work: torch.Tensor) -> int:
    return _vector(work, torch.int64, ZS_WORK_BYTES // 8, "work")


def _matrix(t: torch.Tensor, what: str) -> int:
    """Device pointer of a 2-D tensor whose rows are contiguous; any row stride."""
    if t.dtype not in _TYPES:
        raise TypeError(f"{what}: expected float32, float16 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise TypeError(f"{what}: expected two dimensions with contiguous rows")
    return t.data_ptr()


def _row_stride(t: torch.Tensor) -> int:
    # a single row's stride is never used; torch may report any
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _logits(logits: torch.Tensor, inv_temperature: float) -> Logits:
    ptr = _matrix(logits, "logits")
    return Logits(ptr, logits.shape[0], logits.shape[1], _row_stride(logits), _TYPES[logits.dtype], 0,
                  float(inv_temperature))


def _dlogits(dlogits: torch.Tensor, logits: torch.Tensor):
    ptr = _matrix(dlogits, "dlogits")
    if dlogits.dtype != logits.dtype or dlogits.shape != logits.shape:
        raise TypeError("dlogits: expected the logits' type and shape")
    return ptr, _row_stride(dlogits)


def zero_token_logp_async(logits: torch.Tensor, labels: torch.Tensor, logp: torch.Tensor,
                          entropy: Optional[torch.Tensor] = None, saved: Optional[torch.Tensor] = None,
                          inv_temperature: float = 1.0, stream=None):
    """Log-probability of each row's label (and entropy) under softmax(logits *
    inv_temperature); ``saved`` ([rows, 2] fp32) is what the gradient needs."""
    x = _logits(logits, inv_temperature)
    n = x.rows
    rc = lib().zero_token_logp_async(ctypes.byref(x), _vector(labels, torch.int64, n, "labels"),
                                     _vector(logp, torch.float32, n, "logp"),
                                     _vector(entropy, torch.float32, n, "entropy"),
                                     _vector(saved, torch.float32, 2 * n, "saved"), _stream_of(stream, logits))
    _check(rc, "zero_token_logp_async")


def zero_token_logp_grad_async(logits: torch.Tensor, labels: torch.Tensor, saved: torch.Tensor,
                               dlogp: torch.Tensor, dlogits: torch.Tensor, entropy: Optional[torch.Tensor] = None,
                               dentropy: Optional[torch.Tensor] = None, inv_temperature: float = 1.0,
                               ctrl_dev: Optional[torch.Tensor] = None, stream=None):
    """Loss-scaled gradient of the logits; ``dlogits`` may be ``logits``."""
    x = _logits(logits, inv_temperature)
    n = x.rows
    out, out_stride = _dlogits(dlogits, logits)
    rc = lib().zero_token_logp_grad_async(ctypes.byref(x), _vector(labels, torch.int64, n, "labels"),
                                          _vector(saved, torch.float32, 2 * n, "saved"),
                                          _vector(dlogp, torch.float32, n, "dlogp"),
                                          _vector(entropy, torch.float32, n, "entropy"),
                                          _vector(dentropy, torch.float32, n, "dentropy"),
                                          _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), out, out_stride,
                                          _stream_of(stream, logits))
    _check(rc, "zero_token_logp_grad_async")


def policy(clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0, kl_coef: float = 0.0,
           entropy_coef: float = 0.0) -> Policy:
    """Coefficients of the clipped policy loss (dual_clip 0: off, else > 1)."""
    return Policy(float(clip_low), float(clip_high), float(dual_clip), float(kl_coef), float(entropy_coef))


def zero_policy_loss_async(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor,
                           advantages: torch.Tensor, weights: Optional[torch.Tensor], hp: Policy,
                           totals: torch.Tensor, work: torch.Tensor, ref_logp: Optional[torch.Tensor] = None,
                           logp: Optional[torch.Tensor] = None, entropy: Optional[torch.Tensor] = None,
                           token_loss: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                           inv_temperature: float = 1.0, ctrl_dev: Optional[torch.Tensor] = None, stream=None):
    """Clipped policy loss of the rows' tokens and its loss-scaled gradient
    (``dlogits`` None: forward only; it may be ``logits``).  ``logp`` [rows] is
    required; ``totals``: loss, policy term, KL, entropy, clipped share."""
    x = _logits(logits, inv_temperature)
    n = x.rows
    if logp is None:
        raise ValueError("logp: an output of [rows] fp32 is needed")
    out, out_stride = (None, 0) if dlogits is None else _dlogits(dlogits, logits)
    f32 = torch.float32
    rc = lib().zero_policy_loss_async(ctypes.byref(x), _vector(labels, torch.int64, n, "labels"),
                                      _vector(old_logp, f32, n, "old_logp"),
                                      _vector(advantages, f32, n, "advantages"),
                                      _vector(ref_logp, f32, n, "ref_logp"), _vector(weights, f32, n, "weights"),
                                      ctypes.byref(hp), _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"),
                                      _vector(logp, f32, n, "logp"), _vector(entropy, f32, n, "entropy"),
                                      _vector(token_loss, f32, n, "token_loss"), out, out_stride,
                                      _vector(totals, f32, ZS_POLICY_TOTALS, "totals"), _work_ptr(work),
                                      _stream_of(stream, logits))
    _check(rc, "zero_policy_loss_async")


_PREFERENCE_KINDS = {"sigmoid": ZS_PREFERENCE_SIGMOID, "hinge": ZS_PREFERENCE_HINGE,
                     "squared": ZS_PREFERENCE_SQUARED}


def preference(beta: float, kind="sigmoid", label_smoothing: float = 0.0, margin: float = 0.0,
               average: bool = False) -> Preference:
    """Preference loss; kind "sigmoid", "hinge", "squared" or a ZS_PREFERENCE_* value."""
    return Preference(float(beta), float(label_smoothing), float(margin), int(_PREFERENCE_KINDS.get(kind, kind)),
                      1 if average else 0)


def zero_preference_loss_async(logp: torch.Tensor, cu_seqlens: torch.Tensor, hp: Preference, loss: torch.Tensor,
                               reward: torch.Tensor, totals: torch.Tensor, work: torch.Tensor,
                               ref_logp: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                               weights: Optional[torch.Tensor] = None, dlogp: Optional[torch.Tensor] = None,
                               stream=None):
    """Paired preference loss over packed token log-probabilities (sequence 2 i
    chosen, 2 i + 1 rejected) and its gradient; ``mask`` is bool or uint8."""
    n, sequences = logp.numel(), cu_seqlens.numel() - 1
    if sequences < 0 or sequences % 2:
        raise ValueError("cu_seqlens: expected 2 n_pairs + 1 offsets")
    pairs, f32 = sequences // 2, torch.float32
    if mask is not None and mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"mask: expected bool or uint8, got {mask.dtype}")
    rc = lib().zero_preference_loss_async(_dev_ptr(logp, f32, "logp"), _vector(ref_logp, f32, n, "ref_logp"),
                                          _vector(mask, None if mask is None else mask.dtype, n, "mask"), n,
                                          _dev_ptr(cu_seqlens, torch.int64, "cu_seqlens"),
                                          _vector(weights, f32, pairs, "weights"), pairs, ctypes.byref(hp),
                                          _vector(loss, f32, pairs, "loss"),
                                          _vector(reward, f32, 2 * pairs, "reward"),
                                          _vector(dlogp, f32, n, "dlogp"),
                                          _vector(totals, f32, ZS_PREFERENCE_TOTALS, "totals"), _work_ptr(work),
                                          _stream_of(stream, logp))
    _check(rc, "zero_preference_loss_async")


# ------------------------------------------------- head, norm and embedding ---

def _work_bytes(nbytes: int, what: str, device) -> torch.Tensor:
    """Scratch of a call (uninitialised; calls that may run at once need one each)."""
    if nbytes < 0:
        raise ZeroShardError(nbytes, what, "")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _scratch(work: Optional[torch.Tensor]):
    """Pointer and size of a call's scratch."""
    return (None, 0) if work is None else (_dev_ptr(work, torch.uint8, "work"), work.numel())


def _rows(t: torch.Tensor, what: str):
    """Pointer, rows, width and row stride of a matrix, as _matrix checks it."""
    shape, stride = t.shape, t.stride()
    if t.dtype not in _TYPES or not t.is_cuda or len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        _matrix(t, what)      # says what is wrong
    # a single row's stride is never used; torch may report any
    return t.data_ptr(), shape[0], shape[1], stride[0] if shape[0] > 1 else shape[1]


def _same_matrix(t: torch.Tensor, like: torch.Tensor, what: str):
    """Pointer and row stride of a matrix of the type and shape of another."""
    ptr, _, _, stride = _rows(t, what)
    if t.dtype != like.dtype or t.shape != like.shape:
        raise TypeError(f"{what}: expected {tuple(like.shape)} of {like.dtype}, got {tuple(t.shape)} of {t.dtype}")
    return ptr, stride


def new_head_work(rows: int, width: int, vocab: int, gradient: bool = True, piece: int = 0, device="cuda") -> torch.Tensor:
    """Scratch of the head's calls; gradient: of zero_head_logp_grad_async, which
    then takes ``piece`` entries of the vocabulary at a time (0: the library's choice)."""
    return _work_bytes(int(lib().zero_head_work_bytes(int(rows), int(width), int(vocab), int(piece), 1 if gradient else 0)),
                       "zero_head_work_bytes", device)


def _head(hidden: torch.Tensor, weight: torch.Tensor, inv_temperature: float) -> Head:
    h, rows, width, h_stride = _rows(hidden, "hidden")
    w, vocab, w_width, w_stride = _rows(weight, "weight")
    if hidden.dtype != weight.dtype or hidden.dtype == torch.float32:
        raise TypeError(f"hidden, weight: expected both float16 or both bfloat16, got {hidden.dtype}, {weight.dtype}")
    if width != w_width:
        raise ValueError(f"hidden is {width} wide, weight {w_width}")
    return Head(h, w, rows, vocab, width, h_stride, w_stride, _TYPES[hidden.dtype], 0, inv_temperature)


def zero_head_logp_async(hidden: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor, logp: torch.Tensor,
                         work: torch.Tensor, saved: Optional[torch.Tensor] = None, inv_temperature: float = 1.0,
                         stream=None):
    """Log-probability of each row's label under softmax(hidden weight^T *
    inv_temperature), without the logits; ``saved`` ([rows, 2] fp32) is what the
    gradient needs.  ``work``: new_head_work(..., gradient=False) or larger."""
    h = _head(hidden, weight, inv_temperature)
    n = h.rows
    rc = lib().zero_head_logp_async(ctypes.byref(h), _vector(labels, torch.int64, n, "labels"),
                                    _vector(logp, torch.float32, n, "logp"),
                                    _vector(saved, torch.float32, 2 * n, "saved"), *_scratch(work),
                                    _stream_of(stream, hidden))
    _check(rc, "zero_head_logp_async")


def zero_head_logp_grad_async(hidden: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor, saved: torch.Tensor,
                              dlogp: torch.Tensor, dhidden: Optional[torch.Tensor], dweight: Optional[torch.Tensor],
                              work: torch.Tensor, inv_temperature: float = 1.0,
                              ctrl_dev: Optional[torch.Tensor] = None, stream=None):
    """Loss-scaled gradients of the hidden states and the vocabulary matrix
    (either may be None)."""
    h = _head(hidden, weight, inv_temperature)
    n = h.rows
    dh, dh_stride = (None, 0) if dhidden is None else _same_matrix(dhidden, hidden, "dhidden")
    dw, dw_stride = (None, 0) if dweight is None else _same_matrix(dweight, weight, "dweight")
    rc = lib().zero_head_logp_grad_async(ctypes.byref(h), _vector(labels, torch.int64, n, "labels"),
                                         _vector(saved, torch.float32, 2 * n, "saved"),
                                         _vector(dlogp, torch.float32, n, "dlogp"),
                                         _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), dh, dh_stride, dw, dw_stride,
                                         *_scratch(work), _stream_of(stream, hidden))
    _check(rc, "zero_head_logp_grad_async")


def _norm_vector(t: Optional[torch.Tensor], width: int, kind, what: str):
    """Pointer of one of a norm's vectors (None: NULL), and the type they share."""
    if t is None:
        return None, kind
    if t.dtype not in _TYPES or kind not in (None, t.dtype):
        raise TypeError(f"{what}: expected float32, float16 or bfloat16, the same for all of the norm's vectors")
    if t.numel() != width:
        raise ValueError(f"{what}: {t.numel()} elements, rows have {width}")
    return _dev_ptr(t, t.dtype, what), t.dtype


def zero_layer_norm_async(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], y: torch.Tensor,
                          saved: Optional[torch.Tensor] = None, eps: float = 1e-5, stream=None):
    """Layer norm of the rows of ``x`` into ``y`` (which may be ``x``); ``saved``
    ([rows, 2] fp32: mean, 1 / deviation) is what the gradient needs."""
    ptr, rows, width, stride = _rows(x, "x")
    g, kind = _norm_vector(gamma, width, None, "gamma")
    b, kind = _norm_vector(beta, width, kind, "beta")
    n = Norm(ptr, g, b, rows, width, stride, _TYPES[x.dtype], _TYPES.get(kind, ZS_F32), eps)
    out, out_stride = _same_matrix(y, x, "y")
    rc = lib().zero_layer_norm_async(ctypes.byref(n), out, out_stride, _vector(saved, torch.float32, 2 * rows, "saved"),
                                     _stream_of(stream, x))
    _check(rc, "zero_layer_norm_async")


def new_layer_norm_work(rows: int, width: int, device="cuda") -> torch.Tensor:
    """Scratch of zero_layer_norm_grad_async."""
    return _work_bytes(int(lib().zero_layer_norm_work_bytes(int(rows), int(width))), "zero_layer_norm_work_bytes", device)


def zero_layer_norm_grad_async(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], saved: torch.Tensor,
                               dx: Optional[torch.Tensor], dgamma: Optional[torch.Tensor], dbeta: Optional[torch.Tensor],
                               work: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the norm's input (``dx`` may be ``dy`` or ``x``), weight and
    bias; any of the three may be None."""
    ptr, rows, width, stride = _rows(x, "x")
    g, kind = _norm_vector(gamma, width, None, "gamma")
    dg, kind = _norm_vector(dgamma, width, kind, "dgamma")
    db, kind = _norm_vector(dbeta, width, kind, "dbeta")
    n = Norm(ptr, g, None, rows, width, stride, _TYPES[x.dtype], _TYPES.get(kind, ZS_F32), 0.0)
    dy_ptr, dy_stride = _same_matrix(dy, x, "dy")
    dx_ptr, dx_stride = (None, 0) if dx is None else _same_matrix(dx, x, "dx")
    rc = lib().zero_layer_norm_grad_async(ctypes.byref(n), dy_ptr, dy_stride,
                                          _vector(saved, torch.float32, 2 * rows, "saved"), dx_ptr, dx_stride, dg, db,
                                          *_scratch(work), _stream_of(stream, x))
    _check(rc, "zero_layer_norm_grad_async")


def zero_embed_async(table: torch.Tensor, ids: torch.Tensor, out: torch.Tensor, scale: float = 1.0, stream=None):
    """Rows of ``table`` at ``ids`` (any shape; out of range: zeros) times ``scale``."""
    ptr, vocab, width, stride = _rows(table, "table")
    out_ptr, rows, out_width, out_stride = _rows(out, "out")
    n = ids.numel()
    if out.dtype != table.dtype or rows != n or out_width != width:
        raise TypeError("out: expected one row of the table's type and width for each id")
    e = Embed(ptr, _dev_ptr(ids, torch.int64, "ids"), n, vocab, width, stride, _TYPES[table.dtype], 0, scale)
    _check(lib().zero_embed_async(ctypes.byref(e), out_ptr, out_stride, _stream_of(stream, table)), "zero_embed_async")


def new_embed_work(tokens: int, width: int, device="cuda") -> torch.Tensor:
    """Scratch of zero_embed_grad_async."""
    return _work_bytes(int(lib().zero_embed_work_bytes(int(tokens), int(width))), "zero_embed_work_bytes", device)


def zero_embed_grad_async(ids: torch.Tensor, dout: torch.Tensor, dtable: torch.Tensor, work: torch.Tensor,
                          scale: float = 1.0, accumulate: bool = False, stream=None):
    """Gradient of the table from that of the looked-up rows; ``accumulate`` adds to
    the rows of ``dtable`` whose ids occur and leaves the others as they are."""
    ptr, rows, width, stride = _rows(dout, "dout")
    grad, vocab, grad_width, grad_stride = _rows(dtable, "dtable")
    n = ids.numel()
    if rows != n or width != grad_width:
        raise TypeError("dout: expected one row of the table's width for each id")
    if dtable.dtype is not torch.float32 and dtable.dtype != dout.dtype:
        raise TypeError(f"dtable: expected {dout.dtype} or float32, got {dtable.dtype}")
    e = Embed(None, _dev_ptr(ids, torch.int64, "ids"), n, vocab, width, 0, _TYPES[dout.dtype], 0, scale)
    rc = lib().zero_embed_grad_async(ctypes.byref(e), ptr, stride, grad, grad_stride, _TYPES[dtable.dtype],
                                     1 if accumulate else 0, *_scratch(work), _stream_of(stream, dout))
    _check(rc, "zero_embed_grad_async")


# --------------------------------------------------------- lists of tensors ---

class TensorView:
    """One tensor of an AdamW step over a list, and the C struct that describes it.

    grad: fp32, fp16 or bf16 CUDA tensor; master: fp32, updated in place; m, v:
    both fp32, or both uint8 codes with m_scale, v_scale (fp32, one per
    ZS_ADAM8_BLOCK elements); param: fp16 or bf16 copy of the weights, or None;
    lr_mult, decay_mult: factors of the learning rate and the weight decay.
    All contiguous, of as many elements as master (any shape)."""

    def __init__(self, grad: torch.Tensor, master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                 param: Optional[torch.Tensor] = None, m_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, lr_mult: float = 1.0, decay_mult: float = 1.0):
        self.grad, self.master, self.m, self.v, self.param = grad, master, m, v, param
        self.m_scale, self.v_scale = m_scale, v_scale
        self.n = n = master.numel()
        if grad.dtype not in _TYPES:
            raise TypeError(f"grad: expected float32, float16 or bfloat16, got {grad.dtype}")
        if param is not None and param.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"param: expected float16 or bfloat16, got {param.dtype}")
        if m.dtype not in (torch.float32, torch.uint8):
            raise TypeError(f"m: expected float32 or uint8, got {m.dtype}")
        small = m.dtype == torch.uint8
        if small != (m_scale is not None) or small != (v_scale is not None):
            raise ValueError("m_scale and v_scale go with uint8 states")
        for t, what in ((grad, "grad"), (m, "m"), (v, "v"), (param, "param")):
            if t is not None and t.numel() != n:
                raise ValueError(f"{what}: {t.numel()} elements, master has {n}")
        blocks = (n + ZS_ADAM8_BLOCK - 1) // ZS_ADAM8_BLOCK
        self.struct = Tensor(
            _dev_ptr(grad, grad.dtype, "grad"), _dev_ptr(master, torch.float32, "master"), _dev_ptr(m, m.dtype, "m"),
            _dev_ptr(v, m.dtype, "v"), _vector(m_scale, torch.float32, blocks, "m_scale"),
            _vector(v_scale, torch.float32, blocks, "v_scale"),
            None if param is None else _dev_ptr(param, param.dtype, "param"), n, float(lr_mult), float(decay_mult),
            _TYPES[grad.dtype], ZS_F16 if param is None else _TYPES[param.dtype],
            ZS_STATE_U8 if small else ZS_STATE_F32, 0)


class TensorList:
    """The tensors of one step, described once: the C array is kept, the
    buffers must stay where they are (make a new list when they move)."""

    def __init__(self, views: Sequence[TensorView]):
        self.views = list(views)
        self.array = (Tensor * max(len(self.views), 1))(*[v.struct for v in self.views])

    def __len__(self) -> int:
        return len(self.views)


def zero_tensors_sqnorm_async(tensors: TensorList, sqnorm_dev: torch.Tensor, work: torch.Tensor,
                              ctrl_dev: torch.Tensor, stream=None):
    """Squared norm of the unscaled gradients into sqnorm_dev (fp64), and their
    non-finite test into the control block."""
    rc = lib().zero_tensors_sqnorm_async(tensors.array, len(tensors), _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"),
                                         _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"), _work_ptr(work),
                                         _stream_of(stream, ctrl_dev))
    _check(rc, "zero_tensors_sqnorm_async")


def zero_tensors_adamw_async(tensors: TensorList, hp: Adam, ctrl_dev: torch.Tensor, max_norm: float = 0.0,
                             sqnorm_dev: Optional[torch.Tensor] = None, stream=None):
    """AdamW step of every tensor in place, clipped to max_norm (> 0) by
    sqnorm_dev; skipped on the device if the norm pass met a non-finite value."""
    rc = lib().zero_tensors_adamw_async(tensors.array, len(tensors), ctypes.byref(hp), float(max_norm),
                                        _dev_ptr(sqnorm_dev, torch.float64, "sqnorm_dev"),
                                        _dev_ptr(ctrl_dev, torch.int64, "ctrl_dev"), _stream_of(stream, ctrl_dev))
    _check(rc, "zero_tensors_adamw_async")


def zero_adam8_dequantize(codes: torch.Tensor, scales: torch.Tensor, n: int, signed: bool, out: torch.Tensor,
                          stream=None):
    """fp32 values of an 8-bit state (signed: m; else v)."""
    n = int(n)
    rc = lib().zero_adam8_dequantize(_vector(codes, torch.uint8, n, "codes"),
                                     _vector(scales, torch.float32, (n + ZS_ADAM8_BLOCK - 1) // ZS_ADAM8_BLOCK, "scales"),
                                     n, 1 if signed else 0, _vector(out, torch.float32, n, "out"), _stream_of(stream, codes))
    _check(rc, "zero_adam8_dequantize")


def read_ctrl(ctrl_dev: torch.Tensor) -> dict:
    """Host snapshot of a device control block (synchronises the copy)."""
    raw = ctrl_dev.detach().cpu().numpy().tobytes()[:CTRL_BYTES]
    c = Ctrl.from_buffer_copy(raw)
    return {name: getattr(c, name) for name, _ in Ctrl._fields_}
