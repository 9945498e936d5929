"""Python binding of liblily_q4 (the GB300 MLX-affine Q4 MoE hot path).

Argument marshalling only: every computation runs in the CUDA kernels of
``liblily_q4.so``, reached through its C ABI (``include/lily_q4.h``).  PyTorch
supplies device memory and streams.  There is no CPU fallback: if the library
is missing or cannot load, importing the entry points raises.

The function names are those of the C ABI:

* ``lily_q4_moe_decode(layer, x, y, topk_idx=None, topk_w=None, ws=None, stream=None)``
* ``lily_q4_moe_prefill(layer, x, y, topk_idx=None, topk_w=None, ws=None, stream=None)``
* ``lily_q4_gemv_argmax(W, x, token, logits=None, ws=None, stream=None)``
* ``lily_qk_norm_rope(op, q, k, pos, q_out, k_out, stream=None)`` with ``lily_rope_turns``;
* ``lily_kv8_append(cache, batch, k, v, ws=None, stream=None)``, ``lily_kv8_read(...)``;
* ``lily_kv8_attention(cache, batch, q, out, scale, lse=None, causal=True, window=0, ws=None,
  stream=None)`` with ``lily_kv8_attention_workspace_bytes``;
* ``lily_q4_moe_workspace_bytes``, ``lily_q4_gemv_argmax_workspace_bytes``,
  ``lily_q4_workspace_init``, ``lily_q4_workspace_status``,
  ``lily_q4_status_string``, ``lily_q4_pack``, ``lily_q4_unpack``.

Each compute wrapper returns the C status (0) or raises ``Q4Error``.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional

import numpy as np

from . import build as _build

LIB_PATH = _build.LIB

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE_TOO_SMALL = -3
ERR_CUDA = -4
ERR_TIMEOUT = -5
ERR_INDEX = -6

BF16, F16, F32 = 0, 1, 2
ROPE_SCALING = {"none": 0, "linear": 1, "yarn": 2}


class Q4Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class lily_q4_mat(C.Structure):
    _fields_ = [("w", C.c_void_p), ("s", C.c_void_p), ("b", C.c_void_p)]


class lily_q4_moe_layer(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("inter", C.c_int32),
                ("gate", lily_q4_mat), ("up", lily_q4_mat), ("down", lily_q4_mat),
                ("has_shared", C.c_int32),
                ("sh_gate", lily_q4_mat), ("sh_up", lily_q4_mat), ("sh_down", lily_q4_mat),
                ("router", C.c_void_p), ("router_bias", C.c_void_p),
                ("shared_gate", C.c_void_p),
                ("shared_bits", C.c_int32), ("router_bits", C.c_int32),
                ("router_q8", lily_q4_mat)]


class lily_qk_rope(C.Structure):
    _fields_ = [("head_dim", C.c_int32), ("rotary_dim", C.c_int32), ("interleaved", C.c_int32),
                ("dtype", C.c_int32), ("normalize", C.c_int32), ("eps", C.c_float),
                ("weight_offset", C.c_float), ("rope_scale", C.c_float),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("turns", C.c_void_p)]


class lily_kv8_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_amax", C.c_void_p),
                ("v_amax", C.c_void_p), ("n_pages", C.c_int32), ("kv_heads", C.c_int32),
                ("page", C.c_int32), ("head_dim", C.c_int32)]


class lily_kv8_batch(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("q_start", C.c_void_p), ("kv_len", C.c_void_p),
                ("table_pages", C.c_int32), ("batch", C.c_int32), ("max_q", C.c_int32),
                ("max_kv", C.c_int32)]


_lib = None


def load(path: Optional[str] = None):
    """Load liblily_q4.so (raises if it is absent: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise ImportError(f"liblily_q4.so not built ({path}); run bit_affine_quantized_mlx_gb300.build")
    L = C.CDLL(path)
    vp, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
    L.lily_q4_moe_decode.argtypes = [C.POINTER(lily_q4_moe_layer), vp, i32, vp, vp, vp, vp, sz, vp]
    L.lily_q4_moe_prefill.argtypes = L.lily_q4_moe_decode.argtypes
    L.lily_q4_gemv_argmax.argtypes = [C.POINTER(lily_q4_mat), i32, i32, vp, vp, vp, vp, sz, vp]
    L.lily_q4_moe_workspace_bytes.argtypes = [C.POINTER(lily_q4_moe_layer), i32, i32]
    L.lily_q4_moe_workspace_bytes.restype = sz
    L.lily_q4_gemv_argmax_workspace_bytes.argtypes = [i32, i32]
    L.lily_q4_gemv_argmax_workspace_bytes.restype = sz
    L.lily_q4_moe_launches.argtypes = [C.POINTER(lily_q4_moe_layer), i32, i32]
    L.lily_q4_gemv_argmax_noalloc.argtypes = [C.POINTER(lily_q4_mat), i32, i32, vp, vp, vp, vp]
    L.lily_q4_gemv_argmax_noalloc_status.argtypes = [vp]
    L.lily_q4_gemv_argmax_logprobs.argtypes = [C.POINTER(lily_q4_mat), i32, i32, vp, vp, vp, vp,
                                               vp, sz, vp]
    L.lily_q8_gemv_argmax.argtypes = L.lily_q4_gemv_argmax.argtypes
    L.lily_q8_gemv_argmax_logprobs.argtypes = L.lily_q4_gemv_argmax_logprobs.argtypes
    L.lily_q8_gemv_argmax_workspace_bytes.argtypes = [i32, i32]
    L.lily_q8_gemv_argmax_workspace_bytes.restype = sz
    L.lily_q4_workspace_init.argtypes = [vp, sz, vp]
    L.lily_q4_selftest_timeout.argtypes = [vp, sz, i32, vp]
    L.lily_q4_workspace_status.argtypes = [vp, vp]
    L.lily_q4_status_string.argtypes = [C.c_int]
    L.lily_q4_status_string.restype = C.c_char_p
    L.lily_q4_pack.argtypes = [vp, i32, i32, vp]
    L.lily_q4_unpack.argtypes = [vp, i32, i32, vp]
    i64, f64, rows = C.c_int64, C.c_double, [vp, C.c_int64, C.c_int64]
    cache, batch = C.POINTER(lily_kv8_cache), C.POINTER(lily_kv8_batch)
    L.lily_rope_turns.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    L.lily_qk_norm_rope.argtypes = [C.POINTER(lily_qk_rope), i32, i32, i32, vp, *rows, *rows, *rows,
                                    *rows, vp]
    L.lily_kv8_append.argtypes = [cache, batch, i32, i32, *rows, *rows, vp, sz, vp]
    L.lily_kv8_read.argtypes = L.lily_kv8_append.argtypes
    L.lily_kv8_attention.argtypes = [cache, batch, i32, i32, i32, C.c_float, i32, i32, *rows, *rows,
                                     vp, vp, sz, vp]
    L.lily_kv8_attention_workspace_bytes.argtypes = [cache, batch, i32, i32]
    L.lily_kv8_attention_workspace_bytes.restype = sz
    L.lily_q4_call.argtypes = [i32, C.c_char_p]
    for f in ("lily_q4_call", "lily_rope_turns", "lily_qk_norm_rope", "lily_kv8_append", "lily_kv8_read",
              "lily_kv8_attention",
              "lily_q4_moe_decode", "lily_q4_moe_prefill", "lily_q4_gemv_argmax",
              "lily_q4_workspace_init", "lily_q4_workspace_status", "lily_q4_pack",
              "lily_q4_unpack", "lily_q4_version", "lily_q4_moe_launches",
              "lily_q4_gemv_argmax_noalloc", "lily_q4_gemv_argmax_noalloc_status",
              "lily_q4_gemv_argmax_logprobs",
              "lily_q8_gemv_argmax", "lily_q4_selftest_timeout", "lily_q8_gemv_argmax_logprobs"):
        getattr(L, f).restype = C.c_int
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().lily_q4_status_string(int(status)).decode()


lily_q4_status_string = status_string


def _check(rc: int, what: str) -> int:
    if rc != OK:
        raise Q4Error(rc, what)
    return rc


# --------------------------------------------------------------------------- torch glue

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else int(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(int(stream.cuda_stream))


def to_device(a: np.ndarray, device="cuda"):
    """Upload a numpy array (uint16/uint32/uint64/float32/int32) as a torch tensor of the same bits."""
    torch = _torch()
    a = np.ascontiguousarray(a)
    view = {np.dtype(np.uint16): np.int16, np.dtype(np.uint32): np.int32,
            np.dtype(np.uint64): np.int64}.get(a.dtype)
    if view is not None:
        a = a.view(view)
    return torch.from_numpy(a).to(device)


class DeviceQ4:
    """A Q4 matrix (or expert stack) resident on the GPU."""

    def __init__(self, w, s, b):
        self.w, self.s, self.b = w, s, b

    @classmethod
    def upload(cls, m, device="cuda"):
        return cls(to_device(m.w, device), to_device(m.s, device), to_device(m.b, device))

    def c(self) -> lily_q4_mat:
        return lily_q4_mat(_ptr(self.w), _ptr(self.s), _ptr(self.b))

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.w, self.s, self.b))


class DeviceLayer:
    """One MoE layer on the GPU plus its C struct."""

    def __init__(self, H, E, k, I, gate, up, down, router, router_bias=None, sh_gate=None,
                 sh_up=None, sh_down=None, shared_gate=None, shared_bits=4, router_q8=None):
        self.H, self.E, self.k, self.I = H, E, k, I
        self.gate, self.up, self.down = gate, up, down
        self.router, self.router_bias = router, router_bias
        self.sh_gate, self.sh_up, self.sh_down = sh_gate, sh_up, sh_down
        self.shared_gate = shared_gate
        self.shared_bits = shared_bits   # 8: the shared expert's codes are 8-bit
        self.router_q8 = router_q8       # an 8-bit router (DeviceQ4 of [E, H/4] codes) or None
        self._c = None

    @property
    def has_shared(self) -> bool:
        return self.sh_gate is not None

    @classmethod
    def upload(cls, L, device="cuda"):
        up = lambda m: None if m is None else DeviceQ4.upload(m, device)
        arr = lambda a: None if a is None else to_device(a, device)
        return cls(L.H, L.E, L.k, L.I, up(L.gate), up(L.up), up(L.down), arr(L.router),
                   arr(L.router_bias), up(L.sh_gate), up(L.sh_up), up(L.sh_down),
                   arr(L.shared_gate), getattr(L, "shared_bits", 4),
                   up(getattr(L, "router_q8", None)))

    def c(self) -> lily_q4_moe_layer:
        if self._c is None:
            z = lily_q4_mat(None, None, None)
            st = lily_q4_moe_layer()
            st.hidden, st.n_experts, st.top_k, st.inter = self.H, self.E, self.k, self.I
            st.gate, st.up, st.down = self.gate.c(), self.up.c(), self.down.c()
            st.has_shared = 1 if self.has_shared else 0
            st.sh_gate = self.sh_gate.c() if self.has_shared else z
            st.sh_up = self.sh_up.c() if self.has_shared else z
            st.sh_down = self.sh_down.c() if self.has_shared else z
            st.router = _ptr(self.router)
            st.router_bias = _ptr(self.router_bias)
            st.shared_gate = _ptr(self.shared_gate)
            st.shared_bits = 8 if (self.has_shared and self.shared_bits == 8) else 4
            st.router_bits = 8 if self.router_q8 is not None else 16
            st.router_q8 = self.router_q8.c() if self.router_q8 is not None else z
            self._c = st
        return self._c

    def weight_bytes(self) -> int:
        n = self.gate.nbytes + self.up.nbytes + self.down.nbytes
        n += self.router.numel() * 2 if self.router is not None else self.router_q8.nbytes
        if self.has_shared:
            n += self.sh_gate.nbytes + self.sh_up.nbytes + self.sh_down.nbytes
            n += self.shared_gate.numel() * 2
        return n


# --------------------------------------------------------------------------- entry points

def lily_q4_moe_workspace_bytes(layer: DeviceLayer, T: int, prefill: bool = False) -> int:
    return int(load().lily_q4_moe_workspace_bytes(C.byref(layer.c()), int(T), 1 if prefill else 0))


def lily_q4_moe_launches(layer: DeviceLayer, T: int, prefill: bool = False) -> int:
    return int(load().lily_q4_moe_launches(C.byref(layer.c()), int(T), 1 if prefill else 0))


def lily_q4_gemv_argmax_workspace_bytes(N: int, K: int) -> int:
    return int(load().lily_q4_gemv_argmax_workspace_bytes(int(N), int(K)))


def new_workspace(nbytes: int, device="cuda"):
    """A zero-filled, 256-byte aligned workspace (torch allocations are 256-aligned)."""
    torch = _torch()
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def lily_q4_workspace_init(ws, stream=None) -> int:
    return _check(load().lily_q4_workspace_init(_ptr(ws), ws.numel(), _stream(stream)),
                  "lily_q4_workspace_init")


def lily_q4_workspace_status(ws, stream=None) -> int:
    """0, or ERR_TIMEOUT (returned, not raised) if a bounded device wait gave up."""
    return int(load().lily_q4_workspace_status(_ptr(ws), _stream(stream)))


def _moe(fn, name, layer, x, y, topk_idx, topk_w, ws, stream):
    T = int(x.shape[0])
    return _check(fn(C.byref(layer.c()), _ptr(x), T, _ptr(y), _ptr(topk_idx), _ptr(topk_w),
                     _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)), name)


def lily_q4_moe_decode(layer: DeviceLayer, x, y, topk_idx=None, topk_w=None, ws=None, stream=None):
    """y[T,H] (bf16 bits as int16) = decode MoE of x[T,H]; see include/lily_q4.h."""
    return _moe(load().lily_q4_moe_decode, "lily_q4_moe_decode", layer, x, y, topk_idx, topk_w,
                ws, stream)


def lily_q4_moe_prefill(layer: DeviceLayer, x, y, topk_idx=None, topk_w=None, ws=None, stream=None):
    """Prefill-chunk MoE (grouped tcgen05 GEMM); same arguments as lily_q4_moe_decode."""
    return _moe(load().lily_q4_moe_prefill, "lily_q4_moe_prefill", layer, x, y, topk_idx, topk_w,
                ws, stream)


def lily_q4_gemv_argmax(W: DeviceQ4, x, token, logits=None, ws=None, stream=None):
    N, K = int(W.w.shape[-2]), int(W.w.shape[-1]) * 8
    m = W.c()
    return _check(load().lily_q4_gemv_argmax(C.byref(m), N, K, _ptr(x), _ptr(token), _ptr(logits),
                                             _ptr(ws), ws.numel() if ws is not None else 0,
                                             _stream(stream)), "lily_q4_gemv_argmax")


def lily_q8_gemv_argmax(W, x, token, logits=None, ws=None, stream=None):
    """Greedy token of an 8-bit LM head (W: a DeviceQ4 holding uint32 [N, K/4] codes);
    see include/lily_q4.h."""
    N, K = int(W.w.shape[-2]), int(W.w.shape[-1]) * 4
    m = W.c()
    return _check(load().lily_q8_gemv_argmax(C.byref(m), N, K, _ptr(x), _ptr(token), _ptr(logits),
                                             _ptr(ws), ws.numel() if ws is not None else 0,
                                             _stream(stream)), "lily_q8_gemv_argmax")


def lily_q4_selftest_timeout(ws, which: int, stream=None):
    """Enqueue a wait that runs into its bound (which 0: grid barrier, 1: mbarrier); ws=None
    targets the fixed scratch of lily_q4_gemv_argmax_noalloc.  See include/lily_q4.h."""
    return _check(load().lily_q4_selftest_timeout(_ptr(ws), ws.numel() if ws is not None else 0,
                                                  int(which), _stream(stream)),
                  "lily_q4_selftest_timeout")


def lily_q8_gemv_argmax_logprobs(W, x, token, lse, logprobs=None, ws=None, stream=None):
    """lily_q4_gemv_argmax_logprobs for an 8-bit LM head; see include/lily_q4.h."""
    N, K = int(W.w.shape[-2]), int(W.w.shape[-1]) * 4
    m = W.c()
    return _check(load().lily_q8_gemv_argmax_logprobs(C.byref(m), N, K, _ptr(x), _ptr(token),
                                                      _ptr(lse), _ptr(logprobs), _ptr(ws),
                                                      ws.numel() if ws is not None else 0,
                                                      _stream(stream)),
                  "lily_q8_gemv_argmax_logprobs")


def lily_q8_gemv_argmax_workspace_bytes(N: int, K: int) -> int:
    return int(load().lily_q8_gemv_argmax_workspace_bytes(int(N), int(K)))


def lily_q4_gemv_argmax_logprobs(W: DeviceQ4, x, token, lse, logprobs=None, ws=None, stream=None):
    """Greedy token, full-vocabulary log-sum-exp (fp32 [1]) and optionally logprobs (fp32 [N])
    of a Q4 LM head in one pass; see include/lily_q4.h."""
    N, K = int(W.w.shape[-2]), int(W.w.shape[-1]) * 8
    m = W.c()
    return _check(load().lily_q4_gemv_argmax_logprobs(C.byref(m), N, K, _ptr(x), _ptr(token),
                                                      _ptr(lse), _ptr(logprobs), _ptr(ws),
                                                      ws.numel() if ws is not None else 0,
                                                      _stream(stream)),
                  "lily_q4_gemv_argmax_logprobs")


def lily_q4_gemv_argmax_noalloc(W: DeviceQ4, x, token, logits=None, stream=None):
    """lily_q4_gemv_argmax without a workspace, for callers that cannot allocate device
    memory: the scratch is a fixed array inside the library (see include/lily_q4.h)."""
    N, K = int(W.w.shape[-2]), int(W.w.shape[-1]) * 8
    m = W.c()
    return _check(load().lily_q4_gemv_argmax_noalloc(C.byref(m), N, K, _ptr(x), _ptr(token),
                                                     _ptr(logits), _stream(stream)),
                  "lily_q4_gemv_argmax_noalloc")


def lily_q4_gemv_argmax_noalloc_status(stream=None) -> int:
    """0, or ERR_TIMEOUT (returned, not raised) if a bounded device wait in a call of
    lily_q4_gemv_argmax_noalloc gave up since the last check; clears the record."""
    return int(load().lily_q4_gemv_argmax_noalloc_status(_stream(stream)))


def lily_q4_pack(q: np.ndarray) -> np.ndarray:
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    w = np.empty((N, K // 8), dtype=np.uint32)
    _check(load().lily_q4_pack(q.ctypes.data, N, K, w.ctypes.data), "lily_q4_pack")
    return w


def lily_q4_unpack(w: np.ndarray, N: int, K: int) -> np.ndarray:
    w = np.ascontiguousarray(w, dtype=np.uint32)
    q = np.empty((N, K), dtype=np.uint8)
    _check(load().lily_q4_unpack(w.ctypes.data, N, K, q.ctypes.data), "lily_q4_unpack")
    return q


# --------------------------------------------------------------------------- attention operators

# Filled on the first call (torch is imported lazily); looked up by name, not imported, on later ones.
_DTYPES = {}      # torch.dtype -> code
_HALVES = {}      # the 16-bit ones of them
_raw_stream = None  # device index -> handle of its current stream
_current = None     # -> the current device's index
_int32_t = _float32_t = None
_call = None      # lily_q4_call: one packed argument costs less than a score of them
_ROPE = struct.Struct("18q").pack
_ROWS = struct.Struct("13q").pack
_ATTENTION = struct.Struct("5qd12q").pack


def _first_use():
    global _raw_stream, _current, _int32_t, _float32_t, _call
    torch = _torch()
    _call = load().lily_q4_call
    _int32_t, _float32_t = torch.int32, torch.float32
    _HALVES.update({torch.bfloat16: BF16, torch.int16: BF16, torch.float16: F16})
    _DTYPES.update({**_HALVES, torch.float32: F32})
    _current = torch._C._cuda_getDevice
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _dtype_code(t, what, f32=False):
    """bf16 tensors (or their bits as int16, as elsewhere in this binding), fp16, fp32 if allowed."""
    if _raw_stream is None:
        _first_use()
    code = _DTYPES.get(t.dtype)
    if code is None or (code == F32 and not f32):
        raise Q4Error(ERR_UNSUPPORTED, f"{what}: dtype {t.dtype}")
    return code


def _require(ok, what):
    if not ok:
        raise Q4Error(ERR_INVALID_ARG, what)


def _count(n, what):
    """n as an int that fits the C ABI's 32 bits: ctypes would drop the rest in silence."""
    n = int(n)
    _require(-(1 << 31) <= n < 1 << 31, f"{what} {n}")
    return n


def _device_of(what, *tensors):
    """The index of the one device (-1: the host) that all of these are on."""
    dev = tensors[0].get_device()
    _require(all(t.get_device() == dev for t in tensors), f"{what}: tensors on several devices")
    return dev


def _elsewhere(what):
    raise Q4Error(ERR_INVALID_ARG, f"{what}: every tensor has to be on the current GPU")


def _int32(t, what):
    if _raw_stream is None:
        _first_use()
    if t.dtype is not _int32_t or not t.is_contiguous():
        raise Q4Error(ERR_INVALID_ARG, f"{what}: contiguous int32")
    return t.data_ptr()


def lily_rope_turns(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, original_len: float = 1.0, slow: float = 1.0,
                    fast: float = 32.0) -> np.ndarray:
    """The rotation table of lily_qk_norm_rope: uint64 [rotary_dim / 2] fractions of a turn for
    each position step (host only); see include/lily_q4.h.  ``to_device`` uploads it."""
    _require(scaling in ROPE_SCALING, f"lily_rope_turns: scaling {scaling!r}")
    rotary_dim = _count(rotary_dim, "lily_rope_turns: rotary_dim")
    turns = np.zeros(max(rotary_dim, 0) // 2, dtype=np.uint64)
    _check(load().lily_rope_turns(rotary_dim, float(base), ROPE_SCALING[scaling], float(factor),
                                  float(original_len), float(slow), float(fast), turns.ctypes.data),
           "lily_rope_turns")
    return turns


class QKNormRope:
    """The constants of lily_qk_norm_rope: weights and table on the GPU, and the C struct."""

    def __init__(self, head_dim, rotary_dim, turns, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, weight_offset=0.0, rope_scale=1.0, normalize=True):
        self.head_dim, self.rotary_dim = int(head_dim), int(rotary_dim)
        self.turns, self.q_weight, self.k_weight = turns, q_weight, k_weight
        self.dtype = None
        for w in (q_weight, k_weight):
            if w is None:
                continue
            _require(w.numel() == head_dim and w.is_contiguous(), "QKNormRope: weights of one head")
            code = _dtype_code(w, "QKNormRope")
            _require(self.dtype in (None, code), "QKNormRope: weights of two types")
            self.dtype = code
        if rotary_dim:
            _require(turns is not None and turns.numel() * turns.element_size() == 4 * rotary_dim
                     and turns.is_contiguous(), "QKNormRope: turns is uint64 [rotary_dim / 2]")
        # a struct for each type: without weights one operator may serve both, from several threads
        self._c = {code: lily_qk_rope(self.head_dim, self.rotary_dim, int(bool(interleaved)), code,
                                      int(bool(normalize)), float(eps), float(weight_offset),
                                      float(rope_scale), _ptr(q_weight), _ptr(k_weight),
                                      _ptr(turns) if rotary_dim else None)
                   for code in (BF16, F16) if self.dtype in (None, code)}
        self._at = {code: C.addressof(c) for code, c in self._c.items()}
        held = [t for t in (q_weight, k_weight, turns if rotary_dim else None) if t is not None]
        self._dev = _device_of("QKNormRope", *held) if held else None  # None: whatever the heads are on

    def c(self, dtype):
        """The address of the C struct for heads of this type."""
        at = self._at.get(dtype)
        if at is None:
            raise Q4Error(ERR_INVALID_ARG, "lily_qk_norm_rope: weights and heads of two types")
        return at


def lily_qk_norm_rope(op: QKNormRope, q, k, pos, q_out, k_out, stream=None):
    """Norm and rotation of every head of q [T, q_heads, D] and k [T, k_heads, D] (views with any
    token and head strides) into q_out and k_out, which may be q and k; k may be None."""
    shape, t = q.shape, q.dtype
    if len(shape) != 3:
        raise Q4Error(ERR_INVALID_ARG, f"lily_qk_norm_rope: q {tuple(shape)}")
    T, hq, d = shape
    dtype = _HALVES.get(t)
    if dtype is None:
        dtype = _dtype_code(q, "lily_qk_norm_rope")
    if q_out.shape != shape or q_out.dtype is not t or d != op.head_dim:
        raise Q4Error(ERR_INVALID_ARG, f"lily_qk_norm_rope: q {tuple(shape)}, q_out {tuple(q_out.shape)}, "
                                       f"{t}, {q_out.dtype}, heads of {op.head_dim}")
    dev = q.get_device()
    if dev < 0 or dev != _current() or q_out.get_device() != dev or op._dev not in (None, dev):
        _elsewhere("lily_qk_norm_rope")
    qi, qo = q.stride(), q_out.stride()
    if (qi[2] != 1 or qo[2] != 1) and q.numel():
        raise Q4Error(ERR_INVALID_ARG, f"lily_qk_norm_rope: strides {qi}, {qo}")
    if k is None:
        hk, words = 0, (0, 0, 0, 0, 0, 0)
    else:
        k_shape = k.shape
        hk = k_shape[1]
        if k_shape != (T, hk, d) or k_out.shape != k_shape or k.dtype is not t or k_out.dtype is not t:
            raise Q4Error(ERR_INVALID_ARG, f"lily_qk_norm_rope: k {tuple(k_shape)}, k_out {tuple(k_out.shape)}, "
                                           f"{k.dtype}, {k_out.dtype}")
        if k.get_device() != dev or k_out.get_device() != dev:
            _elsewhere("lily_qk_norm_rope: k")
        ki, ko = k.stride(), k_out.stride()
        if (ki[2] != 1 or ko[2] != 1) and k.numel():
            raise Q4Error(ERR_INVALID_ARG, f"lily_qk_norm_rope: strides {ki}, {ko}")
        words = (k.data_ptr(), ki[0], ki[1], k_out.data_ptr(), ko[0], ko[1])
    at = 0
    if op.rotary_dim:
        at = _int32(pos, "pos")
        if pos.numel() != T:
            raise Q4Error(ERR_INVALID_ARG, "lily_qk_norm_rope: pos")
        if pos.get_device() != dev:
            _elsewhere("lily_qk_norm_rope: pos")
    rc = _call(0, _ROPE(op.c(dtype), T, hq, hk, at, q.data_ptr(), qi[0], qi[1], q_out.data_ptr(), qo[0], qo[1],
                        *words, _raw_stream(dev) if stream is None else stream.cuda_stream))
    return rc if rc == OK else _check(rc, "lily_qk_norm_rope")


class KV8Cache:
    """A paged 8-bit key/value cache on the GPU: int8 codes [pages, kv_heads, page, head_dim] and
    fp32 magnitudes [pages, kv_heads] of the keys and of the values."""

    def __init__(self, k, v, k_amax, v_amax):
        _require(k.dim() == 4 and v.shape == k.shape and str(k.dtype) == str(v.dtype) == "torch.int8"
                 and k.is_contiguous() and v.is_contiguous(), "KV8Cache: codes")
        for a in (k_amax, v_amax):
            _require(tuple(a.shape) == tuple(k.shape[:2]) and str(a.dtype) == "torch.float32"
                     and a.is_contiguous(), "KV8Cache: magnitudes")
        self._dev = _device_of("KV8Cache", k, v, k_amax, v_amax)
        self.k, self.v, self.k_amax, self.v_amax = k, v, k_amax, v_amax
        self.n_pages, self.kv_heads, self.page, self.head_dim = (int(n) for n in k.shape)
        self._c = lily_kv8_cache(_ptr(k), _ptr(v), _ptr(k_amax), _ptr(v_amax), self.n_pages,
                                 self.kv_heads, self.page, self.head_dim)
        self._at = C.addressof(self._c)

    @classmethod
    def new(cls, n_pages, kv_heads, page, head_dim, device="cuda"):
        torch = _torch()
        codes = [torch.zeros((n_pages, kv_heads, page, head_dim), dtype=torch.int8, device=device)
                 for _ in range(2)]
        amax = [torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device)
                for _ in range(2)]
        return cls(*codes, *amax)

    def c(self):
        """The C struct's address."""
        return self._at


class KV8Batch:
    """The sequences of a call: block_table int32 [batch, pages], q_start int32 [batch + 1],
    kv_len int32 [batch], all on the GPU, and the host's bounds of rows and tokens a sequence."""

    def __init__(self, block_table, q_start, kv_len, max_q, max_kv):
        n = int(kv_len.numel())
        _require(block_table.dim() == 2 and block_table.shape[0] == n and q_start.numel() == n + 1,
                 "KV8Batch: block_table [batch, pages], q_start [batch + 1], kv_len [batch]")
        self._dev = _device_of("KV8Batch", block_table, q_start, kv_len)
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        self._c = lily_kv8_batch(_int32(block_table, "block_table"), _int32(q_start, "q_start"),
                                 _int32(kv_len, "kv_len"), int(block_table.shape[1]), n,
                                 _count(max_q, "KV8Batch: max_q"), _count(max_kv, "KV8Batch: max_kv"))
        self._at = C.addressof(self._c)

    def c(self):
        """The C struct's address."""
        return self._at


def _kv8_rows(which, name, cache, batch, k, v, ws, stream, f32):
    shape, step, t = k.shape, k.stride(), k.dtype
    dtype = (_DTYPES if f32 else _HALVES).get(t)
    if dtype is None:
        dtype = _dtype_code(k, name, f32)
    if v.dtype is not t:
        raise Q4Error(ERR_INVALID_ARG, f"{name}: k and v of one type")
    dev = cache._dev
    if dev < 0 or dev != _current() or batch._dev != dev or k.get_device() != dev or v.get_device() != dev:
        _elsewhere(name)
    to = v.stride()
    if (len(shape) != 3 or v.shape != shape or shape[1] != cache.kv_heads or shape[2] != cache.head_dim
            or (step[2] != 1 or to[2] != 1) and k.numel()):
        raise Q4Error(ERR_INVALID_ARG, f"{name}: k {tuple(shape)}, strides {step}, v {tuple(v.shape)}, strides {to}")
    space, size = 0, 0
    if ws is not None:
        if ws.get_device() != dev:
            _elsewhere(f"{name}: workspace")
        space, size = ws.data_ptr(), ws.nbytes
    rc = _call(which, _ROWS(cache._at, batch._at, shape[0], dtype, k.data_ptr(), step[0], step[1], v.data_ptr(), to[0],
                            to[1], space, size, _raw_stream(dev) if stream is None else stream.cuda_stream))
    return rc if rc == OK else _check(rc, name)


def lily_kv8_append(cache: KV8Cache, batch: KV8Batch, k, v, ws=None, stream=None):
    """Writes the batch's tokens k, v [T, kv_heads, head_dim] into the cache; see include/lily_q4.h."""
    return _kv8_rows(1, "lily_kv8_append", cache, batch, k, v, ws, stream, False)


def lily_kv8_read(cache: KV8Cache, batch: KV8Batch, k_out, v_out, ws=None, stream=None):
    """The values of the batch's tokens into k_out, v_out (bf16, fp16 or fp32)."""
    return _kv8_rows(2, "lily_kv8_read", cache, batch, k_out, v_out, ws, stream, True)


def lily_kv8_attention_workspace_bytes(cache: KV8Cache, batch: KV8Batch, T: int, q_heads: int) -> int:
    return int(load().lily_kv8_attention_workspace_bytes(
        C.byref(cache._c), C.byref(batch._c), _count(T, "T"), _count(q_heads, "q_heads")))


def lily_kv8_attention(cache: KV8Cache, batch: KV8Batch, q, out, scale, lse=None, causal=True,
                       window=0, ws=None, stream=None):
    """Attention of q [T, q_heads, head_dim] over the batch's cached tokens into out (same shape)
    and, if given, lse fp32 [T, q_heads]; see include/lily_q4.h."""
    shape, t = q.shape, q.dtype
    if len(shape) != 3:
        raise Q4Error(ERR_INVALID_ARG, f"lily_kv8_attention: q {tuple(shape)}")
    T, heads, d = shape
    dtype = _HALVES.get(t)
    if dtype is None:
        dtype = _dtype_code(q, "lily_kv8_attention")
    if out.shape != shape or out.dtype is not t or d != cache.head_dim:
        raise Q4Error(ERR_INVALID_ARG, f"lily_kv8_attention: q {tuple(shape)}, out {tuple(out.shape)}, {t}, "
                                       f"{out.dtype}, heads of {cache.head_dim}")
    dev = cache._dev
    if dev < 0 or dev != _current() or batch._dev != dev or q.get_device() != dev or out.get_device() != dev:
        _elsewhere("lily_kv8_attention")
    qi, qo = q.stride(), out.stride()
    if (qi[2] != 1 or qo[2] != 1) and q.numel():
        raise Q4Error(ERR_INVALID_ARG, f"lily_kv8_attention: strides {qi}, {qo}")
    at = 0
    if lse is not None:
        if lse.shape != (T, heads) or lse.dtype is not _float32_t or not lse.is_contiguous():
            raise Q4Error(ERR_INVALID_ARG, "lily_kv8_attention: lse is fp32 [T, q_heads]")
        if lse.get_device() != dev:
            _elsewhere("lily_kv8_attention: lse")
        at = lse.data_ptr()
    space, size = 0, 0
    if ws is not None:
        if ws.get_device() != dev:
            _elsewhere("lily_kv8_attention: workspace")
        space, size = ws.data_ptr(), ws.nbytes
    rc = _call(3, _ATTENTION(cache._at, batch._at, T, heads, dtype, scale, 1 if causal else 0, window,
                             q.data_ptr(), qi[0], qi[1], out.data_ptr(), qo[0], qo[1], at, space, size,
                             _raw_stream(dev) if stream is None else stream.cuda_stream))
    return rc if rc == OK else _check(rc, "lily_kv8_attention")
