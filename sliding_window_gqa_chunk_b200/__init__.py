"""Sliding-window GQA attention over a rolling KV cache on B200 (sm_100a).

Thin Python binding of ``libswa.so`` (C ABI in ``include/swa.h``).  Each
function takes torch tensors that already live on the GPU, passes their device
pointers and sizes to the C entry point of the same name, and raises
``SwaError`` on a non-zero status.  All computation happens in the library's
CUDA kernels; nothing here computes attention, and there is no CPU fallback:
if the library is missing the import of any entry point fails loudly.

Mistral 7B, section 2 "Architectural details": sliding-window attention with
window W, a rolling buffer cache of W slots (position i in slot i mod W), and
chunked prefill (chunk <= W) followed by token-by-token decoding; query head h
reads kv head h // (Hq // Hkv).

Typical use for one layer::

    dims = Dims(batch=B, n_q_heads=32, n_kv_heads=8, head_dim=128, window=4096,
                scale=128 ** -0.5)
    kc, vc = new_cache(dims)                       # zeroed [B, Hkv, W, d] bf16
    pws = prefill_workspace(dims, max_tokens=4096)  # zeroed, reused by every call
    for chunk ...:                                  # prompt, chunk by chunk
        prefill_chunk(dims, out, q, k, v, kc, vc, start_pos, n_tokens, workspace=pws)
        cache_append(dims, kc, vc, k, v, start_pos, n_tokens)
    ws = decode_workspace(dims)
    decode(dims, out1, q1, k1, v1, kc, vc, pos, ws)  # one token per sequence

The same over a cache held in 8 bits (half the bytes of a decode step), with the
rotary positions of q and k::

    rot = new_rope(128, base=10000.0)               # table of frequencies
    cache = new_cache_q8(dims, "e4m3")
    pws = prefill_workspace_q8(dims, max_tokens=4096)
    for chunk ...:
        rope(dims, rot, q, k, q, k, start_pos, n_tokens)          # in place
        prefill_chunk_q8(dims, out, q, k, v, cache, start_pos, n_tokens, pws)
        cache_append_q8(dims, cache, k, v, start_pos, n_tokens)
    ws = decode_workspace_q8(dims)
    rope(dims, rot, q1, k1, q1, k1, pos)            # [B, 1, heads, d] views of the step's q, k
    decode_q8(dims, out1, q1, k1, v1, cache, pos, ws)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import os
import threading
from typing import Optional

import torch

__all__ = [
    "Dims", "SwaError", "load_library", "library_path", "cache_append", "prefill_chunk",
    "decode", "decode_static", "decode_workspace_size", "decode_workspace", "decode_launch_info",
    "prefill_workspace_size", "prefill_workspace", "device_status", "new_cache", "abi_version",
    "CacheQ8", "new_cache_q8", "cache_append_q8", "prefill_workspace_size_q8", "prefill_workspace_q8",
    "prefill_chunk_q8", "decode_workspace_size_q8", "decode_workspace_q8", "decode_q8", "Q8_BLOCK",
    "Rope", "new_rope", "rope",
    "SWA_OK", "SWA_ERR_INVALID_ARG", "SWA_ERR_UNSUPPORTED", "SWA_ERR_WORKSPACE_TOO_SMALL",
    "SWA_ERR_CUDA", "SWA_ERR_TIMEOUT", "SWA_ERR_DEVICE_ARG",
]

SWA_OK = 0
SWA_ERR_INVALID_ARG = 1
SWA_ERR_UNSUPPORTED = 2
SWA_ERR_WORKSPACE_TOO_SMALL = 3
SWA_ERR_CUDA = 4
SWA_ERR_TIMEOUT = 5
SWA_ERR_DEVICE_ARG = 6

_DTYPES = {"bf16": 0, "f32": 1}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libswa.so")
_lib = None
_lock = threading.Lock()


class SwaError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"libswa error {code}: {message}")
        self.code = code
        self.message = message


class _CDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("out_dtype", ctypes.c_int32)]


class _CCacheQ8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p),
                ("v_tail", ctypes.c_void_p), ("format", ctypes.c_int32)]


class _CRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float)]


# What the module _native reads of a CacheQ8 and of a Rope, at the address they keep: the C
# structure, and what it checks a call's other tensors against.
class _CacheRecord(ctypes.Structure):
    _fields_ = [("c", _CCacheQ8), ("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("window", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("device", ctypes.c_int32)]


class _RopeRecord(ctypes.Structure):
    _fields_ = [("c", _CRope), ("device", ctypes.c_int32)]


@dataclasses.dataclass(frozen=True)
class Dims:
    """Shape of one attention layer (mirrors ``swa_dims``)."""

    batch: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    window: int
    scale: float
    out_dtype: str = "f32"      # "bf16" or "f32"

    def c(self) -> _CDims:
        return _CDims(self.batch, self.n_q_heads, self.n_kv_heads, self.head_dim, self.window,
                      float(self.scale), _DTYPES[self.out_dtype])

    @property
    def _record(self) -> _CDims:
        # made once, whichever threads ask first: a call may still read it while another one asks
        record = self.__dict__.get("_record_kept")
        return record if record is not None else self.__dict__.setdefault("_record_kept", self.c())

    @functools.cached_property
    def _dims_addr(self) -> int:
        return ctypes.addressof(self._record)

    def __getstate__(self):     # a copy makes its own record
        return {k: v for k, v in self.__dict__.items() if k not in ("_record_kept", "_dims_addr")}

    @property
    def torch_out_dtype(self) -> torch.dtype:
        return torch.float32 if self.out_dtype == "f32" else torch.bfloat16


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libswa.so from the package directory (build it with
    ``python -m sliding_window_gqa_chunk_b200.csrc.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python -m sliding_window_gqa_chunk_b200.csrc.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P = ctypes.c_void_p
        I32 = ctypes.c_int32
        D = ctypes.POINTER(_CDims)
        lib.swa_cache_append.argtypes = [D, P, P, P, P, I32, P, P, P]
        lib.swa_cache_append.restype = ctypes.c_int
        lib.swa_prefill_workspace_size.argtypes = [D, I32]
        lib.swa_prefill_workspace_size.restype = ctypes.c_size_t
        lib.swa_prefill_chunk.argtypes = [D, P, P, P, P, I32, P, P, P, P, P, ctypes.c_size_t, P]
        lib.swa_prefill_chunk.restype = ctypes.c_int
        lib.swa_decode_workspace_size.argtypes = [D]
        lib.swa_decode_workspace_size.restype = ctypes.c_size_t
        lib.swa_decode_launch_info.argtypes = [D, ctypes.POINTER(I32), ctypes.POINTER(I32)]
        lib.swa_decode_launch_info.restype = ctypes.c_int
        lib.swa_decode.argtypes = [D, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.swa_decode.restype = ctypes.c_int
        lib.swa_decode_static.argtypes = [D, P, P, P, P, P, P, P, P]
        lib.swa_decode_static.restype = ctypes.c_int
        C = ctypes.POINTER(_CCacheQ8)
        lib.swa_q8_append.argtypes = [D, C, P, P, I32, P, P, P]
        lib.swa_q8_append.restype = ctypes.c_int
        lib.swa_q8_prefill_workspace_size.argtypes = [D, I32]
        lib.swa_q8_prefill_workspace_size.restype = ctypes.c_size_t
        lib.swa_q8_prefill_chunk.argtypes = [D, P, P, P, P, I32, C, P, P, P, ctypes.c_size_t, P]
        lib.swa_q8_prefill_chunk.restype = ctypes.c_int
        lib.swa_q8_decode_workspace_size.argtypes = [D]
        lib.swa_q8_decode_workspace_size.restype = ctypes.c_size_t
        lib.swa_q8_decode.argtypes = [D, P, P, P, P, C, P, P, ctypes.c_size_t, P]
        lib.swa_q8_decode.restype = ctypes.c_int
        lib.swa_rope.argtypes = [D, ctypes.POINTER(_CRope), P, P, P, P, ctypes.c_int64, ctypes.c_int64,
                                 I32, P, P, I32, P]
        lib.swa_rope.restype = ctypes.c_int
        lib.swa_device_status.argtypes = [P]
        lib.swa_device_status.restype = ctypes.c_int
        lib.swa_last_error.argtypes = []
        lib.swa_last_error.restype = ctypes.c_char_p
        lib.swa_abi_version.argtypes = []
        lib.swa_abi_version.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(rc: int) -> None:
    if rc != SWA_OK:
        msg = load_library().swa_last_error().decode(errors="replace")
        raise SwaError(rc, msg)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libswa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def abi_version() -> int:
    return int(load_library().swa_abi_version())


def new_cache(dims: Dims, device="cuda"):
    """Zeroed (k_cache, v_cache), each [B, Hkv, W, d] bf16 (zero = finite for unwritten slots)."""
    shape = (dims.batch, dims.n_kv_heads, dims.window, dims.head_dim)
    return (torch.zeros(shape, dtype=torch.bfloat16, device=device),
            torch.zeros(shape, dtype=torch.bfloat16, device=device))


def cache_append(dims: Dims, k_cache, v_cache, k, v, start_pos, n_tokens, stream=None) -> None:
    """swa_cache_append: k/v [B, T, Hkv, d] bf16 into the [B, Hkv, W, d] caches at slot p mod W."""
    cd = dims.c()
    _check(load_library().swa_cache_append(
        ctypes.byref(cd), _ptr(k_cache), _ptr(v_cache), _ptr(k), _ptr(v), int(k.shape[1]),
        _ptr(start_pos), _ptr(n_tokens), _stream(stream)))


def prefill_workspace_size(dims: Dims, max_tokens: int) -> int:
    cd = dims.c()
    return int(load_library().swa_prefill_workspace_size(ctypes.byref(cd), int(max_tokens)))


def prefill_workspace(dims: Dims, max_tokens: int, device="cuda") -> torch.Tensor:
    """A zero-filled prefill workspace for these dims (reusable by every later
    call with the same dims on the same stream; calls leave it zero-filled)."""
    return torch.zeros(prefill_workspace_size(dims, max_tokens), dtype=torch.uint8, device=device)


def prefill_chunk(dims: Dims, out, q, k, v, k_cache, v_cache, start_pos, n_tokens,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """swa_prefill_chunk: out [B, T, Hq, d] = attention of chunk q over (cache + chunk k/v).

    ``workspace`` (from ``prefill_workspace``) lets the kernel run persistently
    and split the key ranges of its last query tiles across SMs; without it the
    call launches one CTA per query tile and head pair."""
    cd = dims.c()
    ws_bytes = 0 if workspace is None else int(workspace.numel() * workspace.element_size())
    _check(load_library().swa_prefill_chunk(
        ctypes.byref(cd), _ptr(out), _ptr(q), _ptr(k), _ptr(v), int(q.shape[1]),
        _ptr(k_cache), _ptr(v_cache), _ptr(start_pos), _ptr(n_tokens), _ptr(workspace),
        ws_bytes, _stream(stream)))


def decode_workspace_size(dims: Dims) -> int:
    cd = dims.c()
    return int(load_library().swa_decode_workspace_size(ctypes.byref(cd)))


def decode_workspace(dims: Dims, device="cuda") -> torch.Tensor:
    """A zero-filled decode workspace of decode_workspace_size(dims) bytes."""
    return torch.zeros(decode_workspace_size(dims), dtype=torch.uint8, device=device)


def decode_launch_info(dims: Dims):
    """(n_splits, n_launches) of swa_decode for these dims (host only)."""
    cd = dims.c()
    ns, nl = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().swa_decode_launch_info(ctypes.byref(cd), ctypes.byref(ns), ctypes.byref(nl)))
    return int(ns.value), int(nl.value)


def decode(dims: Dims, out, q, k_new, v_new, k_cache, v_cache, pos, workspace,
           stream=None) -> None:
    """swa_decode: append (k_new, v_new) at slot pos mod W, then out [B, Hq, d] = attention."""
    cd = dims.c()
    _check(load_library().swa_decode(
        ctypes.byref(cd), _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
        _ptr(v_cache), _ptr(pos), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        _stream(stream)))


def decode_static(dims: Dims, out, q, k_new, v_new, k_cache, v_cache, pos, stream=None) -> None:
    """swa_decode_static: the same decode step as ``decode`` with no workspace argument.

    For callers that cannot allocate device memory (an engine with a fixed,
    pre-planned arena, or code that only receives tensor pointers): the scratch
    comes from a 4 MiB array built into the library, shared by every call on a
    device.  Calls that may overlap on the GPU race on it; the first call on a
    device should come before any stream capture.
    """
    cd = dims.c()
    _check(load_library().swa_decode_static(
        ctypes.byref(cd), _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
        _ptr(v_cache), _ptr(pos), _stream(stream)))


def device_status(stream=None) -> None:
    """Synchronise and raise SwaError if a kernel flagged a timeout or a bad device argument."""
    _check(load_library().swa_device_status(_stream(stream)))


# ---- the 8-bit rolling cache and the rotary positions ----
#
# These calls check their tensors (type, shape, device, density) before anything
# is launched, and run on the device that the tensors are on.  The checks and the
# call itself are in the module _native (csrc/binding.cpp).

Q8_BLOCK = 64                                   # slots that share a scale
_Q8_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}
_Q8_DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_binding = None


def _load_binding():
    """The module that takes tensors to the library's calls; like the library, it must have been built."""
    global _binding
    lib = load_library()
    try:
        from . import _native as module
    except ImportError as e:
        raise ImportError(f"{_HERE}/_native.so cannot be loaded ({e}): build it with "
                          "`python -m sliding_window_gqa_chunk_b200.csrc.build`") from e
    calls = (lib.swa_q8_append, lib.swa_q8_prefill_chunk, lib.swa_q8_decode, lib.swa_rope)
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in calls))
    _binding = module
    return module


def _arg(name: str, t: torch.Tensor, shape, dtype: torch.dtype, dev: int) -> int:
    """Address of a dense tensor of this shape, type and device; ValueError for another."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))


def _device_of(name: str, t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return t.get_device()


def _handle(stream, dev: int) -> int:
    """A stream's handle (a torch stream of another device is refused)."""
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"stream of cuda:{stream.device_index} for tensors on cuda:{dev}")
    return _stream(stream).value or 0


@dataclasses.dataclass(frozen=True, eq=False)
class CacheQ8:
    """One layer's rolling cache in 8 bits (mirrors ``swa_q8_cache``).

    ``k``, ``v`` [B, Hkv, W, d] float8_e4m3fn or int8; ``k_scale``, ``v_scale``
    [B, Hkv, ceil(W / 64)] float32: a row stands for its 8-bit numbers times the
    scale of its block of 64 slots (the calls write powers of two; blocks filled
    from elsewhere may have any normal scale > 0, of which a chunk that is written
    out in bf16 rounds the products); ``k_tail``, ``v_tail`` [B, Hkv, 64, d] bf16:
    the rows so far of the block being filled.  The tensors are used where they
    are; keep the handle and pass it to every call.
    """

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_tail: torch.Tensor
    v_tail: torch.Tensor

    def __post_init__(self):
        if self.k.dim() != 4 or self.k.dtype not in _Q8_FORMATS:
            raise ValueError(f"k: expected [B, Hkv, W, d] float8_e4m3fn or int8, got {self.k.dtype} {tuple(self.k.shape)}")
        B, H, W, d = self.k.shape
        dev = _device_of("k", self.k)
        blocks, tail = (B, H, -(-W // Q8_BLOCK)), (B, H, Q8_BLOCK, d)
        ptrs = [_arg("k", self.k, self.k.shape, self.k.dtype, dev), _arg("v", self.v, self.k.shape, self.k.dtype, dev),
                _arg("k_scale", self.k_scale, blocks, torch.float32, dev),
                _arg("v_scale", self.v_scale, blocks, torch.float32, dev),
                _arg("k_tail", self.k_tail, tail, torch.bfloat16, dev),
                _arg("v_tail", self.v_tail, tail, torch.bfloat16, dev)]
        record = _CacheRecord(_CCacheQ8(*ptrs, _Q8_FORMATS[self.k.dtype]), B, H, W, d, dev)
        object.__setattr__(self, "_record", record)
        object.__setattr__(self, "_cache_addr", ctypes.addressof(record))

    def __reduce__(self):       # a copy makes its own record
        return CacheQ8, (self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail)


def new_cache_q8(dims: Dims, format: str = "e4m3", device="cuda") -> CacheQ8:
    """A zeroed 8-bit cache; ``format`` is "e4m3" or "int8" (finer for values of one
    size, coarser for the small ones of a block that holds large ones)."""
    if format not in _Q8_DTYPES:
        raise ValueError(f"format {format!r}: expected one of {sorted(_Q8_DTYPES)}")
    B, H, W, d = dims.batch, dims.n_kv_heads, dims.window, dims.head_dim

    def zeros(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)

    ring, scales, tail = (B, H, W, d), (B, H, -(-W // Q8_BLOCK)), (B, H, Q8_BLOCK, d)
    return CacheQ8(*(zeros(ring, torch.int8).view(_Q8_DTYPES[format]) for _ in range(2)),
                   *(zeros(scales, torch.float32) for _ in range(2)),
                   *(zeros(tail, torch.bfloat16) for _ in range(2)))


def cache_append_q8(dims: Dims, cache: CacheQ8, k, v, start_pos, n_tokens, stream=None) -> None:
    """swa_q8_append: k/v [B, T, Hkv, d] bf16 into the 8-bit cache, blocks that they fill up
    rounded, the rest in the tail."""
    if stream is not None:
        stream = _handle(stream, cache._record.device)
    rc = (_binding or _load_binding()).append(dims, cache, k, v, start_pos, n_tokens, stream)
    if rc:
        _check(rc)


def prefill_workspace_size_q8(dims: Dims, max_tokens: int) -> int:
    return int(load_library().swa_q8_prefill_workspace_size(ctypes.byref(dims._record), int(max_tokens)))


def prefill_workspace_q8(dims: Dims, max_tokens: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for prefill_chunk_q8 with these dims (one serves all layers in turn)."""
    return torch.zeros(prefill_workspace_size_q8(dims, max_tokens), dtype=torch.uint8, device=device)


def prefill_chunk_q8(dims: Dims, out, q, k, v, cache: CacheQ8, start_pos, n_tokens, workspace,
                     stream=None) -> None:
    """swa_q8_prefill_chunk: out [B, T, Hq, d] = attention of chunk q over (8-bit cache + chunk k/v)."""
    if stream is not None:
        stream = _handle(stream, cache._record.device)
    rc = (_binding or _load_binding()).prefill(dims, out, q, k, v, cache, start_pos, n_tokens, workspace, stream)
    if rc:
        _check(rc)


def decode_workspace_size_q8(dims: Dims) -> int:
    return int(load_library().swa_q8_decode_workspace_size(ctypes.byref(dims._record)))


def decode_workspace_q8(dims: Dims, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of decode_workspace_size_q8(dims) bytes."""
    return torch.zeros(decode_workspace_size_q8(dims), dtype=torch.uint8, device=device)


def decode_q8(dims: Dims, out, q, k_new, v_new, cache: CacheQ8, pos, workspace, stream=None) -> None:
    """swa_q8_decode: take (k_new, v_new) in at position pos, then out [B, Hq, d] = attention."""
    if stream is not None:
        stream = _handle(stream, cache._record.device)
    rc = (_binding or _load_binding()).decode(dims, out, q, k_new, v_new, cache, pos, workspace, stream)
    if rc:
        _check(rc)


@dataclasses.dataclass(frozen=True, eq=False)
class Rope:
    """Rotary positions: ``inv_freq`` float32 [r / 2] on the GPU turns the first r elements of each
    head, as pairs (i, i + r / 2) or, ``interleaved``, (2 i, 2 i + 1); turned elements are
    multiplied by ``factor``."""

    inv_freq: torch.Tensor
    interleaved: bool = False
    factor: float = 1.0

    def __post_init__(self):
        dev = _device_of("inv_freq", self.inv_freq)
        n = self.inv_freq.numel()
        ptr = _arg("inv_freq", self.inv_freq, (n,), torch.float32, dev)
        record = _RopeRecord(_CRope(ptr, 2 * n, int(self.interleaved), float(self.factor)), dev)
        object.__setattr__(self, "_record", record)
        object.__setattr__(self, "_rope_addr", ctypes.addressof(record))

    def __reduce__(self):       # a copy makes its own record
        return Rope, (self.inv_freq, self.interleaved, self.factor)


def new_rope(rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
             scale: float = 1.0, original_length: int = 4096, device="cuda") -> Rope:
    """The table base ** (-2 i / rotary_dim), for contexts `scale` times the length a model was
    trained at (``original_length``) in one of the usual forms:

    * "none";
    * "linear": all positions divided by scale;
    * "base": base raised so that the slowest pair turns scale times slower and the fastest as before;
    * "yarn": pairs that turn more than 32 times over original_length are kept, those that turn less
      than once are slowed by scale, and turned elements are multiplied by 0.1 ln(scale) + 1.  Between,
      the share that is slowed grows linearly with the pair's index, from the last index (rounded down)
      with 32 turns to the first (rounded up) with one, as models with such tables are trained.  (The
      method's paper writes the ramp in the number of turns: for that, pass Rope a table.)
    """
    if scaling not in ("none", "linear", "base", "yarn"):
        raise ValueError(f"scaling {scaling!r}: expected none, linear, base or yarn")
    if rotary_dim < 2 or rotary_dim % 2 or not base > 0 or not scale > 0 or not original_length > 0:
        raise ValueError("rotary_dim must be even and positive, base, scale and original_length positive")
    if scaling == "yarn" and not base > 1:
        raise ValueError("yarn needs a base above 1: the pairs' turns have to fall with their index")
    if scaling == "base" and rotary_dim > 2:
        base = base * scale ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    factor = 1.0
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "yarn":
        def index(turns):       # of the pair that turns so often: original_length base ** (-2 i / rotary_dim) = 2 pi turns
            return rotary_dim / 2 * math.log(original_length / (2 * math.pi * turns)) / math.log(base)

        low, high = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rotary_dim - 1)
        slowed = ((torch.arange(rotary_dim // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        # where the ramp's ends fall outside the table
        turns = original_length * freq / (2 * math.pi)
        slowed = torch.where(turns > 32, 0.0, torch.where(turns < 1, 1.0, slowed))
        freq = freq * (1 - slowed) + freq / scale * slowed
        factor = 0.1 * math.log(scale) + 1 if scale > 1 else 1.0
    return Rope(freq.float().to(device), interleaved, factor)


def rope(dims: Dims, spec: Rope, q_out, k_out, q, k, start_pos, n_tokens=None, transpose: bool = False,
         stream=None) -> None:
    """swa_rope: q [B, T, Hq, d] and k [B, T, Hkv, d] (bf16; heads inside a packed projection are
    taken as they lie) turned to positions start_pos[b] + t, into dense q_out and k_out (which may be
    q and k if those are dense).  k and k_out may be None.  ``n_tokens`` None: all T rows.
    ``transpose`` gives the gradient for q and k from that for q_out and k_out."""
    if stream is not None:
        stream = _handle(stream, spec._record.device)
    rc = (_binding or _load_binding()).rope(dims, spec, q_out, k_out, q, k, start_pos, n_tokens, transpose, stream)
    if rc:
        _check(rc)
