"""Python binding of the ARL2 C ABI (include/arl2.h), through ctypes.

Argument marshalling only: each function checks shapes, dtypes and devices of torch
tensors and passes raw pointers and the current CUDA stream to libarl2.so, where every
step of the layer runs in hand-written sm_100a kernels. There is no fallback: if the
library is missing or cannot load, importing the binding's functions raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libarl2.so")

ARL2_OK, ARL2_ERR_INVALID_ARG, ARL2_ERR_UNSUPPORTED, ARL2_ERR_OOM = 0, 1, 2, 3
ARL2_ERR_CUDA, ARL2_ERR_TIMEOUT, ARL2_ERR_STATE = 4, 5, 6
STATUS_NAMES = {
    0: "ARL2_OK", 1: "ARL2_ERR_INVALID_ARG", 2: "ARL2_ERR_UNSUPPORTED", 3: "ARL2_ERR_OOM",
    4: "ARL2_ERR_CUDA", 5: "ARL2_ERR_TIMEOUT", 6: "ARL2_ERR_STATE",
}

_I64 = ctypes.c_int64
_P, _I, _S, _U64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
# name -> (restype, argtypes); the names and order follow include/arl2.h.
SIGNATURES = {
    "arl2_create": (_S, [_I, _I, _I, _I, _I, ctypes.POINTER(_P)]),
    "arl2_set_feature_maps": (_S, [_P, _P, _P, _P, _P]),
    "arl2_frame_query": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_frame_commit": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_frame_query_host": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_frame_commit_host": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_frame_clean_pass": (_S, [_P, _P, _P, _P, _P, _P, _P, _P]),
    "arl2_set_clean_split": (_S, [_P, _I]),
    "arl2_clean_split": (_I, [_P]),
    "arl2_frame_query_token": (_S, [_P, _P, _P, _P, _P, _P, _P, _P]),
    "arl2_frame_commit_token": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_set_gate_weights": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_frame_gates": (_S, [_P, _P, _P, _P, _P]),
    "arl2_frame_commit_gated": (_S, [_P, _P, _P, _P, _P]),
    "arl2_reset": (_S, [_P, _P]),
    "arl2_get_state": (_S, [_P, _P, _P]),
    "arl2_set_state": (_S, [_P, _P, _P]),
    "arl2_frame_index": (_I, [_P]),
    "arl2_get_status": (_S, [_P]),
    "arl2_set_wait_timeout_ns": (_S, [_P, _U64]),
    "arl2_test_stall_next_query": (_S, [_P]),
    "arl2_set_launch_overlap": (_S, [_P, ctypes.c_int]),
    "arl2_memory_bytes": (_SZ, [_P]),
    "arl2_destroy": (None, [_P]),
    "arl2_frame_commit_noalloc": (_S, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "arl2_kvcache_create": (_S, [_I, _I, _I, _I, _I, ctypes.POINTER(_P)]),
    "arl2_kvcache_query": (_S, [_P, _P, _P, _P, _P, _P]),
    "arl2_kvcache_commit": (_S, [_P, _P, _P, _P]),
    "arl2_kvcache_reset": (_S, [_P]),
    "arl2_kvcache_frames": (_I, [_P]),
    "arl2_kvcache_get_status": (_S, [_P]),
    "arl2_kvcache_memory_bytes": (_SZ, [_P]),
    "arl2_kvcache_destroy": (None, [_P]),
    "arl2_attn_create": (_S, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_P)]),
    "arl2_attn_forward": (_S, [_P, _P, _P]),
    "arl2_attn_backward": (_S, [_P, _P, _P]),
    "arl2_attn_get_status": (_S, [_P]),
    "arl2_attn_memory_bytes": (_SZ, [_P]),
    "arl2_attn_destroy": (None, [_P]),
    "arl2_scan_workspace_bytes": (_SZ, [_P]),
    "arl2_scan_forward": (_S, [_P, _P]),
    "arl2_scan_backward": (_S, [_P, _P]),
}

# The argument structs of the training operators, as byte layouts (include/arl2.h): packing one is
# several times faster than filling a ctypes.Structure, which small calls would notice.
_ATTN_SHAPE = "iiPPiif4x"
_TENSOR = "P3q"
_ATTN_FWD = struct.Struct(_ATTN_SHAPE + 4 * _TENSOR + "P")
_ATTN_BWD = struct.Struct(_ATTN_SHAPE + 8 * _TENSOR + "P")

_SCAN_SHAPE = "6iP"
_SCAN_FWD = struct.Struct(_SCAN_SHAPE + "6P7q")
_SCAN_BWD = struct.Struct(_SCAN_SHAPE + "9P9q")

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # arl2_dtype

_lib: Optional[ctypes.CDLL] = None


class Arl2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} failed: {STATUS_NAMES.get(status, status)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libarl2.so and declare its signatures. Raises ImportError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m softmax_attention_ar_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != ARL2_OK:
        raise Arl2Error(status, where)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> int:
    """_dev for arguments that must be device memory (the kernels read them through TMA)."""
    p = _dev(t, dtype, shape, name)
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return p


def _host(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> int:
    """_dev for arguments of the host-buffer calls, which must be host memory."""
    p = _dev(t, dtype, shape, name)
    if t.is_cuda:
        raise ValueError(f"{name}: expected a host (CPU) tensor")
    return p


# ------------------------------------------------------------------ raw C-ABI mirrors
def arl2_create(H: int, T: int, d_k: int, d_v: int, B: int) -> ctypes.c_void_p:
    out = _P()
    _check(load_library().arl2_create(H, T, d_k, d_v, B, ctypes.byref(out)), "arl2_create")
    return out


def arl2_destroy(ctx) -> None:
    load_library().arl2_destroy(ctx)


class ARL2Layer:
    """One ARL2 hybrid attention layer for B streams of H heads, T tokens per frame, head dim d.

    ``query`` is one denoising (or clean) pass of the current frame: it reads the state of
    the previous frame and never writes it. ``commit`` is the clean-pass state update that
    closes the frame. All tensors are CUDA tensors: q, k, v, o bf16 [B, T, H, d]; alpha,
    beta fp32 [B, H, T]; the state fp32 [B, H, d, d]; feature maps bf16 [H, d, d].
    """

    def __init__(self, H: int, T: int, d: int, B: int = 1):
        self.H, self.T, self.d, self.B = H, T, d, B
        self._lib = load_library()
        self._ctx = arl2_create(H, T, d, d, B)

    # -- shapes
    @property
    def act_shape(self):
        return (self.B, self.T, self.H, self.d)

    @property
    def gate_shape(self):
        return (self.B, self.H, self.T)

    @property
    def state_shape(self):
        return (self.B, self.H, self.d, self.d)

    def close(self) -> None:
        if self._ctx is not None:
            self._lib.arl2_destroy(self._ctx)
            self._ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_feature_maps(self, Wq, Wk, Wv, stream=None) -> None:
        shp = (self.H, self.d, self.d)
        _check(self._lib.arl2_set_feature_maps(self._ctx, _dev(Wq, torch.bfloat16, shp, "Wq"),
                                               _dev(Wk, torch.bfloat16, shp, "Wk"),
                                               _dev(Wv, torch.bfloat16, shp, "Wv"), _stream(stream)),
               "arl2_set_feature_maps")

    def query(self, q, k, v, out=None, stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty(self.act_shape, dtype=torch.bfloat16, device=q.device)
        s = self.act_shape
        _check(self._lib.arl2_frame_query(self._ctx, _cuda(q, torch.bfloat16, s, "q"), _cuda(k, torch.bfloat16, s, "k"),
                                          _cuda(v, torch.bfloat16, s, "v"), _cuda(out, torch.bfloat16, s, "o"),
                                          _stream(stream)), "arl2_frame_query")
        return out

    def commit(self, k, v, alpha, beta, stream=None) -> None:
        s, g = self.act_shape, self.gate_shape
        _check(self._lib.arl2_frame_commit(self._ctx, _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
                                           _cuda(alpha, torch.float32, g, "alpha"), _cuda(beta, torch.float32, g, "beta"),
                                           _stream(stream)), "arl2_frame_commit")

    def clean_pass(self, q, k, v, alpha, beta, out=None, stream=None) -> torch.Tensor:
        """The clean pass in one launch: out = the query of (q, k, v) on S_{N-1}, and the commit
        of (k, v, alpha, beta) into S_N."""
        if out is None:
            out = torch.empty(self.act_shape, dtype=torch.bfloat16, device=q.device)
        s, g = self.act_shape, self.gate_shape
        _check(self._lib.arl2_frame_clean_pass(self._ctx, _cuda(q, torch.bfloat16, s, "q"),
                                               _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
                                               _cuda(out, torch.bfloat16, s, "o"),
                                               _cuda(alpha, torch.float32, g, "alpha"),
                                               _cuda(beta, torch.float32, g, "beta"), _stream(stream)),
               "arl2_frame_clean_pass")
        return out

    def set_clean_split(self, commit_sms: int) -> None:
        """SMs the clean pass gives the commit (0: chosen by the library's cost model)."""
        _check(self._lib.arl2_set_clean_split(self._ctx, int(commit_sms)), "arl2_set_clean_split")

    @property
    def clean_split(self) -> int:
        """SMs the clean pass currently gives the commit."""
        return self._lib.arl2_clean_split(self._ctx)

    def query_token(self, q, k, v, alpha, beta, out=None, stream=None) -> torch.Tensor:
        """Token-level access: intra attention plus the token-by-token readout of this pass."""
        if out is None:
            out = torch.empty(self.act_shape, dtype=torch.bfloat16, device=q.device)
        s, g = self.act_shape, self.gate_shape
        _check(self._lib.arl2_frame_query_token(self._ctx, _cuda(q, torch.bfloat16, s, "q"),
                                                _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
                                                _cuda(out, torch.bfloat16, s, "o"),
                                                _cuda(alpha, torch.float32, g, "alpha"),
                                                _cuda(beta, torch.float32, g, "beta"), _stream(stream)),
               "arl2_frame_query_token")
        return out

    def commit_token(self, k, v, alpha, beta, stream=None) -> None:
        """Token-level access: S_N = the state after the clean pass's last token."""
        s, g = self.act_shape, self.gate_shape
        _check(self._lib.arl2_frame_commit_token(self._ctx, _cuda(k, torch.bfloat16, s, "k"),
                                                 _cuda(v, torch.bfloat16, s, "v"),
                                                 _cuda(alpha, torch.float32, g, "alpha"),
                                                 _cuda(beta, torch.float32, g, "beta"), _stream(stream)),
               "arl2_frame_commit_token")

    def query_host(self, q, k, v, out, stream=None) -> torch.Tensor:
        """Host-buffer query: q, k, v, out are CPU tensors (pinned for asynchrony)."""
        s = self.act_shape
        _check(self._lib.arl2_frame_query_host(self._ctx, _host(q, torch.bfloat16, s, "q"),
                                               _host(k, torch.bfloat16, s, "k"), _host(v, torch.bfloat16, s, "v"),
                                               _host(out, torch.bfloat16, s, "o"), _stream(stream)),
               "arl2_frame_query_host")
        return out

    def commit_host(self, k, v, alpha, beta, stream=None) -> None:
        s, g = self.act_shape, self.gate_shape
        _check(self._lib.arl2_frame_commit_host(self._ctx, _host(k, torch.bfloat16, s, "k"),
                                                _host(v, torch.bfloat16, s, "v"),
                                                _host(alpha, torch.float32, g, "alpha"),
                                                _host(beta, torch.float32, g, "beta"), _stream(stream)),
               "arl2_frame_commit_host")

    def set_gate_weights(self, Wa, Wb, ba, bb, stream=None) -> None:
        """Gate projections for gates produced from the hidden state: Wa, Wb bf16 [H, H*d];
        ba, bb fp32 [H]."""
        D = self.H * self.d
        _check(self._lib.arl2_set_gate_weights(self._ctx, _dev(Wa, torch.bfloat16, (self.H, D), "Wa"),
                                               _dev(Wb, torch.bfloat16, (self.H, D), "Wb"),
                                               _dev(ba, torch.float32, (self.H,), "ba"),
                                               _dev(bb, torch.float32, (self.H,), "bb"), _stream(stream)),
               "arl2_set_gate_weights")

    def gates(self, x, alpha=None, beta=None, stream=None):
        """alpha, beta fp32 [B, H, T] from the hidden state x bf16 [B, T, H*d]."""
        if alpha is None:
            alpha = torch.empty(self.gate_shape, dtype=torch.float32, device=x.device)
        if beta is None:
            beta = torch.empty(self.gate_shape, dtype=torch.float32, device=x.device)
        xs, g = (self.B, self.T, self.H * self.d), self.gate_shape
        _check(self._lib.arl2_frame_gates(self._ctx, _cuda(x, torch.bfloat16, xs, "x"),
                                          _cuda(alpha, torch.float32, g, "alpha"),
                                          _cuda(beta, torch.float32, g, "beta"), _stream(stream)),
               "arl2_frame_gates")
        return alpha, beta

    def commit_gated(self, x, k, v, stream=None) -> None:
        """The clean-pass commit with its gates produced from the hidden state x."""
        xs, s = (self.B, self.T, self.H * self.d), self.act_shape
        _check(self._lib.arl2_frame_commit_gated(self._ctx, _cuda(x, torch.bfloat16, xs, "x"),
                                                 _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
                                                 _stream(stream)), "arl2_frame_commit_gated")

    def reset(self, stream=None) -> None:
        _check(self._lib.arl2_reset(self._ctx, _stream(stream)), "arl2_reset")

    def get_state(self, out=None, stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty(self.state_shape, dtype=torch.float32, device="cuda")
        _check(self._lib.arl2_get_state(self._ctx, _dev(out, torch.float32, self.state_shape, "dst"),
                                        _stream(stream)), "arl2_get_state")
        return out

    def set_state(self, S, stream=None) -> None:
        _check(self._lib.arl2_set_state(self._ctx, _dev(S, torch.float32, self.state_shape, "src"), _stream(stream)),
               "arl2_set_state")

    @property
    def frame_index(self) -> int:
        return self._lib.arl2_frame_index(self._ctx)

    def status(self) -> int:
        """Synchronise and return (and clear) the device status (ARL2_OK, ARL2_ERR_TIMEOUT, ...)."""
        return self._lib.arl2_get_status(self._ctx)

    def set_wait_timeout_ns(self, ns: int) -> None:
        _check(self._lib.arl2_set_wait_timeout_ns(self._ctx, int(ns)), "arl2_set_wait_timeout_ns")

    def set_launch_overlap(self, enable: bool) -> None:
        """Queries and commits may start behind the previous kernel in their stream (see arl2.h)."""
        _check(self._lib.arl2_set_launch_overlap(self._ctx, int(bool(enable))), "arl2_set_launch_overlap")

    def test_stall_next_query(self) -> None:
        """Failure-detection hook: the next query's bounded wait runs out (no GPU fault)."""
        _check(self._lib.arl2_test_stall_next_query(self._ctx), "arl2_test_stall_next_query")

    @property
    def memory_bytes(self) -> int:
        return self._lib.arl2_memory_bytes(self._ctx)


def frame_commit_noalloc(k, v, alpha, beta, Wk, Wv, S_prev, S_next, status, stream=None) -> None:
    """Commit without a context or any allocation (arl2_frame_commit_noalloc).

    For callers that cannot allocate device memory: the library's fixed scratch array is
    used instead. k, v bf16 [B, T, H, d]; alpha, beta fp32 [B, H, T]; Wk, Wv bf16 [H, d, d];
    S_prev, S_next fp32 [B, H, d, d] (S_next may be S_prev); status an int32 [1] device word
    the caller zeroed, which reads nonzero after the call if a bounded wait ran out.
    """
    B, T, H, d = k.shape
    s, g, w, st = (B, T, H, d), (B, H, T), (H, d, d), (B, H, d, d)
    if status is None or status.dtype != torch.int32 or status.numel() != 1 or not status.is_cuda:
        raise ValueError("status: expected one int32 element in device memory")
    status_ptr = status.data_ptr()
    _check(load_library().arl2_frame_commit_noalloc(
        B, H, T, d, _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
        _cuda(alpha, torch.float32, g, "alpha"), _cuda(beta, torch.float32, g, "beta"),
        _cuda(Wk, torch.bfloat16, w, "Wk"), _cuda(Wv, torch.bfloat16, w, "Wv"),
        _cuda(S_prev, torch.float32, st, "S_prev"), _cuda(S_next, torch.float32, st, "S_next"),
        status_ptr, _stream(stream)), "arl2_frame_commit_noalloc")


class KVCacheBaseline:
    """The growing-KV-cache full-softmax baseline (comparison only); see arl2_kvcache_* in arl2.h."""

    def __init__(self, H: int, T: int, d: int, B: int = 1, max_frames: int = 1):
        self.H, self.T, self.d, self.B, self.max_frames = H, T, d, B, max_frames
        self._lib = load_library()
        out = _P()
        _check(self._lib.arl2_kvcache_create(H, T, d, B, max_frames, ctypes.byref(out)), "arl2_kvcache_create")
        self._c = out

    @property
    def act_shape(self):
        return (self.B, self.T, self.H, self.d)

    def close(self) -> None:
        if self._c is not None:
            self._lib.arl2_kvcache_destroy(self._c)
            self._c = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def query(self, q, k, v, out=None, stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty(self.act_shape, dtype=torch.bfloat16, device=q.device)
        s = self.act_shape
        _check(self._lib.arl2_kvcache_query(self._c, _cuda(q, torch.bfloat16, s, "q"), _cuda(k, torch.bfloat16, s, "k"),
                                            _cuda(v, torch.bfloat16, s, "v"), _cuda(out, torch.bfloat16, s, "o"),
                                            _stream(stream)), "arl2_kvcache_query")
        return out

    def commit(self, k, v, stream=None) -> None:
        s = self.act_shape
        _check(self._lib.arl2_kvcache_commit(self._c, _cuda(k, torch.bfloat16, s, "k"), _cuda(v, torch.bfloat16, s, "v"),
                                             _stream(stream)), "arl2_kvcache_commit")

    def reset(self) -> None:
        _check(self._lib.arl2_kvcache_reset(self._c), "arl2_kvcache_reset")

    @property
    def frames(self) -> int:
        return self._lib.arl2_kvcache_frames(self._c)

    def status(self) -> int:
        return self._lib.arl2_kvcache_get_status(self._c)

    @property
    def memory_bytes(self) -> int:
        return self._lib.arl2_kvcache_memory_bytes(self._c)


# ------------------------------------------------- training operators: the gated recurrence
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _OnStream:
    """The stream of a call that was given one, or whose tensors' device is not current.

    Without a stream the call runs on the current stream of the tensors' device, as torch's own
    operators do. With one, outputs are allocated for that stream and the inputs are recorded on
    it, so that the allocator does not hand their memory on while the call still reads it.
    """

    def __init__(self, index, stream, tensors):
        if stream is None:
            self.ptr = _raw_stream(index)
            self.ctx = torch.cuda.device(index)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
        if stream.device.index != index:
            raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{index}")
        self.ptr = stream.cuda_stream
        self.ctx = torch.cuda.stream(stream)
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)

    def __enter__(self):
        self.ctx.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _want(t, name, index, dtypes, shape, contiguous=False):
    """Check one tensor argument: a CUDA tensor on device `index`; None passes."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected a tensor on cuda:{index}")
    if t.dtype not in dtypes or t.shape != shape:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if contiguous:
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    elif t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: its last dimension must be adjacent in memory")


_F32, _I32 = (torch.float32,), (torch.int32,)


def _scan_shape(x, a, lens, name):
    """Check the values and gates of a call; (device index, shape, strides of the gates, the
    fields of arl2_scan_shape)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    dtype, shape, index = x.dtype, x.shape, x.get_device()
    if len(shape) != 3 or dtype not in DTYPES:
        raise ValueError(f"{name}: expected bf16, fp16 or fp32 [B, T, C], got {dtype} {tuple(shape)}")
    _want(x, name, index, (dtype,), shape)
    B, T, C = shape
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise TypeError("a must be a torch.Tensor [B, T, C] or [B, heads, T]")
    # A gate tensor of x's shape is per channel; otherwise it is per head.
    st = a.stride()
    if a.shape == shape:
        heads = 0
        _want(a, "a", index, (dtype, torch.float32), shape)
    else:
        heads = a.shape[1]
        if a.get_device() != index or a.dtype != torch.float32 or a.shape != (B, heads, T) or heads < 1 or C % heads:
            raise ValueError(f"a: expected gates {(B, T, C)}, or fp32 [B, heads, T] with heads dividing {C}, got "
                             f"{a.dtype} {tuple(a.shape)} on {a.device}")
        st = (st[0], st[2], st[1])
    if lens is not None:
        _want(lens, "lens", index, _I32, (B,), True)
    return index, shape, st, (B, T, C, heads, DTYPES[dtype], DTYPES[a.dtype], _ptr(lens))


def _scan_workspace(lib, fields, x):
    if fields[1] <= 512:   # one chunk, whatever the width
        return None
    n = lib.arl2_scan_workspace_bytes(struct.pack(_SCAN_SHAPE, *fields))
    return x.new_empty(n, dtype=torch.uint8) if n else None


def scan_forward(x, a, h0=None, lens=None, out=None, final=None, stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + x_t along dim 1; returns (h, final state).

    x bf16, fp16 or fp32 [B, T, C]; a the gates, [B, T, C] of x's type or fp32, or one per head
    and token, fp32 [B, heads, T] with C / heads in {32, 64, 128} (the layout of
    ``ARL2Layer.gates``). h0 fp32 [B, C], 0 if None. lens int32 [B]: behind lens[b] h is 0, and
    the final state is that of the last token inside. With T = 1 this is the serving step. out
    may be x, final may be h0. The outputs carry no autograd graph; scan_backward gives the gradients.
    """
    index, shape, st_a, fields = _scan_shape(x, a, lens, "x")
    B, T, C = shape
    if stream is not None or index != torch._C._cuda_getDevice():
        with _OnStream(index, stream, (x, a, h0, lens, out, final)) as ptr:
            return _scan_forward(x, a, h0, out, final, ptr, index, shape, st_a, fields)
    return _scan_forward(x, a, h0, out, final, _raw_stream(index), index, shape, st_a, fields)


def _scan_forward(x, a, h0, out, final, stream, index, shape, st_a, fields):
    B, _, C = shape
    lib = load_library()
    _want(h0, "h0", index, _F32, (B, C), True)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _want(out, "out", index, (x.dtype,), shape)
    if final is None:
        final = x.new_empty((B, C), dtype=torch.float32) if h0 is None else torch.empty_like(h0)
    else:
        _want(final, "final", index, _F32, (B, C), True)
    ws = _scan_workspace(lib, fields, x)
    sx, so = x.stride(), out.stride()
    f = _SCAN_FWD.pack(*fields, x.data_ptr(), a.data_ptr(), _ptr(h0), out.data_ptr(), final.data_ptr(), _ptr(ws), sx[0],
                       sx[1], *st_a, so[0], so[1])
    _check(lib.arl2_scan_forward(f, stream), "arl2_scan_forward")
    return out, final


def scan_backward(dh, a, h, h0=None, dfinal=None, lens=None, dx=None, da=None, dh0=None, stream=None):
    """The backward pass of scan_forward; returns (dx, da, dh0).

    dh the gradient of h, [B, T, C] of h's type; a, h0, lens as in the forward call and h its
    output; dfinal fp32 [B, C] the gradient of the final state (0 if None). dx has dh's type;
    da the type and shape of a, contiguous; dh0 fp32 [B, C]. dx may be dh.
    """
    index, shape, st_a, fields = _scan_shape(dh, a, lens, "dh")
    if h is None:
        raise TypeError("h must be a torch.Tensor")
    _want(h, "h", index, (dh.dtype,), shape)
    args = (dh, a, h, h0, dfinal, dx, da, dh0)
    if stream is not None or index != torch._C._cuda_getDevice():
        with _OnStream(index, stream, args + (lens,)) as ptr:
            return _scan_backward(*args, ptr, index, shape, st_a, fields)
    return _scan_backward(*args, _raw_stream(index), index, shape, st_a, fields)


def _scan_backward(dh, a, h, h0, dfinal, dx, da, dh0, stream, index, shape, st_a, fields):
    B, _, C = shape
    lib = load_library()
    _want(h0, "h0", index, _F32, (B, C), True)
    _want(dfinal, "dfinal", index, _F32, (B, C), True)
    if dx is None:
        dx = torch.empty_like(dh, memory_format=torch.contiguous_format)
    else:
        _want(dx, "dx", index, (dh.dtype,), shape)
    if da is None:
        da = torch.empty_like(a, memory_format=torch.contiguous_format)
    else:
        _want(da, "da", index, (a.dtype,), a.shape, True)
    if dh0 is None:
        dh0 = dh.new_empty((B, C), dtype=torch.float32)
    else:
        _want(dh0, "dh0", index, _F32, (B, C), True)
    ws = _scan_workspace(lib, fields, dh)
    sg, sh, sx = dh.stride(), h.stride(), dx.stride()
    f = _SCAN_BWD.pack(*fields, dh.data_ptr(), a.data_ptr(), h.data_ptr(), _ptr(h0), _ptr(dfinal), dx.data_ptr(),
                       da.data_ptr(), dh0.data_ptr(), _ptr(ws), sg[0], sg[1], *st_a, sh[0], sh[1], sx[0], sx[1])
    _check(lib.arl2_scan_backward(f, stream), "arl2_scan_backward")
    return dx, da, dh0


# ---------------------------------------------------- training operators: softmax attention
class SoftmaxAttention:
    """Softmax attention with its row statistics and its backward pass (arl2_attn_* in arl2.h).

    For B sequences of H query heads over H_kv key heads (H a multiple of H_kv), head dim d in
    {32, 64, 128}, bf16 or fp16, up to max_Tq queries and max_Tk keys. ``forward`` returns
    (o, lse); ``backward`` takes them with do and returns (dq, dk, dv). q, o, do, dq are
    [B, Tq, H, d], k, v, dk, dv [B, Tk, H_kv, d], lse fp32 [B, H, Tq]; inputs may be strided
    views (16-byte aligned, strides multiples of 8), such as slices of one packed projection.

    Mask: key j is visible to query i if i < q_len[b], j < k_len[b] (int32 [B], None: all) and,
    with frame_len > 0, j < (floor((i + q_start) / frame_len) + 1) * frame_len: its own frame
    and the ones before it (frame_len = 1: causal), q_start being the place of query 0 among
    the keys. Rows that see nothing give o = 0, lse = -inf. scale defaults to 1 / sqrt(d).

    Every call takes B sequences; a shorter batch is one whose last q_len and k_len are 0. The
    outputs carry no autograd graph, whether or not the inputs require gradients: ``backward`` is
    what a ``torch.autograd.Function`` around the two calls would use.

    The scratch belongs to the object: calls on one object, and replays of graphs that captured
    them, must be ordered, normally by one stream.
    """

    def __init__(self, H: int, max_Tq: int, max_Tk: int, d: int, B: int = 1, H_kv: Optional[int] = None,
                 dtype: torch.dtype = torch.bfloat16, device=None):
        self.H, self.d, self.B, self.H_kv, self.dtype = H, d, B, H if H_kv is None else H_kv, dtype
        self.max_Tq, self.max_Tk = max_Tq, max_Tk
        self._c = None
        if dtype not in DTYPES:
            raise ValueError(f"dtype: expected torch.bfloat16 or torch.float16, got {dtype}")
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device: expected a CUDA device, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._lse_shapes = {}
        out = _P()
        with torch.cuda.device(self.device):
            _check(self._lib.arl2_attn_create(B, H, self.H_kv, max_Tq, max_Tk, d, DTYPES[dtype], ctypes.byref(out)),
                   "arl2_attn_create")
        self._c = out

    def close(self) -> None:
        if self._c is not None:
            with torch.cuda.device(self.device):
                self._lib.arl2_attn_destroy(self._c)
            self._c = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _lse_like(self, Tq):
        """A stand-in (4 bytes) of lse's shape: allocating from one is the quicker call."""
        t = self._lse_shapes.get(Tq)
        if t is None:
            if len(self._lse_shapes) > 64:
                self._lse_shapes.clear()
            t = self._lse_shapes[Tq] = torch.empty((1,), dtype=torch.float32, device=self.device).expand(
                self.B, self.H, Tq)
        return t

    def _lengths(self, q, k):
        for t, name in ((q, "q"), (k, "k")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dim() != 4:
                raise ValueError(f"{name}: expected [B, T, heads, d], got {tuple(t.shape)}")
        if self._c is None:
            raise Arl2Error(ARL2_ERR_INVALID_ARG, "a closed SoftmaxAttention")
        return q.shape[1], k.shape[1]

    def _tensor(self, t, name, shape):
        """Check one [B, T, heads, d] tensor; the fields of its arl2_tensor."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        s = t.stride()
        if t.get_device() != self._index or t.dtype is not self.dtype or t.shape != shape or s[3] != 1:
            raise ValueError(f"{name}: expected {self.dtype} {tuple(shape)} on {self.device}, its last dimension "
                             f"adjacent in memory; got {t.dtype} {tuple(t.shape)} on {t.device}, strides {s}")
        return t.data_ptr(), s[0], s[1], s[2]

    def _shape(self, Tq, Tk, q_len, k_len, frame_len, q_start, scale):
        """Check the mask and scale; the fields of arl2_attn_shape."""
        if q_len is not None:
            _want(q_len, "q_len", self._index, _I32, (self.B,), True)
        if k_len is not None:
            _want(k_len, "k_len", self._index, _I32, (self.B,), True)
        for v, name in ((frame_len, "frame_len"), (q_start, "q_start")):
            if not -(1 << 31) <= v < 1 << 31:
                raise ValueError(f"{name}: {v} does not fit an int")
        if scale is None:
            scale = 0.0
        elif not 0.0 < scale < float("inf"):
            raise ValueError(f"scale: expected a positive number, got {scale}")
        return Tq, Tk, _ptr(q_len), _ptr(k_len), frame_len, q_start, scale

    def forward(self, q, k, v, out=None, lse=None, q_len=None, k_len=None, frame_len: int = 0, q_start: int = 0,
                scale: Optional[float] = None, stream=None):
        """o = softmax(scale q k^T + mask) v and the rows' lse; returns (o, lse)."""
        Tq, Tk = self._lengths(q, k)
        shape = self._shape(Tq, Tk, q_len, k_len, frame_len, q_start, scale)
        if stream is not None or self._index != torch._C._cuda_getDevice():
            with _OnStream(self._index, stream, (q, k, v, out, lse, q_len, k_len)) as ptr:
                return self._forward(q, k, v, out, lse, shape, ptr)
        return self._forward(q, k, v, out, lse, shape, _raw_stream(self._index))

    def _forward(self, q, k, v, out, lse, shape, stream):
        qs, ks = (self.B, shape[0], self.H, self.d), (self.B, shape[1], self.H_kv, self.d)
        fields = self._tensor(q, "q", qs) + self._tensor(k, "k", ks) + self._tensor(v, "v", ks)
        if out is None:
            out = torch.empty_like(q)
            s = out.stride()
            o = (out.data_ptr(), s[0], s[1], s[2])
        else:
            o = self._tensor(out, "out", qs)
        if lse is None:
            lse = torch.empty_like(self._lse_like(shape[0]), memory_format=torch.contiguous_format)
        else:
            _want(lse, "lse", self._index, _F32, (self.B, self.H, shape[0]), True)
        f = _ATTN_FWD.pack(*shape, *fields, *o, lse.data_ptr())
        _check(self._lib.arl2_attn_forward(self._c, f, stream), "arl2_attn_forward")
        return out, lse

    def backward(self, do, q, k, v, o, lse, dq=None, dk=None, dv=None, q_len=None, k_len=None, frame_len: int = 0,
                 q_start: int = 0, scale: Optional[float] = None, stream=None):
        """The gradients of q, k and v from do, with o and lse of the forward call and its mask
        and scale; returns (dq, dk, dv)."""
        Tq, Tk = self._lengths(q, k)
        shape = self._shape(Tq, Tk, q_len, k_len, frame_len, q_start, scale)
        args = (do, q, k, v, o, lse, dq, dk, dv)
        if stream is not None or self._index != torch._C._cuda_getDevice():
            with _OnStream(self._index, stream, args + (q_len, k_len)) as ptr:
                return self._backward(*args, shape, ptr)
        return self._backward(*args, shape, _raw_stream(self._index))

    def _backward(self, do, q, k, v, o, lse, dq, dk, dv, shape, stream):
        qs, ks = (self.B, shape[0], self.H, self.d), (self.B, shape[1], self.H_kv, self.d)
        fields = (self._tensor(q, "q", qs) + self._tensor(k, "k", ks) + self._tensor(v, "v", ks)
                  + self._tensor(o, "o", qs) + self._tensor(do, "do", qs))
        if lse is None:
            raise TypeError("lse must be a torch.Tensor")
        _want(lse, "lse", self._index, _F32, (self.B, self.H, shape[0]), True)
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        f = _ATTN_BWD.pack(*shape, *fields, *self._tensor(dq, "dq", qs), *self._tensor(dk, "dk", ks),
                           *self._tensor(dv, "dv", ks), lse.data_ptr())
        _check(self._lib.arl2_attn_backward(self._c, f, stream), "arl2_attn_backward")
        return dq, dk, dv

    def status(self) -> int:
        """Synchronise and return (and clear) the device status (ARL2_OK, ARL2_ERR_TIMEOUT, ...)."""
        with torch.cuda.device(self.device):
            return self._lib.arl2_attn_get_status(self._c)

    @property
    def memory_bytes(self) -> int:
        return self._lib.arl2_attn_memory_bytes(self._c)
