"""Python binding of the GB300 MoE decode library (libmoedecode.so).

Argument marshalling only: every computation runs in the library's CUDA
kernels. PyTorch provides device memory and streams. The names follow the C
ABI in ``include/moe_decode.h``. If the library has not been built, importing
works but every call raises ``RuntimeError``; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoedecode.so")

DEC_OK, DEC_ERR_INVALID_ARG, DEC_ERR_UNSUPPORTED, DEC_ERR_CUDA, DEC_ERR_TIMEOUT = range(5)
VARIANT_AUTO, VARIANT_SMALL_M, VARIANT_SPLIT_K = 0, 1, 2

_lib = None
_bf16 = _i32 = _raw_stream = None  # set by _load


class DecodeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _load().dec_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


def build() -> str:
    """Compile the CUDA library in-tree for sm_103a (nvcc)."""
    from . import _build
    return _build.build()


class _LayerWeights(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("N_in", ctypes.c_int), ("K_out", ctypes.c_int), ("E", ctypes.c_int),
                ("k", ctypes.c_int), ("I", ctypes.c_int), ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in ("gamma1", "W_in", "W_o", "gamma2", "W_r", "Wg", "Wu", "Wd",
                                               "Wg_s", "Wu_s", "Wd_s", "prefetch_next")] + \
               [("prefetch_bytes", ctypes.c_size_t)]


class _MoeWeights(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("I", ctypes.c_int),
                ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in ("gamma", "W_r", "Wg", "Wu", "Wd", "Wg_s", "Wu_s", "Wd_s")]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_stride", ctypes.c_int64),
                ("blocks", ctypes.c_int), ("block_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int)]


class _Batch(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int), ("max_new", ctypes.c_int), ("row_start", ctypes.c_void_p),
                ("own_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int),
                ("prefix_table", ctypes.c_void_p), ("prefix_len", ctypes.c_int)]


class _StepTables(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("row_start", "own_len", "positions", "slots", "left")]


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("phases", ctypes.c_void_p)]


class _LayerAttention(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int), ("scale", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in ("rope", "cache", "batch", "positions", "slots")]


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


class _LayerTrace(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("h1", "idx", "w", "scores")]


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with moe_layers_gb300.build() "
                           "(the CUDA path has no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, U64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_float
    I64 = ctypes.c_int64
    sig = {
        "dec_create": [ctypes.POINTER(P), I],
        "dec_destroy": [P],
        "dec_workspace_init": [P, P, Z, P],
        "dec_set_wait_limit_ns": [P, U64],
        "dec_set_pdl": [P, I],
        "dec_set_force_variant": [P, I],
        "dec_set_shared_sms": [P, I],
        "dec_set_l2_ahead": [P, I],
        "dec_test_set_moe_front": [P, I],
        "dec_test_set_engine_finish": [P, I],
        "dec_check_device_error": [P],
        "dec_linear_workspace_size": [P, I, I, I, ctypes.POINTER(Z)],
        "dec_linear": [P, P, I, P, P, I, I, I, P, Z, P],
        "dec_linear_residual": [P, P, I, P, P, P, I, I, I, P, Z, P],
        "dec_linear_noalloc": [P, P, I, P, P, P, I, I, I, P],
        "dec_rmsnorm": [P, P, P, P, I, I, F, P],
        "moe_route_topk_workspace_size": [P, I, I, I, ctypes.POINTER(Z)],
        "moe_route_topk": [P, P, P, I, I, I, I, P, P, P, P, Z, P],
        "moe_experts_workspace_size": [P, I, I, I, I, I, ctypes.POINTER(Z)],
        "moe_experts": [P, P, P, P, I, I, P, P, P, I, I, I, P, P, P, P, P, P, Z, P],
        "moe_layer_workspace_size": [P, ctypes.POINTER(_MoeWeights), I, ctypes.POINTER(Z)],
        "moe_layer": [P, ctypes.POINTER(_MoeWeights), P, P, P, I, P, P, P, P, Z, P],
        "decode_layer_workspace_size": [P, ctypes.POINTER(_LayerWeights), I, ctypes.POINTER(Z)],
        "decode_layer": [P, ctypes.POINTER(_LayerWeights), P, I, ctypes.POINTER(_LayerTrace), P, Z, P],
        "dec_prefetch_l2": [P, P, Z, P],
        "dec_batch_tables": [P, P, P, I, P, P, P, I, I, I, I, ctypes.POINTER(_StepTables), P],
        "dec_rope_phases": [P, P, I, ctypes.c_double, I, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                            ctypes.c_double, P],
        "dec_rope_append": [P, ctypes.POINTER(_Rope), P, I64, P, I64, P, I64, P, I64, I, I, P, P,
                            ctypes.POINTER(_KvCache), P],
        "dec_attention_workspace_size": [P, I, I, ctypes.POINTER(_KvCache), ctypes.POINTER(_Batch),
                                         ctypes.POINTER(Z)],
        "decode_layer_attention_workspace_size": [P, ctypes.POINTER(_LayerWeights), ctypes.POINTER(_LayerAttention), I,
                                                  ctypes.POINTER(Z)],
        "decode_layer_attention": [P, ctypes.POINTER(_LayerWeights), ctypes.POINTER(_LayerAttention), P, I,
                                   ctypes.POINTER(_LayerTrace), P, Z, P],
        "dec_attention": [P, P, I64, ctypes.POINTER(_KvCache), ctypes.POINTER(_Batch), F, P, I64, I, I, P, Z, P],
        "dec_test_wait_timeout": [P, P],
        "dec_test_routing_wait_timeout": [P, I, P],
        "dec_test_delayed_copy": [P, P, P, Z, U64, P],
        "dec_test_occupy_sms": [P, I, U64, P],
        "dec_set_profiling": [P, I],
        "dec_profile_read": [P, ctypes.POINTER(_KernelTime), I, ctypes.POINTER(I)],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.dec_status_string.argtypes = [ctypes.c_int]
    lib.dec_status_string.restype = ctypes.c_char_p
    lib.dec_last_variant.argtypes = [P]
    lib.dec_last_variant.restype = ctypes.c_int
    lib.dec_last_expert_variant.argtypes = [P]
    lib.dec_last_expert_variant.restype = ctypes.c_int
    lib.dec_launch_count.argtypes = [P]
    lib.dec_launch_count.restype = ctypes.c_uint64
    import torch
    global _bf16, _i32, _raw_stream
    _bf16, _i32 = torch.bfloat16, torch.int32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != DEC_OK:
        raise DecodeError(status, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _require(t, dtype, name: str, ndim: Optional[int] = None):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t


def _rows(t, name: str) -> int:
    """Row stride (elements) of a 2-D tensor whose rows are contiguous."""
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.stride(0) if t.dim() == 2 else t.shape[-1]


class Handle:
    """Owns a dec_handle (side streams, events, device error word) and cached workspaces."""

    def __init__(self, device: int = 0):
        lib = _load()
        h = ctypes.c_void_p()
        _check(lib.dec_create(ctypes.byref(h), int(device)), "dec_create")
        self._h = h
        self.device = int(device)
        self._ws = {}
        self._stream_ws = {}
        self._attention_ws = {}  # workspace bytes by shape
        self._layer_ws = {}      # decode_layer_attention's workspaces by stream and shape

    @property
    def ptr(self):
        return self._h

    def close(self) -> None:
        if self._h:
            _load().dec_destroy(self._h)
            self._h = ctypes.c_void_p()
            self._ws.clear()
            self._stream_ws.clear()
            self._layer_ws.clear()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, key, nbytes: int, layout=None):
        """A workspace of at least nbytes, reused per key. It is zeroed when it
        is created and whenever the layout (entry point and shape) that uses it
        changes, as the C ABI requires; calls with the same layout leave it ready."""
        import torch
        t, last = self._ws.get(key, (None, None))
        if t is None or t.numel() < nbytes:
            t = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=f"cuda:{self.device}")
        elif layout != last:
            t.zero_()
        self._ws[key] = (t, layout)
        return t

    def stream_workspace(self, key, address: int, nbytes: int, stream=None):
        """A workspace of at least nbytes per key and stream (its address; `stream` if it
        is not the current one), for calls that need no zeroed memory. It is memory of
        that stream: a block that another stream gave back may still be in use there.
        One that is outgrown is kept until the handle closes: a captured graph may
        still use it."""
        import torch
        held = self._stream_ws.setdefault((key, address), [])
        if not held or held[-1].numel() < nbytes:
            size = max(int(nbytes), 256, 2 * held[-1].numel() if held else 0)
            with _on_stream(stream):
                held.append(torch.empty(size, dtype=torch.uint8, device=f"cuda:{self.device}"))
        return held[-1]

    def set_force_variant(self, v: int) -> None:
        _check(_load().dec_set_force_variant(self._h, int(v)), "dec_set_force_variant")

    def set_shared_sms(self, n: int) -> None:
        """0: automatic SM share by expected bytes; -1: every SM, overlapped; n > 0: a fixed n-SM partition."""
        _check(_load().dec_set_shared_sms(self._h, int(n)), "dec_set_shared_sms")

    def test_set_moe_front(self, enable: bool) -> None:
        """Test hook: False runs the path taken where an MoE front does not apply."""
        _check(_load().dec_test_set_moe_front(self._h, 1 if enable else 0), "dec_test_set_moe_front")

    def test_set_engine_finish(self, mode: int) -> None:
        """Test hook: how the split-K kernel finishes split tiles (0 default; 1, 2 the fallback paths)."""
        _check(_load().dec_test_set_engine_finish(self._h, int(mode)), "dec_test_set_engine_finish")

    def set_l2_ahead(self, nbytes: int) -> None:
        _check(_load().dec_set_l2_ahead(self._h, int(nbytes)), "dec_set_l2_ahead")

    def set_pdl(self, enable: bool) -> None:
        _check(_load().dec_set_pdl(self._h, 1 if enable else 0), "dec_set_pdl")

    def set_wait_limit_ns(self, ns: int) -> None:
        _check(_load().dec_set_wait_limit_ns(self._h, int(ns)), "dec_set_wait_limit_ns")

    @property
    def last_variant(self) -> int:
        return _load().dec_last_variant(self._h)

    @property
    def last_expert_variant(self) -> int:
        return _load().dec_last_expert_variant(self._h)

    def check_device_error(self) -> int:
        return _load().dec_check_device_error(self._h)

    def set_profiling(self, enable: bool) -> None:
        _check(_load().dec_set_profiling(self._h, 1 if enable else 0), "dec_set_profiling")

    def profile_read(self) -> dict:
        """{kernel tag: (launches, total_ms)} since the last read (synchronises)."""
        buf = (_KernelTime * 64)()
        n = ctypes.c_int()
        _check(_load().dec_profile_read(self._h, buf, 64, ctypes.byref(n)), "dec_profile_read")
        return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n.value)}

    @property
    def launch_count(self) -> int:
        return int(_load().dec_launch_count(self._h))


# ---------------------------------------------------------------------------- projections
def dec_linear(h: Handle, x, W, y=None, stream=None, ws=None):
    """y = x W^T (bf16). x [M,K] (rows may be strided), W [N,K]."""
    import torch
    lib = _load()
    _require(x, torch.bfloat16, "x", 2)
    _require(W, torch.bfloat16, "W", 2)
    M, K = x.shape
    N = W.shape[0]
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    nb = ctypes.c_size_t()
    _check(lib.dec_linear_workspace_size(h.ptr, M, N, K, ctypes.byref(nb)), "dec_linear_workspace_size")
    ws = h.workspace(("linear", id(stream)), nb.value, ("linear", M, N, K)) if ws is None else ws
    _check(lib.dec_linear(h.ptr, _ptr(x), _rows(x, "x"), _ptr(W), _ptr(y), M, N, K, _ptr(ws), ws.numel(),
                          _stream(stream)), "dec_linear")
    return y


def dec_linear_residual(h: Handle, x, W, r, out=None, stream=None, ws=None):
    """out = r + x W^T (bf16); out may be r itself."""
    import torch
    lib = _load()
    _require(x, torch.bfloat16, "x", 2)
    _require(W, torch.bfloat16, "W", 2)
    _require(r, torch.bfloat16, "r", 2)
    M, K = x.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    nb = ctypes.c_size_t()
    _check(lib.dec_linear_workspace_size(h.ptr, M, N, K, ctypes.byref(nb)), "dec_linear_workspace_size")
    ws = h.workspace(("linear", id(stream)), nb.value, ("linear", M, N, K)) if ws is None else ws
    _check(lib.dec_linear_residual(h.ptr, _ptr(x), _rows(x, "x"), _ptr(W), _ptr(r), _ptr(out), M, N, K, _ptr(ws),
                                   ws.numel(), _stream(stream)), "dec_linear_residual")
    return out


def dec_linear_noalloc(h: Handle, x, W, r=None, out=None, stream=None):
    """out = [r +] x W^T through the entry point that takes no workspace and
    allocates nothing (its scratch is a static device array in the library)."""
    import torch
    _require(x, torch.bfloat16, "x", 2)
    _require(W, torch.bfloat16, "W", 2)
    M, K = x.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(_load().dec_linear_noalloc(h.ptr, _ptr(x), _rows(x, "x"), _ptr(W), _ptr(r), _ptr(out), M, N, K,
                                      _stream(stream)), "dec_linear_noalloc")
    return out


def dec_rmsnorm(h: Handle, x, gamma, y=None, eps: float = 1e-6, stream=None):
    import torch
    _require(x, torch.bfloat16, "x", 2)
    _require(gamma, torch.bfloat16, "gamma", 1)
    M, H = x.shape
    if y is None:
        y = torch.empty_like(x)
    _check(_load().dec_rmsnorm(h.ptr, _ptr(x), _ptr(gamma), _ptr(y), M, H, ctypes.c_float(eps), _stream(stream)),
           "dec_rmsnorm")
    return y


# ---------------------------------------------------------------------------- router / experts
def moe_route_topk(h: Handle, x, Wr, k: int, want_scores: bool = True, stream=None):
    """Returns (idx int32 [M,k], w fp32 [M,k], scores fp32 [M,E] or None)."""
    import torch
    lib = _load()
    _require(x, torch.bfloat16, "x", 2)
    _require(Wr, torch.float32, "Wr", 2)
    M, H = x.shape
    E = Wr.shape[0]
    idx = torch.empty((M, k), dtype=torch.int32, device=x.device)
    w = torch.empty((M, k), dtype=torch.float32, device=x.device)
    scores = torch.empty((M, E), dtype=torch.float32, device=x.device) if want_scores else None
    nb = ctypes.c_size_t()
    _check(lib.moe_route_topk_workspace_size(h.ptr, M, H, E, ctypes.byref(nb)), "moe_route_topk_workspace_size")
    ws = h.workspace(("router", id(stream)), nb.value, ("router", M, H, E))
    _check(lib.moe_route_topk(h.ptr, _ptr(x), _ptr(Wr), M, H, E, int(k), _ptr(idx), _ptr(w), _ptr(scores),
                              _ptr(ws), ws.numel(), _stream(stream)), "moe_route_topk")
    return idx, w, scores


def moe_experts(h: Handle, x, idx, w, Wg, Wu, Wd, shared: Optional[Sequence] = None, residual=None, out=None,
                stream=None):
    """out = [residual +] sum_j w_j E_idx_j(x) [+ S(x)] (bf16 [M,H])."""
    import torch
    lib = _load()
    _require(x, torch.bfloat16, "x", 2)
    _require(idx, torch.int32, "idx", 2)
    _require(w, torch.float32, "w", 2)
    for n, t in (("Wg", Wg), ("Wu", Wu), ("Wd", Wd)):
        _require(t, torch.bfloat16, n, 3)
    M, H = x.shape
    k = idx.shape[1]
    E, I, _ = Wg.shape
    sg, su, sd = (None, None, None) if shared is None else shared
    if out is None:
        out = torch.empty_like(x)
    nb = ctypes.c_size_t()
    _check(lib.moe_experts_workspace_size(h.ptr, M, k, E, H, I, ctypes.byref(nb)), "moe_experts_workspace_size")
    ws = h.workspace(("experts", id(stream)), nb.value, ("experts", M, k, E, H, I))
    _check(lib.moe_experts(h.ptr, _ptr(x), _ptr(idx), _ptr(w), M, k, _ptr(Wg), _ptr(Wu), _ptr(Wd), E, H, I,
                           _ptr(sg), _ptr(su), _ptr(sd), _ptr(residual), _ptr(out), _ptr(ws), ws.numel(),
                           _stream(stream)), "moe_experts")
    return out


@dataclass
class MoeWeights:
    """Device tensors of one MoE layer (see dec_moe_weights); gamma None: no RMSNorm."""
    W_r: object
    Wg: object
    Wu: object
    Wd: object
    Wg_s: object = None
    Wu_s: object = None
    Wd_s: object = None
    gamma: object = None
    k: int = 8
    eps: float = 1e-6

    def c_struct(self) -> _MoeWeights:
        E, I, H = self.Wg.shape
        s = _MoeWeights()
        s.H, s.E, s.k, s.I, s.eps = H, E, self.k, I, self.eps
        for n in ("gamma", "W_r", "Wg", "Wu", "Wd", "Wg_s", "Wu_s", "Wd_s"):
            setattr(s, n, _ptr(getattr(self, n)))
        return s


def moe_layer_workspace_size(h: Handle, weights: MoeWeights, M: int) -> int:
    nb = ctypes.c_size_t()
    cw = weights.c_struct()
    _check(_load().moe_layer_workspace_size(h.ptr, ctypes.byref(cw), int(M), ctypes.byref(nb)),
           "moe_layer_workspace_size")
    return nb.value


def moe_layer(h: Handle, weights: MoeWeights, x, residual=None, out=None, trace=False, stream=None, ws=None,
              _cw=None):
    """out = [residual +] MoE([RMSNorm](x)) (bf16 [M,H]): routing and experts in one call.

    trace=True also returns a dict of new device tensors with the routing
    (idx, w, scores); trace may be a dict of preallocated tensors (any of those
    keys). Returns out, or (out, trace dict)."""
    import torch
    lib = _load()
    _require(x, torch.bfloat16, "x", 2)
    M = x.shape[0]
    cw = weights.c_struct() if _cw is None else _cw
    if out is None:
        out = torch.empty_like(x)
    if ws is None:
        ws = h.workspace(("moe_layer", id(stream)), moe_layer_workspace_size(h, weights, M),
                         ("moe_layer", M, cw.H, cw.E, cw.k, cw.I))
    tr = None
    if trace is True:
        tr = dict(idx=torch.empty((M, cw.k), dtype=torch.int32, device=x.device),
                  w=torch.empty((M, cw.k), dtype=torch.float32, device=x.device),
                  scores=torch.empty((M, cw.E), dtype=torch.float32, device=x.device))
    elif isinstance(trace, dict):
        tr = trace
    g = (lambda n: None) if tr is None else tr.get
    _check(lib.moe_layer(h.ptr, ctypes.byref(cw), _ptr(x), _ptr(residual), _ptr(out), M, _ptr(g("idx")),
                         _ptr(g("w")), _ptr(g("scores")), _ptr(ws), ws.numel(), _stream(stream)), "moe_layer")
    return out if tr is None else (out, tr)


@dataclass
class LayerWeights:
    """Device tensors of one decode layer (see dec_layer_weights)."""
    gamma1: object
    W_in: object
    W_o: object
    gamma2: object
    W_r: object
    Wg: object
    Wu: object
    Wd: object
    Wg_s: object = None
    Wu_s: object = None
    Wd_s: object = None
    k: int = 8
    k_out: Optional[int] = None
    eps: float = 1e-6
    prefetch_next: object = None
    prefetch_bytes: int = 0

    def c_struct(self) -> _LayerWeights:
        E, I, H = self.Wg.shape
        s = _LayerWeights()
        s.H, s.N_in = H, self.W_in.shape[0]
        s.K_out = self.W_o.shape[1] if self.k_out is None else self.k_out
        s.E, s.k, s.I, s.eps = E, self.k, I, self.eps
        for n in ("gamma1", "W_in", "W_o", "gamma2", "W_r", "Wg", "Wu", "Wd", "Wg_s", "Wu_s", "Wd_s",
                  "prefetch_next"):
            setattr(s, n, _ptr(getattr(self, n)))
        s.prefetch_bytes = int(self.prefetch_bytes)
        return s


def decode_layer_workspace_size(h: Handle, weights: LayerWeights, M: int) -> int:
    nb = ctypes.c_size_t()
    cw = weights.c_struct()
    _check(_load().decode_layer_workspace_size(h.ptr, ctypes.byref(cw), int(M), ctypes.byref(nb)),
           "decode_layer_workspace_size")
    return nb.value


def decode_layer(h: Handle, weights: LayerWeights, hidden, trace=False, stream=None, ws=None, _cw=None):
    """One decode layer in place on hidden bf16 [M,H].

    trace=True returns a dict of new device tensors with the intermediates
    (h1, idx, w, scores); trace may also be a dict of preallocated tensors
    (any of those keys, others omitted) that receive them."""
    import torch
    lib = _load()
    _require(hidden, torch.bfloat16, "hidden", 2)
    M = hidden.shape[0]
    cw = weights.c_struct() if _cw is None else _cw
    if ws is None:
        ws = h.workspace(("layer", id(stream)), decode_layer_workspace_size(h, weights, M),
                         ("layer", M, cw.H, cw.N_in, cw.K_out, cw.E, cw.k, cw.I))
    tr = None
    out = None
    if trace is True:
        out = dict(h1=torch.empty_like(hidden),
                   idx=torch.empty((M, cw.k), dtype=torch.int32, device=hidden.device),
                   w=torch.empty((M, cw.k), dtype=torch.float32, device=hidden.device),
                   scores=torch.empty((M, cw.E), dtype=torch.float32, device=hidden.device))
    elif isinstance(trace, dict):
        out = trace
    if out is not None:
        tr = _LayerTrace()
        tr.h1, tr.idx, tr.w, tr.scores = (_ptr(out.get(n)) for n in ("h1", "idx", "w", "scores"))
    _check(lib.decode_layer(h.ptr, ctypes.byref(cw), _ptr(hidden), M, ctypes.byref(tr) if tr is not None else None,
                            _ptr(ws), ws.numel(), _stream(stream)), "decode_layer")
    return out


# ---------------------------------------------------------------------------- attention
def _int32(t, name: str, ndim: int = 1):
    import torch
    _require(t, torch.int32, name, ndim)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream_of(h: Handle, stream) -> int:
    """The given stream, else the current one of the handle's device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:  # a microsecond less than a Stream object
        return _raw_stream(h.device)
    import torch
    return torch.cuda.current_stream(h.device).cuda_stream


def _on_stream(stream):
    """Context in which new tensors belong to the stream of the call (None: the current one)."""
    import contextlib
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _rows_of(t, name: str, device: int):
    """(rows, width, row stride) of a 2-D bf16 tensor with contiguous rows on the device."""
    if t.dtype is not _bf16 or t.dim() != 2 or t.get_device() != device:
        _require(t, _bf16, name, 2)
        raise ValueError(f"{name} must be on the handle's device, cuda:{device}")
    rows, width = t.shape
    ld, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # the stride of a single row means nothing
    return rows, width, ld if rows > 1 else -(-width // 8) * 8


def _ints_of(t, name: str, device: int, count: Optional[int] = None) -> int:
    """Address of a contiguous 1-D int32 tensor on the device with `count` elements."""
    if t.dtype is not _i32 or t.dim() != 1 or t.get_device() != device or not t.is_contiguous():
        _int32(t, name)
        raise ValueError(f"{name} must be on the handle's device, cuda:{device}")
    if count is not None and t.numel() != count:
        raise ValueError(f"{name} must have {count} elements")
    return t.data_ptr()


def _ws_bytes(ws, device: int) -> int:
    """Bytes of a caller's workspace, a contiguous tensor of any type on the device."""
    if not ws.is_cuda or ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on the handle's device, cuda:{device}")
    return ws.numel() * ws.element_size()


class KvCache:
    """Paged key / value cache of one layer (see dec_kv_cache): k and v bf16
    [blocks, kv_heads, block_size, head_dim], each block contiguous (the two may
    interleave in one pool). Make a new one to describe other tensors."""

    def __init__(self, k, v):
        import torch
        for n, t in (("k", k), ("v", v)):
            _require(t, torch.bfloat16, n, 4)
            _, heads, size, dim = t.shape
            if t.stride()[1:] != (size * dim, dim, 1):
                raise ValueError(f"{n}: the heads, tokens and elements of a block must be contiguous")
        if k.shape != v.shape or (k.shape[0] > 1 and k.stride(0) != v.stride(0)) or k.device != v.device:
            raise ValueError("k and v must have the same shape, block stride and device")
        self.k, self.v = k, v
        blocks, heads, size, dim = k.shape
        stride = k.stride(0) if blocks > 1 else heads * size * dim
        self._c = _KvCache(k.data_ptr(), v.data_ptr(), stride, blocks, size, heads, dim)
        self._ref = ctypes.byref(self._c)
        self.block_size, self.kv_heads, self.head_dim, self.device_index = size, heads, dim, k.get_device()


class StepTables:
    """Outputs of dec_batch_tables: int32 device tensors row_start [requests + 1],
    own_len [requests], positions [rows], slots [rows] and left [2]."""

    def __init__(self, row_start, own_len, positions, slots, left):
        for n, t in (("row_start", row_start), ("own_len", own_len), ("positions", positions), ("slots", slots),
                     ("left", left)):
            _int32(t, n)
        if any(t.device != row_start.device for t in (own_len, positions, slots, left)):
            raise ValueError("the tables must be on one device")
        if row_start.numel() != own_len.numel() + 1 or positions.numel() != slots.numel() or left.numel() != 2:
            raise ValueError("row_start needs one element more than own_len, positions as many as slots, left two")
        self.row_start, self.own_len, self.positions, self.slots, self.left = row_start, own_len, positions, slots, left
        self._c = _StepTables(*(t.data_ptr() for t in (row_start, own_len, positions, slots, left)))
        self._ref = ctypes.byref(self._c)
        self.requests, self.rows, self.device_index = own_len.numel(), positions.numel(), row_start.get_device()

    @classmethod
    def empty(cls, requests: int, rows: int, device="cuda"):
        import torch
        return cls(*(torch.empty(n, dtype=torch.int32, device=device) for n in (requests + 1, requests, rows, rows, 2)))


class Batch:
    """The requests of one step as attention reads them (see dec_batch): int32
    row_start [requests + 1], own_len [requests], block_table [requests,
    max_blocks]; max_new bounds the rows of one request; prefix_table holds the
    blocks of a prefix of prefix_len tokens that all requests share."""

    def __init__(self, row_start, own_len, block_table, max_new: int = 1, prefix_table=None, prefix_len: int = 0):
        _int32(row_start, "row_start")
        _int32(own_len, "own_len")
        _int32(block_table, "block_table", 2)
        if row_start.numel() != own_len.numel() + 1 or block_table.shape[0] != own_len.numel():
            raise ValueError("row_start needs one element more than own_len, block_table as many rows")
        if prefix_len > 0:
            _int32(prefix_table, "prefix_table")
        if any(t.device != own_len.device for t in (row_start, block_table) + ((prefix_table,) if prefix_len > 0 else ())):
            raise ValueError("the tables must be on one device")
        self.row_start, self.own_len, self.block_table, self.prefix_table = row_start, own_len, block_table, prefix_table
        self.max_new, self.prefix_len = int(max_new), int(prefix_len)
        self._c = _Batch(own_len.numel(), self.max_new, row_start.data_ptr(), own_len.data_ptr(),
                         block_table.data_ptr(), block_table.shape[1], prefix_table.data_ptr() if prefix_len > 0 else None,
                         self.prefix_len)
        self._ref = ctypes.byref(self._c)
        self.device_index = own_len.get_device()


ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


class Rope:
    """Rotary positions of the first rotary_dim elements of each head (see
    dec_rope and dec_rope_phases; rotary_dim 0: none). scaling: "none",
    "linear", "ntk", "bands" or "yarn" by `factor`; low and high are the turns
    within original_len between which "bands" (default 1 and 4) and "yarn"
    (1 and 32) blend."""

    def __init__(self, h: Handle, rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 8192.0, low: float = 1.0,
                 high: Optional[float] = None, magnitude: float = 1.0, stream=None):
        import torch
        if scaling not in ROPE_SCALING:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
        high = (4.0 if scaling == "bands" else 32.0) if high is None else high
        self.phases = None
        if rotary_dim:
            with _on_stream(stream):
                self.phases = torch.empty(max(rotary_dim // 2, 1), dtype=torch.int64, device=f"cuda:{h.device}")
            _check(_load().dec_rope_phases(h.ptr, self.phases.data_ptr(), int(rotary_dim), float(base),
                                           ROPE_SCALING[scaling], float(factor), float(original_len), float(low),
                                           float(high), _stream_of(h, stream)), "dec_rope_phases")
        self._c = _Rope(int(rotary_dim), 1 if interleaved else 0, float(magnitude), _ptr(self.phases))
        self._ref = ctypes.byref(self._c)
        self.device_index = h.device


def _described(h: Handle, thing, name: str) -> None:
    if thing.device_index != h.device:
        raise ValueError(f"{name} must be on the handle's device, cuda:{h.device}")


def dec_batch_tables(h: Handle, ctx_len, new_len, free_blocks, free_count, block_table, block_size: int,
                     out: Optional[StepTables] = None, rows: Optional[int] = None, position_offset: int = 0,
                     stream=None) -> StepTables:
    """Positions, slots and block-table entries of one step from the requests'
    lengths (int32 tensors); block_table [requests, max_blocks] is updated in
    place. free_count is at most free_blocks' elements (0 if it has none). `out`
    gives the output tensors, else they are made for `rows` rows."""
    dev = h.device
    n = ctx_len.numel()
    if out is None:
        if rows is None:
            raise ValueError("rows is required without out")
        with _on_stream(stream):
            out = StepTables.empty(n, rows, ctx_len.device)
    elif rows is not None and rows != out.rows:
        raise ValueError("rows differs from out's")
    _int32(block_table, "block_table", 2)
    width = block_table.shape[1]
    if block_table.shape[0] != n or out.requests != n or free_count.numel() < 1 or block_table.get_device() != dev:
        raise ValueError("block_table and out must be of as many requests as ctx_len, free_count of one value, all on "
                         "the handle's device")
    _described(h, out, "out")
    count = _ints_of(free_count, "free_count", dev)
    st = _load().dec_batch_tables(h.ptr, _ints_of(ctx_len, "ctx_len", dev), _ints_of(new_len, "new_len", dev, n), n,
                                  _ints_of(free_blocks, "free_blocks", dev) or count,  # no address without elements
                                  count, block_table.data_ptr(), width, block_size, position_offset, out.rows, out._ref,
                                  _stream_of(h, stream))
    if st:
        _check(st, "dec_batch_tables")
    return out


def dec_rope_append(h: Handle, rope: Rope, q, k, v, positions, slots, cache: KvCache, q_out=None, stream=None):
    """Turn q and k (bf16 [rows, heads * head_dim], rows may be strided) by their
    positions, write k and v into the cache at their slots; returns the turned
    q (q_out, which may be q; None with q None: only the cache is written)."""
    dev, d = h.device, cache.head_dim
    rows, width, ldk = _rows_of(k, "k", dev)
    rows_v, width_v, ldv = _rows_of(v, "v", dev)
    if rows_v != rows or width_v != width or width != cache.kv_heads * d:
        raise ValueError("k and v must be [rows, kv_heads * head_dim]")
    heads, ldq, ldqo, pq, pqo = 0, 0, 0, None, None
    if q is not None:
        rows_q, width_q, ldq = _rows_of(q, "q", dev)
        if rows_q != rows or width_q % d != 0:
            raise ValueError("q must be [rows, q_heads * head_dim]")
        heads = width_q // d
        if q_out is None:
            import torch
            with _on_stream(stream):
                q_out = torch.empty((rows, width_q), dtype=q.dtype, device=q.device)
        rows_o, width_o, ldqo = _rows_of(q_out, "q_out", dev)
        if rows_o != rows or width_o != width_q:
            raise ValueError("q_out must have q's shape")
        pq, pqo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    _described(h, cache, "cache")
    _described(h, rope, "rope")
    st = _load().dec_rope_append(h.ptr, rope._ref, pq, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, pqo, ldqo, rows,
                                 heads, _ints_of(positions, "positions", dev, rows),
                                 _ints_of(slots, "slots", dev, rows), cache._ref, _stream_of(h, stream))
    if st:
        _check(st, "dec_rope_append")
    return q_out


def dec_attention_workspace_size(h: Handle, M: int, q_heads: int, cache: KvCache, batch: Batch) -> int:
    nb = ctypes.c_size_t()
    _check(_load().dec_attention_workspace_size(h.ptr, int(M), int(q_heads), cache._ref, batch._ref,
                                                ctypes.byref(nb)), "dec_attention_workspace_size")
    return nb.value


def dec_attention(h: Handle, q, cache: KvCache, batch: Batch, scale: float, out=None, stream=None, ws=None):
    """Attention of a step's rows q (bf16 [M, q_heads * head_dim], rows may be
    strided) over the batch's shared prefix and own tokens in the cache. Without
    `out`, rows that belong to no request are zero. Without `ws`, the calls of one
    stream share a workspace: give graphs that may run at the same time one each
    (dec_attention_workspace_size bytes, any contents)."""
    dev = h.device
    M, width, ldq = _rows_of(q, "q", dev)
    if width % cache.head_dim != 0:
        raise ValueError("q must be [M, q_heads * head_dim]")
    heads = width // cache.head_dim
    if out is None:
        import torch
        with _on_stream(stream):
            out = torch.zeros((M, width), dtype=q.dtype, device=q.device)
    M_o, width_o, ldo = _rows_of(out, "out", dev)
    if M_o != M or width_o != width:
        raise ValueError("out must have q's shape")
    if batch.prefix_len > 0 and batch.prefix_table.numel() * cache.block_size < batch.prefix_len:
        raise ValueError("prefix_table holds fewer blocks than prefix_len tokens need")
    _described(h, cache, "cache")
    _described(h, batch, "batch")
    sp = _stream_of(h, stream)
    if ws is not None:
        nbytes = _ws_bytes(ws, dev)
    else:
        shape = (M, heads, cache.head_dim, cache.kv_heads, batch.prefix_len > 0)
        size = h._attention_ws.get(shape)
        if size is None:
            size = h._attention_ws[shape] = dec_attention_workspace_size(h, M, heads, cache, batch)
        ws = h.stream_workspace("attention", sp, size, stream)
        nbytes = ws.numel()
    st = _load().dec_attention(h.ptr, q.data_ptr(), ldq, cache._ref, batch._ref, scale, out.data_ptr(), ldo, M, heads,
                               ws.data_ptr(), nbytes, sp)
    if st:
        _check(st, "dec_attention")
    return out


class LayerAttention:
    """The attention core of one decode layer (see dec_layer_attention):
    positions and slots are int32 [M] (StepTables), rope None turns nothing."""

    def __init__(self, q_heads: int, scale: float, cache: KvCache, batch: Batch, positions, slots,
                 rope: Optional[Rope] = None):
        for n, t in (("positions", positions), ("slots", slots)):
            _int32(t, n)
        if positions.numel() != slots.numel() or positions.device != slots.device:
            raise ValueError("positions and slots must be of the same rows")
        if any(x is not None and x.device_index != positions.get_device() for x in (cache, batch, rope)):
            raise ValueError("cache, batch, rope, positions and slots must be on one device")
        if batch.prefix_len > 0 and batch.prefix_table.numel() * cache.block_size < batch.prefix_len:
            raise ValueError("prefix_table holds fewer blocks than prefix_len tokens need")
        self.q_heads, self.cache, self.batch, self.rope = int(q_heads), cache, batch, rope
        self.positions, self.slots = positions, slots
        self.rows, self.device_index = positions.numel(), positions.get_device()
        at = ctypes.addressof
        self._c = _LayerAttention(self.q_heads, float(scale), None if rope is None else at(rope._c), at(cache._c),
                                  at(batch._c), positions.data_ptr(), slots.data_ptr())
        self._ref = ctypes.byref(self._c)


def decode_layer_attention_workspace_size(h: Handle, weights: LayerWeights, attention: LayerAttention, M: int) -> int:
    nb = ctypes.c_size_t()
    cw = weights.c_struct()
    _check(_load().decode_layer_attention_workspace_size(h.ptr, ctypes.byref(cw), attention._ref, int(M),
                                                         ctypes.byref(nb)), "decode_layer_attention_workspace_size")
    return nb.value


def decode_layer_attention(h: Handle, weights: LayerWeights, attention: LayerAttention, hidden, trace=False,
                           stream=None, ws=None, _cw=None):
    """decode_layer with attention between the projections, in place on hidden
    bf16 [M,H]; trace as in decode_layer. Without `ws`, a workspace is made at the
    first call of a stream and shape, which cannot be one that is captured; the
    calls and captured graphs of one stream and shape share it: give graphs that
    may run at the same time one each (decode_layer_attention_workspace_size
    bytes, zeroed)."""
    import torch
    _require(hidden, torch.bfloat16, "hidden", 2)
    _described(h, attention, "attention")
    M = hidden.shape[0]
    cw = weights.c_struct() if _cw is None else _cw
    if hidden.get_device() != h.device or not hidden.is_contiguous() or attention.rows != M or hidden.shape[1] != cw.H:
        raise ValueError("hidden must be contiguous on the handle's device, as wide as the weights' H and with as many "
                         "rows as attention's positions")
    forms = dict(h1=(cw.H, torch.bfloat16), idx=(cw.k, torch.int32), w=(cw.k, torch.float32),
                 scores=(cw.E, torch.float32))
    for n, t in trace.items() if isinstance(trace, dict) else ():
        if t is not None and n in forms:
            width, dtype = forms[n]
            _require(t, dtype, n, 2)
            if t.shape[0] < M or t.shape[1] != width or not t.is_contiguous() or t.get_device() != h.device:
                raise ValueError(f"trace: {n} must be contiguous [{M}, {width}] (or more rows) on the handle's device")
    sp = _stream_of(h, stream)
    if ws is None:
        # one per stream and shape, kept until the handle closes: a captured graph may
        # hold its address, and its counters must stay as its own calls leave them
        c = attention.cache
        key = (sp, M, cw.H, cw.N_in, cw.K_out, cw.E, cw.k, cw.I, cw.Wg_s is not None, attention.q_heads, c.kv_heads,
               c.head_dim, attention.batch.prefix_len > 0)
        ws = h._layer_ws.get(key)
        if ws is None:
            # on the call's stream, which is another device's than the current one if the handle is
            with torch.cuda.stream(torch.cuda.current_stream(h.device) if stream is None else stream):
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("decode_layer_attention: the first call of a shape makes its zeroed workspace; "
                                       "make it before the capture, or pass ws")
                ws = torch.zeros(decode_layer_attention_workspace_size(h, weights, attention, M), dtype=torch.uint8,
                                 device=hidden.device)
            h._layer_ws[key] = ws
    out = trace if isinstance(trace, dict) else None
    if trace is True:
        with _on_stream(stream):
            out = {n: torch.empty((M, width), dtype=dtype, device=hidden.device) for n, (width, dtype) in forms.items()}
    tr = None
    if out is not None:
        tr = _LayerTrace()
        tr.h1, tr.idx, tr.w, tr.scores = (_ptr(out.get(n)) for n in ("h1", "idx", "w", "scores"))
    _check(_load().decode_layer_attention(h.ptr, ctypes.byref(cw), attention._ref, _ptr(hidden), M,
                                          ctypes.byref(tr) if tr is not None else None, _ptr(ws),
                                          _ws_bytes(ws, h.device), sp), "decode_layer_attention")
    return out


def dec_prefetch_l2(h: Handle, t, nbytes: Optional[int] = None, stream=None) -> None:
    n = t.numel() * t.element_size() if nbytes is None else int(nbytes)
    _check(_load().dec_prefetch_l2(h.ptr, _ptr(t), n, _stream(stream)), "dec_prefetch_l2")


def test_wait_timeout(h: Handle, stream=None) -> None:
    _check(_load().dec_test_wait_timeout(h.ptr, _stream(stream)), "dec_test_wait_timeout")

def test_routing_wait_timeout(h: Handle, tokens: int = 1, stream=None) -> None:
    _check(_load().dec_test_routing_wait_timeout(h.ptr, int(tokens), _stream(stream)),
           "dec_test_routing_wait_timeout")


def test_occupy_sms(h: Handle, ctas: int, hold_ns: int, stream=None) -> None:
    """Hold `ctas` SMs for hold_ns with a sleeping kernel on `stream` (a test hook)."""
    _check(_load().dec_test_occupy_sms(h.ptr, int(ctas), int(hold_ns), _stream(stream)), "dec_test_occupy_sms")


def test_delayed_copy(h: Handle, dst, src, delay_ns: int, stream=None) -> None:
    n = src.numel() * src.element_size()
    _check(_load().dec_test_delayed_copy(h.ptr, _ptr(dst), _ptr(src), n, int(delay_ns), _stream(stream)),
           "dec_test_delayed_copy")
