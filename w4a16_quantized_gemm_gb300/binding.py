"""Thin ctypes binding of ``include/tm_w4a16.h``, ``include/tm_w8a8.h``,
``include/tm_kvb.h`` and ``include/tm_lora.h`` (argument marshalling only).

Every step of the computation runs in the CUDA library; PyTorch provides
device memory and streams.  If the library is missing this module raises --
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

TM_OK = 0
_STATUS = {0: "ok", 1: "invalid argument", 2: "pointer not 16-byte aligned", 3: "unsupported configuration",
           4: "CUDA call failed", 5: "device barrier timeout", 6: "code or zero above 15",
           7: "request exceeds the static staging array"}

EXPORTS = ("tm_status_str", "tm_packed_bytes", "tm_pack_weights", "tm_unpack_weights", "tm_packed_info",
           "tm_packed_free", "tm_w4a16_gemm", "tm_w4a16_gemm_ex", "tm_gemm_plan", "tm_device_error",
           "tm_last_launch_count", "tm_quantize_rtn", "tm_w4a16_gemm_silu_mul", "tm_selftest_wait_timeout",
           "tm_kv_quantize", "tm_kv_decode_attention", "tm_kv_pack_v", "tm_w8a8_quantize_act", "tm_w8_pack",
           "tm_w8_unpack", "tm_w8_packed_info", "tm_w8_packed_free", "tm_w8a8_gemm", "tm_w8a8_gemm_ex",
           "tm_w8_quantize_weight", "tm_kv_append", "tm_w4a16_gemm_host", "tm_w4a16_gemm_host_batch",
           "tm_w8a8_quantize_act_f16", "tm_w8a8_gemm_f16", "tm_w4a16_gemm_host_static",
           "tm_w4a16_gemm_grouped", "tm_gemm_plan_grouped", "tm_kvb_append", "tm_kvb_attention",
           "tm_kvb_attention_workspace", "tm_kvb_evict", "tm_kvb_append_rope", "tm_kvb_attention_tree",
           "tm_kvb_attention_tree_workspace", "tm_kvb_accept", "tm_lora_add")

GROUP_MAX = 4  # TM_GROUP_MAX


class TMError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)} (status {status})")
        self.status = status


class KVBCacheStruct(ctypes.Structure):
    """``tm_kvb_cache``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("format", ctypes.c_int)]


class KVBBatchStruct(ctypes.Structure):
    """``tm_kvb_batch``."""
    _fields_ = [("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("B", ctypes.c_int), ("table_stride", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_len", ctypes.c_int), ("rows", ctypes.c_longlong)]


class KVBRopeStruct(ctypes.Structure):
    """``tm_kvb_rope``."""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int), ("dims", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("pos", ctypes.c_void_p)]


class LoraAdaptersStruct(ctypes.Structure):
    """``tm_lora_adapters``."""
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("n", ctypes.c_int),
                ("K", ctypes.c_int), ("N", ctypes.c_int), ("R", ctypes.c_int)]


class GemmConfig(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("split_k", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("stages", ctypes.c_int), ("warp_n", ctypes.c_int), ("tile_m", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class GemmProblem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("p", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("silu", ctypes.c_int)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None):
    """Load the CUDA library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing; run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, ci, csz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.tm_status_str.restype = ctypes.c_char_p
    lib.tm_status_str.argtypes = [ci]
    lib.tm_packed_bytes.restype = ci
    lib.tm_packed_bytes.argtypes = [ci, ci, ci, ctypes.POINTER(csz)]
    lib.tm_pack_weights.restype = ci
    lib.tm_pack_weights.argtypes = [vp, vp, vp, ci, ci, ci, ctypes.POINTER(vp)]
    lib.tm_unpack_weights.restype = ci
    lib.tm_unpack_weights.argtypes = [vp, vp, vp, vp]
    lib.tm_packed_info.restype = ci
    lib.tm_packed_info.argtypes = [vp, ctypes.POINTER(ci), ctypes.POINTER(ci), ctypes.POINTER(ci),
                                   ctypes.POINTER(csz)]
    lib.tm_packed_free.restype = None
    lib.tm_packed_free.argtypes = [vp]
    lib.tm_w4a16_gemm.restype = ci
    lib.tm_w4a16_gemm.argtypes = [vp, vp, vp, ci, vp]
    lib.tm_w4a16_gemm_ex.restype = ci
    lib.tm_w4a16_gemm_ex.argtypes = [vp, vp, vp, ci, ctypes.POINTER(GemmConfig), vp]
    lib.tm_w4a16_gemm_host.restype = ci
    lib.tm_w4a16_gemm_host.argtypes = [vp, vp, vp, ci, vp, vp, ctypes.POINTER(GemmConfig), vp]
    lib.tm_w4a16_gemm_host_static.restype = ci
    lib.tm_w4a16_gemm_host_static.argtypes = [vp, vp, vp, ci, ctypes.POINTER(GemmConfig), vp]
    lib.tm_w4a16_gemm_host_batch.restype = ci
    lib.tm_w4a16_gemm_host_batch.argtypes = [ci, ctypes.POINTER(vp), ctypes.POINTER(ci), vp, vp, vp, vp, vp]
    lib.tm_gemm_plan.restype = ci
    lib.tm_gemm_plan.argtypes = [vp, ci, ctypes.POINTER(GemmConfig), ctypes.POINTER(GemmConfig)]
    lib.tm_device_error.restype = ci
    lib.tm_device_error.argtypes = [ci, ctypes.POINTER(ctypes.c_uint32)]
    lib.tm_last_launch_count.restype = ci
    lib.tm_last_launch_count.argtypes = []
    lib.tm_kv_quantize.restype = ci
    lib.tm_kv_quantize.argtypes = [vp, ctypes.c_longlong, ci, ci, vp, vp, vp, vp]
    lib.tm_kv_pack_v.restype = ci
    lib.tm_kv_pack_v.argtypes = [vp, ci, ci, ci, ci, vp, vp]
    lib.tm_kv_append.restype = ci
    lib.tm_kv_append.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci] + [vp] * 7
    lib.tm_kv_decode_attention.restype = ci
    lib.tm_kv_decode_attention.argtypes = [vp] * 8 + [ci] * 7 + [vp, vp]
    lib.tm_selftest_wait_timeout.restype = ci
    lib.tm_selftest_wait_timeout.argtypes = [vp]
    lib.tm_w4a16_gemm_silu_mul.restype = ci
    lib.tm_w4a16_gemm_silu_mul.argtypes = [vp, vp, vp, ci, ctypes.POINTER(GemmConfig), vp]
    lib.tm_quantize_rtn.restype = ci
    lib.tm_quantize_rtn.argtypes = [vp, ci, ci, ci, vp, vp, vp, vp]
    lib.tm_w8a8_quantize_act.restype = ci
    lib.tm_w8a8_quantize_act.argtypes = [vp, ci, ci, vp, vp, vp]
    lib.tm_w8_pack.restype = ci
    lib.tm_w8_pack.argtypes = [vp, vp, ci, ci, ctypes.POINTER(vp)]
    lib.tm_w8_unpack.restype = ci
    lib.tm_w8_unpack.argtypes = [vp, vp, vp]
    lib.tm_w8_packed_info.restype = ci
    lib.tm_w8_packed_info.argtypes = [vp, ctypes.POINTER(ci), ctypes.POINTER(ci), ctypes.POINTER(csz)]
    lib.tm_w8_packed_free.restype = None
    lib.tm_w8_packed_free.argtypes = [vp]
    lib.tm_w8a8_gemm.restype = ci
    lib.tm_w8a8_gemm.argtypes = [vp, vp, vp, vp, ci, ci, vp]
    lib.tm_w8_quantize_weight.restype = ci
    lib.tm_w8_quantize_weight.argtypes = [vp, ci, ci, vp, vp, vp]
    lib.tm_w8a8_gemm_ex.restype = ci
    lib.tm_w8a8_gemm_ex.argtypes = [vp, vp, vp, vp, ci, ci, ci, vp]
    lib.tm_w8a8_quantize_act_f16.restype = ci
    lib.tm_w8a8_quantize_act_f16.argtypes = [vp, ci, ci, vp, vp, vp]
    lib.tm_w8a8_gemm_f16.restype = ci
    lib.tm_w8a8_gemm_f16.argtypes = [vp, vp, vp, vp, ci, ci, ci, vp]
    lib.tm_w4a16_gemm_grouped.argtypes = [ctypes.POINTER(GemmProblem), ci, ci, ctypes.POINTER(GemmConfig), vp]
    lib.tm_gemm_plan_grouped.argtypes = [ctypes.POINTER(GemmProblem), ci, ci, ctypes.POINTER(GemmConfig),
                                         ctypes.POINTER(GemmConfig), ctypes.POINTER(ci)]
    pc, pb, ll = ctypes.POINTER(KVBCacheStruct), ctypes.POINTER(KVBBatchStruct), ctypes.c_longlong
    lib.tm_kvb_append.restype = ci
    lib.tm_kvb_append.argtypes = [pc, pb, vp, ll, vp, ll, ci, vp, ll, vp]
    for query in (lib.tm_kvb_attention_workspace, lib.tm_kvb_attention_tree_workspace):
        query.restype = ci
        query.argtypes = [pc, pb, ci, ci, ctypes.POINTER(csz)]
    lib.tm_kvb_attention.restype = ci
    lib.tm_kvb_attention.argtypes = [pc, pb, vp, ll, ci, ci, ctypes.c_float, vp, vp, vp, vp, ll, vp, csz, vp]
    lib.tm_kvb_evict.restype = ci
    lib.tm_kvb_evict.argtypes = [pc, pb, vp, ci, vp, ll, vp, ll, ci, ci, ci, vp, vp, vp]
    lib.tm_kvb_append_rope.restype = ci
    lib.tm_kvb_append_rope.argtypes = [pc, pb, vp, ll, vp, ll, vp, ll, ci, vp, ll, ctypes.POINTER(KVBRopeStruct), ci, vp,
                                       ll, vp]
    lib.tm_kvb_attention_tree.restype = ci
    lib.tm_kvb_attention_tree.argtypes = [pc, pb, vp, ll, ci, ci, ctypes.c_float, vp, ll, vp, vp, vp, vp, ll, vp, csz, vp]
    lib.tm_kvb_accept.restype = ci
    lib.tm_kvb_accept.argtypes = [pc, pb, vp, ci, vp, vp, ll, vp, vp]
    lib.tm_lora_add.restype = ci
    lib.tm_lora_add.argtypes = [ctypes.POINTER(LoraAdaptersStruct), vp, ll, vp, ll, vp, ll, ll, vp, vp, ci, vp]
    _lib = lib
    return lib


def _check(st: int, what: str):
    if st != TM_OK:
        raise TMError(st, what)


def status_str(st: int) -> str:
    return load().tm_status_str(st).decode()


def packed_bytes(K: int, N: int, g: int) -> int:
    out = ctypes.c_size_t()
    _check(load().tm_packed_bytes(K, N, g, ctypes.byref(out)), "tm_packed_bytes")
    return out.value


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Device memory for a call on ``stream`` (None: the current one).  It is that stream's own: a block that
    the current stream gave back may still be in use by work that is pending there, which ``stream`` does not
    wait for.  The caller may use the tensor on its current stream as well."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _contiguous(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """t, or its copy made on the call's stream, in that stream's memory."""
    if stream is None or t.is_contiguous():
        return t.contiguous()
    with torch.cuda.stream(stream):
        return t.contiguous()


class PackedWeights:
    """Owns a ``tm_packed`` handle (device memory on the device of ``q``)."""

    def __init__(self, q: torch.Tensor, z: torch.Tensor, s: torch.Tensor, g: int):
        lib = load()
        K, N = q.shape
        handle = ctypes.c_void_p()
        with torch.cuda.device(q.device):
            st = lib.tm_pack_weights(_dev(q, torch.uint8, "q"), _dev(z, torch.uint8, "z"),
                                     _dev(s, torch.float16, "s"), K, N, g, ctypes.byref(handle))
        _check(st, "tm_pack_weights")
        self._h = handle
        self.K, self.N, self.g = K, N, g
        self.device = q.device
        b = ctypes.c_size_t()
        _check(lib.tm_packed_info(handle, None, None, None, ctypes.byref(b)), "tm_packed_info")
        self.nbytes = b.value

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("packed weights were freed")
        return self._h

    def unpack(self):
        q = torch.empty((self.K, self.N), dtype=torch.uint8, device=self.device)
        z = torch.empty((self.K // self.g, self.N), dtype=torch.uint8, device=self.device)
        s = torch.empty((self.K // self.g, self.N), dtype=torch.float16, device=self.device)
        with torch.cuda.device(self.device):
            _check(load().tm_unpack_weights(self.handle, q.data_ptr(), z.data_ptr(), s.data_ptr()),
                   "tm_unpack_weights")
        return q, z, s

    def free(self):
        if self._h is not None:
            load().tm_packed_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def pack(q: torch.Tensor, z: torch.Tensor, s: torch.Tensor, g: int) -> PackedWeights:
    return PackedWeights(q, z, s, g)


def _cfg(config) -> Optional[GemmConfig]:
    if config is None:
        return None
    if isinstance(config, GemmConfig):
        return config
    c = GemmConfig()
    for k, v in dict(config).items():
        setattr(c, k, int(v))
    return c


def plan(w: PackedWeights, M: int, config=None) -> dict:
    out = GemmConfig()
    c = _cfg(config)
    _check(load().tm_gemm_plan(w.handle, M, ctypes.byref(c) if c else None, ctypes.byref(out)), "tm_gemm_plan")
    return out.as_dict()


def gemm(X: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None, config=None,
         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Y = X . dequant(W) on the GPU.

    X: fp16 [M][K].  On a CUDA tensor the call is asynchronous on ``stream``
    (default: the current stream).  On a CPU tensor (pinned for speed) X is
    copied to the device, the product runs, and Y comes back to the host --
    the end-to-end form of the same call.
    """
    if X.dim() != 2 or X.shape[1] != w.K or X.dtype != torch.float16:
        raise ValueError("X must be fp16 [M][K]")
    if not X.is_cuda:
        return _gemm_host(X, w, out, config, stream)
    M = X.shape[0]
    if out is None:
        out = _empty((M, w.N), torch.float16, X.device, stream)
    elif out.shape != (M, w.N) or out.dtype != torch.float16 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA fp16 [M][N] tensor")
    X = _contiguous(X, stream)
    s = stream if stream is not None else torch.cuda.current_stream(X.device)
    c = _cfg(config)
    lib = load()
    if c is None:
        st = lib.tm_w4a16_gemm(X.data_ptr(), w.handle, out.data_ptr(), M, ctypes.c_void_p(s.cuda_stream))
    else:
        st = lib.tm_w4a16_gemm_ex(X.data_ptr(), w.handle, out.data_ptr(), M, ctypes.byref(c),
                                  ctypes.c_void_p(s.cuda_stream))
    _check(st, "tm_w4a16_gemm")
    return out


def gemm_silu_mul(X: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None, config=None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """H = silu(X . W_gate) * (X . W_up) from one packed gate/up weight whose
    columns interleave gate and up in blocks of 4 (see tm_w4a16_gemm_silu_mul).
    X: CUDA fp16 [M][K]; returns fp16 [M][N/2]; asynchronous on ``stream``."""
    if X.dim() != 2 or X.shape[1] != w.K or X.dtype != torch.float16 or not X.is_cuda:
        raise ValueError("X must be a CUDA fp16 [M][K] tensor")
    M = X.shape[0]
    if out is None:
        out = _empty((M, w.N // 2), torch.float16, X.device, stream)
    elif out.shape != (M, w.N // 2) or out.dtype != torch.float16 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA fp16 [M][N/2] tensor")
    X = _contiguous(X, stream)
    s = stream if stream is not None else torch.cuda.current_stream(X.device)
    c = _cfg(config)
    _check(load().tm_w4a16_gemm_silu_mul(X.data_ptr(), w.handle, out.data_ptr(), M,
                                         ctypes.byref(c) if c else None, ctypes.c_void_p(s.cuda_stream)),
           "tm_w4a16_gemm_silu_mul")
    return out


def _problems(items, M, check_out=True):
    arr = (GemmProblem * len(items))()
    for i, (X, w, out, silu) in enumerate(items):
        arr[i].X = X.data_ptr() if X is not None else None
        arr[i].p = w.handle
        arr[i].Y = out.data_ptr() if out is not None else None
        arr[i].silu = 1 if silu else 0
    return arr


def plan_grouped(weights, M: int, config=None, silu=None) -> dict:
    """Settings tm_w4a16_gemm_grouped would use for these packed weights at M
    rows; "splits" lists each product's split along K ("split_k" is the
    launch's cluster size)."""
    silu = list(silu) if silu is not None else [False] * len(weights)
    arr = _problems([(None, w, None, f) for w, f in zip(weights, silu)], M)
    out = GemmConfig()
    splits = (ctypes.c_int * max(1, len(weights)))()
    c = _cfg(config)
    _check(load().tm_gemm_plan_grouped(arr, len(weights), M, ctypes.byref(c) if c else None, ctypes.byref(out),
                                       splits), "tm_gemm_plan_grouped")
    d = out.as_dict()
    d["splits"] = [splits[i] for i in range(len(weights))]
    return d


def gemm_grouped(problems, config=None, stream: Optional[torch.cuda.Stream] = None):
    """Independent products of the same M in one launch (tm_w4a16_gemm_grouped).

    problems: up to GROUP_MAX tuples (X, w, out, silu) -- X CUDA fp16 [M][K],
    w PackedWeights, out a CUDA fp16 [M][N] tensor ([M][N/2] with silu) or
    None to allocate, silu a bool.  No out may overlap any X or another out.
    Returns the list of outputs; asynchronous on ``stream``."""
    items = []
    M = None
    for X, w, out, silu in problems:
        if X.dim() != 2 or X.shape[1] != w.K or X.dtype != torch.float16 or not X.is_cuda:
            raise ValueError("every X must be a CUDA fp16 [M][K] tensor")
        if M is None:
            M = X.shape[0]
        elif X.shape[0] != M:
            raise ValueError("every X must have the same number of rows")
        cols = w.N // 2 if silu else w.N
        if out is None:
            out = _empty((M, cols), torch.float16, X.device, stream)
        elif out.shape != (M, cols) or out.dtype != torch.float16 or not out.is_cuda or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous CUDA fp16 [{M}][{cols}] tensor")
        items.append((_contiguous(X, stream), w, out, bool(silu)))
    if not items:
        raise ValueError("at least one problem")
    s = stream if stream is not None else torch.cuda.current_stream(items[0][0].device)
    c = _cfg(config)
    arr = _problems(items, M)
    _check(load().tm_w4a16_gemm_grouped(arr, len(items), M, ctypes.byref(c) if c else None,
                                        ctypes.c_void_p(s.cuda_stream)), "tm_w4a16_gemm_grouped")
    return [it[2] for it in items]


def _gemm_host(X, w, out, config, stream):
    return gemm_host(X, w, out, config, stream)


def _host_fp16(t: torch.Tensor, shape, name: str):
    if t.is_cuda or t.dtype != torch.float16 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host fp16 tensor of shape {tuple(shape)}")


def _staging(t: Optional[torch.Tensor], numel: int, device, name: str, stream) -> torch.Tensor:
    if t is None:
        return _empty(numel, torch.float16, device, stream)
    if not t.is_cuda or t.dtype != torch.float16 or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be a contiguous CUDA fp16 buffer of at least {numel} elements")
    return t


def gemm_host(X: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None, config=None,
              stream: Optional[torch.cuda.Stream] = None, X_dev: Optional[torch.Tensor] = None,
              Y_dev: Optional[torch.Tensor] = None, sync: bool = True) -> torch.Tensor:
    """tm_w4a16_gemm_host: X fp16 [M][K] in host memory (pinned for speed) is
    copied to the device buffer ``X_dev``, the product runs into ``Y_dev``, and
    the result comes back into ``out`` (host fp16 [M][N]; pinned, allocated
    when None).  Staging buffers are allocated when None.  With ``sync`` the
    call waits for the stream; otherwise read ``out`` after synchronising it."""
    if X.dim() != 2:
        raise ValueError("X must be fp16 [M][K]")
    M = X.shape[0]
    _host_fp16(X, (M, w.K), "X")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.float16, pin_memory=True)
    _host_fp16(out, (M, w.N), "out")
    X_dev = _staging(X_dev, M * w.K, w.device, "X_dev", stream)
    Y_dev = _staging(Y_dev, M * w.N, w.device, "Y_dev", stream)
    s = stream if stream is not None else torch.cuda.current_stream(w.device)
    c = _cfg(config)
    _check(load().tm_w4a16_gemm_host(X.data_ptr(), w.handle, out.data_ptr(), M, X_dev.data_ptr(), Y_dev.data_ptr(),
                                     ctypes.byref(c) if c else None, ctypes.c_void_p(s.cuda_stream)),
           "tm_w4a16_gemm_host")
    if sync:
        s.synchronize()
    return out


STATIC_STAGING_BYTES = 8 << 20  # TM_STATIC_STAGING_BYTES


def gemm_host_static(X: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None, config=None,
                     stream: Optional[torch.cuda.Stream] = None, sync: bool = True) -> torch.Tensor:
    """tm_w4a16_gemm_host_static: as ``gemm_host``, but staged through the
    library's fixed device array, so that the call allocates no device memory
    (``out``, the host result, is allocated here when None).  Calls share the
    array: issue them on one stream."""
    if X.dim() != 2:
        raise ValueError("X must be fp16 [M][K]")
    M = X.shape[0]
    _host_fp16(X, (M, w.K), "X")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.float16, pin_memory=True)
    _host_fp16(out, (M, w.N), "out")
    s = stream if stream is not None else torch.cuda.current_stream(w.device)
    c = _cfg(config)
    with torch.cuda.device(w.device):
        _check(load().tm_w4a16_gemm_host_static(X.data_ptr(), w.handle, out.data_ptr(), M,
                                                ctypes.byref(c) if c else None, ctypes.c_void_p(s.cuda_stream)),
               "tm_w4a16_gemm_host_static")
    if sync:
        s.synchronize()
    return out


class HostBatch:
    """A fixed list of products with host inputs and outputs for
    tm_w4a16_gemm_host_batch: ``X_host`` / ``Y_host`` are pinned buffers that
    hold every X_i / Y_i back to back (``x(i)`` and ``y(i)`` are views of
    them), staged through one device buffer each way."""

    def __init__(self, weights, Ms, device=None):
        if len(weights) != len(Ms) or any(m < 0 for m in Ms):
            raise ValueError("one non-negative M per weight")
        self.weights, self.Ms = list(weights), [int(m) for m in Ms]
        dev = device if device is not None else (self.weights[0].device if self.weights else 0)
        self.x_off, self.y_off = [0], [0]
        for w, m in zip(self.weights, self.Ms):
            self.x_off.append(self.x_off[-1] + m * w.K)
            self.y_off.append(self.y_off[-1] + m * w.N)
        self.X_host = torch.empty(self.x_off[-1], dtype=torch.float16, pin_memory=True)
        self.Y_host = torch.empty(self.y_off[-1], dtype=torch.float16, pin_memory=True)
        self.X_dev = torch.empty(self.x_off[-1], dtype=torch.float16, device=dev)
        self.Y_dev = torch.empty(self.y_off[-1], dtype=torch.float16, device=dev)
        n = len(self.weights)
        self._p = (ctypes.c_void_p * max(1, n))(*[w.handle for w in self.weights])
        self._m = (ctypes.c_int * max(1, n))(*self.Ms)

    def x(self, i: int) -> torch.Tensor:
        return self.X_host[self.x_off[i]:self.x_off[i + 1]].view(self.Ms[i], self.weights[i].K)

    def y(self, i: int) -> torch.Tensor:
        return self.Y_host[self.y_off[i]:self.y_off[i + 1]].view(self.Ms[i], self.weights[i].N)

    def run(self, stream: Optional[torch.cuda.Stream] = None, sync: bool = True):
        s = stream if stream is not None else torch.cuda.current_stream(self.X_dev.device)
        _check(load().tm_w4a16_gemm_host_batch(len(self.weights), self._p, self._m, self.X_host.data_ptr(),
                                               self.Y_host.data_ptr(), self.X_dev.data_ptr(),
                                               self.Y_dev.data_ptr(), ctypes.c_void_p(s.cuda_stream)),
               "tm_w4a16_gemm_host_batch")
        if sync:
            s.synchronize()


def quantize_rtn(W: torch.Tensor, g: int, stream: Optional[torch.cuda.Stream] = None):
    """Round-to-nearest INT4 quantisation of fp16 W [K][N] on the GPU:
    returns (q uint8 [K][N], z uint8 [K/g][N], s fp16 [K/g][N]), the inputs of
    ``pack``.  Asynchronous on ``stream`` (default: the current stream)."""
    if W.dim() != 2 or W.dtype != torch.float16:
        raise ValueError("W must be fp16 [K][N]")
    K, N = W.shape
    Wd = _contiguous(W, stream)
    _dev(Wd, torch.float16, "W")
    q = _empty((K, N), torch.uint8, Wd.device, stream)
    z = _empty((K // g if g > 0 else 0, N), torch.uint8, Wd.device, stream)
    s = _empty((K // g if g > 0 else 0, N), torch.float16, Wd.device, stream)
    st = stream if stream is not None else torch.cuda.current_stream(Wd.device)
    with torch.cuda.device(Wd.device):
        _check(load().tm_quantize_rtn(Wd.data_ptr(), K, N, g, q.data_ptr(), z.data_ptr(), s.data_ptr(),
                                      ctypes.c_void_p(st.cuda_stream)), "tm_quantize_rtn")
    return q, z, s


def kv_quantize(X: torch.Tensor, bits: int, stream: Optional[torch.cuda.Stream] = None):
    """Quantise fp16 vectors X [..., D] (one per (token, head)) to int8 / int4:
    returns (codes uint8 [..., D or D/2], s fp16 [...], z uint8 [...])."""
    if X.dtype != torch.float16 or not X.is_cuda or X.dim() < 1:
        raise ValueError("X must be a CUDA fp16 tensor [..., D]")
    X = _contiguous(X, stream)
    D = X.shape[-1]
    lead = tuple(X.shape[:-1])
    rows = X.numel() // D if D else 0
    codes = _empty(lead + (D if bits == 8 else D // 2,), torch.uint8, X.device, stream)
    s = _empty(lead, torch.float16, X.device, stream)
    z = _empty(lead, torch.uint8, X.device, stream)
    st = stream if stream is not None else torch.cuda.current_stream(X.device)
    _check(load().tm_kv_quantize(X.data_ptr(), rows, D, bits, codes.data_ptr(), s.data_ptr(), z.data_ptr(),
                                 ctypes.c_void_p(st.cuda_stream)), "tm_kv_quantize")
    return codes, s, z


def kv_pack_v(codes: torch.Tensor, bits: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Value codes [B][Hkv][L][D*bits/8] -> the 16-token tiles in MMA lane
    order the attention kernel reads (see tm_kv_pack_v)."""
    if codes.dim() != 4 or codes.dtype != torch.uint8 or codes.shape[3] != 128 * bits // 8:
        raise ValueError("codes must be uint8 [B][Hkv][L][128*bits/8]")
    B, Hkv, L, _ = codes.shape
    codes = _contiguous(codes, stream)
    tiles = _empty(B * Hkv * L * 128 * bits // 8, torch.uint8, codes.device, stream)
    st = stream if stream is not None else torch.cuda.current_stream(codes.device)
    _check(load().tm_kv_pack_v(codes.data_ptr(), B, L, Hkv, bits, tiles.data_ptr(), ctypes.c_void_p(st.cuda_stream)),
           "tm_kv_pack_v")
    return tiles


def kv_append(Kn: torch.Tensor, Vn: torch.Tensor, pos: torch.Tensor, k: tuple, v: tuple, bits: int,
              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise the new token's K and V (fp16 [B][Hkv][D]) into the head-major
    cache at positions pos (int32 [B]); k = (codes, s, z), v = (tiles, s, z) as
    for kv_decode_attention (see tm_kv_append)."""
    kc, ks, kz = k
    vc, vs, vz = v
    B, Hkv, D = Kn.shape
    if tuple(Vn.shape) != (B, Hkv, D) or kc.dim() != 4 or kc.shape[0] != B or kc.shape[1] != Hkv:
        raise ValueError("Kn, Vn must be [B][Hkv][D] over a [B][Hkv][L][.] cache")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (B,):
        raise ValueError("pos must be int32 [B]")
    L = kc.shape[2]
    ts = [Kn, Vn, pos, kc, ks, kz, vc, vs, vz]
    if any((not t.is_cuda) or (not t.is_contiguous()) for t in ts):
        raise ValueError("all tensors must be contiguous CUDA tensors")
    st = stream if stream is not None else torch.cuda.current_stream(Kn.device)
    _check(load().tm_kv_append(Kn.data_ptr(), Vn.data_ptr(), pos.data_ptr(), B, Hkv, L, D, bits, kc.data_ptr(),
                               ks.data_ptr(), kz.data_ptr(), vc.data_ptr(), vs.data_ptr(), vz.data_ptr(),
                               ctypes.c_void_p(st.cuda_stream)), "tm_kv_append")


def kv_decode_attention(Q: torch.Tensor, k: tuple, v: tuple, lengths: torch.Tensor, bits: int, split: int = 0,
                        out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Q fp16 [B][Hq][D]; k = (codes [B][Hkv][L][D*bits/8], s fp16 [B][Hkv][L],
    z uint8 [B][Hkv][L]) -- the head-major cache; v = (tiles from kv_pack_v,
    s, z as for k); lengths int32 [B].  Returns fp16 [B][Hq][D]."""
    B, Hq, D = Q.shape
    kc, ks, kz = k
    vc, vs, vz = v
    if kc.dim() != 4 or kc.shape[0] != B or tuple(lengths.shape) != (B,):
        raise ValueError("key codes must be [B][Hkv][L][D*bits/8] and lengths [B], B as in Q")
    if Q.dtype != torch.float16 or kc.dtype != torch.uint8 or vc.dtype != torch.uint8:
        raise ValueError("Q must be fp16 and the codes uint8")
    Hkv, L = kc.shape[1], kc.shape[2]
    if kc.shape[3] != D * bits // 8 or vc.numel() != B * Hkv * L * D * bits // 8:
        raise ValueError("code sizes do not match D and bits")
    if tuple(ks.shape) != (B, Hkv, L) or tuple(vs.shape) != (B, Hkv, L):
        raise ValueError("scales and zeros must be [B][Hkv][L] like the key codes")
    if out is None:
        out = _empty((B, Hq, D), torch.float16, Q.device, stream)
    ts = [Q, kc, ks, kz, vc, vs, vz, lengths]
    if any((not t.is_cuda) or (not t.is_contiguous()) for t in ts) or lengths.dtype != torch.int32:
        raise ValueError("all inputs must be contiguous CUDA tensors; lengths int32")
    st = stream if stream is not None else torch.cuda.current_stream(Q.device)
    _check(load().tm_kv_decode_attention(*(t.data_ptr() for t in ts), B, Hq, Hkv, L, D, bits, split,
                                         out.data_ptr(), ctypes.c_void_p(st.cuda_stream)), "tm_kv_decode_attention")
    return out


def selftest_wait_timeout(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Launch the bounded-wait self-test (see tm_selftest_wait_timeout)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(load().tm_selftest_wait_timeout(ctypes.c_void_p(s.cuda_stream)), "tm_selftest_wait_timeout")


def device_error(clear: bool = True) -> int:
    bits = ctypes.c_uint32()
    st = load().tm_device_error(1 if clear else 0, ctypes.byref(bits))
    if st not in (TM_OK, 5):
        raise TMError(st, "tm_device_error")
    return bits.value


def last_launch_count() -> int:
    return load().tm_last_launch_count()


# ------------------------------------------------------------------ W8A8 ---

def w8a8_quantize_act(X: torch.Tensor, out: Optional[tuple] = None, stream: Optional[torch.cuda.Stream] = None):
    """Per-token int8 quantisation of fp16 X [M][K] (see tm_w8a8_quantize_act):
    returns (xq int8 [M][K], sx fp32 [M]), into `out` when given."""
    if X.dim() != 2 or X.dtype != torch.float16:
        raise ValueError("X must be fp16 [M][K]")
    M, K = X.shape
    if out is None:
        xq = _empty((M, K), torch.int8, X.device, stream)
        sx = _empty((M,), torch.float32, X.device, stream)
    else:
        xq, sx = out
        if tuple(xq.shape) != (M, K) or tuple(sx.shape) != (M,):
            raise ValueError("out must be (int8 [M][K], fp32 [M])")
    st = stream if stream is not None else torch.cuda.current_stream(X.device)
    _check(load().tm_w8a8_quantize_act(_dev(X, torch.float16, "X"), M, K, _dev(xq, torch.int8, "xq"),
                                       _dev(sx, torch.float32, "sx"), ctypes.c_void_p(st.cuda_stream)),
           "tm_w8a8_quantize_act")
    return xq, sx


def w8a8_quantize_act_f16(X: torch.Tensor, out: Optional[tuple] = None, stream: Optional[torch.cuda.Stream] = None):
    """tm_w8a8_quantize_act_f16: the same per-token codes as exact fp16 integers:
    returns (xq16 fp16 [M][K], sx fp32 [M]), into `out` when given."""
    if X.dim() != 2 or X.dtype != torch.float16:
        raise ValueError("X must be fp16 [M][K]")
    M, K = X.shape
    if out is None:
        xq = _empty((M, K), torch.float16, X.device, stream)
        sx = _empty((M,), torch.float32, X.device, stream)
    else:
        xq, sx = out
        if tuple(xq.shape) != (M, K) or tuple(sx.shape) != (M,):
            raise ValueError("out must be (fp16 [M][K], fp32 [M])")
    st = stream if stream is not None else torch.cuda.current_stream(X.device)
    _check(load().tm_w8a8_quantize_act_f16(_dev(X, torch.float16, "X"), M, K, _dev(xq, torch.float16, "xq16"),
                                           _dev(sx, torch.float32, "sx"), ctypes.c_void_p(st.cuda_stream)),
           "tm_w8a8_quantize_act_f16")
    return xq, sx


def w8_quantize_weight(W: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
    """Per-output-channel int8 quantisation of fp16 W [K][N] on the GPU (see
    tm_w8_quantize_weight): returns (q int8 [K][N], sw fp32 [N]), the inputs of
    ``pack_w8``."""
    if W.dim() != 2 or W.dtype != torch.float16:
        raise ValueError("W must be fp16 [K][N]")
    K, N = W.shape
    q = _empty((K, N), torch.int8, W.device, stream)
    sw = _empty((N,), torch.float32, W.device, stream)
    st = stream if stream is not None else torch.cuda.current_stream(W.device)
    _check(load().tm_w8_quantize_weight(_dev(W, torch.float16, "W"), K, N, q.data_ptr(), sw.data_ptr(),
                                        ctypes.c_void_p(st.cuda_stream)), "tm_w8_quantize_weight")
    return q, sw


class W8Packed:
    """Owns a ``tm_w8_packed`` handle (device memory on the device of ``q``)."""

    def __init__(self, q: torch.Tensor, sw: torch.Tensor):
        lib = load()
        K, N = q.shape
        handle = ctypes.c_void_p()
        with torch.cuda.device(q.device):
            st = lib.tm_w8_pack(_dev(q, torch.int8, "q"), _dev(sw, torch.float32, "sw"), K, N, ctypes.byref(handle))
        _check(st, "tm_w8_pack")
        self._h = handle
        self.K, self.N = K, N
        self.device = q.device
        b = ctypes.c_size_t()
        _check(lib.tm_w8_packed_info(handle, None, None, ctypes.byref(b)), "tm_w8_packed_info")
        self.nbytes = b.value

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("packed weights were freed")
        return self._h

    def unpack(self):
        q = torch.empty((self.K, self.N), dtype=torch.int8, device=self.device)
        sw = torch.empty((self.N,), dtype=torch.float32, device=self.device)
        with torch.cuda.device(self.device):
            _check(load().tm_w8_unpack(self.handle, q.data_ptr(), sw.data_ptr()), "tm_w8_unpack")
        return q, sw

    def free(self):
        if self._h is not None:
            load().tm_w8_packed_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def pack_w8(q: torch.Tensor, sw: torch.Tensor) -> W8Packed:
    return W8Packed(q, sw)


def w8a8_gemm(xq: torch.Tensor, sx: torch.Tensor, w: W8Packed, out: Optional[torch.Tensor] = None, split: int = 0,
              tile_m: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Y = fp16(sx sw^T (xq . q_w)) for int8 xq [M][K] and fp32 sx [M] (tm_w8a8_gemm_ex)."""
    if xq.dim() != 2 or xq.shape[1] != w.K:
        raise ValueError("xq must be int8 [M][K]")
    M = xq.shape[0]
    if tuple(sx.shape) != (M,):
        raise ValueError("sx must be fp32 [M]")
    if out is None:
        out = _empty((M, w.N), torch.float16, xq.device, stream)
    if tuple(out.shape) != (M, w.N):
        raise ValueError("out must be fp16 [M][N]")
    st = stream if stream is not None else torch.cuda.current_stream(xq.device)
    _check(load().tm_w8a8_gemm_ex(_dev(xq, torch.int8, "xq"), _dev(sx, torch.float32, "sx"), w.handle,
                                  _dev(out, torch.float16, "out"), M, split, tile_m, ctypes.c_void_p(st.cuda_stream)),
           "tm_w8a8_gemm_ex")
    return out


def w8a8_gemm_f16(xq16: torch.Tensor, sx: torch.Tensor, w: W8Packed, out: Optional[torch.Tensor] = None,
                  split: int = 0, tile_m: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """tm_w8a8_gemm_f16: the product with the codes as fp16 integers [M][K]
    (from w8a8_quantize_act_f16), on the tensor-memory kernel for every M."""
    if xq16.dim() != 2 or xq16.shape[1] != w.K:
        raise ValueError("xq16 must be fp16 [M][K]")
    M = xq16.shape[0]
    if tuple(sx.shape) != (M,):
        raise ValueError("sx must be fp32 [M]")
    if out is None:
        out = _empty((M, w.N), torch.float16, xq16.device, stream)
    if tuple(out.shape) != (M, w.N):
        raise ValueError("out must be fp16 [M][N]")
    st = stream if stream is not None else torch.cuda.current_stream(xq16.device)
    _check(load().tm_w8a8_gemm_f16(_dev(xq16, torch.float16, "xq16"), _dev(sx, torch.float32, "sx"), w.handle,
                                   _dev(out, torch.float16, "out"), M, split, tile_m, ctypes.c_void_p(st.cuda_stream)),
           "tm_w8a8_gemm_f16")
    return out


# ---- paged 8-bit KV cache with a scale per page and head (include/tm_kvb.h) ----

_KVB_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}
_KVB_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


class KVBlocks:
    """The pages of one layer: codes ``k``, ``v`` [pages][Hkv][T][D] (int8 or
    float8_e4m3fn: the dtype is the format) and scales ``ks``, ``vs`` fp32
    [pages][Hkv], all contiguous on one device.  ``KVBlocks.empty`` allocates them."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, ks: torch.Tensor, vs: torch.Tensor):
        if k.dim() != 4 or k.dtype not in _KVB_FORMATS:
            raise ValueError("k must be int8 or float8_e4m3fn [pages][Hkv][T][D]")
        if v.shape != k.shape:
            raise ValueError("v must have the shape of k")
        for t, name in ((ks, "ks"), (vs, "vs")):
            if t.shape != k.shape[:2]:
                raise ValueError(f"{name} must be fp32 [pages][Hkv]")
        pages, Hkv, T, D = k.shape
        if T not in (16, 32, 64, 128) or D not in (64, 128) or Hkv < 1:
            raise ValueError("a page holds 16, 32, 64 or 128 tokens of Hkv >= 1 heads of 64 or 128 dimensions")
        if not (k.device == v.device == ks.device == vs.device):
            raise ValueError("k, v, ks and vs must be on one device")
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.pages, self.Hkv, self.T, self.D = pages, Hkv, T, D
        self.device = k.device
        self.index = self.device.index
        self._c = KVBCacheStruct(_dev(k, k.dtype, "k"), _dev(v, k.dtype, "v"), _dev(ks, torch.float32, "ks"),
                           _dev(vs, torch.float32, "vs"), pages, Hkv, T, D, _KVB_FORMATS[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages: int, Hkv: int, T: int, D: int, dtype=torch.int8, device="cuda") -> "KVBlocks":
        """Pages of zeros."""
        codes = lambda: torch.zeros((pages, Hkv, T, D), dtype=torch.uint8, device=device).view(dtype)  # noqa: E731
        scales = lambda: torch.zeros((pages, Hkv), dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(), codes(), scales(), scales())


class KVBatch:
    """The sequences of one step, shared by every layer's calls.

    table:   int32 [B][n], row-contiguous: the page of each block of T tokens
             (entries that name no page are holes)
    kv_len:  int32 [B], the tokens of each sequence, this step's included
    q_start: int32 [B + 1], where each sequence's rows begin in Q, K and V;
             None: one row each
    max_q, max_len: bounds of a sequence's rows and tokens that the host knows
             (max_len 0: the room of the table; the work is planned by it, so that
             a tight one is faster)

    The tensors are kept and read on the device at each call: a program advances
    kv_len, and fills in table entries, in place."""

    def __init__(self, table: torch.Tensor, kv_len: torch.Tensor, q_start: Optional[torch.Tensor] = None,
                 max_q: int = 1, max_len: int = 0):
        if table.dim() != 2 or kv_len.shape != table.shape[:1]:
            raise ValueError("table must be int32 [B][n] and kv_len int32 [B]")
        if q_start is not None and q_start.shape != (table.shape[0] + 1,):
            raise ValueError("q_start must be int32 [B + 1]")
        if max_q < 1 or max_len < 0:
            raise ValueError("max_q must be at least 1 and max_len at least 0")
        self.table, self.kv_len, self.q_start = table, kv_len, q_start
        self.B, self.max_q, self.max_len = table.shape[0], max_q, max_len
        self.device = table.device
        self._c = KVBBatchStruct(_dev(table, torch.int32, "table"), _dev(kv_len, torch.int32, "kv_len"),
                           None if q_start is None else _dev(q_start, torch.int32, "q_start"), table.shape[0],
                           table.shape[1], max_q, max_len, table.shape[0])
        self._ref = ctypes.byref(self._c)

    def _rows(self, rows: int):
        if self.q_start is None and rows != self.B:
            raise ValueError("without q_start there is one row per sequence")
        if rows == self._c.rows:
            return self._ref
        c = KVBBatchStruct.from_buffer_copy(self._c)  # the call's own: another thread may call with other rows
        c.rows = rows
        return ctypes.byref(c)


def _kvb_rows(t: torch.Tensor, heads, D: int, name: str):
    """Device pointer, token stride, dtype code and shape of [rows][heads][D] whose heads lie together."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [rows][heads][{D}]")
    dtype = _KVB_DTYPES.get(t.dtype)
    if dtype is None:
        raise ValueError(f"{name} must be fp16 or bf16")
    if stride[2] != 1 or (stride[1] != D and shape[1] > 1):
        raise ValueError(f"{name}'s heads must be contiguous (its rows may have a stride)")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * D, dtype, shape


def _kvb_weights(t: Optional[torch.Tensor], B: int, Hkv: int, name: str):
    if t is None:
        return None, 0
    shape = t.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != Hkv:
        raise ValueError(f"{name} must be fp32 [B][Hkv][tokens]")
    return _dev(t, torch.float32, name), shape[2]


def _kvb_stream(cache, stream):
    """Handle of the call's stream."""
    return torch._C._cuda_getCurrentRawStream(cache.index) if stream is None else stream.cuda_stream


def kvb_append(cache: KVBlocks, batch: KVBatch, K: torch.Tensor, V: torch.Tensor, w: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise the step's keys and values, fp16 or bf16 [rows][Hkv][D] (rows may
    be strided), into the pages of the last tokens of each sequence
    (tm_kvb_append).  w: token weights fp32 [B][Hkv][tokens], set to 0 for the
    new tokens."""
    Hkv, D = cache.Hkv, cache.D
    kp, ks, dtype, shape = _kvb_rows(K, Hkv, D, "K")
    vp, vs, vdtype, vshape = _kvb_rows(V, Hkv, D, "V")
    if vshape != shape or vdtype != dtype:
        raise ValueError("V must have the shape and dtype of K")
    wp, wn = _kvb_weights(w, batch.B, Hkv, "w")
    st = (_lib or load()).tm_kvb_append(cache._ref, batch._rows(shape[0]), kp, ks, vp, vs, dtype, wp, wn,
                                        _kvb_stream(cache, stream))
    if st:
        raise TMError(st, "tm_kvb_append")


def kvb_attention_workspace(cache: KVBlocks, batch: KVBatch, Hq: int, rows: int, weights: bool = False) -> int:
    """Bytes of workspace that kvb_attention needs (tm_kvb_attention_workspace)."""
    n = ctypes.c_size_t()
    _check(load().tm_kvb_attention_workspace(cache._ref, batch._rows(rows), Hq, 1 if weights else 0, ctypes.byref(n)),
           "tm_kvb_attention_workspace")
    return n.value


def kvb_attention_tree_workspace(cache: KVBlocks, batch: KVBatch, Hq: int, rows: int, weights: bool = False) -> int:
    """Bytes of workspace for kvb_attention_tree (tm_kvb_attention_tree_workspace)."""
    n = ctypes.c_size_t()
    _check(load().tm_kvb_attention_tree_workspace(cache._ref, batch._rows(rows), Hq, 1 if weights else 0, ctypes.byref(n)),
           "tm_kvb_attention_tree_workspace")
    return n.value


def _kvb_attention_args(size_of, cache, batch, Q, out, lse, w_in, w_out, scale, workspace, stream):
    """Arguments that kvb_attention and kvb_attention_tree share, before and after the tree's, out, and the workspace
    (of size_of bytes where none is given; the caller holds it until its launches are made)."""
    if scale and ctypes.c_float(scale).value == 0.0:
        raise ValueError("scale rounds to 0 in fp32, which stands for 1 / sqrt(D)")
    qp, qs, dtype, shape = _kvb_rows(Q, None, cache.D, "Q")
    rows, Hq = shape[0], shape[1]
    if out is None:
        out = _empty(shape, Q.dtype, Q.device, stream)
    elif out.shape != shape:
        raise ValueError("out must have the shape of Q")
    lp = None
    if lse is not None:
        if lse.shape != shape[:2]:
            raise ValueError("lse must be fp32 [rows][Hq]")
        lp = _dev(lse, torch.float32, "lse")
    wi, ni = _kvb_weights(w_in, batch.B, cache.Hkv, "w_in")
    wo, no = _kvb_weights(w_out, batch.B, cache.Hkv, "w_out")
    if wi is not None and (wo is None or ni != no):
        raise ValueError("w_in comes with a w_out of its shape")
    if workspace is None:
        size = size_of(cache, batch, Hq, rows, wo is not None)
        if size:
            workspace = _empty(size, torch.uint8, Q.device, stream)
    sp, size = (None, 0) if workspace is None else (_dev(workspace, torch.uint8, "workspace"), workspace.numel())
    return ((cache._ref, batch._rows(rows), qp, qs, Hq, dtype, 0.0 if scale is None else scale),
            (_dev(out, Q.dtype, "out"), lp, wi, wo, no, sp, size, _kvb_stream(cache, stream)), out, workspace)


def kvb_attention(cache: KVBlocks, batch: KVBatch, Q: torch.Tensor, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, w_in: Optional[torch.Tensor] = None,
                  w_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention of the step's queries, fp16 or bf16 [rows][Hq][D] (rows may
    be strided), over the cache (tm_kvb_attention); append the step's keys and
    values first.  Returns out [rows][Hq][D].

    scale: of the scores, finite; None or 0: 1 / sqrt(D)
    lse:   fp32 [rows][Hq], receives the logarithm of each row's softmax sum
    w_out: fp32 [B][Hkv][tokens], receives w_in (None: 0) plus the weight that each
           token drew in this call; may be w_in
    workspace: a uint8 tensor of kvb_attention_workspace bytes; None: allocated"""
    head, tail, out, held = _kvb_attention_args(kvb_attention_workspace, cache, batch, Q, out, lse, w_in, w_out, scale,
                                                workspace, stream)
    st = (_lib or load()).tm_kvb_attention(*head, *tail)
    if st:
        raise TMError(st, "tm_kvb_attention")
    return out


def kvb_attention_tree(cache: KVBlocks, batch: KVBatch, Q: torch.Tensor, tree: torch.Tensor,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       w_in: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of a tree of drafted tokens (tm_kvb_attention_tree): each row sees the tokens before its
    sequence's new ones, and of the new ones those that its mask names.

    tree: int32 [rows][>= ceil(max_q / 32)], rows may be strided: bit k % 32 of word k / 32 stands for the
          sequence's new token k (``tree_masks`` builds them from parents)

    workspace: a uint8 tensor of kvb_attention_tree_workspace bytes (with fewer it takes fewer slices;
          kvb_attention_workspace's are always enough); None: allocated

    The rest as in kvb_attention."""
    if (tree.dim() != 2 or tree.shape[0] != Q.shape[0] or tree.dtype is not torch.int32 or not tree.is_cuda
            or 32 * tree.shape[1] < batch.max_q or (tree.stride(1) != 1 and tree.shape[1] > 1)):
        raise ValueError("tree must be CUDA int32 [rows][ceil(max_q / 32)], its words contiguous")
    head, tail, out, held = _kvb_attention_args(kvb_attention_tree_workspace, cache, batch, Q, out, lse, w_in, w_out, scale,
                                                workspace, stream)
    stride = tree.stride(0) if tree.shape[0] > 1 else tree.shape[1]
    st = (_lib or load()).tm_kvb_attention_tree(*head, tree.data_ptr(), stride, *tail)
    if st:
        raise TMError(st, "tm_kvb_attention_tree")
    return out


def tree_masks(parents) -> torch.Tensor:
    """Masks for kvb_attention_tree from each sequence's parents: a list per sequence with every node's parent, an
    earlier node of it, or -1.  Returns int32 [rows][words] on the host, the sequences' nodes one after another."""
    words = max([(len(p) + 31) // 32 for p in parents] + [1])
    rows = []
    for p in parents:
        sees = []
        for i, up in enumerate(p):
            if not -1 <= up < i:
                raise ValueError("a node's parent is an earlier node, or -1")
            sees.append((sees[up] if up >= 0 else 0) | 1 << i)
        rows += [[(m >> 32 * k) & 0xffffffff for k in range(words)] for m in sees]
    t = torch.tensor(rows, dtype=torch.int64).reshape(len(rows), words)
    return torch.where(t >= 2 ** 31, t - 2 ** 32, t).to(torch.int32)


class Rope:
    """Rotation by position (tm_kvb_rope): table fp32 [positions][dims] with a position's dims / 2
    cosines, then its sines; pairs (i, i + dims / 2), or neighbours where interleaved."""

    def __init__(self, table: torch.Tensor, interleaved: bool = False):
        if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] % 16 or table.shape[1] < 16:
            raise ValueError("table must be fp32 [positions][dims], dims a multiple of 16")
        self.table, self.interleaved = table, bool(interleaved)
        self.positions, self.dims = table.shape
        self._p = _dev(table, torch.float32, "table")
        self._c = KVBRopeStruct(self._p, self.positions, self.dims, self.interleaved, None)  # positions: the slots
        self._ref = ctypes.byref(self._c)


def kvb_append_rope(cache: KVBlocks, batch: KVBatch, K: torch.Tensor, V: torch.Tensor, rope: Rope,
                    Q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    pos: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """kvb_append with the keys rotated by their positions, and the queries beside them (tm_kvb_append_rope).

    Q:     fp16 or bf16 [rows][Hq][D] (rows may be strided); None: keys and values alone
    q_out: receives the rotated queries, like Q; may be Q (None: allocated).  Returned
    pos:   int32 [rows], each row's position; None: its slot in the cache"""
    Hkv, D = cache.Hkv, cache.D
    kp, ks, dtype, shape = _kvb_rows(K, Hkv, D, "K")
    vp, vs, vdtype, vshape = _kvb_rows(V, Hkv, D, "V")
    if vshape != shape or vdtype != dtype:
        raise ValueError("V must have the shape and dtype of K")
    rows = shape[0]
    qp, qs, Hq, op, os_ = None, 0, 0, None, 0
    if Q is not None:
        qp, qs, qdtype, qshape = _kvb_rows(Q, None, D, "Q")
        if qshape[0] != rows or qdtype != dtype:
            raise ValueError("Q must have the rows and dtype of K")
        Hq = qshape[1]
        if q_out is None:
            q_out = _empty(qshape, Q.dtype, Q.device, stream)
        op, os_, odtype, oshape = _kvb_rows(q_out, Hq, D, "q_out")
        if oshape != qshape or odtype != dtype:
            raise ValueError("q_out must have the shape and dtype of Q")
    elif q_out is not None:
        raise ValueError("q_out comes with Q")
    ref = rope._ref
    if pos is not None:
        if pos.shape != (rows,):
            raise ValueError("pos must be int32 [rows]")
        ref = ctypes.byref(KVBRopeStruct(rope._p, rope.positions, rope.dims, rope.interleaved,
                                         _dev(pos, torch.int32, "pos")))
    wp, wn = _kvb_weights(w, batch.B, Hkv, "w")
    st = (_lib or load()).tm_kvb_append_rope(cache._ref, batch._rows(rows), kp, ks, vp, vs, qp, qs, Hq, op, os_,
                                             ref, dtype, wp, wn, _kvb_stream(cache, stream))
    if st:
        raise TMError(st, "tm_kvb_append_rope")
    return q_out


def kvb_accept(cache: KVBlocks, batch: KVBatch, path: torch.Tensor, count: torch.Tensor,
               w: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Keep a path through the new tokens of each sequence (tm_kvb_accept): path int32 [B][n], ascending indices of
    the sequence's new tokens, of which the first count[b] (int32 [B]) hold.  w: token weights fp32
    [B][Hkv][tokens], moved along.  Returns new_len int32 [B]; batch.kv_len is left as it is."""
    B = batch.B
    if path.dim() != 2 or path.shape[0] != B or count.shape != (B,):
        raise ValueError("path must be int32 [B][n] and count int32 [B]")
    if new_len is None:
        new_len = _empty(B, torch.int32, path.device, stream)
    elif new_len.shape != (B,):
        raise ValueError("new_len must be int32 [B]")
    wp, wn = _kvb_weights(w, B, cache.Hkv, "w")
    st = (_lib or load()).tm_kvb_accept(cache._ref, batch._ref, _dev(path, torch.int32, "path"), path.shape[1],
                                        _dev(count, torch.int32, "count"), wp, wn, _dev(new_len, torch.int32, "new_len"),
                                        _kvb_stream(cache, stream))
    if st:
        raise TMError(st, "tm_kvb_accept")
    return new_len


def kvb_evict(cache: KVBlocks, batch: KVBatch, w: torch.Tensor, budget: int, first: int = 0, recent: int = 0,
              dst_table: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None,
              kept: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
    """Cut every sequence to ``budget`` tokens per KV head (tm_kvb_evict): the first
    ``first``, the last ``recent`` and the heaviest of the rest by w, fp32
    [B][Hkv][tokens].  dst_table int32 [B][n]: the pages that take them (None: in
    place: no page may then belong to two sequences of the batch; move sequences that
    share pages into fresh ones).  w_out: their weights, fp32 [B][Hkv][>= budget] (None: into w).
    Returns (kept int32 [B][Hkv][budget], new_len int32 [B]); batch.kv_len is
    left as it is."""
    wp, wn = _kvb_weights(w, batch.B, cache.Hkv, "w")
    op, on = (wp, wn) if w_out is None else _kvb_weights(w_out, batch.B, cache.Hkv, "w_out")
    if kept is None:
        kept = _empty((batch.B, cache.Hkv, max(budget, 0)), torch.int32, w.device, stream)
    elif kept.shape != (batch.B, cache.Hkv, budget):
        raise ValueError("kept must be int32 [B][Hkv][budget]")
    if new_len is None:
        new_len = _empty(batch.B, torch.int32, w.device, stream)
    elif new_len.shape != (batch.B,):
        raise ValueError("new_len must be int32 [B]")
    dst = batch.table if dst_table is None else dst_table
    if dst.dim() != 2 or dst.shape[0] != batch.B:
        raise ValueError("dst_table must be int32 [B][n]")
    st = load().tm_kvb_evict(cache._ref, batch._ref, _dev(dst, torch.int32, "dst_table"), dst.shape[1], wp, wn, op, on,
                             budget, first, recent, _dev(kept, torch.int32, "kept"),
                             _dev(new_len, torch.int32, "new_len"), _kvb_stream(cache, stream))
    _check(st, "tm_kvb_evict")
    return kept, new_len


# ---- low-rank adapters beside a shared projection (include/tm_lora.h) ----

class Adapters:
    """The low-rank adapters of one projection: A fp16 [n][R][K], B fp16 [n][N][R], contiguous on one device; scale
    fp32 [n] (None: 1).  R is a multiple of 8, 8 .. 128: pad lower ranks with zeros."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: Optional[torch.Tensor] = None):
        if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2]:
            raise ValueError("A must be fp16 [n][R][K] and B fp16 [n][N][R]")
        if scale is not None and scale.shape != A.shape[:1]:
            raise ValueError("scale must be fp32 [n]")
        n, R, K = A.shape
        N = B.shape[1]
        if R % 8 or not 8 <= R <= 128 or K % 8 or N % 8 or K < 8 or N < 8:
            raise ValueError("R must be a multiple of 8 up to 128, K and N multiples of 8")
        if A.device != B.device or (scale is not None and scale.device != A.device):
            raise ValueError("A, B and scale must be on one device")
        self.A, self.B, self.scale = A, B, scale
        self.n, self.R, self.K, self.N, self.device, self.index = n, R, K, N, A.device, A.device.index
        self._c = LoraAdaptersStruct(_dev(A, torch.float16, "A"), _dev(B, torch.float16, "B"),
                                     None if scale is None else _dev(scale, torch.float32, "scale"), n, K, N, R)
        self._ref = ctypes.byref(self._c)


def _lora_rows(t: torch.Tensor, cols: int, name: str):
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != cols or t.dtype is not torch.float16 or not t.is_cuda or stride[1] != 1:
        raise ValueError(f"{name} must be a CUDA fp16 tensor [rows][{cols}] (its rows may have a stride)")
    return t.data_ptr(), stride[0] if shape[0] > 1 else cols


def lora_add(Y: torch.Tensor, X: torch.Tensor, adapters: Adapters, ids: torch.Tensor,
             q_start: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out = Y + scale[a] (X . A[a]^T) . B[a]^T with a the adapter of each row's sequence (tm_lora_add): Y fp16
    [rows][N], a projection's output, X fp16 [rows][K], its input (rows may be strided).

    ids:     int32 [B], each sequence's adapter; outside 0 .. n-1: none
    q_start: int32 [B + 1], where each sequence's rows begin; None: one row each
    out:     fp16 [rows][N]; None: Y itself.  Rows of no sequence are left as they are"""
    yp, ys = _lora_rows(Y, adapters.N, "Y")
    xp, xs = _lora_rows(X, adapters.K, "X")
    rows = X.shape[0]
    if Y.shape[0] != rows:
        raise ValueError("Y must have the rows of X")
    op, os_ = yp, ys
    if out is None:
        out = Y
    else:
        op, os_ = _lora_rows(out, adapters.N, "out")
        if out.shape[0] != rows:
            raise ValueError("out must have the rows of X")
    B = ids.shape[0] if ids.dim() == 1 else -1
    if B < 0 or (q_start is None and B != rows) or (q_start is not None and q_start.shape != (B + 1,)):
        raise ValueError("ids must be int32 [B], q_start int32 [B + 1] (None: one row each)")
    st = (_lib or load()).tm_lora_add(adapters._ref, xp, xs, yp, ys, op, os_, rows, _dev(ids, torch.int32, "ids"),
                                      None if q_start is None else _dev(q_start, torch.int32, "q_start"), B,
                                      _kvb_stream(adapters, stream))
    if st:
        raise TMError(st, "tm_lora_add")
    return out
