"""Thin ctypes binding of the C ABI in include/petit.h.

Argument marshalling only: every computation runs in the CUDA library.  The
functions take torch tensors for device memory and use torch's current CUDA
stream.  If the library cannot be built or loaded, :func:`load` raises --
there is no CPU fallback.
"""

import contextlib
import ctypes
import functools
import os
import threading

import torch

from . import build as _build

PETIT_FMT_NVFP4 = 0
PETIT_FMT_MXFP4 = 1
PETIT_FMT_NVFP4_F16 = 2
FORMATS = {"nvfp4": PETIT_FMT_NVFP4, "mxfp4": PETIT_FMT_MXFP4, "nvfp4_f16": PETIT_FMT_NVFP4_F16}

STATUS = {
    0: "PETIT_OK",
    1: "PETIT_ERR_INVALID_ARG",
    2: "PETIT_ERR_UNSUPPORTED_SHAPE",
    3: "PETIT_ERR_MISALIGNED",
    4: "PETIT_ERR_WORKSPACE",
    5: "PETIT_ERR_ARCH",
    6: "PETIT_ERR_CUDA",
    7: "PETIT_ERR_TIMEOUT",
    8: "PETIT_ERR_BOUNDS",
}

_lib = None
_lock = threading.Lock()

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_sz = ctypes.c_size_t


class PlanInfo(ctypes.Structure):
    """petit_plan_info_t"""
    _fields_ = [("bn", ctypes.c_int32), ("ku", ctypes.c_int32), ("cta_pairs", ctypes.c_int32),
                ("num_ranges", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
                ("units_per_tile", ctypes.c_int32), ("num_tiles", ctypes.c_int64),
                ("units", ctypes.c_int64), ("workspace_bytes", ctypes.c_uint64)]


class KvCacheInfo(ctypes.Structure):
    """petit_kv_cache_t"""
    _fields_ = [("data", _c_p), ("scales", _c_p), ("num_pages", _c_i64), ("page_stride", _c_i64),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class Rows(ctypes.Structure):
    """petit_rows_t"""
    _fields_ = [("data", _c_p), ("token_stride", _c_i64), ("head_stride", _c_i64)]


class KvAttentionArgs(ctypes.Structure):
    """petit_kv_attention_t"""
    _fields_ = [("q", Rows), ("out", Rows), ("lse", _c_p), ("block_table", _c_p), ("seq_lens", _c_p),
                ("q_offsets", _c_p), ("batch", _c_i64), ("total_q", _c_i64), ("max_q", _c_i64),
                ("max_pages", _c_i64), ("table_stride", _c_i64), ("num_q_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", _c_i64)]


# name -> (restype, argtypes)
SIGNATURES = {
    "petit_layout_version": (ctypes.c_int, []),
    "petit_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "petit_repacked_bytes": (_c_sz, [_c_i64, _c_i64, ctypes.c_int]),
    "petit_gemm_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, ctypes.c_int]),
    "petit_absmax_bf16": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p]),
    "petit_nvfp4_global_scale": (ctypes.c_float, [ctypes.c_float]),
    "petit_quantize_nvfp4": (ctypes.c_int, [_c_p, ctypes.c_float, _c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_quantize_mxfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_repack_nvfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_repack_mxfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_repack_nvfp4_f16": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_dequant_f16": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_gemm_f16_nvfp4": (ctypes.c_int, [_c_p, _c_p, ctypes.c_float, _c_p, _c_i64, _c_i64, _c_i64,
                                            _c_p, _c_sz, _c_p]),
    "petit_dequant_bf16": (ctypes.c_int, [_c_p, ctypes.c_int, _c_p, _c_i64, _c_i64, _c_p]),
    "petit_gemm_bf16_nvfp4": (ctypes.c_int, [_c_p, _c_p, ctypes.c_float, _c_p, _c_i64, _c_i64, _c_i64,
                                             _c_p, _c_sz, _c_p]),
    "petit_gemm_bf16_mxfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_sz,
                                             _c_p]),
    "petit_gemm_bf16_nvfp4_dscale": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                                                    _c_p, _c_sz, _c_p]),
    "petit_gemm_bf16_nvfp4_noalloc": (ctypes.c_int, [_c_p, _c_p, ctypes.c_float, _c_p, _c_i64, _c_i64, _c_i64,
                                                     _c_p]),
    "petit_moe_workspace_bytes": (_c_sz, [_c_p, _c_i64, _c_i64, _c_i64, ctypes.c_int]),
    "petit_moe_gemm_bf16_mxfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_i64, _c_p,
                                                 _c_sz, _c_p]),
    "petit_moe_gemm_bf16_nvfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_i64,
                                                 _c_p, _c_sz, _c_p]),
    "petit_get_device_status": (ctypes.c_int, [_c_p, _c_sz, _c_p]),
    "petit_set_tile_config": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "petit_set_pair_mode": (ctypes.c_int, [ctypes.c_int]),
    "petit_bounds_checking": (ctypes.c_int, []),
    "petit_check_set_limits": (ctypes.c_int, [_c_i64, _c_i64]),
    "petit_selftest_timeout": (ctypes.c_int, [_c_p, _c_sz, ctypes.c_uint32, _c_p]),
    "petit_plan_gemm": (ctypes.c_int, [_c_i64, _c_i64, _c_i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(PlanInfo), _c_p, _c_i64]),
    "petit_plan_moe": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.POINTER(PlanInfo), _c_p, _c_i64]),
    "petit_kv_page_bytes": (_c_sz, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int]),
    "petit_kv_append": (ctypes.c_int, [_c_p, _c_p, _c_p, ctypes.c_int, _c_p, _c_i64, _c_p, _c_sz, _c_p]),
    "petit_kv_read": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p, ctypes.c_int, _c_p, _c_sz, _c_p]),
    "petit_kv_attention_workspace_bytes": (_c_sz, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int]),
    "petit_kv_attention": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_sz, _c_p]),
    "petit_device_limits": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
}


class PetitError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def _open(path):
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(build=True):
    """Build (if stale) and load the CUDA library; raises on failure."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            _lib = _open(_build.build() if build else _build.LIB)
    return _lib


_check_lib = None


def load_check(build=True):
    """Build (if stale) and load the bounds-checking build of the library
    (``_petit_check.so``: same API; the GEMM kernel checks every buffer
    index and copy and reports a failed check as PETIT_ERR_BOUNDS)."""
    global _check_lib
    with _lock:
        if _check_lib is None:
            _check_lib = _open(_build.build_check() if build else _build.CHECK_LIB)
    return _check_lib


@contextlib.contextmanager
def bounds_checked():
    """Inside the block every call of this module goes through the
    bounds-checking build (process-wide; not for concurrent use)."""
    global _lib
    chk = load_check()
    prev = load()
    _lib = chk
    try:
        yield chk
    finally:
        _lib = prev


def lib_path():
    return _build.LIB


def _check(status, where):
    if status != 0:
        raise PetitError(status, where)


# The raw handle of torch's current stream without building a Stream object
# (a per-call cost on the GEMM path); the public call where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return t.data_ptr()


def _need(t, dtype, name):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor")


# ---------------------------------------------------------------------- API
def layout_version():
    return load().petit_layout_version()


def absmax(x):
    """max |x| of a BF16 CUDA tensor, as a 1-element FP32 CUDA tensor."""
    _need(x, torch.bfloat16, "x")
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(load().petit_absmax_bf16(_ptr(x), x.numel(), _ptr(out), _stream()), "absmax")
    return out


def nvfp4_global_scale(amax):
    return float(load().petit_nvfp4_global_scale(ctypes.c_float(float(amax))))


def quantize(W, fmt="nvfp4", global_scale=1.0):
    """BF16 [n, k] -> (packed codes uint8 [n, k/2], scales uint8 [n, k/G])."""
    _need(W, torch.bfloat16, "W")
    n, k = W.shape
    group = 16 if fmt == "nvfp4" else 32
    wp = torch.empty((n, k // 2), dtype=torch.uint8, device=W.device)
    sp = torch.empty((n, max(k // group, 1)), dtype=torch.uint8, device=W.device)
    L = load()
    if fmt == "nvfp4":
        st = L.petit_quantize_nvfp4(_ptr(W), ctypes.c_float(global_scale), _ptr(wp), _ptr(sp), n, k, _stream())
    else:
        st = L.petit_quantize_mxfp4(_ptr(W), _ptr(wp), _ptr(sp), n, k, _stream())
    _check(st, "quantize_" + fmt)
    return wp, sp


def repack(w_packed, scales, fmt="nvfp4"):
    """Packed codes [n, k/2] + scales -> one repacked uint8 buffer."""
    _need(w_packed, torch.uint8, "w_packed")
    _need(scales, torch.uint8, "scales")
    n, half_k = w_packed.shape
    k = half_k * 2
    L = load()
    out = torch.empty(max(L.petit_repacked_bytes(n, k, FORMATS[fmt]), 1), dtype=torch.uint8,
                      device=w_packed.device)
    fn = {"nvfp4": L.petit_repack_nvfp4, "mxfp4": L.petit_repack_mxfp4,
          "nvfp4_f16": L.petit_repack_nvfp4_f16}[fmt]
    _check(fn(_ptr(w_packed), _ptr(scales), _ptr(out), n, k, _stream()), "repack_" + fmt)
    return out


def dequant(rep, n, k, fmt="nvfp4"):
    """Repacked weights -> Wq [n, k] (test hook; bit-exact): BF16, or FP16 for
    the "nvfp4_f16" layout."""
    if fmt == "nvfp4_f16":
        out = torch.empty((n, k), dtype=torch.float16, device=rep.device)
        _check(load().petit_dequant_f16(_ptr(rep), _ptr(out), n, k, _stream()), "dequant_f16")
        return out
    out = torch.empty((n, k), dtype=torch.bfloat16, device=rep.device)
    _check(load().petit_dequant_bf16(_ptr(rep), FORMATS[fmt], _ptr(out), n, k, _stream()), "dequant")
    return out


@functools.lru_cache(maxsize=1024)
def workspace_bytes(m, n, k, fmt="nvfp4"):
    return int(load().petit_gemm_workspace_bytes(m, n, k, FORMATS[fmt]))


class Workspace:
    """A zero-filled device workspace that grows on demand.  What it has
    outgrown is kept: calls that are queued or captured in a graph still use it
    and record their errors there."""

    def __init__(self, device=None, nbytes=0):
        self.device = torch.device(device or "cuda")
        self.buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=self.device)
        self._outgrown = []

    def ensure(self, nbytes):
        if nbytes > self.buf.numel():
            self._outgrown.append(self.buf)
            self.buf = torch.zeros(int(nbytes), dtype=torch.uint8, device=self.device)
        return self.buf

    def status(self):
        """PETIT_OK (0) or the error the kernels recorded (clears it)."""
        found = [load().petit_get_device_status(_ptr(b), b.numel(), _stream()) for b in (*self._outgrown, self.buf)]
        return next((s for s in found if s), 0)


def gemm(A, rep, n, fmt="nvfp4", global_scale=1.0, workspace=None, out=None):
    """C[m, n] = g * A @ dequant(W)^T in BF16 (FP32 accumulation).  For NVFP4,
    `global_scale` is a float or a one-element FP32 CUDA tensor (read by the
    kernel, so a CUDA graph picks up a changed value on replay).  With the
    "nvfp4_f16" layout, A and C are FP16."""
    act = torch.float16 if fmt == "nvfp4_f16" else torch.bfloat16
    _need(A, act, "A")
    m, k = A.shape
    ws = workspace or Workspace(A.device)
    need = workspace_bytes(m, n, k, fmt)
    if need == 0:
        raise PetitError(2, "gemm workspace size")
    buf = ws.ensure(need)
    C = out if out is not None else torch.empty((m, n), dtype=act, device=A.device)
    L = load()
    if fmt == "nvfp4_f16":
        st = L.petit_gemm_f16_nvfp4(_ptr(A), _ptr(rep), ctypes.c_float(global_scale), _ptr(C),
                                    m, n, k, _ptr(buf), buf.numel(), _stream())
    elif fmt == "nvfp4" and isinstance(global_scale, torch.Tensor):
        _need(global_scale, torch.float32, "global_scale")
        st = L.petit_gemm_bf16_nvfp4_dscale(_ptr(A), _ptr(rep), _ptr(global_scale), _ptr(C),
                                            m, n, k, _ptr(buf), buf.numel(), _stream())
    elif fmt == "nvfp4":
        st = L.petit_gemm_bf16_nvfp4(_ptr(A), _ptr(rep), ctypes.c_float(global_scale), _ptr(C),
                                     m, n, k, _ptr(buf), buf.numel(), _stream())
    else:
        st = L.petit_gemm_bf16_mxfp4(_ptr(A), _ptr(rep), _ptr(C), m, n, k, _ptr(buf), buf.numel(),
                                     _stream())
    _check(st, "gemm_" + fmt)
    return C


def moe_gemm(A, rep, expert_offsets, n, fmt="mxfp4", global_scales=None, workspace=None, out=None):
    """Grouped GEMM of an MoE layer: rows [off[e], off[e+1]) of A (BF16,
    grouped by expert) times expert e's weights; `rep` holds the experts'
    repacked weights back to back; `expert_offsets` is a host sequence of
    E + 1 ints; `global_scales` (NVFP4) a host sequence of E floats."""
    _need(A, torch.bfloat16, "A")
    T, k = A.shape
    off = (ctypes.c_int64 * len(expert_offsets))(*[int(x) for x in expert_offsets])
    E = len(expert_offsets) - 1
    if int(off[E]) != T:
        raise ValueError("expert_offsets[-1] must equal A.shape[0]")
    L = load()
    ws = workspace or Workspace(A.device)
    need = int(L.petit_moe_workspace_bytes(off, E, n, k, FORMATS[fmt]))
    if need == 0 and T > 0:
        raise PetitError(2, "moe workspace size")
    buf = ws.ensure(max(need, 256))
    C = out if out is not None else torch.empty((T, n), dtype=torch.bfloat16, device=A.device)
    if fmt == "mxfp4":
        st = L.petit_moe_gemm_bf16_mxfp4(_ptr(A), _ptr(rep), off, E, _ptr(C), n, k, _ptr(buf),
                                         buf.numel(), _stream())
    else:
        gs = (ctypes.c_float * E)(*[float(x) for x in (global_scales or [1.0] * E)])
        st = L.petit_moe_gemm_bf16_nvfp4(_ptr(A), _ptr(rep), gs, off, E, _ptr(C), n, k, _ptr(buf),
                                         buf.numel(), _stream())
    _check(st, "moe_gemm_" + fmt)
    return C


def set_tile_config(bn=0, ku=0):
    """Force the GEMM tile shape (bn activation rows, ku 128-k chunks per
    unit) for later calls in this process; (0, 0) restores the planner."""
    _check(load().petit_set_tile_config(int(bn), int(ku)), "set_tile_config")
    workspace_bytes.cache_clear()


def set_pair_mode(mode=0):
    """CTA pairs (cta_group::2) for 128/256-row tiles in later calls of this
    process: 0 where the planner expects a gain, 1 never, 2 wherever they
    apply."""
    _check(load().petit_set_pair_mode(int(mode)), "set_pair_mode")
    workspace_bytes.cache_clear()


_MAX_RANGES = 1025   # kernel grids have at most 1024 work ranges


def _limits(num_sms, pair_capacity):
    """The given SM count and pair capacity, the current device's for any left out."""
    if num_sms is None or pair_capacity is None:
        dev_sms, dev_pc = device_limits()
        num_sms = dev_sms if num_sms is None else num_sms
        pair_capacity = dev_pc if pair_capacity is None else pair_capacity
    return int(num_sms), int(pair_capacity)


def _plan_result(info, starts):
    d = {f: getattr(info, f) for f, _ in PlanInfo._fields_}
    d["cta_pairs"] = bool(d["cta_pairs"])
    d["range_starts"] = list(starts[:info.num_ranges + 1]) if info.num_ranges else []
    return d


def plan(m, n, k, fmt="nvfp4", num_sms=None, pair_capacity=None):
    """The plan of a GEMM (tile shape, CTA pairs, work units and ranges,
    workspace bytes) on a device with num_sms SMs and pair_capacity resident
    CTA pairs; by default the current device's (petit_device_limits).  With
    both given, no GPU is needed."""
    L = load()
    num_sms, pair_capacity = _limits(num_sms, pair_capacity)
    info = PlanInfo()
    starts = (ctypes.c_int64 * _MAX_RANGES)()
    _check(L.petit_plan_gemm(int(m), int(n), int(k), FORMATS[fmt], num_sms, pair_capacity,
                             ctypes.byref(info), starts, _MAX_RANGES), "plan_gemm")
    return _plan_result(info, starts)


def moe_plan(expert_offsets, n, k, fmt="mxfp4", num_sms=None, pair_capacity=None):
    """:func:`plan` for the grouped MoE GEMM (expert_offsets: E + 1 row offsets)."""
    L = load()
    num_sms, pair_capacity = _limits(num_sms, pair_capacity)
    E = len(expert_offsets) - 1
    off = (ctypes.c_int64 * (E + 1))(*[int(x) for x in expert_offsets])
    info = PlanInfo()
    starts = (ctypes.c_int64 * _MAX_RANGES)()
    _check(L.petit_plan_moe(off, E, int(n), int(k), FORMATS[fmt], num_sms, pair_capacity,
                            ctypes.byref(info), starts, _MAX_RANGES), "plan_moe")
    return _plan_result(info, starts)


def device_limits():
    """(SM count, resident CTA pairs) of the current device, as the GEMMs plan with."""
    sms, pc = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().petit_device_limits(ctypes.byref(sms), ctypes.byref(pc)), "device_limits")
    return sms.value, pc.value


def selftest_timeout(workspace, timeout_us=1000):
    _check(load().petit_selftest_timeout(_ptr(workspace.buf), workspace.buf.numel(), timeout_us, _stream()),
           "selftest_timeout")


# ------------------------------------------------------------ 4-bit K/V cache
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class KVCache:
    """A paged cache of attention keys and values in 4 bits (petit.h gives its
    memory order): `num_pages` pages of `page_size` tokens of `num_kv_heads`
    heads.  NVFP4 scales are relative to an FP32 scale per head, for K and for
    V: `scales`, an FP32 CUDA tensor [2, num_kv_heads] (by default ones).
    `data` takes over existing memory, uint8 [num_pages, >= page bytes] with
    contiguous rows; by default it is allocated and zero-filled."""

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, fmt="nvfp4", scales=None, data=None,
                 device=None):
        if fmt not in ("nvfp4", "mxfp4"):
            raise ValueError("fmt: need 'nvfp4' or 'mxfp4'")
        page = load().petit_kv_page_bytes(page_size, num_kv_heads, head_dim, FORMATS[fmt])
        if page == 0 or num_pages < 1:
            raise PetitError(2, "kv cache geometry")
        if data is None:
            data = torch.zeros((num_pages, page), dtype=torch.uint8, device=torch.device(device or "cuda"))
        elif (not data.is_cuda or data.dtype != torch.uint8 or data.dim() != 2 or data.shape[0] != num_pages
              or data.shape[1] < page or data.stride(1) != 1 or (num_pages > 1 and data.stride(0) < page)):
            raise ValueError(f"data: need a CUDA uint8 tensor [{num_pages}, >= {page}] with contiguous rows")
        if scales is not None:
            if fmt == "mxfp4":
                raise ValueError("scales: MXFP4 has none")
            _need(scales, torch.float32, "scales")
            if tuple(scales.shape) != (2, num_kv_heads):
                raise ValueError(f"scales: need shape (2, {num_kv_heads})")
            if scales.device != data.device:
                raise ValueError("scales: need the cache's device")
        self.data, self.scales, self.fmt = data, scales, fmt
        self.device, self.device_index = data.device, data.get_device()
        self.num_pages, self.page_size = num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.page_bytes = page
        self.info = KvCacheInfo(_ptr(data), _ptr(scales) if scales is not None else None, num_pages,
                                data.stride(0) if num_pages > 1 else page, page_size, num_kv_heads, head_dim,
                                FORMATS[fmt])
        self._ref = ctypes.addressof(self.info)
        self._workspace_bytes = 0

    def workspace_bytes(self):
        """Bytes of workspace :meth:`attention` needs on the current device."""
        if not self._workspace_bytes:
            self._workspace_bytes = int(load().petit_kv_attention_workspace_bytes(
                self.num_kv_heads, self.head_dim, FORMATS[self.fmt]))
        return self._workspace_bytes

    def append(self, k, v, slots, workspace=None):
        return kv_append(self, k, v, slots, workspace)

    def read(self, slots, dtype=torch.bfloat16, workspace=None, out=None):
        return kv_read(self, slots, dtype, workspace, out)

    def attention(self, q, block_table, seq_lens, q_offsets=None, max_q=1, **kwargs):
        return kv_attention(self, q, block_table, seq_lens, q_offsets, max_q, **kwargs)


def _rows(t, cache, heads, dtype, name, tokens=None):
    """petit_rows_t of a [tokens, heads, D] tensor whose last dimension is contiguous."""
    if t.dim() == 3 and t.dtype is dtype and t.get_device() == cache.device_index:
        n, h, d = t.shape
        st, sh, sd = t.stride()
        if h == heads and d == cache.head_dim and sd == 1 and (tokens is None or n == tokens):
            return Rows(t.data_ptr(), st, sh)
    raise ValueError(f"{name}: need a {dtype} tensor [{'tokens' if tokens is None else tokens}, {heads}, "
                     f"{cache.head_dim}] on the cache's device, contiguous in its last dimension")


def _new_rows(cache, tokens, heads, dtype):
    """A new tensor [tokens, heads, D] and its petit_rows_t."""
    t = torch.empty((tokens, heads, cache.head_dim), dtype=dtype, device=cache.device)
    return t, Rows(t.data_ptr(), heads * cache.head_dim, cache.head_dim)


def _indices(t, cache, dtype, shape, name):
    if t.dtype is dtype and t.shape == shape and t.get_device() == cache.device_index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: need a contiguous {dtype} tensor {list(shape)} on the cache's device")


def _status_buf(workspace):
    return (None, 0) if workspace is None else (_ptr(workspace.buf), workspace.buf.numel())


def kv_append(cache, k, v, slots, workspace=None):
    """Quantise rows k and v ([tokens, num_kv_heads, head_dim], BF16 or FP16,
    any token and head stride that is a multiple of 8) and write token i to
    slot slots[i] (int64; slot = page * page_size + offset).  Negative slots
    are skipped; a slot past the cache is skipped and, if a `workspace` is
    given, recorded in it (see :meth:`Workspace.status`)."""
    if k.dtype not in _DTYPES:
        raise ValueError("k: need BF16 or FP16")
    n = k.shape[0]
    rk = _rows(k, cache, cache.num_kv_heads, k.dtype, "k")
    rv = _rows(v, cache, cache.num_kv_heads, k.dtype, "v", n)
    buf, nbytes = _status_buf(workspace)
    _check(load().petit_kv_append(cache._ref, ctypes.byref(rk), ctypes.byref(rv), _DTYPES[k.dtype],
                                  _indices(slots, cache, torch.int64, (n,), "slots"), n, buf, nbytes, _stream()),
           "kv_append")


def kv_read(cache, slots, dtype=torch.bfloat16, workspace=None, out=None):
    """The values of the tokens in `slots` as (K, V), each [tokens,
    num_kv_heads, head_dim] in `dtype`; a negative slot (or one past the
    cache, which is recorded in `workspace`) gives zeros."""
    if dtype not in _DTYPES:
        raise ValueError("dtype: need torch.bfloat16 or torch.float16")
    n = slots.numel()
    if out is None:
        k, rk = _new_rows(cache, n, cache.num_kv_heads, dtype)
        v, rv = _new_rows(cache, n, cache.num_kv_heads, dtype)
        out = k, v
    else:
        rk = _rows(out[0], cache, cache.num_kv_heads, dtype, "out[0]", n)
        rv = _rows(out[1], cache, cache.num_kv_heads, dtype, "out[1]", n)
    buf, nbytes = _status_buf(workspace)
    _check(load().petit_kv_read(cache._ref, _indices(slots, cache, torch.int64, (n,), "slots"), n, ctypes.byref(rk),
                                ctypes.byref(rv), _DTYPES[dtype], buf, nbytes, _stream()), "kv_read")
    return out


def kv_attention(cache, q, block_table, seq_lens, q_offsets=None, max_q=1, scale=None, causal=True, window=0,
                 workspace=None, out=None, lse=None):
    """softmax(scale * q k^T + mask) v over the cached sequences.

    q: BF16 or FP16 [total_q, num_q_heads, head_dim], the queries of all
    sequences one after the other; block_table: int32 [batch, max_pages];
    seq_lens: int32 [batch], the cached tokens of each sequence, its queries'
    own among them.  q_offsets: int32 [batch + 1], where each sequence's
    queries begin; None: max_q queries for every sequence.  max_q: the most
    queries of a sequence.  scale: by default head_dim ** -0.5.  causal: the
    last query sees every key, the one before it all but the last, and so on;
    window > 0 keeps the nearest `window` of them (pages whose keys no query
    sees may have been given back: any entry will do).  lse: an FP32 tensor
    [total_q, num_q_heads] that receives the log of the softmax's sum.  A
    query that sees no key gives zeros (and an lse of -inf).  workspace: keep
    one; without it a call makes and zero-fills one of its own (some 40 MB),
    and what it records of lengths and pages out of range is lost with it."""
    if q.dtype not in _DTYPES or q.dim() != 3:
        raise ValueError("q: need a BF16 or FP16 tensor [total_q, num_q_heads, head_dim]")
    total_q, heads = q.shape[0], q.shape[1]
    if heads < 1 or heads % cache.num_kv_heads:
        raise ValueError(f"q: need a multiple of {cache.num_kv_heads} heads")
    if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table: need [batch, max_pages] with contiguous rows")
    batch, max_pages = block_table.shape
    if block_table.dtype is not torch.int32 or block_table.get_device() != cache.device_index:
        raise ValueError("block_table: need int32 on the cache's device")
    # (with one row, or rows without entries, torch's stride says nothing)
    table_stride = block_table.stride(0) if batch > 1 and max_pages > 0 else max(max_pages, 1)
    if table_stride < max_pages:
        raise ValueError("block_table: need rows of their own (an expanded one: make it contiguous)")
    rq = _rows(q, cache, heads, q.dtype, "q")
    if out is None:
        out, ro = _new_rows(cache, total_q, heads, q.dtype)
    else:
        ro = _rows(out, cache, heads, q.dtype, "out", total_q)
    args = KvAttentionArgs(
        rq, ro, None if lse is None else _ptr(lse), _ptr(block_table),
        _indices(seq_lens, cache, torch.int32, (batch,), "seq_lens"),
        None if q_offsets is None else _indices(q_offsets, cache, torch.int32, (batch + 1,), "q_offsets"),
        batch, total_q, int(max_q), max_pages, table_stride, heads, _DTYPES[q.dtype],
        cache.head_dim ** -0.5 if scale is None else float(scale), int(bool(causal)), int(window))
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (total_q, heads)
                            or not lse.is_contiguous() or lse.get_device() != cache.device_index):
        raise ValueError(f"lse: need a contiguous FP32 tensor [{total_q}, {heads}] on the cache's device")
    ws = workspace or Workspace(cache.device)
    buf = ws.ensure(cache.workspace_bytes())
    _check(load().petit_kv_attention(cache._ref, ctypes.byref(args), _ptr(buf), buf.numel(), _stream()),
           "kv_attention")
    return out


class FP4Weight:
    """Offline-prepared FP4 weight: quantised, repacked, ready for gemm()."""

    def __init__(self, W, fmt="nvfp4", global_scale=None):
        n, k = W.shape
        self.n, self.k, self.fmt = n, k, fmt
        if fmt in ("nvfp4", "nvfp4_f16"):
            if global_scale is None:
                global_scale = 1.0
            elif global_scale == "amax":
                global_scale = nvfp4_global_scale(absmax(W).item())
            self.global_scale = float(global_scale)
        else:
            self.global_scale = 1.0
        w_packed, scales = quantize(W, "mxfp4" if fmt == "mxfp4" else "nvfp4", self.global_scale)
        self.rep = repack(w_packed, scales, fmt)

    def __call__(self, A, workspace=None, out=None):
        return gemm(A, self.rep, self.n, self.fmt, self.global_scale, workspace, out)
