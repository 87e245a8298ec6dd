"""Python binding of the C ABI in ``include/mla_decode.h`` and
``include/mla_paging.h`` (ctypes).

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels.  PyTorch tensors supply device memory and the current stream;
their data pointers are handed to the library unchanged.  There is no
fallback path: if the compiled library is missing, loading it raises.

The plan / run split, and the plan arguments (head_dim_ckv = kv_lora_rank,
head_dim_kpe = qk_rope_head_dim, page_size, sm_scale, no causal mask), follow
the decode_wrapper.plan call reviewed in "[WIP] support flashinfer_mla"
(vLLM-metax PR #113).
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libmla_decode.so")

# mla_status_t
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CAPACITY, ERR_CUDA, ERR_DEVICE_TIMEOUT, \
    ERR_DEVICE_BOUNDS, ERR_NOT_PLANNED = range(8)
# mla_dtype_t
DTYPE_BF16, DTYPE_FP8_E4M3, DTYPE_FP32, DTYPE_FP16, DTYPE_Q4 = 0, 1, 2, 3, 4
# mla_kernel_t
KERNEL_DEFAULT, KERNEL_TCGEN05, KERNEL_MMA_SYNC, KERNEL_PAIR, KERNEL_Q4 = 0, 1, 2, 3, 4
KERNELS = {"default": KERNEL_DEFAULT, "tcgen05": KERNEL_TCGEN05, "mma_sync": KERNEL_MMA_SYNC,
           "pair": KERNEL_PAIR, "q4": KERNEL_Q4}
Q4_ROW_BYTES = 304           # of a token in a 4-bit cache, uint8 [num_pages, page_size, Q4_ROW_BYTES]

EXPORTED = ("mla_plan_create", "mla_decode_plan", "mla_decode_run", "mla_decode_run_host",
            "mla_plan_check_status", "mla_plan_info", "mla_plan_destroy", "mla_status_string",
            "mla_plan_last_error", "mla_plan_partition_host", "mla_plan_set_profile_events",
            "mla_decode_noalloc", "mla_decode_plan_multi", "mla_merge_states",
            "mla_absorb_q", "mla_project_out", "mla_build_tables", "mla_rope_append",
            "mla_summarize_pages", "mla_page_scores", "mla_select_pages", "mla_quantize_append",
            "mla_read_cache", "mla_decode_run_q4")


class MLAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("num_sms", ctypes.c_int32), ("num_workers", ctypes.c_int32),
                ("num_units", ctypes.c_int32), ("num_partial_slots", ctypes.c_int32),
                ("num_merge", ctypes.c_int32), ("total_tiles", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kernel", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class RopeSpec(ctypes.Structure):
    """mla_rope_t (see mla_paging.h); made by ``rope_spec``."""
    _fields_ = [("n_axes", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("axis_of_pair", ctypes.c_int32 * 32), ("inv_freq", ctypes.c_double * 32)]


_lib = None
_I32P = ctypes.POINTER(ctypes.c_int32)
_VP = ctypes.c_void_p


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = bind_library(path)
    return _lib


def bind_library(path: str) -> ctypes.CDLL:
    """Open a build of the library at ``path`` and declare the C signatures
    on it (a separate handle; the module's own calls keep using
    ``load_library``'s)."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "paged_mla_decode_02_gb300.build.build() (nvcc, sm_103a)")
    lib = ctypes.CDLL(path)
    c_int, c_float = ctypes.c_int, ctypes.c_float
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [c_int]
    lib.mla_plan_last_error.restype = ctypes.c_char_p
    lib.mla_plan_last_error.argtypes = [_VP]
    lib.mla_plan_create.restype = c_int
    lib.mla_plan_create.argtypes = [c_int, c_int, c_int, ctypes.POINTER(_VP)]
    lib.mla_plan_destroy.restype = c_int
    lib.mla_plan_destroy.argtypes = [_VP]
    lib.mla_decode_plan.restype = c_int
    lib.mla_decode_plan.argtypes = [_VP, _I32P, _VP, _I32P, c_int, c_int, c_int, c_int, c_int,
                                    c_float, _VP]
    lib.mla_absorb_q.restype = c_int
    lib.mla_absorb_q.argtypes = [_VP, _VP, _VP, c_int, c_int, c_int, c_int, _VP]
    lib.mla_project_out.restype = c_int
    lib.mla_project_out.argtypes = [_VP, _VP, _VP, c_int, c_int, c_int, c_int, _VP]
    lib.mla_merge_states.restype = c_int
    lib.mla_merge_states.argtypes = [_VP, _VP, _VP, _VP, _VP, c_int, _VP, c_int, _VP]
    lib.mla_decode_plan_multi.restype = c_int
    lib.mla_decode_plan_multi.argtypes = [_VP, _I32P, _VP, _I32P, c_int, c_int, c_int, c_int,
                                          c_int, c_int, c_float, _VP]
    lib.mla_decode_run.restype = c_int
    lib.mla_decode_run.argtypes = [_VP, _VP, _VP, c_int, _VP, _VP, c_int, c_float, c_int, _VP,
                                   c_int, _VP, _VP]
    lib.mla_decode_run_host.restype = c_int
    lib.mla_decode_run_host.argtypes = lib.mla_decode_run.argtypes
    lib.mla_plan_check_status.restype = c_int
    lib.mla_plan_check_status.argtypes = [_VP]
    lib.mla_plan_info.restype = c_int
    lib.mla_plan_info.argtypes = [_VP, ctypes.POINTER(PlanInfo)]
    lib.mla_plan_set_profile_events.restype = c_int
    lib.mla_plan_set_profile_events.argtypes = [_VP, _VP, _VP]
    lib.mla_plan_partition_host.restype = c_int
    lib.mla_plan_partition_host.argtypes = [_I32P, _I32P, c_int, c_int, c_int, c_int, c_float,
                                            c_int, c_int, _I32P, c_int, _I32P, _I32P, c_int,
                                            _I32P]
    lib.mla_decode_noalloc.restype = c_int
    lib.mla_decode_noalloc.argtypes = [_I32P, _VP, _I32P, c_int, c_int, c_int, c_float, _VP, _VP,
                                       _VP, _VP, c_float, c_int, _VP, c_int, _VP, c_int, _VP]
    c_i64 = ctypes.c_int64
    lib.mla_build_tables.restype = c_int
    lib.mla_build_tables.argtypes = [_VP, _VP, _VP, _VP, c_i64, c_int, _VP, _VP, _VP, c_int, c_int, c_int, _VP,
                                     _VP, c_i64, _VP, _VP, _VP, c_i64, _VP, _VP]
    lib.mla_rope_append.restype = c_int
    lib.mla_rope_append.argtypes = [ctypes.POINTER(RopeSpec), _VP, c_i64, _VP, _VP, c_i64, c_i64, _VP, _VP, c_i64,
                                    _VP, c_i64, _VP, c_float, _VP, _VP, c_int, c_float, c_int, c_int, c_i64, c_int,
                                    c_int, _VP]
    lib.mla_summarize_pages.restype = c_int
    lib.mla_summarize_pages.argtypes = [_VP, c_i64, _VP, _VP, c_int, c_float, c_int, c_int, _VP, c_int, _VP]
    lib.mla_page_scores.restype = c_int
    lib.mla_page_scores.argtypes = [_VP, _VP, _VP, c_int, _VP, _VP, c_i64, c_int, c_int, _VP, c_i64, c_i64, c_int,
                                    _VP]
    lib.mla_select_pages.restype = c_int
    lib.mla_select_pages.argtypes = [_VP, c_i64, c_i64, _VP, _VP, c_i64, c_int, c_int, c_int, c_int, _VP, _VP,
                                     c_i64, c_int, _VP]
    lib.mla_decode_run_q4.restype = c_int
    lib.mla_decode_run_q4.argtypes = [_VP, _VP, _VP, c_int, _VP, c_int, _VP, c_int, _VP, _VP]
    lib.mla_quantize_append.restype = c_int
    lib.mla_quantize_append.argtypes = [_VP, c_i64, _VP, c_i64, c_int, _VP, _VP, c_int, c_int, c_i64, c_int, _VP]
    lib.mla_read_cache.restype = c_int
    lib.mla_read_cache.argtypes = [_VP, _VP, c_int, c_float, c_int, c_int, _VP, _VP, c_i64, _VP, _VP, c_int, _VP,
                                   c_i64, _VP, c_i64, c_int, c_i64, c_int, _VP]
    return lib


def status_string(status: int) -> str:
    return load_library().mla_status_string(status).decode()


def _check(status: int, plan=None, what: str = "") -> None:
    if status != OK:
        lib = load_library()
        detail = lib.mla_plan_last_error(plan).decode() if plan else ""
        msg = f"{what}: {status_string(status)}"
        if detail:
            msg += f" ({detail})"
        raise MLAError(status, msg)


def _i32_host(a) -> np.ndarray:
    """A contiguous host int32 array from a numpy array, list or CPU tensor."""
    if hasattr(a, "detach"):
        if a.device.type != "cpu":
            raise ValueError("kv_indptr / kv_len must be host (CPU) arrays")
        a = a.detach().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(t) -> int:
    return int(t.data_ptr())


def _stream_handle(stream, device=None) -> int:
    import torch
    if stream is None:   # the handle alone: a Stream object costs the host several times as much
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


_dtype_codes: dict = {}


def _dtype_code(t, what: str) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32,
                             torch.float8_e4m3fn: DTYPE_FP8_E4M3, torch.uint8: DTYPE_FP8_E4M3})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _on_cuda(names: str, *tensors) -> None:
    """Each tensor (named in order in ``names``) is a contiguous CUDA tensor."""
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            break
    else:
        return
    for name, t in zip(names.split(), tensors):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")


# ---------------------------------------------------------------------------
# The C ABI entry points, under the same names
# ---------------------------------------------------------------------------

def mla_plan_create(max_batch: int, num_heads: int, kernel="default") -> int:
    """Create a plan on the current CUDA device; returns an opaque handle."""
    lib = load_library()
    handle = _VP()
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    _check(lib.mla_plan_create(int(max_batch), int(num_heads), k, ctypes.byref(handle)), None,
           "mla_plan_create")
    return handle.value


def mla_plan_destroy(plan) -> None:
    if plan:
        load_library().mla_plan_destroy(plan)


def mla_decode_plan(plan, kv_indptr, kv_indices, kv_len, num_heads: int, head_dim_ckv: int,
                    head_dim_kpe: int, page_size: int, sm_scale: float, stream=None) -> None:
    """Plan one batch.  kv_indptr / kv_len are HOST int32 arrays, kv_indices a
    device int32 tensor that must stay alive until the plan's last run."""
    lib = load_library()
    indptr = _i32_host(kv_indptr)
    lens = _i32_host(kv_len)
    batch = lens.shape[0]
    if indptr.shape[0] != batch + 1:
        raise ValueError("kv_indptr must have batch + 1 entries")
    idx_ptr = _ptr(kv_indices) if kv_indices is not None and kv_indices.numel() > 0 else None
    st = lib.mla_decode_plan(plan, indptr.ctypes.data_as(_I32P), idx_ptr,
                             lens.ctypes.data_as(_I32P), batch, int(num_heads),
                             int(head_dim_ckv), int(head_dim_kpe), int(page_size),
                             float(sm_scale), _stream_handle(stream))
    _check(st, plan, "mla_decode_plan")


def mla_decode_plan_multi(plan, kv_indptr, kv_indices, kv_len, q_len: int, num_heads: int,
                          head_dim_ckv: int, head_dim_kpe: int, page_size: int, sm_scale: float,
                          stream=None) -> None:
    """Plan a step of q_len query tokens per request (causal inside the query
    block; see mla_decode.h).  Arrays as for ``mla_decode_plan``."""
    lib = load_library()
    indptr = _i32_host(kv_indptr)
    lens = _i32_host(kv_len)
    batch = lens.shape[0]
    if indptr.shape[0] != batch + 1:
        raise ValueError("kv_indptr must have batch + 1 entries")
    idx_ptr = _ptr(kv_indices) if kv_indices is not None and kv_indices.numel() > 0 else None
    st = lib.mla_decode_plan_multi(plan, indptr.ctypes.data_as(_I32P), idx_ptr,
                                   lens.ctypes.data_as(_I32P), batch, int(q_len), int(num_heads),
                                   int(head_dim_ckv), int(head_dim_kpe), int(page_size),
                                   float(sm_scale), _stream_handle(stream))
    _check(st, plan, "mla_decode_plan_multi")


def _bf16_contig(name, t):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 tensor")


def mla_absorb_q(q_raw, w_uk, q_nope=None, check_status: bool = False, stream=None):
    """q_nope[b,h] = W_UK[h] . q_raw[b,h]: q_raw bf16 [B,H,dn], w_uk bf16
    [H,512,dn]; returns (or fills) q_nope bf16 [B,H,512]."""
    import torch
    B, H, dn = q_raw.shape
    if q_nope is None:
        q_nope = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q_raw.device)
    for name, t in (("q_raw", q_raw), ("w_uk", w_uk), ("q_nope", q_nope)):
        _bf16_contig(name, t)
    if tuple(w_uk.shape) != (H, 512, dn) or tuple(q_nope.shape) != (B, H, 512):
        raise ValueError("w_uk must be [H, 512, dn] and q_nope [B, H, 512]")
    st = load_library().mla_absorb_q(_ptr(q_raw), _ptr(w_uk), _ptr(q_nope), B, H, dn,
                                     int(bool(check_status)), _stream_handle(stream))
    _check(st, None, "mla_absorb_q")
    return q_nope


def mla_project_out(out, w_uv, o=None, check_status: bool = False, stream=None):
    """o[b,h] = out[b,h] . W_UV[h]: out bf16 [B,H,512], w_uv bf16 [H,512,dv];
    returns (or fills) o bf16 [B,H,dv]."""
    import torch
    B, H, _ = out.shape
    dv = w_uv.shape[2]
    if o is None:
        o = torch.empty((B, H, dv), dtype=torch.bfloat16, device=out.device)
    for name, t in (("out", out), ("w_uv", w_uv), ("o", o)):
        _bf16_contig(name, t)
    if tuple(out.shape) != (B, H, 512) or tuple(w_uv.shape) != (H, 512, dv) or tuple(o.shape) != (B, H, dv):
        raise ValueError("out must be [B, H, 512], w_uv [H, 512, dv] and o [B, H, dv]")
    st = load_library().mla_project_out(_ptr(out), _ptr(w_uv), _ptr(o), B, H, dv,
                                        int(bool(check_status)), _stream_handle(stream))
    _check(st, None, "mla_project_out")
    return o


def mla_merge_states(o_a, lse_a, o_b, lse_b, out, lse_out, stream=None) -> None:
    """Combine two attention states of the same rows over disjoint token sets
    by log-sum-exp (see mla_decode.h).  o_a / o_b fp32 [..., 512], lse_a /
    lse_b fp32 [...] on the device; out (bf16 or fp32) and lse_out may alias
    the inputs."""
    import torch
    lib = load_library()
    rows = int(lse_a.numel())
    for name, t in (("o_a", o_a), ("o_b", o_b), ("out", out)):
        if not t.is_contiguous() or t.numel() != rows * 512:
            raise ValueError(f"{name} must be a contiguous [rows, 512] tensor")
    for name, t in (("o_a", o_a), ("o_b", o_b), ("lse_a", lse_a), ("lse_b", lse_b), ("lse_out", lse_out)):
        if t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    if lse_b.numel() != rows or lse_out.numel() != rows:
        raise ValueError("lse tensors must have one entry per row")
    st = lib.mla_merge_states(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(out),
                              _dtype_code(out, "out"), _ptr(lse_out), rows, _stream_handle(stream))
    _check(st, None, "mla_merge_states")


def _check_layouts(q_nope, q_pe, ckv_cache, kpe_cache, out, lse, page_size=None) -> None:
    """The shapes and types mla_decode.h documents, checked before the library
    reads and writes through the raw pointers: the cache [pages, page_size, 512]
    and [pages, page_size, 64] of one dtype, q [..., 512] / [..., 64] of one
    dtype, out [..., 512] and fp32 lse [...] over the same leading dims."""
    cache = ckv_cache.shape
    if len(cache) != 3 or cache[2] != 512:
        raise ValueError(f"ckv_cache must be [num_pages, page_size, 512], got {tuple(cache)}")
    if kpe_cache.shape != (cache[0], cache[1], 64):
        raise ValueError(f"kpe_cache must be [num_pages, page_size, 64] like ckv_cache, "
                         f"got {tuple(kpe_cache.shape)}")
    if kpe_cache.dtype != ckv_cache.dtype:
        raise ValueError("ckv_cache and kpe_cache must have the same dtype")
    if page_size is not None and cache[1] != page_size:
        raise ValueError(f"the cache holds pages of {cache[1]} tokens, the plan {page_size}")
    _check_queries(q_nope, q_pe, out, lse)


def _check_queries(q_nope, q_pe, out, lse) -> None:
    """The queries and outputs of _check_layouts."""
    q = q_nope.shape
    lead = tuple(q[:-1])
    if q[-1] != 512 or q_pe.shape != lead + (64,):
        raise ValueError("q_nope must be [..., 512] and q_pe [..., 64] over the same leading dims")
    if out.shape != q or lse.shape != lead:
        raise ValueError("out must be [..., 512] and lse [...] over q_nope's leading dims")
    if q_pe.dtype != q_nope.dtype:
        raise ValueError(f"q_pe must have q_nope's dtype, got {q_pe.dtype}")
    if _dtype_code(lse, "lse") != DTYPE_FP32:
        raise ValueError(f"lse must be float32, got {lse.dtype}")


def mla_decode_run(plan, q_nope, q_pe, ckv_cache, kpe_cache, out, lse, kv_scale: float = 1.0,
                   stream=None, page_size=None) -> None:
    """Run the planned batch on device tensors (see mla_decode.h for layouts)."""
    lib = load_library()
    _on_cuda("q_nope q_pe ckv_cache kpe_cache out lse", q_nope, q_pe, ckv_cache, kpe_cache, out, lse)
    _check_layouts(q_nope, q_pe, ckv_cache, kpe_cache, out, lse, page_size)
    st = lib.mla_decode_run(plan, q_nope.data_ptr(), q_pe.data_ptr(), _dtype_code(q_nope, "q_nope"),
                            ckv_cache.data_ptr(), kpe_cache.data_ptr(), _dtype_code(ckv_cache, "ckv_cache"),
                            float(kv_scale), ckv_cache.shape[0], out.data_ptr(), _dtype_code(out, "out"),
                            lse.data_ptr(), _stream_handle(stream))
    if st != OK:
        _check(st, plan, "mla_decode_run")


def mla_decode_run_q4(plan, q_nope, q_pe, cache, out, lse, stream=None, page_size=None) -> None:
    """Run the planned batch over a 4-bit cache, uint8 [num_pages, page_size,
    304] (see mla_decode.h); the plan's kernel is "q4"."""
    import torch
    lib = load_library()
    names, tensors = "q_nope q_pe cache out lse", (q_nope, q_pe, cache, out, lse)
    _on_cuda(names, *tensors)
    device = torch.cuda.current_device()
    for i, t in enumerate(tensors):
        if t.get_device() != device:
            raise ValueError(f"{names.split()[i]} must be on the current CUDA device")
    shape = cache.shape
    if cache.dtype != torch.uint8 or len(shape) != 3 or shape[2] != Q4_ROW_BYTES:
        raise ValueError(f"cache must be uint8 [num_pages, page_size, {Q4_ROW_BYTES}], got {cache.dtype} "
                         f"{tuple(shape)}")
    if page_size is not None and shape[1] != page_size:
        raise ValueError(f"the cache holds pages of {shape[1]} tokens, the plan {page_size}")
    _check_queries(q_nope, q_pe, out, lse)
    st = lib.mla_decode_run_q4(plan, q_nope.data_ptr(), q_pe.data_ptr(), _dtype_code(q_nope, "q_nope"),
                               cache.data_ptr(), shape[0], out.data_ptr(), _dtype_code(out, "out"), lse.data_ptr(),
                               _stream_handle(stream, device))
    if st != OK:
        _check(st, plan, "mla_decode_run_q4")


def mla_decode_noalloc(kv_indptr, kv_indices, kv_len, page_size: int, sm_scale: float, q_nope,
                       q_pe, ckv_cache, kpe_cache, out, lse, kv_scale: float = 1.0,
                       check_status: bool = True, stream=None) -> None:
    """Plan + run one batch from the library's fixed scratch memory: the call
    allocates no device memory (out / lse are the caller's tensors).  Calls
    must not overlap; see mla_decode.h for the limits."""
    lib = load_library()
    indptr = _i32_host(kv_indptr)
    lens = _i32_host(kv_len)
    batch = lens.shape[0]
    if indptr.shape[0] != batch + 1:
        raise ValueError("kv_indptr must have batch + 1 entries")
    _on_cuda("q_nope q_pe ckv_cache kpe_cache out lse", q_nope, q_pe, ckv_cache, kpe_cache, out, lse)
    if _dtype_code(q_nope, "q_nope") != DTYPE_BF16 or _dtype_code(ckv_cache, "ckv_cache") != DTYPE_BF16:
        raise ValueError("mla_decode_noalloc takes bf16 queries and caches")
    _check_layouts(q_nope, q_pe, ckv_cache, kpe_cache, out, lse, int(page_size))
    idx_ptr = _ptr(kv_indices) if kv_indices is not None and kv_indices.numel() > 0 else None
    st = lib.mla_decode_noalloc(indptr.ctypes.data_as(_I32P), idx_ptr, lens.ctypes.data_as(_I32P),
                                batch, int(q_nope.shape[1]), int(page_size), float(sm_scale),
                                _ptr(q_nope), _ptr(q_pe), _ptr(ckv_cache), _ptr(kpe_cache),
                                float(kv_scale), int(ckv_cache.shape[0]), _ptr(out),
                                _dtype_code(out, "out"), _ptr(lse), int(bool(check_status)),
                                _stream_handle(stream))
    _check(st, None, "mla_decode_noalloc")


def mla_decode_run_host(plan, q_nope_host, q_pe_host, ckv_cache, kpe_cache, out_host, lse_host,
                        kv_scale: float = 1.0, stream=None) -> None:
    """One decode step from host q buffers to host out / lse (the cache stays on the device)."""
    lib = load_library()
    for name, t in (("q_nope", q_nope_host), ("q_pe", q_pe_host), ("out", out_host),
                    ("lse", lse_host)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    if not ckv_cache.is_cuda or not kpe_cache.is_cuda:
        raise ValueError("the cache must be on the device")
    _check_layouts(q_nope_host, q_pe_host, ckv_cache, kpe_cache, out_host, lse_host)
    st = lib.mla_decode_run_host(plan, _ptr(q_nope_host), _ptr(q_pe_host),
                                 _dtype_code(q_nope_host, "q_nope"), _ptr(ckv_cache),
                                 _ptr(kpe_cache), _dtype_code(ckv_cache, "ckv_cache"),
                                 float(kv_scale), int(ckv_cache.shape[0]), _ptr(out_host),
                                 _dtype_code(out_host, "out"), _ptr(lse_host),
                                 _stream_handle(stream))
    _check(st, plan, "mla_decode_run_host")


def mla_plan_check_status(plan) -> int:
    """Synchronise and return the device status (raises on a device error)."""
    st = load_library().mla_plan_check_status(plan)
    _check(st, plan, "mla_plan_check_status")
    return st


def mla_plan_set_profile_events(plan, start_event, stop_event) -> None:
    """Record torch.cuda.Event start/stop around the decode kernel of every run (None: off)."""
    h0 = int(start_event.cuda_event) if start_event is not None else None
    h1 = int(stop_event.cuda_event) if stop_event is not None else None
    _check(load_library().mla_plan_set_profile_events(plan, h0, h1), plan,
           "mla_plan_set_profile_events")


def mla_plan_info(plan) -> dict:
    info = PlanInfo()
    _check(load_library().mla_plan_info(plan, ctypes.byref(info)), plan, "mla_plan_info")
    return info.as_dict()


def mla_plan_partition_host(kv_indptr, kv_len, num_workers: int, tile_tokens: int,
                            page_size: int, head_dim_ckv: int = 512, head_dim_kpe: int = 64,
                            sm_scale: float = 1.0):
    """The host planner alone: returns (units [n,6], worker_ptr [W+1], merge [m,3], n_slots)."""
    lib = load_library()
    indptr = _i32_host(kv_indptr)
    lens = _i32_host(kv_len)
    batch = lens.shape[0]
    ucap = num_workers + batch
    units = np.zeros((ucap, 6), np.int32)
    wptr = np.zeros(num_workers + 1, np.int32)
    merge = np.zeros((batch, 3), np.int32)
    counts = np.zeros(3, np.int32)
    st = lib.mla_plan_partition_host(indptr.ctypes.data_as(_I32P), lens.ctypes.data_as(_I32P),
                                     batch, head_dim_ckv, head_dim_kpe, page_size, sm_scale,
                                     num_workers, tile_tokens, units.ctypes.data_as(_I32P), ucap,
                                     wptr.ctypes.data_as(_I32P), merge.ctypes.data_as(_I32P),
                                     batch, counts.ctypes.data_as(_I32P))
    if st != OK:
        raise MLAError(st, f"mla_plan_partition_host: {status_string(st)}")
    return units[:counts[0]].copy(), wptr, merge[:counts[2]].copy(), int(counts[1])


# ---------------------------------------------------------------------------
# Around the decode (include/mla_paging.h)
# ---------------------------------------------------------------------------

def _on_device(device: int, dtype, names: str, *tensors, contiguous: bool = True) -> None:
    """Each tensor (named in order in ``names``) is on CUDA device ``device``
    (the current one), of ``dtype`` and (by default) contiguous."""
    for t in tensors:
        if t.get_device() != device or t.dtype is not dtype or (contiguous and not t.is_contiguous()):
            break
    else:
        return
    for name, t in zip(names.split(), tensors):
        if t.get_device() != device:
            raise ValueError(f"{name} must be on the current CUDA device")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _torch_stream(stream):
    import torch
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))


def _empty(shape, dtype, device, stream):
    """Memory for what a call fills, of the stream it fills it on: a block that
    another stream gave back may still be read there."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_stride(name: str, t, rows: int, cols=None) -> int:
    """The row stride of a [rows, cols] tensor whose rows are runs of adjacent
    entries (strides of dimensions of one entry or none say nothing)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be [{rows}, {'columns' if cols is None else cols}], got {tuple(shape)}")
    if shape[1] > 1 and rows > 0 and stride[1] != 1:
        raise ValueError(f"{name} must have adjacent entries in a row")
    if rows < 2:
        return shape[1]
    if stride[0] < 0:
        raise ValueError(f"{name} must not have a negative stride")
    return stride[0]


def _check_cache(device: int, ckv_cache, kpe_cache) -> int:
    """The layout of a paged cache; returns its dtype code."""
    code = _dtype_code(ckv_cache, "ckv_cache")
    if code == DTYPE_FP32:
        raise ValueError("ckv_cache must be bfloat16 or float8_e4m3fn")
    _on_device(device, ckv_cache.dtype, "ckv_cache kpe_cache", ckv_cache, kpe_cache)
    shape = ckv_cache.shape
    if len(shape) != 3 or shape[2] != 512:
        raise ValueError(f"ckv_cache must be [num_pages, page_size, 512], got {tuple(shape)}")
    if kpe_cache.shape != (shape[0], shape[1], 64):
        raise ValueError(f"kpe_cache must be [num_pages, page_size, 64] like ckv_cache, "
                         f"got {tuple(kpe_cache.shape)}")
    return code


def mla_build_tables(kv_len, new_len, block_table, free_pages, free_count, page_size: int, kv_indptr, kv_indices,
                     q_indptr, slots, positions, status, kv_len_out=None, free_count_out=None, stream=None) -> None:
    """One step of the page tables on the device (see mla_paging.h): kv_len,
    new_len [B]; block_table [B, max_pages] (rows may be strided); free_pages
    [num_pages]; outputs kv_indptr, q_indptr [B + 1], kv_indices, slots
    (int64), positions, status [1].  Without kv_len_out / free_count_out the
    lengths and the count are updated in place.  Decodes are planned from host
    lengths: the caller keeps those as well, and reads ``status`` to learn of a
    step that was refused."""
    import torch
    if kv_len_out is None:
        kv_len_out = kv_len
    if free_count_out is None:
        free_count_out = free_count
    device = torch.cuda.current_device()
    _on_device(device, torch.int32, "kv_len new_len kv_len_out free_pages free_count free_count_out kv_indptr kv_indices "
               "q_indptr positions status", kv_len, new_len, kv_len_out, free_pages, free_count, free_count_out,
               kv_indptr, kv_indices, q_indptr, positions, status)
    _on_device(device, torch.int32, "block_table", block_table, contiguous=False)
    _on_device(device, torch.int64, "slots", slots)
    batch = kv_len.numel()
    stride = _row_stride("block_table", block_table, batch)
    if new_len.numel() != batch or kv_len_out.numel() != batch:
        raise ValueError("kv_len, new_len and kv_len_out must have one entry per request")
    if kv_indptr.numel() != batch + 1 or q_indptr.numel() != batch + 1:
        raise ValueError("kv_indptr and q_indptr must have batch + 1 entries")
    if positions.numel() != slots.numel():
        raise ValueError("slots and positions must have the same length")
    if free_count.numel() != 1 or free_count_out.numel() != 1 or status.numel() != 1:
        raise ValueError("free_count, free_count_out and status must have one entry")
    st = load_library().mla_build_tables(
        kv_len.data_ptr(), new_len.data_ptr(), kv_len_out.data_ptr(), block_table.data_ptr(), stride,
        block_table.shape[1], free_pages.data_ptr(), free_count.data_ptr(), free_count_out.data_ptr(),
        free_pages.numel(), batch, int(page_size), kv_indptr.data_ptr(), kv_indices.data_ptr(), kv_indices.numel(),
        q_indptr.data_ptr(), slots.data_ptr(), positions.data_ptr(), slots.numel(), status.data_ptr(),
        _stream_handle(stream, device))
    _check(st, None, "mla_build_tables")


def rope_spec(inv_freq, axis_of_pair=None, interleaved: bool = False, scale: float = 1.0) -> RopeSpec:
    """The rotary embedding of the 64 rope dims: 32 inverse frequencies
    (radians per position), for each pair the position axis it follows (all
    the first by default), and the layout of a pair: dims (2i, 2i+1) if
    interleaved, else (i, i+32).  ``scale`` multiplies cos and sin."""
    freq = [float(f) for f in inv_freq]
    axes = [0] * 32 if axis_of_pair is None else [int(a) for a in axis_of_pair]
    if len(freq) != 32 or len(axes) != 32:
        raise ValueError("inv_freq and axis_of_pair must have 32 entries")
    spec = RopeSpec(max(axes) + 1, int(bool(interleaved)), float(scale))
    spec.axis_of_pair[:] = axes
    spec.inv_freq[:] = freq
    return spec


def mla_rope_append(rope: RopeSpec, positions, slots, q_pe, ckv, kpe, norm_weight, eps: float, ckv_cache, kpe_cache,
                    q_pe_out=None, kv_scale: float = 1.0, check_status: bool = False, stream=None):
    """Rotate the queries and rope keys of a step's tokens, norm their latent
    rows and write both into the cache at ``slots`` (see mla_paging.h).
    positions int32 [n_axes, T] (or [T] for one axis; an expanded first
    dimension is taken as it is), slots int64 [T], q_pe [T, H, 64] or None,
    ckv [T, 512], kpe [T, 64] bf16 (rows may be strided), norm_weight bf16
    [512] or None.  Returns (or fills) q_pe_out, contiguous."""
    import torch
    device = torch.cuda.current_device()
    code = _check_cache(device, ckv_cache, kpe_cache)
    if positions.dim() == 1:
        positions = positions[None]
    _on_device(device, torch.int32, "positions", positions, contiguous=False)
    _on_device(device, torch.int64, "slots", slots)
    if q_pe is None:
        _on_device(device, torch.bfloat16, "ckv kpe", ckv, kpe, contiguous=False)
    else:
        _on_device(device, torch.bfloat16, "ckv kpe q_pe", ckv, kpe, q_pe, contiguous=False)
    T = slots.numel()
    n_axes = rope.n_axes
    if positions.dim() != 2 or positions.shape[0] < n_axes:
        raise ValueError("positions must be [n_axes, tokens]")
    axis_stride = _row_stride("positions", positions, positions.shape[0], T)
    ckv_stride, kpe_stride = _row_stride("ckv", ckv, T, 512), _row_stride("kpe", kpe, T, 64)
    if norm_weight is not None:
        _on_device(device, torch.bfloat16, "norm_weight", norm_weight)
        if norm_weight.numel() != 512:
            raise ValueError("norm_weight must have 512 entries")
    H, q_ptr, q_t, q_h, out_ptr = 0, None, 0, 0, None
    if q_pe is not None:
        if q_pe.dim() != 3 or q_pe.shape[0] != T or q_pe.shape[2] != 64 or (q_pe.numel() and q_pe.stride(2) != 1):
            raise ValueError("q_pe must be [tokens, heads, 64] with adjacent dims")
        H = q_pe.shape[1]
        q_t, q_h = q_pe.stride(0) if T > 1 else 0, q_pe.stride(1) if H > 1 else 0
        if q_pe_out is None:
            q_pe_out = _empty((T, H, 64), torch.bfloat16, q_pe.device, stream)
        else:
            _on_device(device, torch.bfloat16, "q_pe_out", q_pe_out)
            if q_pe_out.shape != q_pe.shape:
                raise ValueError("q_pe_out must have the shape of q_pe")
        q_ptr, out_ptr = q_pe.data_ptr(), q_pe_out.data_ptr()
    elif q_pe_out is not None:
        raise ValueError("q_pe_out needs q_pe")
    st = load_library().mla_rope_append(
        ctypes.byref(rope), positions.data_ptr(), axis_stride, slots.data_ptr(), q_ptr,
        q_t, q_h, out_ptr, ckv.data_ptr(), ckv_stride, kpe.data_ptr(), kpe_stride,
        None if norm_weight is None else norm_weight.data_ptr(), eps, ckv_cache.data_ptr(), kpe_cache.data_ptr(),
        code, kv_scale, ckv_cache.shape[0], ckv_cache.shape[1], T, H, int(bool(check_status)),
        _stream_handle(stream, device))
    _check(st, None, "mla_rope_append")
    return q_pe_out


def mla_summarize_pages(slots, ckv_cache, kpe_cache, summaries, kv_scale: float = 1.0, check_status: bool = False,
                        stream=None) -> None:
    """Mean rows of the pages that the tokens at ``slots`` completed, into
    summaries bf16 [num_pages, 576] (see mla_paging.h)."""
    import torch
    device = torch.cuda.current_device()
    code = _check_cache(device, ckv_cache, kpe_cache)
    _on_device(device, torch.int64, "slots", slots)
    _on_device(device, torch.bfloat16, "summaries", summaries)
    if summaries.shape != (ckv_cache.shape[0], 576):
        raise ValueError("summaries must be [num_pages, 576]")
    st = load_library().mla_summarize_pages(slots.data_ptr(), slots.numel(), ckv_cache.data_ptr(),
                                            kpe_cache.data_ptr(), code, kv_scale, ckv_cache.shape[0],
                                            ckv_cache.shape[1], summaries.data_ptr(), int(bool(check_status)),
                                            _stream_handle(stream, device))
    _check(st, None, "mla_summarize_pages")


def mla_page_scores(q_nope, q_pe, summaries, kv_indptr, kv_indices, scores, check_status: bool = False,
                    stream=None) -> None:
    """scores[r, p] = best score over the heads of row r of the p-th page of
    its list (see mla_paging.h): q_nope bf16 [R, H, 512], q_pe bf16 [R, H, 64]
    (or [R, tokens, heads, .]: one choice for all of a request's query tokens),
    kv_indptr / kv_indices int32 device tensors, scores fp32 [R, >= longest
    list] (rows may be strided)."""
    import torch
    device = torch.cuda.current_device()
    _on_device(device, torch.bfloat16, "q_nope q_pe summaries", q_nope, q_pe, summaries)
    _on_device(device, torch.int32, "kv_indptr kv_indices", kv_indptr, kv_indices)
    _on_device(device, torch.float32, "scores", scores, contiguous=False)
    rows = kv_indptr.numel() - 1
    lead = q_nope.shape[:-1]
    if len(lead) not in (2, 3) or lead[0] != rows or q_nope.shape[-1] != 512 or q_pe.shape != lead + (64,):
        raise ValueError("q_nope must be [rows, ..., 512] and q_pe [rows, ..., 64], kv_indptr [rows + 1]")
    if summaries.dim() != 2 or summaries.shape[1] != 576:
        raise ValueError("summaries must be [num_pages, 576]")
    stride = _row_stride("scores", scores, rows)
    if stride < scores.shape[1]:
        raise ValueError("scores must not overlap")
    heads = lead[1] if len(lead) == 2 else lead[1] * lead[2]
    st = load_library().mla_page_scores(q_nope.data_ptr(), q_pe.data_ptr(), summaries.data_ptr(),
                                        summaries.shape[0], kv_indptr.data_ptr(), kv_indices.data_ptr(),
                                        kv_indices.numel(), rows, heads, scores.data_ptr(), stride, scores.shape[1],
                                        int(bool(check_status)), _stream_handle(stream, device))
    _check(st, None, "mla_page_scores")


def mla_select_pages(scores, kv_indptr, kv_indices, top_k: int, keep_first: int, keep_last: int, sel_indptr,
                     sel_indices, check_status: bool = False, stream=None) -> None:
    """The page lists of a sparse decode: of each row's pages the first
    keep_first, the last keep_last and the best scoring others, min(top_k, n)
    in all, in their order (see mla_paging.h)."""
    import torch
    device = torch.cuda.current_device()
    _on_device(device, torch.int32, "kv_indptr kv_indices sel_indptr sel_indices", kv_indptr, kv_indices, sel_indptr,
               sel_indices)
    _on_device(device, torch.float32, "scores", scores, contiguous=False)
    rows = kv_indptr.numel() - 1
    stride = _row_stride("scores", scores, rows)
    if stride < scores.shape[1]:
        raise ValueError("scores must not overlap")
    if sel_indptr.numel() != rows + 1:
        raise ValueError("sel_indptr must have rows + 1 entries")
    st = load_library().mla_select_pages(scores.data_ptr(), stride, scores.shape[1], kv_indptr.data_ptr(),
                                         kv_indices.data_ptr(), kv_indices.numel(), rows, int(top_k),
                                         int(keep_first), int(keep_last), sel_indptr.data_ptr(),
                                         sel_indices.data_ptr(), sel_indices.numel(), int(bool(check_status)),
                                         _stream_handle(stream, device))
    _check(st, None, "mla_select_pages")


_row_codes: dict = {}


def _row_code(name: str, t) -> int:
    """The dtype code of plain rows given to or taken from a cache."""
    if not _row_codes:
        import torch
        _row_codes.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32})
    code = _row_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _check_q4_cache(device: int, cache):
    """The layout of a 4-bit cache; returns its shape."""
    import torch
    _on_device(device, torch.uint8, "cache", cache)
    shape = cache.shape
    if len(shape) != 3 or shape[2] != Q4_ROW_BYTES:
        raise ValueError(f"cache must be [num_pages, page_size, {Q4_ROW_BYTES}], got {tuple(shape)}")
    return shape


def mla_quantize_append(ckv, kpe, slots, cache, check_status: bool = False, stream=None) -> None:
    """Rows into a 4-bit cache, uint8 [num_pages, page_size, 304], at ``slots``
    (see mla_paging.h): ckv [T, 512] and kpe [T, 64] of one type (bf16, fp16 or
    fp32; rows may be strided), slots int64 [T], negative for padding."""
    import torch
    device = torch.cuda.current_device()
    shape = _check_q4_cache(device, cache)
    code = _row_code("ckv", ckv)
    _on_device(device, ckv.dtype, "ckv kpe", ckv, kpe, contiguous=False)
    _on_device(device, torch.int64, "slots", slots)
    T = slots.numel()
    ckv_stride, kpe_stride = _row_stride("ckv", ckv, T, 512), _row_stride("kpe", kpe, T, 64)
    st = load_library().mla_quantize_append(ckv.data_ptr(), ckv_stride, kpe.data_ptr(), kpe_stride, code,
                                            slots.data_ptr(), cache.data_ptr(), shape[0], shape[1], T,
                                            int(bool(check_status)), _stream_handle(stream, device))
    _check(st, None, "mla_quantize_append")


def mla_read_cache(cache, kpe_cache, kv_indptr, kv_indices, starts, row_indptr, ckv_out, kpe_out,
                   kv_scale: float = 1.0, check_status: bool = False, stream=None) -> None:
    """Tokens starts[b], starts[b] + 1, .. of each request out of a paged cache
    into the rows row_indptr[b] .. row_indptr[b + 1] - 1 of ckv_out [N, 512]
    and kpe_out [N, 64] (bf16, fp16 or fp32; rows may be strided; see
    mla_paging.h).  ``cache``: a 4-bit cache, with kpe_cache None, or the ckv
    part of a bf16 or e4m3 one.  kv_indptr, row_indptr int32 [B + 1], starts
    int32 [B] and kv_indices int32 on the device."""
    import torch
    device = torch.cuda.current_device()
    if kpe_cache is None:
        _check_q4_cache(device, cache)
        kind, kpe_ptr = DTYPE_Q4, None
    else:
        kind, kpe_ptr = _check_cache(device, cache, kpe_cache), kpe_cache.data_ptr()
    _on_device(device, torch.int32, "kv_indptr kv_indices starts row_indptr", kv_indptr, kv_indices, starts,
               row_indptr)
    batch = starts.numel()
    if kv_indptr.numel() != batch + 1 or row_indptr.numel() != batch + 1:
        raise ValueError("kv_indptr and row_indptr must have one entry more than starts")
    code = _row_code("ckv_out", ckv_out)
    _on_device(device, ckv_out.dtype, "ckv_out kpe_out", ckv_out, kpe_out, contiguous=False)
    N = ckv_out.shape[0]
    ckv_stride, kpe_stride = _row_stride("ckv_out", ckv_out, N, 512), _row_stride("kpe_out", kpe_out, N, 64)
    st = load_library().mla_read_cache(cache.data_ptr(), kpe_ptr, kind, kv_scale, cache.shape[0], cache.shape[1],
                                       kv_indptr.data_ptr(), kv_indices.data_ptr(), kv_indices.numel(),
                                       starts.data_ptr(), row_indptr.data_ptr(), batch, ckv_out.data_ptr(),
                                       ckv_stride, kpe_out.data_ptr(), kpe_stride, code, N, int(bool(check_status)),
                                       _stream_handle(stream, device))
    _check(st, None, "mla_read_cache")


# ---------------------------------------------------------------------------
# Convenience wrappers
# ---------------------------------------------------------------------------

class MLADecoder:
    """Owns one plan: ``plan(...)`` once per batch layout, ``run(...)`` per step."""

    def __init__(self, max_batch: int, num_heads: int, kernel="default"):
        self.num_heads = int(num_heads)
        self.handle = mla_plan_create(max_batch, num_heads, kernel)
        self._kv_indices = None
        self.page_size = None
        self._rows = 0                    # query rows of the planned batch

    def plan(self, kv_indptr, kv_indices, kv_len, page_size: int, sm_scale: float,
             head_dim_ckv: int = 512, head_dim_kpe: int = 64, stream=None, q_len: int = 0) -> None:
        """q_len 0: one query token per request (q and out [B, H, .]);
        q_len >= 1: that many, causal inside the block (q and out [B, Q, H, .])."""
        if q_len:
            mla_decode_plan_multi(self.handle, kv_indptr, kv_indices, kv_len, q_len,
                                  self.num_heads, head_dim_ckv, head_dim_kpe, page_size,
                                  sm_scale, stream)
        else:
            mla_decode_plan(self.handle, kv_indptr, kv_indices, kv_len, self.num_heads,
                            head_dim_ckv, head_dim_kpe, page_size, sm_scale, stream)
        self.q_len = int(q_len)
        self.page_size = int(page_size)
        self._rows = len(kv_len) * max(1, self.q_len) * self.num_heads
        self._kv_indices = kv_indices     # keep the borrowed page table alive

    def run(self, q_nope, q_pe, ckv_cache, kpe_cache, out=None, lse=None,
            kv_scale: float = 1.0, out_dtype=None, stream=None):
        import torch
        lead = tuple(q_nope.shape[:-1])          # (B, H) or (B, Q, H)
        if out is None:
            out = torch.empty(lead + (512,), dtype=out_dtype or torch.bfloat16, device=q_nope.device)
        if lse is None:
            lse = torch.empty(lead, dtype=torch.float32, device=q_nope.device)
        mla_decode_run(self.handle, q_nope, q_pe, ckv_cache, kpe_cache, out, lse, kv_scale, stream,
                       page_size=self.page_size)
        return out, lse

    def run_q4(self, q_nope, q_pe, cache, out=None, lse=None, out_dtype=None, stream=None):
        """run() over a 4-bit cache, for a decoder made with kernel="q4": q_nope
        [B, H, 512], with q_len [B, Q, H, 512] (or a view of that as [B, Q * H, 512]
        or [B * Q, H, 512]).  Rows of q_nope behind the planned batch are not read,
        theirs of out and lse left as they were."""
        import torch
        lead = tuple(q_nope.shape[:-1])
        if self.page_size is not None:        # (else there is no plan, which the call below says)
            q_len = max(1, self.q_len)
            rows = (self.num_heads,), (q_len * self.num_heads,), (q_len, self.num_heads)
            if not (lead[1:] in rows and math.prod(lead) >= self._rows):
                raise ValueError(f"q_nope must hold the plan's {self._rows} query rows as [batch, "
                                 f"{f'{q_len}, ' if q_len > 1 else ''}{self.num_heads}, 512], got {tuple(q_nope.shape)}")
        if out is None:
            out = _empty(lead + (512,), out_dtype or torch.bfloat16, q_nope.device, stream)
        if lse is None:
            lse = _empty(lead, torch.float32, q_nope.device, stream)
        mla_decode_run_q4(self.handle, q_nope, q_pe, cache, out, lse, stream, page_size=self.page_size)
        return out, lse

    def info(self) -> dict:
        return mla_plan_info(self.handle)

    def check_status(self) -> int:
        return mla_plan_check_status(self.handle)

    def close(self) -> None:
        if self.handle:
            mla_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MLASparseDecoder:
    """A decode that reads at most ``top_k`` pages of each request: the first
    ``keep_first``, the last ``keep_last`` and those whose mean rows score best
    against the query.  ``plan(...)`` once per batch layout, ``run(...)`` per
    step or layer: mla_page_scores, mla_select_pages, then the decode over the
    selected pages, all queued on the stream without synchronisation.

    Holds lists of up to ``max_pages`` pages for each of ``max_batch`` requests
    (of which a plan takes at most 4096, and batch x top_k <= 2^31 - 1).
    A captured run replays after re-plans of at most the captured batch and of
    the captured q_len; like a decode plan's graph it keeps the addresses it was
    captured with, that of the page list included.  The list may be passed
    shorter or longer there at every plan (``indices[:n]`` of one buffer).

    With q_len query tokens per request (q_len x heads <= 128, batch x q_len <=
    max_batch) the choice is theirs together, and keep_last must cover the
    pages that hold them.

    Its runs share its buffers, as those of a plan do: one at a time."""

    def __init__(self, max_batch: int, num_heads: int, max_pages: int, top_k: int, keep_first: int = 1,
                 keep_last: int = 1, kernel="default"):
        import torch
        if top_k < 1 or keep_first < 0 or keep_last < 1 or keep_first + keep_last > top_k:
            raise ValueError("top_k must cover keep_first >= 0 and keep_last >= 1 pages")
        if max_pages < 1:
            raise ValueError("max_pages must be >= 1")
        self.decoder = MLADecoder(max_batch, num_heads, kernel)
        self.max_batch, self.max_pages = int(max_batch), int(max_pages)
        self.top_k, self.keep_first, self.keep_last = int(top_k), int(keep_first), int(keep_last)
        dev = torch.device("cuda", torch.cuda.current_device())
        self.sel_indices = torch.zeros(self.max_batch * self.top_k, dtype=torch.int32, device=dev)
        self._sel_indptr = torch.zeros(self.max_batch + 1, dtype=torch.int32, device=dev)
        self._kv_indptr = torch.zeros(self.max_batch + 1, dtype=torch.int32, device=dev)
        # the offsets on their way there: written again once the last upload has read them
        self._staged_indptr = torch.zeros(self.max_batch + 1, dtype=torch.int32, pin_memory=True)
        self._uploaded = torch.cuda.Event()
        self._scores = torch.empty((self.max_batch, self.max_pages), dtype=torch.float32, device=dev)
        self._kv_indices, self.sel_indptr, self.batch = None, None, 0
        torch.cuda.current_stream().synchronize()   # the zeros are in place for a run on any stream

    def plan(self, kv_indptr, kv_indices, kv_len, page_size: int, sm_scale: float, stream=None,
             q_len: int = 0) -> None:
        """Arguments as for ``MLADecoder.plan``: the whole page lists, of which
        run() reads the selected pages.  Like that plan it queues its uploads on
        the stream and waits for those of the plan before it alone."""
        import torch
        indptr, lens = _i32_host(kv_indptr), _i32_host(kv_len)
        if lens.ndim != 1 or indptr.shape != (lens.shape[0] + 1,):
            raise ValueError("kv_indptr must have batch + 1 entries")
        if page_size not in (16, 32, 64):
            raise MLAError(ERR_UNSUPPORTED, "page_size must be 16, 32 or 64")
        batch = lens.shape[0]
        pages = np.diff(indptr.astype(np.int64))
        if indptr[0] != 0 or np.any(lens < 0) or np.any(pages != -(-lens.astype(np.int64) // page_size)):
            raise ValueError("kv_indptr must count ceil(kv_len / page_size) pages for each request")
        if batch > self.max_batch or np.any(pages > self.max_pages):
            raise MLAError(ERR_CAPACITY, "the batch exceeds the decoder's max_batch or max_pages")
        if batch > 4096 or batch * self.top_k > 2 ** 31 - 1:   # what the scores and the selection take
            raise MLAError(ERR_CAPACITY, "more than 4096 requests, or batch x top_k past 2^31 - 1")
        _on_device(torch.cuda.current_device(), torch.int32, "kv_indices", kv_indices)
        if kv_indices.numel() < indptr[-1]:
            raise ValueError("kv_indices is shorter than kv_indptr says")
        if q_len * self.decoder.num_heads > 128:
            raise MLAError(ERR_UNSUPPORTED, "q_len x heads exceeds 128")
        if q_len > 1 and (self.keep_last - 1) * page_size + 1 < q_len:
            raise ValueError("keep_last must cover the pages of the q_len query tokens")
        kept = np.minimum(pages, self.top_k)
        sel_indptr = np.zeros(batch + 1, np.int32)
        sel_indptr[1:] = np.cumsum(kept)
        sel_len = (lens - (pages - kept) * page_size).astype(np.int32)
        self.decoder.plan(sel_indptr, self.sel_indices, sel_len, page_size, sm_scale, stream=stream, q_len=q_len)
        # rows past the batch get empty lists: a graph of a larger batch replays this plan
        self._uploaded.synchronize()
        whole = self._staged_indptr.numpy()
        whole[:batch + 1] = indptr
        whole[batch + 1:] = indptr[-1]
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else _torch_stream(stream)):
            self._kv_indptr.copy_(self._staged_indptr, non_blocking=True)
            self._uploaded.record()
        self._kv_indices, self.batch = kv_indices, batch   # keep the borrowed page list alive
        self.sel_indptr = self._sel_indptr[:batch + 1]   # device offsets of the selected pages, after a run
        # the arguments of run()'s calls that stay as they are.  A captured run keeps
        # them while later plans lengthen the list at its place, so its bound is not
        # the list's length (the plan checked that) but the memory behind its first
        # entry, or what the decoder holds.
        behind = kv_indices.untyped_storage().nbytes() // kv_indices.element_size() - kv_indices.storage_offset()
        lists = (self._kv_indptr.data_ptr(), kv_indices.data_ptr(), min(behind, self.max_batch * self.max_pages), batch)
        self._heads = self.decoder.num_heads * max(q_len, 1)
        self._choice = (self._scores.data_ptr(), self.max_pages, self.max_pages)
        self._score_args = lists
        self._select_args = self._choice + lists + (self.top_k, self.keep_first, self.keep_last,
                                                    self._sel_indptr.data_ptr(), self.sel_indices.data_ptr(),
                                                    self.sel_indices.numel(), 0)

    def run(self, q_nope, q_pe, ckv_cache, kpe_cache, summaries, out=None, lse=None, kv_scale: float = 1.0,
            out_dtype=None, stream=None):
        """One step: q_nope [B, H, 512] and q_pe [B, H, 64] (or [B, Q, H, .]),
        the cache and its page summaries [num_pages, 576]; returns out, lse."""
        out, lse, stream = self._choose(q_nope, q_pe, summaries, out, lse, out_dtype, stream)
        return self.decoder.run(q_nope, q_pe, ckv_cache, kpe_cache, out, lse, kv_scale, out_dtype, stream)

    def run_q4(self, q_nope, q_pe, cache, summaries, out=None, lse=None, out_dtype=None, stream=None):
        """run() over a 4-bit cache, for a decoder made with kernel="q4".  Its
        pages' summaries are those of the rows before they were quantised, or of
        the rows that mla_read_cache brings back."""
        out, lse, stream = self._choose(q_nope, q_pe, summaries, out, lse, out_dtype, stream)
        return self.decoder.run_q4(q_nope, q_pe, cache, out, lse, out_dtype, stream)

    def _choose(self, q_nope, q_pe, summaries, out, lse, out_dtype, stream):
        """Queues the choice of pages; returns what the decode over them takes."""
        if self._kv_indices is None:
            raise MLAError(ERR_NOT_PLANNED, "MLASparseDecoder.run before plan")
        import torch
        device = torch.cuda.current_device()
        _on_device(device, torch.bfloat16, "q_nope q_pe summaries", q_nope, q_pe, summaries)
        if self._scores.get_device() != device:
            raise ValueError("the decoder was made on another CUDA device than the current one")
        q, rows = q_nope.shape, summaries.shape
        if len(q) not in (3, 4) or q[0] != self.batch or q[-1] != 512 or q_pe.shape != q[:-1] + (64,):
            raise ValueError("q_nope must be [batch, ..., heads, 512] and q_pe [batch, ..., heads, 64]")
        if len(rows) != 2 or rows[1] != 576:
            raise ValueError("summaries must be [num_pages, 576]")
        heads = q[1] if len(q) == 3 else q[1] * q[2]
        if heads != self._heads:   # the decode reads as many rows as were planned
            raise ValueError(f"q_nope must have {self._heads} query rows (tokens x heads) per request, got {heads}")
        if stream is not None:   # (the decode would take them from the current stream)
            if out is None:
                out = _empty(tuple(q), out_dtype or torch.bfloat16, q_nope.device, stream)
            if lse is None:
                lse = _empty(tuple(q[:-1]), torch.float32, q_nope.device, stream)
        lib, stream = load_library(), _stream_handle(stream)
        st = lib.mla_page_scores(q_nope.data_ptr(), q_pe.data_ptr(), summaries.data_ptr(), rows[0], *self._score_args,
                                 heads, *self._choice, 0, stream)
        if st == OK:
            st = lib.mla_select_pages(*self._select_args, stream)
        if st != OK:
            _check(st, None, "MLASparseDecoder.run")
        return out, lse, stream

    def check_status(self) -> int:
        """Synchronise and raise on a device error of the decode, or of any call of
        mla_paging.h on this device since the last check: those calls and all
        sparse decoders share one word, which the first to ask reads and clears."""
        import torch
        torch.cuda.synchronize()
        # a call of no rows queues nothing and reports what the kernels recorded
        _check(load_library().mla_page_scores(None, None, None, 1, None, None, 0, 0, 1, None, 0, 0, 1,
                                              _stream_handle(None)), None, "MLASparseDecoder")
        return self.decoder.check_status()

    def close(self) -> None:
        self.decoder.close()
