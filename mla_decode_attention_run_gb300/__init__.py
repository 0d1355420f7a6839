"""Paged MLA decode over an FP8 E4M3 or 4-bit KV cache on GB300 (sm_103a).

Thin Python binding of libmla_decode.so (C ABI in include/mla_decode.h).  The
functions below carry the C entry points' names and only marshal arguments:
torch tensors provide device memory and streams, every step of the path runs
in the library's CUDA kernels.  There is no CPU fallback: if the library is
missing or cannot load, importing a function raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "MLA_KV_FP8_E4M3", "MLA_KV_BF16", "MLAError", "library", "library_path",
    "mla_decode_plan", "mla_decode_run", "mla_decode_plan_destroy", "mla_decode_plan_info",
    "mla_decode_schedule", "kv_store_fp8", "kv_gather_cast", "mla_get_last_error",
    "exported_symbols", "D_CKV", "D_KPE", "D_QK", "mla_decode_run_static_scratch",
    "STATIC_SCRATCH_BYTES", "mla_extend_plan", "mla_extend_run", "mla_extend_schedule",
    "kv_proj_store_fp8", "mla_debug_set_wait_limit", "MLA_KV_FP4_E2M1", "kv_store_fp4",
    "kv_gather_fp4", "mla_norm_rope_store", "kv_tables_update", "FP4_CKV_BYTES", "FP4_KPE_BYTES",
    "FP4_ROW_BYTES",
]

D_CKV, D_KPE, D_QK = 512, 64, 576
MLA_KV_FP8_E4M3, MLA_KV_BF16, MLA_KV_FP4_E2M1 = 0, 1, 2
FLAG_INDEX_OOB, FLAG_PLAN_MISMATCH, FLAG_WAIT_TIMEOUT, FLAG_TABLES_REFUSED = 0x1, 0x2, 0x4, 0x8
FP4_CKV_BYTES, FP4_KPE_BYTES, FP4_ROW_BYTES = 272, 34, 320   # a 4-bit row's parts; a combined row
STATIC_SCRATCH_BYTES = 8 << 20       # MLA_STATIC_SCRATCH_BYTES

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla_decode.so")
_lib = None

_P = ctypes.c_void_p
_i32, _i64, _f32, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_PI32 = ctypes.POINTER(ctypes.c_int32)


class MLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = library().mla_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{where}: status {status} ({msg})")


def library():
    """Load libmla_decode.so (built by build.py); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(
            f"{library_path} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python mla_decode_attention_run_gb300/build.py)")
    lib = ctypes.CDLL(library_path)
    lib.mla_decode_plan.argtypes = [ctypes.POINTER(_P), _P, _P, _i32, _i32, _i32, ctypes.c_int,
                                    ctypes.POINTER(_sz), _P]
    lib.mla_decode_run.argtypes = [_P, _P, _i64, _i64, _P, _i64, _P, _i64, _i64, _P, _P, _P, _f32,
                                   _f32, _P, _P, _P, _sz, _P]
    lib.mla_decode_run_static_scratch.argtypes = [_P, _P, _i64, _i64, _P, _i64, _P, _i64, _i64,
                                                  _P, _P, _P, _f32, _f32, _P, _P, _P]
    lib.mla_decode_plan_destroy.argtypes = [_P]
    lib.mla_decode_plan_info.argtypes = [_P, _PI32, _PI32, _PI32, ctypes.POINTER(_sz)]
    lib.mla_decode_schedule.argtypes = [_P, _P, _i32, _i32, _i32, ctypes.c_int, _i32, _P, _i32,
                                        _PI32, _PI32, _PI32, _PI32, _PI32, ctypes.POINTER(_sz)]
    lib.mla_extend_plan.argtypes = [ctypes.POINTER(_P), _P, _P, _P, _i32, _i32, _i32, ctypes.c_int,
                                    ctypes.POINTER(_sz), _P]
    lib.mla_extend_run.argtypes = lib.mla_decode_run.argtypes
    lib.mla_extend_schedule.argtypes = [_P, _P, _P, _i32, _i32, _i32, ctypes.c_int, _i32, _P, _i32,
                                        _P, _i32, _P, ctypes.POINTER(_sz)]
    lib.kv_store_fp8.argtypes = [_P, _P, _P, _i64, _f32, _P, _i64, _P, _i64, _i64, _P]
    lib.kv_proj_store_fp8.argtypes = [_P, _i64, _P, _i64, _i64, _i32, _P, _f32, _P, _i64, _P, _i64,
                                      _i64, _P, _P]
    lib.kv_gather_cast.argtypes = [_P, _i64, _P, _i64, _i64, _P, _i64, _i32, _f32, _P, _P, _P]
    lib.kv_store_fp4.argtypes = lib.kv_store_fp8.argtypes
    lib.kv_gather_fp4.argtypes = [_P, _i64, _P, _i64, _i64, _P, _i64, _i32, _P, _i64, _P, _i64, _P]
    lib.mla_norm_rope_store.argtypes = [_P, _i64, _i64, _P, _i64, _i64, _P, _i64, _P, _P, _P, _P, _f32,
                                        _P, _P, _i64, _i32, _i64, _i32, _P, _i64, _i64, _P, _P, _f32,
                                        ctypes.c_int, _P, _i64, _P, _i64, _i64, _P]
    lib.kv_tables_update.argtypes = [_P, _P, _i32, _i32, _P, _i64, _i32, _P, _i32, _P, _P, _P, _P, _i64,
                                     _P, _P, _P, _i64, _P]
    lib.mla_get_last_error.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
    lib.mla_debug_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    for name in ("mla_decode_plan", "mla_decode_run", "mla_decode_plan_destroy",
                 "mla_decode_plan_info", "mla_decode_schedule", "kv_store_fp8", "kv_gather_cast",
                 "mla_get_last_error", "mla_decode_run_static_scratch", "mla_extend_plan",
                 "mla_extend_run", "mla_extend_schedule", "kv_proj_store_fp8",
                 "mla_debug_set_wait_limit", "kv_store_fp4", "kv_gather_fp4",
                 "mla_norm_rope_store", "kv_tables_update"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def exported_symbols() -> list[str]:
    """Names of the C entry points declared in include/mla_decode.h that the
    loaded library resolves."""
    lib = library()
    names = []
    for n in ("mla_decode_plan", "mla_decode_run", "mla_decode_plan_destroy",
              "mla_decode_plan_info", "mla_decode_schedule", "kv_store_fp8", "kv_gather_cast",
              "mla_get_last_error", "mla_status_string", "mla_decode_run_static_scratch",
              "mla_extend_plan", "mla_extend_run", "mla_extend_schedule", "kv_proj_store_fp8",
              "mla_debug_set_wait_limit", "kv_store_fp4", "kv_gather_fp4", "mla_norm_rope_store",
              "kv_tables_update"):
        getattr(lib, n)
        names.append(n)
    return names


def _check(status: int, where: str):
    if status != 0:
        raise MLAError(status, where)


def _stream(stream, dev=None):
    """The handle of a stream; of the current one (of device dev, the current
    device) where it is None."""
    if stream is None:
        import torch
        # the current stream's handle without a Stream object around it (0.1 against 3.2 us of host time)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _host_i32(a) -> np.ndarray:
    if hasattr(a, "detach"):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.int32)


def _dptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _row_stride_bytes(t) -> int:
    return t.stride(0) * t.element_size()


def _refuse(where: str, name: str, t, dtype, shape, dev: int):
    if t.dtype is not dtype:
        raise TypeError(f"{where}: {name} has dtype {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} is not on the current CUDA device")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{where}: {name} has strides {t.stride()}")


def _tensor(where: str, name: str, t, dtype, shape, dev: int) -> int:
    """The address of a tensor that the kernels will read as dtype[shape] with
    a contiguous last dimension, on the current device; anything else is
    refused here, where the library sees only a pointer."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or (
            not t.is_contiguous() and shape[-1] > 1 and t.stride(-1) != 1):
        _refuse(where, name, t, dtype, shape, dev)
    return t.data_ptr()


def _flat(where: str, name: str, t, dtype, shape, dev: int) -> int:
    """_tensor for arguments that have to be contiguous as a whole."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(where, name, t, dtype, shape, dev)
    return t.data_ptr()


def _pool(where: str, name: str, t, row_bytes: int, slots: int, dev: int):
    """(address, row stride in bytes) of byte rows [>= slots, >= row_bytes]."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or t.element_size() != 1 or t.get_device() != dev or shape[1] < row_bytes or (
            shape[0] < slots or strides[1] != 1):
        raise ValueError(f"{where}: {name} is not {slots} or more rows of {row_bytes} or more bytes on the "
                         f"current CUDA device (dtype {t.dtype}, shape {tuple(shape)}, strides {strides})")
    return t.data_ptr(), strides[0]


def _device(where: str, t) -> int:
    """The device of a tensor, which has to be the current one."""
    dev = t.get_device()
    if dev >= 0:
        import torch
        if dev == torch.cuda.current_device():
            return dev
    raise ValueError(f"{where}: a tensor is not on the current CUDA device")


def _check_pools(where: str, plan, ckv_pool, kpe_pool, slots: int):
    """Refuses pools that cannot be of the plan's type: rows narrower than the
    kernels read (a 4-bit pool on another plan), and on a 4-bit plan typed
    8-bit or wider elements, fewer rows than slots, another device.  (Strides
    are checked by the library.  Byte pools as such do not tell whether they
    hold E4M3 or 4-bit rows.)  Returns the device where it was looked up."""
    if plan.kv_dtype != MLA_KV_FP4_E2M1:
        if ckv_pool.size(-1) < D_CKV or kpe_pool.size(-1) < D_KPE:
            raise ValueError(f"{where}: pool rows of {ckv_pool.size(-1)} and {kpe_pool.size(-1)} channels, "
                             f"not {D_CKV} and {D_KPE} (a 4-bit pool needs a 4-bit plan)")
        return None
    if ckv_pool.element_size() != 1 or kpe_pool.element_size() != 1 or (
            ckv_pool.is_floating_point() or kpe_pool.is_floating_point()):
        raise TypeError(f"{where}: pools of dtypes {ckv_pool.dtype} and {kpe_pool.dtype}; a 4-bit plan reads byte rows")
    dev = _device(where, ckv_pool)
    (n, width), (n_pe, width_pe) = ckv_pool.shape, kpe_pool.shape
    if n < slots or n_pe < slots or width < FP4_CKV_BYTES <= ckv_pool.stride(0) or (
            width_pe < FP4_KPE_BYTES <= kpe_pool.stride(0)) or kpe_pool.get_device() != dev:
        raise ValueError(f"{where}: pools are not {slots} or more rows of {FP4_CKV_BYTES} and {FP4_KPE_BYTES} or more bytes "
                         f"on one device (shapes {(n, width)}, {(n_pe, width_pe)})")
    return dev


class Plan:
    """Owns a plan handle; destroyed explicitly or when garbage collected."""

    def __init__(self):
        self.handle = _P(None)
        self.workspace_bytes = 0
        self.kv_dtype = MLA_KV_FP8_E4M3      # what its pools hold

    def __del__(self):
        try:
            if self.handle and self.handle.value and _lib is not None:
                _lib.mla_decode_plan_destroy(self.handle)
                self.handle = _P(None)
        except Exception:
            pass


def mla_decode_plan(kv_indptr_host, seq_lens_host, batch: int, num_heads: int, page_size: int,
                    kv_dtype: int = MLA_KV_FP8_E4M3, stream=None, plan: Plan | None = None) -> Plan:
    """Build (or rebuild in place) a plan; returns it with .workspace_bytes."""
    lib = library()
    indptr, lens = _host_i32(kv_indptr_host), _host_i32(seq_lens_host)
    plan = plan if plan is not None else Plan()
    ws = _sz(0)
    _check(lib.mla_decode_plan(ctypes.byref(plan.handle), indptr.ctypes.data, lens.ctypes.data,
                               batch, num_heads, page_size, kv_dtype, ctypes.byref(ws),
                               _stream(stream)), "mla_decode_plan")
    plan.workspace_bytes = ws.value
    plan.kv_dtype = kv_dtype
    plan._keep = (indptr, lens)          # host arrays live until the upload is done
    return plan


def mla_decode_run(plan: Plan, q, ckv_pool, kpe_pool, num_pool_slots: int, kv_indptr_dev,
                   kv_indices_dev, seq_lens_dev, k_scale: float, softmax_scale: float, out, lse,
                   workspace=None, stream=None):
    """q: bf16 [B, H, 576] (any strides with contiguous last dim); pools:
    uint8 / float8 (FP8 plans), bf16 (BF16 plans) or uint8 (4-bit plans) with
    rows along dim 0, at least 512 and 64 channels wide (4-bit plans:
    FP4_CKV_BYTES and FP4_KPE_BYTES bytes);
    out: bf16 [B, H, 512]; lse: fp32 [B, H]; workspace: >= plan.workspace_bytes."""
    lib = library()
    dev = _check_pools("mla_decode_run", plan, ckv_pool, kpe_pool, num_pool_slots)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.mla_decode_run(plan.handle, q.data_ptr(), q.stride(0), q.stride(1),
                              ckv_pool.data_ptr(), _row_stride_bytes(ckv_pool),
                              kpe_pool.data_ptr(), _row_stride_bytes(kpe_pool), num_pool_slots,
                              kv_indptr_dev.data_ptr(), _dptr(kv_indices_dev),
                              seq_lens_dev.data_ptr(), k_scale, softmax_scale, out.data_ptr(),
                              lse.data_ptr(), _dptr(workspace), ws_bytes, _stream(stream, dev)),
           "mla_decode_run")


def mla_decode_run_static_scratch(plan: Plan, q, ckv_pool, kpe_pool, num_pool_slots: int,
                                  kv_indptr_dev, kv_indices_dev, seq_lens_dev, k_scale: float,
                                  softmax_scale: float, out, lse, stream=None):
    """mla_decode_run without a workspace argument, for callers that cannot
    allocate device memory: the split-KV partials go to a fixed array inside
    the library (STATIC_SCRATCH_BYTES per GPU, kept until exit).  Calls that
    overlap on the GPU share that array and race; calls on one stream are
    ordered.  Raises MLAError (status 3) if the plan needs more scratch."""
    dev = _check_pools("mla_decode_run_static_scratch", plan, ckv_pool, kpe_pool, num_pool_slots)
    _check(library().mla_decode_run_static_scratch(
        plan.handle, q.data_ptr(), q.stride(0), q.stride(1), ckv_pool.data_ptr(),
        _row_stride_bytes(ckv_pool), kpe_pool.data_ptr(), _row_stride_bytes(kpe_pool),
        num_pool_slots, kv_indptr_dev.data_ptr(), _dptr(kv_indices_dev),
        seq_lens_dev.data_ptr(), k_scale, softmax_scale, out.data_ptr(), lse.data_ptr(),
        _stream(stream, dev)), "mla_decode_run_static_scratch")


def mla_decode_plan_destroy(plan: Plan):
    if plan.handle and plan.handle.value:
        _check(library().mla_decode_plan_destroy(plan.handle), "mla_decode_plan_destroy")
        plan.handle = _P(None)


def mla_decode_plan_info(plan: Plan) -> dict:
    c, s, p, w = _i32(), _i32(), _i32(), _sz()
    _check(library().mla_decode_plan_info(plan.handle, ctypes.byref(c), ctypes.byref(s),
                                          ctypes.byref(p), ctypes.byref(w)), "mla_decode_plan_info")
    return dict(num_ctas=c.value, num_segments=s.value, num_partials=p.value,
                workspace_bytes=w.value)


def mla_decode_schedule(kv_indptr_host, seq_lens_host, batch: int, num_heads: int,
                        page_size: int, kv_dtype: int = MLA_KV_FP8_E4M3, num_sms: int = 152):
    """Host-only schedule: returns (segments int32 [n, 5] = cta, request, t0,
    t1, partial; info dict with kernel 0 = mma.sync, 1 = tcgen05).  Raises
    MLAError on invalid input."""
    lib = library()
    indptr, lens = _host_i32(kv_indptr_host), _host_i32(seq_lens_host)
    n, p, c, t, k, w = _i32(), _i32(), _i32(), _i32(), _i32(), _sz()
    args = (indptr.ctypes.data, lens.ctypes.data, batch, num_heads, page_size, kv_dtype, num_sms)
    outs = (ctypes.byref(n), ctypes.byref(p), ctypes.byref(c), ctypes.byref(t), ctypes.byref(k),
            ctypes.byref(w))
    _check(lib.mla_decode_schedule(*args, None, 0, *outs), "mla_decode_schedule")
    segs = np.zeros((max(n.value, 1), 5), np.int32)
    _check(lib.mla_decode_schedule(*args, segs.ctypes.data, n.value, *outs),
           "mla_decode_schedule")
    return segs[:n.value], dict(num_ctas=c.value, num_partials=p.value, tile_tokens=t.value,
                                kernel=k.value, workspace_bytes=w.value)


def mla_extend_plan(qo_indptr_host, kv_indptr_host, seq_lens_host, batch: int, num_heads: int,
                    page_size: int, kv_dtype: int = MLA_KV_FP8_E4M3, stream=None,
                    plan: Plan | None = None) -> Plan:
    """Plan causal extend attention: request b's new tokens are query rows
    qo_indptr[b] .. qo_indptr[b+1]-1 and already count in seq_lens[b]."""
    lib = library()
    qo, indptr, lens = _host_i32(qo_indptr_host), _host_i32(kv_indptr_host), _host_i32(seq_lens_host)
    plan = plan if plan is not None else Plan()
    ws = _sz(0)
    _check(lib.mla_extend_plan(ctypes.byref(plan.handle), qo.ctypes.data, indptr.ctypes.data,
                               lens.ctypes.data, batch, num_heads, page_size, kv_dtype,
                               ctypes.byref(ws), _stream(stream)), "mla_extend_plan")
    plan.workspace_bytes = ws.value
    plan.kv_dtype = kv_dtype
    plan._keep = (qo, indptr, lens)
    return plan


def mla_extend_run(plan: Plan, q, ckv_pool, kpe_pool, num_pool_slots: int, kv_indptr_dev,
                   kv_indices_dev, seq_lens_dev, k_scale: float, softmax_scale: float, out, lse,
                   workspace=None, stream=None):
    """q: bf16 [n_q, H, 576] (contiguous last dim); out: bf16 [n_q, H, 512];
    lse: fp32 [n_q, H]; the rest as mla_decode_run."""
    dev = _check_pools("mla_extend_run", plan, ckv_pool, kpe_pool, num_pool_slots)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(library().mla_extend_run(plan.handle, q.data_ptr(), q.stride(0), q.stride(1),
                                    ckv_pool.data_ptr(), _row_stride_bytes(ckv_pool),
                                    kpe_pool.data_ptr(), _row_stride_bytes(kpe_pool),
                                    num_pool_slots, kv_indptr_dev.data_ptr(),
                                    _dptr(kv_indices_dev), seq_lens_dev.data_ptr(), k_scale,
                                    softmax_scale, out.data_ptr(), lse.data_ptr(),
                                    _dptr(workspace), ws_bytes, _stream(stream, dev)),
           "mla_extend_run")


def mla_extend_schedule(qo_indptr_host, kv_indptr_host, seq_lens_host, batch: int,
                        num_heads: int, page_size: int, kv_dtype: int = MLA_KV_FP8_E4M3,
                        num_sms: int = 152):
    """Host-only extend schedule: (segments int32 [n, 5] = cta, block, t0, t1,
    partial; blocks int32 [m, 4] = request, first row, rows, causal base;
    info dict)."""
    lib = library()
    qo, indptr, lens = _host_i32(qo_indptr_host), _host_i32(kv_indptr_host), _host_i32(seq_lens_host)
    counts = np.zeros(5, np.int32)
    w = _sz()
    args = (qo.ctypes.data, indptr.ctypes.data, lens.ctypes.data, batch, num_heads, page_size,
            kv_dtype, num_sms)
    _check(lib.mla_extend_schedule(*args, None, 0, None, 0, counts.ctypes.data, ctypes.byref(w)),
           "mla_extend_schedule")
    segs = np.zeros((max(int(counts[0]), 1), 5), np.int32)
    blocks = np.zeros((max(int(counts[3]), 1), 4), np.int32)
    _check(lib.mla_extend_schedule(*args, segs.ctypes.data, int(counts[0]), blocks.ctypes.data,
                                   int(counts[3]), counts.ctypes.data, ctypes.byref(w)),
           "mla_extend_schedule")
    return segs[:counts[0]], blocks[:counts[3]], dict(
        num_segments=int(counts[0]), num_partials=int(counts[1]), num_ctas=int(counts[2]),
        num_blocks=int(counts[3]), block_rows=int(counts[4]), workspace_bytes=w.value)


def kv_store_fp8(ckv_new, kpe_new, slots, k_scale: float, ckv_pool, kpe_pool,
                 num_pool_slots: int | None = None, stream=None):
    """ckv_new bf16 [n, 512], kpe_new bf16 [n, 64] (contiguous), slots int64 [n]."""
    n = slots.shape[0]
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    _check(library().kv_store_fp8(ckv_new.data_ptr(), kpe_new.data_ptr(), slots.data_ptr(), n,
                                  k_scale, ckv_pool.data_ptr(), _row_stride_bytes(ckv_pool),
                                  kpe_pool.data_ptr(), _row_stride_bytes(kpe_pool), nps,
                                  _stream(stream)), "kv_store_fp8")


def kv_proj_store_fp8(x, w, slots, k_scale: float, ckv_pool, kpe_pool,
                      num_pool_slots: int | None = None, latent_out=None, stream=None):
    """x bf16 [n, d_model], w bf16 [576, d_model] (row j = channel j's
    weights), slots int64 [n]: latent = BF16(x @ w.T) quantized into the pool
    rows like kv_store_fp8; latent_out (optional) bf16 [n, 576] receives the
    rounded latents."""
    n, d = x.shape
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    _check(library().kv_proj_store_fp8(x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), n, d,
                                       slots.data_ptr(), k_scale, ckv_pool.data_ptr(),
                                       _row_stride_bytes(ckv_pool), kpe_pool.data_ptr(),
                                       _row_stride_bytes(kpe_pool), nps, _dptr(latent_out),
                                       _stream(stream)), "kv_proj_store_fp8")


def kv_gather_cast(ckv_pool, kpe_pool, kv_indices, page_size: int, k_scale: float, ckv_out,
                   kpe_out, num_pool_slots: int | None = None, stream=None):
    """Gather the listed pages into compact bf16 [n_pages*page_size, 512 / 64]."""
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    _check(library().kv_gather_cast(ckv_pool.data_ptr(), _row_stride_bytes(ckv_pool),
                                    kpe_pool.data_ptr(), _row_stride_bytes(kpe_pool), nps,
                                    kv_indices.data_ptr(), kv_indices.shape[0], page_size,
                                    k_scale, ckv_out.data_ptr(), kpe_out.data_ptr(),
                                    _stream(stream)), "kv_gather_cast")


def kv_store_fp4(ckv_new, kpe_new, slots, k_scale: float, ckv_pool, kpe_pool,
                 num_pool_slots: int | None = None, stream=None):
    """kv_store_fp8 for 4-bit pools: ckv_new bf16 [n, 512], kpe_new bf16
    [n, 64] (contiguous), slots int64 [n]; pools of byte rows of at least
    FP4_CKV_BYTES and FP4_KPE_BYTES, e.g. pool[:, :272] and pool[:, 272:] of a
    uint8 [slots, FP4_ROW_BYTES] pool."""
    import torch
    where, n = "kv_store_fp4", slots.shape[0]
    dev = _device(where, ckv_pool)
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    ckv, ckv_stride = _pool(where, "ckv_pool", ckv_pool, FP4_CKV_BYTES, nps, dev)
    kpe, kpe_stride = _pool(where, "kpe_pool", kpe_pool, FP4_KPE_BYTES, nps, dev)
    _check(library().kv_store_fp4(_flat(where, "ckv_new", ckv_new, torch.bfloat16, (n, D_CKV), dev),
                                  _flat(where, "kpe_new", kpe_new, torch.bfloat16, (n, D_KPE), dev),
                                  _flat(where, "slots", slots, torch.int64, (n,), dev), n, k_scale, ckv,
                                  ckv_stride, kpe, kpe_stride, nps, _stream(stream, dev)), where)


def kv_gather_fp4(ckv_pool, kpe_pool, kv_indices, page_size: int, ckv_out, kpe_out,
                  num_pool_slots: int | None = None, stream=None):
    """Widen the listed pages (int32 [n_pages]) of a 4-bit pool to E4M3 rows:
    ckv_out, kpe_out byte rows [>= n_pages*page_size, >= 512 / >= 64], e.g. an
    FP8 pool's two parts.  Exact; the pool's k_scale still applies."""
    import torch
    where, n = "kv_gather_fp4", kv_indices.shape[0]
    dev = _device(where, ckv_pool)
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    ckv, ckv_stride = _pool(where, "ckv_pool", ckv_pool, FP4_CKV_BYTES, nps, dev)
    kpe, kpe_stride = _pool(where, "kpe_pool", kpe_pool, FP4_KPE_BYTES, nps, dev)
    co, co_stride = _pool(where, "ckv_out", ckv_out, D_CKV, n * page_size, dev)
    ko, ko_stride = _pool(where, "kpe_out", kpe_out, D_KPE, n * page_size, dev)
    _check(library().kv_gather_fp4(ckv, ckv_stride, kpe, kpe_stride, nps,
                                   _flat(where, "kv_indices", kv_indices, torch.int32, (n,), dev), n, page_size,
                                   co, co_stride, ko, ko_stride, _stream(stream, dev)), where)


def mla_norm_rope_store(q_lat, q_pe, latent, positions, cos_sin, slots, eps: float, k_scale: float, ckv_pool,
                        kpe_pool, q_out, kv_dtype: int = MLA_KV_FP8_E4M3, interleaved: bool = False,
                        q_lat_weight=None, q_pe_weight=None, ckv_weight=None, kpe_weight=None,
                        latent_out=None, num_pool_slots: int | None = None, stream=None):
    """Norms and position rotation of a step's queries and latent keys, and the
    keys' cache write, in one pass.  q_lat bf16 [n, H, 512], q_pe bf16
    [n, H, 64], latent bf16 [n, 576] (any strides, contiguous last dim); the
    weights bf16 [512] / [64], None for no norm of that part; positions int32
    [n]; cos_sin fp32 [max_positions, 64]; slots int64 [n]; q_out bf16
    [n, H, 576]; latent_out bf16 [n, 576].  q_lat and q_pe may be
    q_out[..., :512] and q_out[..., 512:]."""
    import torch
    where, bf16 = "mla_norm_rope_store", torch.bfloat16
    dev = _device(where, q_out)
    n, h = q_out.shape[:2]
    fp4 = kv_dtype == MLA_KV_FP4_E2M1
    nps = ckv_pool.shape[0] if num_pool_slots is None else num_pool_slots
    ckv, ckv_stride = _pool(where, "ckv_pool", ckv_pool, FP4_CKV_BYTES if fp4 else D_CKV, nps, dev)
    kpe, kpe_stride = _pool(where, "kpe_pool", kpe_pool, FP4_KPE_BYTES if fp4 else D_KPE, nps, dev)

    def weight(name, w, width):
        return _flat(where, name, w, bf16, (width,), dev) if w is not None else 0

    ql_n, ql_h, _ = q_lat.stride()
    qp_n, qp_h, _ = q_pe.stride()
    qo_n, qo_h, _ = q_out.stride()
    _check(library().mla_norm_rope_store(
        _tensor(where, "q_lat", q_lat, bf16, (n, h, D_CKV), dev), ql_n, ql_h,
        _tensor(where, "q_pe", q_pe, bf16, (n, h, D_KPE), dev), qp_n, qp_h,
        _tensor(where, "latent", latent, bf16, (n, D_QK), dev), latent.stride(0),
        weight("q_lat_weight", q_lat_weight, D_CKV), weight("q_pe_weight", q_pe_weight, D_KPE),
        weight("ckv_weight", ckv_weight, D_CKV), weight("kpe_weight", kpe_weight, D_KPE), eps,
        _flat(where, "positions", positions, torch.int32, (n,), dev),
        _flat(where, "cos_sin", cos_sin, torch.float32, (cos_sin.shape[0], D_KPE), dev), cos_sin.shape[0],
        1 if interleaved else 0, n, h, _tensor(where, "q_out", q_out, bf16, (n, h, D_QK), dev), qo_n, qo_h,
        0 if latent_out is None else _flat(where, "latent_out", latent_out, bf16, (n, D_QK), dev),
        _flat(where, "slots", slots, torch.int64, (n,), dev), k_scale, kv_dtype, ckv, ckv_stride, kpe,
        kpe_stride, nps, _stream(stream, dev)), where)


def kv_tables_update(held_lens, wanted_lens, page_size: int, block_table, free_pages, free_state, kv_indptr,
                     kv_indices, qo_indptr=None, slots=None, positions=None, free_state_out=None,
                     stream=None):
    """Page tables of a step from the requests' lengths (int32 [batch], held
    now and wanted): takes and returns pages, updates block_table int32
    [batch, max_pages] (rows strided as they like), the ring free_pages int32
    [capacity] and free_state int32 [4] = {head, count, 0, 0} (in place, or
    into free_state_out int32 [2]); writes kv_indptr int32 [batch + 1],
    kv_indices int32 [capacity] and, where given, qo_indptr int32 [batch + 1],
    slots int64 [capacity] and positions int32 [capacity].  A step that does
    not fit is refused on the device as a whole (FLAG_TABLES_REFUSED)."""
    import torch
    where, i32 = "kv_tables_update", torch.int32
    dev = _device(where, block_table)
    batch, pages = block_table.shape
    tokens = min(t.shape[0] for t in (slots, positions) if t is not None) if (
        slots is not None or positions is not None) else 0
    out = free_state if free_state_out is None else free_state_out
    _check(library().kv_tables_update(
        _flat(where, "held_lens", held_lens, i32, (batch,), dev),
        _flat(where, "wanted_lens", wanted_lens, i32, (batch,), dev), batch, page_size,
        _tensor(where, "block_table", block_table, i32, (batch, pages), dev), block_table.stride(0), pages,
        _flat(where, "free_pages", free_pages, i32, (free_pages.shape[0],), dev), free_pages.shape[0],
        _flat(where, "free_state", free_state, i32, (4,), dev),
        _flat(where, "free_state_out", out, i32, (4,) if out is free_state else (2,), dev),
        _flat(where, "kv_indptr", kv_indptr, i32, (batch + 1,), dev),
        _flat(where, "kv_indices", kv_indices, i32, (kv_indices.shape[0],), dev), kv_indices.shape[0],
        0 if qo_indptr is None else _flat(where, "qo_indptr", qo_indptr, i32, (batch + 1,), dev),
        0 if slots is None else _flat(where, "slots", slots, torch.int64, (slots.shape[0],), dev),
        0 if positions is None else _flat(where, "positions", positions, i32, (positions.shape[0],), dev),
        tokens, _stream(stream, dev)), where)


def mla_get_last_error(stream=None) -> int:
    """Synchronise the stream; return and clear the device flag word."""
    flags = ctypes.c_uint32(0)
    st = library().mla_get_last_error(_stream(stream), ctypes.byref(flags))
    if st not in (0, 4):
        raise MLAError(st, "mla_get_last_error")
    return flags.value


def mla_debug_set_wait_limit(limit_ns: int):
    """Time limit (ns) of the decode kernels' bounded in-kernel waits on the
    current device; 0 restores the default (2 s).  A test hook: a tiny limit
    makes the next decode calls give up and set FLAG_WAIT_TIMEOUT."""
    _check(library().mla_debug_set_wait_limit(ctypes.c_uint64(int(limit_ns))),
           "mla_debug_set_wait_limit")
