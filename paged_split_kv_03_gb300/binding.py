"""Thin ctypes binding of the C ABI in include/pda.h (argument marshalling only).

The names mirror the C entry points: ``pda_plan``, ``pda_decode``,
``pda_get_status``, ``pda_reset_status``, ``pda_strerror``. Tensors are
passed as raw pointers (``data_ptr()``) and streams as their CUDA handle;
every step of the computation runs in the library's kernels. There is no
fallback: if ``_lib/libpda.so`` has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libpda.so")

PDA_BF16, PDA_E4M3, PDA_INT8 = 0, 1, 2
PDA_SCALE_MLA_BLOCK = 3
PDA_SCALE_NONE, PDA_SCALE_TENSOR, PDA_SCALE_TOKEN_HEAD = 0, 1, 2
PDA_KERNEL_AUTO, PDA_KERNEL_MMA, PDA_KERNEL_TC = 0, 1, 2
PDA_OK = 0
PDA_ERR_NULL, PDA_ERR_INVALID, PDA_ERR_UNSUPPORTED = -1, -2, -3
PDA_ERR_ALIGNMENT, PDA_ERR_SCRATCH, PDA_ERR_CUDA, PDA_ERR_PLAN = -4, -5, -6, -7
PDA_ERR_TOO_LARGE = -8
PDA_STATIC_SCRATCH_BYTES = 32 << 20
PDA_STATUS_KV_LEN_LT_ROWS = 0x1
PDA_STATUS_ROWS_GT_MAX = 0x2
PDA_STATUS_KV_LEN_GT_MAX = 0x4
PDA_STATUS_PAGE_OOB = 0x8
PDA_STATUS_ROWS_GT_CAP = 0x10
PDA_STATUS_WAIT_TIMEOUT = 0x20
PDA_STATUS_SMEM_MISALIGNED = 0x40
PDA_STATUS_TABLE_INVALID = 0x80
PDA_STATUS_NO_PAGES = 0x100
PDA_STATUS_TABLE_FULL = 0x200
PDA_STATUS_TOKENS_GT_CAP = 0x400
PDA_PLAN_MAGIC = 0x50444131
PDA_PREFILL_MAGIC = 0x50444631
PDA_INJECT_WITHHOLD_KV = 0x1
PDA_INJECT_WITHHOLD_CTA0 = 0x2
PDA_INJECT_WITHHOLD_CTA1 = 0x4

# every entry point include/pda.h declares
EXPORTED = ("pda_plan", "pda_decode", "pda_decode_stages", "pda_decode_static", "pda_append_kv",
            "pda_build_tables", "pda_append_slots", "pda_mla_absorb", "pda_mla_project",
            "pda_mla_expand", "pda_prefill_plan", "pda_mla_prefill", "pda_get_status", "pda_reset_status", "pda_strerror", "pda_version",
            "pda_struct_sizes")

_i32, _i64, _u32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p


class PdaParams(ctypes.Structure):
    _fields_ = [("num_qo_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("page_size", _i32), ("q_dtype", _i32), ("kv_dtype", _i32),
                ("scale_mode", _i32), ("max_batch", _i32), ("max_q_len", _i32),
                ("max_kv_len", _i32), ("num_pages", _i32), ("kv_stride_page", _i64),
                ("kv_stride_token", _i64), ("kv_stride_head", _i64), ("device", _i32),
                ("num_sms", _i32), ("host_kv_len", ctypes.POINTER(_i32)), ("batch", _i32),
                ("chunk_pages", _i32), ("kernel", _i32), ("head_dim_v", _i32),
                ("wait_limit_us", _i32), ("inject", _u32),
                ("host_qo_indptr", ctypes.POINTER(_i32)), ("host_window", ctypes.POINTER(_i32))]


class PdaPlan(ctypes.Structure):
    _fields_ = [("magic", _u32), ("num_qo_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("page_size", _i32), ("q_dtype", _i32), ("kv_dtype", _i32),
                ("scale_mode", _i32), ("max_batch", _i32), ("max_q_len", _i32),
                ("max_kv_len", _i32), ("num_pages", _i32), ("batch", _i32),
                ("kv_stride_page", _i64), ("kv_stride_token", _i64), ("kv_stride_head", _i64),
                ("group", _i32), ("kernel", _i32), ("rows_per_cta", _i32),
                ("heads_per_cta", _i32 * 9), ("head_blocks", _i32), ("chunk_pages", _i32),
                ("max_splits", _i32), ("num_sms", _i32), ("grid_ctas", _i64),
                ("rows_cap", _i64), ("scratch_bytes", _i64), ("scratch_lse_offset", _i64),
                ("scratch_o_offset", _i64), ("stage1_smem_bytes", _i32),
                ("tail_from", _i32), ("tail_chunk_pages", _i32), ("head_splits", _i32),
                ("tail_splits", _i32), ("head_dim_v", _i32), ("device", _i32),
                ("wait_limit_us", _i32), ("inject", _u32), ("reserved", _i32 * 7)]


class PdaTables(ctypes.Structure):
    _fields_ = [("cached_len", _vp), ("new_len", _vp), ("request", _vp), ("block_table", _vp),
                ("table_stride", _i64), ("free_pages", _vp), ("free_count", _vp),
                ("free_left", _vp), ("kv_len", _vp), ("kv_indptr", _vp), ("page_table", _vp),
                ("qo_indptr", _vp), ("tok_indptr", _vp), ("slot_map", _vp), ("positions", _vp),
                ("table_rows", _i32), ("table_cols", _i32), ("page_table_cap", _i32),
                ("rows_cap", _i32)]


class PdaPrefillPlan(ctypes.Structure):
    _fields_ = [("magic", _u32), ("struct_bytes", _u32), ("num_qo_heads", _i32), ("batch", _i32),
                ("max_kv_len", _i32), ("num_sms", _i32), ("device", _i32), ("rows", _i32),
                ("tokens", _i32), ("tiles", _i32), ("splits", _i32), ("chunk_tokens", _i32),
                ("wait_limit_us", _i32), ("inject", _u32), ("reserved", _i32 * 2),
                ("scratch_bytes", _i64)]


class PdaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where} failed: {pda_strerror(code)} ({code})")


_LIB = None


def load_library(path: Optional[str] = None):
    """Load libpda.so (built by paged_split_kv_03_gb300.build); raises if absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with paged_split_kv_03_gb300.build.build() "
                           "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    lib.pda_plan.argtypes = [ctypes.POINTER(PdaParams), ctypes.POINTER(PdaPlan),
                             ctypes.POINTER(ctypes.c_size_t)]
    lib.pda_plan.restype = ctypes.c_int
    lib.pda_decode.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _i32, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.pda_decode.restype = ctypes.c_int
    lib.pda_decode_stages.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i32, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _u32,
                                      _vp]
    lib.pda_decode_stages.restype = ctypes.c_int
    lib.pda_decode_static.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _i32, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp]
    lib.pda_decode_static.restype = ctypes.c_int
    lib.pda_append_kv.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                  _vp, _vp, _vp, _vp, _vp, _vp]
    lib.pda_append_kv.restype = ctypes.c_int
    lib.pda_build_tables.argtypes = [ctypes.POINTER(PdaPlan), ctypes.POINTER(PdaTables), _vp, _vp]
    lib.pda_build_tables.restype = ctypes.c_int
    lib.pda_append_slots.argtypes = [ctypes.POINTER(PdaPlan), _vp, _i64, _vp, _i64, _vp, _i32, _vp,
                                     _vp, _vp, _vp, _vp, _vp, _vp]
    lib.pda_append_slots.restype = ctypes.c_int
    lib.pda_mla_absorb.argtypes = [ctypes.POINTER(PdaPlan), _vp, _i64, _i64, _vp, _i64,
                                   ctypes.c_float, _vp, _i32, _vp, _vp, _vp]
    lib.pda_mla_absorb.restype = ctypes.c_int
    lib.pda_mla_project.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _i64, _vp, _i32, _vp, _vp,
                                    _vp]
    lib.pda_mla_project.restype = ctypes.c_int
    lib.pda_mla_expand.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                   _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp]
    lib.pda_mla_expand.restype = ctypes.c_int
    lib.pda_prefill_plan.argtypes = [ctypes.POINTER(PdaPlan), _i32, _i32,
                                     ctypes.POINTER(PdaPrefillPlan),
                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.pda_prefill_plan.restype = ctypes.c_int
    lib.pda_mla_prefill.argtypes = [ctypes.POINTER(PdaPrefillPlan), _vp, _i64, _i64, _vp, _vp, _i64,
                                    _i64, _vp, _i64, _vp, _vp, _vp, _i32, ctypes.c_float, _vp, _vp,
                                    _vp, _vp]
    lib.pda_mla_prefill.restype = ctypes.c_int
    lib.pda_get_status.argtypes = [ctypes.POINTER(PdaPlan), _vp, ctypes.POINTER(_u32), _vp]
    lib.pda_get_status.restype = ctypes.c_int
    lib.pda_reset_status.argtypes = [ctypes.POINTER(PdaPlan), _vp, _vp]
    lib.pda_reset_status.restype = ctypes.c_int
    lib.pda_strerror.argtypes = [ctypes.c_int]
    lib.pda_strerror.restype = ctypes.c_char_p
    lib.pda_version.restype = ctypes.c_int
    lib.pda_struct_sizes.argtypes = [ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.pda_struct_sizes.restype = ctypes.c_int
    if path is None:
        _LIB = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_RAW_STREAM = None


def _stream(stream, dev=None) -> Optional[int]:
    """The raw handle of a stream; None: the current one (of ``dev``, where it is known that
    tensors of that device exist)."""
    if stream is None:
        global _RAW_STREAM
        if _RAW_STREAM is None:
            # the handle alone: a torch Stream object costs ten times as much
            from torch._C import _cuda_getCurrentRawStream
            from torch.cuda import current_device
            _RAW_STREAM = _cuda_getCurrentRawStream, current_device
        return _RAW_STREAM[0](_RAW_STREAM[1]() if dev is None else dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def pda_strerror(code: int) -> str:
    return load_library().pda_strerror(int(code)).decode()


def pda_plan(params: PdaParams, check: bool = True):
    """-> (PdaPlan, scratch_bytes, rc)."""
    plan = PdaPlan()
    nbytes = ctypes.c_size_t(0)
    rc = load_library().pda_plan(ctypes.byref(params), ctypes.byref(plan), ctypes.byref(nbytes))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_plan")
    return plan, int(nbytes.value), rc


def pda_decode(plan: PdaPlan, q, k_pages, v_pages, page_table, kv_indptr, kv_len, qo_indptr,
               max_q_len: int, window, sm_scale: float, k_scale, v_scale, out, lse,
               split_scratch, stream=None, check: bool = True) -> int:
    rc = load_library().pda_decode(
        ctypes.byref(plan), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
        _ptr(kv_indptr), _ptr(kv_len), _ptr(qo_indptr), int(max_q_len), _ptr(window),
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(split_scratch),
        _stream(stream))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_decode")
    return rc


PDA_STAGE_PARTIAL, PDA_STAGE_MERGE = 1, 2


def pda_decode_stages(plan: PdaPlan, q, k_pages, v_pages, page_table, kv_indptr, kv_len,
                      qo_indptr, max_q_len: int, window, sm_scale: float, k_scale, v_scale, out,
                      lse, split_scratch, stages: int, stream=None, check: bool = True) -> int:
    """pda_decode's stage 1 (PDA_STAGE_PARTIAL) and / or merge (PDA_STAGE_MERGE)."""
    rc = load_library().pda_decode_stages(
        ctypes.byref(plan), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
        _ptr(kv_indptr), _ptr(kv_len), _ptr(qo_indptr), int(max_q_len), _ptr(window),
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(split_scratch),
        int(stages), _stream(stream))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_decode_stages")
    return rc


def pda_decode_static(plan: PdaPlan, q, k_pages, v_pages, page_table, kv_indptr, kv_len,
                      qo_indptr, max_q_len: int, window, sm_scale: float, k_scale, v_scale, out,
                      lse, stream=None, check: bool = True) -> int:
    """pda_decode for callers that cannot allocate device memory: the split
    scratch is the library's own fixed array (PDA_STATIC_SCRATCH_BYTES), so
    nothing is allocated. Calls share that array: do not overlap them."""
    rc = load_library().pda_decode_static(
        ctypes.byref(plan), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
        _ptr(kv_indptr), _ptr(kv_len), _ptr(qo_indptr), int(max_q_len), _ptr(window),
        float(sm_scale), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _stream(stream))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_decode_static")
    return rc


def pda_append_kv(plan: PdaPlan, k_new, v_new, page_table, kv_indptr, kv_len, qo_indptr,
                  max_q_len: int, k_pages, v_pages, k_scale, v_scale, split_scratch,
                  stream=None, check: bool = True) -> int:
    """Quantise-on-append of the new rows' K/V (bf16 [rows, Hkv, D]) into the
    paged cache of the plan's dtype and scale mode (see include/pda.h)."""
    rc = load_library().pda_append_kv(
        ctypes.byref(plan), _ptr(k_new), _ptr(v_new), _ptr(page_table), _ptr(kv_indptr),
        _ptr(kv_len), _ptr(qo_indptr), int(max_q_len), _ptr(k_pages), _ptr(v_pages),
        _ptr(k_scale), _ptr(v_scale), _ptr(split_scratch), _stream(stream))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_append_kv")
    return rc


def _types():
    """(bfloat16, int32, int64, float32, float8_e4m3fn, uint8) of torch, looked up once."""
    global _TYPES, _INT8
    if _TYPES is None:
        import torch
        _INT8 = torch.int8
        _TYPES = (torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.float8_e4m3fn,
                  torch.uint8)
    return _TYPES


_TYPES = _INT8 = None


def _chk(where: str, name: str, t, dev: int, dtype, shape, tail=None) -> None:
    """The device, type, sizes and strides that a call with raw pointers assumes and the library
    cannot see: ``tail`` are the strides of the last dimensions (None: contiguous)."""
    if (t.dtype is dtype and t.get_device() == dev and t.shape == shape and
            (t.is_contiguous() if tail is None else t.stride()[-len(tail):] == tail)):
        return
    if t.dtype is not dtype:
        raise ValueError(f"{where}: {name} is {t.dtype}, not {dtype}")
    _chk_device(where, name, t, dev)
    if t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    got = t.stride()
    for d in range(-1, -1 - len(tail or ()), -1):  # a dimension of one has any stride
        if t.shape[d] > 1 and got[d] != tail[d]:
            raise ValueError(f"{where}: {name} has strides {got}, its last ones not {tail}")
    if tail is None:
        raise ValueError(f"{where}: {name} is not contiguous")


def _chk_device(where: str, name: str, t, dev: int) -> None:
    got = t.get_device()
    if got == dev:
        return
    if got < 0:
        raise ValueError(f"{where}: {name} is not on a CUDA device")
    raise PdaError(PDA_ERR_INVALID, f"{where}: {name} is on cuda:{got}, the plan on cuda:{dev};")


def _room(t) -> int:
    """Bytes from a tensor's first element to the end of its memory."""
    return t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()


def _scratch(where: str, t, dev: int, need: int):
    """Address of a scratch; a tensor has to be on the plan's device, with ``need`` bytes."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev or t.nbytes < need:
        _chk_device(where, "the scratch", t, dev)
        if _room(t) < need:
            raise PdaError(PDA_ERR_SCRATCH, f"{where}: {_room(t)} bytes of scratch, not {need};")
    return t.data_ptr()


def _cache_needs(plan: PdaPlan):
    """(device, types of the cache, its bytes, values of its scales), kept with the plan."""
    bf16, _, _, _, e4m3, u8 = _types()
    kv, mode = plan.kv_dtype, plan.scale_mode
    typed = bf16 if kv == PDA_BF16 else e4m3 if kv == PDA_E4M3 else _INT8
    width = 640 if mode == PDA_SCALE_MLA_BLOCK else plan.head_dim
    nbytes = ((plan.num_pages - 1) * plan.kv_stride_page +
              (plan.page_size - 1) * plan.kv_stride_token +
              (plan.num_kv_heads - 1) * plan.kv_stride_head + width) * (2 if kv == PDA_BF16 else 1)
    values = 0 if mode == PDA_SCALE_NONE else 1 if mode == PDA_SCALE_TENSOR else \
        plan.num_pages * plan.page_size * plan.num_kv_heads * (4 if mode == PDA_SCALE_MLA_BLOCK else 1)
    plan.cache_needs = plan.device, (typed, u8, _INT8), nbytes, values
    return plan.cache_needs


def _cache(where: str, side: str, pages, scale, plan: PdaPlan):
    """Addresses of the cache and its scales; tensors have to be on the plan's device, of its
    type (the cache: or raw bytes, uint8 or int8), and large enough for its pages and strides."""
    try:
        dev, types, need, values = plan.cache_needs
    except AttributeError:
        dev, types, need, values = _cache_needs(plan)
    if pages is not None and not isinstance(pages, int):
        if not (pages.dtype in types and pages.get_device() == dev and pages.nbytes >= need and
                pages.is_contiguous()):
            if pages.dtype not in types:
                raise ValueError(f"{where}: {side}_pages is {pages.dtype}, not {types[0]} or bytes")
            _chk_device(where, side + "_pages", pages, dev)
            if _room(pages) < need:
                raise ValueError(
                    f"{where}: {side}_pages has {_room(pages)} bytes, the plan's pages {need}")
        pages = pages.data_ptr()
    if scale is not None and not isinstance(scale, int):
        if values and not (scale.dtype is _TYPES[3] and scale.get_device() == dev and
                           scale.numel() >= values and scale.is_contiguous()):
            _chk_device(where, side + "_scale", scale, dev)
            raise ValueError(f"{where}: {side}_scale has to hold {values} contiguous float32")
        scale = scale.data_ptr()
    return pages, scale


def pda_build_tables(plan: PdaPlan, cached_len, new_len, request, block_table, free_pages,
                     free_count, free_left, kv_len, kv_indptr, page_table, qo_indptr, tok_indptr,
                     slot_map, positions, split_scratch, stream=None, check: bool = True) -> int:
    """Block tables and slot maps of one step from the request lengths, on the GPU (see
    include/pda.h). ``block_table`` is [rows, cols] int32, ``slot_map`` int64, the others int32;
    ``request``, ``tok_indptr``, ``slot_map`` and ``positions`` may be None."""
    _, i32, i64, _, _, _ = _TYPES or _types()
    where, n, dev = "pda_build_tables", plan.batch, plan.device
    per, ptrs, one = (n,), (n + 1,), (1,)
    _chk(where, "cached_len", cached_len, dev, i32, per)
    _chk(where, "new_len", new_len, dev, i32, per)
    _chk(where, "kv_len", kv_len, dev, i32, per)
    _chk(where, "kv_indptr", kv_indptr, dev, i32, ptrs)
    _chk(where, "qo_indptr", qo_indptr, dev, i32, ptrs)
    _chk(where, "free_count", free_count, dev, i32, one)
    _chk(where, "free_left", free_left, dev, i32, one)
    _chk(where, "free_pages", free_pages, dev, i32, (free_pages.numel(),))
    _chk(where, "page_table", page_table, dev, i32, (page_table.numel(),))
    rows, cols = block_table.shape
    _chk(where, "block_table", block_table, dev, i32, (rows, cols), (1,))
    cap = 0x7fffffff
    if request is not None:
        _chk(where, "request", request, dev, i32, per)
        request = request.data_ptr()
    if tok_indptr is not None:
        _chk(where, "tok_indptr", tok_indptr, dev, i32, ptrs)
        tok_indptr = tok_indptr.data_ptr()
    if slot_map is not None:
        cap = slot_map.numel()
        _chk(where, "slot_map", slot_map, dev, i64, (cap,))
        slot_map = slot_map.data_ptr()
    if positions is not None:
        _chk(where, "positions", positions, dev, i32, (positions.numel(),))
        cap = min(cap, positions.numel())
        positions = positions.data_ptr()
    split_scratch = _scratch(where, split_scratch, dev, 4)
    t = PdaTables(cached_len.data_ptr(), new_len.data_ptr(), request, block_table.data_ptr(),
                  block_table.stride(0) if rows > 1 else cols,
                  # (an empty list has no address: any will do, none of it is read)
                  free_pages.data_ptr() or free_count.data_ptr(),
                  free_count.data_ptr(), free_left.data_ptr(), kv_len.data_ptr(),
                  kv_indptr.data_ptr(), page_table.data_ptr(), qo_indptr.data_ptr(), tok_indptr,
                  slot_map, positions, rows, cols, page_table.numel(), cap)
    rc = (_LIB or load_library()).pda_build_tables(ctypes.byref(plan), ctypes.byref(t), split_scratch,
                                         _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def _num_rows(where: str, t, dev: int):
    """Address of a one-element int32 device tensor, or None."""
    if t is None:
        return None
    _chk(where, "num_rows", t, dev, _TYPES[1], (1,))
    return t.data_ptr()


def pda_append_slots(plan: PdaPlan, k_new, v_new, slot_map, num_rows, k_pages, v_pages, k_scale,
                     v_scale, split_scratch, stream=None, check: bool = True) -> int:
    """Append rows (bf16 [rows, Hkv, D], any row stride) through a slot map (int64 [rows]);
    ``num_rows``: an int32 device tensor of one element bounding the rows, or None."""
    bf16, _, i64, _, _, _ = _TYPES or _types()
    where, dev = "pda_append_slots", plan.device
    rows, d = slot_map.numel(), plan.head_dim
    new, tail = (rows, plan.num_kv_heads, d), (d, 1)
    _chk(where, "k_new", k_new, dev, bf16, new, tail)
    _chk(where, "slot_map", slot_map, dev, i64, (rows,))
    if v_new is not None:
        _chk(where, "v_new", v_new, dev, bf16, new, tail)
    k_pages, k_scale = _cache(where, "k", k_pages, k_scale, plan)
    if d != 576:
        v_pages, v_scale = _cache(where, "v", v_pages, v_scale, plan)
    else:  # one latent: no v
        v_pages = v_scale = None
    split_scratch = _scratch(where, split_scratch, dev, 4)
    rc = (_LIB or load_library()).pda_append_slots(
        ctypes.byref(plan), k_new.data_ptr(), _row_stride(k_new), _ptr(v_new),
        0 if v_new is None else _row_stride(v_new), slot_map.data_ptr(), rows,
        _num_rows(where, num_rows, dev), k_pages, v_pages, k_scale, v_scale,
        split_scratch, _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def _row_stride(x) -> int:
    """Elements between rows; a lone row's stride has no meaning in torch."""
    if x.shape[0] > 1:
        return x.stride(0)
    n = 1
    for s in x.shape[1:]:
        n *= s
    return n


def _head_strides(x):
    """(row, head) strides in elements of [rows, heads, channels]."""
    row, head, _ = x.stride()
    if x.shape[1] == 1:
        head = x.shape[2]
    return (row if x.shape[0] > 1 else x.shape[1] * head), head


def pda_mla_absorb(plan: PdaPlan, q, w_uk, q_scale: float, q_lat, num_rows, split_scratch,
                   stream=None, check: bool = True) -> int:
    """The query absorbed into the latent space: q bf16 [rows, Hq, 192], w_uk bf16
    [Hq, 128, 512] (any head stride), q_lat [rows, Hq, 576] bf16 or E4M3 codes."""
    bf16, _, _, _, e4m3, u8 = _TYPES or _types()
    where, dev = "pda_mla_absorb", plan.device
    rows, h = q.shape[0], plan.num_qo_heads
    _chk(where, "q", q, dev, bf16, (rows, h, 192), (1,))
    _chk(where, "w_uk", w_uk, dev, bf16, (h, 128, 512), (512, 1))
    _chk(where, "q_lat", q_lat, dev,
         bf16 if plan.q_dtype == PDA_BF16 else u8 if q_lat.dtype is u8 else e4m3, (rows, h, 576))
    split_scratch = _scratch(where, split_scratch, dev, 4)
    row, head = _head_strides(q)
    rc = (_LIB or load_library()).pda_mla_absorb(
        ctypes.byref(plan), q.data_ptr(), row, head, w_uk.data_ptr(), _row_stride(w_uk),
        float(q_scale), q_lat.data_ptr(), rows, _num_rows(where, num_rows, dev), split_scratch,
        _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def pda_mla_project(plan: PdaPlan, o_lat, w_uv, out, num_rows, split_scratch, stream=None,
                    check: bool = True) -> int:
    """The decode's latent output projected: o_lat bf16 [rows, Hq, 512], w_uv bf16
    [Hq, 128, 512] (any head stride), out bf16 [rows, Hq, 128]."""
    bf16 = (_TYPES or _types())[0]
    where, dev = "pda_mla_project", plan.device
    rows, h = o_lat.shape[0], plan.num_qo_heads
    _chk(where, "o_lat", o_lat, dev, bf16, (rows, h, 512))
    _chk(where, "w_uv", w_uv, dev, bf16, (h, 128, 512), (512, 1))
    _chk(where, "out", out, dev, bf16, (rows, h, 128))
    split_scratch = _scratch(where, split_scratch, dev, 4)
    rc = (_LIB or load_library()).pda_mla_project(
        ctypes.byref(plan), o_lat.data_ptr(), w_uv.data_ptr(), _row_stride(w_uv), out.data_ptr(),
        rows, _num_rows(where, num_rows, dev), split_scratch, _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def _same_strides(where: str, k, v):
    got = _head_strides(k)
    if got != _head_strides(v):
        raise ValueError(f"{where}: k and v differ in their strides")
    return got


def pda_mla_expand(plan: PdaPlan, k_pages, page_table, kv_indptr, tok_indptr, k_scale, w_uk, w_uv,
                   latent, k, v, split_scratch, stream=None, check: bool = True) -> int:
    """Keys and values of cached tokens: latent bf16 [tokens, 576], k and v bf16
    [tokens, Hq, 128] (strided alike) are written; w_uk and w_uv bf16 [Hq, 128, 512]."""
    bf16, i32, _, _, _, _ = _TYPES or _types()
    where, dev = "pda_mla_expand", plan.device
    tokens, h, ptrs = latent.shape[0], plan.num_qo_heads, (plan.batch + 1,)
    _chk(where, "w_uk", w_uk, dev, bf16, (h, 128, 512), (512, 1))
    _chk(where, "w_uv", w_uv, dev, bf16, (h, 128, 512), (512, 1))
    _chk(where, "latent", latent, dev, bf16, (tokens, 576))
    _chk(where, "k", k, dev, bf16, (tokens, h, 128), (1,))
    _chk(where, "v", v, dev, bf16, (tokens, h, 128), (1,))
    _chk(where, "kv_indptr", kv_indptr, dev, i32, ptrs)
    _chk(where, "tok_indptr", tok_indptr, dev, i32, ptrs)
    _chk(where, "page_table", page_table, dev, i32, (page_table.numel(),))
    k_pages, k_scale = _cache(where, "k", k_pages, k_scale, plan)
    split_scratch = _scratch(where, split_scratch, dev, 4)
    w_head = _row_stride(w_uk)
    if w_head != _row_stride(w_uv):
        raise ValueError(f"{where}: w_uk and w_uv differ in their head strides")
    tok, head = _same_strides(where, k, v)
    rc = (_LIB or load_library()).pda_mla_expand(
        ctypes.byref(plan), k_pages, page_table.data_ptr(), kv_indptr.data_ptr(),
        tok_indptr.data_ptr(), k_scale, w_uk.data_ptr(), w_uv.data_ptr(), w_head,
        latent.data_ptr(), k.data_ptr(), v.data_ptr(), tok, head, tokens, split_scratch,
        _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def pda_prefill_plan(plan: PdaPlan, rows: int, tokens: int, check: bool = True):
    """-> (PdaPrefillPlan, scratch_bytes, rc)."""
    pre = PdaPrefillPlan()
    nbytes = ctypes.c_size_t(0)
    rc = (_LIB or load_library()).pda_prefill_plan(ctypes.byref(plan), int(rows), int(tokens),
                                         ctypes.byref(pre), ctypes.byref(nbytes))
    if check and rc != PDA_OK:
        raise PdaError(rc, "pda_prefill_plan")
    return pre, int(nbytes.value), rc


def pda_mla_prefill(pre: PdaPrefillPlan, q, k, v, k_rope, qo_indptr, tok_indptr, window,
                    causal: bool, sm_scale: float, out, lse, scratch, stream=None,
                    check: bool = True) -> int:
    """Expanded latent attention of ragged requests: q bf16 [rows, Hq, 192], k and v bf16
    [tokens, Hq, 128] (strided alike), k_rope bf16 [tokens, 64], out bf16 [rows, Hq, 128],
    lse fp32 [rows, Hq] or None; rows and tokens are the plan's."""
    bf16, i32, _, f32, _, _ = _TYPES or _types()
    where, dev = "pda_mla_prefill", pre.device
    rows, tokens, h, n = pre.rows, pre.tokens, pre.num_qo_heads, pre.batch
    _chk(where, "q", q, dev, bf16, (rows, h, 192), (1,))
    _chk(where, "k", k, dev, bf16, (tokens, h, 128), (1,))
    _chk(where, "v", v, dev, bf16, (tokens, h, 128), (1,))
    _chk(where, "k_rope", k_rope, dev, bf16, (tokens, 64), (1,))
    _chk(where, "qo_indptr", qo_indptr, dev, i32, (n + 1,))
    _chk(where, "tok_indptr", tok_indptr, dev, i32, (n + 1,))
    _chk(where, "out", out, dev, bf16, (rows, h, 128))
    if window is not None:
        _chk(where, "window", window, dev, i32, (n,))
        window = window.data_ptr()
    if lse is not None:
        _chk(where, "lse", lse, dev, f32, (rows, h))
        lse = lse.data_ptr()
    scratch = _scratch(where, scratch, dev, pre.scratch_bytes)
    tok, head = _same_strides(where, k, v)
    row, qhead = _head_strides(q)
    rc = (_LIB or load_library()).pda_mla_prefill(
        ctypes.byref(pre), q.data_ptr(), row, qhead, k.data_ptr(), v.data_ptr(), tok, head,
        k_rope.data_ptr(), _row_stride(k_rope), qo_indptr.data_ptr(), tok_indptr.data_ptr(), window,
        1 if causal else 0, float(sm_scale), out.data_ptr(), lse, scratch, _stream(stream, dev))
    if check and rc != PDA_OK:
        raise PdaError(rc, where)
    return rc


def pda_get_status(plan: PdaPlan, split_scratch, stream=None) -> int:
    """Device status bits; ``split_scratch=None`` reads those of the
    built-in array that pda_decode_static uses."""
    bits = _u32(0)
    rc = load_library().pda_get_status(ctypes.byref(plan), _ptr(split_scratch),
                                       ctypes.byref(bits), _stream(stream))
    if rc != PDA_OK:
        raise PdaError(rc, "pda_get_status")
    return int(bits.value)


def pda_reset_status(plan: PdaPlan, split_scratch, stream=None) -> None:
    rc = load_library().pda_reset_status(ctypes.byref(plan), _ptr(split_scratch),
                                         _stream(stream))
    if rc != PDA_OK:
        raise PdaError(rc, "pda_reset_status")


# ---------------------------------------------------------------- helpers

def params_for(wl, *, max_batch=None, max_q_len=None, max_kv_len=None, device=0, num_sms=0,
               chunk_pages=0, kernel=PDA_KERNEL_AUTO, batch=0, wait_limit_us=0,
               inject=0, host_plan=False) -> PdaParams:
    """PdaParams describing a workload object (synth.Workload or alike).
    ``host_plan``: pass the batch's host lengths, rows and windows, so the
    planner sizes the KV chunk for this batch (the plan still serves any
    lengths within its maxima)."""
    p = PdaParams()
    p.num_qo_heads = wl.num_qo_heads
    p.num_kv_heads = wl.num_kv_heads
    p.head_dim = wl.head_dim
    p.page_size = wl.page_size
    p.q_dtype = PDA_E4M3 if wl.q_e4m3 else PDA_BF16
    p.kv_dtype = (PDA_E4M3 if wl.kv_e4m3 else
                  PDA_INT8 if getattr(wl, "kv_int8", False) else PDA_BF16)
    p.scale_mode = wl.scale_mode
    p.max_batch = max_batch or wl.batch
    p.max_q_len = max_q_len or max(1, wl.max_q_len)
    p.max_kv_len = max_kv_len or max(1, int(wl.kv_len.max().item()))
    p.num_pages = wl.num_pages
    p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = (int(s) for s in wl.strides)
    p.device = device
    p.num_sms = num_sms
    p.batch = batch or wl.batch
    p.chunk_pages = chunk_pages
    p.kernel = kernel
    p.head_dim_v = getattr(wl, "head_dim_v", None) or 0
    p.wait_limit_us = wait_limit_us
    p.inject = inject
    if host_plan:
        def arr(xs):
            a = (_i32 * len(xs))(*[int(x) for x in xs])
            return a, ctypes.cast(a, ctypes.POINTER(_i32))
        p._keep = [arr(wl.kv_len.cpu().tolist()), arr(wl.qo_indptr.cpu().tolist())]
        p.host_kv_len, p.host_qo_indptr = p._keep[0][1], p._keep[1][1]
        if wl.window is not None:
            p._keep.append(arr(wl.window.cpu().tolist()))
            p.host_window = p._keep[2][1]
    return p


class Decoder:
    """A plan plus its split scratch (allocated once with torch) for one
    workload shape; ``run`` enqueues one pda_decode on the current stream."""

    def __init__(self, params: PdaParams, device="cuda"):
        import torch
        self.params = params
        self.plan, self.scratch_bytes, _ = pda_plan(params)
        n = (max(self.scratch_bytes, 256) + 255) // 256 * 256
        self.scratch = torch.zeros(n, dtype=torch.uint8, device=device)

    def run(self, wl, out, lse, max_q_len=None, stream=None, sm_scale=None, stages=None):
        args = (self.plan, wl.q, wl.k_pages, wl.v_pages, wl.page_table, wl.kv_indptr, wl.kv_len,
                wl.qo_indptr, max_q_len or max(1, wl.max_q_len), wl.window,
                wl.sm_scale if sm_scale is None else sm_scale, wl.k_scale, wl.v_scale, out, lse,
                self.scratch)
        if stages is None:
            return pda_decode(*args, stream)
        return pda_decode_stages(*args, stages, stream)

    def status(self, stream=None) -> int:
        return pda_get_status(self.plan, self.scratch, stream)

    def reset_status(self, stream=None) -> None:
        pda_reset_status(self.plan, self.scratch, stream)


class Prefill:
    """A prefill plan plus its scratch (allocated once with torch), for up to ``rows`` query
    rows and ``tokens`` keys of the MLA plan's requests; ``run`` enqueues one pda_mla_prefill."""

    def __init__(self, plan: PdaPlan, rows: int, tokens: int, device=None):
        import torch
        self.decode_plan = plan
        self.plan, self.scratch_bytes, _ = pda_prefill_plan(plan, rows, tokens)
        self.scratch = torch.zeros(self.scratch_bytes, dtype=torch.uint8,
                                   device=f"cuda:{plan.device}" if device is None else device)

    def run(self, q, k, v, k_rope, qo_indptr, tok_indptr, sm_scale, out, lse, window=None,
            causal=True, stream=None):
        return pda_mla_prefill(self.plan, q, k, v, k_rope, qo_indptr, tok_indptr, window, causal,
                               sm_scale, out, lse, self.scratch, stream)

    def status(self, stream=None) -> int:
        return pda_get_status(self.decode_plan, self.scratch, stream)

    def reset_status(self, stream=None) -> None:
        pda_reset_status(self.decode_plan, self.scratch, stream)
