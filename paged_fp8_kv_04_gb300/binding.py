"""Thin Python binding of libpagedfp8 (include/pa.h): argument marshalling only.

Every step of the attention runs in the library's CUDA kernels; this module checks
tensor dtypes and devices, passes data pointers and the current torch stream, and
raises on a non-OK status.  It fails loudly when the shared library is missing.
The cache operators between two decode steps and those on a prompt's way into the cache are marshalled
by a compiled module (csrc/pa_torch.cpp), since most of their kernels are shorter than the same checks in Python.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import numpy as np

from . import build as _build

KV_FP8_E4M3, KV_BF16 = 0, 1
SCALE_NONE, SCALE_SCALAR, SCALE_PER_TOKEN = 0, 1, 2
Q_UNIFORM, Q_RAGGED = 0, 1
OUT_BF16, OUT_F32 = 0, 1
PLAN_NO_PDL = 0x1
PLAN_TCGEN05 = 0x2

STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_CAPACITY",
          4: "PA_ERR_RAGGED", 5: "PA_ERR_ALIGN", 6: "PA_ERR_CUDA", 7: "PA_ERR_DEVICE_DATA",
          8: "PA_ERR_WORKSPACE"}
DEV_FLAGS = {0x01: "BAD_PAGE", 0x02: "BAD_CONTEXT", 0x04: "BAD_QLEN", 0x08: "NOT_UNIFORM",
             0x10: "BAD_SELECTED", 0x20: "Q_RANGE", 0x40: "TIMEOUT", 0x80: "DUMP_RANGE"}


class PaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class PlanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_kv_heads", "group_size", "head_dim", "page_size", "kv_dtype", "scale_mode",
        "q_mode", "q_len", "max_batch", "max_rows", "max_context_len", "max_selected_pages",
        "partition_tokens", "out_dtype", "num_sms", "flags")] + [("reserved", ctypes.c_int32 * 2)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("k_scale_scalar", ctypes.c_float), ("v_scale_scalar", ctypes.c_float),
        ("num_pages", ctypes.c_int64), ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("context_lens", ctypes.c_void_p), ("cu_seqlens_q", ctypes.c_void_p),
        ("cu_seqlens_q_host", ctypes.c_void_p), ("selected_pages", ctypes.c_void_p),
        ("num_selected", ctypes.c_void_p), ("selected_stride", ctypes.c_int32),
        ("num_rows", ctypes.c_int32), ("sm_scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [("grid_ctas", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("threads_per_cta", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("partial_slots", ctypes.c_int64), ("kernel", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class KvWriteArgs(ctypes.Structure):
    _fields_ = [("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("num_tokens", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32)]


DEV_BAD_SLOT = 0x100
DEV_BAD_INDEX_ROW = 0x200
DEV_BAD_KEEP = 0x400
DEV_BAD_BEAM = 0x800
DEV_PAGE_POOL = 0x1000
ROPE_BF16, ROPE_F32 = 0, 1
ROPE_HALF, ROPE_PAIRS = 0, 1
LOGITS_BF16, LOGITS_F32 = 0, 1
MAX_BEAM_STATES = 4


class IndexArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
                ("cu_seqlens_q", ctypes.c_void_p), ("selected", ctypes.c_void_p),
                ("num_selected", ctypes.c_void_p), ("scores", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("num_seqs", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("index_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("block_table_stride", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("reserved", ctypes.c_int32)]

class LseMergeArgs(ctypes.Structure):
    _fields_ = [("part_out", ctypes.c_void_p), ("part_lse", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("num_parts", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _struct(name, pointers, i64="", i32="", f32=""):
    """A ctypes structure of pointers, then int64, int32 and float fields, then a reserved word."""
    fields = [(n, ctypes.c_void_p) for n in pointers.split()]
    fields += [(n, ctypes.c_int64) for n in i64.split()]
    fields += [(n, ctypes.c_int32) for n in i32.split()]
    fields += [(n, ctypes.c_float) for n in f32.split()]
    return type(name, (ctypes.Structure,), {"_fields_": fields + [("reserved", ctypes.c_int32)]})


AttnMassArgs = _struct(
    "AttnMassArgs", "q k_cache k_scale block_table context_lens cu_seqlens_q lse mass mass_out status",
    "num_pages", "num_seqs num_rows num_kv_heads group_size head_dim page_size kv_dtype scale_mode "
    "block_table_stride mass_stride max_q_len", "k_scale_scalar sm_scale decay")
EvictSelectArgs = _struct(
    "EvictSelectArgs", "mass context_lens keep new_lens status", "",
    "num_seqs num_kv_heads mass_stride budget keep_first keep_recent")
KvCompactArgs = _struct(
    "KvCompactArgs", "keep new_lens block_table dst_block_table k_cache v_cache k_scale v_scale mass mass_out "
    "status", "num_pages", "num_seqs num_kv_heads head_dim page_size kv_dtype scale_mode keep_stride "
    "block_table_stride dst_block_table_stride mass_stride mass_out_stride")
BeamSelectArgs = _struct(
    "BeamSelectArgs", "logits scores finished lengths tokens parents scores_out finished_out lengths_out",
    "logits_stride", "num_reqs num_beams vocab logits_dtype eos_token", "length_penalty")


class BeamReorderArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "parents", "context_lens", "block_table", "block_table_out", "k_cache", "v_cache", "k_scale",
        "v_scale", "status")] + [
        ("state_in", ctypes.c_void_p * MAX_BEAM_STATES), ("state_out", ctypes.c_void_p * MAX_BEAM_STATES),
        ("state_bytes", ctypes.c_int64 * MAX_BEAM_STATES), ("num_pages", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in (
            "num_states", "num_reqs", "num_beams", "num_kv_heads", "head_dim", "page_size", "kv_dtype",
            "scale_mode", "block_table_stride", "reserved")]


PageAssignArgs = _struct(
    "PageAssignArgs", "context_lens cu_seqlens_q block_table free_pages num_free num_free_out new_lens slot_mapping positions "
    "status", "num_pages", "num_seqs num_rows block_table_stride page_size free_capacity")
PageReleaseArgs = _struct(
    "PageReleaseArgs", "context_lens new_lens block_table free_pages num_free num_free_out status", "num_pages",
    "num_seqs block_table_stride page_size free_capacity")
RopeArgs = _struct(
    "RopeArgs", "q k positions freqs q_out k_out", "q_stride k_stride q_out_stride k_out_stride",
    "num_tokens num_q_heads num_kv_heads head_dim rot_dim dtype layout inverse", "scale")
PromptAttnArgs = _struct(
    "PromptAttnArgs", "q k v cu_seqlens out lse status", "q_stride k_stride v_stride",
    "num_seqs num_rows num_kv_heads group_size head_dim out_dtype", "sm_scale")


_lib = None
P = ctypes.c_void_p


def header_functions() -> list:
    """Names of every function include/pa.h declares."""
    with open(os.path.join(_build.INCLUDE, "pa.h")) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_[a-z_0-9]+)\s*\(", text)))


def lib(path: Optional[str] = None):
    """Loads libpagedfp8.so (built in-tree by __graft_entry__.build()); raises if missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libpagedfp8.so is not built ({p}); run __graft_entry__.build()")
    L = ctypes.CDLL(p)
    L.pa_plan_validate.argtypes = [ctypes.POINTER(PlanDesc)]
    L.pa_plan_validate.restype = ctypes.c_int
    L.pa_plan_workspace_size.argtypes = [ctypes.POINTER(PlanDesc)]
    L.pa_plan_workspace_size.restype = ctypes.c_size_t
    L.pa_plan_create.argtypes = [ctypes.POINTER(PlanDesc), P, ctypes.c_size_t, ctypes.POINTER(P)]
    L.pa_plan_create.restype = ctypes.c_int
    L.pa_decode_check.argtypes = [P, ctypes.POINTER(DecodeArgs)]
    L.pa_decode_check.restype = ctypes.c_int
    L.pa_decode.argtypes = [P, ctypes.POINTER(DecodeArgs), P]
    L.pa_decode.restype = ctypes.c_int
    L.pa_plan_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
    L.pa_plan_get_device_status.restype = ctypes.c_int
    L.pa_plan_get_info.argtypes = [P, ctypes.POINTER(PlanInfo)]
    L.pa_plan_get_info.restype = ctypes.c_int
    L.pa_plan_destroy.argtypes = [P]
    L.pa_plan_destroy.restype = None
    L.pa_status_string.argtypes = [ctypes.c_int]
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_debug_row_map.argtypes = [P, ctypes.POINTER(DecodeArgs), P, P]
    L.pa_debug_row_map.restype = ctypes.c_int
    L.pa_debug_gather_tile_bytes.argtypes = [P]
    L.pa_debug_gather_tile_bytes.restype = ctypes.c_size_t
    L.pa_debug_gather.argtypes = [P, ctypes.POINTER(DecodeArgs), P, ctypes.c_size_t, P]
    L.pa_debug_gather.restype = ctypes.c_int
    L.pa_decode_noalloc.argtypes = [ctypes.POINTER(PlanDesc), ctypes.POINTER(DecodeArgs), P]
    L.pa_decode_noalloc.restype = ctypes.c_int
    L.pa_kv_quantize_write.argtypes = [ctypes.POINTER(KvWriteArgs), P]
    L.pa_kv_quantize_write.restype = ctypes.c_int
    L.pa_index_topk.argtypes = [ctypes.POINTER(IndexArgs), P]
    L.pa_index_topk.restype = ctypes.c_int
    L.pa_lse_merge.argtypes = [ctypes.POINTER(LseMergeArgs), P]
    L.pa_lse_merge.restype = ctypes.c_int
    for name, args in (("pa_attn_mass", AttnMassArgs), ("pa_evict_select", EvictSelectArgs),
                       ("pa_kv_compact", KvCompactArgs), ("pa_beam_select", BeamSelectArgs),
                       ("pa_beam_reorder", BeamReorderArgs), ("pa_page_assign", PageAssignArgs),
                       ("pa_page_release", PageReleaseArgs), ("pa_rope", RopeArgs), ("pa_prompt_attn", PromptAttnArgs)):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(args), P]
        f.restype = ctypes.c_int
    L.pa_debug_trace.argtypes = [P, ctypes.c_size_t]
    L.pa_debug_trace.restype = ctypes.c_int
    if path is None:
        _lib = L
    return L


def make_desc(*, num_kv_heads=1, group_size=16, head_dim=128, page_size=128, kv_dtype="fp8",
              scale_mode="per_token", q_mode="uniform", q_len=1, max_batch=1, max_rows=None,
              max_context_len=1, max_selected_pages=0, partition_tokens=0, out_dtype="bf16",
              num_sms=0, pdl=True, tcgen05=False) -> PlanDesc:
    d = PlanDesc()
    d.num_kv_heads, d.group_size, d.head_dim, d.page_size = num_kv_heads, group_size, head_dim, page_size
    d.kv_dtype = {"fp8": KV_FP8_E4M3, "bf16": KV_BF16}[kv_dtype] if isinstance(kv_dtype, str) else kv_dtype
    d.scale_mode = ({"none": SCALE_NONE, "scalar": SCALE_SCALAR, "per_token": SCALE_PER_TOKEN}[scale_mode]
                    if isinstance(scale_mode, str) else scale_mode)
    d.q_mode = {"uniform": Q_UNIFORM, "ragged": Q_RAGGED}[q_mode] if isinstance(q_mode, str) else q_mode
    d.q_len, d.max_batch = q_len, max_batch
    d.max_rows = max_rows if max_rows is not None else max_batch * q_len
    d.max_context_len, d.max_selected_pages = max_context_len, max_selected_pages
    d.partition_tokens = partition_tokens
    d.out_dtype = {"bf16": OUT_BF16, "f32": OUT_F32}[out_dtype] if isinstance(out_dtype, str) else out_dtype
    d.num_sms = num_sms
    d.flags = (0 if pdl else PLAN_NO_PDL) | (PLAN_TCGEN05 if tcgen05 else 0)
    return d


def _ptr(t):
    return None if t is None else t.data_ptr()


class Plan:
    """A plan over a capacity bucket, owning its device workspace (a torch uint8 tensor)."""

    def __init__(self, device=None, check_only: bool = False, **desc_kw):
        import torch
        self._lib = lib()
        self.desc = make_desc(**desc_kw)
        self.kv_dtype = desc_kw.get("kv_dtype", "fp8")
        self.scale_mode = desc_kw.get("scale_mode", "per_token")
        self.out_dtype = desc_kw.get("out_dtype", "bf16")
        self._plan = P()
        self.workspace = None
        if check_only:
            st = self._lib.pa_plan_create(ctypes.byref(self.desc), None, 0, ctypes.byref(self._plan))
        else:
            self.device = torch.device(device if device is not None else "cuda")
            nbytes = self._lib.pa_plan_workspace_size(ctypes.byref(self.desc))
            if nbytes == 0:
                raise PaError(self._lib.pa_plan_validate(ctypes.byref(self.desc)) or 2,
                              "pa_plan_workspace_size")
            with torch.cuda.device(self.device):
                self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
                st = self._lib.pa_plan_create(ctypes.byref(self.desc), self.workspace.data_ptr(),
                                              nbytes, ctypes.byref(self._plan))
        if st != 0:
            raise PaError(st, "pa_plan_create")

    def __del__(self):
        try:
            if getattr(self, "_plan", None):
                self._lib.pa_plan_destroy(self._plan)
                self._plan = P()
        except Exception:
            pass

    def info(self) -> dict:
        inf = PlanInfo()
        st = self._lib.pa_plan_get_info(self._plan, ctypes.byref(inf))
        if st != 0:
            raise PaError(st, "pa_plan_get_info")
        return {n: getattr(inf, n) for n, _ in PlanInfo._fields_}

    # ------------------------------------------------------------------ argument building
    def args(self, q, k_cache, v_cache, block_table, context_lens, *, k_scale=None, v_scale=None,
             k_scale_scalar=1.0, v_scale_scalar=1.0, cu_seqlens_q=None, cu_seqlens_q_host=None,
             selected_pages=None, num_selected=None, sm_scale=None, out=None, lse=None,
             num_pages=None, keep=None):
        a = DecodeArgs()
        a.q, a.k_cache, a.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
        a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
        a.k_scale_scalar, a.v_scale_scalar = float(k_scale_scalar), float(v_scale_scalar)
        a.num_pages = int(num_pages if num_pages is not None else k_cache.shape[0])
        a.block_table = _ptr(block_table)
        a.block_table_stride = int(block_table.shape[1]) if block_table is not None else 0
        a.num_seqs = int(context_lens.shape[0]) if context_lens is not None else 0
        a.context_lens = _ptr(context_lens)
        a.cu_seqlens_q = _ptr(cu_seqlens_q)
        if cu_seqlens_q_host is not None:
            h = np.ascontiguousarray(cu_seqlens_q_host, dtype=np.int32)
            if keep is not None:
                keep.append(h)
            a.cu_seqlens_q_host = h.ctypes.data
        a.selected_pages = _ptr(selected_pages)
        a.selected_stride = int(selected_pages.shape[1]) if selected_pages is not None else 0
        a.num_selected = _ptr(num_selected)
        a.num_rows = int(q.shape[0]) if q is not None else 0
        hd = self.desc.head_dim
        a.sm_scale = float(sm_scale if sm_scale is not None else 1.0 / np.sqrt(hd))
        a.out = _ptr(out)
        a.lse = _ptr(lse)
        return a

    def check(self, a: DecodeArgs) -> int:
        return self._lib.pa_decode_check(self._plan, ctypes.byref(a))

    def _stream(self, stream):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        return ctypes.c_void_p(s.cuda_stream)

    def decode(self, q, k_cache, v_cache, block_table, context_lens, *, out=None, lse=None,
               stream=None, **kw):
        """Enqueues one decode; returns `out` ([rows, Hq, D], bf16 or fp32 per the plan)."""
        import torch
        if out is None:
            dt = torch.float32 if self.out_dtype == "f32" else torch.bfloat16
            out = torch.empty(q.shape, dtype=dt, device=q.device)
        keep = []
        a = self.args(q, k_cache, v_cache, block_table, context_lens, out=out, lse=lse,
                      keep=keep, **kw)
        st = self._lib.pa_decode(self._plan, ctypes.byref(a), self._stream(stream))
        if st != 0:
            raise PaError(st, "pa_decode")
        return out

    def decode_args(self, a: DecodeArgs, stream=None) -> None:
        """Enqueues a decode from prepared arguments (for timing loops and graph capture)."""
        st = self._lib.pa_decode(self._plan, ctypes.byref(a), self._stream(stream))
        if st != 0:
            raise PaError(st, "pa_decode")

    def device_status(self, clear: bool = True) -> int:
        v = ctypes.c_uint32(0)
        st = self._lib.pa_plan_get_device_status(self._plan, ctypes.byref(v), int(clear))
        if st != 0:
            raise PaError(st, "pa_plan_get_device_status")
        return int(v.value)

    def _scratch_out(self, q, kw):
        import torch
        out = kw.pop("out", None)
        if out is None:
            dt = torch.float32 if self.out_dtype == "f32" else torch.bfloat16
            out = torch.empty(q.shape, dtype=dt, device=q.device)
        return out

    def row_map(self, q, k_cache, v_cache, block_table, context_lens, **kw):
        import torch
        keep = []
        a = self.args(q, k_cache, v_cache, block_table, context_lens, keep=keep,
                      out=self._scratch_out(q, kw), **kw)
        rm = torch.full((a.num_rows, 3), -1, dtype=torch.int32, device=q.device)
        st = self._lib.pa_debug_row_map(self._plan, ctypes.byref(a), rm.data_ptr(),
                                        self._stream(None))
        if st != 0:
            raise PaError(st, "pa_debug_row_map")
        return rm

    def gather(self, q, k_cache, v_cache, block_table, context_lens, num_tiles, **kw):
        import torch
        keep = []
        a = self.args(q, k_cache, v_cache, block_table, context_lens, keep=keep,
                      out=self._scratch_out(q, kw), **kw)
        tb = self._lib.pa_debug_gather_tile_bytes(self._plan)
        dump = torch.zeros(max(num_tiles, 1) * tb, dtype=torch.uint8, device=q.device)
        st = self._lib.pa_debug_gather(self._plan, ctypes.byref(a), dump.data_ptr(),
                                       num_tiles * tb, self._stream(None))
        if st != 0:
            raise PaError(st, "pa_debug_gather")
        return dump, tb


def kv_write_args(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, status=None,
                  num_tokens=None) -> KvWriteArgs:
    """pa_kv_write_args_t over torch tensors: k_new / v_new bf16 [T, Hkv, D], slot_mapping
    int64 [T], caches uint8 [num_pages, Hkv, page_size, D], scales fp32
    [num_pages, Hkv, page_size], status an optional int32/uint32 device word."""
    a = KvWriteArgs()
    a.k_new, a.v_new, a.slot_mapping = _ptr(k_new), _ptr(v_new), _ptr(slot_mapping)
    a.k_cache, a.v_cache, a.k_scale, a.v_scale = (_ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                                  _ptr(v_scale))
    a.status = _ptr(status)
    a.num_tokens = int(num_tokens if num_tokens is not None else k_new.shape[0])
    a.num_pages = int(k_cache.shape[0])
    a.num_kv_heads = int(k_cache.shape[1])
    a.page_size = int(k_cache.shape[2])
    a.head_dim = int(k_cache.shape[3])
    a.reserved = 0
    return a


def kv_quantize_write(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                      status=None, stream=None, args: Optional[KvWriteArgs] = None) -> None:
    """Enqueues pa_kv_quantize_write on `stream` (default: torch's current stream)."""
    import torch
    a = args if args is not None else kv_write_args(k_new, v_new, slot_mapping, k_cache, v_cache,
                                                    k_scale, v_scale, status)
    s = stream if stream is not None else torch.cuda.current_stream(k_cache.device)
    st = lib().pa_kv_quantize_write(ctypes.byref(a), ctypes.c_void_p(s.cuda_stream))
    if st != 0:
        raise PaError(st, "pa_kv_quantize_write")


def index_args(q, k_cache, k_scale, block_table, context_lens, cu_seqlens_q, selected,
               num_selected, scores, *, topk, max_q_len, sm_scale, status=None) -> IndexArgs:
    """pa_index_args_t over torch tensors: q bf16 [rows, heads, 128], k_cache uint8
    [num_pages, page_size, 128], k_scale fp32 [num_pages, page_size] or None, int32 block
    table / context lens / cu_seqlens_q, outputs selected int32 [rows, topk], num_selected
    int32 [rows], scores fp32 [rows, stride]."""
    a = IndexArgs()
    a.q, a.k_cache, a.k_scale = _ptr(q), _ptr(k_cache), _ptr(k_scale)
    a.block_table, a.context_lens, a.cu_seqlens_q = _ptr(block_table), _ptr(context_lens), _ptr(cu_seqlens_q)
    a.selected, a.num_selected, a.scores, a.status = (_ptr(selected), _ptr(num_selected),
                                                      _ptr(scores), _ptr(status))
    a.num_pages = int(k_cache.shape[0])
    a.num_seqs = int(context_lens.shape[0])
    a.num_rows = int(q.shape[0])
    a.index_heads = int(q.shape[1])
    a.head_dim = int(q.shape[2])
    a.page_size = int(k_cache.shape[1])
    a.topk = int(topk)
    a.block_table_stride = int(block_table.shape[1])
    a.max_q_len = int(max_q_len)
    a.sm_scale = float(sm_scale)
    a.reserved = 0
    return a


def index_topk(args: IndexArgs, device=None, stream=None) -> None:
    """Enqueues pa_index_topk on `stream` (default: torch's current stream)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    st = lib().pa_index_topk(ctypes.byref(args), ctypes.c_void_p(s.cuda_stream))
    if st != 0:
        raise PaError(st, "pa_index_topk")


def lse_merge_args(part_out, part_lse, out, lse=None) -> LseMergeArgs:
    """pa_lse_merge_args_t over torch tensors: part_out fp32 [parts, rows, heads, D],
    part_lse fp32 [parts, rows, heads], out bf16 or fp32 [rows, heads, D], lse fp32
    [rows, heads] or None."""
    import torch
    a = LseMergeArgs()
    a.part_out, a.part_lse, a.out, a.lse = _ptr(part_out), _ptr(part_lse), _ptr(out), _ptr(lse)
    a.num_parts, a.num_rows, a.num_heads, a.head_dim = (int(x) for x in part_out.shape)
    a.out_dtype = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    a.reserved = 0
    return a


def lse_merge(part_out, part_lse, out, lse=None, stream=None, args: Optional[LseMergeArgs] = None):
    """Enqueues pa_lse_merge on `stream` (default: torch's current stream); returns out."""
    import torch
    a = args if args is not None else lse_merge_args(part_out, part_lse, out, lse)
    s = stream if stream is not None else torch.cuda.current_stream(out.device)
    st = lib().pa_lse_merge(ctypes.byref(a), ctypes.c_void_p(s.cuda_stream))
    if st != 0:
        raise PaError(st, "pa_lse_merge")
    return out


# ----------------------------------------------- the cache between two decode steps
#
# These calls take tensors, check types, shapes and layout (the library sees only
# pointers), allocate the outputs that are not given on the launching stream, and run on
# the device of their tensors whatever the current device is.  Wrong tensors raise TypeError
# or ValueError, a refusal by the library PaError.

_module = None


def torch_module():
    """pa_torch.so (built in-tree by __graft_entry__.build()), bound to the library; raises if missing."""
    global _module
    if _module is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries are loaded first)
        path = _build.torch_module_path()
        if not os.path.exists(path):
            raise ImportError(f"pa_torch.so is not built ({path}); run __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("pa_torch", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("pa_torch", loader))
        loader.exec_module(m)
        L = lib()
        m.bind(PaError, *(ctypes.cast(f, P).value for f in (
            L.pa_attn_mass, L.pa_evict_select, L.pa_kv_compact, L.pa_beam_select, L.pa_beam_reorder, L.pa_page_assign,
            L.pa_page_release, L.pa_rope, L.pa_prompt_attn)))
        _module = m
    return _module


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def attn_mass(q, k_cache, block_table, context_lens, cu_seqlens_q, lse, mass, *, max_q_len,
              sm_scale=None, decay=1.0, out=None, k_scale=None, k_scale_scalar=1.0, status=None,
              stream=None):
    """Adds a decode step's attention weights to the cached tokens' mass (pa_attn_mass).

    q bf16 [rows, Hq, D], k_cache as pa_decode's, lse fp32 [rows, Hq] of the same step's pa_decode
    over the whole context (a sparse decode's lse covers the selected pages alone, and would give
    weight to tokens that nobody attended),
    mass fp32 [B, Hkv, stride]; updated in place, or into `out` when given (positions past a
    request's context are not written).  max_q_len bounds every request's rows.  Returns
    the updated tensor."""
    return (_module or torch_module()).attn_mass(
        q, k_cache, block_table, context_lens, cu_seqlens_q, lse, mass, out, k_scale, status, _handle(stream),
        max_q_len, sm_scale, decay, k_scale_scalar)


def evict_select(mass, context_lens, *, budget, first=0, recent=0, keep=None, new_lens=None,
                 status=None, stream=None):
    """The positions that stay when every cache is cut to `budget` tokens (pa_evict_select):
    the first `first`, the last `recent` and the largest mass between.  mass fp32
    [B, Hkv, stride], context_lens int32 [B].  Returns (keep int32 [B, Hkv, budget], ascending,
    -1 after; new_lens int32 [B]).

    A decode on a plan with pdl (the default) reads its context lengths while the kernel before it is
    still running: between this call and a decode that reads new_lens there has to be another kernel that
    is not a decode, such as kv_compact or the write of the step's new tokens."""
    return (_module or torch_module()).evict_select(
        mass, context_lens, keep, new_lens, status, _handle(stream), budget, first, recent)


def kv_compact(keep, new_lens, block_table, k_cache, v_cache, *, dst_block_table=None, k_scale=None,
               v_scale=None, mass=None, mass_out=None, status=None, stream=None) -> None:
    """Moves the kept tokens to the front of their own pages, or of dst_block_table's
    (pa_kv_compact).  keep int32 [B, Hkv, n] and new_lens int32 [B] as evict_select gives
    them; mass fp32 [B, Hkv, stride] moves along, in place or, with dst_block_table, into
    mass_out.  Afterwards new_lens are the context lengths.  The indexer's key cache is not moved:
    index_topk scores pages by the tokens that were there before until the caller has moved its
    index keys and scales by the same keep."""
    (_module or torch_module()).kv_compact(
        keep, new_lens, block_table, dst_block_table, k_cache, v_cache, k_scale, v_scale, mass, mass_out, status,
        _handle(stream))


def beam_select(logits, scores, *, eos=-1, finished=None, lengths=None, length_penalty=0.0, tokens=None,
                parents=None, scores_out=None, finished_out=None, lengths_out=None, stream=None):
    """One step of beam search (pa_beam_select): the W best continuations of each request's W
    beams.  logits bf16 or fp32 [N, W, V] or [N * W, V] (rows may be strided: a padded
    vocabulary), scores fp32 [N, W] (-inf: no such beam yet), finished uint8 and lengths int32
    [N, W], both optional; length_penalty is rounded to fp32.  Returns (tokens, parents, scores, finished, lengths), each [N, W];
    the last two are None where their input is and no output is given."""
    return (_module or torch_module()).beam_select(
        logits, scores, finished, lengths, tokens, parents, scores_out, finished_out, lengths_out, _handle(stream),
        eos, length_penalty)


def beam_reorder(parents, context_lens, block_table, block_table_out, k_cache, v_cache, *, k_scale=None,
                 v_scale=None, states=(), status=None, stream=None) -> None:
    """Lets the beams' histories follow their parents (pa_beam_reorder).  parents int32 [N, W],
    context_lens int32 [N * W], block tables int32 [N * W, stride]; states: up to four
    (in, out) pairs of tensors with N * W rows, gathered by parent.

    A decode on a plan with pdl (the default) reads its block table while the kernel before it is still
    running: between this call and a decode that reads block_table_out there has to be another kernel that is
    not a decode, such as the write of the step's new tokens.  The indexer's key cache is not copied: a
    further child's partial page keeps the keys of the childless beam it came from, and index_topk scores it by
    them until the caller has copied the parent's."""
    (_module or torch_module()).beam_reorder(
        parents, context_lens, block_table, block_table_out, k_cache, v_cache, k_scale, v_scale, states, status,
        _handle(stream))


# ----------------------------------------------------- a prompt's way into the cache

def page_assign(context_lens, cu_seqlens_q, block_table, free_pages, num_free, *, page_size, num_pages, num_rows=None,
                num_free_out=None, new_lens=None, slot_mapping=None, positions=None, status=None, stream=None):
    """Gives requests that grow their pages, and their new tokens slots and positions (pa_page_assign).

    context_lens int32 [B], cu_seqlens_q int32 [B + 1], block_table int32 [B, stride] (updated in place), free_pages
    int32 [capacity] a stack of which num_free (int32 [1]) pages are left, updated in place or into num_free_out.
    num_rows rows in all, padding behind the last request's among them, unless slot_mapping is given.  Returns
    (new_lens int32 [B], slot_mapping int64 [rows] as kv_quantize_write takes it, positions int32 [rows] as rope
    does); new_lens may be context_lens.  A request that the pool has no pages for keeps its length and
    gets slots of -1 (DEV_PAGE_POOL in status).

    A decode on a plan with pdl (the default) reads its context lengths and block table while the kernel before it is still
    running: between this call and that decode there has to be another kernel that is not a decode, such as rope
    or the write of the step's new tokens."""
    return (_module or torch_module()).page_assign(
        context_lens, cu_seqlens_q, block_table, free_pages, num_free, num_free_out, new_lens, slot_mapping, positions, status,
        _handle(stream), page_size, num_pages, num_rows)


def page_release(context_lens, new_lens, block_table, free_pages, num_free, *, page_size, num_pages, num_free_out=None,
                 status=None, stream=None) -> None:
    """Takes back the pages behind the requests' new lengths (pa_page_release): 0 for a request that has ended, evict_select's
    for one that was cut.  They go on top of free_pages; num_free int32 [1] is updated in place or into
    num_free_out.  The block table is left as it is.  Pages that another request reads too (a common prefix, beams) must not
    be given back by this call: who counts references is the caller."""
    (_module or torch_module()).page_release(
        context_lens, new_lens, block_table, free_pages, num_free, num_free_out, status, _handle(stream), page_size, num_pages)


def rope_frequencies(rot_dim, *, base=10000.0, scaling=None, factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0,
                     device="cuda"):
    """The frequencies that rope takes, and the scale that belongs to them: (int64 [rot_dim / 2], float).

    Pair i turns by base ** (-2 i / rot_dim) radians per position.  For contexts `factor` times as long as the
    original_len that a model was trained on, scaling is "linear" (all pairs slower by factor), "ntk" (a larger base, so that the
    slowest pair is slower by factor) or "yarn" (pairs that turn more than beta_fast times within original_len stay, those
    that turn less than beta_slow times are slower by factor, a ramp between; queries and keys scaled by
    0.1 ln(factor) + 1 each).  Kept in units of 2^-64 turns, modulo one: a program makes them once."""
    import math

    import torch
    if rot_dim < 2 or rot_dim % 2 or rot_dim > 128:
        raise ValueError(f"rot_dim: {rot_dim}, expected an even number of 2 .. 128")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'ntk' or 'yarn'")
    if not (base > 1.0 and math.isfinite(base)) or (scaling is not None and not (factor >= 1.0 and math.isfinite(factor))):
        raise ValueError(f"base {base} and factor {factor}: expected finite, above 1 and at least 1")
    half, scale = rot_dim // 2, 1.0
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    elif scaling == "ntk":
        base = base * factor
    w = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    if scaling == "linear":
        w = [x / factor for x in w]
    elif scaling == "yarn":
        if not (original_len > 0 and beta_fast > beta_slow > 0):
            raise ValueError("original_len, beta_fast and beta_slow: expected beta_fast > beta_slow > 0")
        # the pair that turns so many times within original_len
        pair = lambda turns: rot_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot_dim - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(half)]
        w = [x / factor * r + x * (1.0 - r) for x, r in zip(w, ramp)]
        scale = 0.1 * math.log(factor) + 1.0
    turns = [round(x / (2.0 * math.pi) * 2.0 ** 64) % 2 ** 64 for x in w]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device), scale


def rope(q, k, positions, freqs, *, layout="half", inverse=False, scale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions (pa_rope).  q bf16 or fp32 [T, Hq, 128] and k [T, Hkv, 128] (or None), views of one projection's output
    among them; positions int32 [T]; freqs and scale from rope_frequencies.  Pair i is elements (i, i + rot / 2) with layout
    "half", (2 i, 2 i + 1) with "pairs"; elements past rot are carried over.  inverse turns back, which is also the
    rotation's gradient.  In place, or into q_out and k_out; returns (q_out, k_out)."""
    kinds = {"half": ROPE_HALF, "pairs": ROPE_PAIRS}
    if layout not in kinds:
        raise ValueError(f"layout: {layout!r}, expected 'half' or 'pairs'")
    return (_module or torch_module()).rope(
        q, k, positions, freqs, q_out, k_out, _handle(stream), kinds[layout], 1 if inverse else 0, scale)


def prompt_attn(q, k, v, cu_seqlens, *, sm_scale=None, out=None, lse=None, out_dtype="bf16", want_lse=False, status=None,
                stream=None):
    """Causal attention over whole prompts packed one behind the other (pa_prompt_attn).

    q bf16 [T, Hq, 128], k and v bf16 [T, Hkv, 128], views of one projection's output among them; cu_seqlens int32 [S + 1].
    Returns (out [T, Hq, 128], bf16 or, with out_dtype "f32" or a given fp32 `out`, fp32; lse fp32 [T, Hq], or None unless
    it is given or wanted).  Rows of no sequence are not written.  With an fp32 output and an lse the result joins, by
    lse_merge, with that of a decode over what is already cached of the same requests."""
    if out_dtype not in ("bf16", "f32"):
        raise ValueError(f"out_dtype: {out_dtype!r}, expected 'bf16' or 'f32'")
    return (_module or torch_module()).prompt_attn(
        q, k, v, cu_seqlens, out, lse, status, _handle(stream), sm_scale, OUT_F32 if out_dtype == "f32" else OUT_BF16,
        1 if want_lse else 0)
