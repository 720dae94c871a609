"""Thin ctypes binding of libsimoe (include/si_moe.h, include/si_kv.h).

The functions below carry the C entry points' names and only marshal
arguments: tensors become device pointers, torch streams become
cudaStream_t, and a non-OK status raises SiError.  Every step of the MoE
path runs in the library's CUDA kernels; there is no fallback.  If the
library has not been built, loading it raises immediately.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
LIB_PATH = os.path.join(PKG_DIR, "_build", "libsimoe.so")
HEADER_PATH = os.path.join(ROOT, "include", "si_moe.h")
KV_HEADER_PATH = os.path.join(ROOT, "include", "si_kv.h")

SI_OK = 0
SI_ERR_INVALID_ARG = 1
SI_ERR_UNSUPPORTED = 2
SI_ERR_MISALIGNED = 3
SI_ERR_SCRATCH_TOO_SMALL = 4
SI_ERR_CUDA = 5
SI_ERR_TIMEOUT = 6
SI_ERR_DEVICE = 7
SI_ERR_RANGE = 8
SI_WTYPE_Q4_K = 12
SI_WTYPE_NVFP4 = 100
SI_WTYPE_Q5_K = 13
SI_FLAG_ACT_INT8 = 1
SI_MODE_DECODE = 0
SI_MODE_PREFILL = 1
SI_MODE_DECODE_HOST = 2
SI_MAX_EXPERTS = 256
SI_MAX_TOPK = 16
SI_MAX_DECODE_TOKENS = 4
SI_STATIC_SCRATCH_BYTES = 1 << 20
SI_KV_INT8 = 1
SI_KV_E4M3 = 2
SI_KV_BF16 = 1
SI_KV_F16 = 2
SI_KV_MAX_SEQS = 1024
SI_KV_MAX_HEADS = 256
SI_KV_MAX_LEN = 1 << 22
SI_KV_MAX_EVICT_PAGES = 16384


class SiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {si_status_string(status)} (status {status})")


class si_moe_desc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("wtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class si_moe_layer(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("w_scale", ctypes.c_void_p)]


class si_moe_route_out(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("logits", ctypes.c_void_p)]


class si_kv_desc(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("code", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class si_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("n_slots", ctypes.c_int32)]


class si_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("total_new", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("q_start", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("table_stride", ctypes.c_int32)]


class si_kv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libsimoe; raise if it is missing (build it first)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libsimoe is not built ({p} missing): run "
                           "`python -m quantized_moe_expert_gemv_gb300.build` first")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.si_status_string.restype = ctypes.c_char_p
    lib.si_status_string.argtypes = [ctypes.c_int]
    lib.si_moe_plan.restype = ctypes.c_int
    lib.si_moe_plan.argtypes = [ctypes.POINTER(si_moe_desc), ctypes.c_int, ctypes.POINTER(vp)]
    lib.si_moe_plan_destroy.restype = None
    lib.si_moe_plan_destroy.argtypes = [vp]
    lib.si_moe_scratch_bytes.restype = ctypes.c_int
    lib.si_moe_scratch_bytes.argtypes = [vp, ctypes.c_int, i32, ctypes.POINTER(sz)]
    lib.si_moe_scratch_init.restype = ctypes.c_int
    lib.si_moe_scratch_init.argtypes = [vp, vp, sz, vp]
    for name in ("si_moe_forward_decode", "si_moe_forward_prefill", "si_moe_forward_decode_host"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [vp, ctypes.POINTER(si_moe_layer), vp, i32, vp, ctypes.POINTER(si_moe_route_out),
                      vp, sz, vp]
    lib.si_debug_decode_events.restype = ctypes.c_int
    lib.si_debug_decode_events.argtypes = [vp, ctypes.POINTER(si_moe_layer), vp, i32, vp,
                                           ctypes.POINTER(si_moe_route_out), vp, sz,
                                           ctypes.POINTER(vp), vp]
    lib.si_debug_prefill_events.argtypes = [vp, ctypes.POINTER(si_moe_layer), vp, i32, vp,
                                            ctypes.POINTER(si_moe_route_out), vp, sz,
                                            ctypes.POINTER(vp), vp]
    lib.si_debug_prefill_events.restype = ctypes.c_int
    lib.si_moe_forward_decode_noalloc.restype = ctypes.c_int
    lib.si_moe_forward_decode_noalloc.argtypes = [vp, ctypes.POINTER(si_moe_layer), vp, i32, vp,
                                                  ctypes.POINTER(si_moe_route_out), vp]
    lib.si_debug_plan_info.restype = ctypes.c_int
    lib.si_debug_plan_info.argtypes = [vp, ctypes.POINTER(i32), i32]
    lib.si_debug_decode_fused.restype = ctypes.c_int
    lib.si_debug_decode_fused.argtypes = [vp, i32]
    lib.si_moe_read_status.restype = ctypes.c_int
    lib.si_moe_read_status.argtypes = [vp, vp, vp]
    lib.si_debug_q4k_dequant.restype = ctypes.c_int
    lib.si_debug_q4k_dequant.argtypes = [vp, i64, vp, vp, vp]
    lib.si_debug_q4k_dequant_f16.restype = ctypes.c_int
    lib.si_debug_q4k_dequant_f16.argtypes = [vp, i64, vp, vp, vp]
    lib.si_debug_nvfp4_dequant_f16.restype = ctypes.c_int
    lib.si_debug_nvfp4_dequant_f16.argtypes = [vp, i64, ctypes.c_float, vp, vp]
    lib.si_debug_q5k_dequant_f16.restype = ctypes.c_int
    lib.si_debug_q5k_dequant_f16.argtypes = [vp, i64, vp, vp, vp]
    lib.si_moe_read_status_noalloc.restype = ctypes.c_int
    lib.si_moe_read_status_noalloc.argtypes = [vp]
    lib.si_debug_topk.restype = ctypes.c_int
    lib.si_debug_topk.argtypes = [vp, i32, ctypes.POINTER(si_moe_desc),
                                  ctypes.POINTER(si_moe_route_out), vp]
    _declare_kv(lib)
    if path is None:
        _lib = lib
    return lib


def _declare_kv(lib) -> None:
    """Argument and result types of include/si_kv.h's functions."""
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.si_kv_plan.restype = ctypes.c_int
    lib.si_kv_plan.argtypes = [ctypes.POINTER(si_kv_desc), ctypes.c_int, ctypes.POINTER(vp)]
    lib.si_kv_plan_destroy.restype = None
    lib.si_kv_plan_destroy.argtypes = [vp]
    lib.si_kv_scratch_bytes.restype = ctypes.c_int
    lib.si_kv_scratch_bytes.argtypes = [vp, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.si_kv_scratch_init.restype = ctypes.c_int
    lib.si_kv_scratch_init.argtypes = [vp, vp, sz, vp]
    cache, batch, rows = ctypes.POINTER(si_kv_cache), ctypes.POINTER(si_kv_batch), ctypes.POINTER(si_kv_rows)
    f32 = ctypes.c_float
    for name, args in (
            ("si_kv_append", [vp, cache, batch, rows, rows, vp, vp, sz, vp]),
            ("si_kv_read", [vp, cache, vp, i32, vp, vp, vp, sz, vp]),
            ("si_kv_attend", [vp, cache, batch, rows, rows, vp, f32, vp, sz, vp]),
            ("si_kv_weigh", [vp, cache, batch, rows, vp, vp, vp, i64, f32, f32, vp, sz, vp]),
            ("si_kv_evict", [vp, cache, batch, vp, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            ("si_kv_read_status", [vp, vp, vp])):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = args


def declared_symbols() -> list[str]:
    """Names of the functions include/si_moe.h and include/si_kv.h declare."""
    text = ""
    for path in (HEADER_PATH, KV_HEADER_PATH):
        with open(path) as f:
            text += f.read()
    return sorted(set(re.findall(r"^\s*(?:si_status|void|int|const char \*)\s*\*?\s*(si_\w+)\s*\(",
                                 text, flags=re.M)))


# ------------------------------------------------------------ marshalling
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "__array_interface__"):  # a numpy array in host memory
        return t.__array_interface__["data"][0]
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != SI_OK:
        raise SiError(status, where)


def si_status_string(status: int) -> str:
    return load_library().si_status_string(int(status)).decode()


def make_desc(hidden, intermediate, n_experts, top_k, max_tokens=1, wtype=SI_WTYPE_Q4_K, flags=0):
    return si_moe_desc(hidden, intermediate, n_experts, top_k, max_tokens, wtype, flags)


class Plan:
    """Owns an si_moe_plan_t (host memory only)."""

    def __init__(self, handle: int, desc: si_moe_desc):
        self.handle = handle
        self.desc = desc

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.si_moe_plan_destroy(self.handle)
            self.handle = None


def si_moe_plan(desc: si_moe_desc, cuda_device: int = 0) -> Plan:
    h = ctypes.c_void_p()
    _check(load_library().si_moe_plan(ctypes.byref(desc), cuda_device, ctypes.byref(h)), "si_moe_plan")
    return Plan(h.value, desc)


def si_moe_plan_status(desc: si_moe_desc, cuda_device: int = 0) -> int:
    """si_moe_plan's status without raising (frees a plan it made)."""
    lib = load_library()
    h = ctypes.c_void_p()
    st = lib.si_moe_plan(ctypes.byref(desc), cuda_device, ctypes.byref(h))
    if st == SI_OK:
        lib.si_moe_plan_destroy(h)
    return st


def si_moe_scratch_bytes(plan: Plan, mode: int, n_tokens: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().si_moe_scratch_bytes(plan.handle, mode, n_tokens, ctypes.byref(out)),
           "si_moe_scratch_bytes")
    return out.value


def si_moe_scratch_init(plan: Plan, scratch, stream=None):
    _check(load_library().si_moe_scratch_init(plan.handle, _ptr(scratch), scratch.numel() *
                                              scratch.element_size(), _stream(stream)),
           "si_moe_scratch_init")


def layer_struct(w_gate, w_up, w_down, router_w, router_bias=None, norm_weight=None,
                 norm_eps: float = 0.0, w_scale=None) -> si_moe_layer:
    return si_moe_layer(_ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(router_w), _ptr(router_bias),
                        _ptr(norm_weight), float(norm_eps), _ptr(w_scale))


def route_struct(topk_ids=None, topk_w=None, expert_counts=None, expert_offsets=None, perm=None,
                 logits=None) -> si_moe_route_out:
    return si_moe_route_out(_ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts), _ptr(expert_offsets),
                            _ptr(perm), _ptr(logits))


def _forward(fn_name, plan, layer, x, n_tokens, out, route_out, scratch, stream, raw_status):
    lib = load_library()
    ro = ctypes.byref(route_out) if route_out is not None else None
    nbytes = scratch.numel() * scratch.element_size()
    st = getattr(lib, fn_name)(plan.handle, ctypes.byref(layer), _ptr(x), int(n_tokens), _ptr(out), ro,
                               _ptr(scratch), nbytes, _stream(stream))
    if raw_status:
        return st
    _check(st, fn_name)
    return st


def si_moe_forward_decode(plan, layer: si_moe_layer, x, n_tokens, out, route_out=None, scratch=None,
                          stream=None, raw_status=False):
    return _forward("si_moe_forward_decode", plan, layer, x, n_tokens, out, route_out, scratch, stream,
                    raw_status)


def si_moe_forward_prefill(plan, layer: si_moe_layer, x, n_tokens, out, route_out=None, scratch=None,
                           stream=None, raw_status=False):
    return _forward("si_moe_forward_prefill", plan, layer, x, n_tokens, out, route_out, scratch, stream,
                    raw_status)


def si_moe_forward_decode_host(plan, layer: si_moe_layer, x_host, n_tokens, out_host, route_out=None,
                               scratch=None, stream=None, raw_status=False):
    """Decode with x and out in host memory (numpy arrays or CPU tensors);
    returns once out_host holds the result.  scratch:
    si_moe_scratch_bytes(plan, SI_MODE_DECODE_HOST, n)."""
    return _forward("si_moe_forward_decode_host", plan, layer, x_host, n_tokens, out_host, route_out, scratch,
                    stream, raw_status)


def si_moe_forward_decode_noalloc(plan, layer: si_moe_layer, x, n_tokens, out, route_out=None,
                                  stream=None, raw_status=False):
    """Decode with the library's built-in device scratch (no caller buffer,
    no allocation); see include/si_moe.h for its limits."""
    ro = ctypes.byref(route_out) if route_out is not None else None
    st = load_library().si_moe_forward_decode_noalloc(plan.handle, ctypes.byref(layer), _ptr(x),
                                                      int(n_tokens), _ptr(out), ro, _stream(stream))
    if not raw_status:
        _check(st, "si_moe_forward_decode_noalloc")
    return st


def si_debug_decode_events(plan, layer: si_moe_layer, x, n_tokens, out, route_out=None, scratch=None,
                           events=(None, None, None, None), stream=None):
    """Decode with torch.cuda.Event objects (enable_timing=True) recorded
    before/between/after the three kernels."""
    lib = load_library()
    ev = (ctypes.c_void_p * 4)(*[None if e is None else e.cuda_event for e in events])
    ro = ctypes.byref(route_out) if route_out is not None else None
    nbytes = scratch.numel() * scratch.element_size()
    _check(lib.si_debug_decode_events(plan.handle, ctypes.byref(layer), _ptr(x), int(n_tokens), _ptr(out),
                                      ro, _ptr(scratch), nbytes, ev, _stream(stream)),
           "si_debug_decode_events")


def si_debug_prefill_events(plan, layer: si_moe_layer, x, n_tokens, out, route_out=None, scratch=None,
                            events=(None, None, None, None, None), stream=None):
    """Prefill with torch.cuda.Event objects recorded before routing, before
    each GEMM, before the combine and after it."""
    lib = load_library()
    ev = (ctypes.c_void_p * 5)(*[None if e is None else e.cuda_event for e in events])
    ro = ctypes.byref(route_out) if route_out is not None else None
    nbytes = scratch.numel() * scratch.element_size()
    _check(lib.si_debug_prefill_events(plan.handle, ctypes.byref(layer), _ptr(x), int(n_tokens), _ptr(out),
                                       ro, _ptr(scratch), nbytes, ev, _stream(stream)),
           "si_debug_prefill_events")


def si_debug_plan_info(plan: Plan) -> dict:
    buf = (ctypes.c_int32 * 6)()
    load_library().si_debug_plan_info(plan.handle, buf, 6)
    keys = ("sm_count", "cluster_ok", "cluster_size", "clusters_resident", "clusters_needed", "smem_optin")
    return dict(zip(keys, list(buf)))


def si_debug_decode_fused(plan: Plan, n_tokens: int) -> int:
    return load_library().si_debug_decode_fused(plan.handle, int(n_tokens))


def si_moe_read_status(plan: Plan, scratch, stream=None) -> int:
    return load_library().si_moe_read_status(plan.handle, _ptr(scratch), _stream(stream))


def si_debug_q4k_dequant(blocks, n_blocks, out_f32=None, out_bf16=None, stream=None):
    _check(load_library().si_debug_q4k_dequant(_ptr(blocks), int(n_blocks), _ptr(out_f32),
                                               _ptr(out_bf16), _stream(stream)), "si_debug_q4k_dequant")


def si_debug_q4k_dequant_f16(blocks, n_blocks, out_f16, gamma=None, stream=None):
    _check(load_library().si_debug_q4k_dequant_f16(_ptr(blocks), int(n_blocks), _ptr(gamma), _ptr(out_f16),
                                                   _stream(stream)), "si_debug_q4k_dequant_f16")


def si_debug_nvfp4_dequant_f16(blocks, n_blocks, g, out_f16, stream=None):
    _check(load_library().si_debug_nvfp4_dequant_f16(_ptr(blocks), int(n_blocks), float(g), _ptr(out_f16),
                                                     _stream(stream)), "si_debug_nvfp4_dequant_f16")


def si_debug_q5k_dequant_f16(blocks, n_blocks, gamma, out_f16, stream=None):
    _check(load_library().si_debug_q5k_dequant_f16(_ptr(blocks), int(n_blocks), _ptr(gamma), _ptr(out_f16),
                                                   _stream(stream)), "si_debug_q5k_dequant_f16")


def si_moe_read_status_noalloc(stream=None) -> int:
    return load_library().si_moe_read_status_noalloc(_stream(stream))


def si_debug_topk(logits, n, desc: si_moe_desc, route_out: si_moe_route_out, stream=None):
    _check(load_library().si_debug_topk(_ptr(logits), int(n), ctypes.byref(desc),
                                        ctypes.byref(route_out), _stream(stream)), "si_debug_topk")


# ------------------------------------------------------------ attention block (include/si_kv.h)
_KV_CODES = {"int8": SI_KV_INT8, "e4m3": SI_KV_E4M3}
_KV_DTYPES = {"bf16": SI_KV_BF16, "f16": SI_KV_F16}


def make_kv_desc(n_heads, n_kv_heads, head_dim, page_tokens, code="int8", dtype="bf16") -> si_kv_desc:
    """code: "int8" or "e4m3"; dtype: "bf16" or "f16" (or the SI_KV_* numbers)."""
    return si_kv_desc(n_heads, n_kv_heads, head_dim, page_tokens, _KV_CODES.get(code, code),
                      _KV_DTYPES.get(dtype, dtype))


class KvPlan:
    """Owns an si_kv_plan_t (host memory only)."""

    def __init__(self, handle: int, desc: si_kv_desc):
        self.handle = handle
        self.desc = desc

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.si_kv_plan_destroy(self.handle)
            self.handle = None


def si_kv_plan(desc: si_kv_desc, cuda_device: int = 0) -> KvPlan:
    h = ctypes.c_void_p()
    _check(load_library().si_kv_plan(ctypes.byref(desc), cuda_device, ctypes.byref(h)), "si_kv_plan")
    return KvPlan(h.value, desc)


def si_kv_plan_status(desc: si_kv_desc, cuda_device: int = 0) -> int:
    """si_kv_plan's status without raising (frees a plan it made)."""
    lib = load_library()
    h = ctypes.c_void_p()
    st = lib.si_kv_plan(ctypes.byref(desc), cuda_device, ctypes.byref(h))
    if st == SI_OK:
        lib.si_kv_plan_destroy(h)
    return st


def kv_cache(k_codes, v_codes, k_scale, v_scale, k_tail, v_tail) -> si_kv_cache:
    """k_codes, v_codes [n_pages, Hkv, P, D] 8-bit; k_scale, v_scale [n_pages, Hkv] float32; k_tail, v_tail
    [n_slots, Hkv, 2P, D] 16-bit; all contiguous.  The structure keeps them alive."""
    tensors = (k_codes, v_codes, k_scale, v_scale, k_tail, v_tail)
    if not all(t.is_contiguous() for t in tensors):
        raise ValueError("the cache's tensors are contiguous")
    if [t.element_size() for t in tensors] != [1, 1, 4, 4, 2, 2]:
        raise ValueError("codes have 8 bits, scales 32 and the rings 16")
    n, heads, page, dim = k_codes.shape if k_codes.dim() == 4 else (0, 0, 0, 0)
    if not (v_codes.shape == k_codes.shape and tuple(k_scale.shape) == tuple(v_scale.shape) == (n, heads)
            and k_tail.shape == v_tail.shape and tuple(k_tail.shape[1:]) == (heads, 2 * page, dim)):
        raise ValueError("codes [n_pages, Hkv, P, D], scales [n_pages, Hkv], rings [n_slots, Hkv, 2P, D]")
    c = si_kv_cache(_ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), _ptr(k_tail), _ptr(v_tail),
                    k_codes.shape[0], k_tail.shape[0])
    c.held = (k_codes, v_codes, k_scale, v_scale, k_tail, v_tail)
    return c


def kv_batch(n_seqs, total_new, max_new, max_len, q_start, lens, page_table, slots=None) -> si_kv_batch:
    """q_start [n_seqs + 1], lens [n_seqs], page_table [n_seqs, columns] and slots [n_seqs]: int32 on the device
    (page_table's rows may be strided).  The structure keeps them alive."""
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table is [n_seqs, columns] with columns next to each other")
    if any("int32" not in str(t.dtype) for t in (q_start, lens, page_table, slots) if t is not None):
        raise ValueError("q_start, lens, page_table and slots are int32")
    for t, n in ((q_start, n_seqs + 1), (lens, n_seqs), (slots, n_seqs)):
        if t is not None and (t.dim() != 1 or t.shape[0] < n or not t.is_contiguous()):
            raise ValueError("q_start [n_seqs + 1], lens [n_seqs] and slots [n_seqs], each contiguous")
    if page_table.shape[0] < n_seqs:
        raise ValueError("page_table has a row for each sequence")
    stride = page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]
    b = si_kv_batch(n_seqs, total_new, max_new, max_len, _ptr(q_start), _ptr(lens), _ptr(page_table), _ptr(slots),
                    stride)
    b.held = (q_start, lens, page_table, slots)
    return b


def _rows(t) -> si_kv_rows:
    """A [rows, heads, D] tensor (or a view with D contiguous) as si_kv_rows."""
    strides = t.stride()
    if len(strides) != 3 or strides[2] != 1:
        raise ValueError("q, k, v and out are [rows, heads, D] with D contiguous")
    return si_kv_rows(t.data_ptr(), strides[0], strides[1])


def _sums(batch, acc_in, acc_out) -> int:
    """The one stride of both arrays of sums."""
    if not acc_out.is_contiguous() or acc_out.dim() != 3 or acc_out.shape[0] < batch.n_seqs:
        raise ValueError("acc_out is [n_seqs, Hkv, acc_stride], contiguous")
    if acc_in is not None and (acc_in.shape != acc_out.shape or not acc_in.is_contiguous()):
        raise ValueError("acc_in has acc_out's shape, contiguous")
    return acc_out.shape[2]


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _opt(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# A decode step makes a few of these calls for each layer, and on the host each should cost little more than
# its launch: the functions are looked up once, and the current stream is read without making a Stream object.
_kv_fns: dict = {}
_raw_stream = None


def _kv_fn(name):
    f = _kv_fns.get(name)
    if f is None:
        f = _kv_fns[name] = getattr(load_library(), name)
    return f


def _kv_stream(stream) -> Optional[int]:
    global _raw_stream
    if stream is not None:
        return _stream(stream)
    if _raw_stream is None:
        import torch
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
        torch.cuda.current_stream()  # (brings CUDA up)
        _raw_stream = (lambda: raw(device())) if raw else lambda: torch.cuda.current_stream().cuda_stream
    return _raw_stream()


def _kv_done(st, name, raw_status):
    if st != SI_OK and not raw_status:
        raise SiError(st, name)
    return st


def si_kv_scratch_bytes(plan: KvPlan, n_seqs, total_new, max_new, max_len) -> int:
    out = ctypes.c_size_t()
    _check(load_library().si_kv_scratch_bytes(plan.handle, n_seqs, total_new, max_new, max_len, ctypes.byref(out)),
           "si_kv_scratch_bytes")
    return out.value


def si_kv_scratch_init(plan: KvPlan, scratch, stream=None):
    _check(load_library().si_kv_scratch_init(plan.handle, _ptr(scratch), _nbytes(scratch), _stream(stream)),
           "si_kv_scratch_init")


def si_kv_append(plan, cache: si_kv_cache, batch: si_kv_batch, k, v, lens_out, scratch, stream=None,
                 raw_status=False):
    st = _kv_fn("si_kv_append")(plan.handle, cache, batch, _rows(k), _rows(v), lens_out.data_ptr(), scratch.data_ptr(),
                                _nbytes(scratch), _kv_stream(stream))
    return _kv_done(st, "si_kv_append", raw_status)


def si_kv_read(plan, cache: si_kv_cache, pages, n, k_out, v_out, scratch, stream=None, raw_status=False):
    st = _kv_fn("si_kv_read")(plan.handle, cache, pages.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(),
                              scratch.data_ptr(), _nbytes(scratch), _kv_stream(stream))
    return _kv_done(st, "si_kv_read", raw_status)


def si_kv_attend(plan, cache: si_kv_cache, batch: si_kv_batch, q, out, lse, sm_scale, scratch, stream=None,
                 raw_status=False):
    """lse: [rows, n_heads] float32, or None."""
    st = _kv_fn("si_kv_attend")(plan.handle, cache, batch, _rows(q), _rows(out), _opt(lse), sm_scale,
                                scratch.data_ptr(), _nbytes(scratch), _kv_stream(stream))
    return _kv_done(st, "si_kv_attend", raw_status)


def si_kv_weigh(plan, cache: si_kv_cache, batch: si_kv_batch, q, lse, acc_in, acc_out, decay, sm_scale, scratch,
                stream=None, raw_status=False):
    """acc_in (or None) and acc_out: [n_seqs, Hkv, acc_stride] float32, contiguous."""
    stride = _sums(batch, acc_in, acc_out)
    st = _kv_fn("si_kv_weigh")(plan.handle, cache, batch, _rows(q), lse.data_ptr(), _opt(acc_in), acc_out.data_ptr(),
                               stride, decay, sm_scale, scratch.data_ptr(), _nbytes(scratch), _kv_stream(stream))
    return _kv_done(st, "si_kv_weigh", raw_status)


def si_kv_evict(plan, cache: si_kv_cache, batch: si_kv_batch, acc_in, acc_out, budget, sink, recent, new_table,
                new_slots, keep, lens_out, scratch, stream=None, raw_status=False):
    """new_table [n_seqs, budget], keep [n_seqs, Hkv, budget] int32; acc_in, acc_out [n_seqs, Hkv, acc_stride];
    new_slots [n_seqs] int32 or None (the batch's own)."""
    stride = _sums(batch, acc_in, acc_out)
    if not (new_table.is_contiguous() and keep.is_contiguous() and new_table.shape[-1] == keep.shape[-1] == budget):
        raise ValueError("new_table [n_seqs, budget] and keep [n_seqs, Hkv, budget] are contiguous")
    st = _kv_fn("si_kv_evict")(plan.handle, cache, batch, acc_in.data_ptr(), acc_out.data_ptr(), stride, budget,
                               sink, recent, new_table.data_ptr(), _opt(new_slots), keep.data_ptr(),
                               lens_out.data_ptr(), scratch.data_ptr(), _nbytes(scratch), _kv_stream(stream))
    return _kv_done(st, "si_kv_evict", raw_status)


def si_kv_read_status(plan: KvPlan, scratch, stream=None) -> int:
    return load_library().si_kv_read_status(plan.handle, _ptr(scratch), _stream(stream))
