"""Python binding of libmoe_ffn.so (the GB300 routed FP4 MoE expert-FFN library).

Argument marshalling only: every function forwards to the C entry point of the
same name in include/moe_ffn.h.  Pointers may be given as ints or as torch
tensors (their data_ptr() is passed); streams as ints, torch streams or None
(the legacy default stream).  A nonzero return code raises MoeError.  There is
no fallback: if the CUDA library cannot be built or loaded, importing the
binding's functions raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_CUDA = -2
MOE_ERR_OOM = -3
MOE_ERR_UNSUPPORTED = -4
MOE_ERR_BAD_INDEX = -5
MOE_ERR_DEVICE_TIMEOUT = -6

MOE_ACT_BF16 = 0
MOE_ACT_E4M3_UE8M0_128 = 1
MOE_ACT_E2M1_UE8M0_32 = 2
MOE_OUT_BF16 = 0
MOE_OUT_F32 = 1
DEFAULT_GEMM_MIN_TOKENS = 16   # MOE_DEFAULT_GEMM_MIN_TOKENS

EXPORTS = [
    "moe_ffn_packed_expert_bytes", "moe_ffn_create",
    "moe_ffn_pack_expert", "moe_ffn_forward", "moe_ffn_forward_host", "moe_ffn_route",
    "moe_ffn_act_quant", "moe_stack_forward", "moe_stack_forward_host", "moe_ffn_profile_enable",
    "moe_ffn_profile_read",
    "moe_ffn_status", "moe_ffn_strerror", "moe_ffn_destroy", "moe_ffn_forward_noalloc",
    "moe_router_topk", "moe_router_select", "moe_batch_plan", "moe_batch_distinct",
    "moe_expert_cache_create", "moe_expert_cache_fetch", "moe_expert_cache_prefetch", "moe_expert_cache_slot",
    "moe_expert_cache_stats", "moe_expert_cache_destroy", "moe_ffn_test_set_wait", "moe_ffn_test_fail_allocs",
    "moe_ffn_test_copy_h",
    "moe_ffn_set_mma_kind", "moe_ffn_set_routing_wait",
    "moe_ffn_profile_layer_only",
    "moe_kv_pool_bytes", "moe_kv_create", "moe_kv_status", "moe_kv_destroy", "moe_rope_table", "moe_rope",
    "moe_kv_append", "moe_attn_decode", "moe_kv_copy_pages", "moe_kv_call",
    "moe_kv_pages_create", "moe_kv_pages_open", "moe_kv_pages_extend", "moe_kv_pages_fork", "moe_kv_pages_free",
    "moe_kv_pages_compact", "moe_kv_pages_row", "moe_kv_pages_length", "moe_kv_pages_free_pages",
    "moe_kv_pages_refs", "moe_kv_pages_destroy",
]

MOE_KV_BF16 = 0
MOE_KV_E4M3_UE8M0 = 1
MOE_ROPE_HALF = 0
MOE_ROPE_INTERLEAVED = 1
MOE_ROPE_SCALE_NONE = 0
MOE_ROPE_SCALE_LINEAR = 1
MOE_ROPE_SCALE_NTK = 2
MOE_ROPE_SCALE_YARN = 3

MOE_MMA_AUTO = 0
MOE_MMA_MXF4_PIECES = 1
MOE_MMA_MXF8F6F4 = 2

MOE_PHASE_PREP = 0
MOE_PHASE_GATE_UP = 1
MOE_PHASE_DOWN = 2
MOE_PHASE_ROUTE = 3
MOE_PHASE_ACT_QUANT = 4
MOE_PHASE_ROUTER = 5
MOE_NUM_PHASES = 8


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


class moe_ffn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_experts", "hidden", "inter", "topk", "max_tokens", "act_mode", "out_dtype",
        "gemm_min_tokens")]


class moe_expert_table(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_void_p)]


class moe_kv_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_q_heads", "num_kv_heads", "head_dim", "page_size", "num_pages", "max_seqs", "max_pages_per_seq",
        "kv_dtype", "out_dtype")]


class moe_kv_pool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")]


class moe_rope_desc(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("scale", ctypes.c_float)]


_lib = None


def build(force: bool = False) -> str:
    """Compile libmoe_ffn.so for sm_103a (in-tree)."""
    return _build.build(force=force)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        cfgp = ctypes.POINTER(moe_ffn_config)
        tblp = ctypes.POINTER(moe_expert_table)
        D, F, LL = ctypes.c_double, ctypes.c_float, ctypes.c_longlong
        kvcp, poolp, ropep = (ctypes.POINTER(t) for t in (moe_kv_config, moe_kv_pool, moe_rope_desc))
        sig = {
            "moe_ffn_packed_expert_bytes": (S, [cfgp]),
            "moe_ffn_create": (I, [ctypes.POINTER(P), cfgp, I]),
            "moe_ffn_pack_expert": (I, [P, P, P, P, P]),
            "moe_ffn_forward": (I, [P, P, P, P, tblp, P, I, P]),
            "moe_ffn_forward_host": (I, [P, P, P, P, tblp, P, I, P]),
            "moe_ffn_route": (I, [P, P, I, P, P, P, P, P]),
            "moe_ffn_act_quant": (I, [P, P, I, I, P, P, P]),
            "moe_stack_forward": (I, [P, P, tblp, P, P, I, I, P]),
            "moe_stack_forward_host": (I, [P, P, tblp, P, P, I, I, P]),
            "moe_ffn_profile_enable": (I, [P, I]),
            "moe_ffn_profile_read": (I, [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I)]),
            "moe_ffn_status": (I, [P, P]),
            "moe_ffn_strerror": (ctypes.c_char_p, [I]),
            "moe_ffn_destroy": (None, [P]),
            "moe_ffn_forward_noalloc": (I, [cfgp, I, P, P, P, tblp, P, I, P, P]),
            "moe_router_topk": (I, [P, P, P, I, P, P, P, P]),
            "moe_router_select": (I, [P, P, I, P, P, P]),
            "moe_batch_plan": (I, [P, I, I, I, I, I, P]),
            "moe_batch_distinct": (I, [P, P, I, I, I, I, I, P]),
            "moe_expert_cache_create": (I, [cfgp, I, P, I, ctypes.POINTER(P)]),
            "moe_expert_cache_fetch": (I, [P, P, I, P, tblp]),
            "moe_expert_cache_prefetch": (I, [P, P, I, P]),
            "moe_expert_cache_slot": (I, [P, I]),
            "moe_expert_cache_stats": (I, [P, ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_longlong),
                                           ctypes.POINTER(ctypes.c_longlong)]),
            "moe_expert_cache_destroy": (None, [P]),
            "moe_ffn_test_set_wait": (I, [P, ctypes.c_ulonglong, I]),
            "moe_ffn_test_fail_allocs": (None, [I]),
            "moe_ffn_test_copy_h": (I, [P, P, P, I, P]),
            "moe_ffn_set_mma_kind": (I, [P, I]),
            "moe_ffn_set_routing_wait": (I, [P, I]),
            "moe_ffn_profile_layer_only": (I, [P, I]),
            "moe_kv_pool_bytes": (I, [kvcp, ctypes.POINTER(S), ctypes.POINTER(S)]),
            "moe_kv_create": (I, [ctypes.POINTER(P), kvcp, I]),
            "moe_kv_status": (I, [P, P]),
            "moe_kv_destroy": (None, [P]),
            "moe_rope_table": (I, [I, D, I, D, I, P, ctypes.POINTER(F)]),
            "moe_rope": (I, [P, ropep, P, I, P, LL, P, P, LL, P, P]),
            "moe_kv_append": (I, [P, poolp, P, LL, P, LL, P, P, P, I, ropep, P, LL, P, P]),
            "moe_attn_decode": (I, [P, poolp, P, P, P, I, F, F, I, P, P, P]),
            "moe_kv_copy_pages": (I, [P, poolp, I, P, I, P]),
            "moe_kv_call": (I, [I, ctypes.c_char_p]),
            "moe_kv_pages_create": (I, [I, I, I, I, ctypes.POINTER(P)]),
            "moe_kv_pages_open": (I, [P, ctypes.POINTER(I)]),
            "moe_kv_pages_extend": (I, [P, I, I, P]),
            "moe_kv_pages_fork": (I, [P, I, ctypes.POINTER(I)]),
            "moe_kv_pages_free": (I, [P, I]),
            "moe_kv_pages_compact": (I, [P, P, I, ctypes.POINTER(I)]),
            "moe_kv_pages_row": (I, [P, I, P, I]),
            "moe_kv_pages_length": (I, [P, I]),
            "moe_kv_pages_free_pages": (I, [P]),
            "moe_kv_pages_refs": (I, [P, I]),
            "moe_kv_pages_destroy": (None, [P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def library_path() -> str:
    return os.path.abspath(_build.LIB)


def _p(x) -> int | None:
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, ctypes.Array):
        return ctypes.addressof(x)
    return int(x)


def _s(stream) -> int | None:
    if stream is None:
        return None
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _check(rc: int, where: str) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, where)


def strerror(code: int) -> str:
    return lib().moe_ffn_strerror(int(code)).decode()


moe_ffn_strerror = strerror


def config(num_experts, hidden, inter, topk, max_tokens, act_mode=MOE_ACT_BF16,
           out_dtype=MOE_OUT_F32, gemm_min_tokens=0) -> moe_ffn_config:
    return moe_ffn_config(num_experts, hidden, inter, topk, max_tokens, act_mode, out_dtype,
                          gemm_min_tokens)


def moe_ffn_packed_expert_bytes(cfg: moe_ffn_config) -> int:
    return lib().moe_ffn_packed_expert_bytes(ctypes.byref(cfg))


def moe_ffn_create(cfg: moe_ffn_config, device: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(lib().moe_ffn_create(ctypes.byref(h), ctypes.byref(cfg), int(device)), "moe_ffn_create")
    return h.value


def moe_ffn_pack_expert(h, canon_codes, canon_scales, packed, stream=None):
    _check(lib().moe_ffn_pack_expert(h, _p(canon_codes), _p(canon_scales), _p(packed), _s(stream)),
           "moe_ffn_pack_expert")


def expert_table(expert_ptrs) -> moe_expert_table:
    """expert_ptrs: a device array (e.g. a torch int64 tensor on the GPU)
    holding one device pointer per expert, each to a packed blob."""
    return moe_expert_table(_p(expert_ptrs))


def moe_ffn_forward(h, x, topk_idx, topk_w, table: moe_expert_table, y, T: int, stream=None):
    _check(lib().moe_ffn_forward(h, _p(x), _p(topk_idx), _p(topk_w), ctypes.byref(table), _p(y),
                                 int(T), _s(stream)), "moe_ffn_forward")


def moe_ffn_forward_host(h, x, topk_idx, topk_w, table: moe_expert_table, y, T: int, stream=None):
    _check(lib().moe_ffn_forward_host(h, _p(x), _p(topk_idx), _p(topk_w), ctypes.byref(table),
                                      _p(y), int(T), _s(stream)), "moe_ffn_forward_host")


def moe_ffn_route(h, topk_idx, T: int, counts, offsets, perm, inv, stream=None):
    _check(lib().moe_ffn_route(h, _p(topk_idx), int(T), _p(counts), _p(offsets), _p(perm), _p(inv),
                               _s(stream)), "moe_ffn_route")


def moe_ffn_act_quant(h, x, rows: int, n: int, codes, scales, stream=None):
    _check(lib().moe_ffn_act_quant(h, _p(x), int(rows), int(n), _p(codes), _p(scales), _s(stream)),
           "moe_ffn_act_quant")


def moe_stack_forward(h, x, tables, topk_idx, topk_w, L: int, T: int, stream=None):
    """tables: a sequence of moe_expert_table, one per layer."""
    arr = (moe_expert_table * len(tables))(*tables)
    _check(lib().moe_stack_forward(h, _p(x), arr, _p(topk_idx), _p(topk_w), int(L), int(T),
                                   _s(stream)), "moe_stack_forward")


def moe_stack_forward_host(h, x_host, tables, topk_idx_host, topk_w_host, L: int, T: int, stream=None):
    """Host buffers (CPU tensors or ints holding host addresses): x fp32 [T][H]
    updated in place, topk_idx int32 / topk_w fp32 [L][T][k]; waits for the
    stream.  tables: a sequence of moe_expert_table, one per layer."""
    arr = (moe_expert_table * len(tables))(*tables)
    _check(lib().moe_stack_forward_host(h, _p(x_host), arr, _p(topk_idx_host), _p(topk_w_host), int(L), int(T),
                                        _s(stream)), "moe_stack_forward_host")


def moe_ffn_profile_enable(h, on: bool = True) -> None:
    _check(lib().moe_ffn_profile_enable(h, 1 if on else 0), "moe_ffn_profile_enable")


def moe_ffn_profile_read(h):
    """Returns (ms, launches): per-phase summed milliseconds and launch counts."""
    ms = (ctypes.c_double * MOE_NUM_PHASES)()
    n = (ctypes.c_int * MOE_NUM_PHASES)()
    _check(lib().moe_ffn_profile_read(h, ms, n), "moe_ffn_profile_read")
    return list(ms), list(n)


def moe_ffn_profile_layer_only(h, on: bool = True) -> None:
    """Measurement mode: slot-major forwards launch the layer kernel alone,
    reusing the last full call's activation pieces (see include/moe_ffn.h)."""
    _check(lib().moe_ffn_profile_layer_only(h, 1 if on else 0), "moe_ffn_profile_layer_only")


def moe_ffn_set_mma_kind(h, kind: int) -> None:
    """The expert-major path's MMA in the E4M3 mode (MOE_MMA_*)."""
    _check(lib().moe_ffn_set_mma_kind(h, int(kind)), "moe_ffn_set_mma_kind")


def moe_ffn_set_routing_wait(h, on: int) -> None:
    """1: the layer's kernels read the routing only after their dependency wait."""
    _check(lib().moe_ffn_set_routing_wait(h, int(on)), "moe_ffn_set_routing_wait")


def moe_ffn_status(h, stream=None) -> int:
    """Returns the (cleared) sticky device status code; does not raise."""
    return lib().moe_ffn_status(h, _s(stream))


def moe_ffn_forward_noalloc(cfg: moe_ffn_config, device: int, x, topk_idx, topk_w,
                            table: moe_expert_table, y, T: int, status=None, stream=None):
    """The layer without a handle, using the library's fixed device scratch
    array instead of allocating (see include/moe_ffn.h)."""
    _check(lib().moe_ffn_forward_noalloc(ctypes.byref(cfg), int(device), _p(x), _p(topk_idx),
                                         _p(topk_w), ctypes.byref(table), _p(y), int(T),
                                         _p(status), _s(stream)), "moe_ffn_forward_noalloc")


def moe_ffn_test_copy_h(h, n: int, inter: int, stream=None):
    """Test hook: (h [n][inter] fp32, perm [n] int32) of the last kind::mxf8f6f4
    expert-major call, as device tensors (see include/moe_ffn.h)."""
    import torch

    hd = torch.empty((n, inter), dtype=torch.float32, device="cuda")
    pd = torch.empty(n, dtype=torch.int32, device="cuda")
    _check(lib().moe_ffn_test_copy_h(h, hd.data_ptr(), pd.data_ptr(), int(n), _s(stream)), "moe_ffn_test_copy_h")
    return hd, pd


def moe_ffn_test_set_wait(h, wait_ns: int, withhold: bool) -> None:
    """Test hook: bounded-wait limit of the slot-major kernel and the withheld
    partial sums that make its waits run out (see include/moe_ffn.h)."""
    _check(lib().moe_ffn_test_set_wait(h, int(wait_ns), 1 if withhold else 0), "moe_ffn_test_set_wait")


def moe_ffn_test_fail_allocs(n: int) -> None:
    """Test hook: the library's next n allocations fail as if out of memory."""
    lib().moe_ffn_test_fail_allocs(int(n))


def moe_ffn_destroy(h) -> None:
    lib().moe_ffn_destroy(h)


def moe_router_topk(h, x, router_w, T: int, topk_idx, topk_w, logits=None, stream=None):
    _check(lib().moe_router_topk(h, _p(x), _p(router_w), int(T), _p(logits), _p(topk_idx), _p(topk_w),
                                 _s(stream)), "moe_router_topk")


def moe_router_select(h, logits, T: int, topk_idx, topk_w, stream=None):
    _check(lib().moe_router_select(h, _p(logits), int(T), _p(topk_idx), _p(topk_w), _s(stream)),
           "moe_router_select")


def _host_i32(a, ndim):
    import numpy as np

    a = np.ascontiguousarray(a, dtype=np.int32)
    if a.ndim != ndim:
        raise ValueError(f"expected a {ndim}-d int32 array, got shape {a.shape}")
    return a


def moe_batch_plan(sig, E: int, B: int):
    """Batch order of N sequences from their signatures sig [N][L][topk] (host
    int32 expert ids, -1 for none): returns order [N] (host int32)."""
    import numpy as np

    sig = _host_i32(sig, 3)
    N, L, k = sig.shape
    order = np.empty(N, np.int32)
    _check(lib().moe_batch_plan(sig.ctypes.data, N, L, k, int(E), int(B), order.ctypes.data), "moe_batch_plan")
    return order


def moe_batch_distinct(routing, order, E: int, B: int):
    """Distinct experts per (batch, layer) [ceil(N/B)][L] of routing [N][L][topk]
    cut into batches of B in the given order."""
    import numpy as np

    routing = _host_i32(routing, 3)
    order = _host_i32(order, 1)
    N, L, k = routing.shape
    if order.size != N:
        raise ValueError("order must hold N entries")
    out = np.empty(((N + B - 1) // B, L), np.int32)
    _check(lib().moe_batch_distinct(routing.ctypes.data, order.ctypes.data, N, L, k, int(E), int(B),
                                    out.ctypes.data), "moe_batch_distinct")
    return out


# ------------------------------------------------------ host-resident experts

def moe_expert_cache_create(cfg, device: int, host_ptrs, slots: int):
    """Cache of `slots` device slots over experts whose packed blobs sit at the
    host addresses host_ptrs [E] (page-locked)."""
    arr = (ctypes.c_void_p * len(host_ptrs))(*[int(p) for p in host_ptrs])
    out = ctypes.c_void_p()
    _check(lib().moe_expert_cache_create(ctypes.byref(cfg), int(device), arr, int(slots), ctypes.byref(out)),
           "moe_expert_cache_create")
    return out.value


def moe_expert_cache_fetch(c, ids, stream=None):
    """Makes the experts of ids (host int32) resident; returns the layer's table."""
    import numpy as np

    ids = np.ascontiguousarray(ids, dtype=np.int32).reshape(-1)
    tbl = moe_expert_table()
    _check(lib().moe_expert_cache_fetch(c, ids.ctypes.data, ids.size, _s(stream), ctypes.byref(tbl)),
           "moe_expert_cache_fetch")
    return tbl


def moe_expert_cache_prefetch(c, ids, stream=None):
    import numpy as np

    ids = np.ascontiguousarray(ids, dtype=np.int32).reshape(-1)
    _check(lib().moe_expert_cache_prefetch(c, ids.ctypes.data, ids.size, _s(stream)), "moe_expert_cache_prefetch")


def moe_expert_cache_slot(c, expert: int) -> int:
    return int(lib().moe_expert_cache_slot(c, int(expert)))


def moe_expert_cache_stats(c):
    h, m, b = ctypes.c_longlong(), ctypes.c_longlong(), ctypes.c_longlong()
    _check(lib().moe_expert_cache_stats(c, ctypes.byref(h), ctypes.byref(m), ctypes.byref(b)),
           "moe_expert_cache_stats")
    return h.value, m.value, b.value


def moe_expert_cache_destroy(c) -> None:
    lib().moe_expert_cache_destroy(c)


# ------------------------------------------- key-value cache and its attention

def kv_config(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_seqs, max_pages_per_seq,
              kv_dtype=MOE_KV_BF16, out_dtype=MOE_OUT_BF16) -> moe_kv_config:
    return moe_kv_config(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_seqs, max_pages_per_seq,
                         kv_dtype, out_dtype)


def moe_kv_pool_bytes(cfg: moe_kv_config):
    """Bytes of one pool's k (and of its v), and of its k_scales (and of its v_scales)."""
    kv, sc = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_kv_pool_bytes(ctypes.byref(cfg), ctypes.byref(kv), ctypes.byref(sc)), "moe_kv_pool_bytes")
    return kv.value, sc.value


def moe_kv_create(cfg: moe_kv_config, device: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(lib().moe_kv_create(ctypes.byref(h), ctypes.byref(cfg), int(device)), "moe_kv_create")
    return h.value


def moe_kv_status(h, stream=None) -> int:
    """Returns the (cleared) sticky device status code; does not raise."""
    return lib().moe_kv_status(h, _s(stream))


def moe_kv_destroy(h) -> None:
    lib().moe_kv_destroy(h)


def kv_pool(k, v, k_scales=None, v_scales=None) -> moe_kv_pool:
    """One layer's pool (device memory; the scales for MOE_KV_E4M3_UE8M0 only)."""
    return moe_kv_pool(_p(k), _p(v), _p(k_scales), _p(v_scales))


def moe_rope_table(rot_dim: int, base: float, kind: int = MOE_ROPE_SCALE_NONE, factor: float = 1.0,
                   trained_len: int = 0):
    """(turns, scale): the frequencies as host uint64 [rot_dim / 2], to be
    copied to the device, and the factor on cos and sin."""
    import numpy as np

    turns = np.zeros(max(1, int(rot_dim) // 2), np.uint64)
    scale = ctypes.c_float()
    _check(lib().moe_rope_table(int(rot_dim), float(base), int(kind), float(factor), int(trained_len),
                                turns.ctypes.data, ctypes.byref(scale)), "moe_rope_table")
    return turns, scale.value


def rope(freqs, rot_dim: int, layout: int, scale: float = 1.0) -> moe_rope_desc:
    """freqs: moe_rope_table's turns in device memory."""
    return moe_rope_desc(_p(freqs), int(rot_dim), int(layout), float(scale))


# The calls of a decode step go through moe_kv_call: one ctypes argument where
# each of a dozen would cost a conversion.  Tensors and streams are read first as
# torch's; what is none (an address, a raw stream) takes _p and _s.
_ROPE, _APPEND, _ATTN, _COPY = struct.Struct("=3Qq Qq QQq QQ"), struct.Struct("=3QqQq 3Qq QQq QQ"), \
    struct.Struct("=5QqddqQQQ"), struct.Struct("=QQqQqQ")


def _kv_call(op: int, words: bytes, where: str) -> None:
    rc = (_lib or lib()).moe_kv_call(op, words)
    if rc:
        raise MoeError(rc, where)


def moe_rope(h, rope: moe_rope_desc, pos, T: int, q=None, q_out=None, k=None, k_out=None, ldq: int = 0, ldk: int = 0,
             stream=None):
    d = ctypes.addressof(rope)
    try:
        w = _ROPE.pack(h, d, pos.data_ptr(), T, 0 if q is None else q.data_ptr(), ldq, 0 if q_out is None else q_out.data_ptr(),
                       0 if k is None else k.data_ptr(), ldk, 0 if k_out is None else k_out.data_ptr(), stream.cuda_stream)
    except (AttributeError, struct.error):
        w = _ROPE.pack(h or 0, d, _p(pos) or 0, T, _p(q) or 0, ldq, _p(q_out) or 0, _p(k) or 0, ldk, _p(k_out) or 0,
                       _s(stream) or 0)
    _kv_call(0, w, "moe_rope")


def moe_kv_append(h, pool: moe_kv_pool, k, v, pos, page_table, T: int, seq=None, rope: moe_rope_desc | None = None,
                  q=None, q_out=None, ldq: int = 0, ldk: int = 0, ldv: int = 0, stream=None):
    p, d = ctypes.addressof(pool), 0 if rope is None else ctypes.addressof(rope)
    try:
        w = _APPEND.pack(h, p, k.data_ptr(), ldk, v.data_ptr(), ldv, pos.data_ptr(), 0 if seq is None else seq.data_ptr(),
                         page_table.data_ptr(), T, d, 0 if q is None else q.data_ptr(), ldq,
                         0 if q_out is None else q_out.data_ptr(), stream.cuda_stream)
    except (AttributeError, struct.error):
        w = _APPEND.pack(h or 0, p, _p(k) or 0, ldk, _p(v) or 0, ldv, _p(pos) or 0, _p(seq) or 0, _p(page_table) or 0, T, d,
                         _p(q) or 0, ldq, _p(q_out) or 0, _s(stream) or 0)
    _kv_call(1, w, "moe_kv_append")


def moe_attn_decode(h, pool: moe_kv_pool, q, seq_lens, page_table, B: int, out, lse=None, scale: float = 0.0,
                    softcap: float = 0.0, window: int = 0, stream=None):
    """scale 0: 1 / sqrt(head_dim)."""
    p = ctypes.addressof(pool)
    try:
        w = _ATTN.pack(h, p, q.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), B, scale, softcap, window,
                       out.data_ptr(), 0 if lse is None else lse.data_ptr(), stream.cuda_stream)
    except (AttributeError, struct.error):
        w = _ATTN.pack(h or 0, p, _p(q) or 0, _p(seq_lens) or 0, _p(page_table) or 0, B, scale, softcap, window,
                       _p(out) or 0, _p(lse) or 0, _s(stream) or 0)
    _kv_call(2, w, "moe_attn_decode")


def moe_kv_copy_pages(h, pools, pairs, n: int, stream=None):
    """pools: a sequence of moe_kv_pool, one per layer; pairs: device int32 [n][2] of (src, dst) page ids."""
    arr = ctypes.create_string_buffer(b"".join(pools))
    _kv_call(3, _COPY.pack(h or 0, ctypes.addressof(arr), len(pools), _p(pairs) or 0, n, _s(stream) or 0),
             "moe_kv_copy_pages")


def moe_kv_pages_create(num_pages: int, page_size: int, max_seqs: int, max_pages_per_seq: int) -> int:
    m = ctypes.c_void_p()
    _check(lib().moe_kv_pages_create(int(num_pages), int(page_size), int(max_seqs), int(max_pages_per_seq),
                                     ctypes.byref(m)), "moe_kv_pages_create")
    return m.value


def moe_kv_pages_open(m) -> int:
    s = ctypes.c_int()
    _check(lib().moe_kv_pages_open(m, ctypes.byref(s)), "moe_kv_pages_open")
    return s.value


def moe_kv_pages_extend(m, seq: int, tokens: int):
    """Returns the (src, dst) copy to make first, or None."""
    c = (ctypes.c_int32 * 2)()
    _check(lib().moe_kv_pages_extend(m, int(seq), int(tokens), c), "moe_kv_pages_extend")
    return (c[0], c[1]) if c[0] >= 0 else None


def moe_kv_pages_fork(m, parent: int) -> int:
    s = ctypes.c_int()
    _check(lib().moe_kv_pages_fork(m, int(parent), ctypes.byref(s)), "moe_kv_pages_fork")
    return s.value


def moe_kv_pages_free(m, seq: int) -> None:
    _check(lib().moe_kv_pages_free(m, int(seq)), "moe_kv_pages_free")


def moe_kv_pages_compact(m, max_pairs: int):
    """The copies to make, host int32 [n][2] of (src, dst)."""
    import numpy as np

    pairs = np.empty((max(0, int(max_pairs)), 2), np.int32)
    n = ctypes.c_int()
    _check(lib().moe_kv_pages_compact(m, pairs.ctypes.data, int(max_pairs), ctypes.byref(n)), "moe_kv_pages_compact")
    return pairs[:n.value]


def moe_kv_pages_row(m, seq: int, entries: int):
    """The sequence's page-table row, host int32 [entries], -1 behind its last page."""
    import numpy as np

    row = np.empty(max(0, int(entries)), np.int32)
    _check(lib().moe_kv_pages_row(m, int(seq), row.ctypes.data, row.size), "moe_kv_pages_row")
    return row


def _count(rc: int, where: str) -> int:
    if rc < 0:
        raise MoeError(rc, where)
    return rc


def moe_kv_pages_length(m, seq: int) -> int:
    return _count(lib().moe_kv_pages_length(m, int(seq)), "moe_kv_pages_length")


def moe_kv_pages_free_pages(m) -> int:
    return _count(lib().moe_kv_pages_free_pages(m), "moe_kv_pages_free_pages")


def moe_kv_pages_refs(m, page: int) -> int:
    return _count(lib().moe_kv_pages_refs(m, int(page)), "moe_kv_pages_refs")


def moe_kv_pages_destroy(m) -> None:
    lib().moe_kv_pages_destroy(m)
