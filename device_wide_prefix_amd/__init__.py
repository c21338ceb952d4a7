"""Python binding of libdws_scan.so, the gfx950 device-wide + prefix scan.

Argument marshalling only: every step of the scan runs in the library's HIP
kernels. torch supplies device buffers and the current stream. There is no CPU
fallback; if the library is not built, importing the binding's functions raises.

    scan_inclusive(x, out=None)            -> out
    scan_exclusive(x, out=None)            -> out      (out may be x: in place)
    scan_ex(x, out=None, exclusive=False, variant=SINGLE_PASS) -> out
    scan_opts(x, out=None, exclusive=False, variant=..., memory_order=...,
              tile_shape=0, nontemporal=None, tile_index=...) -> out
    scan_seeded(x, seed, exclusive=False, out=None) -> out  (seed: 1-element GPU tensor)
    reduce(x, out=None)                    -> 1-element GPU tensor holding the + of x
    scan_debug(x, out, tile_elems, ...)    -> descriptor words (numpy uint64)
    watchdog_trips()                       -> int
    selftest_wave(x)                       -> (incl, shift)
    pages_grow(refs, table, lengths, rows, new_lengths, page_tokens) -> granted
    pages_fork(refs, table, lengths, parents, children, page_tokens) -> (granted, src, dst, count)
    pages_free(refs, table, lengths, rows, page_tokens) -> freed
    pages_compact(refs, table)             -> (count, remap, src, dst, moves)
    pages_copy(pool, src, dst, count=None, page_dim=0) -> pool
    pages_append(keys, values, table, lengths, k, v, ..., q=None) -> q turned, or None (pools updated)
    pages_attention(q, keys, values, table, lengths, ...) -> out or (out, lse)
    beam_select(logits, scores, k=None, ..., rows=None) -> (scores, parents, tokens[, rows, src, dst])
    delta_rule(q, k, v, g, beta, ...)      -> out or (out, final_state)
    delta_rule_backward(d_out, q, ...)     -> (dq, dk, dv, dg, dbeta, d_initial_state)
    delta_rule_step(q, k, v, g, beta, state, slots=None, ...) -> out (state updated)
The C entry points take raw device pointers; the *_ptr functions expose them.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libdws_scan.so")

# dws_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_OVERLAP, ERR_HIP, ERR_OOM, ERR_MISALIGNED = range(7)
# dws_dtype
INT32, UINT32, FLOAT32, PAIR_I32_F32, PAIR_U32, FLOAT16, BFLOAT16 = 0, 1, 2, 3, 4, 5, 6
# dws_op
OP_SUM, OP_MAX, OP_MIN, OP_AFFINE, OP_SEGMENTED_SUM = 0, 1, 2, 3, 4
# dws_variant
SINGLE_PASS, REDUCE_THEN_SCAN, CHAINED, SCAN_THEN_PROPAGATE = 0, 1, 2, 3
# dws_memory_order
ORDER_RELAXED, ORDER_ACQ_REL = 0, 1
# dws_tile_index
TILE_AUTO, TILE_DRAWN, TILE_DISPATCH = 0, 1, 2
# dws_pred
PRED_EQ, PRED_NE, PRED_LT, PRED_LE, PRED_GT, PRED_GE = range(6)
# dws_options.nontemporal
NT_AUTO, NT_ON, NT_OFF = 0, 1, 2

EXPORTED_SYMBOLS = (
    "scan_inclusive", "scan_exclusive", "dws_scan_ex", "dws_scan_opts", "dws_status_string", "dws_version",
    "dws_num_tile_shapes", "dws_tile_elems", "dws_tile_threads", "dws_reserve",
    "dws_release_workspaces", "dws_watchdog_trips", "dws_scan_debug", "dws_selftest_wave",
    "dws_scan_profiled", "dws_select_flagged", "dws_scan_op", "dws_partition_flagged", "dws_reduce_by_key",
    "dws_run_length_encode", "dws_device_memory_info", "dws_scan_noalloc", "dws_scan_plan", "dws_scan_seeded",
    "dws_reduce", "dws_scan_op_seeded", "dws_reduce_op", "dws_select_if", "dws_partition_if",
    "dws_delta_rule_workspace", "dws_delta_rule", "dws_delta_rule_backward", "dws_delta_rule_step",
    "dws_pages_workspace", "dws_pages_grow", "dws_pages_fork", "dws_pages_free", "dws_pages_compact", "dws_pages_copy",
    "dws_pages_append", "dws_pages_attention_workspace", "dws_pages_attention", "dws_beam_select_workspace",
    "dws_beam_select",
)


class ScanError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class DwsOptions(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("memory_order", ctypes.c_int),
                ("tile_shape", ctypes.c_int), ("nontemporal", ctypes.c_int),
                ("tile_index", ctypes.c_int)]


class LaunchPlan(ctypes.Structure):
    """dws_launch_plan: what a single-pass or chained call would launch."""
    _fields_ = [("threads", ctypes.c_uint), ("tile_elems", ctypes.c_uint), ("num_tiles", ctypes.c_uint),
                ("tile_index", ctypes.c_int), ("nontemporal", ctypes.c_int), ("pause_units", ctypes.c_int)]


class Rows(ctypes.Structure):
    """dws_rows: a (tokens, heads, dim) array."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class DeltaRuleArgs(ctypes.Structure):
    """dws_delta_rule_args."""
    _fields_ = ([(x, ctypes.c_longlong) for x in ("tokens", "n_seqs")] + [("d_offsets", ctypes.c_void_p)] +
                [(x, ctypes.c_int) for x in ("heads_qk", "heads_v", "dim_k", "dim_v", "dtype", "g_dtype", "beta_dtype")] +
                [("scale", ctypes.c_float)] + [(x, Rows) for x in ("q", "k", "v", "g", "beta", "out")] +
                [(x, ctypes.c_void_p) for x in ("d_initial_state", "d_final_state", "d_slots")] +
                [("n_states", ctypes.c_longlong), ("out_grad", Rows), ("d_final_grad", ctypes.c_void_p)] +
                [(x, Rows) for x in ("q_grad", "k_grad", "v_grad", "g_grad", "beta_grad")] +
                [("d_initial_grad", ctypes.c_void_p), ("zero_rest", ctypes.c_int), ("options", ctypes.c_int),
                 ("d_workspace", ctypes.c_void_p),
                 ("workspace_bytes", ctypes.c_size_t)])


class PageCache(ctypes.Structure):
    """dws_page_cache."""
    _fields_ = [("d_refs", ctypes.c_void_p), ("n_pages", ctypes.c_longlong), ("d_table", ctypes.c_void_p),
                ("n_rows", ctypes.c_longlong), ("max_pages", ctypes.c_longlong), ("d_lengths", ctypes.c_void_p),
                ("page_tokens", ctypes.c_longlong)]


class PagePool(ctypes.Structure):
    """dws_page_pool: the keys or values of a pool's pages."""
    _fields_ = [("data", ctypes.c_void_p)] + [(x, ctypes.c_longlong) for x in ("page_stride", "token_stride", "head_stride")]


class KvCache(ctypes.Structure):
    """dws_kv_cache."""
    _fields_ = ([("keys", PagePool), ("values", PagePool), ("d_table", ctypes.c_void_p), ("d_lengths", ctypes.c_void_p)] +
                [(x, ctypes.c_longlong) for x in ("n_pages", "n_rows", "max_pages", "page_tokens")] +
                [(x, ctypes.c_int) for x in ("heads", "dim_k", "dim_v", "dtype")])


class PageSeqs(ctypes.Structure):
    """dws_page_seqs."""
    _fields_ = [("tokens", ctypes.c_longlong), ("n", ctypes.c_longlong), ("d_offsets", ctypes.c_void_p),
                ("d_rows", ctypes.c_void_p)]


class PagesAppendArgs(ctypes.Structure):
    """dws_pages_append_args."""
    _fields_ = ([("cache", KvCache), ("seqs", PageSeqs)] +
                [(x, ctypes.c_void_p) for x in ("d_granted", "d_positions", "d_freqs")] +
                [(x, ctypes.c_int) for x in ("pairs", "adjacent", "heads_q", "zero_rest")] +
                [(x, Rows) for x in ("k", "v", "q", "q_out")])


class PagesAttentionArgs(ctypes.Structure):
    """dws_pages_attention_args."""
    _fields_ = [("cache", KvCache), ("seqs", PageSeqs), ("heads_q", ctypes.c_int), ("scale", ctypes.c_float),
                ("n_groups", ctypes.c_longlong), ("d_groups", ctypes.c_void_p), ("d_shared", ctypes.c_void_p),
                ("zero_rest", ctypes.c_int), ("options", ctypes.c_int), ("q", Rows), ("out", Rows), ("d_lse", ctypes.c_void_p),
                ("d_workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class BeamArgs(ctypes.Structure):
    """dws_beam_args."""
    _fields_ = ([("d_logits", ctypes.c_void_p)] +
                [(x, ctypes.c_longlong) for x in ("batch", "beams", "vocab", "batch_stride", "beam_stride")] +
                [("dtype", ctypes.c_int), ("k", ctypes.c_int), ("d_scores", ctypes.c_void_p), ("d_finished", ctypes.c_void_p),
                 ("end_token", ctypes.c_longlong)] +
                [(x, ctypes.c_void_p) for x in ("d_rows", "d_out_scores", "d_parents", "d_tokens", "d_out_rows", "d_src",
                                                "d_dst", "d_workspace")] + [("workspace_bytes", ctypes.c_size_t)])


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load libdws_scan.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m device_wide_prefix_amd.build` "
                          "(or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, ci, cu = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint
    for name in ("scan_inclusive", "scan_exclusive"):
        f = getattr(lib, name)
        f.argtypes = [vp, vp, sz, ci, vp]
        f.restype = ci
    lib.dws_scan_ex.argtypes = [vp, vp, sz, ci, ci, ci, vp]
    lib.dws_scan_ex.restype = ci
    lib.dws_scan_opts.argtypes = [vp, vp, sz, ci, ci, ctypes.POINTER(DwsOptions), vp]
    lib.dws_scan_opts.restype = ci
    lib.dws_scan_noalloc.argtypes = [vp, vp, sz, ci, ci, vp]
    lib.dws_scan_noalloc.restype = ci
    lib.dws_scan_plan.argtypes = [vp, vp, sz, ci, ci, ctypes.POINTER(DwsOptions), ctypes.POINTER(LaunchPlan)]
    lib.dws_scan_plan.restype = ci
    lib.dws_scan_seeded.argtypes = [vp, vp, sz, ci, ci, vp, vp]
    lib.dws_scan_seeded.restype = ci
    lib.dws_reduce.argtypes = [vp, sz, ci, vp, vp]
    lib.dws_reduce.restype = ci
    lib.dws_scan_op_seeded.argtypes = [vp, vp, sz, ci, ci, ci, vp, vp]
    lib.dws_scan_op_seeded.restype = ci
    lib.dws_reduce_op.argtypes = [vp, sz, ci, ci, vp, vp]
    lib.dws_reduce_op.restype = ci
    for name in ("dws_select_if", "dws_partition_if"):
        f = getattr(lib, name)
        f.argtypes = [vp, vp, sz, ci, ci, vp, vp, vp]
        f.restype = ci
    lib.dws_status_string.argtypes = [ci]
    lib.dws_status_string.restype = ctypes.c_char_p
    lib.dws_version.restype = ci
    lib.dws_num_tile_shapes.restype = ci
    lib.dws_tile_elems.argtypes = [ci, sz, ci]
    lib.dws_tile_elems.restype = cu
    lib.dws_tile_threads.argtypes = [ci, sz, ci]
    lib.dws_tile_threads.restype = cu
    lib.dws_reserve.argtypes = [sz, vp]
    lib.dws_reserve.restype = ci
    lib.dws_release_workspaces.restype = ci
    lib.dws_watchdog_trips.argtypes = [ctypes.POINTER(ctypes.c_ulonglong)]
    lib.dws_watchdog_trips.restype = ci
    lib.dws_device_memory_info.argtypes = [ctypes.POINTER(ctypes.c_int)] * 3
    lib.dws_device_memory_info.restype = ci
    lib.dws_scan_debug.argtypes = [vp, vp, sz, ci, ci, ci, cu, cu, cu, cu,
                                   ctypes.POINTER(ctypes.c_ulonglong), vp]
    lib.dws_scan_debug.restype = ci
    lib.dws_scan_profiled.argtypes = [vp, vp, sz, ci, ci, vp, sz, ctypes.POINTER(cu), vp]
    lib.dws_scan_profiled.restype = ci
    lib.dws_scan_op.argtypes = [vp, vp, sz, ci, ci, ci, vp]
    lib.dws_scan_op.restype = ci
    lib.dws_partition_flagged.argtypes = [vp, vp, vp, sz, ci, vp, vp]
    lib.dws_partition_flagged.restype = ci
    lib.dws_reduce_by_key.argtypes = [vp, vp, vp, vp, sz, ci, vp, vp]
    lib.dws_reduce_by_key.restype = ci
    lib.dws_run_length_encode.argtypes = [vp, vp, vp, sz, vp, vp]
    lib.dws_run_length_encode.restype = ci
    lib.dws_select_flagged.argtypes = [vp, vp, vp, sz, ci, vp, vp]
    lib.dws_select_flagged.restype = ci
    # (dws_delta_rule_args by address: a DeltaRuleArgs or its bytes)
    lib.dws_delta_rule_workspace.argtypes = [vp, ci, ctypes.POINTER(sz)]
    lib.dws_delta_rule_workspace.restype = ci
    for name in ("dws_delta_rule", "dws_delta_rule_backward", "dws_delta_rule_step"):
        f = getattr(lib, name)
        f.argtypes = [vp, vp]
        f.restype = ci
    # (dws_page_cache likewise: a PageCache or its bytes)
    pc, ll = vp, ctypes.c_longlong
    for name, args in (("workspace", [pc, ll, ctypes.POINTER(sz)]), ("grow", [pc, vp, vp, ll, vp, vp, sz, vp]),
                       ("fork", [pc, vp, vp, ll, vp, vp, vp, vp, vp, sz, vp]), ("free", [pc, vp, ll, vp, vp, sz, vp]),
                       ("compact", [pc, vp, vp, vp, vp, vp, vp, sz, vp]),
                       ("copy", [vp, ll, ll, ll, ll, vp, vp, ll, vp, vp])):
        f = getattr(lib, "dws_pages_" + name)
        f.argtypes = args
        f.restype = ci
    # (and the arguments of the calls on cached keys and values and of the beam selection)
    for name in ("dws_pages_append", "dws_pages_attention", "dws_beam_select"):
        f = getattr(lib, name)
        f.argtypes = [vp, vp]
        f.restype = ci
    for name in ("dws_pages_attention_workspace", "dws_beam_select_workspace"):
        f = getattr(lib, name)
        f.argtypes = [vp, ctypes.POINTER(sz)]
        f.restype = ci
    lib.dws_selftest_wave.argtypes = [vp, vp, vp, sz, ci, vp]
    lib.dws_selftest_wave.restype = ci
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().dws_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != OK:
        raise ScanError(status, what)


# ---- raw-pointer entry points (same names as the C ABI, plus _ptr) --------

def scan_inclusive_ptr(d_in: int, d_out: int, n: int, dtype: int, stream: int = 0) -> int:
    return load_library().scan_inclusive(d_in, d_out, n, dtype, stream)


def scan_exclusive_ptr(d_in: int, d_out: int, n: int, dtype: int, stream: int = 0) -> int:
    return load_library().scan_exclusive(d_in, d_out, n, dtype, stream)


def scan_ex_ptr(d_in: int, d_out: int, n: int, dtype: int, exclusive: bool, variant: int,
                stream: int = 0) -> int:
    return load_library().dws_scan_ex(d_in, d_out, n, dtype, int(bool(exclusive)), int(variant), stream)


def scan_noalloc_ptr(d_in: int, d_out: int, n: int, dtype: int, exclusive: bool, stream: int = 0) -> int:
    return load_library().dws_scan_noalloc(d_in, d_out, n, dtype, int(bool(exclusive)), stream)


def scan_seeded_ptr(d_in: int, d_out: int, n: int, dtype: int, exclusive: bool, d_seed: int,
                    stream: int = 0) -> int:
    return load_library().dws_scan_seeded(d_in, d_out, n, dtype, int(bool(exclusive)), d_seed, stream)


def reduce_ptr(d_in: int, n: int, dtype: int, d_total: int, stream: int = 0) -> int:
    return load_library().dws_reduce(d_in, n, dtype, d_total, stream)


def scan_opts_ptr(d_in: int, d_out: int, n: int, dtype: int, exclusive: bool,
                  options: DwsOptions | None, stream: int = 0) -> int:
    opt = ctypes.byref(options) if options is not None else None
    return load_library().dws_scan_opts(d_in, d_out, n, dtype, int(bool(exclusive)), opt, stream)


def scan_plan_ptr(d_in: int, d_out: int, n: int, dtype: int, exclusive: bool,
                  options: DwsOptions | None = None) -> tuple[int, LaunchPlan]:
    """dws_scan_plan: (status, plan) for what dws_scan_opts would launch with
    these arguments; the pointers are only compared and checked for alignment."""
    plan = LaunchPlan()
    opt = ctypes.byref(options) if options is not None else None
    st = load_library().dws_scan_plan(d_in, d_out, n, dtype, int(bool(exclusive)), opt, ctypes.byref(plan))
    return st, plan


# ---- torch-tensor entry points --------------------------------------------

def _dtype_code(t) -> int:
    import torch
    codes = {torch.int32: INT32, torch.float32: FLOAT32}
    u32 = getattr(torch, "uint32", None)
    if u32 is not None:
        codes[u32] = UINT32
    if t.dtype not in codes:
        raise TypeError(f"scan supports int32, uint32 and float32 tensors, got {t.dtype}")
    return codes[t.dtype]


def _prepare(x, out):
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("scan expects a GPU tensor (there is no CPU path)")
    if not x.is_contiguous():
        raise ValueError("input tensor must be contiguous")
    code = _dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.numel() != x.numel() or not out.is_contiguous() or \
            out.device != x.device:
        raise ValueError("out must be a contiguous tensor with the dtype, size and device of x")
    return code, out


def _stream(x, stream):
    import torch
    if stream is not None:
        return int(stream)
    return int(torch.cuda.current_stream(x.device).cuda_stream)


def scan_inclusive(x, out=None, stream=None):
    """Inclusive + scan of a contiguous GPU tensor; returns ``out``."""
    code, out = _prepare(x, out)
    with _device_of(x):
        _check(scan_inclusive_ptr(x.data_ptr(), out.data_ptr(), x.numel(), code, _stream(x, stream)),
               "scan_inclusive")
    return out


def scan_exclusive(x, out=None, stream=None):
    """Exclusive + scan of a contiguous GPU tensor; returns ``out`` (may be x)."""
    code, out = _prepare(x, out)
    with _device_of(x):
        _check(scan_exclusive_ptr(x.data_ptr(), out.data_ptr(), x.numel(), code, _stream(x, stream)),
               "scan_exclusive")
    return out


def scan_ex(x, out=None, exclusive=False, variant=SINGLE_PASS, stream=None):
    """Scan by the global strategy ``variant`` (dws_variant); returns ``out``."""
    code, out = _prepare(x, out)
    with _device_of(x):
        _check(scan_ex_ptr(x.data_ptr(), out.data_ptr(), x.numel(), code, exclusive, variant,
                           _stream(x, stream)), "dws_scan_ex")
    return out


def scan_opts(x, out=None, exclusive=False, variant=SINGLE_PASS, memory_order=ORDER_RELAXED,
              tile_shape=0, nontemporal=None, tile_index=TILE_AUTO, stream=None):
    """Scan with explicit options (variant, descriptor memory order, tile shape,
    non-temporal loads: None for the library's choice, True or False to force
    them on or off; tile index source); returns ``out``."""
    code, out = _prepare(x, out)
    nt = NT_AUTO if nontemporal is None else (NT_ON if nontemporal else NT_OFF)
    opt = DwsOptions(int(variant), int(memory_order), int(tile_shape), nt, int(tile_index))
    with _device_of(x):
        _check(scan_opts_ptr(x.data_ptr(), out.data_ptr(), x.numel(), code, exclusive, opt,
                             _stream(x, stream)), "dws_scan_opts")
    return out


def scan_seeded(x, seed, exclusive=False, out=None, stream=None):
    """Scan of x with the 1-element GPU tensor ``seed`` (dtype of x) as the
    prefix of the whole array (dws_scan_seeded); returns ``out`` (may be x)."""
    import torch
    code, out = _prepare(x, out)
    if not isinstance(seed, torch.Tensor) or seed.device != x.device or seed.dtype != x.dtype or \
            seed.numel() != 1:
        raise ValueError("seed must be a 1-element tensor with the dtype and device of x")
    with _device_of(x):
        _check(scan_seeded_ptr(x.data_ptr(), out.data_ptr(), x.numel(), code, exclusive, seed.data_ptr(),
                               _stream(x, stream)), "dws_scan_seeded")
    return out


def reduce(x, out=None, stream=None):
    """+ of every element of x (dws_reduce) into the 1-element GPU tensor
    ``out`` (a new one by default); returns ``out``."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("reduce expects a GPU tensor (there is no CPU path)")
    if not x.is_contiguous():
        raise ValueError("input tensor must be contiguous")
    code = _dtype_code(x)
    if out is None:
        out = torch.empty(1, dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.numel() != 1 or out.device != x.device:
        raise ValueError("out must be a 1-element tensor with the dtype and device of x")
    with _device_of(x):
        _check(reduce_ptr(x.data_ptr(), x.numel(), code, out.data_ptr(), _stream(x, stream)), "dws_reduce")
    return out


def scan_debug(x, out, tile_elems, exclusive=False, variant=SINGLE_PASS, delay_every=0,
               delay_phase=0, delay_ticks=0, want_descriptors=True, stream=None):
    """Run the protocol-inspection kernel (one wavefront per tile of
    ``tile_elems`` <= 64 elements). Returns the final descriptor words as a numpy
    uint64 array (synchronises) or None."""
    import numpy as np
    code, out = _prepare(x, out)
    n = x.numel()
    num_tiles = max(1, -(-n // int(tile_elems))) if n else 0
    desc = None
    ptr = None
    if want_descriptors and n:
        desc = np.zeros(num_tiles, dtype=np.uint64)
        ptr = desc.ctypes.data_as(ctypes.POINTER(ctypes.c_ulonglong))
    with _device_of(x):
        _check(load_library().dws_scan_debug(x.data_ptr(), out.data_ptr(), n, code, int(bool(exclusive)),
                                             int(variant), int(tile_elems), int(delay_every),
                                             int(delay_phase), int(delay_ticks), ptr, _stream(x, stream)),
               "dws_scan_debug")
    return desc


STAMPS_PER_TILE = 5
STAMP_NAMES = ("start", "tile_index_known", "aggregate_published", "prefix_known", "stores_issued")


def profiled_num_tiles(n: int) -> int:
    t = ctypes.c_uint(0)
    _check(load_library().dws_scan_profiled(None, None, int(n), INT32, 0, None, 0, ctypes.byref(t), None),
           "dws_scan_profiled")
    return int(t.value)


def scan_profiled(x, out=None, exclusive=False, stream=None):
    """Instrumented single-pass scan. Returns (out, stamps) where stamps is a
    (num_tiles, 5) int64 GPU tensor of 100 MHz real-time counter values:
    start, tile index known, aggregate published, prefix known, stores issued."""
    import torch
    code, out = _prepare(x, out)
    tiles = profiled_num_tiles(x.numel())
    stamps = torch.zeros((max(tiles, 1), STAMPS_PER_TILE), dtype=torch.int64, device=x.device)
    t = ctypes.c_uint(0)
    with _device_of(x):
        _check(load_library().dws_scan_profiled(x.data_ptr(), out.data_ptr(), x.numel(), code, int(bool(exclusive)),
                                                stamps.data_ptr(), stamps.numel(), ctypes.byref(t),
                                                _stream(x, stream)), "dws_scan_profiled")
    return out, stamps[:tiles]


def scan_op_ptr(d_in: int, d_out: int, n: int, dtype: int, op: int, exclusive: bool, stream: int = 0) -> int:
    return load_library().dws_scan_op(d_in, d_out, n, dtype, op, int(bool(exclusive)), stream)


def scan_op_seeded_ptr(d_in: int, d_out: int, n: int, dtype: int, op: int, exclusive: bool, d_seed: int,
                       stream: int = 0) -> int:
    return load_library().dws_scan_op_seeded(d_in, d_out, n, dtype, op, int(bool(exclusive)), d_seed, stream)


def select_if_ptr(d_in: int, d_out: int, n: int, dtype: int, pred: int, threshold, d_count: int,
                  stream: int = 0, partition: bool = False) -> int:
    """dws_select_if (dws_partition_if with partition=True); ``threshold`` is a
    Python number converted to dtype on the host."""
    import numpy as np
    np_t = {INT32: np.int32, UINT32: np.uint32, FLOAT32: np.float32}.get(int(dtype), np.uint32)
    buf = np.array([threshold], dtype=np_t)
    f = load_library().dws_partition_if if partition else load_library().dws_select_if
    return f(d_in, d_out, n, dtype, int(pred), buf.ctypes.data, d_count, stream)


def reduce_op_ptr(d_in: int, n: int, dtype: int, op: int, d_total: int, stream: int = 0) -> int:
    return load_library().dws_reduce_op(d_in, n, dtype, op, d_total, stream)


def reduce_op(x, op, dtype=None, out=None, stream=None):
    """Combination under ``op`` of every element of x in order (dws_reduce_op)
    into ``out``: a GPU tensor of one element's bytes (a new int32 tensor of 1
    or 2 words by default, bits as for scan_op). Returns ``out``."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("reduce_op expects a GPU tensor (there is no CPU path)")
    if not x.is_contiguous():
        raise ValueError("input tensor must be contiguous")
    if dtype is None:
        dtype = _dtype_code(x)
    esize = 8 if dtype in (PAIR_I32_F32, PAIR_U32) else 4
    nbytes = x.numel() * x.element_size()
    if nbytes % esize:
        raise ValueError(f"tensor of {nbytes} bytes does not hold whole {esize}-byte elements")
    if out is None:
        out = torch.empty(esize // 4, dtype=torch.int32, device=x.device)
    if out.numel() * out.element_size() != esize or not out.is_contiguous() or out.device != x.device:
        raise ValueError(f"out must be a contiguous tensor of {esize} bytes on the device of x")
    with _device_of(x):
        _check(reduce_op_ptr(x.data_ptr(), nbytes // esize, int(dtype), int(op), out.data_ptr(),
                             _stream(x, stream)), "dws_reduce_op")
    return out


def scan_op(x, op, dtype=None, exclusive=False, out=None, stream=None, seed=None):
    """Scan of a contiguous GPU tensor under a generic operator (OP_*).

    For the 32-bit types dtype defaults from the tensor. Pair types
    (PAIR_I32_F32, PAIR_U32) take any contiguous tensor whose bytes hold the
    pairs, e.g. an (n, 2) int32 tensor of bits; n is its byte size / 8.
    ``seed``: a GPU tensor on x's device whose bytes hold one element, the
    initial value before the whole array (dws_scan_op_seeded).
    Returns ``out`` (same shape and dtype as x; may be x)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("scan_op expects a GPU tensor (there is no CPU path)")
    if not x.is_contiguous():
        raise ValueError("input tensor must be contiguous")
    if dtype is None:
        dtype = _dtype_code(x)
    esize = 8 if dtype in (PAIR_I32_F32, PAIR_U32) else 4
    nbytes = x.numel() * x.element_size()
    if nbytes % esize:
        raise ValueError(f"tensor of {nbytes} bytes does not hold whole {esize}-byte elements")
    if out is None:
        out = torch.empty_like(x)
    if out.numel() * out.element_size() != nbytes or not out.is_contiguous() or out.device != x.device:
        raise ValueError("out must be a contiguous tensor of the same byte size on the device of x")
    if seed is not None:
        if not isinstance(seed, torch.Tensor) or seed.device != x.device or not seed.is_contiguous() or \
                seed.numel() * seed.element_size() != esize:
            raise ValueError(f"seed must be a contiguous tensor of {esize} bytes on the device of x")
        with _device_of(x):
            _check(scan_op_seeded_ptr(x.data_ptr(), out.data_ptr(), nbytes // esize, int(dtype), int(op),
                                      exclusive, seed.data_ptr(), _stream(x, stream)), "dws_scan_op_seeded")
        return out
    with _device_of(x):
        _check(scan_op_ptr(x.data_ptr(), out.data_ptr(), nbytes // esize, int(dtype), int(op), exclusive,
                           _stream(x, stream)), "dws_scan_op")
    return out


def select_flagged_ptr(d_in: int, d_flags: int, d_out: int, n: int, dtype: int, d_count: int,
                      stream: int = 0) -> int:
    return load_library().dws_select_flagged(d_in, d_flags, d_out, n, dtype, d_count, stream)


def select_flagged(x, flags, out=None, count=None, stream=None):
    """Stream compaction: the elements of x whose int32 flag is non-zero, in
    order, written to out[:count]. Returns (out, count) with count a one-element
    int64 GPU tensor (no synchronisation). out may be x (in place)."""
    import torch
    code, out = _prepare(x, out)
    if not isinstance(flags, torch.Tensor) or flags.dtype != torch.int32 or \
            flags.numel() != x.numel() or not flags.is_contiguous() or flags.device != x.device:
        raise ValueError("flags must be a contiguous int32 tensor with the size and device of x")
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=x.device)
    if count.dtype != torch.int64 or count.numel() < 1 or count.device != x.device:
        raise ValueError("count must be an int64 tensor on the device of x")
    with _device_of(x):
        _check(select_flagged_ptr(x.data_ptr(), flags.data_ptr(), out.data_ptr(), x.numel(), code,
                                  count.data_ptr(), _stream(x, stream)), "dws_select_flagged")
    return out, count


def _count_tensor(x, count):
    import torch
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=x.device)
    if count.dtype != torch.int64 or count.numel() < 1 or count.device != x.device:
        raise ValueError("count must be an int64 tensor on the device of x")
    return count


def _check_like(t, x, what):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.device != x.device or \
            t.numel() != x.numel() or t.element_size() != 4:
        raise ValueError(f"{what} must be a contiguous 4-byte GPU tensor with the size and device of the keys")


def partition_flagged(x, flags, out=None, count=None, stream=None):
    """Partition by flags: out[:count] the selected elements in order,
    out[count:] the rejected ones in reverse order. Returns (out, count) with
    count a one-element int64 GPU tensor. out must not overlap x."""
    import torch
    code, _ = _prepare(x, x)
    if out is None:
        out = torch.empty_like(x)
    _check_like(out, x, "out")
    _check_like(flags, x, "flags")
    count = _count_tensor(x, count)
    with _device_of(x):
        _check(load_library().dws_partition_flagged(x.data_ptr(), flags.data_ptr(), out.data_ptr(), x.numel(), code,
                                                    count.data_ptr(), _stream(x, stream)), "dws_partition_flagged")
    return out, count


def reduce_by_key(keys, values, unique_keys=None, aggregates=None, count=None, stream=None):
    """Runs of equal keys (32-bit patterns): unique_keys[:r], aggregates[:r]
    (+ of the values per run), r in the int64 GPU tensor ``count``."""
    import torch
    _check_like(keys, keys, "keys")
    code = _dtype_code(values)
    _check_like(values, keys, "values")
    unique_keys = torch.empty_like(keys) if unique_keys is None else unique_keys
    aggregates = torch.empty_like(values) if aggregates is None else aggregates
    _check_like(unique_keys, keys, "unique_keys")
    _check_like(aggregates, keys, "aggregates")
    count = _count_tensor(keys, count)
    with _device_of(keys):
        _check(load_library().dws_reduce_by_key(keys.data_ptr(), values.data_ptr(), unique_keys.data_ptr(),
                                                aggregates.data_ptr(), keys.numel(), code, count.data_ptr(),
                                                _stream(keys, stream)), "dws_reduce_by_key")
    return unique_keys, aggregates, count


def run_length_encode(keys, unique_keys=None, lengths=None, count=None, stream=None):
    """Runs of equal keys: unique_keys[:r], int32 tensor of uint32 lengths[:r],
    r in the int64 GPU tensor ``count``."""
    import torch
    _check_like(keys, keys, "keys")
    unique_keys = torch.empty_like(keys) if unique_keys is None else unique_keys
    lengths = torch.empty(keys.numel(), dtype=torch.int32, device=keys.device) if lengths is None else lengths
    _check_like(unique_keys, keys, "unique_keys")
    _check_like(lengths, keys, "lengths")
    count = _count_tensor(keys, count)
    with _device_of(keys):
        _check(load_library().dws_run_length_encode(keys.data_ptr(), unique_keys.data_ptr(), lengths.data_ptr(),
                                                    keys.numel(), count.data_ptr(), _stream(keys, stream)),
               "dws_run_length_encode")
    return unique_keys, lengths, count


# ---- the gated delta rule ---------------------------------------------------

# dws_delta_rule_args as a struct: packing one tuple takes a third of the time
# of setting the members of a ctypes structure, and these calls are short. Where
# each member starts in the list of values:
_DELTA = struct.Struct("@qqPiiiiiiif" + 6 * "Pqq" + "PPPq" + "Pqq" + "P" + 5 * "Pqq" + "PiPQ")
_DELTA_OPTIONS = struct.Struct(_DELTA.format[:-2] + "iPQ")      # with `options`, which is 0 in the other's padding
DELTA_FP32_GRADS, DELTA_PRECISE = 1, 2
(_N_SEQS, _OFFSETS, _G_DTYPE, _Q, _K, _V, _G, _BETA, _OUT, _INITIAL, _FINAL, _SLOTS, _N_STATES, _OUT_GRAD, _FINAL_GRAD,
 _Q_GRAD, _K_GRAD, _V_GRAD, _G_GRAD, _BETA_GRAD, _INITIAL_GRAD, _ZERO_REST, _WORKSPACE) = (
    1, 2, 8, 11, 14, 17, 20, 23, 26, 29, 30, 31, 32, 33, 36, 37, 40, 43, 46, 49, 52, 53, 54)

_float_codes = {}


def _int32():
    import torch
    return torch.int32


def _int64():
    import torch
    return torch.int64


def _float_code(dtype, what) -> int:
    if not _float_codes:
        import torch
        _float_codes.update({torch.float32: FLOAT32, torch.float16: FLOAT16, torch.bfloat16: BFLOAT16})
    code = _float_codes.get(dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, float16 or bfloat16, got {dtype}")
    return code


def _gpu_tensor(t, what):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a GPU tensor (there is no CPU path)")


def _rows(t, what, shape, dtype, device):
    """dws_rows of t: (tokens, heads, dim), or (tokens, heads) with dtype None."""
    try:
        if t.shape == shape and t.device == device and (dtype is None or t.dtype == dtype):
            strides = t.stride()
            if len(strides) == 2 or strides[2] == 1 or shape[2] <= 1 or not t.numel():
                return t.data_ptr(), strides[0], strides[1]
            raise ValueError(f"{what} must be contiguous in its last dimension")
    except AttributeError:
        pass
    _gpu_tensor(t, what)
    raise ValueError(f"{what} must have shape {tuple(shape)}" + (f", dtype {dtype}" if dtype is not None else "") +
                     f" and be on {device}, got {tuple(t.shape)}, {t.dtype} on {t.device}")


def _device_ints(t, what, dtype, n, device):
    try:
        if t.dtype == dtype and t.device == device and t.dim() == 1 and (n is None or t.shape[0] == n) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{what} must be a contiguous one-dimensional {dtype} tensor on {device}" +
                     (f" of {n} elements" if n is not None else ""))


def _state_ptr(t, what, count, shape, device):
    try:
        if t.dim() == 4 and _float_code(t.dtype, what) == FLOAT32 and t.shape[1:] == shape and t.device == device and \
                (count is None or t.shape[0] == count) and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    raise ValueError(f"{what} must be a contiguous float32 tensor {('count' if count is None else count, *shape)} on {device}")


def _delta_args(q, k, v, g, beta, offsets, n_seqs, scale):
    """The values that all three delta-rule calls share; checks shapes, types and devices. Returns (values, device)."""
    _gpu_tensor(q, "q")
    _gpu_tensor(v, "v")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be (tokens, heads, dim)")
    device, dtype = q.device, q.dtype
    tokens, heads_qk, dim_k = shape = q.shape
    heads_v, dim_v = v.shape[1:]
    code = _float_code(dtype, "q")
    gates = (tokens, heads_v)
    a = [0] * 56
    if offsets is not None:
        a[_OFFSETS] = _device_ints(offsets, "offsets", _int64(), None, device)
        n_seqs = offsets.shape[0] - 1
    if g is not None:
        a[_G: _G + 3] = _rows(g, "g", gates, None, device)
        a[_G_DTYPE] = _float_code(g.dtype, "g")
    a[_BETA: _BETA + 3] = _rows(beta, "beta", gates, None, device)
    a[:2] = tokens, n_seqs
    a[3:8] = heads_qk, heads_v, dim_k, dim_v, code
    a[9:11] = _float_code(beta.dtype, "beta"), dim_k ** -0.5 if scale is None else float(scale)
    a[_Q: _Q + 9] = (*_rows(q, "q", shape, dtype, device), *_rows(k, "k", shape, dtype, device),
                     *_rows(v, "v", (tokens, heads_v, dim_v), dtype, device))
    return a, device


def _records_no_graph(name, *tensors):
    """Refuses tensors whose gradients the result would silently lack."""
    import torch
    for t in tensors:
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise RuntimeError(f"{name} records no graph: call it with detached tensors or under torch.no_grad(), as the "
                               "forward and backward of a torch.autograd.Function are; delta_rule_backward gives "
                               "delta_rule's gradients")


class _on_stream:
    """Make x's device current, and allocate on the stream that the call runs on: memory that is freed when the binding
    returns is then reused in that stream's order only. Gives the stream's handle."""
    __slots__ = ("x", "given", "contexts")

    def __init__(self, x, stream):
        self.x, self.given, self.contexts = x, stream, ()

    def __enter__(self):
        import torch
        device = self.x.device
        if self.given is None:
            try:
                # the handle alone: current_stream() would make a Stream object, as much time as a launch takes
                if device.index == torch._C._cuda_getDevice():
                    return torch._C._cuda_getCurrentRawStream(device.index)
            except AttributeError:      # another version of torch
                pass
        current = int(torch.cuda.current_stream(device).cuda_stream)
        handle = current if self.given is None else int(self.given)
        self.contexts = (torch.cuda.device(device),)
        if handle != current:
            self.contexts += (torch.cuda.stream(torch.cuda.default_stream(device) if handle == 0 else
                                                torch.cuda.ExternalStream(handle, device=device)),)
        for c in self.contexts:
            c.__enter__()
        return handle

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)
        return False


def _delta_packed(a, options):
    if not options:
        return _DELTA.pack(*a)
    return _DELTA_OPTIONS.pack(*a[:_ZERO_REST + 1], options, *a[_ZERO_REST + 1:])


def _delta_workspace(a, options, backward, device):
    import torch
    need = ctypes.c_size_t(0)
    _check(load_library().dws_delta_rule_workspace(_delta_packed(a, options), backward, ctypes.byref(need)),
           "dws_delta_rule_workspace")
    work = torch.empty(need.value, dtype=torch.uint8, device=device)
    a[_WORKSPACE:] = work.data_ptr(), need.value
    return work


def delta_rule(q, k, v, g, beta, offsets=None, initial_state=None, final_state=None, slots=None, scale=None, out=None,
               stream=None, precise=False):
    """The gated delta rule over whole sequences (dws_delta_rule).

    q, k: (tokens, heads_qk, dim_k); v: (tokens, heads_v, dim_v), all float32, float16 or bfloat16, any strides with a
    contiguous last dimension. g (log decays, or None) and beta: (tokens, heads_v), each any of the three types.
    offsets: int64 GPU tensor of n + 1 ascending row numbers (None: one sequence). initial_state: float32
    (n, heads_v, dim_k, dim_v) or None for zero. final_state: None, a tensor like it to write (may be initial_state),
    or True for a new one. slots: int32 GPU tensor of n places when the states are a pool (count, heads_v, dim_k,
    dim_v); sequences with a place below 0, outside the pool or named before are left out. scale: dim_k^-0.5 by
    default. Rows of ``out`` in no sequence stay as they were, and are 0 in a new one. precise: the states in 16-bit
    products with fp32 accuracy also where no final one is asked for; ``out`` then has the same bits as where it is.
    Records no graph: tensors that require gradients are refused unless gradients are off (torch.no_grad()).
    Returns out, or (out, final_state) when the final state is asked for."""
    import torch
    _records_no_graph("delta_rule", q, k, v, g, beta, initial_state, final_state, out)
    a, device = _delta_args(q, k, v, g, beta, offsets, 1, scale)
    n_seqs, state_shape = a[_N_SEQS], (v.shape[1], q.shape[2], v.shape[2])
    count, options = n_seqs, DELTA_PRECISE if precise else 0
    if slots is not None:
        a[_SLOTS] = _device_ints(slots, "slots", torch.int32, n_seqs, device)
        count = None
        if final_state is True or (initial_state is None and final_state is None):
            raise ValueError("slots name places of a given state tensor")
    with _on_stream(q, stream) as s:
        if out is None:
            # a sequence that is left out keeps its rows: 0 in a new tensor
            out = (torch.empty if slots is None else torch.zeros)(v.shape, dtype=q.dtype, device=device)
            a[_ZERO_REST] = int(offsets is not None)
        a[_OUT: _OUT + 3] = _rows(out, "out", v.shape, q.dtype, device)
        if final_state is True:
            final_state = torch.empty((n_seqs, *state_shape), dtype=torch.float32, device=device)
        for t, what, at in ((initial_state, "initial_state", _INITIAL), (final_state, "final_state", _FINAL)):
            if t is not None:
                a[at] = _state_ptr(t, what, count, state_shape, device)
                if slots is not None:
                    count = a[_N_STATES] = t.shape[0]
        work = _delta_workspace(a, options, 0, device)
        _check(load_library().dws_delta_rule(_delta_packed(a, options), s), "dws_delta_rule")
        del work
    return out if final_state is None else (out, final_state)


def delta_rule_backward(d_out, q, k, v, g, beta, offsets=None, initial_state=None, d_final_state=None, scale=None,
                        stream=None, fp32_grads=False, precise=False):
    """Gradients of delta_rule (dws_delta_rule_backward): the arguments of the forward call and the gradient(s) of its
    result(s). Returns (dq, dk, dv, dg, dbeta, d_initial_state) in the type of q, dg None without g and
    d_initial_state None without initial_state; rows in no sequence are 0. fp32_grads: dg, dbeta and d_initial_state in
    float32, as g and the states may be; the last is then d_final_state for the sequence's part before. precise: the
    states' gradients in 16-bit products in two parts, so that only each result's own rounding is left. They have no graph
    of their own (no second derivatives)."""
    import torch
    a, device = _delta_args(q, k, v, g, beta, offsets, 1, scale)
    a[_OUT_GRAD: _OUT_GRAD + 3] = _rows(d_out, "d_out", v.shape, q.dtype, device)
    n_seqs, state_shape = a[_N_SEQS], (v.shape[1], q.shape[2], v.shape[2])
    for t, what, at in ((initial_state, "initial_state", _INITIAL), (d_final_state, "d_final_state", _FINAL_GRAD)):
        if t is not None:
            a[at] = _state_ptr(t, what, n_seqs, state_shape, device)
    with _on_stream(q, stream) as s:
        options = (DELTA_FP32_GRADS if fp32_grads else 0) | (DELTA_PRECISE if precise else 0)
        grads, narrow = [], torch.float32 if fp32_grads else q.dtype
        for like, at in ((q, _Q_GRAD), (k, _K_GRAD), (v, _V_GRAD), (g, _G_GRAD), (beta, _BETA_GRAD)):
            t = None if like is None else torch.empty(like.shape, dtype=q.dtype if like.dim() == 3 else narrow, device=device)
            if t is not None:
                a[at: at + 3] = t.data_ptr(), t.stride(0), t.stride(1)
            grads.append(t)
        d_initial = None if initial_state is None else torch.empty(initial_state.shape, dtype=narrow, device=device)
        if d_initial is not None:
            a[_INITIAL_GRAD] = d_initial.data_ptr()
        a[_ZERO_REST] = int(offsets is not None)
        work = _delta_workspace(a, options, 1, device)
        _check(load_library().dws_delta_rule_backward(_delta_packed(a, options), s), "dws_delta_rule_backward")
        del work
    return (*grads, d_initial)


def delta_rule_step(q, k, v, g, beta, state, slots=None, offsets=None, scale=None, out=None, stream=None):
    """A few more tokens for each sequence (dws_delta_rule_step), fp32 arithmetic, ``state`` updated in place.

    state: float32 (count, heads_v, dim_k, dim_v); sequence i uses state i, or slots[i] (int32 GPU tensor; places below
    0, outside the pool or named before are left out: their rows of ``out`` and the states stay, and the rows are 0 in
    a new ``out``). The tokens are shared out evenly over the sequences, or by offsets (int64 GPU tensor, n + 1).
    Other arguments, and tensors that require gradients, as delta_rule. Returns out."""
    import torch
    _records_no_graph("delta_rule_step", q, k, v, g, beta, state, out)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a (count, heads_v, dim_k, dim_v) tensor")
    n = slots.numel() if isinstance(slots, torch.Tensor) else state.shape[0]
    a, device = _delta_args(q, k, v, g, beta, offsets, n, scale)
    if a[_N_SEQS] != n or n < 1 or (offsets is None and a[0] % n):
        raise ValueError(f"{n} sequences do not fit {a[0]} tokens or {a[_N_SEQS] + 1} offsets")
    a[_INITIAL] = a[_FINAL] = _state_ptr(state, "state", None, (v.shape[1], q.shape[2], v.shape[2]), device)
    if slots is not None:
        a[_SLOTS] = _device_ints(slots, "slots", torch.int32, n, device)
        a[_N_STATES] = state.shape[0]
    with _on_stream(q, stream) as s:
        if out is None:
            out = torch.zeros(v.shape, dtype=q.dtype, device=device)
        a[_OUT: _OUT + 3] = _rows(out, "out", v.shape, q.dtype, device)
        _check(load_library().dws_delta_rule_step(_DELTA.pack(*a), s), "dws_delta_rule_step")
    return out


# ---- pages of a cache --------------------------------------------------------

_PAGES = struct.Struct("@PqPqqPq")      # dws_page_cache


def _page_cache(refs, table, lengths=None, page_tokens=0):
    """dws_page_cache, packed; and the number of pages."""
    _gpu_tensor(refs, "refs")
    device, int32 = refs.device, refs.dtype
    pages, at = refs.shape[0] if refs.dim() else 0, _device_ints(refs, "refs", _int32(), None, device)
    try:
        ok = table.dtype == int32 and table.dim() == 2 and table.device == device and table.is_contiguous()
    except AttributeError:
        ok = False
    if not ok:
        raise ValueError(f"table must be a contiguous int32 tensor (rows, pages) on {device}")
    rows, most = table.shape
    held = 0 if lengths is None else _device_ints(lengths, "lengths", int32, rows, device)
    return _PAGES.pack(at, pages, table.data_ptr(), rows, most, held, int(page_tokens)), pages


def _page_workspace(c, n, device):
    import torch
    need = ctypes.c_size_t(0)
    _check(load_library().dws_pages_workspace(c, n, ctypes.byref(need)), "dws_pages_workspace")
    return torch.empty(need.value, dtype=torch.uint8, device=device)


def _new_ints(n, like, dtype=None):
    import torch
    return torch.empty(n, dtype=dtype or torch.int32, device=like.device)


def pages_grow(refs, table, lengths, rows, new_lengths, page_tokens, stream=None):
    """Pages for ``rows`` to hold ``new_lengths`` tokens, lowest free page first (dws_pages_grow). refs (pages,), table
    (rows, max_pages) and lengths (rows,) are int32 GPU tensors, updated in place. Returns an int32 tensor: 1 where
    granted, 0 where the row stays as it was."""
    import torch
    c, _ = _page_cache(refs, table, lengths, page_tokens)
    n = rows.numel() if isinstance(rows, torch.Tensor) else 0
    a, b = _device_ints(rows, "rows", torch.int32, n, refs.device), _device_ints(new_lengths, "new_lengths", torch.int32, n, refs.device)
    with _on_stream(refs, stream) as s:
        granted, work = _new_ints(n, refs), _page_workspace(c, n, refs.device)
        _check(load_library().dws_pages_grow(c, a, b, n, granted.data_ptr(), work.data_ptr(), work.numel(), s),
               "dws_pages_grow")
    return granted


def pages_fork(refs, table, lengths, parents, children, page_tokens, stream=None):
    """Rows ``children`` (empty) with the tokens of rows ``parents``: whole pages shared, an unfinished last page new
    (dws_pages_fork). Returns (granted, src, dst, count): the pages to copy are src[:count] to dst[:count], count an
    int64 GPU tensor, for pages_copy on each pool."""
    import torch
    c, _ = _page_cache(refs, table, lengths, page_tokens)
    n = parents.numel() if isinstance(parents, torch.Tensor) else 0
    a, b = _device_ints(parents, "parents", torch.int32, n, refs.device), _device_ints(children, "children", torch.int32, n, refs.device)
    with _on_stream(refs, stream) as s:
        granted, src, dst = _new_ints((3, n), refs).unbind(0)
        count, work = _new_ints(1, refs, torch.int64), _page_workspace(c, n, refs.device)
        _check(load_library().dws_pages_fork(c, a, b, n, granted.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                             count.data_ptr(), work.data_ptr(), work.numel(), s), "dws_pages_fork")
    return granted, src, dst, count


def pages_free(refs, table, lengths, rows, page_tokens, stream=None):
    """Empties ``rows`` (dws_pages_free). Returns the number of pages that became free, a one-element int64 GPU tensor."""
    import torch
    c, _ = _page_cache(refs, table, lengths, page_tokens)
    a = _device_ints(rows, "rows", torch.int32, None, refs.device)
    n = rows.numel()
    with _on_stream(refs, stream) as s:
        freed, work = _new_ints(1, refs, torch.int64), _page_workspace(c, n, refs.device)
        _check(load_library().dws_pages_free(c, a, n, freed.data_ptr(), work.data_ptr(), work.numel(), s),
               "dws_pages_free")
    return freed


def pages_compact(refs, table, stream=None):
    """Pages in use renumbered to the front, with the fewest moves (dws_pages_compact); refs and table are updated.
    Returns (count, remap, src, dst, moves): pages in use, new number of each page (-1: free), and the pages to copy,
    src[:moves] to dst[:moves], for pages_copy on each pool. count and moves are int64 GPU tensors."""
    import torch
    c, pages = _page_cache(refs, table)
    with _on_stream(refs, stream) as s:
        half = pages // 2
        remap = _new_ints(pages, refs)
        src, dst = _new_ints((2, half), refs).unbind(0)
        moves, count = _new_ints(1, refs, torch.int64), _new_ints(1, refs, torch.int64)
        work = _page_workspace(c, 0, refs.device)
        _check(load_library().dws_pages_compact(c, remap.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                                moves.data_ptr(), count.data_ptr(), work.data_ptr(), work.numel(), s),
               "dws_pages_compact")
    return count, remap, src, dst, moves


def pages_copy(pool, src, dst, count=None, page_dim=0, stream=None):
    """pool[dst[i]] = pool[src[i]] for the pairs (the first ``count``, an int64 GPU tensor, of them) whose pages are in
    the pool (dws_pages_copy). pool: contiguous, of any type; page_dim 1: (layers, pages, ...). A written page must be
    in one pair only. Returns pool."""
    import torch
    _gpu_tensor(pool, "pool")
    if page_dim not in (0, 1) or pool.dim() <= page_dim or not pool.is_contiguous():
        raise ValueError("pool must be contiguous, its pages in dimension 0 or 1")
    n = src.numel() if isinstance(src, torch.Tensor) else 0
    device = pool.device
    a, b = _device_ints(src, "src", torch.int32, n, device), _device_ints(dst, "dst", torch.int32, n, device)
    k = None if count is None else _device_ints(count, "count", torch.int64, 1, pool.device)
    layers, pages = (1 if page_dim == 0 else pool.shape[0]), pool.shape[page_dim]
    layer_bytes = pool.numel() * pool.element_size() // max(1, layers)
    with _on_stream(pool, stream) as s:
        _check(load_library().dws_pages_copy(pool.data_ptr(), pages, layer_bytes // pages if pages else 0, layers,
                                             layer_bytes, a, b, n, k, s), "dws_pages_copy")
    return pool


# ---- keys and values in pages ------------------------------------------------

_KV = "PqqqPqqqPPqqqqiiii" + "qqPP"      # dws_kv_cache, dws_page_seqs
_APPEND = struct.Struct("@" + _KV + "PPPiiii" + 4 * "Pqq")
_ATTENTION = struct.Struct("@" + _KV + "ifqPPii" + 2 * "Pqq" + "PPQ")
_BEAM = struct.Struct("@PqqqqqiiPPq" + 8 * "P" + "Q")
ATTENTION_ONE_PART = 1      # dws_pages_attention_args.options

_workspaces = {}        # bytes by a call's sizes: asking again takes as long as a kernel's launch


def _workspace_bytes(query, key, make):
    need = _workspaces.get(key)
    if need is None:
        out = ctypes.c_size_t(0)
        _check(getattr(load_library(), query)(make(), ctypes.byref(out)), query)
        if len(_workspaces) >= 4096:
            _workspaces.clear()
        need = _workspaces[key] = out.value
    return need


def _kv_args(keys, values, table, lengths, tokens, rows, offsets):
    """The values of dws_kv_cache and dws_page_seqs; checks shapes, types and devices. Returns (values, device, n)."""
    import torch
    _gpu_tensor(keys, "keys")
    try:
        pages, page_tokens, heads, dim_k = keys.shape
    except ValueError:
        raise ValueError("keys and values must be (pages, page_tokens, heads, dim)") from None
    device, dtype, int32 = keys.device, keys.dtype, torch.int32
    code = _float_codes.get(dtype) or _float_code(dtype, "keys")
    k, v, dim_v = keys.stride(), (), -1
    try:
        if values.dtype == dtype and values.device == device:
            *same, dim_v = values.shape
            v = values.stride() if same == [pages, page_tokens, heads] else ()
    except AttributeError:
        pass
    if k[3] != 1 and dim_k > 1 or not v or v[3] != 1 and dim_v > 1:
        raise ValueError(f"keys and values must have shape {(pages, page_tokens, heads)} + (dim,), dtype {dtype} and a "
                         f"contiguous last dimension, and be on {device}")
    try:
        n_rows, max_pages = table.shape if table.dtype == int32 and table.device == device and table.is_contiguous() else ()
    except (AttributeError, ValueError):
        raise ValueError(f"table must be a contiguous int32 tensor (rows, pages) on {device}") from None
    held = _device_ints(lengths, "lengths", int32, n_rows, device)
    at = of = 0
    n = n_rows
    if offsets is not None:
        of = _device_ints(offsets, "offsets", torch.int64, None, device)
        n = offsets.shape[0] - 1
        if n < 0:
            raise ValueError("offsets holds one more than there are sequences")
    if rows is not None:
        at = _device_ints(rows, "rows", int32, n if offsets is not None else None, device)
        n = rows.shape[0]
    elif n > n_rows:
        raise ValueError(f"{n} sequences, but the table has {n_rows} rows")
    if offsets is None and (tokens % n if n else tokens):
        raise ValueError(f"{tokens} tokens cannot be shared out to {n} sequences")
    return (keys.data_ptr(), k[0], k[1], k[2], values.data_ptr(), v[0], v[1], v[2], table.data_ptr(), held, pages, n_rows,
            max_pages, page_tokens, heads, dim_k, dim_v, code, tokens, n, of, at), device, n


def pages_append(keys, values, table, lengths, k, v, rows=None, offsets=None, granted=None, positions=None, freqs=None,
                 adjacent=False, q=None, q_out=None, stream=None):
    """Keys and values of new tokens into the pages of a cache, turned by their positions on the way (dws_pages_append).

    keys, values: (pages, page_tokens, heads, dim) views of one layer's pool, float32, float16 or bfloat16, any strides with
    a contiguous last dimension; table (rows, max_pages) and lengths (rows,): int32 GPU tensors, as the other page calls
    have them, the new tokens counted already (pages_grow). k: (tokens, heads, dim_k), v: (tokens, heads, dim_v): the last
    tokens of rows ``rows`` (int32 GPU tensor; None: rows 0, 1, ...), shared out evenly or by offsets (int64 GPU tensor,
    n + 1). granted (as pages_grow returns it): sequences with 0 are left out, as are rows outside the table, those that an
    earlier sequence names, and sequences that have more tokens than their row.

    freqs: float32 GPU tensor, the angle between neighbouring positions for each pair of the first 2 * len(freqs) dimensions
    of k and q; pairs are (j, j + len(freqs)), or (2 j, 2 j + 1) with adjacent. positions (int32, one a token) replaces the
    place in the row in the angles. q: (tokens, heads_q, dim_k) to be turned likewise, into q_out, which may be q (None: a new
    tensor, 0 where the token is left out). Returns q_out, or None without q."""
    import torch
    _records_no_graph("pages_append", keys, values, k, v, q, q_out)
    try:
        tokens, _, _ = k.shape
    except (AttributeError, ValueError):
        _gpu_tensor(k, "k")
        raise ValueError(f"k must be (tokens, heads, dim), got {tuple(k.shape)}") from None
    a, device, n = _kv_args(keys, values, table, lengths, tokens, rows, offsets)
    dtype, heads, dim_k, dim_v = keys.dtype, a[14], a[15], a[16]
    kr, vr = _rows(k, "k", (tokens, heads, dim_k), dtype, device), _rows(v, "v", (tokens, heads, dim_v), dtype, device)
    ok = 0 if granted is None else _device_ints(granted, "granted", torch.int32, n, device)
    at = 0 if positions is None else _device_ints(positions, "positions", torch.int32, tokens, device)
    pairs = by = 0
    if freqs is not None:
        by, pairs = _device_ints(freqs, "freqs", torch.float32, None, device), freqs.shape[0]
        if 2 * pairs > dim_k:
            raise ValueError(f"{pairs} pairs do not fit {dim_k} dimensions")
    if q is None and q_out is not None:
        raise ValueError("q_out needs q")
    with _on_stream(keys, stream) as s:
        heads_q, zero, qr, to = 0, 0, (0, 0, 0), (0, 0, 0)
        if q is not None:
            try:
                shape = _, heads_q, _ = q.shape
            except (AttributeError, ValueError):
                _gpu_tensor(q, "q")
                raise ValueError("q must be (tokens, heads_q, dim_k)") from None
            qr = _rows(q, "q", (tokens, heads_q, dim_k), dtype, device)
            if q_out is None:
                q_out, zero = torch.empty(shape, dtype=dtype, device=device), 1
                to = q_out.data_ptr(), heads_q * dim_k, dim_k
            else:
                to = _rows(q_out, "q_out", shape, dtype, device)
        _check(load_library().dws_pages_append(
            _APPEND.pack(*a, ok, at, by, pairs, bool(adjacent), heads_q, zero, *kr, *vr, *qr, *to), s),
            "dws_pages_append")
    return q_out


def pages_attention(q, keys, values, table, lengths, rows=None, offsets=None, groups=None, shared=None, scale=None, out=None,
                    lse=None, stream=None, one_part=False):
    """Attention of each token's queries with the tokens of its row up to its own (dws_pages_attention).

    q: (tokens, heads_q, dim_k); keys, values, table, lengths, rows and offsets as pages_append, whose tokens these are, one
    a sequence or as many as a prompt has; heads_q is a multiple of the cache's heads. groups (int64 GPU tensor, groups + 1)
    and shared (int32 GPU tensor): the first shared[g] tokens of sequences groups[g] .. groups[g + 1] - 1 are in the same
    pages, as pages_fork leaves them, and are read once for all of these (while they have fewer than 64 queries a key head each, on
    average; through the first one that has a row). scale: dim_k^-0.5 by default. Queries that see
    nothing give 0. Rows of ``out`` in no sequence stay as they were, and are 0 in a new one. lse: None, True for a new
    float32 (tokens, heads_q) tensor of the logarithms of the exponentials' sums, or one to write; its rows in no sequence
    stay as they were, and are -infinity in a new one. one_part: 16-bit
    probabilities rounded once for their product with the values where more than 32 queries share keys: 1.4 times the
    error, a fifth less time for long prompts.
    Returns out, or (out, lse)."""
    import torch
    _records_no_graph("pages_attention", q, keys, values, out, lse if lse is not True else None)
    try:
        tokens, heads_q, _ = q.shape
    except (AttributeError, ValueError):
        _gpu_tensor(q, "q")
        raise ValueError("q must be (tokens, heads_q, dim_k)") from None
    a, device, n = _kv_args(keys, values, table, lengths, tokens, rows, offsets)
    dtype, heads, dim_k, dim_v = keys.dtype, a[14], a[15], a[16]
    if heads_q < 1 or heads_q % heads:
        raise ValueError(f"{heads_q} query heads are no multiple of {heads}")
    qr = _rows(q, "q", (tokens, heads_q, dim_k), dtype, device)
    n_groups = gp = sh = 0
    if (groups is None) != (shared is None):
        raise ValueError("groups and shared go together")
    if groups is not None:
        gp, n_groups = _device_ints(groups, "groups", torch.int64, None, device), groups.shape[0] - 1
        sh = _device_ints(shared, "shared", torch.int32, n_groups, device)
    with _on_stream(q, stream) as s:
        zero, shape = 0, (tokens, heads_q, dim_v)
        if out is None:
            # (dws_pages_attention sets the rest of both results, or of none: a given lse keeps its own)
            kept = offsets is not None and lse is not None and lse is not True
            out, zero = (torch.zeros if kept else torch.empty)(shape, dtype=dtype, device=device), int(offsets is not None and not kept)
            to = out.data_ptr(), heads_q * dim_v, dim_v
        else:
            if lse is True and offsets is not None:
                lse = torch.full((tokens, heads_q), float("-inf"), dtype=torch.float32, device=device)
            to = _rows(out, "out", shape, dtype, device)
        to_lse = 0
        if lse is not None:
            if lse is True:
                lse = torch.empty((tokens, heads_q), dtype=torch.float32, device=device)
            if not (isinstance(lse, torch.Tensor) and lse.dtype == torch.float32 and lse.device == device and
                    lse.shape == (tokens, heads_q) and lse.is_contiguous()):
                raise ValueError(f"lse must be a contiguous float32 tensor {(tokens, heads_q)} on {device}")
            to_lse = lse.data_ptr()
        rest = (heads_q, dim_k ** -0.5 if scale is None else float(scale), n_groups, gp, sh, zero,
                ATTENTION_ONE_PART if one_part else 0, *qr, *to, to_lse)
        need = _workspace_bytes("dws_pages_attention_workspace", (heads_q, n_groups, *a[10:20]),
                                lambda: _ATTENTION.pack(*a, *rest, 0, 0))
        work = torch.empty(need, dtype=torch.uint8, device=device)
        _check(load_library().dws_pages_attention(_ATTENTION.pack(*a, *rest, work.data_ptr(), need), s),
               "dws_pages_attention")
        del work
    return out if lse is None else (out, lse)


# ---- beam search ---------------------------------------------------------------

def beam_select(logits, scores, k=None, finished=None, end_token=0, rows=None, stream=None):
    """For each request the k (None: as many as beams) continuations of its beams with the largest
    scores[beam] + log softmax(logits[beam])[token], in descending order, the lowest beam and token first among equal ones
    (dws_beam_select).

    logits: (batch, beams, vocab), float32, float16 or bfloat16, any strides with a contiguous last dimension; scores:
    float32 (batch, beams). finished: bool or uint8 (batch, beams), beams that go on with end_token alone, at their score,
    whatever their logits hold.
    Returns (scores (batch, k) float32, parents (batch, k) int32, tokens (batch, k) int32).
    With rows (int32 (batch, beams): cache rows or state slots of the beams; needs k == beams) also (rows, src, dst): the
    continuations' rows, and which to copy where (batch * beams each, -1: none). States follow with
    pages_copy(pool, src, dst), rows of pages with pages_free(.., dst, ..), pages_fork(.., src, dst, ..) and pages_copy."""
    import torch
    _records_no_graph("beam_select", logits, scores)
    _gpu_tensor(logits, "logits")
    if logits.dim() != 3 or (logits.stride(2) != 1 and logits.shape[2] > 1):
        raise ValueError("logits must be (batch, beams, vocab), contiguous in the last dimension")
    device, code = logits.device, _float_code(logits.dtype, "logits")
    batch, beams, vocab = logits.shape
    k = beams if k is None else int(k)

    shape, int32 = (batch, beams), torch.int32

    def plain(t, what, dtype, other=None):
        try:
            if t.shape == shape and (t.dtype == dtype or t.dtype == other) and t.device == device and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            pass
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {shape} on {device}")

    of = plain(scores, "scores", torch.float32)
    over = 0 if finished is None else plain(finished, "finished", torch.bool, torch.uint8)
    at = 0 if rows is None else plain(rows, "rows", int32)
    if rows is not None and k != beams:
        raise ValueError("rows can be followed only with as many continuations as beams")
    with _on_stream(logits, stream) as s:
        best = torch.empty_like(scores) if k == beams else torch.empty((batch, k), dtype=torch.float32, device=device)
        parents = torch.empty_like(best, dtype=int32)
        tokens = torch.empty_like(parents)
        new = src = dst = None
        if rows is not None:
            new = torch.empty_like(parents)
            src = torch.empty(batch * beams, dtype=int32, device=device)
            dst = torch.empty_like(src)
            at = at, best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), new.data_ptr(), src.data_ptr(), dst.data_ptr()
        else:
            at = 0, best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), 0, 0, 0
        a = (logits.data_ptr(), batch, beams, vocab, *logits.stride()[:2], code, k, of, over, int(end_token), *at)
        need = _workspace_bytes("dws_beam_select_workspace", a[1:8], lambda: _BEAM.pack(*a, 0, 0))
        work = torch.empty(need, dtype=torch.uint8, device=device)
        _check(load_library().dws_beam_select(_BEAM.pack(*a, work.data_ptr(), need), s), "dws_beam_select")
        del work
    return (best, parents, tokens) if rows is None else (best, parents, tokens, new, src, dst)


def device_memory_info() -> dict:
    """Memory clock (kHz), memory bus width (bits) and compute units of the
    current device, as the HIP runtime reports them."""
    clk, width, cus = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(load_library().dws_device_memory_info(ctypes.byref(clk), ctypes.byref(width), ctypes.byref(cus)),
           "dws_device_memory_info")
    return {"memory_clock_khz": clk.value, "memory_bus_width_bits": width.value, "compute_units": cus.value}


def watchdog_trips() -> int:
    v = ctypes.c_ulonglong(0)
    _check(load_library().dws_watchdog_trips(ctypes.byref(v)), "dws_watchdog_trips")
    return int(v.value)


def selftest_wave(x, stream=None):
    """Apply the kernels' wave64 primitives to each group of 64 elements of x:
    returns (in-wave inclusive scan, previous-lane value)."""
    import torch
    code, _ = _prepare(x, None)
    if x.numel() % 64:
        raise ValueError("selftest_wave needs a multiple of 64 elements")
    incl = torch.empty_like(x)
    shift = torch.empty_like(x)
    with _device_of(x):
        _check(load_library().dws_selftest_wave(x.data_ptr(), incl.data_ptr(), shift.data_ptr(),
                                                x.numel() // 64, code, _stream(x, stream)),
               "dws_selftest_wave")
    return incl, shift


def reserve(n: int, stream=None, device=None):
    import torch
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    with torch.cuda.device(dev):
        s = int(torch.cuda.current_stream(dev).cuda_stream) if stream is None else int(stream)
        _check(load_library().dws_reserve(int(n), s), "dws_reserve")


def release_workspaces():
    _check(load_library().dws_release_workspaces(), "dws_release_workspaces")


def tile_elems(tile_shape: int = 0, n: int = 1 << 28, aligned: bool = True) -> int:
    """Elements per tile the single-pass kernel uses (tile_shape 0 = automatic
    choice for n)."""
    return int(load_library().dws_tile_elems(int(tile_shape), int(n), int(bool(aligned))))


def tile_threads(tile_shape: int = 0, n: int = 1 << 28, aligned: bool = True) -> int:
    return int(load_library().dws_tile_threads(int(tile_shape), int(n), int(bool(aligned))))


def num_tile_shapes() -> int:
    return int(load_library().dws_num_tile_shapes())


class _device_of:
    """Make x's device current for the C call (the library works on the
    current HIP device)."""

    def __init__(self, x):
        self.x = x
        self.ctx = None

    def __enter__(self):
        import torch
        self.ctx = torch.cuda.device(self.x.device)
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)
        return False
