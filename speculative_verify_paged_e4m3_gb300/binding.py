"""Thin ctypes binding over libdflash_verify_attn.so (the C ABI in include/dflash_verify_attn.h,
include/dflash_paged_step.h and include/dflash_mx4_cache.h).

Argument marshalling only: every step of the computation runs in the library's CUDA kernels.
Functions carry the C names; tensors are torch CUDA tensors whose data pointers are passed
through, and the stream is torch's current stream unless one is given. If the library has not
been built, every entry point raises (there is no fallback).
"""
from __future__ import annotations

import collections
import ctypes
import os
import threading

import torch

from . import build as _build

DFLASH_VERIFY_ATTN_VERSION = 3
DFLASH_OK = 0
DFLASH_ERR_INVALID_ARGUMENT = -1
DFLASH_ERR_UNSUPPORTED = -2
DFLASH_ERR_WORKSPACE_TOO_SMALL = -3
DFLASH_ERR_CUDA = -4
DFLASH_FLAG_CONTEXT_CLAMPED = 0x1
DFLASH_FLAG_CONTEXT_SHORT = 0x2
DFLASH_FLAG_PAGE_CLAMPED = 0x4
DFLASH_FLAG_KERNEL_TIMEOUT = 0x8
DFLASH_PROBLEM_FUSED_COMBINE = 0x1
DFLASH_PROBLEM_PDL = 0x2
DFLASH_KERNEL_AUTO = 0
DFLASH_KERNEL_SIMT = 1
DFLASH_KERNEL_TCGEN05 = 2

DFLASH_PAGED_STEP_VERSION = 1
DFLASH_FLAG_PAGES_EXHAUSTED = 0x10
DFLASH_FLAG_TOKENS_DROPPED = 0x20
DFLASH_FLAG_SLOT_RANGE = 0x40
DFLASH_ROPE_HALF = 0
DFLASH_ROPE_INTERLEAVED = 1
DFLASH_ROPE_SCALE_NONE = 0
DFLASH_ROPE_SCALE_LINEAR = 1
DFLASH_ROPE_SCALE_NTK = 2
DFLASH_ROPE_SCALE_YARN = 3
DFLASH_ROPE_SCALE_WAVELENGTH = 4
DFLASH_FP16 = 0
DFLASH_BF16 = 1
DFLASH_PREFIX_KERNEL_AUTO = 0
DFLASH_PREFIX_KERNEL_ROWS = 1
DFLASH_PREFIX_KERNEL_PAIRS = 2
DFLASH_E5M2 = 2
DFLASH_KERNEL_MX4 = 3
DFLASH_MX4_CHUNK_TOKENS = 16
DFLASH_MX4_CHUNK_BYTES = 2176

EXPORTED = (
    "dflash_verify_attn_plan",
    "dflash_verify_attn_split_bounds",
    "dflash_verify_attn_split_slots",
    "dflash_verify_attn_run",
    "dflash_verify_attn_combine",
    "dflash_verify_attn_forward",
    "dflash_verify_attn_debug_dequant",
    "dflash_verify_attn_read_flags",
    "dflash_verify_attn_forward_static_scratch",
    "dflash_verify_attn_kv_write",
    "dflash_paged_tables",
    "dflash_rope_plan",
    "dflash_rope_apply",
    "dflash_rope_kv_write",
    "dflash_rope_kv_write_live",
    "dflash_prefix_attn_plan",
    "dflash_prefix_attn_forward",
    "dflash_norm_rope_apply",
    "dflash_norm_rope_kv_write",
    "dflash_mx4_kv_write",
    "dflash_mx4_read",
    "dflash_mx4_attn_plan",
    "dflash_mx4_attn_forward",
    "dflash_verify_attn_status_string",
)


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "batch", "q_len", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pages", "max_context", "device", "num_splits", "kernel",
        "flags")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "kernel", "num_splits", "tile_keys", "min_split_keys", "rows", "threads",
        "smem_bytes", "sm_count", "combine_fused", "row_blocks", "num_slots")] + [
        ("workspace_bytes", ctypes.c_size_t),
        ("ws_state_offset", ctypes.c_size_t),
        ("ws_acc_offset", ctypes.c_size_t),
        ("problem", Problem),
    ]


class PagedTablesProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "batch", "page_size", "max_pages_per_seq", "num_pages", "max_context",
        "max_tokens", "num_free", "prefix_capacity")]


class RopeProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "num_q_heads", "num_kv_heads", "head_dim", "rotary_dim", "layout", "dtype",
        "scaling", "trained_context", "page_size", "num_pages", "reserved")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "beta_fast", "beta_slow", "low_turns",
                                       "high_turns")]


class RopePlan(ctypes.Structure):
    _fields_ = [("version", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("problem", RopeProblem)]


class PrefixAttnProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "batch", "q_len", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pages", "max_context", "max_prefix", "device", "kernel",
        "flags")]


class PrefixAttnPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "prefix_kernel", "prefix_rows", "prefix_row_blocks", "prefix_splits",
        "prefix_slots", "prefix_slot_rows", "sm_count")] + [
        ("suffix", Plan),
        ("ws_prefix_state_offset", ctypes.c_size_t),
        ("ws_prefix_acc_offset", ctypes.c_size_t),
        ("ws_unit_offset", ctypes.c_size_t),
        ("workspace_bytes", ctypes.c_size_t),
        ("problem", PrefixAttnProblem),
    ]


class HeadNormArgs(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class DflashError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load the built library (raises if it is missing: build it with build.build())."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is not built; run "
                                   "speculative_verify_paged_e4m3_gb300.build.build() first")
            lib = ctypes.CDLL(path)
            vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
            pp = ctypes.POINTER(Plan)
            lib.dflash_verify_attn_plan.argtypes = [ctypes.POINTER(Problem), pp]
            lib.dflash_verify_attn_split_bounds.argtypes = [
                pp, i32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
            i32p = ctypes.POINTER(ctypes.c_int32)
            lib.dflash_verify_attn_split_slots.argtypes = [pp, i32p, i32p, i32p, i32p]
            lib.dflash_verify_attn_run.argtypes = [pp] + [vp] * 8 + [sz, vp]
            lib.dflash_verify_attn_combine.argtypes = [pp, vp, sz, vp, vp, vp, vp]
            lib.dflash_verify_attn_forward.argtypes = [pp] + [vp] * 8 + [sz, vp, vp, vp]
            lib.dflash_verify_attn_forward_static_scratch.argtypes = [pp] + [vp] * 10
            lib.dflash_verify_attn_kv_write.argtypes = [pp] + [vp] * 9 + [sz, vp]
            lib.dflash_paged_tables.argtypes = [ctypes.POINTER(PagedTablesProblem)] + [vp] * 16
            lib.dflash_rope_plan.argtypes = [ctypes.POINTER(RopeProblem),
                                             ctypes.POINTER(RopePlan),
                                             ctypes.POINTER(ctypes.c_uint64)]
            rp = ctypes.POINTER(RopePlan)
            lib.dflash_rope_apply.argtypes = [rp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                              vp]
            lib.dflash_rope_kv_write.argtypes = [rp, i64, vp, i64, vp, i64, vp, i64] + [vp] * 6 + [
                i64] + [vp] * 4
            lib.dflash_rope_kv_write_live.argtypes = [rp, i64, vp, i64, vp, i64, vp, i64] + [vp] * 7 + [
                i64] + [vp] * 4
            xp = ctypes.POINTER(PrefixAttnPlan)
            lib.dflash_prefix_attn_plan.argtypes = [ctypes.POINTER(PrefixAttnProblem), xp]
            lib.dflash_prefix_attn_forward.argtypes = [xp] + [vp] * 10 + [sz, vp, vp, vp]
            np_ = ctypes.POINTER(HeadNormArgs)
            lib.dflash_norm_rope_apply.argtypes = [rp, np_, i64, vp, i64, vp, i64, vp, vp, vp, i64,
                                                   vp, i64, vp]
            lib.dflash_norm_rope_kv_write.argtypes = [rp, np_, i64, vp, i64, vp, i64, vp,
                                                      i64] + [vp] * 7 + [i64] + [vp] * 4
            lib.dflash_mx4_kv_write.argtypes = [rp, np_, i64, vp, i64, vp, i64, vp,
                                                i64] + [vp] * 5 + [i64] + [vp] * 4
            lib.dflash_mx4_read.argtypes = [i32, i32, i32, i32, vp, vp, i64, vp, i32, vp, i64, vp,
                                            i64, vp, vp]
            lib.dflash_mx4_attn_plan.argtypes = [ctypes.POINTER(Problem), pp]
            lib.dflash_mx4_attn_forward.argtypes = [pp] + [vp] * 6 + [sz, vp, vp, vp]
            lib.dflash_verify_attn_debug_dequant.argtypes = [vp, i64, vp, vp, vp, vp]
            lib.dflash_verify_attn_read_flags.argtypes = [vp, ctypes.POINTER(ctypes.c_int32),
                                                          ctypes.c_int, vp]
            lib.dflash_verify_attn_status_string.argtypes = [ctypes.c_int]
            lib.dflash_verify_attn_status_string.restype = ctypes.c_char_p
            for name in EXPORTED[:-1]:
                getattr(lib, name).restype = ctypes.c_int
            _lib = lib
        return _lib


def status_string(status: int) -> str:
    return load_library().dflash_verify_attn_status_string(int(status)).decode()


dflash_verify_attn_status_string = status_string


def _check(fn: str, status: int):
    if status != DFLASH_OK:
        raise DflashError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_problem(batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                 max_pages_per_seq, num_pages, max_context, device=0, num_splits=0,
                 kernel=DFLASH_KERNEL_AUTO, flags=0) -> Problem:
    return Problem(DFLASH_VERIFY_ATTN_VERSION, batch, q_len, num_q_heads, num_kv_heads,
                   head_dim, page_size, max_pages_per_seq, num_pages, max_context, device,
                   num_splits, kernel, flags)


def dflash_verify_attn_plan(problem: Problem) -> Plan:
    plan = Plan()
    _check("dflash_verify_attn_plan",
           load_library().dflash_verify_attn_plan(ctypes.byref(problem), ctypes.byref(plan)))
    return plan


def dflash_verify_attn_plan_status(problem: Problem) -> int:
    """The raw status of planning (for tests of the error paths)."""
    plan = Plan()
    return load_library().dflash_verify_attn_plan(ctypes.byref(problem), ctypes.byref(plan))


def dflash_verify_attn_split_bounds(plan: Plan, n: int):
    starts = (ctypes.c_int32 * (plan.num_splits + 1))()
    active = ctypes.c_int32()
    _check("dflash_verify_attn_split_bounds",
           load_library().dflash_verify_attn_split_bounds(ctypes.byref(plan), int(n), starts,
                                                          ctypes.byref(active)))
    return list(starts), active.value


def dflash_verify_attn_split_slots(plan: Plan, context_lens):
    """(slot_start [units + 1], keys_per_split [units], active [units]) for the given host-side
    context lengths (units = batch * Hkv, unit u = b * Hkv + h)."""
    lens = list(int(x) for x in context_lens)
    units = plan.problem.batch * plan.problem.num_kv_heads
    if len(lens) != plan.problem.batch:
        raise ValueError("context_lens must have batch entries")
    cl = (ctypes.c_int32 * len(lens))(*lens)
    start = (ctypes.c_int32 * (units + 1))()
    per = (ctypes.c_int32 * units)()
    act = (ctypes.c_int32 * units)()
    _check("dflash_verify_attn_split_slots",
           load_library().dflash_verify_attn_split_slots(ctypes.byref(plan), cl, start, per, act))
    return list(start), list(per), list(act)


def dflash_verify_attn_run(plan: Plan, q, k_pool, v_pool, block_table, context_lens, k_scale,
                           v_scale, workspace, stream=None, check=True) -> int:
    rc = load_library().dflash_verify_attn_run(
        ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
        _ptr(context_lens), _ptr(k_scale), _ptr(v_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0,
        _stream(stream))
    if check:
        _check("dflash_verify_attn_run", rc)
    return rc


def dflash_verify_attn_combine(plan: Plan, workspace, context_lens, out, lse, stream=None,
                               check=True) -> int:
    rc = load_library().dflash_verify_attn_combine(
        ctypes.byref(plan), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(context_lens), _ptr(out), _ptr(lse), _stream(stream))
    if check:
        _check("dflash_verify_attn_combine", rc)
    return rc


def dflash_verify_attn_forward(plan: Plan, q, k_pool, v_pool, block_table, context_lens,
                               k_scale, v_scale, workspace, out, lse, stream=None,
                               check=True) -> int:
    rc = load_library().dflash_verify_attn_forward(
        ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
        _ptr(context_lens), _ptr(k_scale), _ptr(v_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _stream(stream))
    if check:
        _check("dflash_verify_attn_forward", rc)
    return rc


def dflash_verify_attn_forward_static_scratch(plan: Plan, q, k_pool, v_pool, block_table,
                                              context_lens, k_scale, v_scale, out, lse,
                                              stream=None, check=True) -> int:
    """Forward pass using the library's built-in device scratch array (no workspace argument)."""
    rc = load_library().dflash_verify_attn_forward_static_scratch(
        ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
        _ptr(context_lens), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse),
        _stream(stream))
    if check:
        _check("dflash_verify_attn_forward_static_scratch", rc)
    return rc


def dflash_verify_attn_kv_write(plan: Plan, k_new, v_new, block_table, context_lens, k_scale,
                                v_scale, k_pool, v_pool, workspace, stream=None,
                                check=True) -> int:
    rc = load_library().dflash_verify_attn_kv_write(
        ctypes.byref(plan), _ptr(k_new), _ptr(v_new), _ptr(block_table), _ptr(context_lens),
        _ptr(k_scale), _ptr(v_scale), _ptr(k_pool), _ptr(v_pool), _ptr(workspace),
        workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0,
        _stream(stream))
    if check:
        _check("dflash_verify_attn_kv_write", rc)
    return rc


def dflash_verify_attn_debug_dequant(codes, scale, decoded, scaled=None, stream=None):
    _check("dflash_verify_attn_debug_dequant",
           load_library().dflash_verify_attn_debug_dequant(
               _ptr(codes), codes.numel(), _ptr(scale), _ptr(decoded), _ptr(scaled),
               _stream(stream)))


def dflash_verify_attn_read_flags(workspace, clear=False, stream=None) -> int:
    v = ctypes.c_int32()
    _check("dflash_verify_attn_read_flags",
           load_library().dflash_verify_attn_read_flags(_ptr(workspace), ctypes.byref(v),
                                                        int(bool(clear)), _stream(stream)))
    return v.value


def make_rope_problem(num_q_heads, num_kv_heads, head_dim, rotary_dim, layout=DFLASH_ROPE_HALF,
                      dtype=DFLASH_FP16, base=10000.0, scaling=DFLASH_ROPE_SCALE_NONE, factor=1.0,
                      trained_context=1, beta_fast=32.0, beta_slow=1.0, low_turns=1.0,
                      high_turns=4.0, page_size=16, num_pages=1) -> RopeProblem:
    return RopeProblem(DFLASH_PAGED_STEP_VERSION, num_q_heads, num_kv_heads, head_dim, rotary_dim,
                       layout, dtype, scaling, trained_context, page_size, num_pages, 0, base,
                       factor, beta_fast, beta_slow, low_turns, high_turns)


def dflash_rope_plan(problem: RopeProblem):
    """(plan, phases): phases is a ctypes array of rotary_dim / 2 64-bit fractions of a turn."""
    plan = RopePlan()
    phases = (ctypes.c_uint64 * max(1, problem.rotary_dim // 2))()
    _check("dflash_rope_plan",
           load_library().dflash_rope_plan(ctypes.byref(problem), ctypes.byref(plan), phases))
    return plan, phases


def make_prefix_problem(batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                        max_pages_per_seq, num_pages, max_context, max_prefix, device=0,
                        kernel=DFLASH_PREFIX_KERNEL_AUTO, flags=0) -> PrefixAttnProblem:
    return PrefixAttnProblem(DFLASH_PAGED_STEP_VERSION, batch, q_len, num_q_heads, num_kv_heads,
                             head_dim, page_size, max_pages_per_seq, num_pages, max_context,
                             max_prefix, device, kernel, flags)


def dflash_prefix_attn_plan(problem: PrefixAttnProblem) -> PrefixAttnPlan:
    plan = PrefixAttnPlan()
    _check("dflash_prefix_attn_plan",
           load_library().dflash_prefix_attn_plan(ctypes.byref(problem), ctypes.byref(plan)))
    return plan


def dflash_mx4_attn_plan(problem: Problem) -> Plan:
    plan = Plan()
    _check("dflash_mx4_attn_plan",
           load_library().dflash_mx4_attn_plan(ctypes.byref(problem), ctypes.byref(plan)))
    return plan


# ---------------------------------------------------------------------------------------------
# convenience layer (still marshalling only)

class VerifyAttention:
    """One layer shape: a plan plus its workspace; call() runs partial attention and combine."""

    def __init__(self, batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                 max_pages_per_seq, num_pages, max_context, device=None, num_splits=0,
                 kernel=DFLASH_KERNEL_AUTO, workspace=None, flags=0):
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.device = dev
        self.problem = make_problem(batch, q_len, num_q_heads, num_kv_heads, head_dim,
                                    page_size, max_pages_per_seq, num_pages, max_context,
                                    dev.index, num_splits, kernel, flags)
        self.plan = dflash_verify_attn_plan(self.problem)
        if workspace is None:
            workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)
        elif workspace.numel() * workspace.element_size() < self.plan.workspace_bytes:
            raise ValueError("workspace smaller than plan.workspace_bytes")
        self.workspace = workspace

    def workspace_views(self):
        """(status int32[1], state float32 [slots,R,2], acc float32 [slots,R,D]) views; for a
        single sequence slot h * num_splits + s is split s of KV head h."""
        pr, pl = self.problem, self.plan
        shape = (pl.num_slots, pl.rows)
        ws = self.workspace
        n_state = pl.num_slots * pl.rows * 2
        state = ws[pl.ws_state_offset:pl.ws_state_offset + 4 * n_state].view(torch.float32)
        n_acc = n_state // 2 * pr.head_dim
        acc = ws[pl.ws_acc_offset:pl.ws_acc_offset + 4 * n_acc].view(torch.float32)
        return (ws[:4].view(torch.int32), state.view(shape + (2,)),
                acc.view(shape + (pr.head_dim,)))

    def __call__(self, q, k_pool, v_pool, block_table, context_lens, k_scale, v_scale,
                 out=None, lse=None, stream=None):
        pr = self.problem
        if out is None:
            out = torch.empty((pr.batch, pr.q_len, pr.num_q_heads, pr.head_dim),
                              dtype=torch.float16, device=self.device)
        if lse is None:
            lse = torch.empty((pr.batch, pr.q_len, pr.num_q_heads), dtype=torch.float32,
                              device=self.device)
        dflash_verify_attn_forward(self.plan, q, k_pool, v_pool, block_table, context_lens,
                                   k_scale, v_scale, self.workspace, out, lse, stream)
        return out, lse

    def kv_write(self, k_new, v_new, block_table, context_lens, k_scale, v_scale, k_pool,
                 v_pool, stream=None):
        """Write the drafted tokens' K/V rows ([B, q_len, Hkv, D] FP16) into the pools."""
        dflash_verify_attn_kv_write(self.plan, k_new, v_new, block_table, context_lens, k_scale,
                                    v_scale, k_pool, v_pool, self.workspace, stream)


# ---------------------------------------------------------------------------------------------
# a paged decoding step (include/dflash_paged_step.h): tables, rotary positions with the cache
# write, attention over a shared prefix. These classes check types, shapes, strides and devices
# before they pass pointers on, and launch on their own device whichever is current. Small calls
# are bound by the host, so the checks and the look-ups of device and stream are kept short.

# (torch.cuda.current_stream builds a Stream object, 3 us on the host of a GB300)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(name, t, dtype, shape, index, form="contiguous "):
    got = (f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}"
           if isinstance(t, torch.Tensor) else type(t).__name__)
    raise ValueError(f"{name}: want {form}{dtype} {tuple(shape)} on cuda:{index}, got {got}")


def _want(name, t, dtype, shape, index):
    """Raise unless t is a contiguous tensor of this type and shape on this device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or t.get_device() != index or not t.is_contiguous()):
        _refuse(name, t, dtype, shape, index)


def _want_rows(name, t, dtype, shape, index):
    """Raise unless t is [tokens, heads, head_dim] with heads one after the other (tokens may be
    further apart: a slice of a fused projection); returns the token stride in elements."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or t.get_device() != index):
        _refuse(name, t, dtype, shape, index, "")
    st = t.stride()
    if st[2] != 1 or (st[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: heads must lie one after the other, got strides {st}")
    return st[0] if shape[0] > 1 else shape[1] * shape[2]


class _OnDevice:
    """The device of an operator and its launches."""

    def __init__(self, device, *functions):
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.device, self._index = dev, dev.index
        lib = load_library()
        self._functions = {name: getattr(lib, name) for name in functions}

    def _launch(self, name, stream, *args):
        stream = _raw_stream(self._index) if stream is None else _stream(stream)
        if _current_device() == self._index:
            rc = self._functions[name](*args, stream)
        else:
            with torch.cuda.device(self._index):
                rc = self._functions[name](*args, stream)
        if rc != DFLASH_OK:
            raise DflashError(name, rc)

    def _empty(self, shape, dtype, stream):
        """A buffer for a launch on this stream, from that stream's memory: memory that was freed on the
        current one may still be in use there."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=self.device) if stream
                      else torch.cuda.default_stream(self.device))
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _ready(self):
        """Wait for what a constructor has put on the current stream: the first call may be on another.
        (A capture cannot wait; made inside one, an operator is ready once the graph has run.)"""
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()

    def _status_word(self, status):
        """The given status word, or one of this operator's own."""
        if status is None:
            return torch.zeros(4, dtype=torch.int32, device=self.device)
        if status.dtype is not torch.int32 or status.numel() < 1 or status.device != self.device:
            raise ValueError(f"status: want an int32 tensor on {self.device}")
        return status

    def _read_flags(self, word, clear, stream):
        with torch.cuda.device(self._index):
            return dflash_verify_attn_read_flags(word, clear, stream)


TablesOut = collections.namedtuple("TablesOut", (
    "context_lens", "held_pages", "free_head", "token_starts", "positions", "slots"))


class _MadeTables(TablesOut):
    """Buffers that a PagedTables made: of the right types and shapes on its device."""
    maker = None


class PagedTables(_OnDevice):
    """The block-table entries, positions and cache slots of each step's new tokens, from request
    lengths on the GPU (dflash_paged_tables)."""

    def __init__(self, batch, page_size, max_pages_per_seq, num_pages, max_context, max_tokens,
                 device=None, status=None):
        super().__init__(device, "dflash_paged_tables")
        self.batch, self.page_size, self.max_tokens = batch, page_size, max_tokens
        self.max_pages_per_seq, self.num_pages = max_pages_per_seq, num_pages
        self.max_context = max_context
        self._problem = PagedTablesProblem(DFLASH_PAGED_STEP_VERSION, batch, page_size,
                                           max_pages_per_seq, num_pages, max_context, max_tokens,
                                           0, 0)
        self.status = self._status_word(status)
        self._ready()

    def empty(self, stream=None) -> TablesOut:
        """Output buffers of one step, of the current stream's memory or the given one's."""
        def i32(n):
            return self._empty(n, torch.int32, stream)
        out = _MadeTables(i32(self.batch), i32(self.batch), i32(1), i32(self.batch + 1),
                          i32(self.max_tokens),
                          self._empty(self.max_tokens, torch.int64, stream))
        out.maker = self
        return out

    def __call__(self, cached_lens, new_lens, held_pages, free_pages, free_head, block_table,
                 prefix_table=None, prefix_pages=None, out=None, stream=None) -> TablesOut:
        """Fill the rows' new entries of block_table in place; the rest goes to out (buffers of
        empty(), made anew when not given)."""
        ix, i32, each = self._index, torch.int32, (self.batch,)
        if out is None:
            out = self.empty(stream)
        num_free = free_pages.numel()
        _want("cached_lens", cached_lens, i32, each, ix)
        _want("new_lens", new_lens, i32, each, ix)
        _want("held_pages", held_pages, i32, each, ix)
        _want("free_pages", free_pages, i32, (num_free,), ix)
        _want("free_head", free_head, i32, (1,), ix)
        _want("block_table", block_table, i32, (self.batch, self.max_pages_per_seq), ix)
        ctx, held, head, starts, positions, slots = out
        if getattr(out, "maker", None) is not self:
            _want("out.context_lens", ctx, i32, each, ix)
            _want("out.held_pages", held, i32, each, ix)
            _want("out.free_head", head, i32, (1,), ix)
            _want("out.token_starts", starts, i32, (self.batch + 1,), ix)
            _want("out.positions", positions, i32, (self.max_tokens,), ix)
            _want("out.slots", slots, torch.int64, (self.max_tokens,), ix)
        capacity, prefix, pages = 0, None, None
        if prefix_table is not None:
            capacity = min(prefix_table.numel(), self.max_pages_per_seq)
            _want("prefix_table", prefix_table, i32, (prefix_table.numel(),), ix)
            _want("prefix_pages", prefix_pages, i32, (1,), ix)
            if capacity:
                prefix, pages = prefix_table.data_ptr(), prefix_pages.data_ptr()
        elif prefix_pages is not None:
            raise ValueError("prefix_pages without prefix_table")
        problem = self._problem
        if problem.num_free != num_free or problem.prefix_capacity != capacity:
            # (another object: a call on another thread may be using this one)
            problem = PagedTablesProblem.from_buffer_copy(problem)
            problem.num_free, problem.prefix_capacity = num_free, capacity
            self._problem = problem
        self._launch("dflash_paged_tables", stream, ctypes.byref(problem), cached_lens.data_ptr(),
                     new_lens.data_ptr(), held_pages.data_ptr(), free_pages.data_ptr(),
                     free_head.data_ptr(), prefix, pages, block_table.data_ptr(), ctx.data_ptr(),
                     held.data_ptr(), head.data_ptr(), starts.data_ptr(), positions.data_ptr(),
                     slots.data_ptr(), self.status.data_ptr())
        return out

    def read_flags(self, clear=False, stream=None) -> int:
        """The sticky status word behind what is on the stream, the current one or the given (waits for
        it): flags of calls on other streams may still be to come."""
        return self._read_flags(self.status, clear, stream)


_ROPE_LAYOUTS = {"half": DFLASH_ROPE_HALF, "interleaved": DFLASH_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"none": DFLASH_ROPE_SCALE_NONE, "linear": DFLASH_ROPE_SCALE_LINEAR,
                  "ntk": DFLASH_ROPE_SCALE_NTK, "yarn": DFLASH_ROPE_SCALE_YARN,
                  "wavelength": DFLASH_ROPE_SCALE_WAVELENGTH}
_ROPE_DTYPES = {torch.float16: DFLASH_FP16, torch.bfloat16: DFLASH_BF16}


class HeadNorm(collections.namedtuple("HeadNorm", ("q_weight", "k_weight", "eps",
                                                   "weight_offset"), defaults=(1e-6, 0.0))):
    """Norms of one layer's heads before their rotation: x * (weight_offset + weight) / sqrt(mean of
    x^2 + eps). Weights [head_dim] of the rotary's dtype; one that is None leaves its operand without
    a norm."""
    __slots__ = ()


class Rotary(_OnDevice):
    """Rotary positions of one model's heads: apply() rotates Q and K, kv_write() rotates Q and
    writes the rotated K and V into the paged E4M3 pools, mx4_write() into the 4-bit ones
    (dflash_rope_apply, dflash_rope_kv_write_live, dflash_mx4_kv_write). Each takes a HeadNorm for
    heads that are normed first."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, rotary_dim=None, layout="half",
                 dtype=torch.float16, base=10000.0, scaling="none", factor=1.0,
                 trained_context=1, beta_fast=32.0, beta_slow=1.0, low_turns=1.0, high_turns=4.0,
                 page_size=16, num_pages=1, device=None, status=None):
        super().__init__(device, "dflash_rope_apply", "dflash_rope_kv_write_live",
                         "dflash_norm_rope_apply", "dflash_norm_rope_kv_write",
                         "dflash_mx4_kv_write")
        if layout not in _ROPE_LAYOUTS or scaling not in _ROPE_SCALINGS:
            raise ValueError(f"unknown layout {layout!r} or scaling {scaling!r}")
        if dtype not in _ROPE_DTYPES:
            raise ValueError(f"dtype {dtype}: want float16 or bfloat16")
        self.dtype, self.shape = dtype, (num_q_heads, num_kv_heads, head_dim)
        self.pool_shape = (num_pages, page_size, num_kv_heads, head_dim)
        self.mx4_pool_shape = (num_pages, page_size // DFLASH_MX4_CHUNK_TOKENS, num_kv_heads,
                               DFLASH_MX4_CHUNK_BYTES)
        self.plan, phases = dflash_rope_plan(make_rope_problem(
            num_q_heads, num_kv_heads, head_dim, head_dim if rotary_dim is None else rotary_dim,
            _ROPE_LAYOUTS[layout], _ROPE_DTYPES[dtype], base, _ROPE_SCALINGS[scaling], factor,
            trained_context, beta_fast, beta_slow, low_turns, high_turns, page_size, num_pages))
        self._plan_ref = ctypes.byref(self.plan)
        # below 2^62: the same bits as int64
        self.phases = torch.tensor(list(phases), dtype=torch.int64, device=self.device)
        self.status = self._status_word(status)
        self._ready()

    def _norm_args(self, norm):
        """The C struct of a HeadNorm (None of None)."""
        if norm is None:
            return None
        D, ix = self.shape[2], self._index
        if norm.q_weight is not None:
            _want("norm.q_weight", norm.q_weight, self.dtype, (D,), ix)
        if norm.k_weight is not None:
            _want("norm.k_weight", norm.k_weight, self.dtype, (D,), ix)
        return ctypes.byref(HeadNormArgs(_ptr(norm.q_weight), _ptr(norm.k_weight), norm.eps,
                                         norm.weight_offset))

    def apply(self, q, k, positions, q_out=None, k_out=None, stream=None, norm=None):
        """(q_out, k_out): q [T, Hq, D] and k [T, Hkv, D] (or None), normed if a HeadNorm is given, rotated
        to positions [T]. q_out may be q itself, k_out k itself."""
        (Hq, Hkv, D), T, dt, ix = self.shape, positions.numel(), self.dtype, self._index
        q_shape, k_shape = (T, Hq, D), (T, Hkv, D)
        if q_out is None:
            q_out = self._empty(q_shape, dt, stream)
        qs = _want_rows("q", q, dt, q_shape, ix)
        qo = _want_rows("q_out", q_out, dt, q_shape, ix)
        _want("positions", positions, torch.int32, (T,), ix)
        ks = ko = 0
        if k is not None:
            if k_out is None:
                k_out = self._empty(k_shape, dt, stream)
            ks = _want_rows("k", k, dt, k_shape, ix)
            ko = _want_rows("k_out", k_out, dt, k_shape, ix)
        elif k_out is not None:
            raise ValueError("k_out without k")
        args = (T, q.data_ptr(), qs, _ptr(k), ks, positions.data_ptr(), self.phases.data_ptr(),
                q_out.data_ptr(), qo, _ptr(k_out), ko)
        if norm is None:
            self._launch("dflash_rope_apply", stream, self._plan_ref, *args)
        else:
            self._launch("dflash_norm_rope_apply", stream, self._plan_ref, self._norm_args(norm),
                         *args)
        return q_out, k_out

    def _write_args(self, q, k, v, positions, slots, pool_shape, k_pool, v_pool, q_out, stream,
                    token_starts):
        """Checks of both cache writes: q_out, the arguments up to num_live, and q_out's stride."""
        (Hq, Hkv, D), T, dt, ix = self.shape, positions.numel(), self.dtype, self._index
        q_shape, k_shape = (T, Hq, D), (T, Hkv, D)
        if q_out is None:
            q_out = self._empty(q_shape, dt, stream)
        qs = _want_rows("q", q, dt, q_shape, ix)
        qo = _want_rows("q_out", q_out, dt, q_shape, ix)
        ks = _want_rows("k", k, dt, k_shape, ix)
        vs = _want_rows("v", v, dt, k_shape, ix)
        _want("positions", positions, torch.int32, (T,), ix)
        _want("slots", slots, torch.int64, (T,), ix)
        _want("k_pool", k_pool, torch.uint8, pool_shape, ix)
        _want("v_pool", v_pool, torch.uint8, pool_shape, ix)
        live = None
        if token_starts is not None:
            n = token_starts.numel()
            _want("token_starts", token_starts, torch.int32, (n,), ix)
            if n < 1:
                raise ValueError("token_starts: want at least one entry")
            live = token_starts.data_ptr() + 4 * (n - 1)
        return q_out, (T, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                       positions.data_ptr(), slots.data_ptr(), live,
                       self.phases.data_ptr()), (q_out.data_ptr(), qo, k_pool.data_ptr(),
                                                 v_pool.data_ptr(), self.status.data_ptr())

    def kv_write(self, q, k, v, positions, slots, k_scale, v_scale, k_pool, v_pool, q_out=None,
                 stream=None, token_starts=None, norm=None):
        """q_out: q [T, Hq, D] rotated to positions [T] (it may be q itself); the rotated k and v
        [T, Hkv, D] go to the pools at slots [T]. A token with a negative slot is padding and left
        alone (its row of a q_out made here is not initialised). With token_starts (of PagedTables) only
        tokens past its last entry are: those inside the shared pages have no slot to write to either,
        but a query. With a HeadNorm q and k are normed before they are rotated."""
        q_out, args, outs = self._write_args(q, k, v, positions, slots, self.pool_shape, k_pool,
                                             v_pool, q_out, stream, token_starts)
        _want("k_scale", k_scale, torch.float32, (1,), self._index)
        _want("v_scale", v_scale, torch.float32, (1,), self._index)
        scales = k_scale.data_ptr(), v_scale.data_ptr()
        if norm is None:
            self._launch("dflash_rope_kv_write_live", stream, self._plan_ref, *args, *scales, *outs)
        else:
            self._launch("dflash_norm_rope_kv_write", stream, self._plan_ref,
                         self._norm_args(norm), *args, *scales, *outs)
        return q_out

    def mx4_write(self, q, k, v, positions, slots, k_pool, v_pool, q_out=None, norm=None,
                  stream=None, token_starts=None):
        """kv_write into the pools of an Mx4Cache, which need no scales."""
        q_out, args, outs = self._write_args(q, k, v, positions, slots, self.mx4_pool_shape, k_pool,
                                             v_pool, q_out, stream, token_starts)
        self._launch("dflash_mx4_kv_write", stream, self._plan_ref, self._norm_args(norm), *args,
                     *outs)
        return q_out

    def read_flags(self, clear=False, stream=None) -> int:
        """The sticky status word behind what is on the stream, the current one or the given (waits for
        it): flags of calls on other streams may still be to come."""
        return self._read_flags(self.status, clear, stream)


class SharedPrefixAttention(_OnDevice):
    """Verification attention of a batch whose sequences share their first tokens: the shared
    pages are read once for all of them (dflash_prefix_attn_forward). A plan plus its workspace;
    calls that may overlap on the GPU need an instance (or a workspace) each."""

    def __init__(self, batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                 max_pages_per_seq, num_pages, max_context, max_prefix, device=None,
                 kernel=DFLASH_PREFIX_KERNEL_AUTO, workspace=None):
        super().__init__(device, "dflash_prefix_attn_forward")
        self.problem = make_prefix_problem(batch, q_len, num_q_heads, num_kv_heads, head_dim,
                                           page_size, max_pages_per_seq, num_pages, max_context,
                                           max_prefix, self.device.index, kernel)
        self.plan = dflash_prefix_attn_plan(self.problem)
        self._plan_ref = ctypes.byref(self.plan)
        if workspace is None:
            workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8,
                                    device=self.device)
        elif (workspace.numel() * workspace.element_size() < self.plan.workspace_bytes
              or workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError("workspace: want plan.workspace_bytes contiguous bytes on "
                             f"{self.device}")
        self.workspace = workspace
        self._workspace_bytes = workspace.numel() * workspace.element_size()
        self.q_shape = (batch, q_len, num_q_heads, head_dim)
        self.pool_shape = (num_pages, page_size, num_kv_heads, head_dim)
        self._ready()

    def __call__(self, q, k_pool, v_pool, prefix_table, prefix_len, block_table, context_lens,
                 k_scale, v_scale, out=None, lse=None, stream=None):
        """(out, lse) of q over the pools. prefix_table: int32, the shared pages in order (at least
        floor(max_prefix / page_size) entries, None if that is 0); prefix_len: int32 [1], None when
        the plan's max_prefix is 0."""
        pr, ix, i32, f32 = self.problem, self._index, torch.int32, torch.float32
        q_shape, pool_shape = self.q_shape, self.pool_shape
        if out is None:
            out = self._empty(q_shape, torch.float16, stream)
        if lse is None:
            lse = self._empty(q_shape[:3], f32, stream)
        _want("q", q, torch.float16, q_shape, ix)
        _want("k_pool", k_pool, torch.uint8, pool_shape, ix)
        _want("v_pool", v_pool, torch.uint8, pool_shape, ix)
        _want("block_table", block_table, i32, (pr.batch, pr.max_pages_per_seq), ix)
        _want("context_lens", context_lens, i32, (pr.batch,), ix)
        _want("k_scale", k_scale, f32, (1,), ix)
        _want("v_scale", v_scale, f32, (1,), ix)
        _want("out", out, torch.float16, q_shape, ix)
        _want("lse", lse, f32, q_shape[:3], ix)
        if pr.max_prefix > 0:
            _want("prefix_len", prefix_len, i32, (1,), ix)
            pages = 0 if prefix_table is None else prefix_table.numel()
            if prefix_table is not None:
                _want("prefix_table", prefix_table, i32, (pages,), ix)
            if pages < pr.max_prefix // pr.page_size:
                raise ValueError("prefix_table has fewer pages than max_prefix fills")
        self._launch("dflash_prefix_attn_forward", stream, self._plan_ref, q.data_ptr(),
                     k_pool.data_ptr(), v_pool.data_ptr(), _ptr(prefix_table), _ptr(prefix_len),
                     block_table.data_ptr(), context_lens.data_ptr(), k_scale.data_ptr(),
                     v_scale.data_ptr(), self.workspace.data_ptr(), self._workspace_bytes,
                     out.data_ptr(), lse.data_ptr())
        return out, lse

    def read_flags(self, clear=False, stream=None) -> int:
        """The sticky status word behind what is on the stream, the current one or the given (waits for
        it): flags of calls on other streams may still be to come."""
        return self._read_flags(self.workspace, clear, stream)


_MX4_READ_DTYPES = {torch.float16: DFLASH_FP16, torch.bfloat16: DFLASH_BF16,
                    torch.float8_e5m2: DFLASH_E5M2}


class Mx4Cache(_OnDevice):
    """The pools of one layer's cache in 4 bits (include/dflash_mx4_cache.h has the format): empty()
    makes them, Rotary.mx4_write fills them, Mx4Attention attends over them, read() gives the numbers of
    cached tokens (dflash_mx4_read)."""

    def __init__(self, num_kv_heads, head_dim, page_size, num_pages, device=None, status=None):
        super().__init__(device, "dflash_mx4_read")
        if num_kv_heads < 1 or num_pages < 1 or page_size < 1:
            raise ValueError("num_kv_heads, page_size and num_pages: want at least 1")
        if head_dim != 256 or page_size % DFLASH_MX4_CHUNK_TOKENS:
            raise DflashError("Mx4Cache", DFLASH_ERR_UNSUPPORTED)
        self._dims = num_kv_heads, head_dim, page_size, num_pages
        self.pool_shape = (num_pages, page_size // DFLASH_MX4_CHUNK_TOKENS, num_kv_heads,
                           DFLASH_MX4_CHUNK_BYTES)
        self.status = self._status_word(status)
        self._ready()

    def empty(self):
        """(k_pool, v_pool), all zeros."""
        return tuple(torch.zeros(self.pool_shape, dtype=torch.uint8, device=self.device)
                     for _ in range(2))

    def read(self, k_pool, v_pool, slots, k_out=None, v_out=None, dtype=torch.float16, stream=None):
        """(k_out, v_out) [T, Hkv, D]: the tokens at slots [T], as numbers of the outputs' dtype (dtype
        for those made here): float16, bfloat16 or float8_e5m2. A pool that is None is left out. The
        rows of a negative slot stay as they are (not initialised if made here)."""
        (Hkv, D, _, _), T, ix = self._dims, slots.numel(), self._index
        _want("slots", slots, torch.int64, (T,), ix)
        given = next((o for o in (k_out, v_out) if o is not None), None)
        if given is not None:
            dtype = given.dtype
        if dtype not in _MX4_READ_DTYPES:
            raise ValueError(f"dtype {dtype}: want float16, bfloat16 or float8_e5m2")
        args, outs = [], []
        for name, pool, out in (("k", k_pool, k_out), ("v", v_pool, v_out)):
            if pool is None:
                if out is not None:
                    raise ValueError(f"{name}_out without {name}_pool")
                args += [None, 0]
            else:
                _want(f"{name}_pool", pool, torch.uint8, self.pool_shape, ix)
                if out is None:
                    out = self._empty((T, Hkv, D), dtype, stream)
                args += [out.data_ptr(), _want_rows(f"{name}_out", out, dtype, (T, Hkv, D), ix)]
            outs.append(out)
        self._launch("dflash_mx4_read", stream, *self._dims, _ptr(k_pool), _ptr(v_pool), T,
                     slots.data_ptr(), _MX4_READ_DTYPES[dtype], *args, self.status.data_ptr())
        return tuple(outs)

    def read_flags(self, clear=False, stream=None) -> int:
        """The sticky status word behind what is on the stream, the current one or the given (waits for
        it): flags of calls on other streams may still be to come."""
        return self._read_flags(self.status, clear, stream)


class Mx4Attention(_OnDevice):
    """Verification attention over the pools of an Mx4Cache: VerifyAttention without scales
    (dflash_mx4_attn_forward). A plan plus its workspace; calls that may overlap on the GPU need an
    instance (or a workspace) each."""

    def __init__(self, batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                 max_pages_per_seq, num_pages, max_context, device=None, num_splits=0,
                 workspace=None, flags=0):
        super().__init__(device, "dflash_mx4_attn_forward")
        self.problem = make_problem(batch, q_len, num_q_heads, num_kv_heads, head_dim, page_size,
                                    max_pages_per_seq, num_pages, max_context, self.device.index,
                                    num_splits, DFLASH_KERNEL_AUTO, flags)
        self.plan = dflash_mx4_attn_plan(self.problem)
        self._plan_ref = ctypes.byref(self.plan)
        if workspace is None:
            workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8,
                                    device=self.device)
        elif (workspace.numel() * workspace.element_size() < self.plan.workspace_bytes
              or workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError("workspace: want plan.workspace_bytes contiguous bytes on "
                             f"{self.device}")
        self.workspace = workspace
        self._workspace_bytes = workspace.numel() * workspace.element_size()
        self.q_shape = (batch, q_len, num_q_heads, head_dim)
        self.pool_shape = (num_pages, page_size // DFLASH_MX4_CHUNK_TOKENS, num_kv_heads,
                           DFLASH_MX4_CHUNK_BYTES)
        self._ready()

    def __call__(self, q, k_pool, v_pool, block_table, context_lens, out=None, lse=None,
                 stream=None):
        """(out, lse) of q [B, q_len, Hq, D] over the pools."""
        pr, ix, i32 = self.problem, self._index, torch.int32
        if out is None:
            out = self._empty(self.q_shape, torch.float16, stream)
        if lse is None:
            lse = self._empty(self.q_shape[:3], torch.float32, stream)
        _want("q", q, torch.float16, self.q_shape, ix)
        _want("k_pool", k_pool, torch.uint8, self.pool_shape, ix)
        _want("v_pool", v_pool, torch.uint8, self.pool_shape, ix)
        _want("block_table", block_table, i32, (pr.batch, pr.max_pages_per_seq), ix)
        _want("context_lens", context_lens, i32, (pr.batch,), ix)
        _want("out", out, torch.float16, self.q_shape, ix)
        _want("lse", lse, torch.float32, self.q_shape[:3], ix)
        self._launch("dflash_mx4_attn_forward", stream, self._plan_ref, q.data_ptr(),
                     k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
                     context_lens.data_ptr(), self.workspace.data_ptr(), self._workspace_bytes,
                     out.data_ptr(), lse.data_ptr())
        return out, lse

    def read_flags(self, clear=False, stream=None) -> int:
        """The sticky status word behind what is on the stream, the current one or the given (waits for
        it): flags of calls on other streams may still be to come."""
        return self._read_flags(self.workspace, clear, stream)
