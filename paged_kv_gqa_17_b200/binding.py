"""ctypes binding of libpkv.so (include/pkv.h): argument marshalling only.

Every step of the decode path (policy, queue, kernels, merge) runs inside the
C-ABI library; this module converts torch tensors to raw pointers, allocates
caller-owned buffers with torch and passes torch's current CUDA stream.  If
the library is missing or cannot be loaded, every call raises PkvError.
"""
from __future__ import annotations

import contextlib
import ctypes
import json
import os
import weakref
from dataclasses import dataclass
from typing import List, Optional, Sequence, Union

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpkv.so")

NO_SPLIT, SPLIT_S, WORK_QUEUE, BALANCED = 0, 1, 2, 3
FLAG_SEPARATE_MERGE, FLAG_NO_PDL, FLAG_DEEP_RING, FLAG_CLUSTER_MERGE, FLAG_PDL_EARLY = 1, 2, 4, 8, 16
FLAG_DEVICE_FILL = 32
FLAG_SHARED_PREFIX = 64
FLAG_SCORES = 128
EVICT_MAX_PLANES = 8
FILL_MAX_ROWS = 1024  # rows a device-fill plan can plan for on the device
INT32_MAX = 2**31 - 1
_MODE_NAMES = {"NO_SPLIT": NO_SPLIT, "SPLIT_S": SPLIT_S, "WORK_QUEUE": WORK_QUEUE, "BALANCED": BALANCED}

c_i32, c_i64, c_p, c_sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = _lib.pkv_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {name} ({status})" if what else f"{name} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [("B", c_i32), ("H_q", c_i32), ("H_kv", c_i32), ("head_dim", c_i32), ("page_size", c_i32),
                ("max_pages_per_seq", c_i32), ("num_pool_pages", c_i32), ("reserved", c_i32),
                ("kv_stride_page", c_i64), ("kv_stride_head", c_i64), ("kv_stride_token", c_i64)]


class Plan(ctypes.Structure):
    _fields_ = [("mode", c_i32), ("num_splits", c_i32), ("chunk_pages", c_i32), ("flags", c_i32)]

    def tuple(self):
        return (self.mode, self.num_splits, self.chunk_pages, self.flags)

    def __repr__(self):
        return f"Plan{self.tuple()}"


class WorkItem(ctypes.Structure):
    _fields_ = [("row", c_i32), ("kv_head", c_i32), ("tok_begin", c_i32), ("tok_end", c_i32)]


class Rule(ctypes.Structure):
    _fields_ = [("b_lo", c_i32), ("b_hi", c_i32), ("nmax_lo", c_i32), ("nmax_hi", c_i32), ("mode", c_i32),
                ("num_splits", c_i32), ("chunk_pages", c_i32), ("flags", c_i32)]

    def tuple(self):
        return tuple(getattr(self, f) for f, _ in self._fields_)


class Counters(ctypes.Structure):
    _fields_ = [(n, c_i64) for n in ("launches", "work_items", "empty_items", "merge_state_bytes", "kv_bytes",
                                     "kv_bytes_streamed", "q_bytes", "out_bytes", "queue_bytes",
                                     "bucket_launches")]

    def as_dict(self):
        return {f: int(getattr(self, f)) for f, _ in self._fields_}


class Plane(ctypes.Structure):
    """pkv_plane: one paged array that an eviction compacts (strides in bytes)."""
    _fields_ = [("base", c_p), ("stride_page", c_i64), ("stride_head", c_i64), ("stride_token", c_i64),
                ("row_bytes", c_i32), ("reserved", c_i32)]


class HostTiming(ctypes.Structure):
    """Where one pkv_decode_host call's time went (pkv_host_timing), in microseconds."""
    _fields_ = [(n, ctypes.c_double) for n in ("host_plan_us", "host_enqueue_us", "host_wait_us", "host_unpack_us",
                                               "dev_h2d_us", "dev_kernel_us", "dev_d2h_us", "host_events_us")]

    def as_dict(self):
        return {f: float(getattr(self, f)) for f, _ in self._fields_}


class HostCall(ctypes.Structure):
    """pkv_host_call: the arguments of pkv_decode_host as one parameter block."""
    _fields_ = [("q_host", c_p), ("block_table_host", c_p), ("seq_lens_host", c_p), ("out_host", c_p),
                ("k_pool", c_p), ("v_pool", c_p), ("scale", ctypes.c_float), ("shape", c_p), ("rules", c_p),
                ("n_rules", c_i32), ("device_buffer", c_p), ("device_buffer_bytes", c_sz), ("host_staging", c_p),
                ("host_staging_bytes", c_sz), ("stream", c_p), ("plan_out", c_p), ("timing", c_p)]


_lib = None

# (name, restype, argtypes) of every function include/pkv.h declares
SIGNATURES = [
    ("pkv_version", ctypes.c_char_p, []),
    ("pkv_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("pkv_default_policy", ctypes.c_int, [c_p, c_i32, c_p]),
    ("pkv_select_policy", ctypes.c_int, [c_p, c_p, c_p, c_i32, c_p]),
    ("pkv_work_queue_size", ctypes.c_int, [c_p, c_p, c_i32, c_p]),
    ("pkv_build_work_queue", ctypes.c_int, [c_p, c_p, c_i32, c_p, c_i32, c_p, c_p]),
    ("pkv_balanced_queue_size", ctypes.c_int, [c_p, c_p, c_i32, c_p]),
    ("pkv_build_balanced_queue", ctypes.c_int, [c_p, c_p, c_i32, c_p, c_i32, c_p, c_p]),
    ("pkv_balanced_queue_capacity", ctypes.c_int, [c_p, c_i32, c_p]),
    ("pkv_build_balanced_queue_device", ctypes.c_int, [c_p, c_p, c_i32, c_p, c_i32, c_p, c_p, c_p]),
    ("pkv_fill_queue_capacity", ctypes.c_int, [c_p, c_i32, c_p]),
    ("pkv_build_fill_queue_device", ctypes.c_int, [c_p, c_p, c_i32, c_p, c_i32, c_p, c_p, c_p]),
    ("pkv_prefix_queue_size", ctypes.c_int, [c_p, c_p, c_p, c_i32, c_i32, c_p, c_p]),
    ("pkv_build_prefix_queue", ctypes.c_int, [c_p, c_p, c_p, c_i32, c_i32, c_p, c_i32, c_p, c_i32, c_p, c_p]),
    ("pkv_plan_counters", ctypes.c_int, [c_p, c_p, c_p, c_p]),
    ("pkv_workspace_bytes", ctypes.c_int, [c_p, c_p, c_i32, c_p]),
    ("pkv_workspace_init", ctypes.c_int, [c_p, c_sz, c_p]),
    ("pkv_workspace_status", ctypes.c_int, [c_p, c_p, c_p]),
    ("pkv_collect_errors", ctypes.c_int, [c_p, c_p]),
    ("pkv_unplanned_status", ctypes.c_int, [c_p, c_p]),
    ("pkv_selftest_wait_timeout", ctypes.c_int, [c_p, c_sz, ctypes.c_uint32, c_p]),
    ("pkv_paged_decode", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_p, c_i32, ctypes.c_float, c_p, c_p, c_p, c_p, c_p, c_i32, c_p, c_sz, c_p]),
    ("pkv_paged_decode_scored", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_p, c_i32, ctypes.c_float, c_p, c_p, c_i64, c_i64, c_p, c_p, c_p, c_p, c_i32, c_p, c_sz,
      c_p]),
    ("pkv_evict_workspace_bytes", ctypes.c_int, [c_p, c_p]),
    ("pkv_evict_tokens", ctypes.c_int,
     [c_p, c_i64, c_i64, c_p, c_i64, c_i64, c_p, c_i32, c_p, c_p, c_i32, c_i32, c_p, c_p, c_p, c_sz, c_p]),
    ("pkv_mx4_append", ctypes.c_int,
     [c_p, c_p, c_i64, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_p, c_i32, c_p, c_p, c_p]),
    ("pkv_mx4_read", ctypes.c_int, [c_p, c_p, c_p, c_p, c_i32, c_p, c_p, c_p, c_p, c_p]),
    ("pkv_mx4_workspace_bytes", ctypes.c_int, [c_p, c_p, c_p]),
    ("pkv_mx4_decode", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_i32, ctypes.c_float, c_p, c_p, c_i64, c_i64, c_p, c_p, c_p, c_sz, c_p]),
    ("pkv_paged_decode_noalloc", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_p, c_i32, ctypes.c_float, c_p, c_p, c_p, c_p, c_p, c_i32, c_p]),
    ("pkv_noalloc_status", ctypes.c_int, [c_p, c_p]),
    ("pkv_decode_host_bytes", ctypes.c_int, [c_p, c_p, c_p, c_i32, c_p, c_p]),
    ("pkv_decode_host", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_p, c_p, ctypes.c_float, c_p, c_p, c_i32, c_p, c_sz, c_p, c_sz, c_p, c_p]),
    ("pkv_decode_host_timed", ctypes.c_int,
     [c_p, c_p, c_p, c_p, c_p, c_p, ctypes.c_float, c_p, c_p, c_i32, c_p, c_sz, c_p, c_sz, c_p, c_p, c_p]),
    ("pkv_decode_host_call", ctypes.c_int, [c_p]),
    ("pkv_decode_host_replays", ctypes.c_int64, []),
]


def lib(path: Optional[str] = None):
    """Load libpkv.so (built by paged_kv_gqa_17_b200.build); raise if it is missing.
    With `path`, load that build instead and make it the one every later call uses."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise PkvError(-4, f"{p} is missing; build it with `python -m paged_kv_gqa_17_b200.build`")
    handle = ctypes.CDLL(p)
    for name, res, args in SIGNATURES:
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    _lib = handle
    return handle


def _check(rc: int, what: str):
    if rc != 0:
        raise PkvError(rc, what)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _lens_array(seq_lens) -> ctypes.Array:
    if isinstance(seq_lens, torch.Tensor):
        seq_lens = seq_lens.detach().cpu().tolist()
    vals = [int(v) for v in seq_lens]
    return (c_i32 * max(1, len(vals)))(*vals), len(vals)


def make_shape(B: int, H_q: int, H_kv: int, head_dim: int, page_size: int, max_pages: int, num_pool_pages: int,
               layout: str = "HND") -> Shape:
    P, D = page_size, head_dim
    if layout == "HND":
        strides = (H_kv * P * D, P * D, D)
    elif layout == "NHD":
        strides = (P * H_kv * D, D, H_kv * D)
    else:
        raise ValueError(layout)
    return Shape(B, H_q, H_kv, D, P, max_pages, num_pool_pages, 0, *strides)


def shape_of(q: torch.Tensor, k_pool: torch.Tensor, block_table: torch.Tensor, layout: str = "HND",
             v_pool: Optional[torch.Tensor] = None) -> Shape:
    """Shape of a decode step from q [B][H_q][D], a pool and block_table [B][max_pages].

    The pool strides are the tensor's own (in elements), so a pool that is a
    view into a larger cache needs no copy: K and V halves of one combined
    cache ([pages][2][H_kv][P][D] gives k = kv[:, 0], v = kv[:, 1]), or pages
    padded past their last row.  The head_dim axis must be contiguous; with
    `v_pool`, its shape and strides must equal k_pool's (one set of strides
    serves both pools).  Axes of extent 1 take the packed stride, which is
    never used to address an element."""
    if k_pool.dim() != 4:
        raise ValueError(f"k_pool must be 4-D, got shape {tuple(k_pool.shape)}")
    if v_pool is not None and (tuple(v_pool.shape) != tuple(k_pool.shape) or v_pool.stride() != k_pool.stride()):
        raise ValueError("k_pool and v_pool must have the same shape and strides")
    B, H_q, D = (int(x) for x in q.shape)
    if layout == "HND":
        (pages, H_kv, P, _), (sp, sh, st, sd) = k_pool.shape, k_pool.stride()
    elif layout == "NHD":
        (pages, P, H_kv, _), (sp, st, sh, sd) = k_pool.shape, k_pool.stride()
    else:
        raise ValueError(layout)
    if sd != 1 and D > 1:
        raise ValueError("the pool's head_dim axis must be contiguous (stride 1)")
    s = make_shape(B, H_q, int(H_kv), D, int(P), int(block_table.shape[1]), int(pages), layout)
    if pages > 1:
        s.kv_stride_page = sp
    if H_kv > 1:
        s.kv_stride_head = sh
    if P > 1:
        s.kv_stride_token = st
    return s


_DECODE_DTYPES = (torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.int32, torch.int32)


def _check_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, shape: Shape):
    """Reject tensors whose type, layout or device differs from what the
    pointers passed to the library are taken to address.  One combined test
    (a few microseconds) passes every well-formed call; only a failing call
    runs the itemised checks that name the problem."""
    dev = q.get_device()
    kst = k_pool.stride()
    if ((q.dtype, out.dtype, k_pool.dtype, v_pool.dtype, block_table.dtype, seq_lens.dtype) == _DECODE_DTYPES
            and dev >= 0 and out.get_device() == dev and k_pool.get_device() == dev
            and v_pool.get_device() == dev and block_table.get_device() == dev and seq_lens.get_device() == dev
            and q.is_contiguous() and out.is_contiguous() and block_table.is_contiguous()
            and seq_lens.is_contiguous()
            and q.shape == (shape.B, shape.H_q, shape.head_dim) and out.shape == q.shape
            and block_table.shape == (shape.B, shape.max_pages_per_seq) and seq_lens.numel() >= shape.B
            and len(kst) == 4 and v_pool.stride() == kst and v_pool.shape == k_pool.shape
            and k_pool.shape[0] >= shape.num_pool_pages
            and (k_pool.shape[0] <= 1 or kst[0] == shape.kv_stride_page)
            and (kst[3] == 1 or shape.head_dim <= 1)):
        return
    _diagnose_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, shape)
    raise ValueError("tensors do not match the plan's shape")


def _diagnose_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, shape: Shape):
    for name, t, dt in (("q", q, torch.bfloat16), ("out", out, torch.bfloat16), ("k_pool", k_pool, torch.bfloat16),
                        ("v_pool", v_pool, torch.bfloat16), ("block_table", block_table, torch.int32),
                        ("seq_lens", seq_lens, torch.int32)):
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    for name, t in (("q", q), ("out", out), ("block_table", block_table), ("seq_lens", seq_lens)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    want = (shape.B, shape.H_q, shape.head_dim)
    if tuple(q.shape) != want or tuple(out.shape) != want:
        raise ValueError(f"q and out must be {list(want)}, got {list(q.shape)} and {list(out.shape)}")
    if tuple(block_table.shape) != (shape.B, shape.max_pages_per_seq):
        raise ValueError(f"block_table must be [{shape.B}][{shape.max_pages_per_seq}], got {list(block_table.shape)}")
    if seq_lens.numel() < shape.B:
        raise ValueError(f"seq_lens holds {seq_lens.numel()} lengths for {shape.B} rows")
    if k_pool.dim() != 4 or tuple(v_pool.shape) != tuple(k_pool.shape) or v_pool.stride() != k_pool.stride():
        raise ValueError("k_pool and v_pool must be 4-D with the same shape and strides")
    if k_pool.shape[0] < shape.num_pool_pages or (k_pool.shape[0] > 1 and k_pool.stride(0) != shape.kv_stride_page):
        raise ValueError("the pools' pages differ from the plan's shape (page count or page stride)")
    if k_pool.stride(-1) != 1 and shape.head_dim > 1:
        raise ValueError("the pools' head_dim axis must be contiguous (stride 1)")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"q must be on a CUDA device, not {dev}")
    for name, t in (("out", out), ("k_pool", k_pool), ("v_pool", v_pool), ("block_table", block_table),
                    ("seq_lens", seq_lens)):
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, q on {dev}")


def _check_host_call(q_host, block_table_host, seq_lens_host, out_host, k_pool, v_pool, shape: Shape,
                     device_index: int):
    """The tensors of a pkv_decode_host call: host q / out (bf16 [B][H_q][D]),
    host table (int32 [B][max_pages]) and lengths (int32, >= B), contiguous;
    pools on the decoder's CUDA device with the shape's page count and strides."""
    n_q = shape.B * shape.H_q * shape.head_dim
    for name, t, dt, n in (("q_host", q_host, torch.bfloat16, n_q), ("out_host", out_host, torch.bfloat16, n_q),
                           ("block_table_host", block_table_host, torch.int32, shape.B * shape.max_pages_per_seq),
                           ("seq_lens_host", seq_lens_host, torch.int32, None)):
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        if t.device.type != "cpu":
            raise ValueError(f"{name} must be a host tensor, not on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if n is not None and t.numel() != n:
            raise ValueError(f"{name} holds {t.numel()} elements, the shape needs {n}")
    if seq_lens_host.numel() < shape.B:
        raise ValueError(f"seq_lens_host holds {seq_lens_host.numel()} lengths for {shape.B} rows")
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.get_device() != device_index:
            raise ValueError(f"{name} must be on the decoder's device cuda:{device_index}")
    if k_pool.dim() != 4 or tuple(v_pool.shape) != tuple(k_pool.shape) or v_pool.stride() != k_pool.stride():
        raise ValueError("k_pool and v_pool must be 4-D with the same shape and strides")
    if k_pool.shape[0] < shape.num_pool_pages or (k_pool.shape[0] > 1 and k_pool.stride(0) != shape.kv_stride_page):
        raise ValueError("the pools' pages differ from the shape (page count or page stride)")
    if k_pool.stride(-1) != 1 and shape.head_dim > 1:
        raise ValueError("the pools' head_dim axis must be contiguous (stride 1)")


def rules_array(rules: Optional[Sequence]) -> tuple:
    """(ctypes array or None, count) from Rule structs, tuples or dicts."""
    if rules is None:
        return None, 0
    out = []
    for r in rules:
        if isinstance(r, Rule):
            out.append(r)
        elif isinstance(r, dict):
            mode = _MODE_NAMES[r["mode"]] if isinstance(r["mode"], str) else int(r["mode"])
            out.append(Rule(int(r["b_lo"]), int(r.get("b_hi", INT32_MAX)), int(r["nmax_lo"]),
                            int(r.get("nmax_hi", INT32_MAX)), mode, int(r.get("num_splits", 1)),
                            int(r.get("chunk_pages", 0)), int(r.get("flags", 0))))
        else:
            out.append(Rule(*[int(v) for v in r]))
    return (Rule * max(1, len(out)))(*out), len(out)


def load_rules(path: str) -> List[Rule]:
    """Read a policy table JSON ({"rules": [...]}) into Rule structs."""
    with open(path) as f:
        doc = json.load(f)
    arr, n = rules_array(doc["rules"])
    return [arr[i] for i in range(n)]


def default_rules() -> List[Rule]:
    L = lib()
    n = c_i32(0)
    L.pkv_default_policy(None, 0, ctypes.byref(n))
    arr = (Rule * max(1, n.value))()
    _check(L.pkv_default_policy(arr, n.value, ctypes.byref(n)), "pkv_default_policy")
    return [arr[i] for i in range(n.value)]


def select_policy(seq_lens_host, shape: Shape, rules=None) -> Plan:
    L = lib()
    lens, _ = _lens_array(seq_lens_host)
    arr, n = rules_array(rules)
    plan = Plan()
    _check(L.pkv_select_policy(lens, ctypes.byref(shape), arr, n, ctypes.byref(plan)), "pkv_select_policy")
    return plan


def build_work_queue(seq_lens_host, shape: Shape, chunk_pages: int):
    """-> (items int32 tensor [n][4] on the CPU, indptr int32 tensor [B*H_kv + 1])."""
    L = lib()
    lens, _ = _lens_array(seq_lens_host)
    n = c_i32(0)
    _check(L.pkv_work_queue_size(lens, ctypes.byref(shape), chunk_pages, ctypes.byref(n)), "pkv_work_queue_size")
    items = torch.zeros((max(1, n.value), 4), dtype=torch.int32)
    indptr = torch.zeros(shape.B * shape.H_kv + 1, dtype=torch.int32)
    _check(L.pkv_build_work_queue(lens, ctypes.byref(shape), chunk_pages, items.data_ptr(), n.value,
                                  indptr.data_ptr(), ctypes.byref(n)), "pkv_build_work_queue")
    return items[:n.value], indptr


def build_balanced_queue(seq_lens_host, shape: Shape, n_blocks: int):
    """-> (items int32 [n][4], indptr int32 [B*H_kv + 1 + n_blocks + 1]: pair offsets, then block offsets)."""
    L = lib()
    lens, _ = _lens_array(seq_lens_host)
    n = c_i32(0)
    _check(L.pkv_balanced_queue_size(lens, ctypes.byref(shape), n_blocks, ctypes.byref(n)),
           "pkv_balanced_queue_size")
    items = torch.zeros((max(1, n.value), 4), dtype=torch.int32)
    indptr = torch.zeros(shape.B * shape.H_kv + 1 + n_blocks + 1, dtype=torch.int32)
    _check(L.pkv_build_balanced_queue(lens, ctypes.byref(shape), n_blocks, items.data_ptr(), n.value,
                                      indptr.data_ptr(), ctypes.byref(n)), "pkv_build_balanced_queue")
    return items[:n.value], indptr


def build_prefix_queue(seq_lens_host, block_table_host, shape: Shape, chunk_pages: int, max_members: int):
    """-> (items int32 [n][4], indptr int32: pair offsets [B*H_kv + 1], unit offsets
    [n_units + 1], the units' member item indices [n]; n_units).  The queue that
    stages shared prefix pages once for several rows (pkv_build_prefix_queue)."""
    L = lib()
    lens, _ = _lens_array(seq_lens_host)
    bt = torch.as_tensor(block_table_host, dtype=torch.int32).cpu().contiguous()
    n, u = c_i32(0), c_i32(0)
    _check(L.pkv_prefix_queue_size(lens, bt.data_ptr(), ctypes.byref(shape), chunk_pages, max_members,
                                   ctypes.byref(n), ctypes.byref(u)), "pkv_prefix_queue_size")
    items = torch.zeros((max(1, n.value), 4), dtype=torch.int32)
    n_ptr = shape.B * shape.H_kv + 1 + u.value + 1 + n.value
    indptr = torch.zeros(n_ptr, dtype=torch.int32)
    _check(L.pkv_build_prefix_queue(lens, bt.data_ptr(), ctypes.byref(shape), chunk_pages, max_members,
                                    items.data_ptr(), n.value, indptr.data_ptr(), n_ptr, ctypes.byref(n),
                                    ctypes.byref(u)), "pkv_build_prefix_queue")
    return items[:n.value], indptr, int(u.value)


def balanced_queue_capacity(shape: Shape, n_blocks: int) -> int:
    L = lib()
    n = c_i32(0)
    _check(L.pkv_balanced_queue_capacity(ctypes.byref(shape), n_blocks, ctypes.byref(n)), "pkv_balanced_queue_capacity")
    return int(n.value)


def build_balanced_queue_device(seq_lens: torch.Tensor, shape: Shape, n_blocks: int, items: torch.Tensor,
                                indptr: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """pkv_build_balanced_queue_device: the balanced queue built on the GPU from
    device lengths into `items` / `indptr` (see include/pkv.h)."""
    L = lib()
    _check(L.pkv_build_balanced_queue_device(seq_lens.data_ptr(), ctypes.byref(shape), n_blocks, items.data_ptr(),
                                             int(items.shape[0]), indptr.data_ptr(), workspace.data_ptr(),
                                             _stream_ptr(stream)), "pkv_build_balanced_queue_device")


def fill_queue_capacity(shape: Shape, n_blocks: int) -> int:
    L = lib()
    n = c_i32(0)
    _check(L.pkv_fill_queue_capacity(ctypes.byref(shape), n_blocks, ctypes.byref(n)), "pkv_fill_queue_capacity")
    return int(n.value)


def build_fill_queue_device(seq_lens: torch.Tensor, shape: Shape, n_blocks: int, items: torch.Tensor,
                            indptr: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """pkv_build_fill_queue_device: the queue whose chunk fills one wave of
    n_blocks blocks, built on the GPU from device lengths (see include/pkv.h)."""
    L = lib()
    _check(L.pkv_build_fill_queue_device(seq_lens.data_ptr(), ctypes.byref(shape), n_blocks, items.data_ptr(),
                                         int(items.shape[0]), indptr.data_ptr(), workspace.data_ptr(),
                                         _stream_ptr(stream)), "pkv_build_fill_queue_device")


def plan_counters(seq_lens_host, shape: Shape, plan: Plan) -> dict:
    L = lib()
    lens, _ = _lens_array(seq_lens_host)
    c = Counters()
    _check(L.pkv_plan_counters(lens, ctypes.byref(shape), ctypes.byref(plan), ctypes.byref(c)), "pkv_plan_counters")
    return c.as_dict()


def workspace_bytes(shape: Shape, plan: Plan, n_items: int = 0) -> int:
    L = lib()
    b = c_sz(0)
    _check(L.pkv_workspace_bytes(ctypes.byref(shape), ctypes.byref(plan), n_items, ctypes.byref(b)),
           "pkv_workspace_bytes")
    return int(b.value)


def _stream_ptr(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


@dataclass
class DecodePlan:
    """Everything a decode step needs besides the tensors: the plan, the queue
    on the device (WORK_QUEUE, BALANCED) and a zeroed workspace.  Reusable for
    every step with the same sequence lengths and shape; with device_queue
    the queue comes from the device lengths at every step (built by a kernel
    of its own, or derived by each decode block under PKV_FLAG_DEVICE_FILL),
    so the plan serves any lengths up to the shape's maximum."""

    shape: Shape
    plan: Plan
    items: Optional[torch.Tensor]
    indptr: Optional[torch.Tensor]
    n_items: int
    workspace: torch.Tensor
    counters: dict
    device_queue: bool = False
    fill_blocks: int = 0  # device queue of a WORK_QUEUE plan: the wave it fills


def prefix_counters(seq_lens_host, shape: Shape, items: torch.Tensor, indptr: torch.Tensor, n_units: int,
                    flags: int = 0) -> dict:
    """Workload counters of a prefix-sharing plan, counted from its queue: one
    block per unit, a unit's pages streamed once for all its members."""
    lens = [int(n) for n in (seq_lens_host.tolist() if isinstance(seq_lens_host, torch.Tensor) else seq_lens_host)]
    B, H_kv, D, P = shape.B, shape.H_kv, shape.head_dim, shape.page_size
    G = shape.H_q // H_kv
    pairs = B * H_kv
    ptr = indptr.tolist()
    it = items.tolist()
    uptr = ptr[pairs + 1:pairs + 2 + n_units]
    uitems = ptr[pairs + 2 + n_units:]
    per_pair = [ptr[k + 1] - ptr[k] for k in range(pairs)]
    streamed = 0
    for u in range(n_units):
        _, _, tb, te = it[uitems[uptr[u]]]
        streamed += (-(-te // P) - tb // P) if te > tb else 0
    return {"launches": 1 + (1 if flags & FLAG_SEPARATE_MERGE else 0), "work_items": n_units,
            "empty_items": H_kv * sum(1 for n in lens if n == 0),
            "merge_state_bytes": 2 * sum(k for k in per_pair if k > 1) * G * (D + 2) * 4,
            "kv_bytes": sum(lens) * H_kv * 2 * D * 2, "kv_bytes_streamed": streamed * P * 2 * D * 2,
            "q_bytes": B * shape.H_q * D * 2, "out_bytes": B * shape.H_q * D * 2,
            "queue_bytes": 16 * len(it) + 4 * len(ptr), "bucket_launches": 2 * len({n for n in lens if n > 0})}


def plan_decode(seq_lens_host, shape: Shape, device, rules=None, plan: Optional[Plan] = None,
                device_queue: bool = False, fill_blocks: int = 296,
                device_fill: Optional[bool] = None, shared_prefix_table=None, scores: bool = False) -> DecodePlan:
    """Host planning for one batch: policy (unless `plan` is given), queue, workspace.

    scores=True plans for paged_decode_scored (PKV_FLAG_SCORES: the workspace
    also holds every token's logits).  The policy's pick keeps its mode, but
    merges through the workspace rather than in a cluster, and a BALANCED
    pick becomes the work queue that fills one wave of its blocks; a `plan`
    or rule with PKV_FLAG_SCORES asks for the same.

    shared_prefix_table (the host block table) asks for the queue that stages
    the prefix pages rows share once for several rows (pkv_build_prefix_queue
    at the plan's chunk; PKV_FLAG_SHARED_PREFIX); a NO_SPLIT plan stays as is.

    device_queue=True leaves the queue to the GPU, rebuilt from the device
    lengths by every paged_decode call (so one plan, or one captured CUDA
    graph, serves any lengths up to the shape's maximum): a BALANCED plan
    gets the balanced queue of its T blocks, a WORK_QUEUE plan the queue
    whose chunk fills one wave of `fill_blocks` blocks.  For the latter the
    decode blocks derive their own items (PKV_FLAG_DEVICE_FILL, one launch)
    where the plan allows it (B <= 1024, merge fused); device_fill=False
    asks for the builder kernel instead.  NO_SPLIT and SPLIT_S plans have no
    queue and read the lengths on the device anyway; they serve lengths up
    to those they were planned for (SPLIT_S: S' chunks of C pages)."""
    given = plan
    if plan is None:
        plan = select_policy(seq_lens_host, shape, rules)
    if scores or plan.flags & FLAG_SCORES:
        if shared_prefix_table is not None or plan.flags & FLAG_SHARED_PREFIX:
            raise ValueError("a scored plan has no prefix-sharing queue")
        plan = Plan.from_buffer_copy(plan)
        plan.flags = (plan.flags | FLAG_SCORES) & ~FLAG_CLUSTER_MERGE
        if plan.mode == BALANCED:
            if given is not None:
                raise ValueError("a scored plan is NO_SPLIT, SPLIT_S or WORK_QUEUE")
            fill = [Rule(0, INT32_MAX, 0, INT32_MAX, WORK_QUEUE, plan.num_splits, 0, plan.flags)]
            plan = select_policy(seq_lens_host, shape, fill)
    if shared_prefix_table is not None and plan.mode != NO_SPLIT or (plan.flags & FLAG_SHARED_PREFIX):
        # the prefix-sharing queue at the plan's chunk (a queue-free plan's whole rows otherwise)
        if shared_prefix_table is None:
            raise ValueError("a shared-prefix plan needs the host block table (shared_prefix_table)")
        lens = [int(n) for n in (seq_lens_host.tolist() if isinstance(seq_lens_host, torch.Tensor)
                                 else seq_lens_host)]
        pages_max = max([-(-n // shape.page_size) for n in lens] + [1])
        C = plan.chunk_pages if plan.mode in (SPLIT_S, WORK_QUEUE) and plan.chunk_pages > 0 else pages_max
        members = max(1, 16 // (shape.H_q // shape.H_kv))
        items_h, indptr_h, n_units = build_prefix_queue(lens, shared_prefix_table, shape, C, members)
        flags = (plan.flags | FLAG_SHARED_PREFIX) & ~(FLAG_DEVICE_FILL | FLAG_PDL_EARLY | FLAG_CLUSTER_MERGE)
        pplan = Plan(WORK_QUEUE, n_units, C, flags)
        n_items = int(items_h.shape[0])
        ws = torch.zeros(workspace_bytes(shape, pplan, n_items), dtype=torch.uint8, device=device)
        return DecodePlan(shape, pplan, items_h.to(device), indptr_h.to(device), n_items, ws,
                          prefix_counters(lens, shape, items_h, indptr_h, n_units, flags))
    if plan.mode == WORK_QUEUE and plan.flags & FLAG_DEVICE_FILL:
        device_queue, device_fill, fill_blocks = True, True, plan.num_splits
    if device_queue and plan.mode == WORK_QUEUE:
        fill_ok = shape.B <= FILL_MAX_ROWS and not plan.flags & FLAG_SEPARATE_MERGE
        if device_fill is None:
            device_fill = fill_ok
        if device_fill:
            if not fill_ok:
                raise ValueError("a device-fill plan needs B <= 1024 and the fused merge")
            dplan = Plan(WORK_QUEUE, fill_blocks, 0, plan.flags | FLAG_DEVICE_FILL)
            cap = max(fill_blocks, shape.B * shape.H_kv)
            ws = torch.zeros(workspace_bytes(shape, dplan, cap), dtype=torch.uint8, device=device)
            return DecodePlan(shape, dplan, None, None, cap, ws, plan_counters(seq_lens_host, shape, dplan), True,
                              fill_blocks)
    if device_queue and plan.mode in (WORK_QUEUE, BALANCED):
        pairs = shape.B * shape.H_kv
        if plan.mode == BALANCED:
            cap = balanced_queue_capacity(shape, plan.num_splits)
            n_ptr = pairs + 1 + plan.num_splits + 1
        else:
            cap = fill_queue_capacity(shape, fill_blocks)
            n_ptr = pairs + 1
        items = torch.zeros((cap, 4), dtype=torch.int32, device=device)
        indptr = torch.zeros(n_ptr, dtype=torch.int32, device=device)
        ws = torch.zeros(workspace_bytes(shape, plan, cap), dtype=torch.uint8, device=device)
        return DecodePlan(shape, plan, items, indptr, cap, ws, plan_counters(seq_lens_host, shape, plan), True,
                          fill_blocks if plan.mode == WORK_QUEUE else 0)
    items = indptr = None
    n_items = 0
    if plan.mode in (WORK_QUEUE, BALANCED):
        if plan.mode == WORK_QUEUE:
            items_h, indptr_h = build_work_queue(seq_lens_host, shape, plan.chunk_pages)
        else:
            items_h, indptr_h = build_balanced_queue(seq_lens_host, shape, plan.num_splits)
        n_items = int(items_h.shape[0])
        items = items_h.to(device)
        indptr = indptr_h.to(device)
    ws = torch.zeros(workspace_bytes(shape, plan, n_items), dtype=torch.uint8, device=device)
    return DecodePlan(shape, plan, items, indptr, n_items, ws, plan_counters(seq_lens_host, shape, plan))


def _own_decode_plan(q, seq_lens, seq_lens_host, shape: Shape, rules, scores: bool, stream) -> DecodePlan:
    """The plan of a decode that was given none.  All of it belongs to the call's stream: the lengths are read behind
    what is queued there, and the workspace's memory is not reused before the call's kernels are done."""
    with _on(q.get_device(), stream):
        host = seq_lens_host if seq_lens_host is not None else seq_lens.detach().cpu()
        return plan_decode(host, shape, q.device, rules, scores=scores)


def paged_decode(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, page_size: int, scale: float, *, plan: Optional[DecodePlan] = None,
                 seq_lens_host=None, layout: str = "HND", rules=None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out = softmax(scale * q K^T) V per (row, query head), read through the block table.

    q bf16 [B][H_q][D]; pools bf16 (layout "HND" [pages][H_kv][P][D] or "NHD"
    [pages][P][H_kv][D], any strides with a contiguous head_dim axis, see
    shape_of); block_table int32 [B][max_pages]; seq_lens int32 [B], all on one
    CUDA device.  Without `plan`, the policy and queue are built from
    `seq_lens_host` (or a host copy of seq_lens, made in the order of the call's stream).  Tensors of another dtype,
    device or layout raise TypeError / ValueError before anything is launched.
    Errors that the kernels meet on device data: workspace_status(plan), or
    without a plan unplanned_status().
    """
    L = lib()
    own = plan is None
    if own:
        shape = shape_of(q, k_pool, block_table, layout, v_pool)
        plan = _own_decode_plan(q, seq_lens, seq_lens_host, shape, rules, False, stream)
    shape = plan.shape
    if out is None:
        out = torch.empty_like(q)
    _check_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, shape)
    if plan.device_queue and plan.plan.mode == BALANCED:
        build_balanced_queue_device(seq_lens, shape, plan.plan.num_splits, plan.items, plan.indptr, plan.workspace,
                                    stream)
    elif plan.device_queue and plan.plan.flags & FLAG_DEVICE_FILL:
        pass  # every decode block derives its own item from the device lengths
    elif plan.device_queue:
        build_fill_queue_device(seq_lens, shape, plan.fill_blocks, plan.items, plan.indptr, plan.workspace, stream)
    rc = L.pkv_paged_decode(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
                            seq_lens.data_ptr(), page_size, float(scale), out.data_ptr(), ctypes.byref(shape),
                            ctypes.byref(plan.plan), plan.items.data_ptr() if plan.items is not None else None,
                            plan.indptr.data_ptr() if plan.indptr is not None else None, plan.n_items,
                            plan.workspace.data_ptr(), plan.workspace.numel(), _stream_ptr(stream))
    _check(rc, "pkv_paged_decode")
    if own:
        _collect(plan, q.get_device(), stream)
    return out


def paged_decode_noalloc(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, page_size: int, scale: float, plan: DecodePlan,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pkv_paged_decode_noalloc: like paged_decode, but the library's own fixed
    scratch array replaces the plan's workspace (for callers that cannot
    allocate device memory; see include/pkv.h)."""
    L = lib()
    if out is None:
        out = torch.empty_like(q)
    _check_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, plan.shape)
    rc = L.pkv_paged_decode_noalloc(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
                                    seq_lens.data_ptr(), page_size, float(scale), out.data_ptr(),
                                    ctypes.byref(plan.shape), ctypes.byref(plan.plan),
                                    plan.items.data_ptr() if plan.items is not None else None,
                                    plan.indptr.data_ptr() if plan.indptr is not None else None, plan.n_items,
                                    _stream_ptr(stream))
    _check(rc, "pkv_paged_decode_noalloc")
    return out


# The current stream's handle of a device as an integer, without the Stream
# object (a fifth of a microsecond instead of two).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index: int, stream):
    """Context in which a call's kernels and allocations belong to `stream` (default: the current stream of CUDA
    device `index`), whatever device is current.  No device (index -1, a tensor that the checks refuse): none."""
    if index < 0:
        return contextlib.nullcontext()
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{index}")
    return torch.cuda.stream(stream)


def _launch(fn, what: str, index: int, stream, *args):
    """fn(*args, stream handle) with CUDA device `index` current; raises on an error status."""
    if stream is None and torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with _on(index, stream):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise PkvError(rc, what)


def _collect(plan, index: int, stream):
    """The device errors of a call that made its own plan, for unplanned_status()."""
    _launch(lib().pkv_collect_errors, "pkv_collect_errors", index, stream, plan.workspace.data_ptr())


def _empty(shape, dtype, index: int, stream) -> torch.Tensor:
    """A new tensor on CUDA device `index` that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=index)
    with _on(index, stream):
        return torch.empty(shape, dtype=dtype, device=index)


def _empty_like(t: torch.Tensor, index: int, stream) -> torch.Tensor:
    """The same by a (CUDA, contiguous) tensor's example, which is cheaper."""
    if stream is None:
        return torch.empty_like(t)
    with _on(index, stream):
        return torch.empty_like(t)


def _cuda_index(name: str, t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device, not {t.device}")
    return index


def _check_plan(plan, index: int):
    if plan.workspace.get_device() != index:
        raise ValueError(f"the plan was made on {plan.workspace.device}, the tensors are on cuda:{index}")


def _check_tensor(name: str, t: torch.Tensor, dtype, index: int, contiguous: bool = True):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, not {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_scores(name: str, t: torch.Tensor, dtype, B: int, H_kv: int, max_pages: int, index: int) -> tuple:
    """[B][H_kv][>= max_pages * 16] with contiguous tokens, no two elements in one place; returns the strides."""
    _check_tensor(name, t, dtype, index, contiguous=False)
    shape = t.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != H_kv or shape[2] < max_pages * 16:
        raise ValueError(f"{name} must be [{B}][{H_kv}][>= {max_pages * 16}], got {list(shape)}")
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name}'s tokens must be contiguous")
    if st[1] < shape[2] or st[0] < st[1] * H_kv:  # not nested in the plain order
        _check_no_overlap(name, shape, st)
    return st


def _check_no_overlap(name: str, shape, strides):
    """Reject views (expanded, overlapping) in which two elements share memory: they would be written twice."""
    reach = 1
    for size, stride in sorted(((s, st) for s, st in zip(shape, strides) if s > 1), key=lambda x: x[1]):
        if stride < reach:
            raise ValueError(f"{name} has elements that share memory")
        reach = stride * (size - 1) + reach


def paged_decode_scored(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, page_size: int, scale: float, scores: torch.Tensor, *,
                        plan: Optional[DecodePlan] = None, seq_lens_host=None, layout: str = "HND", rules=None,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_decode that also adds every cached token's attention weight, summed over the query heads of its KV
    head, to `scores` (fp32 [B][H_kv][>= max_pages * 16], contiguous tokens, in place):

        scores[i, h, t] += sum over the G heads of KV head h of softmax(scale * q K^T)[t],  t < seq_lens[i]

    the input of evict_tokens.  `plan` comes from plan_decode(..., scores=True); elements past a row's length
    are left alone.  Everything else as paged_decode."""
    L = lib()
    index = _cuda_index("q", q)
    own = plan is None
    if own:
        shape = shape_of(q, k_pool, block_table, layout, v_pool)
        plan = _own_decode_plan(q, seq_lens, seq_lens_host, shape, rules, True, stream)
    shape = plan.shape
    if not plan.plan.flags & FLAG_SCORES:
        raise ValueError("the plan was not made for scores: plan_decode(..., scores=True)")
    _check_plan(plan, index)
    if out is None:
        out = _empty_like(q, index, stream)
    _check_decode_tensors(q, k_pool, v_pool, block_table, seq_lens, out, shape)
    st = _check_scores("scores", scores, torch.float32, shape.B, shape.H_kv, shape.max_pages_per_seq, index)
    ws = plan.workspace
    items = indptr = None
    if plan.items is not None:
        items, indptr = plan.items.data_ptr(), plan.indptr.data_ptr()
        if plan.device_queue:
            _launch(L.pkv_build_fill_queue_device, "pkv_build_fill_queue_device", index, stream, seq_lens.data_ptr(),
                    ctypes.byref(shape), plan.fill_blocks, items, int(plan.items.shape[0]), indptr, ws.data_ptr())
    _launch(L.pkv_paged_decode_scored, "pkv_paged_decode_scored", index, stream, q.data_ptr(), k_pool.data_ptr(),
            v_pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), page_size, scale, out.data_ptr(),
            scores.data_ptr(), st[0], st[1], ctypes.byref(shape), ctypes.byref(plan.plan), items, indptr, plan.n_items,
            ws.data_ptr(), ws.numel())
    if own:
        _collect(plan, index, stream)
    return out


@dataclass
class EvictPlan:
    """What evict_tokens needs besides the tensors: the shape and a zeroed workspace, reusable for any lengths,
    scores, budget and planes of that batch."""

    shape: Shape
    workspace: torch.Tensor


def plan_evict(B: int, H_kv: int, max_pages: int, device) -> EvictPlan:
    """Workspace for evict_tokens over B rows of H_kv KV heads and block tables of max_pages columns."""
    L = lib()
    shape = make_shape(B, H_kv, H_kv, 128, 16, max_pages, 1)
    n = c_sz(0)
    _check(L.pkv_evict_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "pkv_evict_workspace_bytes")
    return EvictPlan(shape, torch.zeros(n.value, dtype=torch.uint8, device=device))


def evict_tokens(scores: torch.Tensor, planes: Sequence[torch.Tensor], block_table: torch.Tensor,
                 seq_lens: torch.Tensor, budget: int, recent: int, *, positions: Optional[torch.Tensor] = None,
                 layout: str = "HND", plan: Optional[EvictPlan] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Evict cached tokens by accumulated attention weight, in place; returns the new lengths (int32 [B]).

    Every row longer than `budget` keeps, per KV head, its `recent` newest tokens and the budget - recent others
    with the highest `scores` (the lowest slot first among equals; NaN counts as -inf).  Of the first
    A = budget - recent slots, those whose tokens go receive, in ascending order, the kept older tokens of later slots;
    the recent tokens move down to [A, budget) in order.  Scores and `positions` (int32, shaped like scores) move
    with their tokens; vacated slots' scores become 0.  Rows within the budget stay as they are.

    planes: the paged arrays to compact, [pages][H_kv][16][X] (layout "HND") or [pages][16][H_kv][X] ("NHD"), any
    dtype, any strides with a contiguous last axis: (k_pool, v_pool), or mx4_planes(pool).  No two may share memory,
    nor may scores and positions.  Pages that rows share
    must be copied first: the call moves tokens within every row's pages.  `seq_lens` is not changed."""
    L = lib()
    index = _cuda_index("scores", scores)
    B, max_pages = block_table.shape
    H_kv = scores.shape[1] if scores.dim() == 3 else 0
    if layout not in ("HND", "NHD"):
        raise ValueError(layout)
    if not 1 <= len(planes) <= EVICT_MAX_PLANES:
        raise ValueError(f"between 1 and {EVICT_MAX_PLANES} planes, got {len(planes)}")
    if not 0 <= recent <= budget or budget > INT32_MAX:
        raise ValueError(f"0 <= recent <= budget, got recent {recent}, budget {budget}")
    score_st = _check_scores("scores", scores, torch.float32, B, H_kv, max_pages, index)
    own = plan is None
    if own:
        with _on(index, stream):
            plan = plan_evict(B, H_kv, max_pages, index)
    shape = plan.shape
    if shape.B != B or shape.H_kv != H_kv or shape.max_pages_per_seq != max_pages:
        raise ValueError("the plan was made for another batch (B, H_kv or max_pages)")
    _check_plan(plan, index)
    pos_ptr, pos_st = None, (0, 0)
    if positions is not None:
        pos_st = _check_scores("positions", positions, torch.int32, B, H_kv, max_pages, index)
        pos_ptr = positions.data_ptr()
        if pos_ptr == scores.data_ptr() and pos_ptr:
            raise ValueError("scores and positions share memory")
    _check_tensor("block_table", block_table, torch.int32, index)
    _check_tensor("seq_lens", seq_lens, torch.int32, index)
    if out is None:
        out = _empty_like(seq_lens, index, stream) if seq_lens.shape == (B,) else _empty(B, torch.int32, index, stream)
    else:
        _check_tensor("out", out, torch.int32, index)
    lens_ptr, out_ptr = seq_lens.data_ptr(), out.data_ptr()
    if seq_lens.numel() < B or out.numel() < B:
        raise ValueError(f"seq_lens and out must hold {B} lengths")
    if out_ptr < lens_ptr + 4 * B and lens_ptr < out_ptr + 4 * B:
        raise ValueError("out must not share memory with seq_lens")
    pages = planes[0].shape[0]
    head_axis, token_axis = (1, 2) if layout == "HND" else (2, 1)
    arr = (Plane * len(planes))()
    rows = []  # the first rows' addresses
    for i, t in enumerate(planes):
        dims, st = t.shape, t.stride()
        if t.get_device() != index:
            raise ValueError(f"plane {i} must be on cuda:{index}, not {t.device}")
        if len(dims) != 4 or dims[0] != pages or dims[head_axis] != H_kv or dims[token_axis] != 16:
            raise ValueError(f"plane {i}'s shape {list(dims)} is not {pages} {layout} pages of {H_kv} heads "
                             "and 16 tokens")
        if dims[3] < 1 or (dims[3] > 1 and st[3] != 1):
            raise ValueError(f"plane {i}'s last axis must be contiguous")
        if st[2] < dims[3] or st[1] < st[2] * dims[2] or st[0] < st[1] * dims[1]:  # not nested in the plain order
            _check_no_overlap(f"plane {i}", dims, st)
        size = t.element_size()
        p = arr[i]
        p.base = base = t.data_ptr()
        p.stride_page, p.stride_head, p.stride_token = st[0] * size, st[head_axis] * size, st[token_axis] * size
        p.row_bytes = row_bytes = dims[3] * size
        for j, (begin, end) in enumerate(rows):
            if begin < base + row_bytes and base < end and base:
                raise ValueError(f"planes {j} and {i} share memory")
        rows.append((base, base + row_bytes))
    shape = Shape.from_buffer_copy(shape)  # the plan may serve several calls at once
    shape.num_pool_pages = pages
    _launch(L.pkv_evict_tokens, "pkv_evict_tokens", index, stream, scores.data_ptr(), score_st[0], score_st[1], pos_ptr,
            pos_st[0], pos_st[1], arr, len(planes), block_table.data_ptr(), lens_ptr, budget, recent, out_ptr,
            ctypes.byref(shape), plan.workspace.data_ptr(), plan.workspace.numel())
    if own:
        _collect(plan, index, stream)
    return out


def mx4_pool(pages: int, H_kv: int, head_dim: int, device) -> torch.Tensor:
    """An empty 4-bit pool: uint8 [pages][H_kv][17 * head_dim], one record per page and KV head (include/pkv.h
    describes it).  Zero bytes are tokens of zeros."""
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
    return torch.zeros(pages, H_kv, 17 * head_dim, dtype=torch.uint8, device=device)


def _mx4_head_dim(pool: torch.Tensor) -> int:
    if pool.dim() != 3 or pool.shape[2] not in (17 * 64, 17 * 128):
        raise ValueError(f"a 4-bit pool is [pages][H_kv][17 * head_dim], head_dim 64 or 128, got {list(pool.shape)}")
    return pool.shape[2] // 17


def mx4_planes(pool: torch.Tensor) -> tuple:
    """The four arrays of a 4-bit pool as views [pages][H_kv][16][...]: K codes, V codes, K scales, V scales (the
    planes of evict_tokens)."""
    D = _mx4_head_dim(pool)
    pages, H_kv = pool.shape[:2]
    page, head, byte = pool.stride()
    if byte != 1:
        raise ValueError("the pool's records must be contiguous")
    at, c, s = pool.storage_offset(), D // 2, D // 32
    return (pool.as_strided((pages, H_kv, 16, c), (page, head, c, 1), at),
            pool.as_strided((pages, H_kv, 16, c), (page, head, c, 1), at + 16 * c),
            pool.as_strided((pages, H_kv, 16, s), (page, head, s, 1), at + 32 * c),
            pool.as_strided((pages, H_kv, 16, s), (page, head, s, 1), at + 32 * c + 16 * s))


def mx4_shape(pool: torch.Tensor, block_table: torch.Tensor, q_heads: Optional[int] = None) -> Shape:
    """Shape of the calls over a 4-bit pool (strides in bytes); q_heads is needed for mx4_decode."""
    D = _mx4_head_dim(pool)
    pages, H_kv = int(pool.shape[0]), int(pool.shape[1])
    B, max_pages = (int(x) for x in block_table.shape)
    if pool.stride(2) != 1:
        raise ValueError("the pool's records must be contiguous")
    _check_no_overlap("pool", pool.shape, pool.stride())
    head = pool.stride(1) if H_kv > 1 else 17 * D
    page = pool.stride(0) if pages > 1 else H_kv * head
    return Shape(B, H_kv if q_heads is None else q_heads, H_kv, D, 16, max_pages, pages, 0, page, head, D // 2)


@dataclass
class Mx4Plan:
    """What the calls over a 4-bit pool need besides the tensors: the shape, the grid and a zeroed workspace.
    Every call derives its work from the device lengths, so one plan serves any of them."""

    shape: Shape
    plan: Plan
    workspace: torch.Tensor


def plan_mx4(shape: Shape, device, scores: bool = False, blocks: Optional[int] = None) -> Mx4Plan:
    """Plan for mx4_append, mx4_read and mx4_decode over mx4_shape(...); scores=True for mx4_decode with scores.
    `blocks` (default: one per SM, which fills the GPU) is the decode's grid."""
    L = lib()
    if blocks is None:
        blocks = torch.cuda.get_device_properties(device).multi_processor_count
    plan = Plan(BALANCED, blocks, 0, FLAG_SCORES if scores else 0)
    n = c_sz(0)
    _check(L.pkv_mx4_workspace_bytes(ctypes.byref(shape), ctypes.byref(plan), ctypes.byref(n)),
           "pkv_mx4_workspace_bytes")
    return Mx4Plan(shape, plan, torch.zeros(n.value, dtype=torch.uint8, device=device))


def _own_mx4_plan(pool, block_table, q_heads, scores: bool, stream) -> Mx4Plan:
    """The plan of a call that was given none; its workspace belongs to the call's stream."""
    index = _cuda_index("pool", pool)
    with _on(index, stream):
        return plan_mx4(mx4_shape(pool, block_table, q_heads), index, scores)


def _check_mx4(pool, block_table, seq_lens, shape: Shape) -> int:
    """The pool, table and lengths of a call against its plan's shape; one combined test passes every well-formed
    call, the itemised ones name what is wrong with another.  Returns the device index."""
    index = pool.get_device()
    dims, st = pool.shape, pool.stride()
    if (index >= 0 and pool.dtype is torch.uint8 and block_table.dtype is torch.int32
            and seq_lens.dtype is torch.int32 and block_table.get_device() == index and seq_lens.get_device() == index
            and len(dims) == 3 and dims[0] >= shape.num_pool_pages and dims[1] == shape.H_kv
            and dims[2] == 17 * shape.head_dim and st[2] == 1 and (st[1] == shape.kv_stride_head or dims[1] == 1)
            and (st[0] == shape.kv_stride_page or dims[0] == 1)
            and block_table.shape == (shape.B, shape.max_pages_per_seq) and block_table.is_contiguous()
            and seq_lens.numel() >= shape.B and seq_lens.is_contiguous()):
        return index
    _cuda_index("pool", pool)
    _check_tensor("pool", pool, torch.uint8, index, contiguous=False)
    if _mx4_head_dim(pool) != shape.head_dim or dims[1] != shape.H_kv or dims[0] < shape.num_pool_pages:
        raise ValueError(f"pool {list(dims)} differs from the plan's shape")
    _check_tensor("block_table", block_table, torch.int32, index)
    _check_tensor("seq_lens", seq_lens, torch.int32, index)
    if tuple(block_table.shape) != (shape.B, shape.max_pages_per_seq):
        raise ValueError(f"block_table must be [{shape.B}][{shape.max_pages_per_seq}], got {list(block_table.shape)}")
    if seq_lens.numel() < shape.B:
        raise ValueError(f"seq_lens holds {seq_lens.numel()} lengths for {shape.B} rows")
    raise ValueError("the pool's strides differ from the plan's shape")


def _check_indptr(indptr, n_tokens: int, shape: Shape, index: int):
    if indptr is None:
        if n_tokens != shape.B:
            raise ValueError(f"without indptr there is one token per row: {n_tokens} tokens for {shape.B} rows")
        return None
    _check_tensor("indptr", indptr, torch.int32, index)
    if indptr.numel() != shape.B + 1:
        raise ValueError(f"indptr must hold {shape.B + 1} offsets, got {indptr.numel()}")
    return indptr.data_ptr()


def _check_token_rows(name: str, t: torch.Tensor, n: int, shape: Shape, index: int) -> tuple:
    """bf16 [n][H_kv][D] with contiguous D; returns the token and head strides."""
    _check_tensor(name, t, torch.bfloat16, index, contiguous=False)
    dims, st = t.shape, t.stride()
    if len(dims) != 3 or dims[0] != n or dims[1] != shape.H_kv or dims[2] != shape.head_dim:
        raise ValueError(f"{name} must be [{n}][{shape.H_kv}][{shape.head_dim}], got {list(dims)}")
    if st[2] != 1:
        raise ValueError(f"{name}'s head_dim axis must be contiguous")
    return (st[0] if n > 1 else 0), (st[1] if dims[1] > 1 else 0)


def mx4_append(k: torch.Tensor, v: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, *, plan: Optional[Mx4Plan] = None, indptr: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Quantise new tokens into a 4-bit pool: k, v bf16 [n][H_kv][D] (contiguous D, other strides multiples of 8).

    Token j belongs to the row i with indptr[i] <= j < indptr[i + 1] (int32 [B + 1] on the device; without it there
    is one token per row) and goes to position seq_lens[i] + j - indptr[i]; seq_lens are the lengths before the call
    and stay unchanged.  Positions past a row's pages and bad page ids are skipped and reported: by
    workspace_status(plan), or without a plan by unplanned_status()."""
    L = lib()
    own = plan is None
    if own:
        plan = _own_mx4_plan(pool, block_table, None, False, stream)
    shape = plan.shape
    index = _check_mx4(pool, block_table, seq_lens, shape)
    _check_plan(plan, index)
    n = k.shape[0]
    k_token, k_head = _check_token_rows("k", k, n, shape, index)
    v_token, v_head = _check_token_rows("v", v, n, shape, index)
    ptr = _check_indptr(indptr, n, shape, index)
    _launch(L.pkv_mx4_append, "pkv_mx4_append", index, stream, k.data_ptr(), v.data_ptr(), k_token, k_head, v_token,
            v_head, pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), ptr, n, ctypes.byref(shape),
            plan.workspace.data_ptr())
    if own:
        _collect(plan, index, stream)


def mx4_read(pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, n_tokens: int, *,
             plan: Optional[Mx4Plan] = None, indptr: Optional[torch.Tensor] = None,
             out: Optional[tuple] = None, stream=None) -> tuple:
    """The stored values, bf16 (k, v) [n_tokens][H_kv][D], of the tokens that mx4_append with the same seq_lens and
    indptr wrote.  Exact.  `out` = (k, v) is written in place; tokens that the append skips get zeros."""
    L = lib()
    own = plan is None
    if own:
        plan = _own_mx4_plan(pool, block_table, None, False, stream)
    shape = plan.shape
    index = _check_mx4(pool, block_table, seq_lens, shape)
    _check_plan(plan, index)
    n = int(n_tokens)
    if n < 0:
        raise ValueError(f"n_tokens must be >= 0, got {n}")
    ptr = _check_indptr(indptr, n, shape, index)
    dims = (n, shape.H_kv, shape.head_dim)
    if out is None:
        k = _empty(dims, torch.bfloat16, index, stream)
        v = _empty_like(k, index, stream)
    else:
        k, v = out
        for name, t in (("k", k), ("v", v)):
            _check_tensor(f"out's {name}", t, torch.bfloat16, index)
            if t.shape != dims:
                raise ValueError(f"out's {name} must be {list(dims)}, got {list(t.shape)}")
    _launch(L.pkv_mx4_read, "pkv_mx4_read", index, stream, pool.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), ptr, n, k.data_ptr(), v.data_ptr(), ctypes.byref(shape), plan.workspace.data_ptr())
    if own:
        _collect(plan, index, stream)
    return k, v


def mx4_decode(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               page_size: int, scale: float, *, plan: Optional[Mx4Plan] = None,
               scores: Union[torch.Tensor, bool, None] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """paged_decode over a 4-bit pool; with `scores` (as in paged_decode_scored, and a plan with scores=True) the
    attention weights are added to them; None and False, as plan_mx4 takes it, both say no scores.  q bf16
    [B][H_q][D], 1 <= H_q / H_kv <= 16.  The plan serves any lengths, so a captured call can be replayed after
    seq_lens changed on the device."""
    L = lib()
    if scores is False:
        scores = None
    elif scores is not None and not isinstance(scores, torch.Tensor):
        raise TypeError(f"scores must be a tensor, None or False, got {type(scores).__name__}")
    own = plan is None
    if own:
        plan = _own_mx4_plan(pool, block_table, int(q.shape[1]), scores is not None, stream)
    shape = plan.shape
    index = _check_mx4(pool, block_table, seq_lens, shape)
    _check_plan(plan, index)
    _check_tensor("q", q, torch.bfloat16, index)
    if q.shape != (shape.B, shape.H_q, shape.head_dim):
        raise ValueError(f"q must be [{shape.B}][{shape.H_q}][{shape.head_dim}], got {list(q.shape)}")
    if (scores is not None) != bool(plan.plan.flags & FLAG_SCORES):
        raise ValueError("scores go with a plan made for them, plan_mx4(..., scores=True), and only with it")
    score_ptr, st = None, (0, 0)
    if scores is not None:
        st = _check_scores("scores", scores, torch.float32, shape.B, shape.H_kv, shape.max_pages_per_seq, index)
        score_ptr = scores.data_ptr()
    if out is None:
        out = _empty_like(q, index, stream)
    else:
        _check_tensor("out", out, torch.bfloat16, index)
        if out.shape != q.shape:
            raise ValueError(f"out must be {list(q.shape)}, got {list(out.shape)}")
    ws = plan.workspace
    _launch(L.pkv_mx4_decode, "pkv_mx4_decode", index, stream, q.data_ptr(), pool.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), page_size, scale, out.data_ptr(), score_ptr, st[0], st[1], ctypes.byref(shape),
            ctypes.byref(plan.plan), ws.data_ptr(), ws.numel())
    if own:
        _collect(plan, index, stream)
    return out


def unplanned_status(stream=None) -> int:
    """Synchronize and return the raw device error mask (0 = clean) of the calls without a plan on `stream`'s device
    (default: the current stream), of which only those queued on that stream are sure to be in; it is zero afterwards.
    Calls with a plan have theirs: workspace_status(plan)."""
    err = c_i32(0)
    index = torch.cuda.current_device() if stream is None else stream.device.index
    with _on(index, stream):
        rc = lib().pkv_unplanned_status(_raw_stream(index), ctypes.byref(err))
    if rc not in (0, -5, -6):
        _check(rc, "pkv_unplanned_status")
    return int(err.value)


def noalloc_status(stream=None) -> int:
    """Synchronize and return the raw device error mask the last
    pkv_paged_decode_noalloc call left in the library's scratch (0 = clean)."""
    L = lib()
    err = c_i32(0)
    rc = L.pkv_noalloc_status(_stream_ptr(stream), ctypes.byref(err))
    if rc not in (0, -5, -6):
        _check(rc, "pkv_noalloc_status")
    return int(err.value)


def workspace_status(plan: DecodePlan, stream=None) -> int:
    """Synchronize and return the raw device error mask of a plan's workspace (0 = clean)."""
    L = lib()
    err = c_i32(0)
    L.pkv_workspace_status(plan.workspace.data_ptr(), _stream_ptr(stream), ctypes.byref(err))
    return int(err.value)


def host_replays() -> int:
    """How many pkv_decode_host calls of this thread replayed a captured graph of their step."""
    return int(lib().pkv_decode_host_replays())


class HostDecoder:
    """Caller-owned buffers for pkv_decode_host, grown on demand: one device
    buffer (torch) and one page-locked host staging buffer.  Calls run on
    `stream` (default: the device's current stream when the decoder is made)
    unless a call passes its own.  The tensors of a call are checked (dtype,
    size, contiguity, pool strides and device) when a tensor object or shape
    is first seen; a serving loop that reuses its buffers pays only identity
    comparisons per step.  Checked tensors must not be resized in place."""

    def __init__(self, device, stream=None):
        self.device = torch.device(device)
        self.dev = torch.empty(0, dtype=torch.uint8, device=self.device)
        self.host = torch.empty(0, dtype=torch.uint8).pin_memory()
        self._stream = _stream_ptr(stream if stream is not None else torch.cuda.current_stream(self.device))
        self._fn = lib().pkv_decode_host
        self._fn_timed = lib().pkv_decode_host_timed
        self._fn_call = lib().pkv_decode_host_call
        self._plan = Plan()
        self._plan_ref = ctypes.byref(self._plan)
        self._bufs = (0, 0, 0, 0)
        self._checked = ()  # weak references to the tensors (and the shape) of the last checked call
        self._args = None   # the argument tuple of the last call with the checked tensors, its scale, no rules
        self._call = HostCall()  # the same arguments as a pkv_host_call block
        self._call_ref = ctypes.byref(self._call)

    def ensure(self, seq_lens_host, shape: Shape, rules=None):
        L = lib()
        lens, _ = _lens_array(seq_lens_host)
        arr, n = rules_array(rules)
        db, hb = c_sz(0), c_sz(0)
        _check(L.pkv_decode_host_bytes(lens, ctypes.byref(shape), arr, n, ctypes.byref(db), ctypes.byref(hb)),
               "pkv_decode_host_bytes")
        if self.dev.numel() < db.value:
            self.dev = torch.zeros(db.value, dtype=torch.uint8, device=self.device)
        if self.host.numel() < hb.value:
            self.host = torch.zeros(hb.value, dtype=torch.uint8).pin_memory()
        bufs = (self.dev.data_ptr(), self.dev.numel(), self.host.data_ptr(), self.host.numel())
        if bufs != self._bufs:  # the stored argument block names the old buffers
            self._bufs = bufs
            self._args = None

    def __call__(self, q_host: torch.Tensor, block_table_host: torch.Tensor, seq_lens_host: torch.Tensor,
                 out_host: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, scale: float, shape: Shape,
                 rules=None, stream=None, timing: Optional[HostTiming] = None) -> Plan:
        """One synchronized step; with `timing` (a HostTiming), pkv_decode_host_timed
        also fills in where the call's time went."""
        seen = self._checked
        if not (seen and seen[6] is shape and seen[0]() is q_host and seen[1]() is block_table_host
                and seen[2]() is seq_lens_host and seen[3]() is out_host and seen[4]() is k_pool
                and seen[5]() is v_pool):
            _check_host_call(q_host, block_table_host, seq_lens_host, out_host, k_pool, v_pool, shape,
                             self.dev.get_device())
            self._checked = tuple(weakref.ref(t) for t in (q_host, block_table_host, seq_lens_host, out_host,
                                                            k_pool, v_pool)) + (shape,)
            self._args = None
        elif rules is None and stream is None and self._args is not None and self._args[6] == scale:
            # the same checked tensors as the last call: its parameter block holds
            self._call.timing = None if timing is None else ctypes.addressof(timing)
            rc = self._fn_call(self._call_ref)
            if rc != 0:
                raise PkvError(rc, "pkv_decode_host")
            return Plan.from_buffer_copy(self._plan)
        arr, n = rules_array(rules) if rules is not None else (None, 0)
        dev, dev_n, host, host_n = self._bufs
        args = (q_host.data_ptr(), block_table_host.data_ptr(), seq_lens_host.data_ptr(), out_host.data_ptr(),
                k_pool.data_ptr(), v_pool.data_ptr(), float(scale), ctypes.byref(shape), arr, n, dev, dev_n,
                host, host_n, self._stream if stream is None else _stream_ptr(stream), self._plan_ref)
        if rules is None and stream is None:
            self._args = args
            c = self._call
            (c.q_host, c.block_table_host, c.seq_lens_host, c.out_host, c.k_pool, c.v_pool, c.scale) = args[:7]
            c.shape = ctypes.addressof(shape)
            c.rules, c.n_rules = None, 0
            (c.device_buffer, c.device_buffer_bytes, c.host_staging, c.host_staging_bytes, c.stream) = args[10:15]
            c.plan_out = ctypes.addressof(self._plan)
        rc = self._fn(*args) if timing is None else self._fn_timed(*args, ctypes.byref(timing))
        if rc != 0:
            raise PkvError(rc, "pkv_decode_host")
        return Plan.from_buffer_copy(self._plan)


def decode_host(*args, **kwargs):
    """One-shot pkv_decode_host with freshly allocated buffers (see HostDecoder)."""
    q_host, bt_host, lens_host, out_host, k_pool, v_pool, scale, shape = args[:8]
    dec = HostDecoder(k_pool.device)
    dec.ensure(lens_host, shape, kwargs.get("rules"))
    return dec(*args, **kwargs)
