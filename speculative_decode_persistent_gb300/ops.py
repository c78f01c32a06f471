"""Operators on one attention layer of the paged KV pool, outside the fused
step (include/mk_ops.h): kv_write stores new rows (rounded, or quantised),
kv_read gathers rows back, attend runs the attention of a chunk of new rows
over the cached tokens. Like the engine binding this is argument marshalling
only; the work runs in the CUDA library, on the current torch stream of the
tensors' device, without waiting, so calls can be captured into CUDA graphs.

    pool = KVPool(k, v)                      # one layer; Engine.kv_pool(layer) gives an engine's
    rows = KVRows(row_start, kv_len, tables) # which rows of the dense tensors are whose
    kv_write(pool, rows, new_k, new_v)       # [rows][kv heads][head dim]
    out = attend(pool, rows, q)              # [rows][query heads][head dim]

The new rows of a sequence are the LAST of its kv_len tokens: kv_len counts
them. Errors are MkError, as everywhere in the package.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .mk import MK_KV_F16, MK_KV_Q8, MkError, i32, lib, sz, vp

PAGE_TOKENS = 16
MK_OPS_MAX_SEQS = 1024
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_INVALID = -1

i64, u64, f32 = ctypes.c_int64, ctypes.c_uint64, ctypes.c_float


class mk_kv_pool(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("k_scale", vp), ("v_scale", vp),
                ("kv_dtype", i32), ("n_pages", i32), ("hkv", i32), ("dh", i32)]


class mk_kv_rows(ctypes.Structure):
    _fields_ = [("row_start", vp), ("kv_len", vp), ("tables", vp),
                ("n_seqs", i32), ("n_rows", i32), ("table_stride", i32), ("max_q", i32)]


class mk_dense(ctypes.Structure):
    _fields_ = [("data", vp), ("row_stride", i64), ("head_stride", i64)]


class mk_attend_args(ctypes.Structure):
    _fields_ = [("q", mk_dense), ("gate", mk_dense), ("out", mk_dense), ("hq", i32), ("dtype", i32), ("scale", f32),
                ("window", i32), ("sinks", i32), ("work", vp), ("work_bytes", u64)]


_P = ctypes.POINTER
for _name, _res, _args in (
        ("mk_kv_write", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_dense), _P(mk_dense), i32, vp]),
        ("mk_kv_read", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_dense), _P(mk_dense), i32, vp]),
        ("mk_attend_work_bytes", sz, [_P(mk_kv_pool), _P(mk_kv_rows), i32]),
        ("mk_attend", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_attend_args), vp])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args
EXPORTS = ["mk_kv_write", "mk_kv_read", "mk_attend_work_bytes", "mk_attend"]


def _refuse(what: str):
    raise MkError(_INVALID, what)


def _check(rc: int, what: str):
    if rc != 0:
        raise MkError(rc, what)


class KVPool:
    """One attention layer of a paged pool.

    k, v: [pages][kv heads][16][head dim], contiguous; binary16 (torch.float16,
    or int16 views of its bits), or int8 codes with k_scale, v_scale
    [pages][kv heads][16][head dim / 32] (binary16 likewise)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.shape[2] != PAGE_TOKENS or k.dtype != v.dtype:
            _refuse("KVPool (k and v are [pages][kv heads][16][head dim] of one type)")
        half = (torch.float16, torch.int16)
        self.q8 = k.dtype == torch.int8
        every = [k, v]
        if self.q8:
            want = k.shape[:3] + (k.shape[3] // 32,)
            for s in (k_scale, v_scale):
                if s is None or s.dtype not in half or tuple(s.shape) != tuple(want):
                    _refuse("KVPool (an int8 pool needs binary16 scales [pages][kv heads][16][head dim / 32])")
                every.append(s)
        elif k.dtype not in half or k_scale is not None or v_scale is not None:
            _refuse("KVPool (binary16, or int8 codes with scales)")
        if not all(t.is_contiguous() for t in every):
            _refuse("KVPool (contiguous tensors)")
        if any(t.device != k.device for t in every):
            _refuse("KVPool (one device)")
        self.tensors, self.device = every, k.device
        self.n_pages, self.hkv, _, self.dh = k.shape
        self.c = mk_kv_pool(k.data_ptr(), v.data_ptr(), every[2].data_ptr() if self.q8 else None,
                            every[3].data_ptr() if self.q8 else None, MK_KV_Q8 if self.q8 else MK_KV_F16,
                            self.n_pages, self.hkv, self.dh)
        self.ref = ctypes.byref(self.c)


class KVRows:
    """Which rows of the dense tensors are whose: int32 tensors on the pool's
    device. Rows row_start[s] .. row_start[s+1]-1 are the last of sequence s's
    kv_len[s] tokens, whose positions 16i .. 16i+15 lie on page tables[s][i]
    (-1: no page). They are read when the work runs. n_rows: rows of the
    dense tensors (default: the tensor's of the call, needed for a kv_read
    that makes its outputs). max_q: the most new rows of one sequence (default
    n_rows), a hint for the choice of a kernel."""

    def __init__(self, row_start, kv_len, tables, n_rows=None, max_q=None):
        for t in (row_start, kv_len, tables):
            if t.dtype != torch.int32 or not t.is_contiguous():
                _refuse("KVRows (contiguous int32 tensors)")
        if tables.dim() != 2 or kv_len.dim() != 1 or row_start.dim() != 1:
            _refuse("KVRows (row_start [n + 1], kv_len [n], tables [n][pages])")
        n = kv_len.shape[0]
        if row_start.shape[0] != n + 1 or tables.shape[0] != n:
            _refuse("KVRows (row_start [n + 1], kv_len [n], tables [n][pages])")
        if row_start.device != kv_len.device or tables.device != kv_len.device:
            _refuse("KVRows (one device)")
        if n_rows is not None and n_rows < 0 or max_q is not None and max_q < 0:
            _refuse("KVRows (counts of rows)")
        self.tensors, self.device = (row_start, kv_len, tables), kv_len.device
        self.n_seqs, self.n_rows, self.max_q = n, n_rows, max_q
        self.c = mk_kv_rows(row_start.data_ptr(), kv_len.data_ptr(), tables.data_ptr(), n, 0, tables.shape[1], 0)
        self.ref = ctypes.byref(self.c)

    def _at(self, n_rows: int):
        """The C view for dense tensors of n_rows rows."""
        self.c.n_rows = n_rows
        self.c.max_q = n_rows if self.max_q is None else min(self.max_q, n_rows)
        return self.ref


def _dense(t, heads: int, dh: int, what: str, out=False):
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dh:
        _refuse(f"{what} ([rows][{heads}][{dh}])")
    if dh > 1 and t.stride(2) != 1:
        _refuse(f"{what} (contiguous head dim)")
    if out and t.shape[0] and not (t.stride(1) >= dh and (t.shape[0] == 1 or t.stride(0) >= (heads - 1) * t.stride(1) + dh)):
        _refuse(f"{what} (rows of an output must not overlap)")
    if t.requires_grad and torch.is_grad_enabled():
        _refuse(f"{what} (no gradient is defined: detach it or use torch.no_grad)")
    return mk_dense(t.data_ptr(), t.stride(0), t.stride(1))


def _same(pool: KVPool, rows: KVRows, *tensors):
    n = tensors[0].shape[0]
    if rows.n_rows is not None and rows.n_rows != n:
        _refuse("rows of the dense tensors differ from KVRows.n_rows")
    if any(t.shape[0] != n or t.dtype != tensors[0].dtype for t in tensors):
        _refuse("dense tensors of one type with one number of rows")
    if tensors[0].dtype not in DTYPES:
        _refuse("dense tensors are float32, float16 or bfloat16")
    if pool.device.type != "cuda" or rows.device != pool.device or any(t.device != pool.device for t in tensors):
        _refuse("pool, rows and dense tensors on one CUDA device")
    return n


class _On:
    """The tensors' device made current for a call."""

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.was = torch.cuda.current_device()
        if self.was != self.device.index:
            torch.cuda.set_device(self.device)
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.was != self.device.index:
            torch.cuda.set_device(self.was)


def kv_write(pool: KVPool, rows: KVRows, k, v) -> None:
    """Store the new rows k, v [rows][kv heads][head dim] at their positions,
    rounded to binary16 or quantised as the fused step does. Two rows of one
    call must not share a slot of the pool."""
    kd, vd = _dense(k, pool.hkv, pool.dh, "kv_write k"), _dense(v, pool.hkv, pool.dh, "kv_write v")
    n = _same(pool, rows, k, v)
    with _On(pool.device) as stream:
        _check(lib.mk_kv_write(pool.ref, rows._at(n), kd, vd, DTYPES[k.dtype], stream), "mk_kv_write")


def kv_read(pool: KVPool, rows: KVRows, dtype=torch.float16, out=None):
    """The rows' cached values as dense (k, v) of type dtype, or into out =
    (k, v). Rows of no sequence are left as they are (undefined when the
    tensors are made here)."""
    if out is None:
        if rows.n_rows is None:
            _refuse("kv_read (KVRows.n_rows or out)")
        out = tuple(torch.empty((rows.n_rows, pool.hkv, pool.dh), dtype=dtype, device=pool.device) for _ in "kv")
    k, v = out
    kd, vd = (_dense(t, pool.hkv, pool.dh, "kv_read out", out=True) for t in (k, v))
    n = _same(pool, rows, k, v)
    with _On(pool.device) as stream:
        _check(lib.mk_kv_read(pool.ref, rows._at(n), kd, vd, DTYPES[k.dtype], stream), "mk_kv_read")
    return k, v


def attend(pool: KVPool, rows: KVRows, q, scale=None, window: int = 0, sinks: int = 0, gate=None, out=None):
    """Attention of the new rows q [rows][query heads][head dim] (float16 or
    bfloat16) over the cached tokens, the rows' own among them (kv_write
    first): causal; with window > 0 a row sees the last `window` tokens and
    the first `sinks` ones. Query heads share kv heads in equal groups, in
    order. scale defaults to 1/sqrt(head dim). With gate (like q) the output
    is multiplied by sigmoid(gate). A row that sees no token gives 0. Returns
    out, like q (made here unless given; it may be q or gate itself; rows of
    no sequence are left as they are, undefined when it is made here)."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    hq = q.shape[1] if q.dim() == 3 else 0
    a = mk_attend_args()
    a.q = _dense(q, hq, pool.dh, "attend q")
    a.out = _dense(out, hq, pool.dh, "attend out", out=True)
    if gate is None:
        n = _same(pool, rows, q, out)
    else:
        a.gate = _dense(gate, hq, pool.dh, "attend gate")
        n = _same(pool, rows, q, out, gate)
    a.hq, a.dtype = hq, DTYPES[q.dtype]
    a.scale = 1.0 / math.sqrt(pool.dh) if scale is None else scale
    a.window, a.sinks = window, sinks
    with _On(pool.device) as stream:
        ref = rows._at(n)
        nbytes = lib.mk_attend_work_bytes(pool.ref, ref, hq)
        # from torch's allocator, so calls on other streams and captured graphs have their own
        work = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=pool.device)
        a.work, a.work_bytes = work.data_ptr(), work.numel()
        _check(lib.mk_attend(pool.ref, ref, ctypes.byref(a), stream), "mk_attend")
    return out
