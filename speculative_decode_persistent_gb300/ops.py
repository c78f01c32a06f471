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
import struct

import torch

from .mk import LIB_PATH, MK_KV_F16, MK_KV_Q8, MkError, i32, lib, sz, vp

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
        ("mk_attend", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_attend_args), vp]),
        ("mk_debug_attend_wait", i32, [i32, i32])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args
EXPORTS = ["mk_kv_write", "mk_kv_read", "mk_attend_work_bytes", "mk_attend", "mk_debug_attend_wait"]

# The calls below pass the structs as packed bytes, which costs a few hundred
# nanoseconds less a field than ctypes structures: a small call is bound by
# this file, not by the GPU.
_fast = ctypes.CDLL(LIB_PATH)
for _name, _n in (("mk_kv_write", 4), ("mk_kv_read", 4), ("mk_attend", 3)):
    _fn = getattr(_fast, _name)
    _fn.restype, _fn.argtypes = i32, [vp] * _n + ([i32] if _n == 4 else []) + [vp]
_kv_write, _kv_read, _attend = _fast.mk_kv_write, _fast.mk_kv_read, _fast.mk_attend
_POOL, _ROWS, _DENSE, _ARGS = (struct.Struct(f).pack for f in ("@4P4i", "@3P4i", "@Pqq", "@PqqPqqPqqiifiiPQ"))
assert all(struct.calcsize(f) <= ctypes.sizeof(t) for f, t in (
    ("@4P4i", mk_kv_pool), ("@3P4i", mk_kv_rows), ("@Pqq", mk_dense), ("@PqqPqqPqqiifiiPQ", mk_attend_args)))
_raw_stream = torch._C._cuda_getCurrentRawStream
_HALF = (torch.float16, torch.int16)


def _refuse(what: str):
    raise MkError(_INVALID, what)


class KVPool:
    """One attention layer of a paged pool.

    k, v: [pages][kv heads][16][head dim], contiguous; binary16 (torch.float16,
    or int16 views of its bits), or int8 codes with k_scale, v_scale
    [pages][kv heads][16][head dim / 32] (binary16 likewise)."""

    __slots__ = ("tensors", "device", "q8", "n_pages", "hkv", "dh", "c")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        shape, dtype, device = k.shape, k.dtype, k.device
        if len(shape) != 4 or v.shape != shape or shape[2] != PAGE_TOKENS or v.dtype != dtype:
            _refuse("KVPool (k and v are [pages][kv heads][16][head dim] of one type)")
        self.q8 = dtype == torch.int8
        self.n_pages, self.hkv, _, self.dh = shape
        if not (k.is_contiguous() and v.is_contiguous()):
            _refuse("KVPool (contiguous tensors)")
        if v.device != device:
            _refuse("KVPool (one device)")
        self.device = device
        if self.q8:
            want = (self.n_pages, self.hkv, PAGE_TOKENS, self.dh // 32)
            for s in (k_scale, v_scale):
                if s is None or s.dtype not in _HALF or s.shape != want or not s.is_contiguous() or s.device != device:
                    _refuse("KVPool (an int8 pool needs binary16 scales [pages][kv heads][16][head dim / 32])")
            self.tensors = (k, v, k_scale, v_scale)
            self.c = _POOL(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), MK_KV_Q8, self.n_pages,
                           self.hkv, self.dh)
        else:
            if dtype not in _HALF or k_scale is not None or v_scale is not None:
                _refuse("KVPool (binary16, or int8 codes with scales)")
            self.tensors = (k, v)
            self.c = _POOL(k.data_ptr(), v.data_ptr(), 0, 0, MK_KV_F16, self.n_pages, self.hkv, self.dh)


class KVRows:
    """Which rows of the dense tensors are whose: int32 tensors on the pool's
    device. Rows row_start[s] .. row_start[s+1]-1 are the last of sequence s's
    kv_len[s] tokens, whose positions 16i .. 16i+15 lie on page tables[s][i]
    (-1: no page). They are read when the work runs. n_rows: rows of the
    dense tensors (default: the tensor's of the call, needed for a kv_read
    that makes its outputs). max_q: the most new rows of one sequence (default:
    their mean), a hint for the choice of a kernel."""

    __slots__ = ("tensors", "device", "n_seqs", "n_rows", "max_q", "_head", "_stride")

    def __init__(self, row_start, kv_len, tables, n_rows=None, max_q=None):
        i = torch.int32
        if row_start.dtype != i or kv_len.dtype != i or tables.dtype != i:
            _refuse("KVRows (contiguous int32 tensors)")
        if not (row_start.is_contiguous() and kv_len.is_contiguous() and tables.is_contiguous()):
            _refuse("KVRows (contiguous int32 tensors)")
        shape, n = tables.shape, kv_len.shape
        if len(shape) != 2 or len(n) != 1 or row_start.shape != (n[0] + 1,) or shape[0] != n[0]:
            _refuse("KVRows (row_start [n + 1], kv_len [n], tables [n][pages])")
        device = kv_len.device
        if row_start.device != device or tables.device != device:
            _refuse("KVRows (one device)")
        if n_rows is not None and n_rows < 0 or max_q is not None and max_q < 0:
            _refuse("KVRows (counts of rows)")
        self.tensors, self.device = (row_start, kv_len, tables), device
        self.n_seqs, self.n_rows, self.max_q = n[0], n_rows, max_q
        self._head, self._stride = (row_start.data_ptr(), kv_len.data_ptr(), tables.data_ptr(), n[0]), shape[1]

    def _at(self, n_rows: int):
        """The C view for dense tensors of n_rows rows."""
        mean = -(-n_rows // max(self.n_seqs, 1))
        return _ROWS(*self._head, n_rows, self._stride, mean if self.max_q is None else min(self.max_q, n_rows))


def _overlap(n: int, heads: int, dh: int, row: int, head: int) -> bool:
    """Whether two of the n x heads vectors of dh elements at r row + h head share an element."""
    if n == 0 or head >= dh and (n == 1 or row >= (heads - 1) * head + dh):  # rows of heads
        return False
    if row >= dh and (heads == 1 or head >= (n - 1) * row + dh):  # heads of rows
        return False
    if n > 1 and row < dh or heads > 1 and head < dh:
        return True
    # the multiples of row on both sides of each multiple of head
    return any(a < n and abs(a * row - b * head) < dh
               for b in range(1, heads) for a in (b * head // row, b * head // row + 1))


def _dense(t, heads: int, dh: int, what: str, out=False):
    """(address, row stride, head stride) of a dense tensor, checked."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dh:
        _refuse(f"{what} ([rows][{heads}][{dh}])")
    row, head, one = t.stride()
    if one != 1:
        _refuse(f"{what} (contiguous head dim)")
    if out and _overlap(shape[0], heads, dh, row, head):
        _refuse(f"{what} (rows of an output must not overlap)")
    if t.requires_grad and torch.is_grad_enabled():
        _refuse(f"{what} (no gradient is defined: detach it or use torch.no_grad)")
    return t.data_ptr(), row, head


def _same(pool: KVPool, rows: KVRows, t, *more):
    """Rows and device index of dense tensors that belong together."""
    n, dtype, device = t.shape[0], t.dtype, pool.device
    if rows.n_rows is not None and rows.n_rows != n:
        _refuse("rows of the dense tensors differ from KVRows.n_rows")
    for x in more:
        if x.shape[0] != n or x.dtype != dtype:
            _refuse("dense tensors of one type with one number of rows")
    if dtype not in DTYPES:
        _refuse("dense tensors are float32, float16 or bfloat16")
    if device.type != "cuda" or rows.device != device or t.device != device:
        _refuse("pool, rows and dense tensors on one CUDA device")
    for x in more:
        if x.device != device:
            _refuse("pool, rows and dense tensors on one CUDA device")
    return n, device.index


def _run(device: int, what: str, fn, *args):
    """fn(*args, stream) with the device current, on its current stream."""
    was = torch._C._cuda_getDevice()
    if was == device:
        rc = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device))
    if rc != 0:
        raise MkError(rc, what)


def kv_write(pool: KVPool, rows: KVRows, k, v) -> None:
    """Store the new rows k, v [rows][kv heads][head dim] at their positions,
    rounded to binary16 or quantised as the fused step does. Two rows of one
    call must not share a slot of the pool."""
    kd, vd = _dense(k, pool.hkv, pool.dh, "kv_write k"), _dense(v, pool.hkv, pool.dh, "kv_write v")
    n, device = _same(pool, rows, k, v)
    _run(device, "mk_kv_write", _kv_write, pool.c, rows._at(n), _DENSE(*kd), _DENSE(*vd), DTYPES[k.dtype])


def kv_read(pool: KVPool, rows: KVRows, dtype=torch.float16, out=None):
    """The rows' cached values as dense (k, v) of type dtype, or into out =
    (k, v). Rows of no sequence are left as they are (undefined when the
    tensors are made here)."""
    hkv, dh = pool.hkv, pool.dh
    if out is None:
        if rows.n_rows is None:
            _refuse("kv_read (KVRows.n_rows or out)")
        shape = (rows.n_rows, hkv, dh)
        k, v = torch.empty(shape, dtype=dtype, device=pool.device), torch.empty(shape, dtype=dtype, device=pool.device)
        kd, vd = (k.data_ptr(), hkv * dh, dh), (v.data_ptr(), hkv * dh, dh)
        n, device = _same(pool, rows, k)
    else:
        k, v = out
        kd, vd = _dense(k, hkv, dh, "kv_read out", True), _dense(v, hkv, dh, "kv_read out", True)
        n, device = _same(pool, rows, k, v)
    _run(device, "mk_kv_read", _kv_read, pool.c, rows._at(n), _DENSE(*kd), _DENSE(*vd), DTYPES[k.dtype])
    return k, v


_work_bytes: dict = {}  # of mk_attend_work_bytes, which goes by the head dim alone


def attend(pool: KVPool, rows: KVRows, q, scale=None, window: int = 0, sinks: int = 0, gate=None, out=None):
    """Attention of the new rows q [rows][query heads][head dim] (float16 or
    bfloat16) over the cached tokens, the rows' own among them (kv_write
    first): causal; with window > 0 a row sees the last `window` tokens and
    the first `sinks` ones. Query heads share kv heads in equal groups, in
    order. scale defaults to 1/sqrt(head dim). With gate (like q) the output
    is multiplied by sigmoid(gate). A row that sees no token gives 0. Returns
    out, like q (made here unless given; it may be q or gate itself; rows of
    no sequence are left as they are, undefined when it is made here)."""
    shape, dtype, dh = q.shape, q.dtype, pool.dh
    hq = shape[1] if len(shape) == 3 else 0
    qd = _dense(q, hq, dh, "attend q")
    gd = (0, 0, 0) if gate is None else _dense(gate, hq, dh, "attend gate")
    more = () if gate is None else (gate,)
    if out is None:
        n, device = _same(pool, rows, q, *more)
        out = torch.empty(shape, dtype=dtype, device=pool.device)
        od = (out.data_ptr(), hq * dh, dh)
    else:
        od = _dense(out, hq, dh, "attend out", True)
        n, device = _same(pool, rows, q, out, *more)
    scale = 1.0 / math.sqrt(dh) if scale is None else float(scale)
    if not (0.0 < scale < 3.4e38 and 0 <= window < 2 ** 31 and 0 <= sinks < 2 ** 31):
        _refuse("attend (a finite positive scale, a window and sinks of at least 0)")
    at = rows._at(n)
    nbytes = _work_bytes.get(dh)
    if nbytes is None:
        nbytes = lib.mk_attend_work_bytes(mk_kv_pool.from_buffer_copy(pool.c),
                                          mk_kv_rows.from_buffer_copy(at), hq)
        if nbytes:
            _work_bytes[dh] = nbytes
    # from torch's allocator, so calls on other streams and captured graphs have their own
    work = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=pool.device)
    args = _ARGS(*qd, *gd, *od, hq, DTYPES[dtype], scale, window, sinks, work.data_ptr(),
                 work.numel())
    _run(device, "mk_attend", _attend, pool.c, at, args)
    return out
