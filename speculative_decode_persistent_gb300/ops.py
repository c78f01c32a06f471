"""Operators on the paged KV pool, outside the fused step (include/mk_ops.h):
kv_write stores new rows of one layer (rounded, or quantised), rope_write does
so behind the heads' norm and the position rotation, kv_read gathers rows back,
attend runs the attention of new rows over the cached tokens, tree_accept
verifies a tree of drafts greedily, kv_keep keeps some of a sequence's tokens in
all layers, kv_copy copies pages. Like the engine binding this is argument
marshalling only; the work runs in the CUDA library, on the current torch stream
of the tensors' device, without waiting, so calls can be captured into CUDA graphs.

    pool = KVPool(k, v)                      # one layer; Engine.kv_pool(layer) gives an engine's
    rows = KVRows(row_start, kv_len, tables) # which rows of the dense tensors are whose
    kv_write(pool, rows, new_k, new_v)       # [rows][kv heads][head dim]
    out = attend(pool, rows, q)              # [rows][query heads][head dim]

A step over trees of drafts, whose nodes are the rows:

    rope = Rope(dims, base, q_gain, k_gain)                        # once per layer
    q = rope_write(pool, rows, rope, q, k, v, parents=parents)     # in each layer
    out = attend(pool, rows, q, parents=parents)
    path, count, emitted = tree_accept(rows, parents, tokens, logits)
    kv_len = kv_keep(KVLayers(k, v), rows, path)                   # in all layers at once

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


class mk_rope(ctypes.Structure):
    _fields_ = [("turns", vp), ("q_gain", vp), ("k_gain", vp), ("rot", i32), ("eps", f32)]


class mk_rope_args(ctypes.Structure):
    _fields_ = [("q", mk_dense), ("out", mk_dense), ("k", mk_dense), ("v", mk_dense), ("hq", i32), ("dtype", i32),
                ("rope", mk_rope), ("parents", vp), ("positions", vp)]


class mk_tree_args(ctypes.Structure):
    _fields_ = [("parents", vp), ("tokens", vp), ("logits", vp), ("row_stride", i64), ("vocab", i32), ("dtype", i32),
                ("path", vp), ("count", vp), ("emitted", vp), ("work", vp), ("work_bytes", u64)]


class mk_kv_layers(ctypes.Structure):
    _fields_ = [("pool", mk_kv_pool), ("n_layers", i32), ("layer_stride", i64)]


_P = ctypes.POINTER
for _name, _res, _args in (
        ("mk_kv_write", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_dense), _P(mk_dense), i32, vp]),
        ("mk_kv_read", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_dense), _P(mk_dense), i32, vp]),
        ("mk_attend_work_bytes", sz, [_P(mk_kv_pool), _P(mk_kv_rows), i32]),
        ("mk_attend", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_attend_args), vp]),
        ("mk_attend_tree", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_attend_args), vp, vp]),
        ("mk_rope_turns", i32, [i32, ctypes.c_double, vp, vp]),
        ("mk_rope_write", i32, [_P(mk_kv_pool), _P(mk_kv_rows), _P(mk_rope_args), vp]),
        ("mk_tree_work_bytes", sz, [i32, i32]),
        ("mk_tree_accept", i32, [_P(mk_kv_rows), _P(mk_tree_args), vp]),
        ("mk_kv_copy", i32, [_P(mk_kv_layers), vp, vp, i32, vp]),
        ("mk_kv_keep", i32, [_P(mk_kv_layers), _P(mk_kv_rows), vp, vp, vp]),
        ("mk_debug_attend_wait", i32, [i32, i32])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args
EXPORTS = ["mk_kv_write", "mk_kv_read", "mk_attend_work_bytes", "mk_attend", "mk_attend_tree", "mk_rope_turns", "mk_rope_write",
           "mk_tree_work_bytes", "mk_tree_accept", "mk_kv_copy", "mk_kv_keep", "mk_debug_attend_wait"]

# The calls below pass the structs as packed bytes, which costs a few hundred
# nanoseconds less a field than ctypes structures: a small call is bound by
# this file, not by the GPU.
_fast = ctypes.CDLL(LIB_PATH)
for _name, _args in (("mk_kv_write", [vp] * 4 + [i32, vp]), ("mk_kv_read", [vp] * 4 + [i32, vp]), ("mk_attend_tree", [vp] * 5),
                     ("mk_rope_write", [vp] * 4), ("mk_tree_accept", [vp] * 3), ("mk_kv_copy", [vp] * 3 + [i32, vp]),
                     ("mk_kv_keep", [vp] * 5)):
    _fn = getattr(_fast, _name)
    _fn.restype, _fn.argtypes = i32, _args
_kv_write, _kv_read, _attend = _fast.mk_kv_write, _fast.mk_kv_read, _fast.mk_attend_tree
_rope_write, _tree_accept, _kv_copy, _kv_keep = _fast.mk_rope_write, _fast.mk_tree_accept, _fast.mk_kv_copy, _fast.mk_kv_keep
_FORMATS = (("@4P4i", mk_kv_pool), ("@3P4i", mk_kv_rows), ("@Pqq", mk_dense), ("@PqqPqqPqqiifiiPQ", mk_attend_args),
            ("@PqqPqqPqqPqqiiPPPifPP", mk_rope_args), ("@PPPqiiPPPPQ", mk_tree_args), ("@4P4iiq", mk_kv_layers))
_POOL, _ROWS, _DENSE, _ARGS, _ROPE, _TREE, _LAYERS = (struct.Struct(f).pack for f, _ in _FORMATS)
assert all(struct.calcsize(f) <= ctypes.sizeof(t) for f, t in _FORMATS)
_tree_work_bytes = _fast.mk_tree_work_bytes
_tree_work_bytes.restype, _tree_work_bytes.argtypes = sz, [i32, i32]
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


class KVLayers:
    """Layers of a paged pool that have their pages in common: the tensors of
    KVPool with the layers in front, [layers][pages][kv heads][16][head dim]
    (a slice of an engine's, say). Each layer is contiguous."""

    __slots__ = ("tensors", "device", "q8", "n_layers", "n_pages", "hkv", "dh", "c")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        shape, dtype, device, step = k.shape, k.dtype, k.device, k.stride()
        if len(shape) != 5 or v.shape != shape or shape[0] == 0 or shape[3] != PAGE_TOKENS or v.dtype != dtype:
            _refuse("KVLayers (k and v are [layers][pages][kv heads][16][head dim] of one type)")
        n, pages, heads, _, dh = shape
        inner, layer = (heads * PAGE_TOKENS * dh, PAGE_TOKENS * dh, dh, 1), step[0]
        if step[1:] != inner or v.stride() != step or n > 1 and (layer < pages * inner[0] or layer % 256):
            _refuse("KVLayers (contiguous layers, equally far apart in all tensors)")
        if v.device != device:
            _refuse("KVLayers (one device)")
        self.q8 = dtype == torch.int8
        if self.q8:
            blocks = dh // 32
            want, at = (n, pages, heads, PAGE_TOKENS, blocks), (heads * PAGE_TOKENS * blocks, PAGE_TOKENS * blocks, blocks, 1)
            for s in (k_scale, v_scale):
                if s is None or s.dtype not in _HALF or s.shape != want or s.device != device:
                    _refuse("KVLayers (an int8 pool needs binary16 scales [layers][pages][kv heads][16][head dim / 32])")
                if s.stride()[1:] != at or n > 1 and s.stride(0) * 32 != layer:
                    _refuse("KVLayers (contiguous layers, equally far apart in all tensors)")
            ks, vs, kind = k_scale.data_ptr(), v_scale.data_ptr(), MK_KV_Q8
        else:
            if dtype not in _HALF or k_scale is not None or v_scale is not None:
                _refuse("KVLayers (binary16, or int8 codes with scales)")
            ks, vs, kind = 0, 0, MK_KV_F16
        self.tensors = (k, v, k_scale, v_scale)
        self.device, self.n_layers, self.n_pages, self.hkv, self.dh = device, n, pages, heads, dh
        self.c = _LAYERS(k.data_ptr(), v.data_ptr(), ks, vs, kind, pages, heads, dh, n, layer if n > 1 else 0)


class Rope:
    """Rotation of the first `dims` dims of a head by position (a multiple of
    64; pairs i and i + dims / 2), pair i at freq[i] radians a position
    (default: base^(-2i / dims)). With q_gain, k_gain (float32 [head dim]) the
    heads of q, k are first normalised by their root mean square (with eps) and
    multiplied by it. Made once, on the gains' device or `device`."""

    __slots__ = ("tensors", "device", "dims", "gain", "c")

    def __init__(self, dims: int, base: float = 1e7, q_gain=None, k_gain=None, eps: float = 1e-6, freq=None, device=None):
        if dims < 0 or dims % 64 or dims > 65536:
            _refuse("Rope (dims: a multiple of 64)")
        if not 0.0 <= eps < 3.4e38:
            _refuse("Rope (eps)")
        gains = [g for g in (q_gain, k_gain) if g is not None]
        device = torch.device(device) if device is not None else gains[0].device if gains else torch.device("cuda")
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        for g in gains:
            if g.dtype != torch.float32 or g.dim() != 1 or not g.is_contiguous() or g.device != device or g.shape != gains[0].shape:
                _refuse("Rope (gains: contiguous float32 [head dim] on one device)")
            if g.requires_grad and torch.is_grad_enabled():
                _refuse("Rope (no gradient is defined: detach the gains or use torch.no_grad)")
            if g.data_ptr() % 16:
                _refuse("Rope (gains: 16-byte aligned)")
        turns = (u64 * max(dims // 2, 1))()
        if freq is not None:
            freq = [float(f) for f in freq]
            if len(freq) != dims // 2:
                _refuse("Rope (dims / 2 frequencies)")
            freq = (ctypes.c_double * max(len(freq), 1))(*freq)
        rc = lib.mk_rope_turns(dims, float(base), freq, turns)
        if rc != 0:
            raise MkError(rc, "mk_rope_turns")
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        table = torch.tensor(signed, dtype=torch.int64).to(device)
        self.tensors, self.device, self.dims = (table, q_gain, k_gain), device, dims
        self.gain = gains[0].shape[0] if gains else 0
        self.c = (table.data_ptr(), *(0 if g is None else g.data_ptr() for g in (q_gain, k_gain)), dims, float(eps))


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


def _index(t, n: int, device, what: str) -> int:
    """Address of a contiguous int32 tensor of n elements (0 for none)."""
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.device != device:
        _refuse(f"{what} (contiguous int32 [{n}] on the pool's device)")
    return t.data_ptr()


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


def rope_write(pool: KVPool, rows: KVRows, rope: Rope, q, k, v, parents=None, positions=None, out=None):
    """New rows into use in one pass: q [rows][query heads][head dim] and k
    [rows][kv heads][head dim] normalised (when rope has gains) and rotated by
    the rows' positions, q into out (made here unless given; it may be q
    itself; rows of no sequence are left as they are, undefined when it is
    made here), k and v into the pool as by kv_write. A row's position is
    positions[row], or that of its slot; for nodes of trees (parents, as for
    attend) the tree's first position plus the node's depth. All tensors are
    of one type; q, k, v may be slices of one projection's output. Two rows of
    one call must not share a slot of the pool. Returns out."""
    hkv, dh, shape = pool.hkv, pool.dh, q.shape
    hq = shape[1] if len(shape) == 3 else 0
    qd = _dense(q, hq, dh, "rope_write q")
    kd, vd = _dense(k, hkv, dh, "rope_write k"), _dense(v, hkv, dh, "rope_write v")
    if out is None:
        n, device = _same(pool, rows, q, k, v)
        out = torch.empty(shape, dtype=q.dtype, device=pool.device)
        od = (out.data_ptr(), hq * dh, dh)
    else:
        od = _dense(out, hq, dh, "rope_write out", True)
        n, device = _same(pool, rows, q, k, v, out)
    if rope.device != pool.device or rope.dims > dh or rope.gain not in (0, dh):
        _refuse("rope_write (a Rope on the pool's device, of no more dims than a head and gains for all of them)")
    if parents is not None and positions is not None:
        _refuse("rope_write (parents or positions)")
    args = _ROPE(*qd, *od, *kd, *vd, hq, DTYPES[q.dtype], *rope.c, _index(parents, n, pool.device, "rope_write parents"),
                 _index(positions, n, pool.device, "rope_write positions"))
    _run(device, "mk_rope_write", _rope_write, pool.c, rows._at(n), args)
    return out


_work_bytes: dict = {}  # of mk_attend_work_bytes, which goes by the head dim alone


def attend(pool: KVPool, rows: KVRows, q, scale=None, window: int = 0, sinks: int = 0, gate=None, out=None, parents=None):
    """Attention of the new rows q [rows][query heads][head dim] (float16 or
    bfloat16) over the cached tokens, the rows' own among them (kv_write
    first): causal; with window > 0 a row sees the last `window` tokens and
    the first `sinks` ones. Query heads share kv heads in equal groups, in
    order. scale defaults to 1/sqrt(head dim). With gate (like q) the output
    is multiplied by sigmoid(gate). A row that sees no token gives 0. With
    parents (int32 [rows]) the rows of a sequence are the nodes of a tree of
    drafts: parents[row] is the row's parent, an index into its sequence's rows
    before its own, or -1 where the node follows the cached tokens directly; a
    node sees the tokens before the tree, its ancestors and itself, and windows
    count positions, the tree's first slot plus a node's depth. Returns out, like q (made here unless given; it may be q or gate itself; rows of
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
    _run(device, "mk_attend", _attend, pool.c, at, args, _index(parents, n, pool.device, "attend parents"))
    return out


def tree_accept(rows: KVRows, parents, tokens, logits):
    """Greedy verification of trees of drafts (parents as for attend; None: a
    chain per sequence): tokens int32 [rows], the nodes' drafts, of which a
    sequence's first, its last emitted token, stands; logits [rows][vocabulary]
    (float32, float16 or bfloat16), the model's after each node. Returns int32
    (path [rows], count [sequences], emitted [rows]): from a sequence's first
    row on the nodes that the model's greedy choices lead through (the lowest
    child that agrees) and those choices, the accepted drafts and one token
    more; -1 behind them; their number. Of equal logits the lowest index
    counts; a node with a NaN among its logits has the choice -1, and none of its children
    is accepted. Rows of no sequence are undefined."""
    if logits.dim() != 2 or logits.dtype not in DTYPES or logits.shape[1] == 0 or logits.stride(1) != 1:
        _refuse("tree_accept (logits [rows][vocabulary], float32, float16 or bfloat16, a row contiguous)")
    n, vocab = logits.shape
    device = rows.device
    if rows.n_rows is not None and rows.n_rows != n:
        _refuse("rows of the logits differ from KVRows.n_rows")
    if device.type != "cuda" or logits.device != device:
        _refuse("tree_accept (rows and logits on one CUDA device)")
    if tokens is None:
        _refuse("tree_accept (tokens)")
    par, tok = _index(parents, n, device, "tree_accept parents"), _index(tokens, n, device, "tree_accept tokens")
    path, emitted = torch.empty(n, dtype=torch.int32, device=device), torch.empty(n, dtype=torch.int32, device=device)
    count = torch.empty(rows.n_seqs, dtype=torch.int32, device=device)
    nbytes = _tree_work_bytes(n, vocab)
    work = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    args = _TREE(par, tok, logits.data_ptr(), logits.stride(0), vocab, DTYPES[logits.dtype], path.data_ptr(), count.data_ptr(),
                 emitted.data_ptr(), work.data_ptr(), nbytes)
    _run(device.index, "mk_tree_accept", _tree_accept, rows._at(n), args)
    return path, count, emitted


def kv_copy(layers: KVLayers, src, dst) -> None:
    """Copy page src[i] to page dst[i] in all layers (int32 tensors of one
    length). Pairs with an id that is no page are passed over. A page may be
    copied several times; one that is written must not be another pair's
    source or target."""
    if src.dim() != 1:
        _refuse("kv_copy (int32 [n])")
    n = src.shape[0]
    if layers.device.type != "cuda":
        _refuse("kv_copy (a CUDA device)")
    _run(layers.device.index, "mk_kv_copy", _kv_copy, layers.c, _index(src, n, layers.device, "kv_copy src"),
         _index(dst, n, layers.device, "kv_copy dst"), n)


def kv_keep(layers: KVLayers, rows: KVRows, keep):
    """Keep some of each sequence's new rows, in all layers: keep int32 [rows]
    lists, from a sequence's first row on, indices into its rows, ascending;
    the first entry that does not ascend (-1, say) ends the list, so that
    tree_accept's path can be given as it is. Row keep[i] moves, in place, to the
    i-th slot behind the tokens before the rows. Returns the new lengths, int32
    [sequences]; the caller frees the pages wholly behind them. Sequences of one
    call must not share pages that a row moves to."""
    device = layers.device
    if device.type != "cuda" or rows.device != device:
        _refuse("kv_keep (layers and rows on one CUDA device)")
    if keep.dim() != 1 or rows.n_rows is not None and rows.n_rows != keep.shape[0]:
        _refuse("kv_keep (an entry per row)")
    n = keep.shape[0]
    at = _index(keep, n, device, "kv_keep keep")
    kv_len = torch.empty(rows.n_seqs, dtype=torch.int32, device=device)
    _run(device.index, "mk_kv_keep", _kv_keep, layers.c, rows._at(n), at, kv_len.data_ptr())
    return kv_len
