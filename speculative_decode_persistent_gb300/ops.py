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

import torch

try:
    from . import _bind
except ImportError as e:
    raise ImportError("_bind.so is missing, or was built for another torch or Python: run __graft_entry__.build() first") from e
from .mk import MkError, i32, lib, sz, vp

MK_OPS_MAX_SEQS = 1024
PAGE_TOKENS = 16
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # MK_F32, MK_F16, MK_BF16
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
        ("mk_tree_work_bytes", sz, [_P(mk_kv_rows), i32]),
        ("mk_tree_accept", i32, [_P(mk_kv_rows), _P(mk_tree_args), vp]),
        ("mk_kv_copy", i32, [_P(mk_kv_layers), vp, vp, i32, vp]),
        ("mk_kv_keep", i32, [_P(mk_kv_layers), _P(mk_kv_rows), vp, vp, vp]),
        ("mk_debug_attend_wait", i32, [i32, i32])):
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args
EXPORTS = ["mk_kv_write", "mk_kv_read", "mk_attend_work_bytes", "mk_attend", "mk_attend_tree", "mk_rope_turns", "mk_rope_write",
           "mk_tree_work_bytes", "mk_tree_accept", "mk_kv_copy", "mk_kv_keep", "mk_debug_attend_wait"]

# The calls below are marshalled by a compiled module (csrc/ops/bind.cpp), which
# takes the library's entries from here: a small call is bound by the host.
_bind.connect(MkError, {n: ctypes.cast(getattr(lib, n), vp).value for n in EXPORTS})


def _refuse(what: str):
    raise MkError(_INVALID, what)


class KVPool:
    """One attention layer of a paged pool.

    k, v: [pages][kv heads][16][head dim], contiguous; binary16 (torch.float16,
    or int16 views of its bits), or int8 codes with k_scale, v_scale
    [pages][kv heads][16][head dim / 32] (binary16 likewise)."""

    __slots__ = ("tensors", "h")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.h = _bind.pool(k, v, k_scale, v_scale)
        self.tensors = (k, v) if k_scale is None else (k, v, k_scale, v_scale)

    device = property(lambda self: self.tensors[0].device)
    q8 = property(lambda self: self.tensors[0].dtype == torch.int8)
    n_pages = property(lambda self: self.tensors[0].shape[-4])
    hkv = property(lambda self: self.tensors[0].shape[-3])
    dh = property(lambda self: self.tensors[0].shape[-1])


class KVLayers:
    """Layers of a paged pool that have their pages in common: the tensors of
    KVPool with the layers in front, [layers][pages][kv heads][16][head dim]
    (a slice of an engine's, say). Each layer is contiguous."""

    __slots__ = ("tensors", "h")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.h = _bind.layers(k, v, k_scale, v_scale)
        self.tensors = (k, v) if k_scale is None else (k, v, k_scale, v_scale)

    device, q8, n_pages, hkv, dh = KVPool.device, KVPool.q8, KVPool.n_pages, KVPool.hkv, KVPool.dh
    n_layers = property(lambda self: self.tensors[0].shape[0])


class Rope:
    """Rotation of the first `dims` dims of a head by position (a multiple of
    64; pairs i and i + dims / 2), pair i at freq[i] radians a position
    (default: base^(-2i / dims)). With q_gain, k_gain (float32 [head dim]) the
    heads of q, k are first normalised by their root mean square (with eps) and
    multiplied by it. Made once, on the gains' device or `device`."""

    __slots__ = ("tensors", "h")

    def __init__(self, dims: int, base: float = 1e7, q_gain=None, k_gain=None, eps: float = 1e-6, freq=None, device=None):
        if dims < 0 or dims % 64 or dims > 65536:
            _refuse("Rope (dims: a multiple of 64)")
        if not 0.0 <= eps < 3.4e38:
            _refuse("Rope (eps)")
        gains = [g for g in (q_gain, k_gain) if g is not None]
        if device is None:
            device = gains[0].device if gains else "cuda"
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
        self.h = _bind.rope(table, q_gain, k_gain, dims, eps)
        self.tensors = (table, q_gain, k_gain)


class KVRows:
    """Which rows of the dense tensors are whose: int32 tensors on the pool's
    device. Rows row_start[s] .. row_start[s+1]-1 are the last of sequence s's
    kv_len[s] tokens, whose positions 16i .. 16i+15 lie on page tables[s][i]
    (-1: no page). They are read when the work runs. n_rows: rows of the
    dense tensors (default: the tensor's of the call, needed for a kv_read
    that makes its outputs). max_q: the most new rows of one sequence (default:
    their mean), a hint for the choice of a kernel."""

    __slots__ = ("tensors", "n_rows", "max_q", "h")

    def __init__(self, row_start, kv_len, tables, n_rows=None, max_q=None):
        self.h = _bind.rows(row_start, kv_len, tables, n_rows, max_q)
        self.tensors, self.n_rows, self.max_q = (row_start, kv_len, tables), n_rows, max_q

    device = property(lambda self: self.tensors[0].device)
    n_seqs = property(lambda self: self.tensors[1].shape[0])


def kv_write(pool: KVPool, rows: KVRows, k, v) -> None:
    """Store the new rows k, v [rows][kv heads][head dim] at their positions,
    rounded to binary16 or quantised as the fused step does. Two rows of one
    call must not share a slot of the pool."""
    _bind.kv_write(pool.h, rows.h, k, v)


def kv_read(pool: KVPool, rows: KVRows, dtype=torch.float16, out=None):
    """The rows' cached values as dense (k, v) of type dtype, or into out =
    (k, v). Rows of no sequence are left as they are (undefined when the
    tensors are made here)."""
    k, v = (None, None) if out is None else out
    return _bind.kv_read(pool.h, rows.h, dtype, k, v)


def rope_write(pool: KVPool, rows: KVRows, rope: Rope, q, k, v, parents=None, positions=None, out=None):
    """New rows into use in one pass: q [rows][query heads][head dim] and k
    [rows][kv heads][head dim] normalised (when rope has gains) and rotated by
    the rows' positions, q into out (made here unless given; it may be q
    itself, and overlaps no input otherwise; rows of no sequence are left as they
    are, undefined when it is made here), k and v into the pool as by kv_write. A row's position is
    positions[row], or that of its slot; for nodes of trees (parents, as for
    attend) the tree's first position plus the node's depth. All tensors are
    of one type; q, k, v may be slices of one projection's output. Two rows of
    one call must not share a slot of the pool. Returns out."""
    return _bind.rope_write(pool.h, rows.h, rope.h, q, k, v, parents, positions, out)


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
    count positions, the tree's first slot plus a node's depth (for drafts: the
    time of the tree's own tokens grows with its nodes times their depth).
    Returns out, like q (made here unless given; it may be q or gate itself; rows of
    no sequence are left as they are, undefined when it is made here)."""
    return _bind.attend(pool.h, rows.h, q, scale, window, sinks, gate, out, parents)


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
    return _bind.tree_accept(rows.h, parents, tokens, logits)


def kv_copy(layers: KVLayers, src, dst) -> None:
    """Copy page src[i] to page dst[i] in all layers (int32 tensors of one
    length). Pairs with an id that is no page are passed over. A page may be
    copied several times; one that is written must not be another pair's
    source or target."""
    _bind.kv_copy(layers.h, src, dst)


def kv_keep(layers: KVLayers, rows: KVRows, keep):
    """Keep some of each sequence's new rows, in all layers: keep int32 [rows]
    lists, from a sequence's first row on, indices into its rows, ascending;
    the first entry that does not ascend (-1, say) ends the list, so that
    tree_accept's path can be given as it is. Row keep[i] moves, in place, to the
    i-th slot behind the tokens before the rows. Returns the new lengths, int32
    [sequences]; the caller frees the pages wholly behind them. Sequences of one
    call must not share pages that a row moves to."""
    return _bind.kv_keep(layers.h, rows.h, keep)
