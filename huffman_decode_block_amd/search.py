"""Binding of the operators for decoding with more than one candidate
(include/df11_search.h): attention of a tree or chain of new tokens over a paged
cache, pages copied, forked and compacted, a beam search's selection.

Argument marshalling only, with the checks, streams and workspaces of the step
module: each call allocates what it returns and its workspace with torch and
launches HIP kernels of the library on `stream`.  No call has a derivative; a
tensor that asks for one is refused.
"""
from __future__ import annotations

import ctypes
import functools

from . import step
from .step import _check, _dense, _last_dense, _no_gradient, _out, _place, _tensor, _workspace, df11_paged_cache

_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_i32 = ctypes.c_int32
_vp = ctypes.c_void_p

DF11_LOGITS_BF16 = 0
DF11_LOGITS_FP32 = 1


class df11_tree(ctypes.Structure):
    _fields_ = [
        ("q", _vp), ("q_batch_stride", _u64), ("q_node_stride", _u64), ("q_head_stride", _u64),
        ("mask", _vp), ("mask_batch_stride", _u64), ("mask_node_stride", _u64),
        ("counts", _vp), ("starts", _vp), ("starts_batch_stride", _u64), ("starts_node_stride", _u64),
        ("batch", _u64), ("nodes", _u64), ("q_heads", _u32), ("scale", ctypes.c_float),
    ]


SEARCH_EXPORTS = [
    "df11_paged_tree_attention", "df11_paged_tree_attention_workspace_bytes", "df11_paged_copy", "df11_paged_compact",
    "df11_paged_fork", "df11_paged_fork_workspace_bytes", "df11_beam_select", "df11_beam_select_workspace_bytes",
]

_SIGNATURES = {
    "df11_paged_tree_attention": ([_vp, _vp, _vp, _u64, _u64, _vp, _vp, _vp, _vp, _u64, _vp], _i32),
    "df11_paged_tree_attention_workspace_bytes": ([_u64, _u64, _u32, _u32, _u32, _u32, _u64], _u64),
    "df11_paged_copy": ([_vp, _u32, _u64, _u64, _vp, _vp, _vp, _u64, _vp], _i32),
    "df11_paged_compact": ([_vp, _u32, _u64, _u64, _vp, _u32, _vp, _vp, _u64, _u64, _vp, _u64, _vp], _i32),
    "df11_paged_fork": ([_vp, _u64, _vp, _u64, _u64, _u32, _vp, _vp, _u64, _u64, _vp, _vp, _vp, _vp, _vp, _u64, _vp], _i32),
    "df11_paged_fork_workspace_bytes": ([_u64, _u64, _u32, _u64, _u64], _u64),
    "df11_beam_select": ([_vp, _u32, _u64, _u64, _u64, _u64, _u64, _vp, _vp, _u32, _i32, _vp, _vp, _vp, _vp, _u64, _vp], _i32),
    "df11_beam_select_workspace_bytes": ([_u64, _u64, _u64, _u32], _u64),
}

_torch = None  # torch and the library, from the first call on
_L = None


def declare(L) -> None:
    """Sets the argument and result types of the entry points."""
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _load():
    global _torch, _L
    torch = step._torch or step._load()
    _L = step._L
    _torch = torch
    return torch


def _whole(t, name, shape, dev):
    """Checks a contiguous tensor of 32-bit whole numbers."""
    _tensor(t, name, _torch.int32, len(shape), dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    _dense(t, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def df11_paged_tree_attention_workspace_bytes(batch: int, nodes: int, q_heads: int, kv_heads: int, head_dim: int,
                                              page_size: int, table_width: int) -> int:
    """Bytes of workspace df11_paged_tree_attention needs."""
    if _torch is None:
        _load()
    return int(_L.df11_paged_tree_attention_workspace_bytes(int(batch), int(nodes), int(q_heads), int(kv_heads),
                                                            int(head_dim), int(page_size), int(table_width)))


@functools.lru_cache(maxsize=1024)
def _tree_need(*sizes):
    return int(_L.df11_paged_tree_attention_workspace_bytes(*sizes))


def df11_paged_tree_attention(q, k_pages, v_pages, page_table, lens, tree=None, nodes=None, starts=None, scale=None,
                              k_scale=None, v_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens ("nodes"), whose keys and values the cache holds
    behind each sequence's length already: node a of sequence b at position
    lens[b] + a.

    q           BF16 [batch, nodes, q_heads, head_dim]; q_heads a multiple of the pages' kv_heads
    k_pages,    as for df11_paged_append
    v_pages
    page_table  int32 [batch, width]
    lens        int32 [batch]: positions in front of the nodes
    tree        int64 [batch, nodes, ceil(nodes / 64)]: bit a % 64 of word a / 64 of node i says whether i reads
                node a (itself only if named); None: a chain, nodes 0..i
    nodes       int32 [batch]: how many nodes each sequence has; None: all
    starts      int32 [batch, nodes]: a node reads positions [start, lens[b]) and nodes; None: from 0.  A start cuts
                nothing of the nodes: a chain longer than its window needs a tree
    scale       of the scores; None: head_dim ** -0.5
    tree and starts may have any strides, 0 among them (one tree for all sequences), but the words of a node lie next
    to each other and nodes share none.
    Returns (out, lse): BF16 like q and float32 [batch, nodes, q_heads]; rows that read nothing get zeros and -inf."""
    torch = _torch or _load()
    i32 = torch.int32
    dev = _tensor(q, "q", torch.bfloat16, 4, -1)
    _last_dense(q, "q")
    c = step._cache(k_pages, v_pages, k_scale, v_scale, dev)
    _tensor(page_table, "page_table", i32, 2, dev)
    _last_dense(page_table, "page_table")
    batch, n, heads, dim = q.shape
    kv_heads = c.kv_heads
    if dim != c.head_dim or kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"q {tuple(q.shape)} does not fit pages of {kv_heads} heads of {c.head_dim}")
    if page_table.shape[0] != batch:
        raise ValueError(f"page_table must hold {batch} sequences")
    _whole(lens, "lens", (batch,), dev)
    if nodes is not None:
        _whole(nodes, "nodes", (batch,), dev)
    t0 = t1 = s0 = s1 = 0
    if tree is not None:
        _tensor(tree, "tree", torch.int64, 3, dev)
        if tree.shape != (batch, n, (n + 63) // 64):
            raise ValueError(f"tree must be {(batch, n, (n + 63) // 64)}, got {tuple(tree.shape)}")
        _last_dense(tree, "tree")
        t0, t1, _ = tree.stride()
        if n <= 1:  # torch leaves the strides of single nodes open
            t1 = 0
        elif t1 < tree.shape[2]:
            raise ValueError("the nodes of tree must not share words")
    if starts is not None:
        _tensor(starts, "starts", i32, 2, dev)
        if starts.shape != (batch, n):
            raise ValueError(f"starts must be {(batch, n)}, got {tuple(starts.shape)}")
        s0, s1 = starts.stride()
    scale = dim ** -0.5 if scale is None else float(scale)
    _no_gradient("df11_paged_tree_attention", q, k_pages, v_pages, k_scale, v_scale, out, lse)
    q0, q1, q2, _ = q.stride()
    t = df11_tree(q.data_ptr(), q0, q1, q2, _ptr(tree), t0, t1, _ptr(nodes), _ptr(starts), s0, s1, batch, n, heads, scale)
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _tree_attention(q, c, t, page_table, lens, out, lse, workspace, dev, handle)
    with ctx:
        return _tree_attention(q, c, t, page_table, lens, out, lse, workspace, dev, handle)


def _tree_attention(q, c, t, page_table, lens, out, lse, workspace, dev, handle):
    batch, n, heads, dim = q.shape
    if out is None:
        out = q.new_empty((batch, n, heads, dim))
    else:
        _dense(_out(out, q, (batch, n, heads, dim), _torch.bfloat16, dev), "out")
    if lse is None:
        lse = q.new_empty((batch, n, heads), dtype=_torch.float32)
    else:
        _dense(_out(lse, q, (batch, n, heads), _torch.float32, dev, "lse"), "lse")
    width = page_table.shape[1]
    need = _tree_need(batch, n, heads, c.kv_heads, dim, c.page_size, width)
    keep, ws, size = _workspace(workspace, need, q, dev)
    st = _L.df11_paged_tree_attention(ctypes.byref(c), ctypes.byref(t), page_table.data_ptr(),
                                      page_table.stride(0) if batch > 1 else width, width, lens.data_ptr(),
                                      out.data_ptr(), lse.data_ptr(), ws, size, handle)
    if st:
        _check(st, "df11_paged_tree_attention")
    return out, lse


def _layers(k_pages, v_pages, dev):
    """(df11_paged_cache without scales, layers, strides of a layer, GPU) of pages [n_pages, kv_heads, page_size,
    head_dim] or [layers, n_pages, ...]."""
    torch = _torch
    dtype = k_pages.dtype if isinstance(k_pages, torch.Tensor) else None
    if dtype is not torch.bfloat16 and dtype is not torch.float8_e4m3fn:
        raise TypeError(f"pages must be device tensors of bfloat16 or float8_e4m3fn, got {dtype}")
    rank = 5 if k_pages.dim() == 5 else 4
    dev = _tensor(k_pages, "k_pages", dtype, rank, dev)
    _tensor(v_pages, "v_pages", dtype, rank, dev)
    shape = k_pages.shape
    if v_pages.shape != shape:
        raise ValueError("k_pages and v_pages differ in shape")
    ks, vs = k_pages.stride(), v_pages.stride()
    layers, kl, vl = 1, 0, 0
    if rank == 5:
        layers = shape[0]
        if layers > 1:
            kl, vl = ks[0], vs[0]
        shape, ks, vs = shape[1:], ks[1:], vs[1:]
    n, h, page, d = shape
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last dimension of the pages must be contiguous")
    k0, k1, k2, _ = ks
    v0, v1, v2, _ = vs
    if n == 1:  # torch leaves the strides of single pages and heads open
        k0 = v0 = 0
    if h == 1:
        k1 = v1 = 0
    c = df11_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(), n, k0, k1, k2, v0, v1, v2, None, None, h, d, page,
                         step.DF11_CACHE_E4M3 if dtype is torch.float8_e4m3fn else step.DF11_CACHE_BF16)
    return c, layers, kl, vl, dev


def df11_paged_copy(src, dst, k_pages, v_pages, rows=None, stream=None) -> None:
    """Copies page src[i] to page dst[i], keys and values of all heads (and
    layers), for pages [n_pages, kv_heads, page_size, head_dim] or [layers,
    n_pages, kv_heads, page_size, head_dim] as for df11_paged_append.  src, dst:
    int32 [n]; a pair with a number outside the cache is skipped.  rows: int32 [n],
    the first positions to copy; None: whole pages.  A page must not be the target
    of two pairs, or of one and the source of another."""
    if _torch is None:
        _load()
    c, layers, kl, vl, dev = _layers(k_pages, v_pages, -1)
    _tensor(src, "src", _torch.int32, 1, dev)
    n = src.shape[0]
    _whole(src, "src", (n,), dev)
    _whole(dst, "dst", (n,), dev)
    if rows is not None:
        _whole(rows, "rows", (n,), dev)
    _no_gradient("df11_paged_copy", k_pages, v_pages)
    handle, ctx = _place(dev, stream)
    args = (ctypes.byref(c), layers, kl, vl, src.data_ptr(), dst.data_ptr(), _ptr(rows), n, handle)
    if ctx is None:
        st = _L.df11_paged_copy(*args)
    else:
        with ctx:
            st = _L.df11_paged_copy(*args)
    if st:
        _check(st, "df11_paged_copy")


def df11_paged_compact(path, accepted, page_table, lens, k_pages, v_pages, stream=None) -> None:
    """Moves keys and values from position lens[b] + path[b, i] of each sequence to
    lens[b] + i, for i < accepted[b]: an accepted path of a drafted tree next to
    what the cache held.  path: int32 [batch, depth], ascending (the first number
    that is not ends it); accepted, lens: int32 [batch]; page_table: int32 [batch,
    width]; pages as for df11_paged_copy.  lens stays as it is: add accepted to it
    when all layers are done."""
    if _torch is None:
        _load()
    c, layers, kl, vl, dev = _layers(k_pages, v_pages, -1)
    _tensor(path, "path", _torch.int32, 2, dev)
    batch, depth = path.shape
    _dense(path, "path")
    _whole(accepted, "accepted", (batch,), dev)
    _whole(lens, "lens", (batch,), dev)
    _tensor(page_table, "page_table", _torch.int32, 2, dev)
    _last_dense(page_table, "page_table")
    if page_table.shape[0] != batch:
        raise ValueError(f"page_table must hold {batch} sequences")
    _no_gradient("df11_paged_compact", k_pages, v_pages)
    width = page_table.shape[1]
    handle, ctx = _place(dev, stream)
    args = (ctypes.byref(c), layers, kl, vl, path.data_ptr(), depth, accepted.data_ptr(), page_table.data_ptr(),
            page_table.stride(0) if batch > 1 else width, width, lens.data_ptr(), batch, handle)
    if ctx is None:
        st = _L.df11_paged_compact(*args)
    else:
        with ctx:
            st = _L.df11_paged_compact(*args)
    if st:
        _check(st, "df11_paged_compact")


def df11_paged_fork_workspace_bytes(batch: int, table_width: int, page_size: int, n_pages: int, room: int) -> int:
    """Bytes of workspace df11_paged_fork needs."""
    if _torch is None:
        _load()
    return int(_L.df11_paged_fork_workspace_bytes(int(batch), int(table_width), int(page_size), int(n_pages), int(room)))


@functools.lru_cache(maxsize=1024)
def _fork_need(*sizes):
    return int(_L.df11_paged_fork_workspace_bytes(*sizes))


def df11_paged_fork(parents, page_table, lens, refs, page_size: int, room: int = 1, workspace=None, stream=None):
    """Reorders the sequences of a page table, in place: row b goes on from row
    parents[b] (outside [0, batch): it ends).  Full pages are shared; the last
    positions, in a page that is not full, and `room` more get pages of the row's
    own, free ones unless the row is the first to go on from its parent; pages that
    nobody holds any longer are free from the next call on.

    parents     int32 [batch], or None: every row goes on from itself (trims and reserves pages)
    page_table  int32 [batch, width], changed: -1 where a row holds no page
    lens        int32 [batch], changed: the length of each row's parent
    refs        int32 [n_pages], changed: holders of each page; 0: free
    Returns (src, dst, rows, missing): int32 [batch] each, what df11_paged_copy has
    to copy in every layer (-1, -1, 0 for a row that needs nothing), and int32 [1],
    the pages that were wanted and not to be had (their entries are -1)."""
    torch = _torch or _load()
    i32 = torch.int32
    dev = _tensor(page_table, "page_table", i32, 2, -1)
    _last_dense(page_table, "page_table")
    batch, width = page_table.shape
    if parents is not None:
        _whole(parents, "parents", (batch,), dev)
    _whole(lens, "lens", (batch,), dev)
    _tensor(refs, "refs", i32, 1, dev)
    _dense(refs, "refs")
    page_size, room = int(page_size), int(room)
    if not 0 <= page_size < 1 << 32 or not 0 <= room < 1 << 64:  # what their C types hold
        raise ValueError("page_size must fit 32 bits and room 64, neither negative")
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _fork(parents, page_table, lens, refs, page_size, room, workspace, dev, handle)
    with ctx:
        return _fork(parents, page_table, lens, refs, page_size, room, workspace, dev, handle)


def _fork(parents, page_table, lens, refs, page_size, room, workspace, dev, handle):
    batch, width = page_table.shape
    pool = refs.shape[0]
    need = _fork_need(batch, width, page_size, pool, room)
    keep, ws, size = _workspace(workspace, need, refs, dev)
    src, dst, rows, missing = refs.new_empty(3 * batch + 1).split_with_sizes((batch, batch, batch, 1))
    st = _L.df11_paged_fork(_ptr(parents), batch, page_table.data_ptr(), page_table.stride(0) if batch > 1 else width,
                            width, page_size, lens.data_ptr(), refs.data_ptr(), pool, room, src.data_ptr(),
                            dst.data_ptr(), rows.data_ptr(), missing.data_ptr(), ws, size, handle)
    if st:
        _check(st, "df11_paged_fork")
    return src, dst, rows, missing


def df11_beam_select_workspace_bytes(batch: int, beams: int, vocab: int, k: int) -> int:
    """Bytes of workspace df11_beam_select needs."""
    if _torch is None:
        _load()
    return int(_L.df11_beam_select_workspace_bytes(int(batch), int(beams), int(vocab), int(k)))


@functools.lru_cache(maxsize=1024)
def _beam_need(*sizes):
    return int(_L.df11_beam_select_workspace_bytes(*sizes))


def df11_beam_select(logits, scores, k: int, done=None, pad: int = 0, workspace=None, stream=None):
    """The k best continuations of each search: scores[b, i] + log softmax of beam
    i's logits, over all beams and tokens.

    logits  BF16 or float32 [batch, beams, vocab], the last dimension contiguous
    scores  float32 [batch, beams]; a beam whose score is no finite number offers nothing
    k       up to 64
    done    bool or uint8 [batch, beams]: beams that have ended go on once, as they are, with token `pad`
    Returns (scores, parents, tokens): float32, int32 and int32 [batch, k], best
    first; parents are rows of the [batch * beams] sequences (what df11_paged_fork
    takes); of equal scores the lower beam and token come first.  Places for which
    no candidate is left hold -inf, -1 and pad."""
    torch = _torch or _load()
    bf16 = isinstance(logits, torch.Tensor) and logits.dtype is torch.bfloat16
    dev = _tensor(logits, "logits", torch.bfloat16 if bf16 else torch.float32, 3, -1)
    _last_dense(logits, "logits")
    batch, beams, vocab = logits.shape
    _tensor(scores, "scores", torch.float32, 2, dev)
    _dense(scores, "scores")
    if scores.shape != (batch, beams):
        raise ValueError(f"scores must be {(batch, beams)}, got {tuple(scores.shape)}")
    if done is not None:
        _tensor(done, "done", torch.bool if getattr(done, "dtype", None) is torch.bool else torch.uint8, 2, dev)
        _dense(done, "done")
        if done.shape != (batch, beams):
            raise ValueError(f"done must be {(batch, beams)}, got {tuple(done.shape)}")
    k, pad = int(k), int(pad)
    if not 0 < k <= 64:
        raise ValueError(f"k must be 1 to 64, got {k}")
    if not -1 << 31 <= pad < 1 << 31:
        raise ValueError("pad must fit 32 bits")
    _no_gradient("df11_beam_select", logits, scores)
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _select(logits, scores, k, done, pad, workspace, bf16, dev, handle)
    with ctx:
        return _select(logits, scores, k, done, pad, workspace, bf16, dev, handle)


def _select(logits, scores, k, done, pad, workspace, bf16, dev, handle):
    batch, beams, vocab = logits.shape
    best = scores.new_empty((batch, k))
    parents = scores.new_empty((batch, k), dtype=_torch.int32)
    tokens = scores.new_empty((batch, k), dtype=_torch.int32)
    need = _beam_need(batch, beams, vocab, k)
    keep, ws, size = _workspace(workspace, need, scores, dev)
    s0, s1, _ = logits.stride()
    st = _L.df11_beam_select(logits.data_ptr(), DF11_LOGITS_BF16 if bf16 else DF11_LOGITS_FP32, batch, beams, vocab, s0, s1,
                             scores.data_ptr(), _ptr(done), k, pad, best.data_ptr(), parents.data_ptr(),
                             tokens.data_ptr(), ws, size, handle)
    if st:
        _check(st, "df11_beam_select")
    return best, parents, tokens
