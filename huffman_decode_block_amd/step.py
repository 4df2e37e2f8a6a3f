"""Binding of the token step's operators (include/df11_step.h): 4-bit weights
and the product that reads them, a paged key-value cache, its writer and the
attention of one token that reads it.

Argument marshalling only, as in the rest of the package: each call checks its
tensors, allocates what it returns and its workspace with torch, and launches
HIP kernels of the library on `stream` (torch stream, raw handle, or None for
the current stream).  With a stream other than the current one, what a call
allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_vp = ctypes.c_void_p

DF11_CACHE_BF16 = 0
DF11_CACHE_E4M3 = 1


class df11_paged_cache(ctypes.Structure):
    _fields_ = [
        ("k_pages", _vp), ("v_pages", _vp), ("n_pages", _u64),
        ("k_page_stride", _u64), ("k_head_stride", _u64), ("k_row_stride", _u64),
        ("v_page_stride", _u64), ("v_head_stride", _u64), ("v_row_stride", _u64),
        ("k_scale", _vp), ("v_scale", _vp),
        ("kv_heads", _u32), ("head_dim", _u32), ("page_size", _u32), ("dtype", _u32),
    ]


STEP_EXPORTS = [
    "df11_mx4_quantize", "df11_mx4_dequantize", "df11_mx4_matmul", "df11_mx4_matmul_workspace_bytes",
    "df11_paged_append", "df11_paged_attention", "df11_paged_attention_workspace_bytes",
]

_SIGNATURES = {
    "df11_mx4_quantize": ([_vp, _u64, _u64, _u64, _vp, _vp, _vp], _i32),
    "df11_mx4_dequantize": ([_vp, _vp, _u64, _u64, _vp, _u64, _vp], _i32),
    "df11_mx4_matmul": ([_vp, _u64, _u64, _u64, _vp, _vp, _u64, _vp, _u64, _vp, _u64, _vp], _i32),
    "df11_mx4_matmul_workspace_bytes": ([_u64, _u64, _u64, _i32], _u64),
    "df11_paged_append": ([_vp, _vp, _u64, _u64, _vp, _u64, _u64, _vp, _u64, _vp], _i32),
    "df11_paged_attention": ([_vp, _vp, _u64, _u64, _u64, _u64, _vp, _u64, _u64, _vp, _vp, _f32, _vp, _vp, _vp, _u64,
                              _vp], _i32),
    "df11_paged_attention_workspace_bytes": ([_u64, _u64, _u32, _u32, _u32, _u64], _u64),
}


def declare(L) -> None:
    """Sets the argument and result types of the step's entry points."""
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _lib():
    from . import lib
    return lib()


def _check(status: int, what: str):
    if status:
        from . import _check as check
        check(status, what)


class _On:
    """The device and stream a call runs on: raw handle, and, where the stream
    is not the current one, a context in which torch allocates for it."""

    __slots__ = ("torch", "device", "handle", "stack")

    def __init__(self, device, stream):
        import torch
        self.torch, self.device, self.stack = torch, device, None
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
        elif isinstance(stream, torch.cuda.Stream):
            self.handle = stream.cuda_stream
        else:
            self.handle = int(stream)
        if device.index != torch.cuda.current_device() or (
                stream is not None and self.handle != torch.cuda.current_stream(device).cuda_stream):
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(self.handle, device=device)
            self.stack = stream

    def __enter__(self):
        if self.stack is not None:
            self.stack = self.torch.cuda.stream(self.stack)
            self.stack.__enter__()
        return self

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.__exit__(*exc)


def _tensor(t, name, dtype, ndim, dev=None):
    """Checks a tensor's place, type and rank."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not {dev}")


def _last_dense(t, name):
    """The last dimension's values lie next to each other and no stride is negative or hidden by expansion."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _row_stride(t):
    """A matrix's row stride; of a single row (torch leaves it open) its length."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(torch, given, need, dev):
    if given is not None:
        if not isinstance(given, torch.Tensor) or not given.is_cuda or given.device != dev or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor on the inputs' GPU")
        return given, given.numel() * given.element_size()
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def df11_mx4_matmul_workspace_bytes(m: int, n: int, k: int, x_aligned: bool = True) -> int:
    """Bytes of workspace df11_mx4_matmul needs."""
    return int(_lib().df11_mx4_matmul_workspace_bytes(int(m), int(n), int(k), 1 if x_aligned else 0))


def df11_mx4_quantize(x, codes=None, scales=None, stream=None):
    """4-bit codes and scale bytes of x (BF16 device matrix [rows, cols], rows
    may be strided): uint8 tensors [rows, 16 * ceil(cols / 32)] and [rows,
    ceil(cols / 32)], allocated when None.  Returns (codes, scales)."""
    import torch
    _tensor(x, "x", torch.bfloat16, 2)
    _last_dense(x, "x")
    rows, cols = x.shape
    if cols == 0:
        raise ValueError("x has no columns")
    blocks = (cols + 31) // 32
    with _On(x.device, stream) as on:
        if codes is None:
            codes = torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=x.device)
        if scales is None:
            scales = torch.empty((rows, blocks), dtype=torch.uint8, device=x.device)
        _codes(codes, scales, cols, x.device)
        if codes.shape[0] != rows:
            raise ValueError(f"codes has {codes.shape[0]} rows, x {rows}")
        st = _lib().df11_mx4_quantize(x.data_ptr(), rows, cols, _row_stride(x), codes.data_ptr(), scales.data_ptr(),
                                      on.handle)
    _check(st, "df11_mx4_quantize")
    return codes, scales


def _codes(codes, scales, cols, dev):
    import torch
    _tensor(codes, "codes", torch.uint8, 2, dev)
    _tensor(scales, "scales", torch.uint8, 2, dev)
    _dense(codes, "codes")
    _dense(scales, "scales")
    blocks = (cols + 31) // 32
    if codes.shape[1] != 16 * blocks or scales.shape[1] != blocks or codes.shape[0] != scales.shape[0]:
        raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold {cols} columns: "
                         f"[rows, {16 * blocks}] and [rows, {blocks}] expected")


def df11_mx4_dequantize(codes, scales, cols: int, out=None, stream=None):
    """The values of 4-bit codes as a BF16 matrix [rows, cols] (exact).  Returns out."""
    import torch
    cols = int(cols)
    if cols <= 0:
        raise ValueError("cols must be positive")
    _codes(codes, scales, cols, None)
    rows, dev = codes.shape[0], codes.device
    if scales.device != dev:
        raise ValueError(f"scales is on {scales.device}, not {dev}")
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        _tensor(out, "out", torch.bfloat16, 2, dev)
        _last_dense(out, "out")
        if tuple(out.shape) != (rows, cols):
            raise ValueError(f"out must be {(rows, cols)}, got {tuple(out.shape)}")
        st = _lib().df11_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(),
                                        _row_stride(out), on.handle)
    _check(st, "df11_mx4_dequantize")
    return out


def df11_mx4_matmul(x, codes, scales, out=None, workspace=None, stream=None):
    """out [m, n] := x [m, k] (BF16, rows may be strided) times the transpose
    of the 4-bit matrix [n, k] in codes and scales; sums in 32 bits, one
    rounding.  workspace: df11_mx4_matmul_workspace_bytes bytes, allocated
    when None and needed.  Returns out."""
    import torch
    _tensor(x, "x", torch.bfloat16, 2)
    _last_dense(x, "x")
    m, k = x.shape
    dev = x.device
    _codes(codes, scales, k, dev)
    n = codes.shape[0]
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        else:
            _tensor(out, "out", torch.bfloat16, 2, dev)
            _last_dense(out, "out")
            if tuple(out.shape) != (m, n):
                raise ValueError(f"out must be {(m, n)}, got {tuple(out.shape)}")
        L = _lib()
        xs, xp = _row_stride(x), x.data_ptr()
        need = L.df11_mx4_matmul_workspace_bytes(m, n, k, 1 if xs % 8 == 0 and xp % 16 == 0 and xs <= 1 << 21 else 0)
        ws, size = _workspace(torch, workspace, need, dev)
        st = L.df11_mx4_matmul(xp, m, k, xs, codes.data_ptr(), scales.data_ptr(), n, out.data_ptr(), _row_stride(out),
                               None if ws is None else ws.data_ptr(), size, on.handle)
    _check(st, "df11_mx4_matmul")
    return out


def _cache(k_pages, v_pages, k_scale, v_scale, dev):
    """The df11_paged_cache of page tensors [n_pages, kv_heads, page_size, head_dim]."""
    import torch
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a device tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [n_pages, kv_heads, page_size, head_dim], got {tuple(t.shape)}")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not {dev}")
        _last_dense(t, name)
    if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
        raise ValueError("k_pages and v_pages differ in shape or type")
    n, h, page, d = k_pages.shape
    e4m3 = k_pages.dtype == torch.float8_e4m3fn
    if not e4m3 and k_pages.dtype != torch.bfloat16:
        raise TypeError(f"pages must be bfloat16 or float8_e4m3fn, got {k_pages.dtype}")
    if e4m3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise ValueError(f"E4M3 pages need {name}")
            _tensor(t, name, torch.float32, 1, dev)
            _dense(t, name)
            if t.shape[0] != h:
                raise ValueError(f"{name} must hold {h} values, one for each head")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to E4M3 pages")
    ks, vs = k_pages.stride(), v_pages.stride()
    return df11_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(), n, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                            k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None, h, d, page,
                            DF11_CACHE_E4M3 if e4m3 else DF11_CACHE_BF16)


def df11_paged_append(k, v, slots, k_pages, v_pages, k_scale=None, v_scale=None, stream=None) -> None:
    """Writes keys and values (BF16 [tokens, kv_heads, head_dim], the last
    dimension contiguous) into pages [n_pages, kv_heads, page_size, head_dim]
    (BF16 or float8_e4m3fn, any layout whose head_dim values are contiguous).
    slots: int64 [tokens], page * page_size + position; negative or past the
    cache: the token is skipped.  E4M3 pages take k_scale and v_scale, float32
    [kv_heads]: what is stored is the value over its head's scale."""
    import torch
    _tensor(k, "k", torch.bfloat16, 3)
    dev = k.device
    _tensor(v, "v", torch.bfloat16, 3, dev)
    _tensor(slots, "slots", torch.int64, 1, dev)
    _dense(slots, "slots")
    _last_dense(k, "k")
    _last_dense(v, "v")
    c = _cache(k_pages, v_pages, k_scale, v_scale, dev)
    t = slots.shape[0]
    want = (t, c.kv_heads, c.head_dim)
    if tuple(k.shape) != want or tuple(v.shape) != want:
        raise ValueError(f"k and v must be {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
    with _On(dev, stream) as on:
        st = _lib().df11_paged_append(ctypes.byref(c), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                      v.stride(0), v.stride(1), slots.data_ptr(), t, on.handle)
    _check(st, "df11_paged_append")


def df11_paged_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                                         table_width: int) -> int:
    """Bytes of workspace df11_paged_attention needs."""
    return int(_lib().df11_paged_attention_workspace_bytes(int(batch), int(q_heads), int(kv_heads), int(head_dim),
                                                           int(page_size), int(table_width)))


def df11_paged_attention(q, k_pages, v_pages, page_table, lens, starts=None, scale=None, k_scale=None, v_scale=None,
                         out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token for each sequence over its pages.

    q           BF16 [batch, q_heads, head_dim]; q_heads a multiple of the pages' kv_heads
    k_pages,    as for df11_paged_append
    v_pages
    page_table  int32 [batch, width]: page of each page_size positions (entries outside the cache mask them)
    lens        int32 [batch]: sequence b reads positions [starts[b], lens[b]); starts None: from 0
    scale       of the scores; None: head_dim ** -0.5
    Returns (out, lse): BF16 [batch, q_heads, head_dim] and float32 [batch,
    q_heads], the natural logarithm of the sum of exponentials; a sequence
    with no position gets zeros and -inf."""
    import torch
    _tensor(q, "q", torch.bfloat16, 3)
    dev = q.device
    _last_dense(q, "q")
    c = _cache(k_pages, v_pages, k_scale, v_scale, dev)
    _tensor(page_table, "page_table", torch.int32, 2, dev)
    _last_dense(page_table, "page_table")
    _tensor(lens, "lens", torch.int32, 1, dev)
    _dense(lens, "lens")
    batch, heads, dim = q.shape
    if dim != c.head_dim or heads % max(1, c.kv_heads) != 0:
        raise ValueError(f"q {tuple(q.shape)} does not fit pages of {c.kv_heads} heads of {c.head_dim}")
    if page_table.shape[0] != batch or lens.shape[0] != batch:
        raise ValueError(f"page_table and lens must hold {batch} sequences")
    if starts is not None:
        _tensor(starts, "starts", torch.int32, 1, dev)
        _dense(starts, "starts")
        if starts.shape[0] != batch:
            raise ValueError(f"starts must hold {batch} sequences")
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((batch, heads, dim), dtype=torch.bfloat16, device=dev)
        else:
            _tensor(out, "out", torch.bfloat16, 3, dev)
            _dense(out, "out")
            if tuple(out.shape) != (batch, heads, dim):
                raise ValueError(f"out must be {(batch, heads, dim)}, got {tuple(out.shape)}")
        if lse is None:
            lse = torch.empty((batch, heads), dtype=torch.float32, device=dev)
        else:
            _tensor(lse, "lse", torch.float32, 2, dev)
            _dense(lse, "lse")
            if tuple(lse.shape) != (batch, heads):
                raise ValueError(f"lse must be {(batch, heads)}, got {tuple(lse.shape)}")
        L = _lib()
        width = page_table.shape[1]
        need = L.df11_paged_attention_workspace_bytes(batch, heads, c.kv_heads, dim, c.page_size, width)
        ws, size = _workspace(torch, workspace, need, dev)
        st = L.df11_paged_attention(
            ctypes.byref(c), q.data_ptr(), batch, heads, q.stride(0), q.stride(1), page_table.data_ptr(),
            page_table.stride(0) if batch > 1 else width, width, lens.data_ptr(),
            None if starts is None else starts.data_ptr(), dim ** -0.5 if scale is None else float(scale),
            out.data_ptr(), lse.data_ptr(), None if ws is None else ws.data_ptr(), size, on.handle)
    _check(st, "df11_paged_attention")
    return out, lse
