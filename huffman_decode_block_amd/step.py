"""Binding of the token step's operators (include/df11_step.h): 4-bit weights
and the product that reads them, a paged key-value cache, its writer and the
attention of one token that reads it.

Argument marshalling only, as in the rest of the package: each call checks its
tensors, allocates what it returns and its workspace with torch, and launches
HIP kernels of the library on `stream` (torch stream, raw handle, or None for
the current stream).  With a stream other than the current one, what a call
allocates belongs to that stream.

No call has a derivative.  df11_mx4_matmul, df11_paged_append and
df11_paged_attention refuse a tensor that asks for one (requires_grad where
gradients are enabled, or a forward-mode tangent) rather than lose it; call them
under torch.no_grad() or with detached tensors.
"""
from __future__ import annotations

import ctypes
import functools

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


_torch = None  # torch, its forward-mode derivatives and the library, from the first call on
_forward_ad = None
_L = None


def declare(L) -> None:
    """Sets the argument and result types of the step's entry points."""
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _load():
    global _torch, _forward_ad, _L
    import torch
    from torch.autograd import forward_ad

    from . import lib
    _L = lib()
    _forward_ad = forward_ad
    _torch = torch
    return torch


def _check(status: int, what: str):
    if status:
        from . import _check as check
        check(status, what)


def _place(dev, stream):
    """Where a call on GPU number `dev` runs: the raw stream handle, and None or
    a context that makes that device and stream torch's current ones (so that
    what the call allocates belongs to its stream)."""
    torch = _torch
    # torch's own calls below the public ones, which build a Stream object and
    # check for initialisation: 2 us less of a call's 9
    here = torch._C._cuda_getDevice() == dev
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev), None if here else torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        if here and handle == torch._C._cuda_getCurrentRawStream(dev):
            return handle, None
        # the null stream has no ExternalStream: torch takes its handle, 0, for one that was not given
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"stream belongs to GPU {stream.device_index}, the tensors to {dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _tensor(t, name, dtype, ndim, dev):
    """Checks a tensor's type, rank and place (a GPU's number; -1 for any GPU)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a device tensor")
    at = t.get_device()
    if at < 0:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if at != dev and dev >= 0:
        raise ValueError(f"{name} is on GPU {at}, not {dev}")
    return at


def _no_gradient(what, *tensors):
    """Refuses tensors (or None) that ask for a derivative: what a call returns has no history."""
    if _torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{what} has no backward and was given a tensor that requires a gradient: call it under "
                                 "torch.no_grad() or with detached tensors")
    if _forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{what} has no derivative and was given a tensor with a tangent")


def _last_dense(t, name):
    """The last dimension's values lie next to each other."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _row_stride(t):
    """A matrix's row stride; of a single row (torch leaves it open) its length."""
    rows, cols = t.shape
    return t.stride(0) if rows > 1 else cols or 1


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(given, need, like, dev):
    """(tensor to keep, address, bytes) of a workspace: the given one or a new one."""
    if given is not None:
        if not isinstance(given, _torch.Tensor) or given.get_device() != dev or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor on the inputs' GPU")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    t = like.new_empty((need,), dtype=_torch.uint8)
    return t, t.data_ptr(), need


def df11_mx4_matmul_workspace_bytes(m: int, n: int, k: int, x_aligned: bool = True) -> int:
    """Bytes of workspace df11_mx4_matmul needs."""
    if _torch is None:
        _load()
    return int(_L.df11_mx4_matmul_workspace_bytes(int(m), int(n), int(k), 1 if x_aligned else 0))


def _codes(codes, scales, cols, dev):
    """Checks codes and scale bytes of a matrix with `cols` columns; returns its rows and GPU."""
    u8 = _torch.uint8
    dev = _tensor(codes, "codes", u8, 2, dev)
    rows, width = codes.shape
    blocks = (cols + 31) // 32
    if not (isinstance(scales, _torch.Tensor) and scales.dtype is u8 and scales.get_device() == dev):
        _tensor(scales, "scales", u8, 2, dev)
    if scales.shape != (rows, blocks) or width != 16 * blocks:
        raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold {cols} columns: "
                         f"[rows, {16 * blocks}] and [rows, {blocks}] expected")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    return rows, dev


def df11_mx4_quantize(x, codes=None, scales=None, stream=None):
    """4-bit codes and scale bytes of x (BF16 device matrix [rows, cols], rows
    may be strided): uint8 tensors [rows, 16 * ceil(cols / 32)] and [rows,
    ceil(cols / 32)], allocated when None.  Returns (codes, scales)."""
    torch = _torch or _load()
    dev = _tensor(x, "x", torch.bfloat16, 2, -1)
    _last_dense(x, "x")
    if x.shape[1] == 0:
        raise ValueError("x has no columns")
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _quantize(x, codes, scales, dev, handle)
    with ctx:
        return _quantize(x, codes, scales, dev, handle)


def _quantize(x, codes, scales, dev, handle):
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    given = codes is not None or scales is not None
    if codes is None:
        codes = x.new_empty((rows, 16 * blocks), dtype=_torch.uint8)
    if scales is None:
        scales = x.new_empty((rows, blocks), dtype=_torch.uint8)
    if given and _codes(codes, scales, cols, dev)[0] != rows:
        raise ValueError(f"codes has {codes.shape[0]} rows, x {rows}")
    _check(_L.df11_mx4_quantize(x.data_ptr(), rows, cols, _row_stride(x), codes.data_ptr(), scales.data_ptr(), handle),
           "df11_mx4_quantize")
    return codes, scales


def df11_mx4_dequantize(codes, scales, cols: int, out=None, stream=None):
    """The values of 4-bit codes as a BF16 matrix [rows, cols] (exact).  Returns out."""
    if _torch is None:
        _load()
    cols = int(cols)
    if cols <= 0:
        raise ValueError("cols must be positive")
    _, dev = _codes(codes, scales, cols, -1)
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _dequantize(codes, scales, cols, out, dev, handle)
    with ctx:
        return _dequantize(codes, scales, cols, out, dev, handle)


def _out(out, like, shape, dtype, dev, name="out"):
    """A new output on the device of `like`, or the given one checked."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _tensor(out, name, dtype, len(shape), dev)
    if out.shape != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(out.shape)}")
    _last_dense(out, name)
    return out


def _dequantize(codes, scales, cols, out, dev, handle):
    rows = codes.shape[0]
    out = _out(out, codes, (rows, cols), _torch.bfloat16, dev)
    _check(_L.df11_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), _row_stride(out),
                                  handle), "df11_mx4_dequantize")
    return out


def df11_mx4_matmul(x, codes, scales, out=None, workspace=None, stream=None):
    """out [m, n] := x [m, k] (BF16, rows may be strided) times the transpose
    of the 4-bit matrix [n, k] in codes and scales; sums in 32 bits, one
    rounding.  workspace: df11_mx4_matmul_workspace_bytes bytes, allocated
    when None and needed.  Returns out."""
    torch = _torch or _load()
    dev = _tensor(x, "x", torch.bfloat16, 2, -1)
    m, k = x.shape
    xs, x1 = x.stride()
    if x1 != 1 and k > 1:
        raise ValueError("the last dimension of x must be contiguous")
    if m <= 1:  # torch leaves the stride of a single row open
        xs = k or 1
    n, _ = _codes(codes, scales, k, dev)
    _no_gradient("df11_mx4_matmul", x, out)
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _matmul(x, m, k, xs, codes, scales, n, out, workspace, dev, handle)
    with ctx:
        return _matmul(x, m, k, xs, codes, scales, n, out, workspace, dev, handle)


def _matmul(x, m, k, xs, codes, scales, n, out, workspace, dev, handle):
    if out is None:
        out, ys = x.new_empty((m, n)), n or 1
    else:
        ys = _row_stride(_out(out, x, (m, n), _torch.bfloat16, dev))
    xp = x.data_ptr()
    keep, ws, size = workspace, None, 0
    if workspace is not None or k % 32 or xs % 8 or xp % 16 or xs > 1 << 21:
        need = _L.df11_mx4_matmul_workspace_bytes(m, n, k, xs % 8 == 0 and xp % 16 == 0 and xs <= 1 << 21)
        keep, ws, size = _workspace(workspace, need, x, dev)
    st = _L.df11_mx4_matmul(xp, m, k, xs, codes.data_ptr(), scales.data_ptr(), n, out.data_ptr(), ys, ws, size, handle)
    if st:
        _check(st, "df11_mx4_matmul")
    return out


def _cache(k_pages, v_pages, k_scale, v_scale, dev):
    """The df11_paged_cache of page tensors [n_pages, kv_heads, page_size, head_dim]."""
    torch = _torch
    dtype = k_pages.dtype if isinstance(k_pages, torch.Tensor) else None
    e4m3 = dtype is torch.float8_e4m3fn
    if not e4m3 and dtype is not torch.bfloat16:
        raise TypeError(f"pages must be device tensors of bfloat16 or float8_e4m3fn, got {dtype}")
    _tensor(k_pages, "k_pages", dtype, 4, dev)
    _tensor(v_pages, "v_pages", dtype, 4, dev)
    shape = k_pages.shape
    if v_pages.shape != shape:
        raise ValueError("k_pages and v_pages differ in shape")
    n, h, page, d = shape
    k0, k1, k2, k3 = k_pages.stride()
    v0, v1, v2, v3 = v_pages.stride()
    if k3 != 1 or v3 != 1:
        raise ValueError("the last dimension of the pages must be contiguous")
    if n == 1:  # torch leaves the strides of single pages and heads open
        k0 = v0 = 0
    if h == 1:
        k1 = v1 = 0
    ks = vs = None
    if e4m3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise ValueError(f"E4M3 pages need {name}")
            _tensor(t, name, torch.float32, 1, dev)
            _dense(t, name)
            if t.shape[0] != h:
                raise ValueError(f"{name} must hold {h} values, one for each head")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to E4M3 pages")
    return df11_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(), n, k0, k1, k2, v0, v1, v2, ks, vs, h, d, page,
                            DF11_CACHE_E4M3 if e4m3 else DF11_CACHE_BF16)


def df11_paged_append(k, v, slots, k_pages, v_pages, k_scale=None, v_scale=None, stream=None) -> None:
    """Writes keys and values (BF16 [tokens, kv_heads, head_dim], the last
    dimension contiguous) into pages [n_pages, kv_heads, page_size, head_dim]
    (BF16 or float8_e4m3fn, any layout whose head_dim values are contiguous).
    slots: int64 [tokens], page * page_size + position; negative or past the
    cache: the token is skipped.  E4M3 pages take k_scale and v_scale, float32
    [kv_heads]: what is stored is the value over its head's scale."""
    torch = _torch or _load()
    bf16 = torch.bfloat16
    dev = _tensor(k, "k", bf16, 3, -1)
    _tensor(v, "v", bf16, 3, dev)
    _tensor(slots, "slots", torch.int64, 1, dev)
    _dense(slots, "slots")
    _last_dense(k, "k")
    _last_dense(v, "v")
    c = _cache(k_pages, v_pages, k_scale, v_scale, dev)
    t = slots.shape[0]
    want = (t, c.kv_heads, c.head_dim)
    if k.shape != want or v.shape != want:
        raise ValueError(f"k and v must be {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
    _no_gradient("df11_paged_append", k, v, k_pages, v_pages, k_scale, v_scale)
    handle, ctx = _place(dev, stream)
    k0, k1, _ = k.stride()
    v0, v1, _ = v.stride()
    args = (ctypes.byref(c), k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, slots.data_ptr(), t, handle)
    if ctx is None:
        st = _L.df11_paged_append(*args)
    else:
        with ctx:
            st = _L.df11_paged_append(*args)
    _check(st, "df11_paged_append")


def df11_paged_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                                         table_width: int) -> int:
    """Bytes of workspace df11_paged_attention needs."""
    if _torch is None:
        _load()
    return int(_L.df11_paged_attention_workspace_bytes(int(batch), int(q_heads), int(kv_heads), int(head_dim),
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
    torch = _torch or _load()
    i32 = torch.int32
    dev = _tensor(q, "q", torch.bfloat16, 3, -1)
    _last_dense(q, "q")
    c = _cache(k_pages, v_pages, k_scale, v_scale, dev)
    _tensor(page_table, "page_table", i32, 2, dev)
    _last_dense(page_table, "page_table")
    batch, heads, dim = q.shape
    kv_heads = c.kv_heads
    if dim != c.head_dim or kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"q {tuple(q.shape)} does not fit pages of {kv_heads} heads of {c.head_dim}")
    _tensor(lens, "lens", i32, 1, dev)
    if page_table.shape[0] != batch or lens.shape[0] != batch:
        raise ValueError(f"page_table and lens must hold {batch} sequences")
    _dense(lens, "lens")
    if starts is not None:
        _tensor(starts, "starts", i32, 1, dev)
        _dense(starts, "starts")
        if starts.shape[0] != batch:
            raise ValueError(f"starts must hold {batch} sequences")
    scale = dim ** -0.5 if scale is None else float(scale)
    _no_gradient("df11_paged_attention", q, k_pages, v_pages, k_scale, v_scale, out, lse)
    handle, ctx = _place(dev, stream)
    if ctx is None:
        return _attention(q, c, page_table, lens, starts, scale, out, lse, workspace, dev, handle)
    with ctx:
        return _attention(q, c, page_table, lens, starts, scale, out, lse, workspace, dev, handle)


def _attention(q, c, page_table, lens, starts, scale, out, lse, workspace, dev, handle):
    batch, heads, dim = q.shape
    if out is None:
        out = q.new_empty((batch, heads, dim))
    else:
        _dense(_out(out, q, (batch, heads, dim), _torch.bfloat16, dev), "out")
    if lse is None:
        lse = q.new_empty((batch, heads), dtype=_torch.float32)
    else:
        _dense(_out(lse, q, (batch, heads), _torch.float32, dev, "lse"), "lse")
    width = page_table.shape[1]
    need = _attention_need(batch, heads, c.kv_heads, dim, c.page_size, width)
    keep, ws, size = _workspace(workspace, need, q, dev)
    q0, q1, _ = q.stride()
    st = _L.df11_paged_attention(ctypes.byref(c), q.data_ptr(), batch, heads, q0, q1, page_table.data_ptr(),
                                 page_table.stride(0) if batch > 1 else width, width, lens.data_ptr(),
                                 None if starts is None else starts.data_ptr(), scale, out.data_ptr(), lse.data_ptr(),
                                 ws, size, handle)
    if st:
        _check(st, "df11_paged_attention")
    return out, lse


@functools.lru_cache(maxsize=1024)
def _attention_need(*sizes):
    return int(_L.df11_paged_attention_workspace_bytes(*sizes))
