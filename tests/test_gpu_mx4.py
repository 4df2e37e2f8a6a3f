"""GPU checks of the 4-bit weights: codes and scales against the definition in
64 bits (exact, every BF16 pattern), their values (exact, every code under
every scale), and the product against 64-bit sums.

Bound of the product, for the result y of k exact products summed in 32 bits
in some order and rounded to BF16 once (8 significant bits: off by at most half
of 2^-7 of the value): |y - ref| <= 2^-8 |ref| + (1 + 2^-8) k 2^-23 sum |x w| (an
addition is off by at most 2^-23 of a partial sum, rounding or truncating, and
no partial sum exceeds sum |x w|).
"""
import numpy as np
import pytest

import huffman_decode_block_amd as hdb

pytestmark = pytest.mark.gpu

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def say(msg):
    print(f"[gpu-test] {msg}", flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "the GPU tests need a GPU"
    return t


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(v):
    """Nearest BF16 (ties to even) of 64-bit values, as 64-bit values."""
    v = np.asarray(v, dtype=np.float64)
    f = v.astype(np.float32)  # exact for what is passed here: at most 24 bits above 2^-149
    b = f.view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(bits):
    """Codes and scale bytes of BF16 bit patterns [rows, cols], from the definition."""
    rows, cols = bits.shape
    blocks = -(-cols // 32)
    full = np.zeros((rows, 32 * blocks), dtype=np.uint16)
    full[:, :cols] = bits
    full = full.reshape(rows, blocks, 32)
    v = bf16_values(full)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(-1)
    e = np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2
    e = np.where(top > 0, np.clip(e, -127, 127), -127)
    m = np.minimum(np.ldexp(np.abs(v), -e[..., None]), 6.0)
    lo = np.searchsorted(GRID, m, side="right") - 1
    hi = np.minimum(lo + 1, 7)
    mid = (GRID[lo] + GRID[hi]) / 2
    code = np.where((m > mid) | ((m == mid) & (hi % 2 == 0)), hi, lo)
    code = code + 8 * (full >> 15)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(rows, 16 * blocks, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, cols):
    rows, blocks = scales.shape
    c = np.stack([codes & 15, codes >> 4], -1).reshape(rows, blocks, 32)
    v = GRID[c & 7] * np.where(c >= 8, -1.0, 1.0)
    v = np.ldexp(v, scales.astype(np.int64)[..., None] - 127)
    v = np.where(scales[..., None] == 255, np.nan, v)
    return v.reshape(rows, 32 * blocks)[:, :cols]


def on_gpu(torch, bits, pad=0, offset=0):
    """Device BF16 matrix of the bit patterns, `pad` NaNs behind every row, the first row `offset` values into its storage."""
    rows, cols = bits.shape
    flat = torch.full((offset + rows * (cols + pad),), 0x7FC1, dtype=torch.int16, device="cuda")
    x = flat[offset:].view(rows, cols + pad)[:, :cols]
    x.copy_(torch.from_numpy(bits.view(np.int16)))
    return x.view(torch.bfloat16)


def check_quantise(torch, bits, pad=0, offset=0):
    codes, scales = hdb.df11_mx4_quantize(on_gpu(torch, bits, pad, offset))
    want_c, want_s = quantise(bits)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    got = hdb.df11_mx4_dequantize(codes, scales, bits.shape[1]).float().cpu().numpy().astype(np.float64)
    assert np.array_equal(got, to_bf16(values(want_c, want_s, bits.shape[1])), equal_nan=True)


@pytest.mark.parametrize("order", ["sorted", "shuffled", "finite shuffled"])
def test_quantise_every_bf16_pattern(torch, order):
    say(f"quantise all patterns, {order}")
    bits = np.arange(65536, dtype=np.uint16)
    if order != "sorted":
        bits = np.random.default_rng(5).permutation(bits)
    if order == "finite shuffled":
        bits = np.where((bits & 0x7F80) == 0x7F80, 0x3F80, bits).astype(np.uint16)
    check_quantise(torch, bits.reshape(512, 128))


@pytest.mark.parametrize("rows,cols,pad,offset", [
    (1, 1, 0, 0), (1, 32, 0, 0), (3, 31, 0, 0), (5, 33, 7, 1), (2, 64, 8, 8), (7, 1000, 0, 0), (129, 257, 3, 4),
    (66, 96, 0, 1), (4, 8200, 8, 0), (1000, 1, 0, 0), (3, 40, 0, 0),
])
def test_quantise_shapes(torch, rows, cols, pad, offset):
    say(f"quantise {rows}x{cols} pad {pad} offset {offset}")
    rng = np.random.default_rng(rows * 10007 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    bits[rng.random((rows, cols)) < 0.1] = 0x8000  # minus zero
    if rows > 4:
        bits[2] = 0
        bits[3, cols // 2] = 0x7F80
        bits[4, 0] = 0xFFC0
    check_quantise(torch, bits, pad, offset)


def test_values_of_every_code_and_scale(torch):
    say("dequantise every code and scale")
    codes = np.tile((np.arange(16) | (np.arange(16)[::-1] << 4)).astype(np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    got = hdb.df11_mx4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32)
    want = to_bf16(np.where(np.isnan(values(codes, scales, 32)), np.nan,
                            np.clip(values(codes, scales, 32), -3.5e38, 3.5e38)))
    big = np.abs(values(codes, scales, 32)) > 3.3961775292304e38  # past BF16's largest: an infinity
    want = np.where(big, np.sign(values(codes, scales, 32)) * np.inf, want)
    assert np.array_equal(got.float().cpu().numpy().astype(np.float64), want, equal_nan=True)


def test_dequantise_into_strided_rows(torch):
    rng = np.random.default_rng(3)
    for cols, pad, offset in ((70, 3, 1), (64, 8, 8), (33, 0, 0)):
        say(f"dequantise into rows of {cols}, pad {pad}")
        codes = rng.integers(0, 256, (9, 16 * -(-cols // 32))).astype(np.uint8)
        scales = rng.integers(100, 140, (9, -(-cols // 32))).astype(np.uint8)
        flat = torch.full((offset + 9 * (cols + pad),), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[offset:].view(9, cols + pad)
        hdb.df11_mx4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), cols, out=out[:, :cols])
        assert np.array_equal(out[:, :cols].float().cpu().numpy(), values(codes, scales, cols))
        assert bool((out[:, cols:] == 7).all()) and bool((flat[:offset] == 7).all())


def product_inputs(torch, m, n, k, pad=0, offset=0, seed=0):
    rng = np.random.default_rng([m, n, k, seed])
    x = rng.standard_normal((m, k)) * np.exp2(rng.integers(-3, 4, (m, 1)))
    xb = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    blocks = -(-k // 32)
    codes = rng.integers(0, 256, (n, 16 * blocks)).astype(np.uint8)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(n, 32 * blocks)
    nib[:, k:] = 0  # as the quantiser leaves what lies past k
    nib = nib.reshape(n, 16 * blocks, 2)
    codes = (nib[..., 0] | (nib[..., 1] << 4)).astype(np.uint8)
    scales = rng.integers(110, 130, (n, blocks)).astype(np.uint8)
    return xb, codes, scales, on_gpu(torch, xb, pad, offset), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()


def product_bound(xb, codes, scales):
    x, w = bf16_values(xb), values(codes, scales, xb.shape[1])
    ref = x @ w.T
    return ref, 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * xb.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


SHAPES = [
    (1, 1, 1), (1, 16, 32), (1, 4096, 4096), (2, 17, 31), (3, 100, 33), (15, 64, 100), (16, 130, 128), (17, 129, 96),
    (31, 33, 1000), (33, 257, 512), (64, 64, 64), (65, 1000, 160), (77, 257, 199), (128, 128, 128), (129, 130, 320),
    (200, 72, 2048), (256, 256, 256), (257, 511, 65), (300, 1024, 1024), (513, 260, 288), (1, 300, 14336),
    (1024, 512, 544), (2, 128300, 64), (5, 8, 8192), (48, 2048, 4096), (700, 640, 32),
    (1500, 1500, 512), (1400, 1600, 200), (2100, 2111, 96), (16, 8200, 512), (32, 5200, 1024), (40, 10300, 160), (129, 8193, 64),
]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_against_64_bits(torch, m, n, k):
    say(f"product {m}x{n}x{k}")
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k)
    ref, bound = product_bound(xb, codes, scales)
    y = hdb.df11_mx4_matmul(x, c, s)
    assert (np.abs(y.float().cpu().numpy() - ref) <= bound).all()
    assert torch.equal(y, hdb.df11_mx4_matmul(x, c, s)), "a second call differs"


# One for each way a product is taken: pieces of 16 x 32, 16 x 64, 32 x 32, 32 x 64, 64 x 32 and
# 64 x 64, tiles of 64 and 128 rows with one group of waves and with two; k in whole
# 512s, whole 32s, and ending inside a block.
FORMS = [
    (16, 8210, 2048), (16, 16390, 2048), (16, 16390, 160), (7, 16390, 77), (32, 5130, 2048), (30, 5130, 99), (32, 10250, 2048),
    (20, 10250, 160), (29, 10250, 45), (130, 2100, 2048), (64, 10250, 2048), (100, 5200, 333), (1100, 5000, 512), (1100, 5000, 96),
    (1024, 4096, 1536), (900, 4100, 1056), (2048, 4100, 512), (2050, 4100, 160), (2048, 4096, 1024), (2040, 4090, 544),
    (2048, 4096, 70), (16, 8192, 11008),
]


@pytest.mark.parametrize("m,n,k", FORMS)
def test_product_in_every_form(torch, m, n, k):
    """The same bound, with the 64-bit sums taken on the GPU."""
    say(f"product {m}x{n}x{k}")
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k)
    xd = torch.from_numpy(bf16_values(xb)).cuda()
    wd = torch.from_numpy(values(codes, scales, k)).cuda().T.contiguous()
    ref, total = xd @ wd, xd.abs() @ wd.abs()
    bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * k * 2.0 ** -23 * total
    y = hdb.df11_mx4_matmul(x, c, s)
    assert bool(((y.double() - ref).abs() <= bound).all())
    assert torch.equal(y, hdb.df11_mx4_matmul(x, c, s)), "a second call differs"


TILES = [
    (100, 5200, 1100), (100, 8192, 2048), (100, 8100, 1999), (64, 10250, 2112), (40, 16390, 2048), (640, 2048, 512), (333, 2050, 333),
    (900, 2100, 96), (1030, 4090, 512), (1100, 3000, 1056), (130, 16380, 45), (512, 14336, 512), (512, 14300, 96), (520, 14300, 96),
    (520, 14336, 1024), (320, 4096, 4096), (45, 16300, 32),
]


@pytest.mark.parametrize("m,n,k", TILES)
def test_product_in_every_tile(torch, m, n, k):
    test_product_in_every_form(torch, m, n, k)


@pytest.mark.parametrize("m,n,k,pad,offset", [(100, 6200, 333, 3, 1), (500, 4100, 96, 1, 0), (450, 14200, 70, 8, 2), (330, 4097, 512, 5, 8)])
def test_tiles_of_strided_rows(torch, m, n, k, pad, offset):
    test_product_of_strided_rows(torch, m, n, k, pad, offset)


@pytest.mark.parametrize("m,n,k,pad,offset", [
    (1, 96, 128, 0, 1), (4, 96, 128, 8, 8), (19, 50, 256, 3, 2), (90, 200, 96, 5, 0), (150, 129, 100, 0, 4), (260, 140, 64, 8, 3),
    (1500, 1500, 70, 1, 0), (1600, 1411, 64, 0, 1), (70, 3000, 515, 0, 0),
])
def test_product_of_strided_rows(torch, m, n, k, pad, offset):
    """What lies between the rows of x is NaN; the rows of y are strided too."""
    say(f"product {m}x{n}x{k} pad {pad} offset {offset}")
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k, pad, offset)
    ref, bound = product_bound(xb, codes, scales)
    flat = torch.full((m, n + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    y = hdb.df11_mx4_matmul(x, c, s, out=flat[:, 2:2 + n])
    assert (np.abs(y.float().cpu().numpy() - ref) <= bound).all()
    assert bool((flat[:, :2] == 9).all()) and bool((flat[:, 2 + n:] == 9).all())


@pytest.mark.parametrize("m", [1, 20, 300])
def test_product_keeps_nan_and_infinity_in_their_rows(torch, m):
    say(f"product with NaN, {m} rows")
    n, k = 150, 320
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k)
    scales[7, 3] = 255
    s[7, 3] = 255
    if m > 2:
        xb[1, 5], xb[2, 9] = 0x7FC0, 0x7F80
        x[1, 5], x[2, 9] = float("nan"), float("inf")
        codes[:, 4] |= 0x60  # column 9 of no row is zero
        c |= 0
        c[:, 4] |= 0x60
    with np.errstate(invalid="ignore"):
        ref, bound = product_bound(xb, codes, scales)
    got = hdb.df11_mx4_matmul(x, c, s).float().cpu().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    assert (np.abs(got - ref)[fine] <= bound[fine]).all()


def test_empty_products(torch):
    say("empty products")
    _, _, _, x, c, s = product_inputs(torch, 3, 40, 64)
    assert hdb.df11_mx4_matmul(x[:0], c, s).shape == (0, 40)
    assert hdb.df11_mx4_matmul(x, c[:0], s[:0]).shape == (3, 0)
    y = hdb.df11_mx4_matmul(x[:, :0], c[:, :0].contiguous(), s[:, :0].contiguous())
    assert y.shape == (3, 40) and bool((y == 0).all())
    codes, scales = hdb.df11_mx4_quantize(x[:0])
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert hdb.df11_mx4_dequantize(codes, scales, 64).shape == (0, 64)


@pytest.mark.parametrize("m,k", [(2, 512), (90, 333), (400, 512)])
def test_product_on_another_stream_and_in_a_graph(torch, m, k):
    say(f"product {m} rows on a side stream and in a graph")
    xb, codes, scales, x, c, s = product_inputs(torch, m, 500, k)
    want = hdb.df11_mx4_matmul(x, c, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = hdb.df11_mx4_matmul(x, c, s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    got = hdb.df11_mx4_matmul(x, c, s, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hdb.df11_mx4_matmul(x, c, s, out=out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, hdb.df11_mx4_matmul(x, c, s))


def test_refusals(torch):
    say("refusals")
    _, _, _, x, c, s = product_inputs(torch, 3, 40, 64)
    with pytest.raises(TypeError):
        hdb.df11_mx4_matmul(x.float(), c, s)
    with pytest.raises(TypeError):
        hdb.df11_mx4_matmul(x.cpu(), c, s)
    with pytest.raises(ValueError):
        hdb.df11_mx4_matmul(x[:, :32], c, s)
    with pytest.raises(ValueError):
        hdb.df11_mx4_matmul(x.T, c, s)
    with pytest.raises(ValueError):
        hdb.df11_mx4_matmul(x, c, s[:-1])
    with pytest.raises(ValueError):
        hdb.df11_mx4_matmul(x, c, s, out=torch.empty(3, 41, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        hdb.df11_mx4_quantize(x[:, :0])
    with pytest.raises(ValueError):
        hdb.df11_mx4_dequantize(c, s, 65)
    wide = torch.zeros(2048, 65, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_mx4_matmul(wide, *hdb.df11_mx4_quantize(wide), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == hdb.DF11_E_BUFFER_TOO_SMALL


def test_derivatives_are_refused(torch):
    """The product loses no gradient and no tangent silently; codes are whole numbers and have none to lose."""
    say("derivatives")
    from torch.autograd import forward_ad
    _, _, _, x, c, s = product_inputs(torch, 3, 40, 64)
    want = hdb.df11_mx4_matmul(x, c, s)
    wants = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        hdb.df11_mx4_matmul(wants, c, s)
    with pytest.raises(ValueError, match="no backward"):
        hdb.df11_mx4_matmul(wants * 2, c, s)
    with pytest.raises(ValueError, match="no backward"):
        hdb.df11_mx4_matmul(x, c, s, out=torch.empty_like(want).requires_grad_())
    with torch.no_grad():
        assert torch.equal(hdb.df11_mx4_matmul(wants, c, s), want)
    assert torch.equal(hdb.df11_mx4_matmul(wants.detach(), c, s), want)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="no derivative"):
            hdb.df11_mx4_matmul(forward_ad.make_dual(x, torch.ones_like(x)), c, s)
    for got, ref in zip(hdb.df11_mx4_quantize(wants), hdb.df11_mx4_quantize(x)):
        assert torch.equal(got, ref)


# A product in each way that it is taken: the token form with scales in one load, by the byte, and with x through
# registers; tiles of 64 x 128 with two groups of waves and with one, of an x that is copied first, of 64 x 256, and
# of 128 x 256 with two groups and with one.
EVERY_WAY = [
    (1, 300, 4096), (4, 130, 320), (20, 200, 96), (64, 520, 2048), (33, 150, 333),
    (640, 2048, 512), (1100, 5000, 96), (333, 2050, 333), (1600, 4096, 512), (2048, 4096, 1536), (2100, 5000, 160),
    (1600, 4096, 4608), (1610, 4090, 1568), (2100, 6200, 160), (3200, 4096, 512),
]


@pytest.mark.parametrize("m,n,k", EVERY_WAY)
def test_product_of_quantised_nan_and_infinity(torch, m, n, k):
    """A weight that is NaN or infinite makes its block NaN, and so its column of the product, for x of zeros too;
    the other columns are those of the matrix without it."""
    say(f"product {m}x{n}x{k} of quantised NaN and infinities")
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
    x[m // 2] = 0
    w = torch.randn(n, k, generator=g, device="cuda").to(torch.bfloat16)
    clean = hdb.df11_mx4_matmul(x, *hdb.df11_mx4_quantize(w))
    at = [(0, 0), (5, k - 1), (n // 2, k // 2), (n - 1, k - 1), (17, 31)]
    for i, (row, col) in enumerate(at):
        w[row, col] = float("nan") if i % 2 else float("-inf")
    codes, scales = hdb.df11_mx4_quantize(w)
    for row, col in at:
        assert int(scales[row, col // 32]) == 255 and bool((codes[row, col // 32 * 16:col // 32 * 16 + 16] == 0).all())
    y = hdb.df11_mx4_matmul(x, codes, scales)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[row for row, _ in at]] = True
    assert bool(y[:, bad].isnan().all())
    assert torch.equal(y[:, ~bad], clean[:, ~bad])


def sums_on_gpu(torch, xb, codes, scales, k):
    """(64-bit products, bound) of bit patterns and codes, taken on the GPU."""
    xd = torch.from_numpy(bf16_values(xb)).cuda()
    wd = torch.from_numpy(values(codes, scales, k)).cuda().T.contiguous()
    ref = xd @ wd
    return ref, 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * k * 2.0 ** -23 * (xd.abs() @ wd.abs())


@pytest.mark.parametrize("m,n,k", EVERY_WAY)
def test_product_of_nan_and_infinity_in_x(torch, m, n, k):
    """NaN and infinities in x, of one sign and of both, stay in their rows."""
    say(f"product {m}x{n}x{k} with NaN and infinities in x")
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k)
    cols = (0, k // 2, k - 1)
    for col in cols:  # of no row of w zero
        codes[:, col // 2] |= 0x66
    if k % 2:
        codes[:, (k - 1) // 2] &= 0x0F
    c.copy_(torch.from_numpy(codes))
    rows = {0: ((0, 0x7FC0),), m // 3: ((k // 2, 0x7F80),), m // 2: ((k - 1, 0xFF80),), m - 1: ((0, 0x7F80), (k - 1, 0x7F80))}
    for row, bits in rows.items():
        for col, b in bits:
            xb[row, col] = b
    x.copy_(torch.from_numpy(xb.view(np.int16)).view(torch.bfloat16))
    ref, bound = sums_on_gpu(torch, xb, codes, scales, k)
    got = hdb.df11_mx4_matmul(x, c, s).double()
    fine = ref.isfinite()
    assert int((~fine).sum()) == n * len(rows) and bool(ref.isinf().any())
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got[ref.isinf()], ref[ref.isinf()])
    assert bool(((got - ref).abs()[fine] <= bound[fine]).all())


@pytest.mark.parametrize("m,n,k", EVERY_WAY)
def test_product_of_denormals(torch, m, n, k):
    """BF16 denormals count: in x (times large weights) and as what small weights expand to (times large x)."""
    say(f"product {m}x{n}x{k} of denormals")
    rng = np.random.default_rng([m, n, k])
    xb, codes, _, _, c, _ = product_inputs(torch, m, n, k)
    for tiny_x in (True, False):
        bits = rng.integers(1, 128, (m, k)).astype(np.uint16) if tiny_x else (xb & 0x807F | (rng.integers(240, 250, (m, k)) << 7)).astype(np.uint16)
        bits[rng.random((m, k)) < 0.5] ^= 0x8000
        sc = rng.integers(230, 240, (n, -(-k // 32))) if tiny_x else rng.integers(0, 3, (n, -(-k // 32)))
        sc = sc.astype(np.uint8)
        ref, bound = sums_on_gpu(torch, bits, codes, sc, k)
        assert float(ref.abs().max()) > 2.0 ** -40
        got = hdb.df11_mx4_matmul(on_gpu(torch, bits), c, torch.from_numpy(sc).cuda()).double()
        assert bool(((got - ref).abs() <= bound).all())


@pytest.mark.parametrize("m,n,k", [(640, 2048, 512), (333, 2050, 333), (1600, 4096, 96), (2048, 4096, 512)])
def test_tiles_on_another_stream_and_in_a_graph(torch, m, n, k):
    """Also where x is copied in front of the product (333 columns): two launches, with a workspace between them."""
    say(f"tiles {m}x{n}x{k} on a side stream and in a graph")
    xb, codes, scales, x, c, s = product_inputs(torch, m, n, k)
    want = hdb.df11_mx4_matmul(x, c, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = hdb.df11_mx4_matmul(x, c, s, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hdb.df11_mx4_matmul(x, c, s, out=out)
    for _ in range(4):
        x.mul_(-0.5)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, hdb.df11_mx4_matmul(x, c, s))


@pytest.mark.parametrize("m,n,k", [
    (2100, 6200, 160), (3137, 4100, 544), (4096, 4096, 512), (2049, 6145, 70), (1300, 10250, 1030), (1290, 10250, 2048),  # one group
    (1600, 4096, 4608), (2040, 4090, 5120), (1610, 4090, 1568), (820, 8190, 1999),                                          # two
    (2100, 4100, 8224),  # one, for a long k
])
def test_product_in_tiles_of_128_rows(torch, m, n, k):
    test_product_in_every_form(torch, m, n, k)
