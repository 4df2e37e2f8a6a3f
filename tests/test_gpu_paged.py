"""GPU checks of the paged key-value cache: what the append writes (exact) and
the attention of one token against 64 bits.

Bounds, for scores s = scale q . k computed in 32 bits from exact products:
each is off by at most e = (head_dim + 4) 2^-23 scale max_j sum |q| |k_j| plus
2^-22 max |s| (the scale, log2 e and the difference from the maximum, rounded);
a weight is off by a factor of at most 1 + 2 e + 2^-16 (its two BF16 parts, the
exponential) and a sum of L terms by L 2^-23 more.  So
  |out - ref| <= 2^-8 |ref| + (4 e + 2^-14 + L 2^-22) sum w |v| / sum w
  |lse - ref| <= 2 e + 2^-14 / 8 + L 2^-22 + 2^-22 |ref|
"""
import math

import numpy as np
import pytest

import huffman_decode_block_amd as hdb

pytestmark = pytest.mark.gpu


def say(msg):
    print(f"[gpu-test] {msg}", flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "the GPU tests need a GPU"
    return t


def make_pages(torch, n, heads, page, dim, dtype, layout, fill):
    """Pages [n, heads, page, dim] in one of three layouts."""
    if layout == "positions first":
        return torch.full((n, page, heads, dim), fill, device="cuda").to(dtype).transpose(1, 2)
    if layout == "joint":  # keys and values of a page next to each other
        return torch.full((n, 2, heads, page, dim), fill, device="cuda").to(dtype)[:, 0]
    return torch.full((n, heads, page, dim), fill, device="cuda").to(dtype)


def e4m3(torch, x, scale):
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


LAYOUTS = ["heads first", "positions first", "joint"]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,page,layout,source", [
    (1, 1, 64, 8, 0, "dense"), (5, 3, 128, 16, 1, "joint"), (33, 8, 128, 64, 2, "odd"), (7, 2, 256, 1024, 0, "joint"),
    (300, 4, 64, 32, 1, "odd"), (64, 1, 256, 16, 2, "dense"),
])
def test_append(torch, fp8, tokens, heads, dim, page, layout, source):
    layout = LAYOUTS[layout]
    say(f"append {tokens} tokens {heads}x{dim} page {page} {layout} {source} fp8={fp8}")
    g = torch.Generator(device="cuda").manual_seed(tokens)
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    n = -(-tokens // page) + 3
    kp = make_pages(torch, n, heads, page, dim, dtype, layout, 1.0)
    vp = make_pages(torch, n, heads, page, dim, dtype, layout, 2.0)
    if source == "odd":  # rows that start off 16 bytes
        flat = torch.randn(tokens * (2 * heads * dim + 3) + 1, generator=g, device="cuda").to(torch.bfloat16)[1:]
        kv = flat.view(tokens, 2 * heads * dim + 3)
        k, v = kv[:, 1:1 + heads * dim].view(tokens, heads, dim), kv[:, 2 + heads * dim:2 + 2 * heads * dim].view(tokens, heads, dim)
    else:
        kv = torch.randn(tokens, 2 * heads, dim, generator=g, device="cuda").to(torch.bfloat16)
        k, v = kv[:, :heads], kv[:, heads:]
        if source == "dense":
            k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(n * page, generator=g, device="cuda")[:tokens]
    if tokens > 4:
        slots[1], slots[2], slots[3] = -1, n * page, 1 << 40
    ks = vs = None
    if fp8:
        ks = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.001
        vs = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.001
    want = []
    for p, x, sc in ((kp, k, ks), (vp, v, vs)):
        w = p.float().cpu().numpy()
        new = e4m3(torch, x, sc.view(1, -1, 1)).float() if fp8 else x.float()
        new = new.cpu().numpy()
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < n * page:
                w[slot // page, :, slot % page] = new[t]
        want.append(w)
    hdb.df11_paged_append(k, v, slots, kp, vp, ks, vs)
    assert np.array_equal(kp.float().cpu().numpy(), want[0])
    assert np.array_equal(vp.float().cpu().numpy(), want[1])


@pytest.mark.parametrize("scale", [1.0, 0.37, 3e-5])
def test_append_every_bf16_pattern_to_e4m3(torch, scale):
    say(f"append every pattern, scale {scale}")
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    kp = torch.zeros(32, 1, 16, 128, device="cuda").to(torch.float8_e4m3fn)
    vp = torch.zeros_like(kp)
    s = torch.full((1,), scale, device="cuda")
    hdb.df11_paged_append(x, x, torch.arange(512, device="cuda"), kp, vp, s, s)
    # the definition on the host: nearest of E4M3's values, held to 448
    v = (x.float() / s).cpu().numpy().reshape(-1).astype(np.float64)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(v), 448)
        e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6)
        want = np.copysign(np.ldexp(np.rint(np.ldexp(a, 3 - e)), e - 3), v)
    for p in (kp, vp):
        assert np.array_equal(p.float().cpu().numpy().reshape(-1), np.where(np.isnan(v), np.nan, want), equal_nan=True)


def reference(torch, q, kp, vp, table, lens, starts, scale, ks, vs):
    """(out, lse, bound of out, bound of lse) in 64 bits on the host."""
    q = q.double().cpu().numpy()
    k, v = kp.float().double().cpu().numpy(), vp.float().double().cpu().numpy()
    n, heads, page, dim = k.shape
    if ks is not None:
        k = k * ks.double().cpu().numpy().reshape(1, -1, 1, 1)
        v = v * vs.double().cpu().numpy().reshape(1, -1, 1, 1)
    table = table.cpu().numpy()
    batch, q_heads, _ = q.shape
    group = q_heads // heads
    out, lse = np.zeros(q.shape), np.full((batch, q_heads), -np.inf)
    out_b, lse_b = np.zeros(q.shape), np.zeros((batch, q_heads))
    for b in range(batch):
        hi = min(max(int(lens[b]), 0), table.shape[1] * page)
        lo = 0 if starts is None else max(int(starts[b]), 0)
        at = np.arange(lo, max(lo, hi))
        pg = table[b][at // page]
        at, pg = at[(pg >= 0) & (pg < n)], pg[(pg >= 0) & (pg < n)]
        if at.size == 0:
            continue
        for h in range(heads):
            kk, vv = k[pg, h, at % page], v[pg, h, at % page]
            for g in range(h * group, (h + 1) * group):
                s = scale * (kk @ q[b, g])
                mag = abs(scale) * (np.abs(kk) @ np.abs(q[b, g])).max()
                e = (dim + 4) * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(s).max()
                top = s.max()
                w = np.exp(s - top)
                lse[b, g] = top + math.log(w.sum())
                w /= w.sum()
                out[b, g] = w @ vv
                out_b[b, g] = 2.0 ** -8 * np.abs(out[b, g]) + (4 * e + 2.0 ** -14 + at.size * 2.0 ** -22) * (w @ np.abs(vv))
                lse_b[b, g] = 2 * e + 2.0 ** -17 + at.size * 2.0 ** -22 + 2.0 ** -22 * abs(lse[b, g])
    return out, lse, out_b, lse_b


def build(torch, lens, heads, group, dim, page, fp8, layout="heads first", extra=2, spread=1.0, seed=1):
    """A cache whose unused positions hold NaN, and a query for each sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, width = len(lens), max(1, -(-max(lens) // page)) + 1
    n = batch * width + extra
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kp = make_pages(torch, n, heads, page, dim, dtype, layout, float("nan"))
    vp = make_pages(torch, n, heads, page, dim, dtype, layout, float("nan"))
    table = torch.randperm(n, generator=g, device="cuda")[:batch * width].int().view(batch, width)
    ks = vs = None
    if fp8:
        ks = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.005
        vs = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.005
    total = sum(lens)
    if total:
        k = (torch.randn(total, heads, dim, generator=g, device="cuda") * spread).to(torch.bfloat16)
        v = torch.randn(total, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
        slots = torch.cat([table[b].long().repeat_interleave(page)[:m] * page + torch.arange(m, device="cuda") % page
                           for b, m in enumerate(lens)])
        hdb.df11_paged_append(k, v, slots, kp, vp, ks, vs)
    q = torch.randn(batch, heads * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    return q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), ks, vs


def check(torch, q, kp, vp, table, lens, starts, ks, vs, scale=None, **more):
    out, lse = hdb.df11_paged_attention(q, kp, vp, table, lens, starts=starts, scale=scale, k_scale=ks, v_scale=vs, **more)
    ref, ref_lse, bound, lse_bound = reference(
        torch, q, kp, vp, table, lens.tolist(), None if starts is None else starts.tolist(),
        q.shape[-1] ** -0.5 if scale is None else scale, ks, vs)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - ref) <= bound).all(), float((np.abs(o - ref) - bound).max())
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(l), empty)
    assert (np.abs(l - ref_lse)[~empty] <= lse_bound[~empty]).all()
    again, again_lse = hdb.df11_paged_attention(q, kp, vp, table, lens, starts=starts, scale=scale, k_scale=ks, v_scale=vs, **more)
    assert torch.equal(out, again) and torch.equal(lse, again_lse), "a second call differs"
    return out, lse


EDGE_LENS = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 65, 100, 127, 128, 255, 256, 257, 300]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,group,layout", [(8, 1, 0), (16, 4, 1), (64, 7, 2), (1024, 16, 0)])
def test_attention_lengths(torch, fp8, dim, page, group, layout):
    say(f"attention dim {dim} page {page} group {group} {LAYOUTS[layout]} fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, EDGE_LENS, 2, group, dim, page, fp8, LAYOUTS[layout])
    check(torch, q, kp, vp, table, lens, None, ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,group", [(1, 2), (3, 3), (1, 17), (2, 32), (1, 40), (8, 1)])
def test_attention_head_layouts(torch, fp8, heads, group):
    say(f"attention {heads} heads group {group} fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, [0, 5, 70, 513], heads, group, 128, 16, fp8)
    check(torch, q, kp, vp, table, lens, None, ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("length,page,dim", [(1024, 16, 128), (1025, 64, 64), (2000, 32, 256), (5003, 128, 128)])
def test_attention_long(torch, fp8, length, page, dim):
    say(f"attention length {length} page {page} dim {dim} fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, [length, 3, length // 2], 2, 4, dim, page, fp8)
    check(torch, q, kp, vp, table, lens, None, ks, vs)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_starts(torch, dim):
    """Windows: starts inside and at the edges of steps and pages, past the length, negative; lengths past the table."""
    say(f"attention starts, dim {dim}")
    lens = [300, 300, 300, 300, 300, 300, 300, 300, 40, 2, 300]
    starts = [0, 1, 16, 31, 32, 33, 255, 299, 40, 5, -7]
    q, kp, vp, table, ln, ks, vs = build(torch, lens, 2, 3, dim, 16, False)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    check(torch, q, kp, vp, table, ln, st, ks, vs)
    narrow = table[:, :4].clone()
    check(torch, q, kp, vp, narrow, ln, st, ks, vs)
    check(torch, q, kp, vp, table, torch.full_like(ln, -3), st, ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_masked_pages(torch, fp8):
    """Table entries outside the cache mask their positions, up to all of a sequence."""
    say(f"attention masked pages fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, [200, 200, 200, 50], 2, 4, 128, 16, fp8)
    table[0, 3], table[0, 12], table[1, 0] = -1, kp.shape[0], 1 << 30
    table[2] = -5
    out, lse = check(torch, q, kp, vp, table, lens, None, ks, vs)
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())


def test_attention_large_and_small_scores(torch):
    """Scores of thousands: the running maximum carries them; weights that vanish against it are zeros."""
    say("attention large scores")
    q, kp, vp, table, lens, ks, vs = build(torch, [1, 40, 700, 1300], 2, 4, 128, 16, False, spread=300.0)
    check(torch, q, kp, vp, table, lens, None, ks, vs)
    check(torch, q, kp, vp, table, lens, None, ks, vs, scale=-0.01)
    check(torch, q, kp, vp, table, lens, None, ks, vs, scale=0.0)


def test_attention_nan_and_infinity_stay_in_their_sequence(torch):
    say("attention NaN")
    q, kp, vp, table, lens, ks, vs = build(torch, [100, 100, 100], 1, 4, 128, 16, False)
    want, want_lse = hdb.df11_paged_attention(q, kp, vp, table, lens)
    q = q.clone()
    q[1, 2] = float("nan")
    vp[int(table[2, 1]), 0, 3, 5] = float("nan")
    out, lse = hdb.df11_paged_attention(q, kp, vp, table, lens)
    assert bool(out[1, 2].isnan().all()) and bool(lse[1, 2].isnan())
    assert bool(out[2, :, 5].isnan().all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, 2], keep[2, :, 5] = False, False
    assert torch.equal(out[keep], want[keep])
    assert torch.equal(lse[2], want_lse[2])


def test_attention_strided_query_and_table(torch):
    say("attention strided query and table")
    q, kp, vp, table, lens, ks, vs = build(torch, [90, 33, 0], 2, 2, 128, 16, False)
    joint = torch.full((3, 9, 131), float("nan"), dtype=torch.bfloat16, device="cuda")
    joint[:, 1:5, 1:129] = q
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    want = hdb.df11_paged_attention(q, kp, vp, table, lens)
    got = hdb.df11_paged_attention(joint[:, 1:5, 1:129], kp, vp, wide[:, :table.shape[1]], lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = hdb.df11_paged_attention(q, kp, vp, wide, lens)
    check(torch, q, kp, vp, wide, lens, None, ks, vs)
    assert torch.equal(torch.isneginf(got[1]), torch.isneginf(want[1]))


def test_attention_past_4_gib(torch):
    """Pages whose offsets pass 32 bits, read through a table that jumps over all of the cache."""
    say("attention over 6 GiB of pages")
    page, heads, dim = 64, 8, 128
    n = (6 << 30) // (page * heads * dim * 2) // 2
    kp = torch.zeros(2 * n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros(2 * n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    small_k = torch.randn(6, heads, page, dim, device="cuda").to(torch.bfloat16)
    small_v = torch.randn(6, heads, page, dim, device="cuda").to(torch.bfloat16)
    at = torch.tensor([0, 2 * n - 1, n // 3, n, 2 * n - 7, 1], device="cuda")
    kp[at], vp[at] = small_k, small_v
    q = torch.randn(1, 32, dim, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([6 * page - 5], dtype=torch.int32, device="cuda")
    want = hdb.df11_paged_attention(q, small_k, small_v, torch.arange(6, device="cuda").int().view(1, 6), lens)
    got = hdb.df11_paged_attention(q, kp, vp, at.int().view(1, 6), lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    new = torch.randn(1, heads, dim, device="cuda").to(torch.bfloat16)
    hdb.df11_paged_append(new, new, torch.tensor([(2 * n - 1) * page + 63], device="cuda"), kp, vp)
    assert torch.equal(kp[2 * n - 1, :, 63], new[0]) and torch.equal(vp[2 * n - 1, :, 63], new[0])
    assert torch.equal(kp[2 * n - 1, :, :63], small_k[1, :, :63])


@pytest.mark.parametrize("length", [60, 3000])
def test_attention_on_another_stream_and_in_a_graph(torch, length):
    say(f"attention on a side stream and in a graph, length {length}")
    q, kp, vp, table, lens, ks, vs = build(torch, [length, 10], 2, 4, 128, 16, False)
    want = hdb.df11_paged_attention(q, kp, vp, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = hdb.df11_paged_attention(q, kp, vp, table, lens, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hdb.df11_paged_attention(q, kp, vp, table, lens, out=out, lse=lse)
    for step in range(4):  # the lengths are read on the device: a replay takes the new ones
        lens[:1].fill_(length - 7 * step)
        q.mul_(-1)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = hdb.df11_paged_attention(q, kp, vp, table, lens)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_refusals(torch):
    say("refusals")
    q, kp, vp, table, lens, ks, vs = build(torch, [20, 3], 2, 2, 128, 16, False)
    with pytest.raises(TypeError):
        hdb.df11_paged_attention(q.float(), kp, vp, table, lens)
    with pytest.raises(TypeError):
        hdb.df11_paged_attention(q, kp, vp, table.long(), lens)
    with pytest.raises(TypeError):
        hdb.df11_paged_attention(q, kp.half(), vp.half(), table, lens)
    with pytest.raises(ValueError):
        hdb.df11_paged_attention(q[:, :3], kp, vp, table, lens)
    with pytest.raises(ValueError):
        hdb.df11_paged_attention(q, kp, vp, table[:1], lens)
    with pytest.raises(ValueError):
        hdb.df11_paged_attention(q, kp, vp, table, lens, k_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        hdb.df11_paged_attention(q, kp.to(torch.float8_e4m3fn), vp.to(torch.float8_e4m3fn), table, lens)
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_paged_attention(q[..., :32], kp[..., :32], vp[..., :32], table, lens)
    assert e.value.status == hdb.DF11_E_UNSUPPORTED
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_paged_attention(q, kp[:, :, :12], vp[:, :, :12], table, lens)
    assert e.value.status == hdb.DF11_E_UNSUPPORTED
    with pytest.raises(ValueError):
        hdb.df11_paged_append(q[:1], q, torch.zeros(2, dtype=torch.int64, device="cuda"), kp, vp)
    with pytest.raises(TypeError):
        hdb.df11_paged_append(q[:, :2], q[:, :2], torch.zeros(2, dtype=torch.int32, device="cuda"), kp, vp)
    assert hdb.df11_paged_attention(q[:0], kp, vp, table[:0], lens[:0])[0].shape == (0, 4, 128)
    hdb.df11_paged_append(q[:0, :2], q[:0, :2], torch.zeros(0, dtype=torch.int64, device="cuda"), kp, vp)


def ragged(batch, most, seed):
    """Lengths with the ends of chunks, steps and classes among them, and sequences of the same length."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, most + 1, batch)
    edges = [0, most, 1, most - 1, 127, 128, 129, 0, most // 2, most // 2, 33, 31]
    lens[g.permutation(batch)[:min(batch, len(edges))]] = edges[:batch]
    return lens.tolist()


# more heads than compute units and one chunk: the longest sequences first
BY_LENGTH = [(33, 8, 1, 64, 16, 520), (64, 5, 3, 128, 32, 1000), (65, 4, 1, 256, 16, 700), (130, 2, 17, 64, 64, 900),
             (256, 2, 1, 64, 16, 1100), (257, 1, 1, 64, 16, 1100), (200, 2, 2, 128, 16, 600)]
# chunks of one length for all sequences
EVENLY = [(16, 8, 2, 64, 16, 4100), (2, 4, 3, 64, 16, 65530), (70, 2, 1, 64, 64, 4200), (9, 16, 17, 64, 32, 4095),
          (17, 8, 1, 128, 128, 4090), (11, 4, 33, 256, 16, 4090), (5, 8, 1, 128, 128, 8300)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch,heads,group,dim,page,most", BY_LENGTH + EVENLY)
def test_attention_ragged(torch, fp8, batch, heads, group, dim, page, most):
    say(f"attention {batch} ragged of {most} {heads}x{group} dim {dim} page {page} fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, ragged(batch, most, most), heads, group, dim, page, fp8)
    check(torch, q, kp, vp, table, lens, None, ks, vs)


@pytest.mark.parametrize("batch,heads,group,dim,page,most", BY_LENGTH[:1] + BY_LENGTH[3:4] + EVENLY[:2])
def test_attention_ragged_starts_masks_and_lengths(torch, batch, heads, group, dim, page, most):
    """Windows, masked pages, equal lengths, one sequence that holds all, none that holds any, one past the table."""
    say(f"attention {batch} of {most} {heads}x{group} dim {dim} page {page}: starts, masks, lengths")
    q, kp, vp, table, lens, ks, vs = build(torch, [most] * batch, heads, group, dim, page, False)
    check(torch, q, kp, vp, table, lens, None, ks, vs)
    starts = torch.tensor(ragged(batch, most, 3), dtype=torch.int32, device="cuda")
    check(torch, q, kp, vp, table, lens, starts, ks, vs)
    table = table.clone()
    table[0] = -1
    table[1, 3], table[1, 7] = -1, kp.shape[0]
    one = torch.zeros_like(lens)
    one[batch - 1] = most
    for ln in (one, torch.zeros_like(lens), torch.full_like(lens, -9), torch.tensor(ragged(batch, most, 4), device="cuda").int()):
        check(torch, q, kp, vp, table, ln, starts, ks, vs)
        check(torch, q, kp, vp, table, ln, None, ks, vs)


@pytest.mark.parametrize("batch,heads,group,dim,page,most", BY_LENGTH[:1] + EVENLY[:1])
def test_attention_ragged_in_a_graph(torch, batch, heads, group, dim, page, most):
    """A replay orders and cuts the sequences by the lengths that it finds."""
    say(f"attention {batch} of {most} in a graph")
    q, kp, vp, table, lens, ks, vs = build(torch, [most] * batch, heads, group, dim, page, False)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    hdb.df11_paged_attention(q, kp, vp, table, lens, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hdb.df11_paged_attention(q, kp, vp, table, lens, out=out, lse=lse)
    for step in range(4):
        lens.copy_(torch.tensor(ragged(batch, most, step), dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = check(torch, q, kp, vp, table, lens, None, ks, vs)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_the_null_stream_by_its_handle(torch):
    """stream=0 is the null stream also where another one is current: the call follows what was put there before it."""
    say("null stream by its handle")
    q, kp, vp, table, lens, ks, vs = build(torch, [3000, 10], 2, 4, 128, 16, False)
    want = hdb.df11_paged_attention(q, kp, vp, table, lens)
    late = torch.zeros_like(q)
    a = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert torch.cuda.default_stream().cuda_stream == 0
    for _ in range(20):  # some milliseconds in front of the query
        a = (a @ a).clamp(max=1)
    late.copy_(q)
    with torch.cuda.stream(side):
        assert hdb.step._place(0, 0)[0] == 0
        got = hdb.df11_paged_attention(late, kp, vp, table, lens, stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def score(q, kp, table, b, h, g, group, length):
    """Scores of one query head over a sequence's first positions, in 64 bits."""
    page, dim = kp.shape[2], kp.shape[3]
    at = np.arange(length)
    rows = kp[table[b, at // page], h, at % page]
    return dim ** -0.5 * (rows @ q[b, h * group + g]), at


@pytest.mark.parametrize("lens,heads,group,dim,page", [
    ([100, 37, 1, 2], 2, 4, 64, 16), ([100, 37, 1, 2], 1, 17, 128, 8), ([250, 33, 5], 2, 3, 256, 64),
    ([3000, 700, 1], 2, 4, 128, 16),  # cut into chunks
    (ragged(33, 520, 1), 8, 1, 64, 16), (ragged(16, 4100, 2), 8, 2, 64, 16),  # by length; chunks of one length
])
def test_attention_infinite_values(torch, lens, heads, group, dim, page):
    """Infinities in V make a sum infinite, of both signs NaN, whatever weight they have, the largest among them."""
    say(f"attention infinite values, {len(lens)} sequences, {heads}x{group} dim {dim}")
    q, kp, vp, table, ln, ks, vs = build(torch, lens, heads, group, dim, page, False)
    clean, clean_lse = check(torch, q, kp, vp, table, ln, None, ks, vs)
    want = clean.float().cpu().numpy().reshape(len(lens), heads, group, dim)
    rng = np.random.default_rng(len(lens))
    qn, kn, tn = q.double().cpu().numpy(), kp.double().cpu().numpy(), table.cpu().numpy()
    inf = float("inf")
    for b, length in enumerate(lens):
        if length == 0:
            continue
        for h in range(heads):
            top = int(np.argmax(score(qn, kn, tn, b, h, 0, group, length)[0]))
            one, two = rng.integers(0, length, 2)
            for col, at, sign in ((3, one, 1), (7, two, -1), (13, top, 1), (20, top, -1), (11, one, 1), (11, two, 1), (9, one, 1), (9, two, -1)):
                if col == 9 and one == two:
                    continue
                vp[int(tn[b, at // page]), h, int(at) % page, col] = sign * inf
            for col, value in ((3, inf), (7, -inf), (13, inf), (20, -inf), (11, inf), (9, np.nan)):
                if col != 9 or one != two:
                    want[b, h, :, col] = value
    out, lse = hdb.df11_paged_attention(q, kp, vp, table, ln)
    assert np.array_equal(out.float().cpu().numpy().reshape(want.shape), want, equal_nan=True)
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("length", [60, 3000])
def test_attention_infinite_keys(torch, length):
    """A score of -infinity is a weight of zero; one of +infinity leaves no number."""
    say(f"attention infinite keys, length {length}")
    q, kp, vp, table, ln, ks, vs = build(torch, [length, 5], 2, 4, 64, 16, False)
    at = length // 2
    q[0, :, 5] = torch.tensor([1.0, -1.0] * 4, device="cuda")
    kp[int(table[0, at // 16]), :, at % 16, 5] = float("inf")
    kp[int(table[0, 0]), :, 3, 5] = float("inf")
    out, lse = hdb.df11_paged_attention(q, kp, vp, table, ln)
    assert bool(out[0, ::2].isnan().all())
    qn, kn, vn, tn = q.double().cpu().numpy(), kp.double().cpu().numpy(), vp.double().cpu().numpy(), table.cpu().numpy()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for head in range(1, 8, 2):
        h, g = head // 4, head % 4
        s, pos = score(qn, kn, tn, 0, h, g, 4, length)
        v = vn[tn[0, pos // 16], h, pos % 16]
        live = np.isfinite(s)
        assert live.sum() == length - 2
        k = kn[tn[0, pos // 16], h, pos % 16][live]
        e = 68 * 2.0 ** -23 / 8 * (np.abs(k) @ np.abs(qn[0, head])).max() + 2.0 ** -22 * np.abs(s[live]).max()
        w = np.exp(s[live] - s[live].max())
        ref_lse, w = s[live].max() + math.log(w.sum()), w / w.sum()
        ref = w @ v[live]
        bound = 2.0 ** -8 * np.abs(ref) + (4 * e + 2.0 ** -14 + length * 2.0 ** -22) * (w @ np.abs(v[live]))
        assert (np.abs(got[0, head] - ref) <= bound).all()
        assert abs(got_lse[0, head] - ref_lse) <= 2 * e + 2.0 ** -17 + length * 2.0 ** -22 + 2.0 ** -22 * abs(ref_lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_derivatives_are_refused(torch, fp8):
    """No call loses a gradient or a tangent silently: not of q, k, v, pages, scales or outputs."""
    say(f"derivatives fp8={fp8}")
    from torch.autograd import forward_ad
    q, kp, vp, table, lens, ks, vs = build(torch, [20, 3], 2, 2, 128, 16, fp8)
    want = hdb.df11_paged_attention(q, kp, vp, table, lens, k_scale=ks, v_scale=vs)
    k, slots = torch.randn(2, 2, 128, device="cuda").to(torch.bfloat16), table[:, -1].long() * 16  # past the lengths
    a = dict(q=q, k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, out=torch.empty_like(q), lse=torch.empty_like(want[1]))
    w = dict(k=k, v=k, k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs)
    held = kp.clone()

    def attend(**more):
        return hdb.df11_paged_attention(page_table=table, lens=lens, **{**a, **more})

    def append(**more):
        hdb.df11_paged_append(slots=slots, **{**w, **more})

    for call, given in ((attend, a), (append, w)):
        for name, t in given.items():
            if t is None:
                continue
            wants = t.detach().clone().requires_grad_()
            with pytest.raises(ValueError, match="no backward"):
                call(**{name: wants})
            if t.dtype is not torch.float8_e4m3fn:
                with forward_ad.dual_level(), torch.no_grad():
                    dual = forward_ad.make_dual(t.detach(), torch.ones_like(t))
                    with pytest.raises(ValueError, match="no derivative"):
                        call(**{name: dual})
    assert torch.equal(kp.view(torch.uint8), held.view(torch.uint8)), "a refused call wrote"
    with torch.no_grad():
        got = attend(q=q.clone().requires_grad_())
        append(k=k.clone().requires_grad_())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def bits_of_e4m3(values):
    """E4M3 bytes of values that E4M3 has (NaN as 0x7F), the sign of zero kept."""
    a = np.abs(values)
    e = np.maximum(np.frexp(np.where(np.isnan(a) | (a == 0), 2.0 ** -6, a))[1] - 1, -6)
    m = np.ldexp(np.where(np.isnan(a), 0, a), 3 - e)
    b = np.where(m >= 8, (e + 7) * 8 + m - 8, m)
    return np.where(np.isnan(values), 0x7F, b + np.where(np.signbit(values), 0x80, 0)).astype(np.uint8)


@pytest.mark.parametrize("scale", [1.0, 0.37, -0.5, 3e-5, 1e-30, 1e-36, 2.0 ** -140, 1e31, 1e38])
def test_append_every_bf16_pattern_with_its_sign(torch, scale):
    """The bytes that are stored, minus zero among them, for scales with a normal reciprocal, past it and negative."""
    say(f"append every pattern to bytes, scale {scale}")
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    kp = torch.zeros(32, 1, 16, 128, device="cuda").to(torch.float8_e4m3fn)
    vp = torch.zeros_like(kp)
    s = torch.full((1,), scale, device="cuda")
    hdb.df11_paged_append(x, x, torch.arange(512, device="cuda"), kp, vp, s, s)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        v = (x.float().cpu().numpy().reshape(-1) / np.float32(scale)).astype(np.float64)  # the 32-bit quotient, on the host
        a = np.minimum(np.abs(v), 448)
        e = np.maximum(np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -6)
        want = bits_of_e4m3(np.copysign(np.ldexp(np.rint(np.ldexp(a, 3 - e)), e - 3), v))
    for p in (kp, vp):
        got = p.view(torch.uint8).cpu().numpy().reshape(-1)
        nan = np.isnan(v)
        assert np.array_equal(got[~nan], want[~nan])
        assert (got[nan] & 0x7F == 0x7F).all()


def test_append_keeps_bf16_bits(torch):
    say("append every pattern to BF16 pages")
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    kp = torch.zeros(32, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    hdb.df11_paged_append(x, x, torch.arange(512, device="cuda"), kp, vp)
    for p in (kp, vp):
        assert torch.equal(p.view(torch.int16).view(-1), x.view(torch.int16).view(-1))


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_chunks_of_one_length_over_few_sequences(torch, fp8):
    """Five sequences of up to 16,500 positions: about 2,400 to a chunk, all sequences cut to one length."""
    say(f"attention 5 ragged of 16500 fp8={fp8}")
    q, kp, vp, table, lens, ks, vs = build(torch, ragged(5, 16500, 1), 8, 1, 128, 128, fp8)
    # more room than chunks of each sequence by itself would take: heads x (128 values, maximum and sum)
    splits = -(-256 // (5 * 8))
    assert hdb.df11_paged_attention_workspace_bytes(5, 8, 8, 128, 128, table.shape[1]) > 5 * splits * 8 * 130 * 4
    check(torch, q, kp, vp, table, lens, None, ks, vs)
