"""GPU checks of the attention of drafted trees and chains over a paged cache,
against 64 bits.

Bounds, for scores s = scale q . k computed in 32 bits from exact products:
each is off by at most e = (head_dim + 4) 2^-23 scale max_j sum |q| |k_j| plus
2^-22 max |s| (the scale, log2 e and the difference from the reference, rounded).
With BF16 pages a weight is off by a factor of at most 1 + 2 e + 2^-16 (its two
parts, the exponential), with E4M3 pages by 1 + 2 e + 2^-11 (FP16) and at least
by 2^-25 of a weight that the largest reaches (FP16's smallest step, halved); a
sum of L terms by L 2^-23 more.  With weights w, the largest 1:
  |out - ref| <= 2^-8 |ref| + (4 e + 2^-14 + L 2^-22 [+ 2^-10]) sum w |v| / sum w [+ 2^-24 sum |v| / sum w]
  |lse - ref| <= 2 e + 2^-17 + L 2^-22 + 2^-22 |ref|
"""
import math

import pytest

import huffman_decode_block_amd as hdb
from test_gpu_paged import LAYOUTS, make_pages

pytestmark = pytest.mark.gpu


def say(msg):
    print(f"[gpu-test] {msg}", flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "the GPU tests need a GPU"
    return t


def bits_of(torch, reads):
    """Mask words of reads [batch, nodes, nodes]."""
    b, t, _ = reads.shape
    words = (t + 63) // 64
    padded = torch.nn.functional.pad(reads, (0, 64 * words - t)).view(b, t, words, 64).long()
    return (padded << torch.arange(64, device=reads.device)).sum(-1)


def random_tree(torch, g, batch, nodes):
    reads = torch.eye(nodes, dtype=torch.bool, device="cuda").repeat(batch, 1, 1)
    parent = (torch.rand(batch, nodes, generator=g, device="cuda") * torch.arange(nodes, device="cuda")).long()
    each = torch.arange(batch, device="cuda")
    for i in range(1, nodes):
        reads[:, i] |= reads[each, parent[:, i]]
    return reads


def build(torch, lens, nodes, heads, group, dim, page, fp8, layout="heads first", counts=None, chain=False, spread=1.0, seed=1,
          fill=float("nan"), extra=1):
    """A call's arguments over a cache whose unused positions hold `fill`, and what each node reads of the nodes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch = len(lens)
    width = -(-(max(lens) + nodes) // page) + extra
    n = batch * width + 2
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kp = make_pages(torch, n, heads, page, dim, dtype, layout, fill)
    vp = make_pages(torch, n, heads, page, dim, dtype, layout, fill)
    table = torch.randperm(n, generator=g, device="cuda")[:batch * width].int().view(batch, width)
    ks = vs = None
    if fp8:
        ks = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.005
        vs = torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.005
    count = [nodes] * batch if counts is None else counts
    total = sum(lens) + sum(count)
    if total:
        k = (torch.randn(total, heads, dim, generator=g, device="cuda") * spread).to(torch.bfloat16)
        v = torch.randn(total, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
        slots = torch.cat([table[b].long().repeat_interleave(page)[:m + c] * page + torch.arange(m + c, device="cuda") % page
                           for b, (m, c) in enumerate(zip(lens, count))])
        hdb.df11_paged_append(k, v, slots, kp, vp, ks, vs)
    q = torch.randn(batch, nodes, heads * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    reads = torch.ones(nodes, nodes, dtype=torch.bool, device="cuda").tril().repeat(batch, 1, 1) if chain else random_tree(torch, g, batch, nodes)
    a = dict(q=q, k_pages=kp, v_pages=vp, page_table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             tree=None if chain else bits_of(torch, reads),
             nodes=None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs)
    return a, reads


def reference(torch, a, reads):
    """(out, lse, bound of out, bound of lse) in 64 bits."""
    q, kp, vp, table = a["q"], a["k_pages"], a["v_pages"], a["page_table"]
    batch, t, q_heads, dim = q.shape
    n, heads, page, _ = kp.shape
    group = q_heads // heads
    fp8 = a["k_scale"] is not None
    scale = a.get("scale")
    scale = dim ** -0.5 if scale is None else scale
    f = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(batch, t, q_heads, dim, **f), torch.full((batch, t, q_heads), -math.inf, **f)
    out_b, lse_b = torch.zeros(batch, t, q_heads, dim, **f), torch.zeros(batch, t, q_heads, **f)
    for b in range(batch):
        m = min(max(int(a["lens"][b]), 0), table.shape[1] * page)
        c = t if a["nodes"] is None else min(max(int(a["nodes"][b]), 0), t)
        at = torch.arange(min(m + c, table.shape[1] * page), device="cuda")
        pg = table[b].long()[at // page]
        ok = (pg >= 0) & (pg < n)
        at, pg = at[ok], pg[ok]
        if at.numel() == 0 or c == 0:
            continue
        start = torch.zeros(c, 1, dtype=torch.long, device="cuda")
        if a.get("starts") is not None:
            start = a["starts"][b, :c].long().clamp(0, m).view(c, 1)
        node = (at - m).clamp(0, t - 1)
        live = ((at < m) & (at >= start)) | ((at >= m) & reads[b, :c][:, node])
        for h in range(heads):
            k, v = kp[:, h].float().double()[pg, at % page], vp[:, h].float().double()[pg, at % page]
            if fp8:
                k, v = k * a["k_scale"][h].double(), v * a["v_scale"][h].double()
            mine = slice(h * group, (h + 1) * group)
            qq = q[b, :c, mine].double().reshape(c * group, dim)
            lv = live.repeat_interleave(group, 0)
            s = (scale * (qq @ k.T.contiguous())).masked_fill(~lv, -math.inf)
            some = lv.any(-1)
            size = lv.sum(-1, keepdim=True)
            mag = abs(scale) * (qq.abs() @ k.abs().T.contiguous()).masked_fill(~lv, 0).amax(-1, keepdim=True)
            e = (dim + 4) * 2.0 ** -23 * mag + 2.0 ** -22 * s.masked_fill(~lv, 0).abs().amax(-1, keepdim=True)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            w = torch.exp(s - top)
            sw = w.sum(-1, keepdim=True)
            odd = ~v.isfinite()
            vf = v.masked_fill(odd, 0)
            o = w @ vf / torch.where(sw == 0, 1.0, sw)
            o_b = 2.0 ** -8 * o.abs() + (4 * e + 2.0 ** -14 + size * 2.0 ** -22 + (2.0 ** -10 if fp8 else 0)) * (w @ vf.abs()) / torch.where(sw == 0, 1.0, sw)
            if fp8:
                o_b += 2.0 ** -24 * (lv.double() @ vf.abs()) / torch.where(sw == 0, 1.0, sw)
            if odd.any():
                r = lv.double()
                plus, minus, nan = (r @ x.double() > 0 for x in (v == math.inf, v == -math.inf, v.isnan()))
                o = torch.where(plus, math.inf, torch.where(minus, -math.inf, o))
                o = torch.where(nan | (plus & minus) | sw.isnan(), math.nan, o)  # a score that is no number leaves none
            put = lambda to, x: to[b, :c, mine].copy_(torch.where(some.view(c, group, *[1] * (x.dim() - 1)), x.view(c, group, *x.shape[1:]), to[b, :c, mine]))  # noqa: E731
            put(out, o)
            put(out_b, o_b)
            put(lse, torch.log(sw)[:, 0] + top[:, 0])
            put(lse_b, (2 * e + 2.0 ** -17 + size * 2.0 ** -22)[:, 0] + 2.0 ** -22 * (torch.log(sw) + top)[:, 0].abs())
    return out, lse, out_b, lse_b


def compare(torch, got, want):
    """Values within their bounds, infinities and NaN where they belong."""
    (out, lse), (ref, ref_lse, bound, lse_bound) = got, want
    for x, y, b, name in ((out, ref, bound, "out"), (lse, ref_lse, lse_bound, "lse")):
        x = x.double()
        fine = y.isfinite()
        assert torch.equal(x.isfinite(), fine), name
        assert torch.equal(x.isnan(), y.isnan()), name
        assert torch.equal(x[y.isinf()], y[y.isinf()]), name
        over = ((x - y).abs() - b)[fine]
        assert over.numel() == 0 or float(over.max()) <= 0, (name, float(over.max()))


def check(torch, a, reads):
    got = hdb.df11_paged_tree_attention(**a)
    compare(torch, got, reference(torch, a, reads))
    again = hdb.df11_paged_tree_attention(**a)
    assert torch.equal(got[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(got[1], again[1]), "a second call differs"
    return got


EDGE_LENS = [0, 1, 2, 7, 8, 15, 31, 32, 33, 63, 65, 100, 127, 128, 200, 257]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,group,nodes,layout", [(8, 1, 1, 0), (16, 4, 3, 1), (64, 7, 9, 2), (1024, 2, 65, 0), (32, 16, 16, 1)])
def test_trees(torch, fp8, dim, page, group, nodes, layout):
    say(f"tree dim {dim} page {page} group {group} nodes {nodes} {LAYOUTS[layout]} fp8={fp8}")
    check(torch, *build(torch, EDGE_LENS, nodes, 2, group, dim, page, fp8, LAYOUTS[layout]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,group,nodes", [(16, 1, 1), (16, 3, 33), (64, 4, 130), (8, 1, 300)])
def test_chains(torch, fp8, dim, page, group, nodes):
    say(f"chain dim {dim} page {page} group {group} nodes {nodes} fp8={fp8}")
    check(torch, *build(torch, [0, 1, 31, 64, 300], nodes, 2, group, dim, page, fp8, chain=True))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,group,nodes", [(1, 1, 15), (1, 1, 17), (3, 5, 7), (1, 33, 3), (8, 2, 128), (2, 3, 129), (1, 40, 64)])
def test_head_layouts(torch, fp8, heads, group, nodes):
    say(f"tree {heads} heads group {group} nodes {nodes} fp8={fp8}")
    check(torch, *build(torch, [0, 70, 513], nodes, heads, group, 128, 16, fp8, counts=[nodes, nodes // 2, nodes]))


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_counts(torch, fp8, chain):
    """Sequences of no node, of all, of more and of less than none; rows behind the last node are zeros."""
    say(f"counts chain={chain} fp8={fp8}")
    counts = [0, 1, 20, 19, 5, 16]
    a, reads = build(torch, [50, 0, 33, 64, 0, 300], 20, 2, 4, 128, 16, fp8, counts=counts, chain=chain)
    out, lse = check(torch, a, reads)
    for b, c in enumerate(counts):
        assert bool((out[b, c:] == 0).all()) and bool((lse[b, c:] == -math.inf).all())
    a["nodes"] = torch.tensor([-1, 1, 99, 19, 5, 16], dtype=torch.int32, device="cuda")
    check(torch, a, reads)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("length,page,dim,nodes", [(1100, 16, 128, 8), (5003, 64, 64, 64), (4097, 32, 256, 20), (40000, 8, 64, 5), (20000, 128, 128, 33)])
def test_long_contexts(torch, fp8, length, page, dim, nodes):
    say(f"tree behind {length}, page {page} dim {dim} nodes {nodes} fp8={fp8}")
    check(torch, *build(torch, [length, 3, length // 2], nodes, 1, 4, dim, page, fp8))


@pytest.mark.parametrize("batch", [40, 300])
def test_many_sequences(torch, batch):
    say(f"trees of {batch} sequences")
    lens = [(37 * i * i) % 700 for i in range(batch)]
    check(torch, *build(torch, lens, 6, 2, 4, 64, 16, False, counts=[i % 7 for i in range(batch)]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,nodes,chain", [([700], 65, False), ([900, 33, 0, 4200], 40, False), ([2500, 60, 1], 130, True)])
def test_wide_tables(torch, fp8, dim, lens, nodes, chain):
    """Tables for far more positions than there are: the largest tiles of rows, short chunks."""
    say(f"tree in a wide table, lens {lens} nodes {nodes} dim {dim} chain={chain} fp8={fp8}")
    a, reads = build(torch, lens, nodes, 2, 4, dim, 32, fp8, chain=chain)
    table = torch.full((len(lens), 1 << 15), -1, dtype=torch.int32, device="cuda")
    table[:, :a["page_table"].shape[1]] = a["page_table"]
    a["page_table"] = table
    check(torch, a, reads)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch,nodes,dim", [(2, 40, 128), (17, 3, 128), (64, 9, 64), (65, 9, 64), (24, 12, 256)])
def test_ragged_batches(torch, batch, nodes, dim, fp8):
    """One long sequence among short and empty ones, with and without windows."""
    say(f"ragged batch of {batch}, nodes {nodes} dim {dim} fp8={fp8}")
    lens = [(97 * i * i) % 160 for i in range(batch)]
    lens[batch // 2] = 6000
    a, reads = build(torch, lens, nodes, 1, 4, dim, 16, fp8, counts=[max(0, nodes - i % 5) for i in range(batch)])
    check(torch, a, reads)
    a["starts"] = (a["lens"].view(-1, 1) - torch.arange(nodes, device="cuda") * 7 - 50).int()
    check(torch, a, reads)
    a["lens"] = torch.zeros_like(a["lens"])
    a["starts"] = None
    a["nodes"] = torch.zeros_like(a["lens"])
    out, lse = hdb.df11_paged_tree_attention(**a)
    assert not bool(out.any()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("fp8,dim,nodes", [(False, 64, 3), (True, 64, 33), (True, 128, 2), (False, 256, 20)])
def test_long_chunks(torch, fp8, dim, nodes):
    """More positions for a workgroup than it keeps the pages of at a time."""
    heads = 520 if dim == 64 else 260
    say(f"{heads} heads behind 4,700 positions, nodes {nodes} dim {dim} fp8={fp8}")
    batch = 520 // heads
    check(torch, *build(torch, [4700] * batch, nodes, heads, 1, dim, 64, fp8))


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("dim,fp8", [(64, False), (128, True), (256, False)])
def test_starts(torch, dim, fp8, chain):
    """Windows of a node's own: inside and at the edges of steps, past the length, negative, none."""
    say(f"starts dim {dim} chain={chain} fp8={fp8}")
    lens, nodes = [300, 300, 40, 0, 1500], 33
    a, reads = build(torch, lens, nodes, 2, 3, dim, 16, fp8, chain=chain)
    g = torch.Generator(device="cuda").manual_seed(5)
    starts = torch.randint(-3, 310, (5, nodes), generator=g, device="cuda").int()
    starts[0, :8] = torch.tensor([0, 1, 31, 32, 33, 299, 300, 301], device="cuda").int()
    starts[4] += 1190
    a["starts"] = starts
    check(torch, a, reads)
    a["starts"] = torch.tensor([128, 290, 5, 0, 1400], dtype=torch.int32, device="cuda").view(5, 1).expand(5, nodes)
    check(torch, a, reads)
    wide = torch.full((5, 2 * nodes), -9, dtype=torch.int32, device="cuda")
    wide[:, ::2] = starts
    a["starts"] = wide[:, ::2]
    check(torch, a, reads)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_read_nothing(torch, fp8):
    """Masks of no node, not even itself, behind windows that are empty."""
    say(f"empty rows fp8={fp8}")
    a, reads = build(torch, [40, 0, 700], 70, 2, 2, 64, 16, fp8)
    reads[:, ::3] = False
    a["tree"] = bits_of(torch, reads)
    a["starts"] = torch.full((3, 70), 1 << 30, dtype=torch.int32, device="cuda")
    out, lse = check(torch, a, reads)
    assert bool((out[:, ::3] == 0).all()) and bool((lse[:, ::3] == -math.inf).all())
    assert bool(lse[:, 1::3].isfinite().all())


def test_one_tree_for_all_sequences(torch):
    """Strides of zero, words between others, bits behind the last node."""
    say("shared tree")
    a, reads = build(torch, [40, 0, 700], 70, 2, 2, 64, 16, False)
    one = a["tree"][:1].clone()
    one[..., 1] |= -1 << 6  # nodes 70 and up
    wide = torch.full((1, 70, 5), -1, dtype=torch.int64, device="cuda")
    wide[..., 1:3] = one
    a["tree"] = wide[..., 1:3].expand(3, 70, 2)
    check(torch, a, reads[:1].expand(3, 70, 70))


@pytest.mark.parametrize("fp8", [False, True])
def test_masked_pages_and_narrow_tables(torch, fp8):
    """Table entries outside the cache mask their positions, up to all of a sequence, nodes among them; nodes past the table."""
    say(f"masked pages fp8={fp8}")
    a, reads = build(torch, [200, 200, 200, 50, 180], 24, 2, 4, 128, 16, fp8)
    t = a["page_table"]
    t[0, 3], t[0, 13], t[1, 0] = -1, a["k_pages"].shape[0], 1 << 30
    t[2] = -5
    out, lse = check(torch, a, reads)
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())
    a["page_table"] = t[:, :13].clone()  # 208 positions
    check(torch, a, reads)
    a["page_table"] = t[:, :4].clone()
    check(torch, a, reads)
    a["lens"] = torch.full_like(a["lens"], -3)
    check(torch, a, reads)


def test_large_small_and_turned_scores(torch):
    say("large scores")
    a, reads = build(torch, [1, 40, 700, 1300], 9, 2, 4, 128, 16, False, spread=300.0)
    for scale in (None, -0.01, 0.0, 1e-3):
        a["scale"] = scale
        check(torch, a, reads)
    a, reads = build(torch, [900], 20, 1, 4, 64, 16, True, spread=30.0)
    a["k_scale"] = -a["k_scale"]
    check(torch, a, reads)


def test_scores_that_rise_and_fall(torch):
    """The reference of the weights follows maxima that grow by little and by much at each step, and stays."""
    say("rising scores")
    a, reads = build(torch, [2000, 2000], 17, 1, 4, 64, 16, False)
    ramp = torch.linspace(0.1, 40, 2000, device="cuda")
    for b, r in enumerate((ramp, ramp.flip(0))):
        at = torch.arange(2000, device="cuda")
        pg = a["page_table"][b].long()[at // 16]
        a["k_pages"][pg, 0, at % 16] = (a["q"][b, 0, 0].float() * r.view(-1, 1) / 8).to(torch.bfloat16)
    check(torch, a, reads)


@pytest.mark.parametrize("dim,fp8,chain", [(64, False, False), (128, False, True), (128, True, False), (256, False, False), (64, True, True)])
def test_what_a_node_does_not_read(torch, dim, fp8, chain):
    """NaN and infinities in the keys and values of some nodes and in front of some windows reach their readers alone."""
    say(f"odd values dim {dim} chain={chain} fp8={fp8}")
    lens, nodes, page = [100, 0, 31, 700], 40, 16
    a, reads = build(torch, lens, nodes, 2, 3, dim, page, fp8, chain=chain)
    g = torch.Generator(device="cuda").manual_seed(9)
    a["starts"] = torch.randint(0, 60, (4, nodes), generator=g, device="cuda").int()
    clean = hdb.df11_paged_tree_attention(**a)
    inf, nan = math.inf, math.nan
    for b, m in enumerate(lens):
        for at, col, value in ((m + 5, 3, nan), (m + 7, 0, inf), (m + 11, 0, -inf), (m + 21, dim - 1, -inf), (m + 39, 6, inf), (17, 9, inf), (18, 10, nan),
                               (40, dim - 2, -inf), (m + 20, 5, inf)):
            if at < m + nodes:
                value = nan if fp8 else value
                a["v_pages"][int(a["page_table"][b, at // page]), b % 2, at % page, col] = value
        at = m + 12  # a key
        a["k_pages"][int(a["page_table"][b, at // page]), 1, at % page, 4] = nan
    want = reference(torch, a, reads)
    got = hdb.df11_paged_tree_attention(**a)
    compare(torch, got, want)
    assert int((~want[0].isfinite()).sum()) > 100 and int(want[0].isfinite().sum()) > got[0].numel() // 4
    same = want[0].isfinite()
    same[:, :, 3:] = False  # the head whose keys stayed: bit for bit what it was
    assert torch.equal(got[0][same], clean[0][same])


def test_infinities_in_front_of_all(torch):
    """Infinities that every node reads, in steps without a mask."""
    say("infinite values in the context")
    a, reads = build(torch, [1500, 200], 9, 1, 4, 128, 16, False)
    for b, at, col, value in ((0, 700, 3, math.inf), (0, 701, 5, -math.inf), (0, 1, 7, math.inf), (0, 1400, 7, -math.inf), (1, 64, 0, math.nan), (1, 65, 1, math.inf)):
        a["v_pages"][int(a["page_table"][b, at // 16]), 0, at % 16, col] = value
    compare(torch, hdb.df11_paged_tree_attention(**a), reference(torch, a, reads))


def test_infinite_keys(torch):
    say("infinite keys")
    a, reads = build(torch, [300], 5, 1, 2, 64, 16, False)
    a["q"][:, :, 0, 5], a["q"][:, :, 1, 5] = 1.0, -1.0
    a["k_pages"][int(a["page_table"][0, 10]), 0, 3, 5] = math.inf
    out, lse = hdb.df11_paged_tree_attention(**a)
    assert bool(out[:, :, 0].isnan().all())
    assert bool(out[:, :, 1].isfinite().all()) and bool(lse[:, :, 1].isfinite().all())


def test_strided_queries(torch):
    say("strided queries")
    a, reads = build(torch, [90, 33], 6, 2, 2, 128, 16, False)
    joint = torch.full((2, 7, 9, 131), float("nan"), dtype=torch.bfloat16, device="cuda")
    joint[:, 1:, 1:5, 1:129] = a["q"]
    want = hdb.df11_paged_tree_attention(**a)
    wide = torch.full((2, a["page_table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :a["page_table"].shape[1]] = a["page_table"]
    got = hdb.df11_paged_tree_attention(**{**a, "q": joint[:, 1:, 1:5, 1:129], "page_table": wide[:, :a["page_table"].shape[1]]})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    turned = a["q"].transpose(0, 1).contiguous().transpose(0, 1)
    got = hdb.df11_paged_tree_attention(**{**a, "q": turned})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_past_4_gib(torch):
    say("tree over 6 GiB of pages")
    page, heads, dim = 64, 8, 128
    n = (6 << 30) // (page * heads * dim * 2)
    kp = torch.zeros(n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros(n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    a, reads = build(torch, [5 * page - 7], 9, heads, 4, dim, page, False, extra=0, fill=0.0)
    at = torch.tensor([0, n - 1, n // 3, n // 2, n - 7, 1], device="cuda")[:a["page_table"].shape[1]]
    pages = a["page_table"][0].long()
    kp[at], vp[at] = a["k_pages"][pages], a["v_pages"][pages]
    want = hdb.df11_paged_tree_attention(**a)
    got = hdb.df11_paged_tree_attention(**{**a, "k_pages": kp, "v_pages": vp, "page_table": at.int().view(1, -1)})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("length", [60, 3000])
def test_streams_and_graphs(torch, length):
    """A side stream, two streams at once, a graph whose replays find other lengths, counts, masks and queries."""
    say(f"tree on side streams and in a graph, length {length}")
    a, reads = build(torch, [length, 10], 20, 2, 4, 128, 16, False, counts=[20, 20])
    want = hdb.df11_paged_tree_attention(**a)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [hdb.df11_paged_tree_attention(**a, stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hdb.df11_paged_tree_attention(**a, out=out, lse=lse)
    for step in range(4):
        a["lens"][:1].fill_(length - 7 * step)
        a["nodes"].fill_(20 - 3 * step)
        a["tree"].bitwise_or_(1 << step)
        a["q"].mul_(-1)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = hdb.df11_paged_tree_attention(**a)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        for i in range(step + 1):
            reads[:, :, i] = True
        compare(torch, eager, reference(torch, a, reads))


def test_one_node_is_the_attention_of_one_token(torch):
    """A chain of one node reads what the single token's attention reads; both within their bounds."""
    say("one node against one token")
    a, reads = build(torch, [0, 40, 300, 2000], 1, 2, 4, 128, 16, False, chain=True)
    out, lse = check(torch, a, reads)
    one, one_lse = hdb.df11_paged_attention(a["q"][:, 0], a["k_pages"], a["v_pages"], a["page_table"], a["lens"] + 1)
    _, _, bound, lse_bound = reference(torch, a, reads)
    assert bool(((out[:, 0].double() - one.double()).abs() <= 2 * bound[:, 0]).all())
    assert bool(((lse[:, 0].double() - one_lse.double()).abs() <= 2 * lse_bound[:, 0]).all())


def test_refusals(torch):
    say("tree refusals")
    a, _ = build(torch, [20, 3], 5, 2, 2, 128, 16, False)

    def call(**more):
        return hdb.df11_paged_tree_attention(**{**a, **more})

    for bad in (dict(q=a["q"].float()), dict(page_table=a["page_table"].long()), dict(k_pages=a["k_pages"].half(), v_pages=a["v_pages"].half()),
                dict(tree=a["tree"].int()), dict(nodes=a["lens"].long()), dict(lens=a["lens"].cpu()), dict(starts=a["tree"][..., 0])):
        with pytest.raises(TypeError):
            call(**bad)
    starts = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    for bad in (dict(q=a["q"][:, :, :3]), dict(q=a["q"][0]), dict(page_table=a["page_table"][:1]), dict(lens=a["lens"][:1]), dict(tree=a["tree"][:, :4]),
                dict(tree=a["tree"][:1]), dict(tree=torch.cat([a["tree"]] * 2, -1)), dict(nodes=a["lens"][:1]), dict(starts=starts[:, :4]),
                dict(tree=a["tree"][:, :1].expand(2, 5, 1)), dict(k_scale=torch.ones(2, device="cuda")),
                dict(k_pages=a["k_pages"].to(torch.float8_e4m3fn), v_pages=a["v_pages"].to(torch.float8_e4m3fn)),
                dict(out=torch.empty_like(a["q"])[:, :, :2]), dict(q=a["q"].clone().requires_grad_()),
                dict(v_pages=a["v_pages"].clone().requires_grad_()), dict(workspace=torch.empty(4))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(hdb.DF11Error) as e:
        call(q=a["q"][..., :32], k_pages=a["k_pages"][..., :32], v_pages=a["v_pages"][..., :32])
    assert e.value.status == hdb.DF11_E_UNSUPPORTED
    long, _ = build(torch, [3000], 5, 2, 2, 128, 16, False)
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_paged_tree_attention(**long, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == hdb.DF11_E_BUFFER_TOO_SMALL
    assert call(q=a["q"][:0], page_table=a["page_table"][:0], lens=a["lens"][:0], tree=a["tree"][:0])[0].shape == (0, 5, 4, 128)
    out, lse = call(q=a["q"][:, :0], tree=a["tree"][:, :0, :0])
    assert out.shape == (2, 0, 4, 128) and lse.shape == (2, 0, 4)


@pytest.mark.parametrize("batch", [1, 2, 64])
def test_no_nodes_behind_long_tables(torch, batch):
    """A call without nodes returns empty tensors, also where a table's positions would be shared among workgroups."""
    say(f"no nodes, {batch} sequences of wide tables")
    kp = torch.zeros(3, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(batch, 64, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), 1000, dtype=torch.int32, device="cuda")
    q = torch.zeros(batch, 0, 32, 128, dtype=torch.bfloat16, device="cuda")
    for tree in (None, torch.zeros(batch, 0, 0, dtype=torch.int64, device="cuda")):
        out, lse = hdb.df11_paged_tree_attention(q, kp, kp, table, lens, tree)
        assert out.shape == (batch, 0, 32, 128) and lse.shape == (batch, 0, 32)


@pytest.mark.parametrize("dim,group,nodes,wide", [(64, 1, 9, False), (128, 4, 8, False), (256, 2, 5, False), (64, 8, 8, False), (128, 4, 12, False), (256, 4, 12, False),
                                                  (64, 16, 9, True), (128, 4, 20, True), (128, 4, 40, True), (64, 4, 40, True)])
def test_small_weights_of_e4m3(torch, dim, group, nodes, wide):
    """Positions 18 (26 powers of two) behind the one that a row mostly reads, whose value is zero: all that there is.
    A weight is off by 2^-11 of itself or, below FP16's normal numbers, by 2^-32 of the largest (1 here); scores are
    whole numbers up to 16, an exponential off by 2^-18; the values' sum by 2^-22 for each of 128 terms at most."""
    say(f"small weights dim {dim} group {group} nodes {nodes} wide={wide}")
    length, page = 80, 16
    a, reads = build(torch, [length, length // 2], nodes, 2, group, dim, page, True, chain=True)
    code = lambda x: torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8).item()  # noqa: E731
    k, v, table = a["k_pages"].view(torch.uint8), a["v_pages"].view(torch.uint8), a["page_table"]
    k.zero_()
    k[..., 0] = code(-2)
    v.bitwise_and_(0x77)  # positive numbers of up to 240
    for b, at in enumerate((37, 3)):
        k[int(table[b, at // page]), :, at % page, 0] = code(16)
        v[int(table[b, at // page]), :, at % page] = 0
    a["q"].zero_()
    a["q"][..., 0] = 1
    a["scale"], a["k_scale"] = 1.0, torch.ones(2, device="cuda")
    if wide:
        a["page_table"] = torch.full((2, 1 << 15), -1, dtype=torch.int32, device="cuda")
        a["page_table"][:, :table.shape[1]] = table
    (out, lse), (ref, ref_lse, _, lse_bound) = hdb.df11_paged_tree_attention(**a), reference(torch, a, reads)
    assert bool(((lse.double() - ref_lse).abs() <= lse_bound).all())
    size = (a["lens"].view(2, 1, 1, 1) + torch.arange(1, nodes + 1, device="cuda").view(1, nodes, 1, 1)).double()
    v_max = 240 * a["v_scale"].double().repeat_interleave(group).view(1, 1, -1, 1)
    bound = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * ref + 2.0 ** -32 * size * v_max
    assert float(ref.min()) >= 0 and float((ref > 4 * bound).double().mean()) > 0.9, "the bound leaves nothing to see"
    over = (out.double() - ref).abs() - bound
    assert float(over.max()) <= 0, float(((out.double() - ref).abs() / bound.clamp_min(1e-30)).max())
