"""GPU checks of pages copied, compacted and forked: whole numbers and bits,
exact against plain host code."""
import numpy as np
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


def random_pages(torch, layers, n, heads, page, dim, fp8, layout, seed=1):
    """K and V pages of random bits, NaN patterns among them; layers None: without that dimension."""
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    got = []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed + i)
        if layers is None:
            p = make_pages(torch, n, heads, page, dim, dtype, layout, 0.0)
        else:
            p = make_pages(torch, layers * n, heads, page, dim, dtype, layout, 0.0)
            p = p.unflatten(0, (layers, n))
        bits = torch.int8 if fp8 else torch.int16
        lo, hi = (-128, 128) if fp8 else (-32768, 32768)
        p.view(bits).copy_(torch.randint(lo, hi, p.shape, generator=g, device="cuda").to(bits))
        got.append(p)
    return got


def host(torch, p):
    return p.view(torch.int8 if p.dtype is torch.float8_e4m3fn else torch.int16).cpu().numpy().copy()


def same(torch, p, want):
    return np.array_equal(host(torch, p), want)


SHAPES = [(None, 1, 8, 64), (None, 3, 16, 128), (1, 2, 64, 256), (3, 5, 32, 64), (2, 8, 16, 128), (7, 1, 1024, 64), (2, 1, 128, 256)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("layers,heads,page,dim", SHAPES)
def test_copy(torch, layers, heads, page, dim, layout, fp8):
    """Whole and partial pages, pairs that are skipped, one source for several targets; nothing else changes."""
    say(f"copy layers {layers} {heads} heads page {page} dim {dim} {LAYOUTS[layout]} fp8={fp8}")
    n = 24
    for partial in (False, True):
        k, v = random_pages(torch, layers, n, heads, page, dim, fp8, LAYOUTS[layout])
        want = [host(torch, k), host(torch, v)]
        src = torch.tensor([1, 1, 5, -1, n, 7, 2, 9, 1 << 30], dtype=torch.int32, device="cuda")
        dst = torch.tensor([12, 13, 14, 15, 16, -7, n, 23, 17], dtype=torch.int32, device="cuda")
        rows = torch.tensor([page, 1, page - 1, 3, 3, 3, 3, 99999, 1], dtype=torch.int32, device="cuda")
        if partial:
            rows[0] = -4  # none
        for i, (a, b) in enumerate(zip(src.tolist(), dst.tolist())):
            if 0 <= a < n and 0 <= b < n:
                m = max(0, min(page, int(rows[i]))) if partial else page
                for w in want:
                    w[..., b, :, :m, :] = w[..., a, :, :m, :]
        hdb.df11_paged_copy(src, dst, k, v, rows=rows if partial else None)
        assert same(torch, k, want[0]) and same(torch, v, want[1])


def test_copy_many_and_past_4_gib(torch):
    say("copy past 4 GiB")
    page, heads, dim = 64, 8, 128
    n = (6 << 30) // (page * heads * dim * 2)
    k = torch.zeros(n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    k[:700] = torch.randn(700, heads, page, dim, device="cuda").to(torch.bfloat16)
    v[:700] = torch.randn(700, heads, page, dim, device="cuda").to(torch.bfloat16)
    src = torch.arange(700, dtype=torch.int32, device="cuda")
    dst = (n - 1 - src).int()
    hdb.df11_paged_copy(src, dst, k, v)
    assert torch.equal(k[dst.long()], k[:700]) and torch.equal(v[dst.long()], v[:700])
    assert int((k[700:n - 700] != 0).sum()) == 0


def plain_compact(arrays, path, accepted, table, lens, page, n):
    width = table.shape[1]
    for b in range(len(lens)):
        last = -1
        for i in range(min(max(int(accepted[b]), 0), path.shape[1])):
            if path[b, i] <= last:
                break
            last = int(path[b, i])
            a, t = max(int(lens[b]), 0) + last, max(int(lens[b]), 0) + i
            if a >= width * page:
                continue
            pa, pt = int(table[b, a // page]), int(table[b, t // page])
            if not (0 <= pa < n and 0 <= pt < n):
                continue
            for w in arrays:
                w[..., pt, :, t % page, :] = w[..., pa, :, a % page, :]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layers,heads,page,dim,layout,depth,nodes", [
    (None, 1, 8, 64, 0, 1, 1), (None, 3, 16, 128, 1, 5, 20), (3, 5, 32, 64, 2, 8, 9), (2, 8, 16, 128, 0, 9, 64), (4, 1, 1024, 256, 1, 64, 130),
    (2, 2, 16, 64, 0, 65, 200), (1, 4, 64, 128, 2, 200, 400),
])
def test_compact(torch, fp8, layers, heads, page, dim, layout, depth, nodes):
    """Paths of every kind: whole, cut by a number that does not ascend, negative numbers, past the table, masked pages."""
    say(f"compact layers {layers} {heads}x{dim} page {page} depth {depth} nodes {nodes} fp8={fp8}")
    rng = np.random.default_rng(depth + nodes)
    batch, longest = 9, 70
    width = -(-(longest + nodes) // page)
    n = batch * width + 2
    k, v = random_pages(torch, layers, n, heads, page, dim, fp8, LAYOUTS[layout])
    path = np.stack([np.sort(rng.permutation(nodes)[:depth]) if nodes >= depth else np.arange(depth) for _ in range(batch)]).astype(np.int32)
    lens = rng.integers(0, longest + 1, batch).astype(np.int32)
    accepted = rng.integers(0, depth + 1, batch).astype(np.int32)
    table = rng.permutation(n)[:batch * width].reshape(batch, width).astype(np.int32)
    accepted[0], accepted[1], accepted[2] = depth, depth + 5, -2
    path[3], accepted[3] = np.arange(depth), depth  # already in place
    accepted[4:] = depth
    path[4, depth // 2] = -1
    path[5, depth // 2:] = path[5, 0]
    path[6, depth - 1] = 1 << 30
    table[7, ::2] = -1
    table[8, -1] = n
    lens[8] = max(longest - 1, 0)
    lens[5] = -4
    want = [host(torch, k), host(torch, v)]
    plain_compact(want, path, accepted, table, lens, page, n)
    d = [torch.from_numpy(x).cuda() for x in (path, accepted, table, lens)]
    held = [x.clone() for x in d]
    hdb.df11_paged_compact(*d, k, v)
    assert same(torch, k, want[0]) and same(torch, v, want[1])
    assert all(torch.equal(x, y) for x, y in zip(d, held))
    wide = torch.full((batch, width + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :width] = d[2]
    plain_compact(want, path, accepted, table, lens, page, n)
    hdb.df11_paged_compact(d[0], d[1], wide[:, :width], d[3], k, v)
    assert same(torch, k, want[0]) and same(torch, v, want[1])


def plain_fork(parents, table, lens, refs, page, room):
    """The definition, row by row."""
    batch, width = table.shape
    pool = len(refs)
    old, was = table.copy(), refs.copy()
    free = [p for p in range(pool) if was[p] == 0]
    new = np.full_like(table, -1)
    new_lens = np.zeros_like(lens)
    src, dst, rows = np.full(batch, -1, np.int32), np.full(batch, -1, np.int32), np.zeros(batch, np.int32)
    taken = missing = 0
    for b in range(batch):
        p = b if parents is None else int(parents[b])
        if not 0 <= p < batch:
            continue
        length = min(max(int(lens[p]), 0), width * page)
        new_lens[b] = length
        first = next(i for i in range(batch) if (i if parents is None else parents[i]) == p) == b
        for col in range(min(-(-(length + room) // page), width)):
            e = int(old[p, col])
            held = 0 <= e < pool
            if col < length // page:
                new[b, col] = e if held else -1
            elif first and held and was[e] <= 1:
                new[b, col] = e
            elif taken < len(free):
                new[b, col] = free[taken]
                taken += 1
                if col == length // page and length % page and held:
                    src[b], dst[b], rows[b] = e, new[b, col], length % page
            else:
                missing += 1
    for t, d in ((old, -1), (new, 1)):
        for e in t.reshape(-1):
            if 0 <= e < pool:
                refs[e] += d
    table[:] = new
    lens[:] = new_lens
    return src, dst, rows, missing


def check_fork(torch, parents, table, lens, refs, page, room, stream=None):
    """One fork against the plain one; the arrays and tensors move on together."""
    d = [None if x is None else torch.from_numpy(x).cuda() for x in (parents, table, lens, refs)]
    got = hdb.df11_paged_fork(*d, page, room=room, stream=stream)
    want = plain_fork(parents, table, lens, refs, page, room)
    torch.cuda.synchronize()
    for x, y, name in zip(got[:3], want[:3], ("src", "dst", "rows")):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert int(got[3]) == want[3]
    for x, y, name in zip(d[1:], (table, lens, refs), ("table", "lens", "refs")):
        assert np.array_equal(x.cpu().numpy(), y), name
    return want


def counted(table, pool):
    refs = np.zeros(pool, np.int32)
    for e in table.reshape(-1):
        if 0 <= e < pool:
            refs[e] += 1
    return refs


@pytest.mark.parametrize("batch,width,page,pool,room", [(1, 1, 8, 3, 0), (1, 1, 8, 3, 1), (5, 7, 16, 60, 1), (33, 9, 8, 700, 20), (64, 40, 16, 5000, 1),
                                                       (300, 5, 32, 3000, 64), (12, 130, 16, 20000, 300), (7, 33, 1024, 300, 5000)])
def test_fork_over_many_steps(torch, batch, width, page, pool, room):
    """A search from one row: children of one prompt, reorderings, rows that end and come back, growth, trims."""
    say(f"fork {batch} rows of {width} pages of {page}, room {room}")
    rng = np.random.default_rng(batch + width)
    table, lens, refs = np.full((batch, width), -1, np.int32), np.zeros(batch, np.int32), np.zeros(pool, np.int32)
    lens[0] = 0
    check_fork(torch, None, table, lens, refs, page, room)  # reserve
    lens[0] = min(room, width * page)
    for step in range(12):
        kind = step % 4
        if kind == 0:
            parents = np.zeros(batch, np.int32)
        elif kind == 1:
            parents = rng.integers(0, batch, batch).astype(np.int32)
        elif kind == 2:
            parents = rng.integers(-3, batch + 3, batch).astype(np.int32)
            parents[rng.integers(0, batch)] = 0
        else:
            parents = None
        _, _, _, missing = check_fork(torch, parents, table, lens, refs, page, room)
        assert np.array_equal(refs, counted(table, pool)) and refs.min() >= 0
        if missing == 0:  # what a page is written to belongs to one row
            for b in range(batch):
                for col in range(lens[b] // page, width):
                    assert table[b, col] < 0 or refs[table[b, col]] == 1
        grow = rng.integers(0, room + 1, batch) if kind != 3 else -rng.integers(0, page, batch)
        live = (table >= 0).sum(1) > 0
        lens[:] = np.where(live, np.clip(lens + grow, 0, width * page), 0)


def test_fork_out_of_pages(torch):
    say("fork without free pages")
    table = np.array([[0, 1, 2, -1], [3, 4, -1, -1], [-1, -1, -1, -1]], np.int32)
    lens = np.array([40, 20, 0], np.int32)
    refs = np.zeros(7, np.int32)
    refs[:5] = 1
    parents = np.array([0, 0, 0], np.int32)  # two copies and room: more than pages 5 and 6
    src, dst, rows, missing = check_fork(torch, parents, table, lens, refs, 16, 20)
    assert missing > 0
    check_fork(torch, None, table, lens, refs, 16, 0)
    check_fork(torch, np.array([1, 2, 0], np.int32), table, lens, refs, 16, 9)


def test_fork_odd_entries(torch):
    """Entries that are no pages, a page held from outside, lengths past the table and below none, a page named twice."""
    say("fork odd entries")
    table = np.array([[5, 99, 7, 8], [-3, 1 << 30, 9, -1], [10, 11, 12, 13], [2, 2, -1, -1]], np.int32)
    lens = np.array([40, 33, 1000, -5], np.int32)
    refs = counted(table, 40)
    refs[7] += 1  # also in a prefix that is kept
    refs[20:24] = 3
    check_fork(torch, np.array([0, 0, 1, 2], np.int32), table, lens, refs, 16, 3)
    check_fork(torch, np.array([2, 3, 3, 3], np.int32), table, lens, refs, 16, 30)
    check_fork(torch, np.array([-1, 4, 1 << 30, -(1 << 31)], np.int32), table, lens, refs, 16, 30)


def test_fork_of_a_large_table(torch):
    """All rows that a call takes, a pool that is nearly full."""
    say("fork 4096 rows")
    rng = np.random.default_rng(4)
    batch, width, page = 4096, 9, 16
    pool = 70001
    names = rng.permutation(pool).astype(np.int32)
    table, lens = np.full((batch, width), -1, np.int32), rng.integers(0, 8 * page, batch).astype(np.int32)
    at = 0
    for b in range(batch):
        m = -(-int(lens[b]) // page)
        table[b, :m] = names[at:at + m]
        at += m
    refs = counted(table, pool)
    refs[rng.permutation(pool)[:60000]] += 1  # others hold pages too
    check_fork(torch, rng.integers(0, batch, batch).astype(np.int32), table, lens, refs, page, 1)
    check_fork(torch, None, table, lens, refs, page, 40)


def test_fork_strides_streams_and_graph(torch):
    say("fork in a graph")
    batch, width, page, pool = 6, 5, 16, 100
    wide = torch.full((batch, width + 3), -7, dtype=torch.int32, device="cuda")
    table = wide[:, 1:1 + width]
    table.fill_(-1)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    parents = torch.zeros(batch, dtype=torch.int32, device="cuda")
    h = [np.full((batch, width), -1, np.int32), np.zeros(batch, np.int32), np.zeros(pool, np.int32)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    hdb.df11_paged_fork(None, table, lens, refs, page, room=5, stream=side)
    side.synchronize()
    plain_fork(None, *h, page, 5)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(hdb.df11_paged_fork_workspace_bytes(batch, width, page, pool, 5), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        got = hdb.df11_paged_fork(parents, table, lens, refs, page, room=5, workspace=ws)
    rng = np.random.default_rng(2)
    for step in range(6):
        p = rng.integers(0, batch, batch).astype(np.int32)
        parents.copy_(torch.from_numpy(p))
        graph.replay()
        torch.cuda.synchronize()
        want = plain_fork(p, *h, page, 5)
        for x, y in zip((*got[:3], table, lens, refs), (*want[:3], *h)):
            assert np.array_equal(x.cpu().numpy(), y), step
        assert int(got[3]) == want[3] == 0
        lens.add_(5)
        h[1] += 5
    assert int((wide[:, 0] != -7).sum()) == 0 and int((wide[:, 1 + width:] != -7).sum()) == 0


@pytest.mark.parametrize("op", ["copy", "compact"])
def test_copy_and_compact_on_streams_and_in_graphs(torch, op):
    say(f"{op} on a stream and in a graph")
    n, page = 40, 16
    k, v = random_pages(torch, 3, n, 2, page, 64, False, "heads first")
    src = torch.arange(8, dtype=torch.int32, device="cuda")
    dst = src + 20
    path = torch.tensor([[1, 3, 4], [0, 2, 9]], dtype=torch.int32, device="cuda")
    accepted = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([13, 20], dtype=torch.int32, device="cuda")

    def call(stream=None):
        if op == "copy":
            hdb.df11_paged_copy(src, dst, k, v, stream=stream)
        else:
            hdb.df11_paged_compact(path, accepted, table, lens, k, v, stream=stream)

    def plain(w):
        if op == "copy":
            for x in w:
                x[:, 20:28] = x[:, src.cpu().numpy()]
        else:
            plain_compact(w, path.cpu().numpy(), accepted.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), page, n)

    want = [host(torch, k), host(torch, v)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    plain(want)
    assert same(torch, k, want[0]) and same(torch, v, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(4):
        if op == "copy":
            src.add_(1)
        else:
            lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        plain(want)
        assert same(torch, k, want[0]) and same(torch, v, want[1])


def test_refusals(torch):
    say("page refusals")
    k, v = random_pages(torch, 2, 10, 2, 16, 64, False, "heads first")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    for bad in ((i.long(), i, k, v), (i, i.cpu(), k, v), (i, i, k.half(), v.half()), (i, i, k, v.to(torch.float8_e4m3fn))):
        with pytest.raises(TypeError):
            hdb.df11_paged_copy(*bad)
    for bad in ((i, i[:2], k, v), (i, i, k, v[:1]), (i, i, k[0], v), (i[::2], i[::2], k, v), (i, i, k.clone().requires_grad_(), v),
                (i, i, k.transpose(-1, -2), v.transpose(-1, -2))):
        with pytest.raises(ValueError):
            hdb.df11_paged_copy(*bad)
    with pytest.raises(ValueError):
        hdb.df11_paged_copy(i, i, k, v, rows=i[:2])
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_paged_copy(i, i, k[..., :32], v[..., :32])
    assert e.value.status == hdb.DF11_E_UNSUPPORTED
    hdb.df11_paged_copy(i[:0], i[:0], k, v)
    path = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    for bad in ((path, i[:2], table, i), (path, i, table[:2], i), (path, i, table, i[:2]), (path[0], i, table, i)):
        with pytest.raises(ValueError):
            hdb.df11_paged_compact(*bad, k, v)
    with pytest.raises(TypeError):
        hdb.df11_paged_compact(path.long(), i, table, i, k, v)
    with pytest.raises(hdb.DF11Error):
        hdb.df11_paged_compact(torch.zeros(3, 1025, dtype=torch.int32, device="cuda"), i, table, i, k, v)
    hdb.df11_paged_compact(path[:0], i[:0], table[:0], i[:0], k, v)
    hdb.df11_paged_compact(path[:, :0], i, table, i, k, v)
    refs = torch.zeros(10, dtype=torch.int32, device="cuda")
    for bad in ((i[:2], table, i, refs, 16), (i, table, i[:2], refs, 16), (i, table[0], i, refs, 16), (i, table, i, refs[::2], 16), (i, table, i, refs, -1)):
        with pytest.raises(ValueError):
            hdb.df11_paged_fork(*bad)
    with pytest.raises(ValueError):
        hdb.df11_paged_fork(i, table, i, refs, 16, room=-1)
    for bad in ((i.long(), table, i, refs, 16), (i, table.long(), i, refs, 16), (i, table, i, refs.float(), 16)):
        with pytest.raises(TypeError):
            hdb.df11_paged_fork(*bad)
    for more in (dict(page_size=12), dict(page_size=2048), dict(page_size=0), dict(page_size=16, room=1 << 31)):
        with pytest.raises(hdb.DF11Error):
            hdb.df11_paged_fork(i, table, i, refs, **more)
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_paged_fork(i, table, i, refs, 16, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == hdb.DF11_E_BUFFER_TOO_SMALL
    assert int(hdb.df11_paged_fork(i[:0], table[:0], i[:0], refs, 16)[3]) == 0
    assert int(refs.sum()) == 0 and int(table.sum()) == 0


def test_fork_sizes_past_their_types(torch):
    """Numbers that C would cut off to allowed ones are refused, and nothing changes."""
    say("fork sizes past 32 and 64 bits")
    table = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    refs = torch.tensor([1, 1, 1, 0, 0], dtype=torch.int32, device="cuda")
    parents = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    for page_size, room in (((1 << 32) + 16, 1), (16 - (1 << 32), 1), (16, (1 << 64) + 1), (16, 1 - (1 << 64))):
        with pytest.raises(ValueError):
            hdb.df11_paged_fork(parents, table, lens, refs, page_size, room=room)
    assert table.tolist() == [[0, 1], [2, -1]] and lens.tolist() == [20, 5] and refs.tolist() == [1, 1, 1, 0, 0]
