"""Cases for timing and checking the operators of decoding with more than one candidate for each sequence.

Operators:
  tree      attention of a tree of drafted tokens (or of a chain, as a chunk of a prompt is) over a paged cache
  beam      the best continuations of a sequence's beams over the vocabulary
  fork      the rows of a page table after a reordering: pages shared, taken and given back by their counts
  copy      pages of all layers copied, whole or their first positions
  compact   an accepted path's keys and values moved next to what the cache holds, in all layers

`run` computes them from elementary torch operations, or with `own` set through the library.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def listed():
    return [
        # a single user's tree of 64 drafted tokens behind 8,192 tokens of context, 8B-shaped heads
        dict(name="tree 1x8192 64 nodes", op="tree", batch=1, heads=32, kv_heads=8, dim=128, page=16, length=8192, nodes=64, chain=False, fp8=False, window=0, ragged=False),
        # a small serving batch, contexts and trees of every size up to 2,048 and 25
        dict(name="tree 16 ragged", op="tree", batch=16, heads=32, kv_heads=8, dim=128, page=16, length=2048, nodes=25, chain=False, fp8=False, window=0, ragged=True),
        # long contexts, 70B-shaped heads, E4M3 pages, small trees
        dict(name="tree 8x32768 fp8", op="tree", batch=8, heads=64, kv_heads=8, dim=128, page=64, length=32768, nodes=16, chain=False, fp8=True, window=0, ragged=False),
        # a chunk of a prompt behind what the cache holds, sliding windows over wide heads
        dict(name="chain 2x509 window", op="tree", batch=2, heads=8, kv_heads=4, dim=256, page=32, length=5003, nodes=509, chain=True, fp8=False, window=1024, ragged=False),
        # the first ranking of a search with four beams over a vocabulary of 32,000, logits in 32 bits
        dict(name="beam 1x4", op="beam", batch=1, beams=4, k=4, vocab=32000, f32=True, done=False, first=True, pad=0),
        # thirty-two searches of eight beams over a large vocabulary, twice as many continuations, some beams ended
        dict(name="beam 32x8", op="beam", batch=32, beams=8, k=16, vocab=128256, f32=False, done=True, first=False, pad=0),
        # eight searches of four beams take their next step, up to 2,048 positions each
        dict(name="fork 32 rows", op="fork", rows=32, beams=4, width=128, page=16, length=2000, room=1, spare=512, ended=False),
        # a large batch's searches with room for a tree, rows that end among them, in a pool of a hundred thousand pages
        dict(name="fork 512 rows", op="fork", rows=512, beams=8, width=513, page=16, length=8100, room=64, spare=16384, ended=True),
        # the pages that such a step copies: the first positions of a page for each beam, in 32 layers
        dict(name="copy 32 partial", op="copy", pairs=32, layers=32, kv_heads=8, dim=128, page=16, pages=160, fp8=False, partial=True),
        # 2,048 whole E4M3 pages moved together, as a prefix that is made a search's own
        dict(name="copy 2048 fp8", op="copy", pairs=2048, layers=2, kv_heads=8, dim=128, page=64, pages=4200, fp8=True, partial=False),
        # one user's accepted path in 32 layers
        dict(name="compact 1", op="compact", batch=1, layers=32, kv_heads=8, dim=128, page=16, length=1000, nodes=64, depth=6, fp8=False),
        # a serving batch's accepted paths, E4M3 pages
        dict(name="compact 64 fp8", op="compact", batch=64, layers=32, kv_heads=8, dim=128, page=32, length=200, nodes=63, depth=9, fp8=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "beam", "beam", "fork", "copy", "compact"])
    if op == "beam":
        batch, beams, vocab = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 100, 160000)
        while batch * beams * vocab > 32 * 8 * 128256:
            batch = (batch + 1) // 2
        return dict(op=op, batch=batch, beams=beams, k=min(rng.choice([1, beams, 2 * beams]), beams * vocab), vocab=vocab, f32=rng.random() < 0.4, done=rng.random() < 0.5,
                    first=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 5]))
    page = rng.choice([16, 32, 64, 128])
    if op == "fork":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        length = _log(rng, 1, 16384)
        rows = beams * _log(rng, 1, 512 // beams)
        while rows * length > 512 * 8100:
            length = (length + 1) // 2
        return dict(op=op, rows=rows, beams=beams, width=(length + page - 1) // page + rng.randint(1, 9), page=page, length=length, room=rng.choice([0, 1, 1, 5, 64, 300]),
                    spare=rows * 24 + _log(rng, 1, 65536), ended=rng.random() < 0.5)
    kv_heads, dim, fp8 = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.random() < 0.4
    if op == "copy":
        pairs, layers = _log(rng, 1, 2048), _log(rng, 1, 40)
        while pairs * layers * kv_heads * page * dim > 2048 * 2 * 8 * 64 * 128 // 2:
            pairs, layers = (pairs + 1) // 2, (layers + 1) // 2
        return dict(op=op, pairs=pairs, layers=layers, kv_heads=kv_heads, dim=dim, page=page, pages=2 * pairs + rng.randint(1, 40), fp8=fp8, partial=rng.random() < 0.6)
    batch = _log(rng, 1, 64)
    if op == "compact":
        nodes, layers, length = _log(rng, 1, 256), _log(rng, 1, 40), _log(rng, 1, 1000)
        while batch * (length + nodes + page) * layers * kv_heads * dim > 1 << 29:
            batch, layers = (batch + 1) // 2, (layers + 1) // 2
        return dict(op=op, batch=batch, layers=layers, kv_heads=kv_heads, dim=dim, page=page, length=length, nodes=nodes, depth=min(nodes, _log(rng, 1, 32)), fp8=fp8)
    chain, length, group = rng.random() < 0.3, _log(rng, 1, 32768), rng.choice([1, 2, 3, 4, 7, 8, 16])
    nodes = _log(rng, 1, 1024 if chain else 256)
    while batch * (length + nodes) * kv_heads * dim > 8 * 32768 * 8 * 128 // 2 or batch * (length + nodes) * nodes * kv_heads * group * dim > 8 * 32768 * 16 * 64 * 128 // 2:
        batch, length, nodes = (batch + 1) // 2, (length + 1) // 2, (nodes + 1) // 2
    return dict(op=op, batch=batch, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, length=length, nodes=nodes, chain=chain, fp8=fp8,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), ragged=rng.random() < 0.6)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    return {"tree": _prepare_tree, "beam": _prepare_beam, "fork": _prepare_fork, "copy": _prepare_copy, "compact": _prepare_compact}[case["op"]](s, g)


def _whole(g, lo, hi, shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def _pages(s, g, lead):
    shape = lead + (s["kv_heads"], s["page"], s["dim"])
    s["k_scale"] = s["v_scale"] = None
    if s["fp8"]:
        s["k_scale"] = torch.rand(s["kv_heads"], generator=g, device="cuda") * 0.02 + 0.005
        s["v_scale"] = torch.rand(s["kv_heads"], generator=g, device="cuda") * 0.02 + 0.005
    for name in ("k", "v"):
        p = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
        if s["fp8"]:
            p = (p / s[name + "_scale"].view(-1, 1, 1).to(BF16)).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name + "_pages"] = p


def _prepare_tree(s, g):
    b, t, page = s["batch"], s["nodes"], s["page"]
    per = (s["length"] + t + page - 1) // page
    s["q"] = torch.randn(b, t, s["heads"], s["dim"], generator=g, device="cuda").to(BF16)
    lens = torch.full((b,), s["length"], device="cuda")
    s["count"] = None
    if s["ragged"]:
        lens, count = _whole(g, 0, s["length"], (b,)), _whole(g, 1, t, (b,))
        if b > 3:  # a sequence without context, one of a single position, one that drafted nothing
            lens[0], lens[1], count[2] = 0, 1, 0
        s["count"] = count.to(I32)
    s["lens"] = lens.to(I32)
    depth = torch.zeros(b, t, dtype=torch.int64, device="cuda")
    s["tree"] = None
    if s["chain"]:
        depth += torch.arange(t, device="cuda")
    else:  # each node but the first hangs on an earlier one
        parent = (torch.rand(b, t, generator=g, device="cuda") * torch.arange(t, device="cuda")).long()
        reads = torch.eye(t, dtype=torch.bool, device="cuda").repeat(b, 1, 1)
        each = torch.arange(b, device="cuda")
        for i in range(1, t):
            reads[:, i] |= reads[each, parent[:, i]]
        depth = reads.sum(-1) - 1
        words = (t + 63) // 64
        bits = torch.nn.functional.pad(reads, (0, 64 * words - t)).view(b, t, words, 64).long()
        s["tree"] = (bits << torch.arange(64, device="cuda")).sum(-1)
    s["starts"] = (lens.view(b, 1) + depth + 1 - s["window"]).clamp(min=0).to(I32) if s["window"] else None
    _pages(s, g, (b * per + 1,))
    s["table"] = (torch.randperm(b * per, generator=g, device="cuda") + 1).to(I32).view(b, per)
    return s


def _prepare_beam(s, g):
    b, n, v = s["batch"], s["beams"], s["vocab"]
    x = torch.randn(b, n, v, generator=g, device="cuda") * 2.5
    x += 6 * (torch.rand(b, n, v, generator=g, device="cuda") < 20 / v)  # a few likely tokens
    s["logits"] = x if s["f32"] else x.to(BF16)
    s["scores"] = -torch.rand(b, n, generator=g, device="cuda") * 5 - 8
    if s["first"]:  # one beam of each holds the prompt
        s["scores"][:, 1:] = -math.inf
        s["scores"][:, 0] = 0
    s["ended"] = None
    if s["done"]:
        s["ended"] = torch.rand(b, n, generator=g, device="cuda") < 0.2
        s["ended"][-1] = True  # a search that is over
    return s


def _pool(case):
    """Pages of a fork's cache: what its rows hold at most, and some more."""
    most = (case["length"] + case["page"] - 1) // case["page"]
    return case["rows"] // case["beams"] * (most * 3 // 4 + case["beams"] * (most - most * 3 // 4 + 2)) + case["spare"]


def _prepare_fork(s, g):
    """Tables in which a search's beams share a prompt's pages and own what follows."""
    rows, n, width, page = s["rows"], s["beams"], s["width"], s["page"]
    groups = rows // n
    lens = _whole(g, max(1, s["length"] // 2), s["length"], (groups, 1)).expand(groups, n)  # the beams of a search are of one length
    if s["ended"] and groups > 1:
        lens = lens.clone()
        lens[0] = 0
    held = ((lens + page - 1) // page).reshape(rows, 1)
    prompt = (lens * 3 // 4 // page).reshape(rows, 1)
    at = torch.arange(width, device="cuda")
    row = torch.arange(rows, device="cuda").view(rows, 1)
    leader = row // n * n
    place = torch.where(at < prompt, leader, row) * width + at  # which (row, column) made the page
    total = _pool(s)
    names = torch.randperm(total, generator=g, device="cuda")
    used = torch.zeros(rows * width, dtype=torch.int64, device="cuda").index_fill_(0, place[at < held], 1)
    s["table"] = torch.where(at < held, names[(used.cumsum(0) - 1)[place].clamp(min=0)], -1).to(I32)
    s["lens"] = lens.reshape(rows).to(I32)
    s["refs"] = torch.zeros(total, dtype=I32, device="cuda")
    live = s["table"] >= 0
    s["refs"].scatter_add_(0, s["table"][live].long(), torch.ones(int(live.sum()), dtype=I32, device="cuda"))
    parents = leader + _whole(g, 0, n - 1, (rows, 1))
    if s["ended"]:
        parents[torch.rand(rows, 1, generator=g, device="cuda") < 0.05] = -1
    s["parents"] = parents.view(rows).to(I32)
    return s


def _prepare_copy(s, g):
    n, p = s["pairs"], s["pages"]
    _pages(s, g, (s["layers"], p))
    names = torch.randperm(p, generator=g, device="cuda")
    s["src"] = names[:p - n][_whole(g, 0, p - n - 1, (n,))].to(I32)  # pages may be copied more than once
    s["dst"] = names[p - n:].to(I32)
    s["filled"] = None
    if s["partial"]:
        s["filled"] = _whole(g, 1, s["page"] - 1, (n,)).to(I32)
        none = torch.rand(n, generator=g, device="cuda") < 0.25  # rows that kept their page
        none[0] = False
        s["src"][none], s["dst"][none], s["filled"][none] = -1, -1, 0
    return s


def _prepare_compact(s, g):
    b, page, t, d = s["batch"], s["page"], s["nodes"], s["depth"]
    per = (s["length"] + t + page - 1) // page
    _pages(s, g, (s["layers"], b * per + 1))
    s["table"] = (torch.randperm(b * per, generator=g, device="cuda") + 1).to(I32).view(b, per)
    s["lens"] = _whole(g, 0, s["length"], (b,)).to(I32)
    s["accepted"] = _whole(g, 1, d, (b,)).to(I32)
    order = torch.rand(b, t, generator=g, device="cuda")
    order[:, 0] = -1  # the first node is on every path
    s["path"] = order.argsort(-1)[:, :d].sort(-1).values.to(I32)
    return s


def run(s):
    if own:
        import huffman_decode_block_amd as df11
        if s["op"] == "tree":
            out, lse = df11.df11_paged_tree_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], tree=s["tree"], nodes=s["count"], starts=s["starts"],
                                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {"out": out, "lse": lse}
        if s["op"] == "beam":
            scores, parents, tokens = df11.df11_beam_select(s["logits"], s["scores"], s["k"], done=s["ended"], pad=s["pad"])
            return {"scores": scores, "parents": parents, "tokens": tokens}
        if s["op"] == "fork":
            src, dst, filled, missing = df11.df11_paged_fork(s["parents"], s["table"], s["lens"], s["refs"], s["page"], room=s["room"])
            return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "src": src, "dst": dst, "filled": filled, "missing": missing}
        if s["op"] == "copy":
            df11.df11_paged_copy(s["src"], s["dst"], s["k_pages"], s["v_pages"], rows=s["filled"])
        else:
            df11.df11_paged_compact(s["path"], s["accepted"], s["table"], s["lens"], s["k_pages"], s["v_pages"])
        return {"k": s["k_pages"], "v": s["v_pages"]}
    return {"tree": _tree, "beam": _beam, "fork": _fork, "copy": _copy, "compact": _compact}[s["op"]](s)


def _tree(s):
    q, table = s["q"].float(), s["table"].long()
    b, t, heads, d = q.shape
    h, page = s["kv_heads"], s["page"]
    total = table.shape[1] * page
    group = heads // h

    def gathered(pages, scale):
        p = pages.view(torch.uint8)[table].view(pages.dtype) if s["fp8"] else pages[table]
        p = p.transpose(1, 2).reshape(b, h, total, d).float()
        return p if scale is None else p * scale.view(1, -1, 1, 1)

    at = torch.arange(total, device=q.device)
    lens = s["lens"].long().view(b, 1, 1)
    context = at < lens
    if s["starts"] is not None:
        context = context & (at >= s["starts"].view(b, t, 1))
    node = at - lens  # which node a position holds
    count = t if s["count"] is None else s["count"].view(b, 1, 1)
    mine = torch.arange(t, device=q.device).view(1, t, 1)
    if s["chain"]:
        reads = node <= mine
    else:
        each = torch.arange(t, device=q.device)
        bits = (s["tree"][..., each // 64] >> (each % 64)) & 1
        reads = bits.bool().gather(2, node.clamp(0, t - 1).expand(b, t, total))
    live = ((context | ((node >= 0) & (node < count) & reads)) & (mine < count)).view(b, 1, t, 1, total).expand(b, h, t, group, total).reshape(b, h, t * group, total)
    score = (q.view(b, t, h, group, d).transpose(1, 2).reshape(b, h, t * group, d) / math.sqrt(d)) @ gathered(s["k_pages"], s["k_scale"]).transpose(-1, -2)
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)  # a row with no position
    p = torch.exp(score - top)
    total_p = p.sum(-1, keepdim=True)
    out = (p / torch.where(total_p == 0, torch.ones_like(total_p), total_p)) @ gathered(s["v_pages"], s["v_scale"])
    lse = torch.log(total_p) + top
    return {"out": out.view(b, h, t, group, d).transpose(1, 2).reshape(b, t, heads, d).to(BF16), "lse": lse.view(b, h, t, group).transpose(1, 2).reshape(b, t, heads)}


def _beam(s):
    x = s["logits"].double()  # scores of different beams may lie next to each other
    b, n, v = x.shape
    top = x.amax(-1, keepdim=True)
    score = s["scores"].double().view(b, n, 1) + (x - (torch.log(torch.exp(x - top).sum(-1, keepdim=True)) + top))
    if s["ended"] is not None:  # an ended beam goes on as it is
        ended = s["ended"].view(b, n, 1)
        score = torch.where(ended, torch.where(torch.arange(v, device=x.device) == s["pad"], s["scores"].double().view(b, n, 1), -math.inf), score)
    score = torch.where(score.isnan(), -math.inf, score)
    best, at = torch.sort(score.view(b, n * v), dim=-1, descending=True, stable=True)
    best, at = best[:, :s["k"]], at[:, :s["k"]]
    some = best > -math.inf
    parents = torch.where(some, at // v + n * torch.arange(b, device=x.device).view(b, 1), -1)
    return {"scores": best.float(), "parents": parents.to(I32), "tokens": torch.where(some, at % v, s["pad"]).to(I32)}


def _fork(s):
    table, refs, page = s["table"].long(), s["refs"], s["page"]
    rows, width = table.shape
    pool = refs.shape[0]
    parents, row, at = s["parents"].long(), torch.arange(rows, device=table.device), torch.arange(width, device=table.device)
    real = (parents >= 0) & (parents < rows)
    of = parents.clamp(0, rows - 1)
    lens = torch.where(real, s["lens"].long()[of], 0).clamp(0, width * page)
    old = table[of]
    held = (old >= 0) & (old < pool)
    full, part = lens // page, lens % page
    need = torch.where(real, ((lens + s["room"] + page - 1) // page).clamp(max=width), 0)
    first = torch.full((rows,), rows, device=table.device).scatter_reduce(0, of, torch.where(real, row, rows), "amin")[of] == row
    shares = at < full.view(rows, 1)
    writes = (at < need.view(rows, 1)) & ~shares
    keeps = writes & first.view(rows, 1) & held & (refs[old.clamp(0, pool - 1)] <= 1)
    takes = writes & ~keeps
    free = refs == 0
    order = torch.argsort((~free).to(torch.uint8), stable=True)  # free pages first, by their numbers
    turn = takes.view(-1).cumsum(0).view(rows, width) - 1
    n_free = free.sum()
    got = torch.where(turn < n_free, order[turn.clamp(0, pool - 1)], -1)
    new = torch.where((shares & held) | keeps, old, torch.where(takes, got, -1))
    one = full.clamp(max=width - 1).view(rows, 1)
    copies = ((part > 0).view(rows, 1) & takes.gather(1, one) & held.gather(1, one) & (got.gather(1, one) >= 0)).view(rows)
    src = torch.where(copies, old.gather(1, one).view(rows), -1)
    dst = torch.where(copies, got.gather(1, one).view(rows), -1)
    for_all = torch.zeros(pool + 1, dtype=I32, device=table.device)  # the last one for entries that name no page
    was = torch.where((table >= 0) & (table < pool), table, pool)
    now = torch.where(new >= 0, new, pool)
    ones = torch.ones(rows * width, dtype=I32, device=table.device)
    refs += for_all.scatter_add(0, now.view(-1), ones).scatter_add(0, was.view(-1), -ones)[:pool]
    s["table"].copy_(new)
    s["lens"].copy_(lens)
    return {"table": s["table"], "lens": s["lens"], "refs": refs, "src": src.to(I32), "dst": dst.to(I32), "filled": torch.where(copies, part, 0).to(I32),
            "missing": (takes & (turn >= n_free)).sum().to(I32).view(1)}


def _copy(s):
    src, dst, filled = s["src"].long(), s["dst"].long(), s["filled"]
    if s["partial"]:
        real = src >= 0
        src, dst, filled = src[real], dst[real], filled[real]
    return {"k": _copied(s["k_pages"], s, src, dst, filled), "v": _copied(s["v_pages"], s, src, dst, filled)}


def _copied(pages, s, src, dst, filled):
    raw = pages.view(torch.uint8) if s["fp8"] else pages
    new = raw[:, src]
    if filled is not None:
        new = torch.where(torch.arange(s["page"], device=raw.device).view(1, 1, 1, -1, 1) < filled.view(1, -1, 1, 1, 1), new, raw[:, dst])
    raw[:, dst] = new
    return pages


def _compact(s):
    b, d = s["path"].shape
    each = torch.arange(d, device=s["path"].device)
    moves = each < s["accepted"].view(b, 1)
    lens, row = s["lens"].long().view(b, 1), torch.arange(b, device=each.device).view(b, 1).expand(b, d)[moves]
    src, dst = (lens + s["path"].long())[moves], (lens + each)[moves]
    table, page = s["table"].long(), s["page"]
    src_page, dst_page = table[row, src // page], table[row, dst // page]
    return {"k": _compacted(s["k_pages"], s, src_page, src % page, dst_page, dst % page), "v": _compacted(s["v_pages"], s, src_page, src % page, dst_page, dst % page)}


def _compacted(pages, s, src_page, src, dst_page, dst):
    raw = pages.view(torch.uint8) if s["fp8"] else pages
    raw[:, dst_page, :, dst] = raw[:, src_page, :, src]
    return pages


def work(case):
    size = 1 if case.get("fp8") else 2
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        n = rows * case["vocab"] * (0.8 if case["done"] else 1) / (case["beams"] if case["first"] else 1)  # rows that are searched
        return {"bytes": n * (4 if case["f32"] else 2) + rows * 5 + case["batch"] * case["k"] * 12, "flops": 4 * n}
    if case["op"] == "fork":
        held = case["rows"] * max(1, case["length"] * 3 // 4 // case["page"])  # entries read and written; a quarter of them name pages whose counts change
        return {"bytes": 8 * held + 4 * held + 24 * case["rows"], "flops": 2 * held}
    if case["op"] == "copy":
        pairs = case["pairs"] * (0.375 if case["partial"] else 1)  # three quarters of the rows, half a page each
        return {"bytes": max(1, pairs) * 4 * case["layers"] * case["kv_heads"] * case["page"] * case["dim"] * size + 12 * case["pairs"], "flops": 0}
    if case["op"] == "compact":
        moved = case["batch"] * (case["depth"] + 1) / 2
        return {"bytes": moved * 4 * case["layers"] * case["kv_heads"] * case["dim"] * size + 8 * case["batch"] * case["depth"], "flops": 0}
    b, t, hd = case["batch"], case["nodes"], case["kv_heads"] * case["dim"]
    length = case["length"] / (2 if case["ragged"] else 1)
    nodes = (t + 1) / 2 if case["ragged"] else t
    seen = min(length, case["window"] + (nodes if case["chain"] else 0)) if case["window"] else length  # positions that some node reads
    each = min(length, case["window"]) if case["window"] else length  # and one node
    up = (nodes + 1) / 2 if case["chain"] else math.log(nodes + 1) + 1  # nodes above a node, and itself
    rows = b * t * case["heads"]
    return {"bytes": b * (seen + nodes) * 2 * hd * size + rows * (4 * case["dim"] + 4), "flops": 4 * b * nodes * case["heads"] * (each + up) * case["dim"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fork":
        return None  # whole numbers only
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "beam":
        return _exact_beam(s)
    out = {}
    for name in ("k", "v"):
        pages = s[name + "_pages"].to(F64)
        if case["op"] == "copy":
            for i, (a, b) in enumerate(zip(s["src"].tolist(), s["dst"].tolist())):
                n = s["page"] if s["filled"] is None else int(s["filled"][i])
                if a >= 0:
                    pages[:, b, :, :n] = pages[:, a, :, :n]
        else:
            for i, (lo, n) in enumerate(zip(s["lens"].tolist(), s["accepted"].tolist())):
                path, table = s["path"][i].tolist(), s["table"][i].tolist()
                for j in range(n):  # a path ascends: no row is overwritten before it has moved
                    a, b = lo + path[j], lo + j
                    pages[:, table[b // s["page"]], :, b % s["page"]] = pages[:, table[a // s["page"]], :, a % s["page"]]
        out[name] = pages
    return out


def _exact_beam(s):
    """The scores; which beam and token they belong to are whole numbers."""
    b, n, v = s["logits"].shape
    best = torch.full((b, s["k"]), -math.inf, dtype=F64, device="cuda")
    for i in range(b):
        found = []
        for j in range(n):
            if s["ended"] is not None and bool(s["ended"][i, j]):
                found.append(s["scores"][i, j].double().view(1))
            else:
                found.append(s["scores"][i, j].double() + torch.log_softmax(s["logits"][i, j].double(), 0))
        top = torch.sort(torch.cat(found), descending=True).values[:s["k"]]
        best[i, :len(top)] = top
    return {"scores": best, "parents": None, "tokens": None}


def _exact_tree(s):
    b, t, heads, d = s["q"].shape
    h, page = s["kv_heads"], s["page"]
    group = heads // h
    out = torch.zeros(b, t, heads, d, dtype=F64, device="cuda")
    lse = torch.full((b, t, heads), -math.inf, dtype=F64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        nodes = t if s["count"] is None else int(s["count"][i])
        if nodes == 0:
            continue
        at = torch.arange(n + nodes, device="cuda")
        where, row = s["table"][i].long()[at // page], at % page
        reads = torch.zeros(nodes, n + nodes, dtype=torch.bool, device="cuda")
        for j in range(nodes):
            reads[j, 0 if s["starts"] is None else min(n, int(s["starts"][i, j])):n] = True
            if s["chain"]:
                reads[j, n:n + j + 1] = True
        if not s["chain"]:
            each = torch.arange(nodes, device="cuda")
            reads[:, n:] = (s["tree"][i, :nodes][:, each // 64] >> (each % 64)) % 2 != 0
        for j in range(h):
            mine = slice(j * group, (j + 1) * group)
            k, v = (s[x + "_pages"][:, j].view(torch.uint8 if s["fp8"] else BF16)[where, row].view(s[x + "_pages"].dtype).to(F32).double() for x in ("k", "v"))
            if s["fp8"]:
                k, v = k * float(s["k_scale"][j]), v * float(s["v_scale"][j])
            score = (s["q"][i, :nodes, mine].double().reshape(nodes * group, d) @ k.T.contiguous() * d ** -0.5).view(nodes, group, -1)
            score = score.masked_fill(~reads.view(nodes, 1, -1), -math.inf)
            lse[i, :nodes, mine] = torch.logsumexp(score, -1)
            out[i, :nodes, mine] = (torch.softmax(score, -1).view(nodes * group, -1) @ v).view(nodes, group, d)
    return {"out": out, "lse": lse}
