"""Cases for timing and checking the operators of a token step that read the library's other two stores.

Operators:
  quantize   BF16 weights to microscaled 4-bit floating point (E2M1 codes, one power-of-two scale for 32
             values) and back to BF16, the round trip a converter of checkpoints makes
  matmul     BF16 activations times 4-bit weights, from one token to a prompt
  append     new keys and values into the pages of a cache (BF16, or E4M3 with a scale for each head)
  attention  one new token for each sequence against its pages

`run` computes them from elementary torch operations in 32 bits, or with `own` set through the library.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # one attention projection of a Llama-3.1-8B-shaped block converted
        dict(name="mx4 quantize 4096x4096", op="quantize", rows=4096, cols=4096, pad=0),
        # a matrix whose rows end inside a block and start off 16 bytes, as an odd-sized head or adapter has
        dict(name="mx4 quantize 9001x1387", op="quantize", rows=9001, cols=1387, pad=2),
        # one token through one attention projection: the smallest product of a token step
        dict(name="mx4 matmul 1 token", op="matmul", m=1, n=4096, k=4096, pad=0),
        # sixteen sequences' tokens through a gate projection
        dict(name="mx4 matmul 16 tokens", op="matmul", m=16, n=14336, k=4096, pad=0),
        # a short ragged batch on sizes that no tile divides, rows of x not next to each other
        dict(name="mx4 matmul 77 ragged", op="matmul", m=77, n=2057, k=1990, pad=6),
        # a prompt of 2,048 tokens through a gate projection
        dict(name="mx4 matmul 2048 prompt", op="matmul", m=2048, n=14336, k=4096, pad=0),
        # the new token of thirty-two sequences
        dict(name="append 32 tokens", op="append", tokens=32, kv_heads=8, dim=128, page=16, pages=4096, fp8=False, padding=False),
        # a prompt's keys and values into E4M3 pages, some rows padding
        dict(name="append 8192 prompt fp8", op="append", tokens=8192, kv_heads=8, dim=128, page=64, pages=2048, fp8=True, padding=True),
        # a single user at 8,192 tokens of context, 8B-shaped heads
        dict(name="attention 1x8192", op="attention", batch=1, heads=32, kv_heads=8, dim=128, page=16, length=8192, fp8=False, window=0, ragged=False),
        # a serving batch with lengths from none to 1,024
        dict(name="attention 64 ragged", op="attention", batch=64, heads=32, kv_heads=8, dim=128, page=16, length=1024, fp8=False, window=0, ragged=True),
        # long contexts, 70B-shaped heads, E4M3 pages
        dict(name="attention 8x32768 fp8", op="attention", batch=8, heads=64, kv_heads=8, dim=128, page=64, length=32768, fp8=True, window=0, ragged=False),
        # a sliding window over wide heads, pages that end inside the window
        dict(name="attention 16x window", op="attention", batch=16, heads=8, kv_heads=4, dim=256, page=32, length=5003, fp8=False, window=1024, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "append", "attention", "attention"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 16384), _log(rng, 1, 16384)
        while rows * cols > 14336 * 4096:
            rows = (rows + 1) // 2
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8]))
    if op == "matmul":
        n, k = _log(rng, 16, 16384), _log(rng, 16, 16384)
        if rng.random() < 0.6:  # most real sizes are whole blocks
            n, k = (n + 31) // 32 * 32, (k + 31) // 32 * 32
        m = _log(rng, 1, 4096)
        while m * n * k > 2048 * 14336 * 4096 or m * n > 2048 * 14336:
            m = (m + 1) // 2
        return dict(op=op, m=m, n=n, k=k, pad=rng.choice([0, 0, 3, 8]))
    kv_heads, dim, page, fp8 = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128]), rng.random() < 0.4
    if op == "append":
        tokens = _log(rng, 1, 16384)
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, page=page, pages=(tokens + page - 1) // page + rng.randint(1, 64), fp8=fp8, padding=rng.random() < 0.5)
    batch, length = _log(rng, 1, 128), _log(rng, 1, 65536)
    while batch * length * kv_heads * dim > 8 * 32768 * 8 * 128 // 2:
        batch, length = (batch + 1) // 2, (length + 1) // 2
    return dict(op=op, batch=batch, heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16]), kv_heads=kv_heads, dim=dim, page=page, length=length, fp8=fp8,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), ragged=rng.random() < 0.6)


def _rows(g, rows, cols, pad, scale):
    """BF16 rows with a scale of their own each, `pad` values of something else behind every row."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    u = torch.rand(rows, 1, generator=g, device="cuda") * 1.5 + 0.5
    return (x * u * scale).to(BF16)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantize":
        x = _rows(g, case["rows"], case["cols"], case["pad"], 0.02)
        x[:, : max(1, case["cols"] // 50)] *= 16  # outlier columns
        x[:: 97] = 0  # rows that were pruned
        s["x"] = x
    elif case["op"] == "matmul":
        s["x"] = _rows(g, case["m"], case["k"], case["pad"], 1.0)
        s["codes"], s["scales"] = _encode(_rows(g, case["n"], case["k"], 0, 0.02))
    elif case["op"] == "append":
        t, h, d, n = case["tokens"], case["kv_heads"], case["dim"], case["pages"] * case["page"]
        kv = torch.randn(t, 2 * h + 4, d, generator=g, device="cuda").to(BF16)  # as the joint projection leaves them
        s["k"], s["v"] = kv[:, :h], kv[:, h:2 * h]
        s["slots"] = torch.randperm(n, generator=g, device="cuda")[:t]
        if case["padding"]:
            s["slots"][torch.rand(t, generator=g, device="cuda") < 0.1] = -1
        _pages(s, case, g, case["pages"])
    else:
        b, page = case["batch"], case["page"]
        per = (case["length"] + page - 1) // page
        s["q"] = torch.randn(b, case["heads"], case["dim"], generator=g, device="cuda").to(BF16)
        lens = torch.full((b,), case["length"], device="cuda")
        if case["ragged"]:
            lens = (torch.rand(b, generator=g, device="cuda") * (case["length"] + 1)).long()
            if b > 3:
                lens[0], lens[1] = 0, 1
        s["lens"] = lens.int()
        s["starts"] = (lens - case["window"]).clamp(min=0).int() if case["window"] else None
        _pages(s, case, g, b * per + 1)
        s["table"] = (torch.randperm(b * per, generator=g, device="cuda") + 1).int().view(b, per)
    return s


def _pages(s, case, g, pages):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    s["k_scale"] = s["v_scale"] = None
    if case["fp8"]:
        s["k_scale"] = torch.rand(case["kv_heads"], generator=g, device="cuda") * 0.02 + 0.005
        s["v_scale"] = torch.rand(case["kv_heads"], generator=g, device="cuda") * 0.02 + 0.005
    for name in ("k", "v"):
        p = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
        if case["fp8"]:
            p = (p / s[name + "_scale"].view(1, -1, 1, 1).to(BF16)).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name + "_pages"] = p


def run(s):
    if own:
        import huffman_decode_block_amd as df11
        if s["op"] == "quantize":
            codes, scales = df11.df11_mx4_quantize(s["x"])
            return {"values": df11.df11_mx4_dequantize(codes, scales, s["cols"]), "scales": scales}
        if s["op"] == "matmul":
            return df11.df11_mx4_matmul(s["x"], s["codes"], s["scales"])
        if s["op"] == "append":
            df11.df11_paged_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
            return {"k": s["k_pages"], "v": s["v_pages"]}
        out, lse = df11.df11_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], starts=s["starts"],
                                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if s["op"] == "quantize":
        codes, scales = _encode(s["x"])
        return {"values": _decode(codes, scales, s["cols"]).to(BF16), "scales": scales}
    if s["op"] == "matmul":
        return (s["x"].float() @ _decode(s["codes"], s["scales"], s["k"]).T).to(BF16)
    if s["op"] == "append":
        slots, k, v = s["slots"], s["k"], s["v"]
        if s["padding"]:
            real = slots >= 0
            slots, k, v = slots[real], k[real], v[real]
        at, row = slots // s["page"], slots % s["page"]
        for new, pages, scale in ((k, s["k_pages"], s["k_scale"]), (v, s["v_pages"], s["v_scale"])):
            if s["fp8"]:
                new = (new.float() / scale.view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                pages.view(torch.uint8)[at, :, row] = new.view(torch.uint8)
            else:
                pages[at, :, row] = new
        return {"k": s["k_pages"], "v": s["v_pages"]}
    return _attention(s)


def _pow2(e):
    """2^e in 32 bits for whole e in [-127, 127], from its bits (a power function need not be exact)."""
    normal = ((e + 127).clamp(min=1) << 23).view(F32)
    return torch.where(e < -126, 0.5 * normal, normal)


def _encode(x):
    """Codes [rows, 16 * blocks] (even columns in the low halves of the bytes) and scale bytes [rows, blocks]."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    v = torch.nn.functional.pad(x.float(), (0, 32 * blocks - cols)).view(rows, blocks, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    a = (v * _pow2(-e)).abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; halfway to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(rows, 16 * blocks, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8).view(rows, blocks)


def _decode(codes, scales, cols):
    """32-bit values of codes and scale bytes."""
    rows, blocks = scales.shape
    c = torch.stack((codes & 15, codes >> 4), -1).view(rows, blocks, 32)
    low, exp = (c & 1).float(), ((c >> 1) & 3).int()
    mag = torch.where(exp == 0, 0.5 * low, (1 + 0.5 * low) * _pow2(exp - 1))
    v = torch.where(c >= 8, -mag, mag)
    return (v * _pow2(scales.int() - 127).unsqueeze(-1)).view(rows, 32 * blocks)[:, :cols]


def _attention(s):
    q, table, lens = s["q"].float(), s["table"].long(), s["lens"].view(-1, 1, 1, 1)
    b, heads, d = q.shape
    h, page = s["kv_heads"], s["page"]
    total = table.shape[1] * page

    def gathered(pages, scale):
        p = pages.view(torch.uint8)[table].view(pages.dtype) if s["fp8"] else pages[table]
        p = p.transpose(1, 2).reshape(b, h, total, d).float()
        return p if scale is None else p * scale.view(1, -1, 1, 1)

    at = torch.arange(total, device=q.device)
    live = at < lens
    if s["starts"] is not None:
        live = live & (at >= s["starts"].view(-1, 1, 1, 1))
    score = (q.view(b, h, heads // h, d) / math.sqrt(d)) @ gathered(s["k_pages"], s["k_scale"]).transpose(-1, -2)
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)  # a row with no position
    p = torch.exp(score - top)
    total_p = p.sum(-1, keepdim=True)
    out = (p / torch.where(total_p == 0, torch.ones_like(total_p), total_p)) @ gathered(s["v_pages"], s["v_scale"])
    return {"out": out.reshape(b, heads, d).to(BF16), "lse": (torch.log(total_p) + top).view(b, heads)}


def _live(s):
    """Positions that attention reads, over all sequences of a case, on average of its draws."""
    total = s["batch"] * s["length"]
    if s["ragged"]:
        total //= 2
    return min(total, s["batch"] * s["window"]) if s["window"] else total


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n + 2 * n + 2 * (n / 2 + n / 32), "flops": 2 * n}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k * 17 / 32 + 2 * m * n, "flops": 2 * m * n * k}
    size = 1 if case["fp8"] else 2
    if case["op"] == "append":
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": n * (2 + size) + 8 * case["tokens"], "flops": n}
    live, hd = _live(case), case["kv_heads"] * case["dim"]
    rows = case["batch"] * case["heads"]
    return {"bytes": max(1, live) * 2 * hd * size + rows * (4 * case["dim"] + 4), "flops": 4 * live * case["heads"] * case["dim"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_round_trip(s["x"])
    if case["op"] == "matmul":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device="cuda")
        c = s["codes"].long()
        w = torch.empty(case["n"], 2 * c.shape[1], dtype=F64, device="cuda")
        for half in (0, 1):
            nib = (c >> (4 * half)) & 15
            w[:, half::2] = grid[nib & 7] * (1 - 2 * (nib >> 3))
        w *= _exact_pow2(s["scales"].long() - 127).repeat_interleave(32, dim=1)
        return s["x"].double() @ w[:, : case["k"]].T.contiguous()
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            pages, new, scale = s[name + "_pages"], s[name], s[name + "_scale"]
            want = pages.to(F64)
            if scale is not None:
                # E4M3 of the 32-bit quotient, by its own grid: 8 steps to a power of two, 2^-9 the smallest
                v = (new.float() / scale.view(1, -1, 1)).double().clamp(-448, 448)
                step = _exact_pow2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.long() - 4)
                new = torch.round(v / step) * step
            t = torch.nonzero(s["slots"] >= 0).flatten()
            at = s["slots"][t]
            want[at // case["page"], :, at % case["page"]] = new.double()[t]
            out[name] = want
        return out
    b, heads, d, h = case["batch"], case["heads"], case["dim"], case["kv_heads"]
    out = torch.zeros(b, heads, d, dtype=F64, device="cuda")
    lse = torch.full((b, heads), -math.inf, dtype=F64, device="cuda")
    first = s["starts"].tolist() if s["starts"] is not None else [0] * b
    for i, (lo, hi) in enumerate(zip(first, s["lens"].tolist())):
        if hi <= lo:
            continue
        at = torch.arange(lo, hi, device="cuda")
        page, row = s["table"][i].long()[at // case["page"]], at % case["page"]
        for j in range(h):
            mine = slice(j * (heads // h), (j + 1) * (heads // h))
            k, v = (_wide(s[n + "_pages"], j, page, row, s[n + "_scale"]) for n in ("k", "v"))
            score = s["q"][i, mine].double() @ k.T.contiguous() * d ** -0.5
            lse[i, mine] = torch.logsumexp(score, -1)
            out[i, mine] = torch.softmax(score, -1) @ v
    return {"out": out, "lse": lse}


def _wide(pages, head, page, row, scale):
    flat = pages[:, head].view(torch.uint8)[page, row].view(pages.dtype).to(F32).double()
    return flat if scale is None else flat * float(scale[head])


def _exact_pow2(e):
    """2^e in 64 bits for whole e, exactly."""
    return ((e + 1023) << 52).view(F64)


def _exact_round_trip(x):
    """Each block's values on the 4-bit grid under its power of two, from the definition: the nearest grid value, of two as near the even code."""
    rows, cols = x.shape
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device="cuda")
    values = torch.empty(rows, cols, dtype=F64, device="cuda")
    blocks = (cols + 31) // 32
    scales = torch.empty(rows, blocks, dtype=torch.uint8, device="cuda")
    for at in range(blocks):
        v = x[:, 32 * at: 32 * at + 32].double()
        a = v.abs().amax(1)
        e = torch.where(a > 0, torch.frexp(a).exponent.long() - 1 - 2, -127).clamp(-127, 127)
        unit = _exact_pow2(e).unsqueeze(1)
        m = (v.abs() / unit).clamp(max=6)
        lo = torch.searchsorted(grid, m.contiguous(), right=True) - 1
        hi = (lo + 1).clamp(max=7)
        mid = (grid[lo] + grid[hi]) / 2
        up = (m > mid) | ((m == mid) & (hi % 2 == 0))
        values[:, 32 * at: 32 * at + 32] = torch.sign(v) * torch.where(up, grid[hi], grid[lo]) * unit
        scales[:, at] = (e + 127).to(torch.uint8)
    return {"values": values, "scales": scales}
