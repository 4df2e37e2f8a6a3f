"""GPU checks of the beam search's selection: which beams and tokens are chosen
and their scores, against 64 bits.

A term exp(-d) of the sum is off by at most (1.5 d + 2) 2^-23 of itself (d, its
product with log2 e and the exponential rounded in 32 bits), where the mean of d
over the softmax is below 12 for these vocabularies, and 64 terms of a lane and
the joins of a workgroup add at most 20 roundings of 2^-24 (sums of eight go in
pairs): the logarithm is off by less than 2^-18.  A score is rounded once to 32
bits: |score - ref| <= 2^-18 + 2^-24 |ref|.  Candidates of different beams may
change places where they lie closer than twice that; those of one beam may not.
Where none lie so close the choice has to be the same, place by place."""
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


def reference(logits, scores, k, done, pad):
    """Scores, parents and tokens in 64 bits; each beam's offers, best first; how near chosen ones of different beams lie."""
    batch, beams, vocab = logits.shape
    best, parents, tokens = np.full((batch, k), -np.inf), np.full((batch, k), -1), np.full((batch, k), pad)
    near, offers = np.inf, {}
    for b in range(batch):
        found = []
        for i in range(beams):
            s, mine = float(scores[b, i]), []
            if np.isfinite(s):
                if done is not None and done[b, i]:
                    mine = [(-s, i, 0.0, pad)]
                else:
                    x = logits[b, i].astype(np.float64)
                    if not (np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all()):
                        top = x.max()
                        lse = math.log(np.exp(x - top).sum()) + top
                        order = np.lexsort((np.arange(vocab), -x))[:k + 1]
                        mine = [(-(s + (x[t] - lse)), i, -x[t], int(t)) for t in order if x[t] > -np.inf]
            offers[b * beams + i] = mine
            found += mine
        found.sort()
        for j, (m, i, _, t) in enumerate(found[:k]):
            best[b, j], parents[b, j], tokens[b, j] = -m, b * beams + i, t
        for u, w in zip(found[:k], found[1:k + 1]):
            if u[1] != w[1]:
                near = min(near, w[0] - u[0])
    return best, parents, tokens, offers, near


def check(torch, logits, scores, k, done=None, pad=0, equal=False, **more):
    """equal: beams are the same to the last bit, their order is that of their numbers."""
    want, parents, tokens, offers, near = reference(logits.float().cpu().numpy(), scores.cpu().numpy(), k, None if done is None else done.cpu().numpy(), pad)
    got = hdb.df11_beam_select(logits, scores, k, done=done, pad=pad, **more)
    torch.cuda.synchronize()
    s, got_parents, got_tokens = got[0].double().cpu().numpy(), got[1].cpu().numpy(), got[2].cpu().numpy()
    some = np.isfinite(want)
    bound = 2.0 ** -18 + 2.0 ** -24 * np.abs(np.where(some, want, 0))
    assert np.array_equal(np.isneginf(s), ~some)
    assert (np.abs(s - want)[some] <= bound[some]).all()
    if equal or near > 2 * bound.max():
        assert np.array_equal(got_parents, parents)
        assert np.array_equal(got_tokens, tokens)
        return got
    beams = logits.shape[1]
    for b in range(logits.shape[0]):
        taken = {}
        for j in range(k):
            row = int(got_parents[b, j])
            assert (row >= 0) == bool(some[b, j])
            if row < 0:
                assert got_tokens[b, j] == pad
                continue
            assert row // beams == b
            m, _, _, t = offers[row][taken.get(row, 0)]  # each beam's in their order
            taken[row] = taken.get(row, 0) + 1
            assert t == got_tokens[b, j] and abs(s[b, j] + m) <= bound[b, j]
    return got


def make(torch, batch, beams, vocab, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(batch, beams, vocab, generator=g, device="cuda") * 160).round() / 64
    scores = -torch.rand(batch, beams, generator=g, device="cuda") * 5 - 1
    return x.to(dtype), scores


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("batch,beams,vocab,k", [
    (1, 1, 1, 1), (2, 3, 2, 4), (1, 4, 7, 8), (3, 2, 63, 5), (2, 5, 100, 64), (1, 4, 511, 4), (2, 2, 513, 16), (1, 3, 2047, 64), (2, 4, 2049, 8),
    (1, 4, 32000, 4), (3, 5, 32003, 10), (2, 16, 9001, 32), (1, 64, 1000, 64), (70, 8, 4100, 16), (1, 2, 128256, 64), (33, 8, 50001, 1), (1, 1000, 33, 20),
])
def test_sizes(torch, f32, batch, beams, vocab, k):
    say(f"beam {batch}x{beams} of {vocab}, best {k}, f32={f32}")
    x, s = make(torch, batch, beams, vocab, torch.float32 if f32 else torch.bfloat16, seed=vocab)
    check(torch, x, s, k)
    g = torch.Generator(device="cuda").manual_seed(2)
    done = torch.rand(batch, beams, generator=g, device="cuda") < 0.4
    check(torch, x, s, k, done=done, pad=min(3, vocab - 1))
    check(torch, x, s, k, done=torch.ones_like(done).to(torch.uint8), pad=-1)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vocab", [300, 5000, 40000])
def test_ties(torch, f32, vocab):
    """Equal logits by the thousand: of one beam the lowest tokens, of equal beams the lowest beam."""
    say(f"ties in {vocab}, f32={f32}")
    dtype = torch.float32 if f32 else torch.bfloat16
    x = torch.zeros(2, 3, vocab, dtype=dtype, device="cuda")
    s = torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -3.0]], device="cuda")
    check(torch, x, s, 64, equal=True)
    x[:, 1, vocab // 2:] = 1.0  # more than there are places for, and ties behind them
    x[0, 2, -1] = 2.0
    check(torch, x, s, 64, equal=True)
    x, s = make(torch, 2, 3, vocab, dtype)
    x = (x / 4).round() * 4
    check(torch, x, s, 40)


def test_equal_beams(torch):
    """Searches whose beams are the same: every score in all of them, the lower beam first."""
    say("equal beams")
    x, s = make(torch, 2, 1, 3001, torch.bfloat16)
    check(torch, x.expand(2, 4, 3001), s.expand(2, 4).contiguous(), 20, equal=True)


@pytest.mark.parametrize("f32", [False, True])
def test_masked_tokens_and_beams(torch, f32):
    """-infinity in nearly all, all and scattered tokens, NaN, infinity, the first step's scores, places left over."""
    say(f"masked tokens f32={f32}")
    x, s = make(torch, 6, 4, 33000, torch.float32 if f32 else torch.bfloat16)
    inf = math.inf
    keep = torch.zeros(33000, dtype=torch.bool, device="cuda")
    keep[::1100] = True
    x[0, :, ~keep] = -inf
    x[1, 1] = -inf
    x[1, 2, 17] = math.nan
    x[1, 3, 32999] = inf
    x[2] = -inf
    x[2, 3, 20] = 1.0
    s[3] = torch.tensor([0.0, -inf, -inf, -inf], device="cuda")
    s[4] = torch.tensor([math.nan, inf, -inf, -3.0], device="cuda")
    x[5, 0] = math.nan
    x[5, 1] = inf
    x[5, 2] = -inf
    x[5, 3] = -inf
    for k in (1, 8, 64):
        check(torch, x, s, k, pad=9)
    lanes = torch.full((1, 1, 16384), -inf, device="cuda")  # few of a wave's lanes hold anything, and those hold much
    lanes.view(1, 1, 8, 256, 8)[:, :, :, ::5] = torch.randn(1, 1, 8, 52, 8, device="cuda")
    check(torch, lanes, torch.zeros(1, 1, device="cuda"), 64)


def test_extreme_values(torch):
    """Logits of thousands, spread beyond what exponentials hold, next to each other in 32 bits; far scores."""
    say("extreme logits")
    x, s = make(torch, 2, 3, 5000, torch.float32)
    check(torch, x * 1000, s, 16)
    check(torch, x - 20000, s, 16)
    check(torch, x * 1e30, s, 3)
    y = torch.arange(5000, device="cuda").flip(0) * 2.0 ** -20 + 1
    y = torch.stack([y, y + 3, y - 5]).expand(2, 3, 5000).contiguous()
    check(torch, y, torch.tensor([[-1.0, -20.0, -40.0], [-60.0, -30.0, -9.0]], device="cuda"), 20)
    check(torch, x, s * 1e6, 16)


def test_strides_and_alignment(torch):
    say("strided logits")
    for dtype in (torch.float32, torch.bfloat16):
        x, s = make(torch, 2, 3, 5003, dtype)
        want = check(torch, x, s, 8)
        wide = torch.full((3, 2, 5011), math.nan, dtype=dtype, device="cuda")
        wide[:, :, 1:5004] = x.transpose(0, 1)
        got = check(torch, wide[:, :, 1:5004].transpose(0, 1), s, 8)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_and_graphs(torch):
    say("beam in a graph")
    x, s = make(torch, 3, 4, 32000, torch.bfloat16)
    want = check(torch, x, s, 8)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [hdb.df11_beam_select(x, s, 8, stream=side) for side in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    done = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = hdb.df11_beam_select(x, s, 8, done=done, pad=2)
    for step in range(4):
        x.copy_(x.roll(7, -1))
        s.sub_(0.37)
        done[step % 3, step] = True
        graph.replay()
        torch.cuda.synchronize()
        eager = check(torch, x, s, 8, done=done, pad=2)
        assert all(torch.equal(a, b) for a, b in zip(held, eager))


def test_refusals(torch):
    say("beam refusals")
    x, s = make(torch, 2, 3, 100, torch.bfloat16)
    for bad in ((x.half(), s), (x, s.double()), (x.cpu(), s), (x, s.cpu())):
        with pytest.raises(TypeError):
            hdb.df11_beam_select(*bad, 4)
    for bad in ((x[0], s), (x, s[:1]), (x, s[0]), (x.transpose(1, 2), s), (x.clone().requires_grad_(), s), (x, s.clone().requires_grad_())):
        with pytest.raises(ValueError):
            hdb.df11_beam_select(*bad, 4)
    for k in (0, 65, -1):
        with pytest.raises(ValueError):
            hdb.df11_beam_select(x, s, k)
    with pytest.raises(ValueError):
        hdb.df11_beam_select(x, s, 4, done=torch.zeros(2, 4, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError):
        hdb.df11_beam_select(x, s, 4, done=torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        hdb.df11_beam_select(x, s, 4, pad=1 << 31)
    with pytest.raises(hdb.DF11Error) as e:
        hdb.df11_beam_select(x, s, 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == hdb.DF11_E_BUFFER_TOO_SMALL
    with pytest.raises(hdb.DF11Error):
        hdb.df11_beam_select(x[:, :, :0], s, 4)
    assert hdb.df11_beam_select(x[:0], s[:0], 4)[1].shape == (0, 4)


@pytest.mark.parametrize("batch,beams,vocab", [(1, 16, 160000), (1, 64, 32000), (1, 4, 128256), (32, 8, 128256), (64, 4, 50000)])
def test_many_continuations_are_not_sought_one_by_one(torch, batch, beams, vocab):
    """64 continuations take at most ten times as long as 8 of the same logits, also 32, of which a workgroup's threads
    are a multiple: sought one after the other they took up to 170 times as long."""
    say(f"beam {batch}x{beams} of {vocab}: time by k")
    x, s = make(torch, batch, beams, vocab, torch.bfloat16, seed=3)
    took = {}
    for k in (8, 32, 64):
        for _ in range(2):
            hdb.df11_beam_select(x, s, k)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                hdb.df11_beam_select(x, s, k)
        times = []
        for _ in range(7):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        took[k] = sorted(times)[3]
    assert took[32] <= 10 * took[8] and took[64] <= 10 * took[8], took


@pytest.mark.parametrize("k", [1, 8, 16, 32, 33, 64])
@pytest.mark.parametrize("batch,beams,vocab", [(2, 3, 20000), (1, 16, 70001), (1, 300, 9000), (2, 1000, 300), (3, 2, 700)])
def test_lists_of_many_kinds(torch, batch, beams, vocab, k):
    """One beam far ahead of the others, its best tokens next to each other; beams with a token or two; ended ones; all alike."""
    say(f"beam {batch}x{beams} of {vocab}, best {k}: uneven beams")
    x, s = make(torch, batch, beams, vocab, torch.float32, seed=vocab + k)
    ahead = s.clone()
    ahead[:, beams // 2] += 40
    x[:, beams // 2, vocab // 3:vocab // 3 + 100] += 20
    check(torch, x, ahead, k)
    y = x.clone()
    y[:, ::2, 2:] = -math.inf
    check(torch, y, s, k, pad=5)
    y[:, 1::2, 40:] = -math.inf
    done = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
    done[:, beams // 3:] = True
    check(torch, y, s, k, done=done, pad=7)
    same = torch.full_like(s, -1.0)
    check(torch, torch.zeros(batch, beams, vocab, device="cuda"), same, k, equal=True)
    z = torch.zeros(batch, beams, vocab, device="cuda")
    z[:, beams // 2, ::2] = 1.0
    check(torch, z, same, k, equal=True)
