"""GPU: the example of drafted trees and beam search over one pool of pages
(append, tree attention, compact, fork, copy and selection together) against the
same decoder in plain 32-bit torch without a cache, on each candidate's own tokens.

Logits are held to the bound of the token-step example's test: about 16 roundings
to BF16 a layer and two outside, 2^-8 each, times the square root of their number,
times 4, in the 2-norm.  Choices are checked against the logits that they were
made from: a selected score is off by the roundings of 32 bits in the sum of
exponentials (a sum of 1,000 positive terms, 2^-14 at most) and in the score
itself."""
import math
import os
import sys

import pytest

from conftest import ROOT
from test_gpu_token_step import plain

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

LAYERS, BOUND = 2, 4 * 2.0 ** -8 * math.sqrt(16 * 2 + 2)


def close(torch, model, logits, tokens, e4m3):
    """Holds logits [rows, vocab] to those behind `tokens`, a list of each row's."""
    import token_step
    by_length = {}
    for i, row in enumerate(tokens):
        by_length.setdefault(len(row), []).append(i)
    for rows in by_length.values():
        ref = plain(torch, model, token_step, torch.tensor([tokens[i] for i in rows], device="cuda"), e4m3)
        off = (logits[rows].float() - ref).norm(dim=-1) / ref.norm(dim=-1)
        assert float(off.max()) <= BOUND, (rows, off.tolist())


def counted(torch, model):
    """Every page's count is the number of entries that name it."""
    held = model.table[model.table >= 0].long()
    assert torch.equal(torch.bincount(held, minlength=model.refs.numel()).int(), model.refs)


@pytest.mark.parametrize("e4m3", [False, True])
def test_beam_steps(e4m3):
    import torch

    import search_step
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    print(f"[gpu-test] beam search example, e4m3={e4m3}", flush=True)
    searches, beams = 3, 4
    model = search_step.Search(searches, beams, layers=LAYERS, e4m3=e4m3, max_tokens=64)
    g = torch.Generator(device="cuda").manual_seed(5)
    prompt = torch.randint(0, 1000, (searches, 29), generator=g, device="cuda")
    logits = model.prompt(prompt).view(searches, 1, -1)
    scores = torch.zeros(searches, 1, device="cuda")
    seen = prompt.tolist()
    close(torch, model, logits[:, 0], seen, e4m3)
    for step in range(8):
        used = logits.shape[1]
        total = scores.double().unsqueeze(-1) + torch.log_softmax(logits.double(), -1)
        best = total.view(searches, -1).topk(beams).values
        before = seen
        logits, scores, parents, tokens = model.beam_step(logits, scores)
        assert float((scores.double() - best).abs().max()) <= 2.0 ** -14 + 2.0 ** -22 * float(best.abs().max())
        p, t = parents.tolist(), tokens.tolist()
        seen = [before[row // beams if used == 1 else row] + [token] for a, b in zip(p, t) for row, token in zip(a, b)]
        assert all(row // beams == i for i, rows in enumerate(p) for row in rows)
        close(torch, model, logits.view(searches * beams, -1), seen, e4m3)
        counted(torch, model)
        assert model.lens.tolist() == [30 + step] * (searches * beams)


@pytest.mark.parametrize("e4m3", [False, True])
def test_drafted_trees(e4m3):
    import torch

    import search_step
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    print(f"[gpu-test] drafted trees example, e4m3={e4m3}", flush=True)
    rows = 3
    model = search_step.Search(rows, 1, layers=LAYERS, e4m3=e4m3, max_tokens=96)
    g = torch.Generator(device="cuda").manual_seed(6)
    prompt = torch.randint(0, 1000, (rows, 27), generator=g, device="cuda")
    following = model.prompt(prompt).argmax(-1, keepdim=True)
    seen = prompt.tolist()
    parents = [-1, 0, 0, 1, 1, 2, 3, 6]
    for step in range(4):
        # a draft that is right for some rows: the model's own choices, found without changing the cache for good
        tokens = torch.randint(0, 1000, (rows, len(parents)), generator=g, device="cuda")
        tokens[:, :1] = following
        model.go_on(room=2)
        guess = model.nodes(tokens[:, :1])[:, 0].argmax(-1)
        tokens[step % rows:, 2] = guess[step % rows:]
        guess = model.nodes(tokens[:, [0, 2]])[:, 1].argmax(-1)
        tokens[step % rows:, 5] = guess[step % rows:]
        depth = [0, 1, 1, 2, 2, 2, 3, 4]
        model.go_on(room=len(parents))
        logits = model.nodes(tokens, torch.tensor(depth, device="cuda"), search_step.mask_words(parents))
        for node in range(len(parents)):
            way = []
            at = node
            while at >= 0:
                way.insert(0, at)
                at = parents[at]
            close(torch, model, logits[:, node], [s + [int(tokens[i, a]) for a in way] for i, s in enumerate(seen)], e4m3)
        path, accepted, following = model.tree_step(tokens, parents)
        choice = logits.argmax(-1)
        for i in range(rows):
            way = path[i, :int(accepted[i])].tolist()
            assert way[0] == 0 and all(parents[b] == a and tokens[i, b] == choice[i, a] for a, b in zip(way, way[1:]))
            assert not any(parents[c] == way[-1] and tokens[i, c] == choice[i, way[-1]] for c in range(len(parents)))
            assert int(following[i]) == int(choice[i, way[-1]])
            seen[i] = seen[i] + [int(tokens[i, a]) for a in way]
        assert model.lens.tolist() == [len(s) for s in seen]
        model.go_on(room=1)
        counted(torch, model)
        # what the cache holds now: one token more, without keeping it
        close(torch, model, model.nodes(following)[:, 0], [s + [int(following[i])] for i, s in enumerate(seen)], e4m3)
