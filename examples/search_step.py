"""Decoding with more than one candidate over a paged cache: drafted trees and
beam search, on the decoder of token_step.py.

A drafted tree: its tokens are appended behind what a sequence has, all of them
attend in one call, the path that the model agrees with is moved together, and the
rest is given back.  A beam step: the best continuations of a search's beams are
chosen, each goes on from its parent's pages, and only a page that is not full is
copied.  Sequences take pages from one pool and count how many hold each.

    python examples/search_step.py [--layers N] [--searches B] [--beams K] [--prompt T] [--steps S] [--e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch  # noqa: E402
import torch.nn.functional as F  # noqa: E402

import token_step  # noqa: E402
from token_step import df11, rms_norm, rotate  # noqa: E402


def mask_words(parents):
    """Words of a tree's mask: node i reads itself and those it comes from, parents[i] < i (-1: none)."""
    reads = [0] * len(parents)
    for i, p in enumerate(parents):
        reads[i] = (reads[p] if p >= 0 else 0) | 1 << i
    words = [[r >> 64 * w & (1 << 64) - 1 for w in range((len(parents) + 63) // 64)] for r in reads]
    return torch.tensor([[w - (1 << 64) if w >> 63 else w for w in r] for r in words], dtype=torch.int64)


class Search(token_step.Decoder):
    def __init__(self, searches=2, beams=4, **sizes):
        super().__init__(batch=searches * beams, **sizes)
        self.searches, self.beams = searches, beams
        self.table.fill_(-1)  # every row takes its pages from the pool
        self.refs = torch.zeros(self.cache[0].k.shape[0], dtype=torch.int32, device=self.device)

    def go_on(self, parents=None, room=1):
        """Rows go on from `parents` (None: from themselves), with pages for `room` positions more.  Returns how
        many pages were not to be had, on the device."""
        src, dst, rows, missing = df11.df11_paged_fork(parents, self.table, self.lens, self.refs, self.page_size, room)
        for c in self.cache:
            df11.df11_paged_copy(src, dst, c.k, c.v, rows)
        return missing

    def nodes(self, tokens, depth=None, tree=None, every=1):
        """Logits [rows, T, vocab] of tokens [rows, T] behind what the cache holds of each `every`-th row; lens stays
        as it is.  depth: int64 [T], positions past the length; tree: mask words; None: a chain."""
        b, t = tokens.shape
        table, lens = self.table[::every].contiguous(), self.lens[::every].contiguous()
        places = torch.arange(t, device=self.device)
        at = lens.view(b, 1) + places
        slots = table.gather(1, at // self.page_size).long() * self.page_size + at % self.page_size  # negative without a page
        position = (lens.view(b, 1) + (places if depth is None else depth)).reshape(-1)
        state = {"x": self.embedding[tokens.reshape(-1)]}
        if tree is not None:
            tree = tree.to(self.device).expand(b, -1, -1)  # one for all rows

        def layer(i, weights):
            wq, wk, wv, wo = weights
            x, c = state["x"], self.cache[i]
            h = rms_norm(x)
            q = rotate(F.linear(h, wq).view(-1, self.heads, self.head_dim), position)
            k = rotate(F.linear(h, wk).view(-1, self.kv_heads, self.head_dim), position)
            v = F.linear(h, wv).view(-1, self.kv_heads, self.head_dim)
            df11.df11_paged_append(k, v, slots.view(-1), c.k, c.v, c.scale, c.scale)
            o, _ = df11.df11_paged_tree_attention(q.view(b, t, self.heads, self.head_dim), c.k, c.v, table, lens, tree,
                                                  k_scale=c.scale, v_scale=c.scale)
            x = x + F.linear(o.view(-1, self.heads * self.head_dim), wo)
            gate, up, down = self.ffn[i]
            h = rms_norm(x)
            h = F.silu(df11.df11_mx4_matmul(h, *gate)) * df11.df11_mx4_matmul(h, *up)
            state["x"] = x + df11.df11_mx4_matmul(h, *down)

        self.ahead.run(layer)
        return F.linear(rms_norm(state["x"]), self.embedding).view(b, t, -1)

    def prompt(self, tokens):
        """A prompt [searches, T] for each search, held once.  Returns the logits behind it."""
        first = torch.arange(self.batch, device=self.device) % self.beams == 0
        row = torch.arange(self.batch, dtype=torch.int32, device=self.device)
        self.go_on(torch.where(first, row, -1).int(), tokens.shape[1])
        logits = self.nodes(tokens, every=self.beams)[:, -1]
        self.lens[::self.beams] += tokens.shape[1]
        return logits

    def beam_step(self, logits, scores, done=None, pad=0):
        """The best continuations of logits [searches, beams in use, vocab] and their rows' pages, one token fed.
        Returns (logits, scores, parents, tokens); parents are rows of the table."""
        k = self.beams
        scores, parents, tokens = df11.df11_beam_select(logits, scores, k, done, pad)
        if logits.shape[1] != k:  # of the prompt: each search's first row
            parents = torch.where(parents >= 0, parents // logits.shape[1] * k, -1).int()
        self.go_on(parents.view(-1))
        tokens = tokens.view(-1, 1)
        out = self.nodes(tokens.clamp_min(0))[:, 0]
        self.lens += 1
        return out.view(self.searches, k, -1), scores, parents, tokens.view(self.searches, k)

    def tree_step(self, tokens, parents):
        """Checks drafted tokens [rows, T] against the model: node 0 is the last token known, node i follows
        parents[i].  Returns (path, accepted, next): nodes [rows, T] that the model agrees with, how many, and the
        token behind them; the cache holds the path."""
        b, t = tokens.shape
        depth = [0] * t
        for i in range(1, t):
            depth[i] = depth[parents[i]] + 1
        self.go_on(room=t)
        logits = self.nodes(tokens, torch.tensor(depth, device=self.device), mask_words(parents))
        choice = logits.argmax(-1)
        of = torch.tensor(parents, device=self.device)
        here = torch.zeros(b, dtype=torch.int64, device=self.device)
        path = torch.full((b, t), -1, dtype=torch.int32, device=self.device)
        path[:, 0] = 0
        accepted = torch.ones(b, dtype=torch.int32, device=self.device)
        alive = torch.ones(b, dtype=torch.bool, device=self.device)
        for step in range(1, max(depth) + 1):
            fits = (of == here.view(b, 1)) & (tokens == choice.gather(1, here.view(b, 1)))
            alive &= fits.any(1)
            here = torch.where(alive, fits.int().argmax(1), here)
            path[:, step] = torch.where(alive, here, -1).int()
            accepted += alive.int()
        for c in self.cache:
            df11.df11_paged_compact(path, accepted, self.table, self.lens, c.k, c.v)
        self.lens += accepted
        return path, accepted, choice.gather(1, here.view(b, 1))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--searches", type=int, default=4)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=64)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--e4m3", action="store_true", help="keys and values in 8 bits")
    a = ap.parse_args()
    model = Search(a.searches, a.beams, layers=a.layers, hidden=4096, heads=32, kv_heads=8, head_dim=128, ffn=14336, vocab=32000,
                   max_tokens=a.prompt + a.steps + 16, e4m3=a.e4m3)
    tokens = torch.randint(0, 32000, (a.searches, a.prompt), device=model.device)
    logits = model.prompt(tokens).view(a.searches, 1, -1)
    scores = torch.zeros(a.searches, 1, device=model.device)
    logits, scores, _, tokens = model.beam_step(logits, scores)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps - 1):
        logits, scores, _, tokens = model.beam_step(logits, scores)
    end.record()
    torch.cuda.synchronize()
    ms = begin.elapsed_time(end) / max(1, a.steps - 1)
    print(f"{a.layers} layers, {a.searches} searches of {a.beams} beams: {ms:.3f} ms a step")


if __name__ == "__main__":
    main()
