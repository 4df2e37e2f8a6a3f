"""A decoder's prompt and token steps over the library's three stores.

Per layer, the attention projections (q, k, v, o) are one DF11 block, decoded
bit-exactly one layer ahead of its use (DecodeAhead); the feed-forward matrices
(gate, up, down) are 4-bit codes that the product reads as they are; keys and
values lie in the pages of a cache, BF16 or E4M3.  Weights are random; norms,
rotary positions and the activation are plain torch.

    python examples/token_step.py [--layers N] [--batch B] [--prompt T] [--steps S] [--e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402
import torch.nn.functional as F  # noqa: E402

import huffman_decode_block_amd as df11  # noqa: E402
from huffman_decode_block_amd.overlap import DecodeAhead  # noqa: E402


def rms_norm(x, eps=1e-5):
    v = x.float()
    return (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)).to(x.dtype)


def rotate(x, positions):
    """Rotary positions on [tokens, heads, dim]."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device) / half)
    angle = positions.view(-1, 1, 1) * freq
    a, b = x.float()[..., :half], x.float()[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(x.dtype)


class Pages:
    """A paged cache of one layer; all layers share the page table."""

    def __init__(self, n_pages, kv_heads, page_size, head_dim, e4m3, device):
        shape = (n_pages, kv_heads, page_size, head_dim)
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        # one scale for each head: values of up to 448 steps of it
        self.scale = torch.full((kv_heads,), 1 / 32, device=device) if e4m3 else None


class Decoder:
    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, ffn=1408, vocab=1000, batch=2,
                 max_tokens=128, page_size=16, e4m3=False, seed=0, device="cuda"):
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.batch = hidden, heads, kv_heads, head_dim, batch
        self.page_size, self.device = page_size, device
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) / cols ** 0.5).to(torch.bfloat16)

        shapes = [(heads * head_dim, hidden), (kv_heads * head_dim, hidden), (kv_heads * head_dim, hidden),
                  (hidden, heads * head_dim)]
        blocks, self.ffn, self.attention_weights = [], [], []
        for _ in range(layers):
            mats = [weight(*s) for s in shapes]
            self.attention_weights.append(mats)
            blocks.append(df11.DeviceBlock.from_encoded(df11.df11_encode_block(mats), device=device))
            self.ffn.append([df11.df11_mx4_quantize(weight(*s).to(device)) for s in
                             ((ffn, hidden), (ffn, hidden), (hidden, ffn))])
        self.embedding = weight(vocab, hidden).to(device) * hidden ** 0.5
        self.ahead = DecodeAhead(blocks, [shapes] * layers)
        per = -(-max_tokens // page_size)
        self.cache = [Pages(batch * per, kv_heads, page_size, head_dim, e4m3, device) for _ in range(layers)]
        self.table = torch.randperm(batch * per, generator=g).int().view(batch, per).to(device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def forward(self, tokens):
        """Logits of `tokens` [batch, T], which follow what the cache holds."""
        b, t = tokens.shape
        at = (self.lens.view(b, 1) + torch.arange(t, device=self.device)).reshape(-1)  # position of each token
        row = torch.arange(b, device=self.device).repeat_interleave(t)
        table = self.table[row]  # each token reads its sequence's pages up to itself
        slots = table.gather(1, (at // self.page_size).view(-1, 1)).view(-1).long() * self.page_size + at % self.page_size
        lens = (at + 1).int()
        state = {"x": self.embedding[tokens.reshape(-1)]}

        def layer(i, weights):
            wq, wk, wv, wo = weights
            x, c = state["x"], self.cache[i]
            h = rms_norm(x)
            q = rotate(F.linear(h, wq).view(-1, self.heads, self.head_dim), at)
            k = rotate(F.linear(h, wk).view(-1, self.kv_heads, self.head_dim), at)
            v = F.linear(h, wv).view(-1, self.kv_heads, self.head_dim)
            df11.df11_paged_append(k, v, slots, c.k, c.v, c.scale, c.scale)
            o, _ = df11.df11_paged_attention(q, c.k, c.v, table, lens, k_scale=c.scale, v_scale=c.scale)
            x = x + F.linear(o.view(-1, self.heads * self.head_dim), wo)
            gate, up, down = self.ffn[i]
            h = rms_norm(x)
            h = F.silu(df11.df11_mx4_matmul(h, *gate)) * df11.df11_mx4_matmul(h, *up)
            state["x"] = x + df11.df11_mx4_matmul(h, *down)

        self.ahead.run(layer)
        self.lens += t
        return F.linear(rms_norm(state["x"]).view(b, t, -1)[:, -1], self.embedding)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=64)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--e4m3", action="store_true", help="keys and values in 8 bits")
    a = ap.parse_args()
    model = Decoder(layers=a.layers, hidden=4096, heads=32, kv_heads=8, head_dim=128, ffn=14336, vocab=32000,
                    batch=a.batch, max_tokens=a.prompt + a.steps, e4m3=a.e4m3)
    tokens = torch.randint(0, 32000, (a.batch, a.prompt), device=model.device)
    token = model.forward(tokens).argmax(-1, keepdim=True)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps - 1):
        token = model.forward(token).argmax(-1, keepdim=True)
    end.record()
    torch.cuda.synchronize()
    ms = begin.elapsed_time(end) / max(1, a.steps - 1)
    print(f"{a.layers} layers, batch {a.batch}: {ms:.3f} ms a token step, {a.batch / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
