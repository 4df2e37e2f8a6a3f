"""GPU: the token-step example (DF11 attention weights, 4-bit feed-forward
weights, paged cache) against the same decoder in plain 32-bit torch without a
cache, on the weights that the stores stand for.

The example rounds to BF16 about 16 times a layer and twice outside; each
rounding is off by at most 2^-8 of a value, and errors of that size pass
through norms and residuals about as they are.  The logits may be off by 2^-8
times the square root of their number, times 4 for the largest of many, in the
2-norm over that of the logits."""
import math
import os
import sys

import pytest

import huffman_decode_block_amd as hdb
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain(torch, model, token_step, tokens, e4m3):
    """Logits behind the last of `tokens`, everything in 32 bits."""
    x = model.embedding[tokens].float()
    b, t, _ = x.shape
    at = torch.arange(t, device=x.device)
    mask = torch.ones(t, t, dtype=torch.bool, device=x.device).tril()
    for i, mats in enumerate(model.attention_weights):
        wq, wk, wv, wo = (m.to(x.device).float() for m in mats)
        h = token_step.rms_norm(x)
        def heads(w, n):
            return (h @ w.T).view(b * t, n, model.head_dim)
        pos = at.repeat(b)
        q, k = token_step.rotate(heads(wq, model.heads), pos), token_step.rotate(heads(wk, model.kv_heads), pos)
        v = heads(wv, model.kv_heads)
        if e4m3:
            s = model.cache[i].scale.view(1, -1, 1)
            k, v = ((y.to(torch.bfloat16).float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s for y in (k, v))
        g = model.heads // model.kv_heads
        q, k, v = (y.view(b, t, -1, model.head_dim).transpose(1, 2).contiguous() for y in (q, k, v))
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        s = (q @ k.transpose(-1, -2).contiguous()) / math.sqrt(model.head_dim)
        o = torch.softmax(s.masked_fill(~mask, -math.inf), -1) @ v
        x = x + o.transpose(1, 2).reshape(b, t, -1) @ wo.T
        gate, up, down = (hdb.df11_mx4_dequantize(*c, n).float() for c, n in
                          zip(model.ffn[i], (model.hidden, model.hidden, model.ffn[i][0][0].shape[0])))
        h = token_step.rms_norm(x)
        x = x + (torch.nn.functional.silu(h @ gate.T) * (h @ up.T)) @ down.T
    return token_step.rms_norm(x)[:, -1] @ model.embedding.float().T


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_and_token_steps(e4m3):
    import torch

    import token_step
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    print(f"[gpu-test] token step example, e4m3={e4m3}", flush=True)
    layers = 2
    model = token_step.Decoder(layers=layers, e4m3=e4m3, batch=3, max_tokens=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(0, 1000, (3, 37), generator=g, device="cuda")
    bound = 4 * 2.0 ** -8 * math.sqrt(16 * layers + 2)
    for new in (tokens[:, :30], *tokens[:, 30:].split(1, dim=1)):  # a prompt, then single tokens
        logits = model.forward(new)
        seen = tokens[:, : int(model.lens[0])]
        ref = plain(torch, model, token_step, seen, e4m3)
        off = float((logits.float() - ref).norm() / ref.norm())
        print(f"[gpu-test] {seen.shape[1]} tokens: off by {off:.2e}", flush=True)
        assert off <= bound
