"""A caption decoder's self-attention layer served in 8 bits, built from this
library's calls.

Layer:
  n = layer norm of the tokens                       (layer_norm)
  n in 8 bits, a scale a token                       (quantize_rows)
  q, k, v = its product with weights in 8 bits       (linear_i8)
  q, k normed per head and rotated by position       (qk_norm_rope)
  k, v into the paged cache in 8 bits                (kv_cache_write)
  o = attention of the new tokens over the cache     (cache_attention)
  y = x + product of o in 8 bits with the output's weights
A prompt goes through the same calls as one token, many tokens at a time; the
sequences of a batch may have different lengths.  norm_step is a training step
of the layer's norm: its gradients from the gradient at its result.

Run on the GPU:  python examples/caption_decoder.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import implicit_gemm_nhwc_amd as igc  # noqa: E402


class PageTable:
    """Hands out a pool's pages to the sequences of a batch as they grow."""

    def __init__(self, pages, page_tokens, batch, max_tokens, device):
        self.free = list(range(pages))
        self.page_tokens = page_tokens
        self.owned = [0] * batch
        self.table = torch.full((batch, -(-max_tokens // page_tokens)), -1, dtype=torch.int32)
        self.device = device

    def grow(self, tokens):
        """The table with room for tokens[b] tokens of sequence b."""
        for b, n in enumerate(tokens):
            while self.owned[b] * self.page_tokens < n:
                self.table[b, self.owned[b]] = self.free.pop()
                self.owned[b] += 1
        return self.table.to(self.device)


class DecoderLayer:
    """Weights of one layer, in 8 bits, with its cache."""

    def __init__(self, channels, heads, kv_heads, head_dim, *, batch, max_tokens, page_tokens=16,
                 dtype=torch.bfloat16, device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weights(out, k):
            w = torch.randn(out, k, generator=gen, device=device) * k ** -0.5
            return igc.quantize_rows(w.to(dtype))      # a scale an output channel

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.w_qkv = weights((heads + 2 * kv_heads) * head_dim, channels)
        self.w_out = weights(channels, heads * head_dim)
        self.norm_weight = torch.ones(channels, device=device)
        self.norm_bias = torch.zeros(channels, device=device)
        self.q_weight = torch.ones(head_dim, device=device)
        self.k_weight = torch.ones(head_dim, device=device)
        self.rotation = igc.rope_table(max_tokens, head_dim, device=device)
        per = -(-max_tokens // page_tokens)
        self.cache = igc.KVCache.empty(batch * per, page_tokens, kv_heads, head_dim, device=device)
        self.pages = PageTable(batch * per, page_tokens, batch, max_tokens, device)
        self.held = [0] * batch        # tokens of each sequence

    def project(self, x, weights):
        q, scale = igc.quantize_rows(x)
        return igc.linear_i8(q, scale, *weights, dtype=x.dtype)

    def forward(self, x, new=None):
        """x [batch, tokens, channels]; new: how many of them each sequence
        really has (a padded prompt; None: all).  Returns the layer's result;
        rows of padding hold nothing of use."""
        b, t, _ = x.shape
        new = [t] * b if new is None else list(new)
        dev = x.device
        start = torch.tensor(self.held, dtype=torch.int32, device=dev)
        lens = torch.tensor(new, dtype=torch.int32, device=dev)
        self.held = [h + n for h, n in zip(self.held, new)]
        table = self.pages.grow(self.held)
        n = igc.layer_norm(x, self.norm_weight, self.norm_bias)
        qkv = self.project(n, self.w_qkv).view(b, t, -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 2)
        at = start[:, None] + torch.arange(t, dtype=torch.int32, device=dev)
        q, k = igc.qk_norm_rope(q, k, q_weight=self.q_weight, k_weight=self.k_weight,
                                q_table=self.rotation, k_table=self.rotation, q_positions=at,
                                k_positions=at)
        igc.kv_cache_write(self.cache, k, v, table, start, lens=lens)
        # the last t places, the padding's among them, are the new tokens'
        o = igc.cache_attention(q, self.cache, table, start + t)
        return x + self.project(o.view(b, t, -1), self.w_out)

    def norm_step(self, x, d_normed):
        """A training step of the norm: its result, the gradient at x and at its
        weight and bias, from the gradient at its result."""
        n = igc.layer_norm(x, self.norm_weight, self.norm_bias)
        return n, igc.layer_norm_bwd(d_normed, x, self.norm_weight)


def main():
    dev = "cuda:0"
    gen = torch.Generator(device=dev).manual_seed(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)

    layer = DecoderLayer(512, heads=8, kv_heads=2, head_dim=64, batch=3, max_tokens=64)
    y = layer.forward(rnd(3, 20, 512), new=[20, 7, 13])
    print("prompt:", tuple(y.shape), "tokens held:", layer.held, flush=True)
    token = y[:, :1]
    for _ in range(5):
        token = layer.forward(token)
    n, (dx, dw, db) = layer.norm_step(rnd(3, 20, 512), rnd(3, 20, 512))
    torch.cuda.synchronize()
    print("5 tokens:", tuple(token.shape), "held:", layer.held, "finite:",
          bool(torch.isfinite(token).all()), "norm's gradients:", tuple(dx.shape), tuple(dw.shape),
          tuple(db.shape), flush=True)


if __name__ == "__main__":
    main()
