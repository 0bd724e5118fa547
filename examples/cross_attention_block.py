"""The attention block of a text-conditioned image model, and a caption
decoder's reading of an image, built from this library's calls.

Block (training and inference): an NHWC map attends to a text encoder's states.
  q  = 1x1 convolution of the map                (conv2d)
  kv = 1x1 convolution of the states, seen as a [N, 1, T, C] map
  q, k normed per head and rotated, the map's pixels by row and column, the
       states by position                        (qk_norm_rope)
  o  = attention of the pixels to the states     (cross_attention)
  y  = map + 1x1 convolution of o                (conv2d with a residual)
The convolution's NHWC output [N, H, W, heads * D] is the attention's
[N, H * W, heads, D] without a copy, and back.

Decoder: tokens one at a time attend to the pixels of the map (their keys and
values made once), which is the single-token form of the same calls.

Run on the GPU:  python examples/cross_attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import implicit_gemm_nhwc_amd as igc  # noqa: E402


class CrossAttentionBlock:
    """Weights and tables of one block; 1x1 filters in RSCF layout."""

    def __init__(self, channels, state_channels, heads, kv_heads, head_dim, *,
                 dtype=torch.bfloat16, device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def filt(c, f):
            w = torch.randn(1, 1, c, f, generator=gen, device=device) * c ** -0.5
            return w.to(dtype)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.wq = filt(channels, heads * head_dim)
        self.wkv = filt(state_channels, 2 * kv_heads * head_dim)
        self.wo = filt(heads * head_dim, channels)
        self.q_weight = torch.ones(head_dim, device=device)
        self.k_weight = torch.ones(head_dim, device=device)
        self.tables = {}

    def _table(self, kind, *size):
        """Rotation tables are made once a size."""
        if (kind, size) not in self.tables:
            make = igc.rope_table_2d if kind == "map" else igc.rope_table
            self.tables[kind, size] = make(*size, self.head_dim, device=self.wq.device)
        return self.tables[kind, size]

    def project(self, x, states):
        """Queries [N, H*W, heads, D] and keys, values [N, T, kv_heads, D],
        before the norm."""
        n, h, w, _ = x.shape
        t = states.shape[1]
        q = igc.conv2d(x, self.wq, filter_is_fcrs=False).view(n, h * w, self.heads, self.head_dim)
        kv = igc.conv2d(states.view(n, 1, t, -1), self.wkv, filter_is_fcrs=False)
        kv = kv.view(n, t, 2, self.kv_heads, self.head_dim)
        return q, kv[:, :, 0], kv[:, :, 1]

    def norm_args(self, x, states):
        n, h, w, _ = x.shape
        return dict(q_weight=self.q_weight, k_weight=self.k_weight,
                    q_table=self._table("map", h, w),
                    k_table=self._table("states", states.shape[1]))

    def forward(self, x, states, kv_lens=None, key_mask=None):
        q, k, v = self.project(x, states)
        qr, kr = igc.qk_norm_rope(q, k, **self.norm_args(x, states))
        o = igc.cross_attention(qr, kr, v, kv_lens=kv_lens, key_mask=key_mask)
        return igc.conv2d(o.view(*x.shape[:3], -1), self.wo, filter_is_fcrs=False, source=x,
                          beta=1.0)

    def attention_step(self, x, states, d_attn, kv_lens=None, key_mask=None):
        """A training step of the block's attention: its output and, from the
        gradient d_attn at it, the gradients at the projections' outputs and
        at the norm's weights."""
        q, k, v = self.project(x, states)
        norm = self.norm_args(x, states)
        qr, kr = igc.qk_norm_rope(q, k, **norm)
        o, lse = igc.cross_attention(qr, kr, v, kv_lens=kv_lens, key_mask=key_mask,
                                     return_lse=True)
        dqr, dkr, dv = igc.cross_attention_bwd(d_attn, qr, kr, v, o, lse, kv_lens=kv_lens,
                                               key_mask=key_mask)
        dq, dk, dqw, dkw = igc.qk_norm_rope_bwd(dqr, dkr, q, k, **norm)
        return o, dict(dq=dq, dk=dk, dv=dv, dq_weight=dqw, dk_weight=dkw)


class CaptionReader:
    """Single tokens attend to an image's pixels, whose keys and values are
    made once an image."""

    def __init__(self, block, image):
        n, h, w, c = image.shape
        self.block = block
        _, k, self.v = block.project(image, image.reshape(n, h * w, c))
        self.k = igc.qk_norm_rope(k, q_weight=block.k_weight, q_table=block._table("map", h, w))

    def step(self, token, positions, table):
        """token [N, 1, 1, channels] at positions int32 [N, 1] of the table."""
        b = self.block
        q = igc.conv2d(token, b.wq, filter_is_fcrs=False).view(-1, 1, b.heads, b.head_dim)
        q = igc.qk_norm_rope(q, q_weight=b.q_weight, q_table=table, q_positions=positions)
        o = igc.cross_attention(q, self.k, self.v)
        return igc.conv2d(o.view(token.shape[0], 1, 1, -1), b.wo, filter_is_fcrs=False,
                          source=token, beta=1.0)


def main():
    dev = "cuda:0"
    gen = torch.Generator(device=dev).manual_seed(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)

    block = CrossAttentionBlock(256, 512, heads=4, kv_heads=2, head_dim=64)
    x, states = rnd(2, 64, 64, 256), rnd(2, 77, 512)
    lens = torch.tensor([77, 31], dtype=torch.int32, device=dev)
    y = block.forward(x, states, kv_lens=lens)
    o, grads = block.attention_step(x, states, rnd(2, 64 * 64, 4, 64), kv_lens=lens)
    print("block:", tuple(y.shape), "attention:", tuple(o.shape),
          {n: tuple(g.shape) for n, g in grads.items()}, flush=True)

    reader = CaptionReader(CrossAttentionBlock(256, 256, heads=8, kv_heads=2, head_dim=128),
                           rnd(2, 28, 28, 256))
    table = igc.rope_table(64, 128, device=dev)
    token = rnd(2, 1, 1, 256)
    for t in range(4):
        at = torch.full((2, 1), t, dtype=torch.int32, device=dev)
        token = reader.step(token, at, table)
    torch.cuda.synchronize()
    print("decoder: 4 tokens,", tuple(token.shape), "finite:",
          bool(torch.isfinite(token).all()), flush=True)


if __name__ == "__main__":
    main()
