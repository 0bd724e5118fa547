"""The example's attention block and caption decoder against float64: the
operators together, as they are used between the convolutions."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

import implicit_gemm_nhwc_amd as igc  # noqa: E402
from oracle import attention as oracle  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(
        torch.bfloat16).to(DEV)


def _rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach().cpu().double()
    assert torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm())


def test_block_forward_and_step():
    """Each stage is compared from the stage before as the GPU rounded it:
    roundings of at most 2^-8 on each result and, inside the attention, on
    the probabilities and ds, which add in the 2-norm to less than 2^-7."""
    from cross_attention_block import CrossAttentionBlock
    block = CrossAttentionBlock(64, 96, heads=4, kv_heads=2, head_dim=32)
    block.q_weight.mul_(1.3)
    block.k_weight.mul_(0.8)
    x, states = _rnd(2, 9, 7, 64, seed=1), _rnd(2, 33, 96, seed=2)
    lens = torch.tensor([33, 12], dtype=torch.int32, device=DEV)
    q, k, v = block.project(x, states)
    wq = block.wq.cpu().double()[0, 0]
    assert _rel(q.reshape(2, 63, -1), x.cpu().double().view(2, 63, 64) @ wq) < 2.0 ** -7
    norm = block.norm_args(x, states)
    qr, kr = igc.qk_norm_rope(q, k, **norm)
    q64 = oracle.qk_norm_rope(q, weight=block.q_weight, table=norm["q_table"], eps=1e-6)
    k64 = oracle.qk_norm_rope(k, weight=block.k_weight, table=norm["k_table"], eps=1e-6)
    assert _rel(qr, q64) < 2.0 ** -8 and _rel(kr, k64) < 2.0 ** -8
    go = _rnd(2, 63, 4, 32, seed=3)
    o, grads = block.attention_step(x, states, go, kv_lens=lens)
    r = oracle.cross_attention(qr, kr, v, kv_lens=lens, dout=go)
    assert _rel(o, r["out"]) < 2.0 ** -7
    dqr, dkr, dv = igc.cross_attention_bwd(
        go, qr, kr, v, o, igc.cross_attention(qr, kr, v, kv_lens=lens, return_lse=True)[1],
        kv_lens=lens)
    for got, name in ((dqr, "dq"), (dkr, "dk"), (dv, "dv")):
        assert _rel(got, r[name]) < 2.0 ** -7, name
    assert torch.equal(grads["dv"], dv)
    rq = oracle.qk_norm_rope(q, weight=block.q_weight, table=norm["q_table"], grad=dqr)
    rk = oracle.qk_norm_rope(k, weight=block.k_weight, table=norm["k_table"], grad=dkr)
    assert _rel(grads["dq"], rq["dx"]) < 2.0 ** -8 and _rel(grads["dk"], rk["dx"]) < 2.0 ** -8
    assert _rel(grads["dq_weight"], rq["dweight"]) < 1e-4
    assert _rel(grads["dk_weight"], rk["dweight"]) < 1e-4
    y = block.forward(x, states, kv_lens=lens)
    wo = block.wo.cpu().double()[0, 0]
    y64 = x.cpu().double().view(2, 63, 64) + o.cpu().double().view(2, 63, -1) @ wo
    assert _rel(y.view(2, 63, 64), y64) < 2.0 ** -7


def test_decoder_reads_as_the_block_does():
    """A token a step gives what one call over all tokens gives."""
    from cross_attention_block import CaptionReader, CrossAttentionBlock
    block = CrossAttentionBlock(64, 64, heads=8, kv_heads=2, head_dim=32)
    image, tokens = _rnd(3, 12, 11, 64, seed=4), _rnd(3, 5, 1, 64, seed=5)
    reader = CaptionReader(block, image)
    table = igc.rope_table(16, 32, device=DEV)
    at = (torch.arange(5)[None] + torch.tensor([[0], [3], [9]])).to(torch.int32).to(DEV)
    steps = [reader.step(tokens[:, t:t + 1].contiguous(), at[:, t:t + 1].contiguous(), table)
             for t in range(5)]
    q = igc.conv2d(tokens, block.wq, filter_is_fcrs=False).view(3, 5, 8, 32)
    q = igc.qk_norm_rope(q, q_weight=block.q_weight, q_table=table, q_positions=at)
    r = oracle.cross_attention(q, reader.k, reader.v)
    y = tokens.cpu().double().view(3, 5, 64) + r["out"].view(3, 5, -1) @ block.wo.cpu().double()[
        0, 0]
    got = torch.cat([s.view(3, 1, 64) for s in steps], 1)
    # out and y rounded once each, the probabilities once
    assert _rel(got, y) < 2.0 ** -7


def test_both_ways_through_the_binding(monkeypatch):
    """The calls that go through the binding's C++ part give the same bits
    and the same refusals through Python alone."""
    from implicit_gemm_nhwc_amd import attention as binding
    assert binding._fast is not None
    q, kv = _rnd(2, 40, 8, 64, seed=6), _rnd(2, 70, 2, 4, 64, seed=7)
    k, v = kv[:, :, 0], kv[:, :, 1]
    go = _rnd(2, 40, 8, 64, seed=8)
    lens = torch.tensor([70, 9], dtype=torch.int32, device=DEV)
    mask = torch.rand(2, 70, device=DEV) < 0.8
    table = igc.rope_table(80, 32, device=DEV)
    at = torch.randint(0, 80, (2, 40), device=DEV).to(torch.int32)
    w = torch.rand(64, device=DEV)

    def calls():
        kw = dict(kv_lens=lens, key_mask=mask, scale=0.2)
        out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
        norm = dict(q_weight=w, q_table=table, k_table=table, q_positions=at, eps=1e-5,
                    interleaved=True)
        alone = {n: x for n, x in norm.items() if n != "k_table"}
        return [out, lse, igc.cross_attention(q, k, v),
                *igc.cross_attention_bwd(go, q, k, v, out, lse, **kw),
                *igc.qk_norm_rope(q, k, **norm), igc.qk_norm_rope(q, **alone),
                *igc.qk_norm_rope_bwd(go, k, q, k, **norm),
                *igc.qk_norm_rope_bwd(go, None, q, **alone)]

    def refusals():
        seen = []
        for bad in (lambda: igc.cross_attention(q, k[:1], v), lambda: igc.cross_attention(q, k, go),
                    lambda: igc.cross_attention(q, k, v, scale=-1.0),
                    lambda: igc.cross_attention(q.float(), k, v),
                    lambda: igc.cross_attention(q, k, v, kv_lens=lens.long()),
                    lambda: igc.qk_norm_rope(q, k, q_table=table),
                    lambda: igc.qk_norm_rope(q, eps=-1.0),
                    lambda: igc.qk_norm_rope_bwd(go[:1], None, q)):
            with pytest.raises((igc.InvalidArgument, igc.Declined)) as e:
                bad()
            seen.append((e.type, str(e.value)))
        return seen

    fast, said = calls(), refusals()
    monkeypatch.setattr(binding, "_fast", None)
    slow = calls()
    assert said == refusals()
    for a, b in zip(fast, slow):
        assert (a is None and b is None) or (a.shape == b.shape and torch.equal(a, b))
        assert a is None or (a.stride() == b.stride() and a.dtype == b.dtype)


def test_example_runs(capsys):
    import cross_attention_block
    cross_attention_block.main()
    text = capsys.readouterr().out
    assert "finite: True" in text
