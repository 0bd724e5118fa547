"""The example's decoder layer against float64: the operators together, as a
program uses them, a padded prompt and then single tokens; and the norm's
training step."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

import implicit_gemm_nhwc_amd as igc  # noqa: E402
from oracle import attention, decoder as oracle  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(
        torch.bfloat16).to(DEV)


def _rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach().cpu().double()
    assert torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm())


def test_prompt_and_tokens(monkeypatch):
    """Each call is compared from its inputs as the GPU rounded them: one
    rounding of at most 2^-8 of each value, which in the 2-norm stays below
    2^-8; integers and scales are equal."""
    from caption_decoder import DecoderLayer
    layer = DecoderLayer(128, heads=6, kv_heads=2, head_dim=40, batch=3, max_tokens=50, seed=3)
    layer.norm_weight.mul_(1.2)
    layer.norm_bias.add_(0.1)
    layer.k_weight.mul_(0.9)
    real = {n: getattr(igc, n) for n in ("layer_norm", "quantize_rows", "linear_i8", "qk_norm_rope",
                                         "kv_cache_write", "cache_attention")}
    calls = []

    def spy(name):
        def call(*a, **kw):
            before = None
            if name == "kv_cache_write":
                before = [t.cpu().clone() for t in (a[0].k, a[0].k_scale, a[0].v, a[0].v_scale)]
            r = real[name](*a, **kw)
            calls.append((name, a, kw, r, before))
            return r
        return call

    for n in real:
        monkeypatch.setattr(igc, n, spy(n))
    steps = [(_rnd(3, 20, 128, seed=1), [20, 7, 13])] + [
        (_rnd(3, 1, 128, seed=2 + i), None) for i in range(3)] + [(_rnd(3, 4, 128, seed=9), None)]
    for x, new in steps:
        calls.clear()
        y = layer.forward(x, new)
        names = [c[0] for c in calls]
        assert names == ["layer_norm", "quantize_rows", "linear_i8", "qk_norm_rope",
                         "kv_cache_write", "cache_attention", "quantize_rows", "linear_i8"]
        b, t, _ = x.shape
        good = torch.arange(t)[None] < torch.tensor(new or [t] * b)[:, None]
        for name, a, kw, r, before in calls:
            if name == "layer_norm":
                assert _rel(r, oracle.layer_norm(a[0], weight=a[1], bias=a[2])["y"]) < 2.0 ** -8
            elif name == "quantize_rows":
                q, s = oracle.rows_i8(a[0])
                assert torch.equal(r[0].cpu().double()[good], q[good])
                assert torch.equal(r[1].cpu()[good], s[good])
            elif name == "linear_i8":
                xq, xs, wq, ws = (u.cpu().double() for u in a)
                ref = (xq @ wq.t()) * xs[..., None] * ws
                assert _rel(r[good.to(DEV)], ref[good]) < 2.0 ** -8
            elif name == "qk_norm_rope":
                for i, n in enumerate("qk"):
                    ref = attention.qk_norm_rope(a[i], weight=kw[n + "_weight"],
                                                 table=kw[n + "_table"],
                                                 positions=kw[n + "_positions"], eps=1e-6)
                    assert _rel(r[i], ref) < 2.0 ** -8
            elif name == "kv_cache_write":
                cache, k, v, table, start = a
                oracle.cache_write(before[0], before[1], k, table.cpu(), start.cpu(), kw["lens"].cpu())
                oracle.cache_write(before[2], before[3], v, table.cpu(), start.cpu(), kw["lens"].cpu())
                for have, want in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), before):
                    assert torch.equal(have.cpu(), want)
            else:
                q, cache, table, lens = a
                ref = oracle.cache_attention(q, cache.k.cpu(), cache.k_scale.cpu(), cache.v.cpu(),
                                             cache.v_scale.cpu(), table.cpu(), lens.cpu())
                assert _rel(r[good.to(DEV)], ref["out"][good]) < 2.0 ** -8
        assert torch.isfinite(y[good.to(DEV)]).all()
    assert layer.held == [27, 14, 20]


def test_tokens_one_by_one_and_together():
    """A prompt through one call, or token by token, leaves the same cache, and
    rows that differ by the attention's order of sums only (two roundings of
    2^-8 and what they move)."""
    from caption_decoder import DecoderLayer
    x = _rnd(2, 9, 64, seed=5)
    one, many = (DecoderLayer(64, heads=4, kv_heads=4, head_dim=32, batch=2, max_tokens=20, seed=4)
                 for _ in range(2))
    y = one.forward(x)
    rows = [many.forward(x[:, t:t + 1]) for t in range(9)]
    for a, b in zip((one.cache.k, one.cache.k_scale, one.cache.v, one.cache.v_scale),
                    (many.cache.k, many.cache.k_scale, many.cache.v, many.cache.v_scale)):
        assert torch.equal(a, b)
    assert _rel(torch.cat(rows, 1), y) < 2.0 ** -6


def test_training_step_of_the_norm():
    """Against the formula and against differences of a loss in 64 bits."""
    from caption_decoder import DecoderLayer
    layer = DecoderLayer(96, heads=2, kv_heads=1, head_dim=32, batch=1, max_tokens=16)
    layer.norm_weight.mul_(1.3)
    x, g = _rnd(2, 11, 96, seed=6), _rnd(2, 11, 96, seed=7)
    n, (dx, dw, db) = layer.norm_step(x, g)
    r = oracle.layer_norm(x, weight=layer.norm_weight, bias=layer.norm_bias, grad=g)
    assert _rel(n, r["y"]) < 2.0 ** -8 and _rel(dx, r["dx"]) < 2.0 ** -8
    assert _rel(dw, r["dweight"]) < 2.0 ** -16 and _rel(db, r["dbias"]) < 2.0 ** -16

    def loss(xx, w, b):
        return float((oracle.layer_norm(xx, weight=w, bias=b)["y"] * g.cpu().double()).sum())

    args = [x.cpu().double(), layer.norm_weight.cpu().double(), layer.norm_bias.cpu().double()]
    for i, (grad, u) in enumerate(((dx, 2.0 ** -8), (dw, 2.0 ** -16), (db, 2.0 ** -16))):
        flat = args[i].view(-1)
        for at in (0, 17, flat.numel() - 1):
            keep, f = float(flat[at]), []
            for s in (1, -1):
                flat[at] = keep + s * 1e-5
                f.append(loss(*args))
            flat[at] = keep
            want = (f[0] - f[1]) / 2e-5
            top = float(grad.abs().max())
            assert abs(float(grad.reshape(-1)[at]) - want) <= u * top + 1e-6 * top


def test_example_runs(capsys):
    import caption_decoder
    caption_decoder.main()
    assert "finite: True" in capsys.readouterr().out
