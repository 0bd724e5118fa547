"""The decoder operators' binding: its two ways (C++ and Python) give the same
results and report the same errors."""
import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from implicit_gemm_nhwc_amd import decoder as binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class NoTruth:
    def __bool__(self):
        raise ValueError("neither true nor false")


def _run():
    """Every operator once; fresh caches, the same inputs."""
    gen = torch.Generator().manual_seed(7)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).to(DEV)

    x, dy, w = rnd(2, 5, 100), rnd(2, 5, 100), torch.rand(100, generator=gen).to(DEV)
    out = [igc.layer_norm(x, w, w, eps=1e-3), igc.layer_norm(x[0, 0]),
           *igc.layer_norm_bwd(dy, x, w, eps=1e-3)]
    q, s = igc.quantize_rows(x)
    wq, ws = igc.quantize_rows(rnd(33, 100))
    out += [q, s, igc.linear_i8(q, s, wq, ws, bias=ws, dtype=torch.float16),
            igc.linear_i8(q[0, 1], s[0, 1], wq, ws)]
    cache = igc.KVCache.empty(9, 16, 2, 40, device=DEV)
    table = torch.arange(8, device=DEV, dtype=torch.int32).view(2, 4)
    start = torch.tensor([3, 0], dtype=torch.int32, device=DEV)
    lens = torch.tensor([30, 12], dtype=torch.int32, device=DEV)
    assert igc.kv_cache_write(cache, rnd(2, 30, 2, 40), rnd(2, 30, 2, 40), table, start,
                              lens=lens) is None
    out += igc.kv_cache_read(cache, table, start, 31, lens=lens, dtype=torch.float16)
    out += igc.cache_attention(rnd(2, 3, 4, 40), cache, table, start + lens, return_lse=True)
    out += [igc.cache_attention(rnd(2, 1, 4, 40), cache, table, start + lens, causal=False,
                                scale=0.3), cache.k.clone(), cache.v_scale.clone()]
    return out


def test_both_ways(monkeypatch):
    assert binding._fast is not None
    fast = _run()
    monkeypatch.setattr(binding, "_fast", None)
    slow = _run()
    for a, b in zip(fast, slow):
        assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride()
        assert torch.equal(a, b)


@pytest.mark.parametrize("way", ["C++", "Python"])
def test_arguments_of_other_types(way, monkeypatch):
    if way == "Python":
        monkeypatch.setattr(binding, "_fast", None)
    x = torch.randn(3, 64, device=DEV).to(torch.bfloat16)
    w = torch.ones(64, device=DEV)
    with pytest.raises((TypeError, ValueError)):
        igc.layer_norm(x, w, eps="small")
    with pytest.raises(igc.InvalidArgument):
        igc.layer_norm_bwd(3, x, w)
    with pytest.raises(igc.InvalidArgument):
        igc.linear_i8(x, w, x, w)
    cache = igc.KVCache.empty(3, 16, 2, 64, device=DEV)
    q = torch.randn(1, 1, 2, 64, device=DEV).to(torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    lens = torch.ones(1, dtype=torch.int32, device=DEV)
    for kw in (dict(causal=NoTruth()), dict(return_lse=NoTruth())):
        with pytest.raises(ValueError, match="neither true nor false"):
            igc.cache_attention(q, cache, table, lens, **kw)
        assert torch.isfinite(igc.cache_attention(q, cache, table, lens)).all()
    assert torch.equal(igc.cache_attention(q, cache, table, lens, causal="yes"),
                       igc.cache_attention(q, cache, table, lens))
    with pytest.raises(AttributeError):
        cache.k = cache.v
