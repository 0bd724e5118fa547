"""Rows in 8 bits and the paged cache on the GPU: integers and scales equal to
the oracle's, bit by bit; read-back values within one rounding to the type (u =
eps / 2) and one of the fp32 product."""
import math
import os

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from oracle import decoder as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


def _rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _same_rows(x, q, scale):
    want, step = oracle.rows_i8(x)
    assert torch.equal(q.cpu().double(), want)
    assert torch.equal(scale.cpu().nan_to_num(-1.0), step.nan_to_num(-1.0))


ROWS = [(BF, (1,), 1), (HF, (3,), 7), (BF, (2, 5), 16), (HF, (33,), 64), (BF, (4, 3, 2), 100),
        (HF, (70,), 130), (BF, (9,), 256), (HF, (31,), 333), (BF, (300,), 512), (HF, (8,), 1000),
        (BF, (8,), 1024), (HF, (5,), 2048), (BF, (3,), 3001), (HF, (7,), 4096), (BF, (2,), 8192),
        (HF, (3,), 11008), (BF, (2,), 16384), (HF, (2,), 16385), (BF, (3,), 40000),
        (HF, (1,), 131071)]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{'x'.join(map(str, c[1]))}-{c[2]}")
def test_quantize_rows(case):
    print(f"quantize rows {case}", flush=True)
    dt, lead, c = case
    x = _rnd(*lead, c, seed=1).to(dt).to(DEV)
    q, scale = igc.quantize_rows(x)
    assert q.shape == x.shape and scale.shape == x.shape[:-1] and q.dtype == torch.int8
    _same_rows(x, q, scale)
    with igc.using_library(igc.POISON_LIB_PATH):
        q2, s2 = igc.quantize_rows(x)
    assert torch.equal(q, q2) and torch.equal(scale, s2)


def test_quotients_on_and_beside_the_half_steps():
    """Maxima of every significand with values at, above and below the middle
    between two steps; bf16 and fp16, several powers of two."""
    for dt, bits, powers in ((BF, 8, (-118, -66, -62, 0, 90, 119)), (HF, 11, (-14, -10, 0, 4))):
        rows = []
        for m in range(1 << (bits - 1), 1 << bits, 1 if bits == 8 else 37):
            k = torch.arange(0, 127).double()
            x = (2 * k + 1) * m / 254
            near = x.to(dt).double()
            step = 2.0 ** (torch.floor(torch.log2(near)) - (bits - 1))
            row = torch.cat([near, near + step, near - step, torch.tensor([float(m)]).double()])
            rows.append(row.clamp(max=float(m)))
        x = torch.stack(rows)
        x[1::2] *= -1
        for p in powers:
            y = (x * 2.0 ** (p - (bits - 1 if dt == HF else 0))).to(dt).to(DEV)
            assert torch.isfinite(y).all()
            _same_rows(y, *igc.quantize_rows(y))


def test_rows_of_zeros_infinities_and_nans():
    for dt in (BF, HF):
        x = _rnd(7, 40, seed=2).to(dt)
        x[0] = 0
        x[1, 3] = math.inf
        x[2, 39] = -math.inf
        x[3, 0] = math.nan
        x[4] = 0
        x[4, 7] = -0.0
        x[5] = torch.finfo(dt).max
        q, scale = igc.quantize_rows(x.to(DEV))
        _same_rows(x, q, scale)
        assert torch.isnan(scale[1:4]).all() and (q[1:4] == 0).all() and scale[0] == 0
        assert (q[5] == 127).all() and torch.isfinite(scale[6])
    tiny = torch.full((2, 24), 2.0 ** -112).to(BF)
    tiny[1] = 2.0 ** -110
    q, scale = igc.quantize_rows(tiny.to(DEV))
    assert (q[0] == 0).all() and scale[0] == 0 and (q[1] == 127).all() and scale[1] > 0


def test_quantize_strides_and_refusals():
    big = _rnd(3, 9, 11, 57, seed=3).to(BF).to(DEV)
    for x in (big[:, 2:7, 1:9, 3:43], big[1, ::3, :, :40], big[0, 0, ::2, 1:41],
              big[:1, :1, :1, 7:47].expand(3, 4, 5, 40), big.transpose(0, 1)[..., :40]):
        q, s = igc.quantize_rows(x)
        q2, s2 = igc.quantize_rows(x.contiguous())
        assert torch.equal(q, q2) and torch.equal(s, s2)
    for shape in ((0, 24), (2, 0, 24)):
        q, s = igc.quantize_rows(torch.zeros(shape, dtype=BF, device=DEV))
        assert q.shape == shape and s.shape == shape[:-1]
    for bad in (big.float(), big.cpu(), big.transpose(2, 3), [1], big[0, 0, 0, 0]):
        with pytest.raises(igc.InvalidArgument):
            igc.quantize_rows(bad)
    with pytest.raises(igc.Declined, match="size_limit"):
        igc.quantize_rows(torch.zeros(1, 131072, dtype=BF, device=DEV))


CACHES = [
    # dt, b, t, heads, d, page, lengths given, fused projection
    (BF, 1, 1, 1, 8, 16, False, False),
    (HF, 3, 1, 4, 128, 16, False, True),
    (BF, 2, 17, 3, 40, 16, True, True),
    (HF, 4, 50, 5, 64, 32, True, False),
    (BF, 3, 130, 8, 80, 64, True, True),
    (HF, 2, 33, 9, 96, 128, False, False),
    (BF, 70, 5, 2, 24, 16, True, False),
    (HF, 1, 300, 2, 120, 1024, False, True),
]


def _setup(case):
    dt, b, t, h, d, page, lens, fused = case
    gen = torch.Generator().manual_seed(5)
    first = torch.randint(0, 40, (b,), generator=gen, dtype=torch.int32)
    per = -(-(t + 40) // page)
    pages = b * per + 3
    table = torch.randperm(pages, generator=gen)[:b * per].view(b, per).to(torch.int32)
    n = torch.randint(0, t + 1, (b,), generator=gen, dtype=torch.int32) if lens else None
    kv = _rnd(b, t, 2, h, d, seed=6).to(dt).to(DEV)
    k, v = kv[:, :, 0], kv[:, :, 1]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    cache = igc.KVCache.empty(pages, page, h, d, device=DEV)
    # what is there stays: noise in all of it
    cache.k.copy_(torch.randint(-128, 128, cache.k.shape, generator=gen))
    cache.v.copy_(torch.randint(-128, 128, cache.v.shape, generator=gen))
    cache.k_scale.copy_(_rnd(*cache.k_scale.shape, seed=7))
    cache.v_scale.copy_(_rnd(*cache.v_scale.shape, seed=8))
    return cache, k, v, table, first, n


@pytest.mark.parametrize("case", CACHES, ids=lambda c: f"{c[1]}x{c[2]}-{c[3]}.{c[4]}-{c[5]}")
def test_write_and_read(case):
    print(f"cache {case}", flush=True)
    dt, b, t, h, d, page, _, _ = case
    cache, k, v, table, first, n = _setup(case)
    want = [x.cpu().clone() for x in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    oracle.cache_write(want[0], want[1], k, table, first, n)
    oracle.cache_write(want[2], want[3], v, table, first, n)
    args = [x.to(DEV) for x in (table, first)]
    lens = None if n is None else n.to(DEV)
    igc.kv_cache_write(cache, k, v, *args, lens=lens)
    for x, y in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), want):
        assert torch.equal(x.cpu(), y)
    # read back, in both types, from the same places
    for out in (BF, HF):
        got = igc.kv_cache_read(cache, *args, t, lens=lens, dtype=out)
        for x, q, s in zip(got, (want[0], want[2]), (want[1], want[3])):
            assert x.shape == (b, t, h, d) and x.dtype == out and x.is_contiguous()
            for i in range(b):
                m = t if n is None else int(n[i])
                ref = oracle.cache_rows(q, s, table[i].tolist(), int(first[i]) + m, d)[int(first[i]):]
                u = torch.finfo(out).eps / 2 + 2.0 ** -24
                far = (x[i, :m].cpu().double() - ref).abs()
                assert (far <= u * ref.abs() + 2.0 ** -25).all()
                assert (x[i, m:] == 0).all()


def test_positions_and_pages_that_do_not_exist():
    """Left out by the write, NaN in the read, everything else untouched."""
    d, h, page = 64, 2, 16
    cache = igc.KVCache.empty(4, page, h, d, device=DEV)
    table = torch.tensor([[0, -1, 2], [4, 3, 1 << 30], [1, 1, 1]], dtype=torch.int32, device=DEV)
    start = torch.tensor([-3, 10, 40], dtype=torch.int32, device=DEV)
    k, v = _rnd(3, 20, h, d, seed=1).to(BF).to(DEV), _rnd(3, 20, h, d, seed=2).to(BF).to(DEV)
    igc.kv_cache_write(cache, k, v, table, start)
    want = [x.cpu().clone().zero_() for x in (cache.k, cache.k_scale)]
    oracle.cache_write(*want, k[:2], table[:2].cpu(), start[:2].cpu())
    for p in (0, 2, 3):
        assert torch.equal(cache.k[p].cpu(), want[0][p])
        assert torch.equal(cache.k_scale[p].cpu(), want[1][p])
    got, _ = igc.kv_cache_read(cache, table, start, 20)
    there = torch.isfinite(got).all(-1).all(-1).cpu()
    for b in range(3):
        for t in range(20):
            p = int(start[b]) + t
            assert bool(there[b, t]) == (oracle.cache_place(table[b].tolist(), p, page, 4) is not None)
    assert torch.isnan(got[~there.to(DEV)]).all()


def test_rows_of_nans_stay_recognisable():
    cache = igc.KVCache.empty(2, 16, 1, 32, device=DEV)
    k = _rnd(1, 3, 1, 32).to(HF)
    k[0, 1, 0, 5] = math.nan
    k[0, 2] = 0
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    igc.kv_cache_write(cache, k.to(DEV), k.to(DEV), table, zero)
    got, _ = igc.kv_cache_read(cache, table, zero, 3, dtype=HF)
    assert torch.isnan(got[0, 1]).all() and (got[0, 2] == 0).all() and torch.isfinite(got[0, 0]).all()


def test_offsets_past_32_bits():
    """The last pages of a pool of 4.8 GB a tensor."""
    pages, page, h, d = 36700, 128, 8, 128
    cache = igc.KVCache.empty(pages, page, h, d, device=DEV)
    assert cache.k.numel() > 1 << 32
    table = torch.tensor([[pages - 1, 5, pages - 2]], dtype=torch.int32, device=DEV)
    start = torch.tensor([100], dtype=torch.int32, device=DEV)
    k, v = _rnd(1, 200, h, d, seed=1).to(BF).to(DEV), _rnd(1, 200, h, d, seed=2).to(BF).to(DEV)
    igc.kv_cache_write(cache, k, v, table, start)
    got = igc.kv_cache_read(cache, table, start, 200)
    for x, y in zip((k, v), got):
        q, s = oracle.rows_i8(x)
        ref = q * s.double()[..., None]
        assert ((y.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs()).all()
    assert (cache.k_scale[6:pages - 2] == 0).all() and (cache.k_scale[:5] == 0).all()
    lens = torch.tensor([300], dtype=torch.int32, device=DEV)
    short = igc.KVCache(cache.k[[pages - 1, 5, pages - 2]], cache.v[[pages - 1, 5, pages - 2]],
                        cache.k_scale[[pages - 1, 5, pages - 2]],
                        cache.v_scale[[pages - 1, 5, pages - 2]], d)
    q = _rnd(1, 2, 16, d, seed=3).to(BF).to(DEV)
    same = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV)
    assert torch.equal(igc.cache_attention(q, cache, table, lens),
                       igc.cache_attention(q, short, same, lens))


def test_empty_extents():
    cache = igc.KVCache.empty(3, 16, 2, 32, device=DEV)
    none = igc.KVCache.empty(0, 16, 2, 32, device=DEV)
    for c in (cache, none):
        for b, t, e in ((0, 4, 2), (2, 0, 2), (2, 3, 0)):
            table = torch.zeros(b, e, dtype=torch.int32, device=DEV)
            start = torch.zeros(b, dtype=torch.int32, device=DEV)
            k = torch.ones(b, t, 2, 32, dtype=BF, device=DEV)
            igc.kv_cache_write(c, k, k, table, start)
            got, _ = igc.kv_cache_read(c, table, start, t)
            assert got.shape == k.shape and torch.isnan(got).all()
    assert (cache.k == 0).all() and (cache.k_scale == 0).all()


def test_graph_and_stream():
    cache, k, v, table, first, n = _setup((BF, 4, 50, 5, 64, 32, True, True))
    table, first, n = table.to(DEV), first.to(DEV), n.to(DEV)
    igc.kv_cache_write(cache, k, v, table, first, lens=n)
    igc.kv_cache_read(cache, table, first, 50, lens=n)
    torch.cuda.synchronize()
    # what the first write left, too
    other = igc.KVCache(*(x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)), 64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        igc.kv_cache_write(cache, k, v, table, first, lens=n)
        got = igc.kv_cache_read(cache, table, first, 50, lens=n)
    s = torch.cuda.Stream()
    for i in range(4):
        k.copy_(torch.randn(k.shape, device=DEV) * (i + 1))
        n.copy_(torch.randint(0, 51, n.shape, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        igc.kv_cache_write(other, k, v, table, first, lens=n, stream=s)
        want = igc.kv_cache_read(other, table, first, 50, lens=n, stream=s.cuda_stream)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(cache.k, other.k) and torch.equal(cache.k_scale, other.k_scale)


def test_binding_refusals():
    cache, k, v, table, first, n = _setup((BF, 4, 50, 5, 64, 32, True, True))
    table, first, n = table.to(DEV), first.to(DEV), n.to(DEV)
    good = dict(cache=cache, k=k, v=v, table=table, start=first, lens=n)
    for bad in (dict(k=k.half()), dict(k=k[:, :, :4]), dict(k=k[..., :32], v=v[..., :32]),
                dict(k=k.cpu()), dict(table=table.long()), dict(table=table[:2]),
                dict(table=table.t()), dict(start=first[:2]), dict(start=first.long()),
                dict(start=None), dict(lens=n.float()), dict(lens=n.cpu()), dict(cache=k),
                dict(k=k.float(), v=v.float()), dict(k=None), dict(table=None)):
        a = {**good, **bad}
        with pytest.raises(igc.InvalidArgument):
            igc.kv_cache_write(a["cache"], a["k"], a["v"], a["table"], a["start"], lens=a["lens"])
    for bad in (dict(dtype=torch.float32), dict(tokens=-1), dict(table=table[0])):
        a = {**dict(table=table, tokens=5, dtype=BF), **bad}
        with pytest.raises(igc.InvalidArgument):
            igc.kv_cache_read(cache, a["table"], first, a["tokens"], dtype=a["dtype"])
    parts = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    for i, t in enumerate((cache.k.float(), cache.v[:1], cache.k_scale.half(), cache.v_scale[0])):
        with pytest.raises(igc.InvalidArgument):
            igc.KVCache(*parts[:i], t, *parts[i + 1:], 64)
    with pytest.raises(igc.InvalidArgument):
        igc.KVCache(*parts, 48)
    same = igc.KVCache(cache.k, cache.k, cache.k_scale, cache.v_scale, 64)
    with pytest.raises(igc.Declined, match="overlap"):
        igc.kv_cache_write(same, k, v, table, first)
    odd = igc.KVCache.empty(3, 24, 5, 64, device=DEV)
    with pytest.raises(igc.Declined, match="shape"):
        igc.kv_cache_write(odd, k, v, table, first)
    wide = igc.KVCache.empty(3, 16, 5, 136, device=DEV)
    with pytest.raises(igc.Declined, match="head_dim"):
        igc.kv_cache_read(wide, table, first, 4)
