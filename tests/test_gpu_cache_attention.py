"""Attention over the 8-bit cache on the GPU against the float64 oracle on the
values that the cache holds.

Bounds, e = 2^-24 and u = eps / 2 of the type: a score sums D exact products in
fp32 and takes two multiplications, so it is off by (D + 16) e S, S the largest
sum of magnitudes of its row; the exponent's argument (at most 2 S + 8) rounds
once and 2^x is good to 2 e, so a probability is off by a factor eta = (D + 16)
e S + 2 (2 S + 12) e.  The output is off by 2 eta + 2^-17 (two bf16 numbers
hold a probability) + 2 (n / 8 + 100) e (its sums: the keys of one of eight
waves) of sum p |v|, and one rounding."""
import os

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from oracle import decoder as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16
E = 2.0 ** -24


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


def _pool(b, entries, hk, d, page, lens, seed=3, spare=2):
    """Cache and table of sequences of lens tokens; every place that none of
    them holds has a NaN scale and noise."""
    gen = torch.Generator().manual_seed(seed)
    pages = b * entries + spare
    table = torch.randperm(pages, generator=gen)[:b * entries].view(b, entries).to(torch.int32)
    cache = igc.KVCache.empty(pages, page, hk, d, device=DEV)
    for q, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        q.copy_(torch.randint(-128, 128, q.shape, generator=gen, dtype=torch.int8))
        w = torch.full(s.shape, float("nan"))
        for i, n in enumerate(lens):
            for j in range(entries):
                m = min(max(n - j * page, 0), page)
                w[table[i, j], :, :m] = 0.02 + 0.02 * torch.rand(hk, m, generator=gen)
        s.copy_(w)
    return cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def _q(dt, b, tq, hq, d, seed=1):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(b, tq, hq, d, generator=gen).to(dt).to(DEV)


def _check(q, cache, table, lens, out, lse, **kw):
    dt, d = q.dtype, q.shape[3]
    o = oracle.cache_attention(q, cache.k.cpu(), cache.k_scale.cpu(), cache.v.cpu(),
                               cache.v_scale.cpu(), table.cpu(), lens.cpu(), **kw)
    s = o["s_abs"].permute(0, 2, 1)[..., None]
    n = o["n"][:, :, None, None].double()
    eta = (d + 16) * E * s + 2 * (2 * s + 12) * E
    bound = (torch.finfo(dt).eps / 2 * o["out"].abs() + 2.0 ** -25
             + o["out_abs"] * (2 * eta + 2.0 ** -17 + 2 * (n / 8 + 100) * E))
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    far = (got - o["out"]).abs()
    print(f"    out: {float((far / bound).max()):.3f} of the bound", flush=True)
    assert (far <= bound).all()
    if lse is not None:
        ref = o["lse"]
        assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(ref))
        ok = torch.isfinite(ref)
        lim = (eta + (n / 8 + 100) * E).permute(0, 2, 1, 3)[..., 0] + 4 * E * ref.abs() + 4 * E
        assert ((lse.cpu().double() - ref).abs()[ok] <= lim.expand_as(ref)[ok]).all()


CASES = [
    # dt, q tokens, q heads, kv heads, d, page, entries, lengths
    (BF, 1, 1, 1, 8, 16, 1, [1]),
    (HF, 1, 4, 4, 16, 16, 2, [0, 17, 32]),
    (BF, 1, 16, 4, 128, 16, 50, [784, 1, 33, 400]),
    (HF, 5, 8, 8, 80, 32, 5, [129, 3, 160, 5, 0, 64]),
    (BF, 8, 8, 2, 40, 64, 3, [130, 192, 7]),              # 32 rows a key head
    (HF, 3, 24, 2, 64, 16, 9, [140, 2, 33]),              # 36 rows: two tiles
    (BF, 70, 3, 1, 96, 128, 2, [200, 70, 30]),            # 210 rows, more than a sequence
    (HF, 1, 8, 8, 128, 64, 20, [1280, 1000, 3]),          # split between workgroups
    (BF, 2, 6, 2, 72, 32, 160, [5100, 0, 2049, 1, 777]),
    (HF, 4, 4, 1, 24, 16, 130, [2080, 1030]),
    (BF, 1, 2, 1, 56, 16, 70, [(97 * i) % 1121 for i in range(100)]),   # sequences past a wave
    (HF, 1, 40, 1, 128, 256, 13, [3071, 2500]),           # two row tiles, split
    (BF, 1, 10, 10, 128, 1024, 3, [2000]),
    # prompts: a causal row tile stops where its last row does, parts of a split
    # may hold none of its keys
    (BF, 300, 4, 2, 64, 64, 40, [2500, 300, 150]),
    (HF, 1200, 2, 1, 32, 32, 40, [1280]),
    (BF, 90, 12, 12, 128, 16, 7, [90, 112, 1]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[7])}x{c[1]}-{c[2]}.{c[3]}.{c[4]}-{c[5]}")
def test_against_the_oracle(case):
    print(f"cache attention {case}", flush=True)
    dt, tq, hq, hk, d, page, entries, lens = case
    cache, table, n = _pool(len(lens), entries, hk, d, page, lens)
    q = _q(dt, len(lens), tq, hq, d)
    for causal in (True, False):
        out, lse = igc.cache_attention(q, cache, table, n, causal=causal, return_lse=True)
        _check(q, cache, table, n, out, lse, causal=causal)
        assert torch.equal(igc.cache_attention(q, cache, table, n, causal=causal), out)
        with igc.using_library(igc.POISON_LIB_PATH):
            assert torch.equal(igc.cache_attention(q, cache, table, n, causal=causal), out)


# the sequences of these share what room there is by their lengths, past a wave's
# 64 of them too; one and two row tiles, one and several key heads
DIVIDED = [
    (BF, 1, 2, 1, 128, 16, 128, [2048, 0, 1, 300, 129, 2047, 7, 256] + [0, 1, 640, 90] * 23),
    (HF, 2, 4, 2, 64, 32, 22, [704, 703, 0, 1, 257] * 20),
    (BF, 1, 3, 1, 40, 16, 44, [(97 * i) % 705 for i in range(200)]),
    (HF, 8, 4, 1, 32, 32, 35, [1120, 5, 0, 900, 256] * 14),
    (BF, 1, 32, 32, 64, 64, 64, [4096, 1, 2300]),
    (HF, 5, 32, 32, 80, 16, 256, [4095, 3, 0]),
    (BF, 5, 24, 8, 128, 128, 64, [8192, 4100, 129]),
]


def _divided(q_shape, cache, entries, dt):
    """Whether a call's workspace holds fewer parts than every sequence's own
    slots would take (256 keys a part at least)."""
    b, tq, hq, d = q_shape
    rows, most = tq * hq // cache.kv_heads, -(-(entries * cache.k.shape[2]) // 256)
    a_part = cache.kv_heads * (rows if rows <= 16 else -(-rows // 32) * min(rows, 32)) * (d + 2) * 4
    room, rest = divmod(igc.cache_attn_fwd_workspace_bytes(q_shape, cache, entries, dt), a_part)
    assert rest == 0
    return b < room < b * most


@pytest.mark.parametrize("case", DIVIDED, ids=lambda c: f"{len(c[7])}x{c[1]}-{c[2]}.{c[3]}.{c[4]}-{c[5]}")
def test_division_by_lengths(case):
    print(f"cache attention, divided {case[:7]}", flush=True)
    dt, tq, hq, hk, d, page, entries, lens = case
    cache, table, n = _pool(len(lens), entries, hk, d, page, lens)
    q = _q(dt, len(lens), tq, hq, d)
    assert _divided(q.shape, cache, entries, dt)
    out, lse = igc.cache_attention(q, cache, table, n, return_lse=True)
    _check(q, cache, table, n, out, lse)
    full = igc.cache_attention(q, cache, table, n, causal=False)
    if tq == 1:
        assert torch.equal(full, out)
    for again in range(2):
        assert torch.equal(igc.cache_attention(q, cache, table, n), out)
        with igc.using_library(igc.POISON_LIB_PATH):
            assert torch.equal(igc.cache_attention(q, cache, table, n), out)
            assert torch.equal(igc.cache_attention(q, cache, table, n, causal=False), full)


def test_a_captured_launch_divides_anew():
    """Between the replays of a graph the lengths change, and with them the
    division: each replay's bits are an eager call's, and each is checked."""
    cache, table, n = _pool(4, 100, 16, 64, 16, [1600, 1600, 1600, 1600])
    q = _q(HF, 4, 2, 32, 64)
    assert _divided(q.shape, cache, 100, HF)
    igc.cache_attention(q, cache, table, n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = igc.cache_attention(q, cache, table, n, return_lse=True)
    for i, lens in enumerate(([1600, 0, 3, 700], [0, 0, 0, 0], [1, 1600, 1600, 2], [5, 1, 0, 1599])):
        q.copy_(torch.randn(q.shape, device=DEV))
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        a, b = igc.cache_attention(q, cache, table, n, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, lse)
        _check(q, cache, table, n, out, lse)


def test_rows_that_attend_to_nothing():
    cache, table, n = _pool(3, 2, 2, 64, 16, [0, 2, 5])
    q = _q(BF, 3, 4, 4, 64)
    out, lse = igc.cache_attention(q, cache, table, n, return_lse=True)
    _check(q, cache, table, n, out, lse)
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all() and (out[1, :2] == 0).all()
    for value in (-5, -(1 << 31)):
        n[2] = value
        out = igc.cache_attention(q, cache, table, n)
        assert (out[2] == 0).all()


def test_lengths_past_the_table():
    cache, table, n = _pool(2, 2, 1, 32, 16, [32, 20])
    q = _q(HF, 2, 1, 2, 32)
    want = igc.cache_attention(q, cache, table, n)
    n[0] = (1 << 31) - 1
    assert torch.equal(igc.cache_attention(q, cache, table, n), want)
    # new tokens keep their places when some lie past the table (padding)
    for entries, tq, lens in ((3, 6, [50, 45]), (80, 4, [1282, 1281])):
        cache, table, n = _pool(2, entries, 1, 32, 16, lens)
        q = _q(BF, 2, tq, 2, 32)
        out, lse = igc.cache_attention(q, cache, table, n, return_lse=True)
        _check(q, cache, table, n, out, lse)
        short = n - 2
        assert torch.equal(igc.cache_attention(q[:, :-2], cache, table, short), out[:, :-2])


def test_pages_outside_the_pool():
    """Rows that attend to such a page are NaN, the others as they were."""
    cache, table, n = _pool(4, 70, 2, 64, 16, [1100, 40, 17, 1120])
    q = _q(BF, 4, 2, 4, 64)
    want = igc.cache_attention(q, cache, table, n)
    for bad in (-1, cache.k.shape[0], (1 << 31) - 1):
        t = table.clone()
        t[0, 68] = bad       # its last tokens but for 12
        t[1, 3] = bad        # past its length
        t[2, 1] = bad        # its last token, which the first new one does not see
        out = igc.cache_attention(q, cache, t, n)
        assert torch.isnan(out[0]).all() and torch.equal(out[1], want[1])
        assert torch.isnan(out[2, 1]).all() and torch.equal(out[2, 0], want[2, 0])
        assert torch.equal(out[3], want[3])


def test_a_token_of_nans_is_seen_from_it_on():
    cache, table, n = _pool(1, 3, 1, 64, 16, [40])
    q = _q(HF, 1, 4, 2, 64)
    want = igc.cache_attention(q, cache, table, n)
    for s in (cache.k_scale, cache.v_scale):
        keep = s.clone()
        s[table[0, 2], 0, 38 - 32] = float("nan")
        out = igc.cache_attention(q, cache, table, n)
        assert torch.equal(out[0, :2], want[0, :2]) and torch.isnan(out[0, 2:]).all()
        s.copy_(keep)


def test_extreme_scores_and_scales():
    """Scores of hundreds, scales far apart, a scale of zero."""
    for dt in (BF, HF):
        cache, table, n = _pool(2, 8, 2, 128, 16, [128, 90])
        cache.k_scale.mul_(20.0)
        cache.v_scale[..., ::3] *= 1e-4
        cache.v_scale[..., 1::5] *= 300.0
        cache.k_scale[table[1, 1].long(), :, 3] = 0.0
        cache.v_scale[table[1, 2].long(), :, 4] = 0.0
        q = _q(dt, 2, 1, 8, 128)
        out, lse = igc.cache_attention(q, cache, table, n, return_lse=True)
        _check(q, cache, table, n, out, lse)
        out = igc.cache_attention(q, cache, table, n, scale=0.5)
        _check(q, cache, table, n, out, None, scale=0.5)


def _edge(entries, hk, tq, lens, page=16, d=64, dt=BF):
    """Pool, table, lengths and queries of four heads a key head."""
    cache, table, n = _pool(len(lens), entries, hk, d, page, lens)
    return cache, table, n, _q(dt, len(lens), tq, 4 * hk, d)


# whole sequences, slots of their own, a division by lengths; one and two row tiles
EDGES = [(3, 2, 1, [1, 40, 0]), (4, 2, 3, [2, 61, 64]), (100, 2, 2, [1600, 700, 1]),
         (300, 16, 1, [4800, 1, 300]), (60, 4, 9, [950, 8, 640])]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("edge", EDGES, ids=str)
def test_rows_whose_scores_are_all_minus_infinity_are_nan(edge, dt):
    """An infinite value of a query makes each of its row's scores infinite; the
    row is NaN by the definition, and zeros are what a row without a key has.
    Rows beside it keep their bits."""
    cache, table, n, q = _edge(*edge, dt=dt)
    cache.k[..., 5].copy_(cache.k[..., 5].abs().clamp(1, 127))
    b, tq, hq, _ = q.shape
    want, lse0 = igc.cache_attention(q, cache, table, n, return_lse=True)
    for value in (-torch.inf, torch.inf, torch.nan):
        for rows in ((slice(None), slice(None), slice(1, None, 3)), (slice(None), 0), (0,)):
            hit = torch.zeros(b, tq, hq, dtype=torch.bool, device=DEV)
            hit[rows] = True
            bad = q.clone()
            bad[..., 5] = torch.where(hit, value, bad[..., 5].float()).to(dt)
            for causal in (True, False):
                first = n[:, None] - (torch.arange(tq - 1, -1, -1, device=DEV) if causal else 0)
                hit_now = hit & (first > 0)[..., None]
                if not causal:
                    want_now, lse_now = igc.cache_attention(q, cache, table, n, causal=False,
                                                            return_lse=True)
                else:
                    want_now, lse_now = want, lse0
                out, lse = igc.cache_attention(bad, cache, table, n, causal=causal,
                                               return_lse=True)
                hit_lse = hit_now.transpose(1, 2)
                assert out[hit_now].isnan().all() and lse[hit_lse].isnan().all()
                assert torch.equal(out[~hit_now], want_now[~hit_now])
                assert torch.equal(lse[~hit_lse], lse_now[~hit_lse])


@pytest.mark.parametrize("edge", [(8, 2, 1, [128, 100, 70]), (100, 2, 2, [1600, 700, 90]),
                                  (300, 16, 1, [4800, 80, 300]), (60, 4, 9, [950, 80, 640])],
                         ids=str)
def test_keys_of_minus_infinity_beside_finite_ones(edge):
    """Scores past fp32's range, of whole blocks, waves and splits: as scores of
    -1000 would, they leave the others their weights, to the bit."""
    cache, table, n, q = _edge(*edge)
    cache.k[..., 5] = -100
    place = torch.arange(32, 64, device=DEV)
    cache.k[table.long()[:, place // 16], :, (place % 16), 5] = 0
    for causal in (True, False):
        got = []
        for value in (1e38, 1e5):
            q[..., 5] = value
            got.append(igc.cache_attention(q, cache, table, n, causal=causal, return_lse=True))
        assert torch.isfinite(got[0][0]).all()
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_strides_guards_and_workspace():
    cache, table, n = _pool(3, 70, 2, 80, 16, [1100, 40, 1117])
    dense = _q(BF, 3, 3, 8, 80)
    want, lse = igc.cache_attention(dense, cache, table, n, return_lse=True)
    wide = _q(BF, 3, 3, 20, 96, seed=9)
    part = wide[:, :, 4:12, 8:88]
    part.copy_(dense)
    assert torch.equal(igc.cache_attention(part, cache, table, n), want)
    heads_first = dense.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(igc.cache_attention(heads_first, cache, table, n), want)
    one = dense[:1].expand(3, 3, 8, 80)
    assert torch.equal(igc.cache_attention(one, cache, table, n)[0], want[0])
    pad = torch.full((3, 5, 10, 96), 3.0, dtype=BF, device=DEV)
    out = pad[:, 1:4, 1:9, 8:88]
    need = igc.cache_attn_fwd_workspace_bytes(dense.shape, cache, 70, BF)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    l2 = torch.empty_like(lse)
    assert igc.cache_attn_fwd(dense, cache, table, n, out, lse=l2, workspace=ws,
                              workspace_bytes=need) == 1
    assert torch.equal(out, want) and torch.equal(l2, lse) and (ws[need:] == 255).all()
    assert igc.cache_attn_fwd(dense, cache, table, n, out) == 1 and torch.equal(out, want)
    out.fill_(3.0)
    assert (pad == 3.0).all()
    wider = torch.zeros(3, 100, dtype=torch.int32, device=DEV)
    wider[:, 5:75] = table
    assert torch.equal(igc.cache_attention(dense, cache, wider[:, 5:75], n), want)
    shared = table[:1].expand(3, 70)
    same = igc.cache_attention(dense, cache, shared, n[:1].expand(3).contiguous())
    assert torch.equal(same[0], want[0])


def test_empty_extents():
    cache, table, n = _pool(2, 2, 2, 32, 16, [20, 5])
    for b, tq, hq in ((0, 1, 4), (2, 0, 4), (2, 1, 0)):
        q = torch.zeros(b, tq, hq, 32, dtype=BF, device=DEV)
        assert igc.cache_attention(q, cache, table[:b], n[:b]).shape == q.shape
        long = torch.zeros(b, 200, dtype=torch.int32, device=DEV)
        assert igc.cache_attention(q, cache, long, n[:b]).shape == q.shape
    q = _q(BF, 2, 1, 4, 32)
    out = igc.cache_attention(q, cache, table[:, :0], n)
    assert (out == 0).all()
    # a pool without pages: every page of a table is outside it
    none = igc.KVCache.empty(0, 16, 2, 32, device=DEV)
    n[1] = 0
    for entries in (2, 200):
        t = torch.zeros(2, entries, dtype=torch.int32, device=DEV)
        out, lse = igc.cache_attention(q, none, t, n, return_lse=True)
        assert out[0].isnan().all() and lse[0].isnan().all()
        assert (out[1] == 0).all() and torch.isinf(lse[1]).all()
        new = _q(BF, 2, 40, 4, 32)   # the first 20 attend to nothing
        out = igc.cache_attention(new, none, t, n)
        assert (out[0, :20] == 0).all() and out[0, 20:].isnan().all() and (out[1] == 0).all()


def test_graph_and_stream():
    """Lengths and queries change between the replays; the division of the work
    follows the lengths."""
    cache, table, n = _pool(4, 100, 2, 64, 16, [1600, 1600, 1600, 1600])
    q = _q(HF, 4, 2, 8, 64)
    igc.cache_attention(q, cache, table, n)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = igc.cache_attention(q, cache, table, n)
    with torch.cuda.graph(g2):
        out2 = igc.cache_attention(q, cache, table, n, causal=False)
    s = torch.cuda.Stream()
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=DEV))
        n.copy_(torch.randint(0, 1601, n.shape, device=DEV))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for st in (s, s.cuda_stream):
            a = igc.cache_attention(q, cache, table, n, stream=st)
            b = igc.cache_attention(q, cache, table, n, causal=False, stream=st)
            s.synchronize()
            assert torch.equal(a, out) and torch.equal(b, out2)


def test_written_tokens_are_attended_to():
    """Write, then attend, step by step: against the oracle on the values that
    the cache holds."""
    cache, table, n = _pool(2, 4, 2, 64, 16, [0, 0])
    gen = torch.Generator().manual_seed(4)
    at = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    for t in (20, 1, 1, 3):
        k, v = (torch.randn(2, t, 2, 64, generator=gen).to(BF).to(DEV) for _ in range(2))
        igc.kv_cache_write(cache, k, v, table, at)
        at += t
        q = torch.randn(2, t, 4, 64, generator=gen).to(BF).to(DEV)
        out, lse = igc.cache_attention(q, cache, table, at, return_lse=True)
        _check(q, cache, table, at, out, lse)


def test_binding_refusals():
    cache, table, n = _pool(2, 2, 2, 32, 16, [20, 5])
    q = _q(BF, 2, 1, 4, 32)
    good = dict(q=q, cache=cache, table=table, lens=n)
    for bad in (dict(q=q.float()), dict(q=q[..., :16]), dict(q=q.cpu()), dict(q=q[0]), dict(q=None),
                dict(table=table.long()), dict(table=table[:1]), dict(lens=n.long()),
                dict(lens=n[:1]), dict(lens=None), dict(cache=None), dict(lens=n.cpu())):
        a = {**good, **bad}
        with pytest.raises(igc.InvalidArgument):
            igc.cache_attention(a["q"], a["cache"], a["table"], a["lens"])
    with pytest.raises(igc.Declined, match="groups"):
        igc.cache_attention(q[:, :, :3], cache, table, n)
    for scale in (0.0, -1.0, float("nan"), 1e300):
        with pytest.raises(igc.Declined, match="scale"):
            igc.cache_attention(q, cache, table, n, scale=scale)
    assert igc.cache_attn_fwd(q, cache, table, n, q) == 0
    lse = torch.empty(2, 4, 2, device=DEV)
    with pytest.raises(igc.InvalidArgument):
        igc.cache_attn_fwd(q, cache, table, n, torch.empty_like(q), lse=lse)
