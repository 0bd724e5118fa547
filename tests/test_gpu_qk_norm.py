"""Per-head norm and rotation on the GPU against the float64 oracle.

Bounds with u = eps / 2 of the element type: one rounding of each result (u
times its value) and fp32 arithmetic before it, whose sums over a row of D
cost at most (D + 16) 2^-24 of the magnitudes of the row; the weight gradient
sums up to n rows in fp32, one thread at most n / 4 + 300 of them in a chain.
"""
import math
import os
import sys

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from oracle import attention as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


def _rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _near(name, got, ref, bound):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), name
    far = (got - ref).abs()
    print(f"    {name}: {float((far / bound.clamp_min(1e-300)).max()) if far.numel() else 0:.3f} "
          "of the bound", flush=True)
    assert (far <= bound).all(), name


def _check(dt, x, y, kw, dy=None, dx=None, dw=None):
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -24 if dt == HF else 2.0 ** -133
    d = x.shape[-1]
    zero = torch.zeros_like(x) if dy is None else dy
    r = oracle.qk_norm_rope(x, grad=zero, **kw)
    slop = (d + 16) * 2.0 ** -24
    row = r["y"].abs().amax(-1, keepdim=True) * 2
    _near("y", y, r["y"], u * r["y"].abs() + slop * row + tiny)
    if dx is not None:
        row = r["dx_abs"].amax(-1, keepdim=True) * 2
        _near("dx", dx, r["dx"], u * r["dx"].abs() + slop * row + tiny)
    if dw is not None:
        n = x.shape[0] * x.shape[1] * x.shape[2]
        chain = (n / 4 + 300 + d) * 2.0 ** -24
        _near("dweight", dw, r["dweight"], chain * r["dweight_abs"] + 1e-30)


CASES = [
    # dt, b, tq, tk, hq, hk, d, rot, positions, interleaved, weights
    (BF, 1, 1, 1, 1, 1, 8, 8, False, False, True),
    (HF, 2, 1, 1, 16, 4, 128, 128, True, False, True),
    (BF, 3, 7, 5, 5, 3, 64, 64, False, True, True),
    (HF, 1, 33, 65, 8, 8, 40, 40, True, False, True),     # 20-value halves: not whole chunks
    (BF, 2, 65, 33, 9, 1, 80, 40, True, True, True),
    (HF, 2, 19, 70, 4, 2, 96, 32, False, False, False),
    (BF, 1, 100, 3, 2, 6, 72, 72, True, False, True),
    (HF, 1, 50, 50, 3, 1, 120, 2, False, False, True),
    (BF, 2, 12, 9, 7, 7, 16, 6, True, True, False),
    (HF, 2, 12, 9, 7, 7, 24, 10, True, False, True),
    (BF, 1, 30, 4, 4, 4, 128, 0, False, False, True),     # the norm alone
    (HF, 4, 700, 300, 8, 4, 64, 64, True, False, True),
    (BF, 2, 3000, 1, 8, 8, 128, 64, False, False, True),
]


def _inputs(case, layout="dense"):
    dt, b, tq, tk, hq, hk, d, rot, given, inter, weights = case
    q, k = _rnd(b, tq, hq, d, seed=1).to(dt).to(DEV), _rnd(b, tk, hk, d, seed=2).to(dt).to(DEV)
    gq, gk = _rnd(b, tq, hq, d, seed=3).to(dt).to(DEV), _rnd(b, tk, hk, d, seed=4).to(dt).to(DEV)
    rows = max(tq, tk) + 50
    a = _rnd(rows, rot // 2, seed=5).double() * 100
    table = torch.cat([a.cos(), a.sin()], 1).float().to(DEV) if rot else None
    gen = torch.Generator().manual_seed(9)
    pos = [torch.randint(0, rows, (b, t), generator=gen, dtype=torch.int32).to(DEV) if given
           else None for t in (tq, tk)]
    w = [(1 + 0.3 * _rnd(d, seed=6 + i)).to(DEV) if weights else None for i in range(2)]
    kw = dict(q_weight=w[0], k_weight=w[1], q_table=table, k_table=table, q_positions=pos[0],
              k_positions=pos[1], eps=1e-5, interleaved=inter)
    one = [dict(weight=w[i], table=table, positions=pos[i], eps=1e-5, interleaved=inter)
           for i in range(2)]
    return q, k, gq, gk, kw, one


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}.{c[7]}")
def test_norm_and_gradients(case):
    print(f"norm {case}", flush=True)
    dt = case[0]
    q, k, gq, gk, kw, one = _inputs(case)
    yq, yk = igc.qk_norm_rope(q, k, **kw)
    dq, dk, dqw, dkw = igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    _check(dt, q, yq, one[0], gq, dq, dqw)
    _check(dt, k, yk, one[1], gk, dk, dkw)
    # queries alone give the same bits; so does a second run
    alone = {n: (None if n.startswith("k_") else v) for n, v in kw.items()}
    assert torch.equal(igc.qk_norm_rope(q, **alone), yq)
    g1 = igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    assert all(torch.equal(x, y) for x, y in zip(g1, (dq, dk, dqw, dkw)))
    g2 = igc.qk_norm_rope_bwd(gq, None, q, **alone)
    assert torch.equal(g2[0], dq) and torch.equal(g2[2], dqw) and g2[1] is None and g2[3] is None
    with igc.using_library(igc.POISON_LIB_PATH):
        assert all(torch.equal(x, y) for x, y in zip(igc.qk_norm_rope(q, k, **kw), (yq, yk)))


def test_extreme_rows():
    """Zero rows (eps alone), the largest finite values, subnormal ones."""
    for dt in (BF, HF):
        x = _rnd(1, 6, 2, 64, seed=3).to(dt)
        x[0, 0] = 0
        x[0, 1] = torch.finfo(dt).max / 64 if dt == HF else 1e17
        x[0, 2] *= 1e-6
        x = x.to(DEV)
        gy = _rnd(1, 6, 2, 64, seed=4).to(dt).to(DEV)
        y = igc.qk_norm_rope(x, eps=1e-6)
        dx, _, dw, _ = igc.qk_norm_rope_bwd(gy, None, x, eps=1e-6)
        _check(dt, x, y, dict(eps=1e-6), gy, None, dw)
        assert (y[0, 0] == 0).all() and torch.isfinite(y).all()
    x[0, 3, 1, 5] = math.nan
    y = igc.qk_norm_rope(x)
    assert torch.isnan(y[0, 3, 1]).all() and torch.isfinite(y[0, 3, 0]).all()


def test_positions_outside_the_table():
    q, table = _rnd(2, 3, 2, 64).to(BF).to(DEV), igc.rope_table(10, 32, device=DEV)
    pos = torch.tensor([[0, 10, 9], [-1, 1 << 30, -(1 << 31)]], dtype=torch.int32, device=DEV)
    y = igc.qk_norm_rope(q, q_table=table, q_positions=pos)
    dx = igc.qk_norm_rope_bwd(q, None, q, q_table=table, q_positions=pos)[0]
    for t in (y, dx):
        ok = torch.isfinite(t).all(-1).all(-1).cpu()
        assert ok.tolist() == [[True, False, True], [False, False, False]]
    assert torch.isfinite(y[..., 32:]).all()     # values that do not turn


def test_strides_in_place_and_guards():
    """Slices of a fused projection, in place and into padded outputs."""
    b, t, hq, hk, d = 2, 45, 6, 3, 64
    table = igc.rope_table(64, d, device=DEV)
    w = (1 + 0.1 * _rnd(d)).to(DEV)
    kw = dict(q_weight=w, k_weight=w, q_table=table, k_table=table)
    qkv = _rnd(b, t, hq + 2 * hk, d).to(HF).to(DEV)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    yq, yk = igc.qk_norm_rope(q.contiguous(), k.contiguous(), **kw)
    sq, sk = igc.qk_norm_rope(q, k, **kw)
    assert torch.equal(sq, yq) and torch.equal(sk, yk)
    pad = torch.full((b, t + 2, hq + 2, d + 16), 3.0, dtype=HF, device=DEV)
    ko = torch.empty_like(yk)
    assert igc.qk_norm_rope_fwd(q, k, pad[:, 1:-1, 1:-1, 8:-8], ko, **kw) == 1
    assert torch.equal(pad[:, 1:-1, 1:-1, 8:-8], yq)
    pad[:, 1:-1, 1:-1, 8:-8] = 3.0
    assert (pad == 3.0).all()
    both = qkv.clone()
    q2, k2 = both[:, :, :hq], both[:, :, hq:hq + hk]
    assert igc.qk_norm_rope_fwd(q2, k2, q2, k2, **kw) == 1
    assert torch.equal(q2, yq) and torch.equal(k2, yk)
    assert torch.equal(both[:, :, hq + hk:], qkv[:, :, hq + hk:])
    # shared input through stride 0
    x = _rnd(1, t, hq, d).to(HF).to(DEV)
    e = igc.qk_norm_rope(x.expand(3, t, hq, d), q_weight=w, q_table=table)
    assert torch.equal(e[2], igc.qk_norm_rope(x, q_weight=w, q_table=table)[0])


def test_head_major_rows():
    """Heads further apart than 2^23 elements, in place in a cache."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    cache = torch.randn(1, 2, 70000, 128, device=DEV, generator=gen).to(torch.bfloat16)
    k = cache.transpose(1, 2)
    assert k.stride(2) > 1 << 23
    g = torch.randn(1, 70000, 2, 128, device=DEV, generator=gen).to(torch.bfloat16)
    table = igc.rope_table(70000, 128, device=DEV)
    want = igc.qk_norm_rope(k.contiguous(), q_table=table)
    assert torch.equal(igc.qk_norm_rope(k, q_table=table), want)
    for x, y in zip(igc.qk_norm_rope_bwd(g, None, k, q_table=table),
                    igc.qk_norm_rope_bwd(g, None, k.contiguous(), q_table=table)):
        assert x is y is None or torch.equal(x, y)


def test_empty_extents():
    table = igc.rope_table(8, 64, device=DEV)
    for shape in ((0, 4, 2, 64), (2, 0, 2, 64), (2, 4, 0, 64)):
        q = torch.zeros(shape, dtype=BF, device=DEV)
        k = _rnd(1, 3, 2, 64).to(BF).to(DEV)
        kw = dict(q_table=table, k_table=table)
        yq, yk = igc.qk_norm_rope(q, k, **kw)
        assert yq.shape == q.shape and torch.isfinite(yk).all()
        dq, dk, dqw, dkw = igc.qk_norm_rope_bwd(q, k, q, k, **kw)
        assert (dqw == 0).all() and (dkw != 0).any() and dq.shape == q.shape
        assert igc.qk_norm_rope(q, **{"q_table": table}).shape == q.shape


def test_graph_and_stream():
    case = (BF, 2, 70, 30, 4, 2, 64, 64, True, False, True)
    q, k, gq, gk, kw, _ = _inputs(case)
    igc.qk_norm_rope(q, k, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = igc.qk_norm_rope(q, k, **kw)
        d = igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    s = torch.cuda.Stream()
    for n in range(4):
        for t in (q, k, gq, gk):
            t.copy_(torch.randn(t.shape, device=DEV) * (n + 1))
        g.replay()
        torch.cuda.synchronize()
        y2 = igc.qk_norm_rope(q, k, stream=s, **kw)
        d2 = igc.qk_norm_rope_bwd(gq, gk, q, k, stream=s.cuda_stream, **kw)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y + d, y2 + d2))


def test_binding_refusals():
    q, k = _rnd(2, 5, 4, 64).to(BF).to(DEV), _rnd(2, 3, 2, 64).to(BF).to(DEV)
    table = igc.rope_table(8, 64, device=DEV)
    pos = torch.zeros(2, 5, dtype=torch.int32, device=DEV)
    kw = dict(q_table=table, k_table=table)
    for bad in (dict(q_weight=torch.ones(64, device=DEV).to(BF)),
                dict(q_weight=torch.ones(32, device=DEV)), dict(k_table=None),
                dict(k_table=igc.rope_table(8, 32, device=DEV)),
                dict(q_table=table.double()), dict(q_positions=pos.long()),
                dict(q_positions=pos[:1]), dict(q_table=table.cpu())):
        with pytest.raises(igc.InvalidArgument):
            igc.qk_norm_rope(q, k, **{**kw, **bad})
    with pytest.raises(igc.InvalidArgument):
        igc.qk_norm_rope(q, k.half(), **kw)
    with pytest.raises(igc.InvalidArgument):
        igc.qk_norm_rope(q, k[..., :32], **kw)
    with pytest.raises(igc.InvalidArgument):
        igc.qk_norm_rope_bwd(q[:1], k, q, k, **kw)
    with pytest.raises(igc.Declined, match="shape"):
        igc.qk_norm_rope(q, k, q_table=table[:4], k_table=table)
    with pytest.raises(igc.Declined, match="scale"):
        igc.qk_norm_rope(q, eps=-1.0)
    with pytest.raises(igc.Declined, match="dtype"):
        igc.qk_norm_rope(q.to(torch.float8_e4m3fn))
