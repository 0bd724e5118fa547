"""Layer norm and its gradient on the GPU against the float64 oracle.

Bounds, with u = eps / 2 of the element type for the one rounding of each
result and e = 2^-24 for each fp32 step.  A row's sum takes at most 8 + 4
additions in a lane, 6 between lanes and 8 between waves: under 32 e of the
magnitudes.  With A = mean |x|, the mean is off by 32 e A and x - mean by
d = e (|x - mean| + 32 A); the variance by 2 d sigma + 32 e sigma^2, so that r
is off by a factor (32 A r + 32) e, and xh by
  X = e (33 A r + |xh|) + |xh| (33 A r + 32) e.
The gradients add their own sums (32 e of the magnitudes) and what X moves.
A weight's gradient adds a lane's rounds, a workgroup's groups of lanes, 1 / 64
of the workgroups' partials a lane and a tree of 6: with a row a workgroup rows /
256 + 8 + 6, otherwise rows / 2048 + 32 + 12 + 6, both under rows / 768 + 64 up to
19000 rows.
"""
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


def _rnd(*shape, seed=0, mean=0.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) + mean


def _near(name, got, ref, bound):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    far = (got - ref).abs()
    print(f"    {name}: {float((far / bound.clamp_min(1e-300)).max()) if far.numel() else 0:.3f} "
          "of the bound", flush=True)
    assert (far <= bound).all(), name


def _check(x, y, kw, dy=None, dx=None, dw=None, db=None):
    dt = x.dtype
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == HF else 2.0 ** -134
    o = oracle.layer_norm(x, grad=dy, **kw)
    xh, w, ar = o["xh"].abs(), o["w"].abs(), o["a"] * o["r"]
    off = E * (33 * ar + xh) + xh * (33 * ar + 32) * E
    if y is not None:
        _near("y", y, o["y"], u * o["y"].abs() + off * w + 2 * E * (xh * w + o["b"].abs()) + tiny)
    if dx is not None:
        t, q = o["u"].abs(), o["q"].abs()
        mt, mtx = t.mean(-1, keepdim=True), (t * xh).mean(-1, keepdim=True)
        top = off.amax(-1, keepdim=True)
        err = o["r"] * (2 * E * t + 34 * E * mt + xh * (34 * E * mtx + top * mt) + off * q
                        + (32 * ar + 40) * E * (t + mt + xh * q))
        _near("dx", dx, o["dx"], u * o["dx"].abs() + err + tiny)
    lead = tuple(range(x.dim() - 1))
    n = x.numel() // x.shape[-1]
    depth = (n / 768 + 64) * E
    if dw is not None:
        g = o["g"].abs()
        _near("dweight", dw, o["dweight"], depth * (g * xh).sum(lead) + (g * off).sum(lead) + 1e-30)
    if db is not None:
        _near("dbias", db, o["dbias"], depth * o["g"].abs().sum(lead) + 1e-30)


CASES = [
    # dt, leading axes, C, weights, mean of the inputs
    (BF, (1,), 1, True, 1.0),
    (HF, (5,), 7, True, 0.0),
    (BF, (3, 5), 8, True, 0.3),
    (HF, (33,), 64, False, 0.3),
    (BF, (2, 31), 65, True, 0.0),
    (HF, (70,), 128, True, 4.0),
    (BF, (9,), 129, False, 0.0),
    (HF, (2, 3, 5), 255, True, 0.0),
    (BF, (300,), 256, True, 0.3),
    (HF, (3, 961), 333, True, 0.3),
    (BF, (2, 7, 9), 512, True, 0.0),
    (HF, (4,), 513, True, 0.0),
    (BF, (1000,), 768, True, 0.3),
    (HF, (8, 1), 1024, True, 0.0),
    (BF, (17,), 1025, False, 0.0),
    (HF, (1, 1, 1), 2048, True, 2.0),
    (BF, (5,), 2049, True, 0.0),
    (HF, (37,), 4096, True, 0.3),
    (BF, (3,), 4103, True, 0.0),
    (HF, (21,), 8192, True, 0.0),
    (BF, (2,), 8195, True, 0.3),
    (HF, (3,), 16384, True, 0.0),
    (BF, (3100, 3), 40, True, 0.0),       # several rounds a workgroup, backward
    (HF, (4000,), 777, True, 0.3),
    (BF, (1600,), 4096, False, 0.0),
    (HF, (2000,), 8200, True, 0.0),
    (BF, (1100,), 6000, True, 0.0),
    (HF, (700,), 7000, True, 0.3),
    (BF, (600,), 12289, True, 0.0),
]


def _inputs(case):
    dt, lead, c, weights, mean = case
    x = _rnd(*lead, c, seed=1, mean=mean).to(dt).to(DEV)
    dy = _rnd(*lead, c, seed=2).to(dt).to(DEV)
    w = (1 + 0.3 * _rnd(c, seed=3)).to(DEV) if weights else None
    b = (0.3 * _rnd(c, seed=4)).to(DEV) if weights else None
    return x, dy, w, b


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{'x'.join(map(str, c[1]))}-{c[2]}")
def test_norm_and_gradients(case):
    print(f"layer norm {case}", flush=True)
    x, dy, w, b = _inputs(case)
    y = igc.layer_norm(x, w, b, eps=1e-5)
    dx, dw, db = igc.layer_norm_bwd(dy, x, w, eps=1e-5)
    _check(x, y, dict(weight=w, bias=b, eps=1e-5), dy, dx, dw, db)
    again = (igc.layer_norm(x, w, b),) + igc.layer_norm_bwd(dy, x, w)
    assert all(torch.equal(p, q) for p, q in zip(again, (y, dx, dw, db)))
    with igc.using_library(igc.POISON_LIB_PATH):
        poison = (igc.layer_norm(x, w, b),) + igc.layer_norm_bwd(dy, x, w)
    assert all(torch.equal(p, q) for p, q in zip(poison, (y, dx, dw, db)))


def test_extreme_rows():
    """Constant rows (eps alone), a mean far above the spread, large and small
    values; a NaN stays in its row."""
    for dt in (BF, HF):
        x = _rnd(8, 96, seed=3).to(dt)
        x[0] = 5.0
        x[1] = (300 + 2 * _rnd(96, seed=5)).to(dt)
        x[2] *= 1e4 if dt == HF else 1e15
        x[3] *= 2.0 ** -14
        x[4] = 0
        x[5, 1:] = 0
        dy = _rnd(8, 96, seed=4).to(dt).to(DEV)
        x = x.to(DEV)
        y = igc.layer_norm(x, eps=1e-5)
        dx, dw, db = igc.layer_norm_bwd(dy, x, eps=1e-5)
        _check(x, y, dict(eps=1e-5), dy, dx, dw, db)
        assert (y[0] == 0).all() and (y[4] == 0).all()
        x[6, 95] = float("nan")
        x[7, 0] = float("inf")
        y2 = igc.layer_norm(x, eps=1e-5)
        assert torch.isnan(y2[6:]).all() and torch.equal(y2[:6], y[:6])
        dx2, dw2, _ = igc.layer_norm_bwd(dy, x, eps=1e-5)
        assert torch.isnan(dx2[6:]).all() and torch.equal(dx2[:6], dx[:6])


def test_rows_without_lanes_stay_out_of_the_gradients():
    """Lane groups without a row, with eps = 0."""
    x, dy = _rnd(3, 24, seed=1).to(BF).to(DEV), _rnd(3, 24, seed=2).to(BF).to(DEV)
    dx, dw, db = igc.layer_norm_bwd(dy, x, eps=0.0)
    _check(x, None, dict(eps=0.0), dy, dx, dw, db)


def test_strides_in_place_and_guards():
    w, b = (1 + 0.1 * _rnd(40, seed=1)).to(DEV), _rnd(40, seed=2).to(DEV)
    for dt in (BF, HF):
        big = _rnd(3, 9, 11, 57, seed=3).to(dt).to(DEV)
        for x in (big[:, 2:7, 1:9, 3:43], big[..., 5:45], big[1, ::3, :, :40], big[0, 0, ::2, 1:41],
                  big[:1, :1, :1, 7:47].expand(3, 4, 5, 40), big.transpose(0, 1)[..., :40]):
            y = igc.layer_norm(x.contiguous(), w, b)
            assert torch.equal(igc.layer_norm(x, w, b), y)
            dy = _rnd(*x.shape, seed=4).to(dt).to(DEV)
            want = igc.layer_norm_bwd(dy, x.contiguous(), w)
            assert all(torch.equal(p, q) for p, q in zip(igc.layer_norm_bwd(dy, x, w), want))
            # into a padded buffer, at an odd offset
            pad = torch.full((*x.shape[:-1], 59), 3.0, dtype=dt, device=DEV)
            assert igc.layer_norm_fwd(x, pad[..., 9:49], weight=w, bias=b) == 1
            assert torch.equal(pad[..., 9:49], y)
            assert igc.layer_norm_grad(dy, x, pad[..., 9:49], weight=w) == 1
            assert torch.equal(pad[..., 9:49], want[0])
            pad[..., 9:49] = 3.0
            assert (pad == 3.0).all()
            z = dy.clone()
            assert igc.layer_norm_grad(z, x, z, weight=w) == 1 and torch.equal(z, want[0])
        z = big.clone()
        part = z[:, 2:7, 1:9, 3:43]
        assert igc.layer_norm_fwd(part, part, weight=w, bias=b) == 1
        assert torch.equal(part, igc.layer_norm(big[:, 2:7, 1:9, 3:43], w, b))
        z[:, 2:7, 1:9, 3:43] = big[:, 2:7, 1:9, 3:43]
        assert torch.equal(z, big)


def test_weight_gradients_alone_and_given_workspace():
    x, dy, w, _ = _inputs((HF, (700,), 200, True, 0.0))
    dx, dw, db = igc.layer_norm_bwd(dy, x, w)
    need = igc.layer_norm_bwd_workspace_bytes(x.shape, x.dtype)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    o, g = torch.empty_like(x), torch.empty_like(dw)
    assert igc.layer_norm_grad(dy, x, o, weight=w, dweight=g, workspace=ws,
                               workspace_bytes=need) == 1
    assert torch.equal(o, dx) and torch.equal(g, dw) and (ws[need:] == 255).all()
    assert igc.layer_norm_grad(dy, x, o, weight=w, dbias=g) == 1 and torch.equal(g, db)
    short = ws[:need - 16]
    assert igc.layer_norm_bwd_check(dy, x, o, weight=w, dweight=g, workspace=short) == 12


def test_empty_extents():
    for shape in ((0, 24), (3, 0, 24), (2, 0, 3, 24)):
        x = torch.zeros(shape, dtype=BF, device=DEV)
        assert igc.layer_norm(x).shape == x.shape
        dx, dw, db = igc.layer_norm_bwd(x, x)
        assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all() and dw.shape == (24,)


def test_graph_and_stream():
    x, dy, w, b = _inputs((BF, (70, 5), 333, True, 0.0))
    igc.layer_norm(x, w, b)
    igc.layer_norm_bwd(dy, x, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = (igc.layer_norm(x, w, b),) + igc.layer_norm_bwd(dy, x, w)
    s = torch.cuda.Stream()
    for n in range(4):
        for t in (x, dy):
            t.copy_(torch.randn(t.shape, device=DEV) * (n + 1))
        g.replay()
        torch.cuda.synchronize()
        for st in (s, s.cuda_stream):
            want = (igc.layer_norm(x, w, b, stream=st),) + igc.layer_norm_bwd(dy, x, w, stream=st)
            s.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_binding_refusals():
    x, dy, w, b = _inputs((BF, (4, 5), 24, True, 0.0))
    for bad in (dict(weight=w.to(BF)), dict(weight=w[:23]), dict(bias=b.cpu()),
                dict(bias=b.double()), dict(weight=w[::2])):
        with pytest.raises(igc.InvalidArgument):
            igc.layer_norm(x, **{**dict(weight=w, bias=b), **bad})
    for bad in (x.float(), x.cpu(), x.transpose(1, 2), x[..., ::2], x[0, 0, 0], [1.0],
                x.view(1, 1, 4, 5, 24)):
        with pytest.raises(igc.InvalidArgument):
            igc.layer_norm(bad)
    for bad in (dy[:1], dy.half(), dy.cpu(), None):
        with pytest.raises(igc.InvalidArgument):
            igc.layer_norm_bwd(bad, x, w)
    for eps in (-1.0, float("nan"), float("inf"), 1e300):
        with pytest.raises(igc.Declined, match="scale"):
            igc.layer_norm(x, eps=eps)
    with pytest.raises(igc.Declined, match="size_limit"):
        igc.layer_norm(torch.zeros(2, 16385, dtype=BF, device=DEV))
    with pytest.raises(igc.Declined, match="shape"):
        igc.layer_norm(torch.zeros(2, 0, dtype=BF, device=DEV))
    out = torch.empty_like(x)
    assert igc.layer_norm_fwd(x[:, 1:], x[:, :-1]) == 0            # shifted in place
    assert igc.layer_norm_fwd(x, out[:1].expand(4, 5, 24)) == 0    # meets itself
    assert igc.layer_norm_grad(dy, x, x) == 0                      # over its own input
    assert igc.layer_norm_grad(dy, x, out, dweight=w, weight=w) == 0
