"""The product of rows in 8 bits on the GPU against whole numbers in 64 bits.
The integer sums are exact, so an output is off by its one rounding (u = eps /
2) and four fp32 steps (2^-24) of the product's and the bias's magnitude."""
import os

import pytest
import torch

import implicit_gemm_nhwc_amd as igc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


def _ints(rows, k, seed, pad=0):
    """int8 [rows, k] of all values, in rows of whole 16-byte pieces and `pad`
    more of noise."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pitch = -(-k // 16) * 16 + pad
    buf = torch.randint(-128, 128, (rows, pitch), generator=gen, device=DEV, dtype=torch.int8)
    return buf[:, :k]


def _scales(n, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return 0.001 + 0.02 * torch.rand(n, generator=gen, device=DEV)


def _check(x, xs, w, ws, bias, y):
    # exact in 64 bits: sums stay below 2^53
    acc = x.double().reshape(-1, x.shape[-1]) @ w.double().t().contiguous()
    p = acc * xs.double().reshape(-1, 1) * ws.double()
    b = torch.zeros_like(ws) if bias is None else bias
    ref = p + b.double()
    got = y.double().reshape(ref.shape)
    assert torch.isfinite(got).all()
    u = torch.finfo(y.dtype).eps / 2
    bound = u * ref.abs() + 4 * 2.0 ** -24 * (p.abs() + b.double().abs()) + 2.0 ** -25
    far = (got - ref).abs()
    print(f"    y: {float((far / bound).max()):.3f} of the bound", flush=True)
    assert (far <= bound).all()


CASES = [
    # dt, m, k, n, bias
    (BF, 1, 1, 1, True), (HF, 1, 16, 16, False), (BF, 3, 17, 5, True), (HF, 16, 64, 33, True),
    (BF, 8, 2048, 8192, True), (HF, 17, 1000, 100, True), (BF, 32, 1025, 47, False),
    (HF, 33, 128, 64, True), (BF, 64, 5000, 129, True), (HF, 5, 131071, 18, True),
    (BF, 65, 64, 64, True), (HF, 65, 1, 3, True), (BF, 100, 127, 65, False),
    (HF, 1001, 1000, 777, True), (BF, 129, 129, 1031, True), (HF, 500, 272, 63, True),
    (BF, 70, 20000, 200, True), (BF, 20, 6000, 6001, True), (HF, 18, 1300, 500, False),
    (BF, 520, 700, 2100, True),
    (HF, 2100, 100, 2111, True), (BF, 1920, 2048, 2048, False), (HF, 2049, 129, 2050, True),
    (BF, 4100, 200, 4200, True), (HF, 4096, 1024, 4096, False), (BF, 8193, 1030, 2300, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}")
def test_against_whole_numbers(case):
    print(f"linear i8 {case}", flush=True)
    dt, m, k, n, with_bias = case
    x, w, xs, ws = _ints(m, k, 1), _ints(n, k, 2), _scales(m, 3), _scales(n, 4)
    bias = _scales(n, 5) * 30 - 0.3 if with_bias else None
    y = igc.linear_i8(x, xs, w, ws, bias=bias, dtype=dt)
    _check(x, xs, w, ws, bias, y)
    assert torch.equal(igc.linear_i8(x, xs, w, ws, bias=bias, dtype=dt), y)
    with igc.using_library(igc.POISON_LIB_PATH):
        assert torch.equal(igc.linear_i8(x, xs, w, ws, bias=bias, dtype=dt), y)
    # other noise past the rows, another pitch
    x2, w2 = _ints(m, k, 7, 32), _ints(n, k, 8, 16)
    x2.copy_(x)
    w2.copy_(w)
    assert torch.equal(igc.linear_i8(x2, xs, w2, ws, bias=bias, dtype=dt), y)


def test_largest_sums():
    """Every product 128 * 128 or -128 * 127, at the largest k."""
    for m in (3, 70):
        x = torch.full((m, 131072), -128, dtype=torch.int8, device=DEV)[:, :131071]
        w = torch.full((18, 131072), -128, dtype=torch.int8, device=DEV)[:, :131071]
        w[1] = 127
        xs, ws = torch.full((m,), 2.0 ** -20, device=DEV), torch.full((18,), 2.0 ** -10, device=DEV)
        _check(x, xs, w, ws, None, igc.linear_i8(x, xs, w, ws))


def test_quantised_projection():
    """Tokens of three axes and weights through quantize_rows: within the steps
    of both of the product in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    for dt, c in ((BF, 256), (HF, 333)):
        x = torch.randn(2, 60, c, generator=gen).to(dt).to(DEV)
        w = (torch.randn(100, c, generator=gen) * c ** -0.5).to(dt).to(DEV)
        xq, xs = igc.quantize_rows(x)
        wq, ws = igc.quantize_rows(w)
        y = igc.linear_i8(xq, xs, wq, ws, dtype=dt)
        assert y.shape == (2, 60, 100) and y.dtype == dt
        _check(xq, xs, wq, ws, None, y)
        ref = x.double() @ w.double().t().contiguous()
        # |dx| <= xs / 2, |dw| <= ws / 2
        step = (xs.double()[..., None] / 2 * w.double().abs().sum(1)
                + ws.double() / 2 * x.double().abs().sum(-1, keepdim=True)
                + c * xs.double()[..., None] * ws.double() / 4)
        assert ((y.double() - ref).abs() <= step * 1.001 + torch.finfo(dt).eps * ref.abs()).all()


def test_rows_without_a_scale():
    """Scales of zero, infinity and NaN reach their row alone."""
    x, w = _ints(70, 64, 1), _ints(40, 64, 2)
    xs, ws = _scales(70, 3), _scales(40, 4)
    want = igc.linear_i8(x, xs, w, ws)
    xs2 = xs.clone()
    xs2[3], xs2[69] = float("nan"), 0.0
    y = igc.linear_i8(x, xs2, w, ws)
    assert torch.isnan(y[3]).all() and (y[69] == 0).all()
    keep = [i for i in range(70) if i not in (3, 69)]
    assert torch.equal(y[keep], want[keep])


def test_empty_extents():
    for m, k, n in ((0, 16, 5), (4, 16, 0), (4, 0, 5), (70, 0, 70)):
        x = torch.zeros(m, k, dtype=torch.int8, device=DEV)
        w = torch.zeros(n, k, dtype=torch.int8, device=DEV)
        bias = torch.arange(n, device=DEV).float()
        y = igc.linear_i8(x, _scales(m, 1), w, _scales(n, 2), bias=bias)
        assert y.shape == (m, n) and torch.equal(y, bias.to(BF).expand(m, n))


def test_layouts():
    """Slices of wider rows, repeated rows, transposed leading axes refused."""
    big = _ints(60, 512, 1)
    xs = _scales(60, 2)
    w, ws = _ints(50, 96, 3), _scales(50, 4)
    want = igc.linear_i8(big[:, 128:224].contiguous(), xs, w, ws)
    assert torch.equal(igc.linear_i8(big[:, 128:224], xs, w, ws), want)
    three = big[:, 128:224].unflatten(0, (3, 20))
    assert torch.equal(igc.linear_i8(three, xs.view(3, 20), w, ws), want.view(3, 20, 50))
    one = igc.linear_i8(big[:1, 128:224].expand(60, 96), xs[:1].expand(60).contiguous(), w, ws)
    assert torch.equal(one, want[:1].expand(60, 50))
    assert torch.equal(igc.linear_i8(big[5, 128:224], xs[5], w, ws), want[5])
    assert torch.equal(igc.linear_i8(big[::2, 128:224], xs[::2].contiguous(), w, ws), want[::2])


def test_graph_and_stream():
    x = torch.randn(90, 200, device=DEV).to(BF)
    wq, ws = igc.quantize_rows(torch.randn(130, 200, device=DEV).to(BF))
    bias = torch.randn(130, device=DEV)

    def step(**kw):
        q, s = igc.quantize_rows(x, **kw)
        return igc.linear_i8(q, s, wq, ws, bias=bias, **kw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    s = torch.cuda.Stream()
    for i in range(4):
        x.copy_(torch.randn(x.shape, device=DEV) * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        for st in (s, s.cuda_stream):
            want = step(stream=st)
            s.synchronize()
            assert torch.equal(y, want)


def test_binding_refusals():
    x, w, xs, ws = _ints(70, 64, 1), _ints(40, 64, 2), _scales(70, 3), _scales(40, 4)
    good = dict(x=x, xs=xs, w=w, ws=ws, bias=None, dtype=BF)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(w=w.half()), dict(w=w[:, :48]),
                dict(w=w[None]), dict(xs=xs[:1]), dict(ws=xs), dict(xs=xs.double()),
                dict(ws=ws.cpu()), dict(bias=xs), dict(dtype=torch.float32), dict(w=None),
                dict(x=x.t()), dict(x=x.view(7, 10, 64).transpose(0, 1), xs=xs.view(10, 7)),
                dict(xs=None)):
        a = {**good, **bad}
        with pytest.raises(igc.InvalidArgument):
            igc.linear_i8(a["x"], a["xs"], a["w"], a["ws"], bias=a["bias"], dtype=a["dtype"])
    # rows that end in the middle of a 16-byte piece without room behind them
    short = torch.zeros(3 * 64 + 40, dtype=torch.int8, device=DEV).as_strided((4, 40), (64, 1))
    with pytest.raises(igc.InvalidArgument, match="storage"):
        igc.linear_i8(short, _scales(4, 1), w[:, :40], ws)
    dense = torch.zeros(4, 40, dtype=torch.int8, device=DEV)   # a pitch of 40 bytes
    with pytest.raises(igc.Declined, match="alignment"):
        igc.linear_i8(torch.zeros(5, 40, dtype=torch.int8, device=DEV)[:4], _scales(4, 1),
                      w[:, :40], ws)
    with pytest.raises(igc.Declined, match="alignment"):
        igc.linear_i8(x[:, 8:56], xs, w[:, 8:56], ws)
    with pytest.raises(igc.Declined, match="size_limit"):
        igc.linear_i8(torch.zeros(1, 131072, dtype=torch.int8, device=DEV), xs[:1],
                      torch.zeros(2, 131072, dtype=torch.int8, device=DEV), ws[:2])
    assert igc.linear_i8_check(x, xs, w, ws, x.view(BF)[:, :40]) == 11
