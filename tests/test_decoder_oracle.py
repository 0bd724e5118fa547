"""Pins of the decoder oracle (CPU): loops in pure Python, whole-number
arithmetic, closed forms and differences."""
import math
from fractions import Fraction

import pytest
import torch

from oracle import attention, decoder as oracle


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).double()


def test_layer_norm_brute_force():
    x, w, b = _rand(2, 3, 7) + 2, _rand(7, seed=1), _rand(7, seed=2)
    y = oracle.layer_norm(x, weight=w, bias=b, eps=0.01)["y"]
    for i in range(2):
        for j in range(3):
            row = [float(v) for v in x[i, j]]
            mean = math.fsum(row) / 7
            sd = math.sqrt(math.fsum((v - mean) ** 2 for v in row) / 7 + 0.01)
            for c in range(7):
                assert math.isclose(float(y[i, j, c]), (row[c] - mean) / sd * float(w[c]) + float(b[c]),
                                    abs_tol=1e-13)


def test_layer_norm_gradients():
    x, w, b = _rand(5, 6), _rand(6, seed=1), _rand(6, seed=2)
    g = _rand(5, 6, seed=3)
    r = oracle.layer_norm(x, weight=w, bias=b, eps=0.01, grad=g)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = torch.nn.functional.layer_norm(leaves[0], (6,), leaves[1], leaves[2], 0.01)
    assert torch.allclose(y, r["y"], atol=1e-13)
    (y * g).sum().backward()
    for t, n in zip(leaves, ("dx", "dweight", "dbias")):
        assert torch.allclose(t.grad, r[n], atol=1e-12), n
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)):
        flat = t.view(-1)
        for at in (0, 3, flat.numel() - 1):
            keep, f = float(flat[at]), []
            for s in (1, -1):
                flat[at] = keep + s * 1e-6
                f.append(float((oracle.layer_norm(x, weight=w, bias=b, eps=0.01)["y"] * g).sum()))
            flat[at] = keep
            assert math.isclose((f[0] - f[1]) / 2e-6, float(r[name].reshape(-1)[at]), rel_tol=1e-6,
                                abs_tol=1e-8)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_rows_by_rational_numbers(dt):
    x = _rand(40, 9, seed=4).to(dt)
    x[0] = 0
    x[1] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5, 127]).to(dt)   # ties
    x[2] = torch.tensor([-254, 1, 3, 5, -1, -3, 253, -253, 7]).to(dt)
    q, s = oracle.rows_i8(x)
    for i in range(40):
        row = [Fraction(float(v)) for v in x[i]]
        m = max(abs(v) for v in row)
        for j, v in enumerate(row):
            want = 0 if m == 0 else round(127 * v / m)    # to even on ties
            assert int(q[i, j]) == want
        assert float(s[i]) == float((torch.tensor(float(m)) / 127).float())
    assert q[1].tolist() == [127, 0, 2, 2, 0, -2, 126, -126, 127]
    assert q[2].tolist() == [-127, 0, 2, 2, 0, -2, 126, -126, 4]


def test_rows_without_a_scale():
    x = torch.zeros(5, 3).to(torch.bfloat16)
    x[1, 0], x[2, 1], x[3] = math.inf, math.nan, 2.0 ** -111
    x[4] = 2.0 ** -110
    q, s = oracle.rows_i8(x)
    assert (q[:4] == 0).all() and s[0] == 0 and s[3] == 0 and torch.isnan(s[1:3]).all()
    assert (q[4] == 127).all() and s[4] > 0


def test_cache_places():
    row = [4, -1, 2, 7]
    assert oracle.cache_place(row, 0, 16, 7) == (4, 0)
    assert oracle.cache_place(row, 47, 16, 7) == (2, 15)
    for p in (-1, 16, 31, 48, 63, 64, 1 << 40):
        assert oracle.cache_place(row, p, 16, 7) is None
    assert oracle.cache_place([], 0, 16, 7) is None


def test_cache_written_and_read():
    x = _rand(2, 5, 3, 8, seed=5).to(torch.float16)
    q = torch.zeros(4, 3, 16, 16, dtype=torch.int8)
    s = torch.full((4, 3, 16), -1.0)
    oracle.cache_write(q, s, x, torch.tensor([[3, 0], [1, 9]]), torch.tensor([14, 12]),
                       torch.tensor([4, 9]))
    rows, steps = oracle.rows_i8(x)
    for b, t, page, place in ((0, 0, 3, 14), (0, 1, 3, 15), (0, 2, 0, 0), (0, 3, 0, 1), (1, 0, 1, 12),
                              (1, 3, 1, 15)):
        assert torch.equal(q[page, :, place, :8].double(), rows[b, t])
        assert torch.equal(s[page, :, place], steps[b, t])
    assert int((s >= 0).sum()) == 3 * 8      # the ninth token's page does not exist
    back = oracle.cache_rows(q, s, [3, 0], 18, 8)
    assert torch.equal(back[16], rows[0, 2] * steps[0, 2].double()[:, None])
    assert torch.isnan(oracle.cache_rows(q, s, [9], 2, 8)).all()


def test_cache_attention_is_attention_to_what_it_holds():
    gen = torch.Generator().manual_seed(6)
    kq, vq = (torch.randint(-127, 128, (5, 2, 16, 16), generator=gen, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(5, 2, 16, generator=gen) * 0.05 for _ in range(2))
    table, lens = torch.tensor([[2, 0], [4, 1], [3, 3]]), torch.tensor([20, 3, 0])
    q = _rand(3, 4, 4, 16, seed=7)
    k, v = (torch.stack([oracle.cache_rows(a, s, t.tolist(), 32, 16) for t in table])
            for a, s in ((kq, ks), (vq, vs)))
    r = oracle.cache_attention(q, kq, ks, vq, vs, table, lens, causal=False)
    want = attention.cross_attention(q, k, v, kv_lens=lens)
    assert torch.allclose(r["out"], want["out"], atol=1e-13)
    assert torch.equal(torch.isinf(r["lse"]), torch.isinf(want["lse"]))
    assert torch.allclose(r["lse"][:2], want["lse"][:2], atol=1e-12)
    r = oracle.cache_attention(q, kq, ks, vq, vs, table, lens, scale=0.1)
    for t in range(4):
        want = attention.cross_attention(q[:, t:t + 1], k, v, kv_lens=lens - (3 - t), scale=0.1)
        assert torch.allclose(r["out"][:, t:t + 1], want["out"], atol=1e-13)
    assert (r["out"][1, 0] == 0).all() and (r["out"][1, 1] != 0).any() and (r["out"][2] == 0).all()
    # a length past the table's 32 positions places the tokens all the same
    far = oracle.cache_attention(q, kq, ks, vq, vs, table, torch.tensor([34, 3, 0]), scale=0.1)
    near = oracle.cache_attention(q[:, :2], kq, ks, vq, vs, table, torch.tensor([32, 1, 0]), scale=0.1)
    assert torch.equal(far["out"][0, :2], near["out"][0])
    assert torch.equal(far["lse"][0, :, 3], near["lse"][0, :, 1] * 0 + oracle.cache_attention(
        q[:, 3:], kq, ks, vq, vs, table, torch.tensor([32, 1, 0]), scale=0.1)["lse"][0, :, 0])
