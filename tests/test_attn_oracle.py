"""Pins of the attention oracle (CPU): loops in pure Python, closed forms and
differences."""
import math

import pytest
import torch

from oracle import attention as oracle


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).double()


def test_attention_brute_force():
    q, k, v = _rand(2, 3, 4, 8), _rand(2, 5, 2, 8, seed=1), _rand(2, 5, 2, 8, seed=2)
    lens = torch.tensor([5, 3])
    mask = torch.tensor([[1, 0, 1, 1, 1], [1, 1, 0, 1, 1]])
    r = oracle.cross_attention(q, k, v, scale=0.3, kv_lens=lens, key_mask=mask)
    for b in range(2):
        for t in range(3):
            for h in range(4):
                w = {j: math.exp(0.3 * math.fsum(float(q[b, t, h, d] * k[b, j, h // 2, d])
                                                 for d in range(8)))
                     for j in range(int(lens[b])) if mask[b, j]}
                n = math.fsum(w.values())
                assert math.isclose(float(r["lse"][b, h, t]), math.log(n), rel_tol=1e-12)
                for d in range(8):
                    o = math.fsum(w[j] * float(v[b, j, h // 2, d]) for j in w) / n
                    assert math.isclose(float(r["out"][b, t, h, d]), o, abs_tol=1e-12)


def test_attention_without_valid_keys():
    q, k = _rand(2, 3, 2, 8), _rand(2, 4, 2, 8, seed=1)
    r = oracle.cross_attention(q, k, k, kv_lens=torch.tensor([0, 2]), dout=q)
    assert (r["out"][0] == 0).all() and (r["lse"][0] == -math.inf).all()
    assert (r["dq"][0] == 0).all() and (r["dk"][0] == 0).all() and (r["dv"][1, 2:] == 0).all()
    assert (r["out"][1] != 0).any()


def test_attention_gradients():
    q, k, v = _rand(1, 3, 4, 8), _rand(1, 5, 2, 8, seed=1), _rand(1, 5, 2, 8, seed=2)
    go = _rand(1, 3, 4, 8, seed=3)
    lens = torch.tensor([4])
    r = oracle.cross_attention(q, k, v, kv_lens=lens, dout=go)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        for at in ((0, 1, 1, 3), (0, 2, 0, 0), (0, 0, 1, 7)):
            h, keep, f = 1e-6, float(t[at]), []
            for s in (1, -1):
                t[at] = keep + s * h
                f.append(float((oracle.cross_attention(q, k, v, kv_lens=lens)["out"] * go).sum()))
            t[at] = keep
            assert math.isclose(float(r[name][at]), (f[0] - f[1]) / (2 * h), abs_tol=1e-7)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    kk, vv = (x[:, :4].repeat_interleave(2, 2) for x in leaves[1:])
    s = torch.einsum("bthd,bjhd->bhtj", leaves[0], kk) / 8 ** 0.5
    out = torch.einsum("bhtj,bjhd->bthd", s.softmax(-1), vv)
    out.backward(go)
    for name, t in zip(("dq", "dk", "dv"), leaves):
        assert torch.allclose(r[name], t.grad, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_brute_force(interleaved):
    x, w = _rand(2, 3, 2, 8), _rand(8, seed=1)
    table = torch.cat([_rand(6, 3, seed=2), _rand(6, 3, seed=3)], 1)
    pos = torch.tensor([[5, 0, 2], [1, 1, 9]], dtype=torch.int32)
    y = oracle.qk_norm_rope(x, weight=w, table=table, positions=pos, eps=1e-3,
                            interleaved=interleaved)
    for b in range(2):
        for t in range(3):
            for h in range(2):
                row = [float(z) for z in x[b, t, h]]
                r = 1 / math.sqrt(sum(z * z for z in row) / 8 + 1e-3)
                n = [z * r * float(s) for z, s in zip(row, w)]
                want = list(n)
                p = int(pos[b, t])
                for i in range(3):
                    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
                    c, s = ((float(table[p, i]), float(table[p, 3 + i])) if p < 6
                            else (math.nan, math.nan))
                    want[lo], want[hi] = n[lo] * c - n[hi] * s, n[hi] * c + n[lo] * s
                got = [float(z) for z in y[b, t, h]]
                for g, e in zip(got, want):
                    assert (math.isnan(g) and math.isnan(e)) or math.isclose(g, e, abs_tol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients(interleaved):
    x, w, dy = _rand(1, 2, 3, 8), _rand(8, seed=1), _rand(1, 2, 3, 8, seed=2)
    a = _rand(2, 2, seed=4)
    table = torch.cat([a.cos(), a.sin()], 1)
    kw = dict(table=table, eps=1e-2, interleaved=interleaved)
    r = oracle.qk_norm_rope(x, weight=w, grad=dy, **kw)
    for grad, t, at in (("dx", x, (0, 1, 2, 1)), ("dx", x, (0, 0, 0, 6)), ("dweight", w, (2,)),
                        ("dweight", w, (7,))):
        h, keep, f = 1e-6, float(t[at]), []
        for s in (1, -1):
            t[at] = keep + s * h
            f.append(float((oracle.qk_norm_rope(x, weight=w, **kw) * dy).sum()))
        t[at] = keep
        assert math.isclose(float(r[grad][at]), (f[0] - f[1]) / (2 * h), abs_tol=1e-7)
