"""Oracle of the attention operators (TEST INFRASTRUCTURE ONLY): the
definitions of include/igemm_attn.h in float64 on the CPU, one batch entry and
head at a time, sharing no code with the HIP library.

cross_attention and its gradients are pinned in tests/test_attn_oracle.py by a
pure-Python sum over the keys, by finite differences and by torch's automatic
differentiation; qk_norm_rope by a pure-Python loop, its inverse rotation and
finite differences."""
import torch


def valid_keys(b, kv_len, kv_lens, key_mask):
    """Boolean [kv_len]: which keys batch entry b attends to."""
    ok = torch.ones(kv_len, dtype=torch.bool)
    if kv_lens is not None:
        ok &= torch.arange(kv_len) < int(kv_lens[b])
    if key_mask is not None:
        ok &= key_mask[b].cpu() != 0
    return ok


def cross_attention(q, k, v, *, scale=None, kv_lens=None, key_mask=None, dout=None):
    """dict of float64 results: out, lse, and with dout also dq, dk, dv; for
    bounds on rounding also the sums of magnitudes behind each result: out_abs
    (sum p |v|), s_abs (the largest scale sum |q| |k| of a row), and with dout
    dv_abs (sum p |do|), and the pieces of the ds bound."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    b, tq, hq, d = q.shape
    tk, hk = k.shape[1], k.shape[2]
    g = hq // max(hk, 1)
    scale = d ** -0.5 if scale is None else scale
    r = {"out": torch.zeros_like(q), "lse": torch.full((b, hq, tq), -torch.inf).double(),
         "out_abs": torch.zeros_like(q), "s_abs": torch.zeros(b, hq, tq).double(),
         "v_abs": torch.zeros(b, hq, d).double()}
    if dout is not None:
        dout = dout.detach().cpu().double()
        r.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v),
                 parts={})
    for i in range(b):
        idx = valid_keys(i, tk, kv_lens, key_mask).nonzero()[:, 0]
        if not len(idx):
            continue
        for h in range(hq):
            qq, kk, vv = q[i, :, h], k[i, idx, h // g], v[i, idx, h // g]
            s = scale * (qq @ kk.t())
            top = s.max(1, keepdim=True).values
            e = torch.exp(s - top)
            total = e.sum(1, keepdim=True)
            p = e / total
            r["lse"][i, h] = (top + total.log())[:, 0]
            r["out"][i, :, h] = p @ vv
            r["out_abs"][i, :, h] = p @ vv.abs()
            r["s_abs"][i, h] = scale * (qq.abs() @ kk.abs().t()).max(1).values
            r["v_abs"][i, h] = vv.abs().sum(0)
            if dout is not None:
                go = dout[i, :, h]
                dp = go @ vv.t()
                delta = (go * r["out"][i, :, h]).sum(1, keepdim=True)
                ds = p * (dp - delta)
                r["dq"][i, :, h] = scale * (ds @ kk)
                r["dk"][i, idx, h // g] += scale * (ds.t() @ qq)
                r["dv"][i, idx, h // g] += p.t() @ go
                r["parts"][i, h] = (idx, p, ds, go, kk, vv, qq)
    return r


def qk_norm_rope(x, *, weight=None, table=None, positions=None, eps=1e-6, interleaved=False,
                 grad=None):
    """y of one part in float64; with grad = dy a dict of y, dx, dweight and
    the magnitudes behind them."""
    x = x.detach().cpu().double()
    b, t, _, d = x.shape
    w = torch.ones(d).double() if weight is None else weight.detach().cpu().double()
    rot = 0 if table is None else table.shape[1]
    h = rot // 2
    cos, sin = torch.ones(b, t, 1, h).double(), torch.zeros(b, t, 1, h).double()
    if rot:
        tab = table.detach().cpu().double()
        pos = (torch.arange(t).expand(b, t) if positions is None else positions.cpu().long())
        bad = (pos < 0) | (pos >= tab.shape[0])
        rows = tab[pos.clamp(0, tab.shape[0] - 1)]
        rows[bad] = float("nan")
        cos, sin = rows[:, :, None, :h], rows[:, :, None, h:]
    a = slice(0, rot, 2) if interleaved else slice(0, h)
    c = slice(1, rot, 2) if interleaved else slice(h, rot)
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5

    def turn(u, sn):
        y = u.clone()
        y[..., a] = u[..., a] * cos - u[..., c] * sn
        y[..., c] = u[..., c] * cos + u[..., a] * sn
        return y

    y = turn(x * r * w, sin)
    if grad is None:
        return y
    g = turn(grad.detach().cpu().double(), -sin)
    u, xh = g * w, x * r
    mean = (u * xh).mean(-1, keepdim=True)
    return {"y": y, "dx": r * (u - xh * mean), "dweight": (g * xh).sum((0, 1, 2)),
            "dx_abs": r * (u.abs() + xh.abs() * (u * xh).abs().mean(-1, keepdim=True)),
            "dweight_abs": (g * xh).abs().sum((0, 1, 2)), "g": g}
