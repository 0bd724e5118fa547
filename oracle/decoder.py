"""Oracle of the decoder block's operators (TEST INFRASTRUCTURE ONLY): the
definitions of include/igemm_decoder.h in float64 on the CPU, sharing no code
with the HIP library.

Pinned in tests/test_decoder_oracle.py by pure-Python loops, finite differences
and torch's automatic differentiation."""
import torch


def _wide(t):
    return t.detach().cpu().double()


def layer_norm(x, *, weight=None, bias=None, eps=1e-5, grad=None):
    """dict of y and, for bounds on rounding, xh and r; with grad = dy also dx,
    dweight and dbias, and what stands behind them."""
    x = _wide(x)
    c = x.shape[-1]
    w = torch.ones(c).double() if weight is None else _wide(weight)
    b = torch.zeros(c).double() if bias is None else _wide(bias)
    d = x - x.mean(-1, keepdim=True)
    r = (d.square().mean(-1, keepdim=True) + eps) ** -0.5
    xh = d * r
    got = {"y": xh * w + b, "xh": xh, "r": r, "w": w, "b": b,
           "a": x.abs().mean(-1, keepdim=True)}
    if grad is not None:
        g = _wide(grad)
        u = g * w
        q = (u * xh).mean(-1, keepdim=True)
        lead = tuple(range(x.dim() - 1))
        got.update(dx=r * (u - u.mean(-1, keepdim=True) - xh * q), u=u, q=q,
                   dweight=(g * xh).sum(lead), dbias=g.sum(lead), g=g)
    return got


def rows_i8(x):
    """(integers as float64, scales as float32) of the rows of x in 8 bits, and
    from exact rational arithmetic: ties are found on whole numbers."""
    x = _wide(x)
    m = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    none = m < 2.0 ** -110
    top = torch.where(bad | none, 1.0, m)
    # x and m have at most 11 bits: 254 |x| and m are compared exactly in 64
    a = torch.where(bad | none, torch.zeros_like(x), x).abs() * 254
    k = torch.floor(a / (2 * top))          # whole steps below
    k = torch.where((k + 1) * 2 * top <= a, k + 1, k)
    k = torch.where(k * 2 * top > a, k - 1, k)
    rest = a - k * 2 * top                  # in units of m: half a step is m
    up = (rest > top) | ((rest == top) & (k % 2 == 1))
    q = (k + up) * torch.sign(torch.where(bad | none, torch.zeros_like(x), x))
    scale = torch.where(none, torch.zeros_like(m), (m.float() / 127).double())
    scale = torch.where(bad, torch.full_like(m, float("nan")), scale)
    return q, scale.squeeze(-1).float()


def cache_place(table_row, position, page_tokens, pages):
    """(page, token) of a position, or None."""
    if position < 0 or position // page_tokens >= len(table_row):
        return None
    page = int(table_row[position // page_tokens])
    return (page, position % page_tokens) if 0 <= page < pages else None


def cache_write(q, scale, x, table, start, lens=None):
    """Writes x [b, t, h, d] into integers q [pages, h, page, >= d] and scales
    (CPU tensors, changed in place)."""
    rows, steps = rows_i8(x)
    pages, _, tokens, _ = q.shape
    for b in range(x.shape[0]):
        n = x.shape[1] if lens is None else min(int(lens[b]), x.shape[1])
        for t in range(n):
            at = cache_place(table[b].tolist(), int(start[b]) + t, tokens, pages)
            if at:
                q[at[0], :, at[1], :x.shape[3]] = rows[b, t].to(q.dtype)
                scale[at[0], :, at[1]] = steps[b, t]


def cache_rows(q, scale, table_row, n, d):
    """The values [n, h, d] in float64 that a sequence's first n positions
    hold (NaN without a page)."""
    pages, h, tokens, _ = q.shape
    out = torch.full((n, h, d), float("nan")).double()
    for p in range(n):
        at = cache_place(table_row, p, tokens, pages)
        if at:
            out[p] = q[at[0], :, at[1], :d].double() * scale[at[0], :, at[1], None].double()
    return out


def cache_attention(q, kq, ks, vq, vs, table, lens, *, causal=True, scale=None):
    """dict of out and lse, and for bounds out_abs (sum p |v|) and s_abs."""
    q = _wide(q)
    b, tq, hq, d = q.shape
    hk, tokens = kq.shape[1], kq.shape[2]
    g = hq // max(hk, 1)
    scale = d ** -0.5 if scale is None else scale
    r = {"out": torch.zeros_like(q), "out_abs": torch.zeros_like(q),
         "lse": torch.full((b, hq, tq), -torch.inf).double(), "s_abs": torch.zeros(b, hq, tq).double(),
         "n": torch.zeros(b, tq).long()}
    for i in range(b):
        row = table[i].tolist()
        given = max(int(lens[i]), 0)
        n = min(given, len(row) * tokens)
        k, v = cache_rows(kq, ks, row, n, d), cache_rows(vq, vs, row, n, d)
        for t in range(tq):
            m = min(given - (tq - 1 - t) if causal else given, n)
            if m <= 0:
                continue
            r["n"][i, t] = m
            for h in range(hq):
                z = scale * (k[:m, h // g] @ q[i, t, h])
                p = torch.softmax(z, 0)
                r["lse"][i, h, t] = torch.logsumexp(z, 0)
                r["out"][i, t, h] = p @ v[:m, h // g]
                r["out_abs"][i, t, h] = p @ v[:m, h // g].abs()
                r["s_abs"][i, h, t] = scale * (k[:m, h // g].abs() @ q[i, t, h].abs()).max()
    return r
