"""Cases of the operators around the attention of a decoder that reads maps
and text: layer norm (forward, training), the product in 8-bit integers with a
scale a token and a channel, the cache of keys and values held in 8 bits
(written, read back), and the attention of new tokens over that cache.

With own = False, run() computes the operators from elementary torch
operations; with own = True it makes the calls of implicit_gemm_nhwc_amd.
exact() has the definitions in 64 bits.

The cache is pages of `page` tokens, [pages, kv heads, page, D] in int8 with D
rounded up to a multiple of 16, and one fp32 scale a row of D; position p of
sequence b is token p % page of page table[b][p // page].
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-5


# ------------------------------------------------------------------ cases
def _ln(name, op, dt, rows, c, affine=True):
    """op: "ln" (inference), "ln_train" (forward and backward)."""
    return _named(name, {"op": op, "dt": dt, "rows": rows, "c": c, "affine": affine})


def _i8(name, dt, m, k, n, bias=True):
    """Tokens quantised as they come, times weights quantised beforehand."""
    return _named(name, {"op": "i8", "dt": dt, "m": m, "k": k, "n": n, "bias": bias})


def _cache(name, dt, b, t, hk, d, page, ragged, past, fused_kv=True):
    """t tokens a sequence written behind `past` earlier ones, and read back.
    ragged: a padded batch with lengths.  fused_kv: k and v are the halves of
    one projection's output."""
    return _named(name, {"op": "cache", "dt": dt, "b": b, "t": t, "hk": hk, "d": d,
                         "page": page, "ragged": ragged, "past": past, "fused_kv": fused_kv})


def _attn(name, dt, b, tq, tk, hq, hk, d, page, causal=True):
    """tq new tokens a sequence over up to tk cached ones (themselves among
    them), each attending up to its own position where causal."""
    return _named(name, {"op": "attn", "dt": dt, "b": b, "tq": tq, "tk": tk, "hq": hq, "hk": hk,
                         "d": d, "page": page, "causal": causal})


def _named(name, c):
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token of eight sequences: latency
        _ln("ln_token", "ln", "bf16", 8, 1024),
        # inference over sixteen 64x64 maps of 512 channels
        _ln("ln_map", "ln", "fp16", 16 * 64 * 64, 512),
        # training, small map of an odd channel count
        _ln("ln_train_odd", "ln_train", "fp16", 3 * 31 * 31, 333),
        # training, 56x56 maps, batch 32
        _ln("ln_train_map", "ln_train", "bf16", 32 * 56 * 56, 768),
        # projection of one token of eight sequences: the weights' bytes
        _i8("i8_token", "bf16", 8, 2048, 8192),
        # odd number of tokens, inputs and outputs
        _i8("i8_odd", "fp16", 1001, 1000, 777),
        # projection of four 64x64 maps: the largest product
        _i8("i8_map", "bf16", 4 * 64 * 64, 4096, 4096, False),
        # the step of a caption decoder: one token of eight sequences
        _cache("cache_token", "bf16", 8, 1, 4, 128, 16, False, 300),
        # prompts of a padded batch
        _cache("cache_prompt", "fp16", 16, 4096, 8, 128, 64, True, 0),
        # caption decoder over a 28x28 map's states
        _attn("attn_cache_token", "bf16", 8, 1, 784, 16, 4, 128, 16),
        # one token of a few long ragged sequences
        _attn("attn_cache_long", "bf16", 4, 1, 65537, 32, 8, 128, 64),
        # drafted tokens in a row, odd head width
        _attn("attn_cache_drafts", "fp16", 16, 5, 4099, 8, 8, 80, 32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_train", "i8", "i8", "cache", "attn", "attn"])
    dt = rng.choice(["bf16", "fp16"])
    if op.startswith("ln"):
        c = _log(rng, 33, 8192)
        if rng.random() < 0.6:
            c = (c + 7) // 8 * 8
        rows = _log(rng, 1, max(1, min(100352, 32 * 56 * 56 * 768 // c)))
        return _ln(None, op, dt, rows, c, rng.random() < 0.8)
    if op == "i8":
        k, n = _log(rng, 65, 8192), _log(rng, 33, 8192)
        if rng.random() < 0.6:
            k, n = (k + 63) // 64 * 64, (n + 63) // 64 * 64
        m = _log(rng, 1, max(1, min(16384, 16384 * 4096 * 4096 // (k * n))))
        return _i8(None, dt, m, k, n, rng.random() < 0.5)
    d = rng.choice([40, 64, 64, 80, 128, 128])
    hk = rng.choice([1, 2, 4, 8, 10])
    page = rng.choice([16, 32, 64, 128])
    b = _log(rng, 1, 32)
    if op == "cache":
        t = _log(rng, 1, 8192)
        while b * t * hk * d > 16 * 4096 * 8 * 128:
            b, t = (b + 1) // 2, (t * 3 + 3) // 4
        return _cache(None, dt, b, t, hk, d, page, rng.random() < 0.6, rng.choice([0, 1, 300]),
                      rng.random() < 0.5)
    tk = _log(rng, 33, 65537)
    while b * tk * hk * d > 4 * 65537 * 8 * 128:
        b, tk = (b + 1) // 2, (tk * 3 + 3) // 4
    return _attn(None, dt, b, rng.choice([1, 1, 1, 2, 5, 8]), tk, hk * rng.choice([1, 1, 2, 4]),
                 hk, d, page, rng.random() < 0.8)


# ----------------------------------------------------------------- inputs
def _lens(b, most, gen, dev):
    """Ragged lengths between a third of `most` and `most`, the first full."""
    n = torch.randint(max(1, most // 3), most + 1, (b,), generator=gen, device=dev,
                      dtype=torch.int32)
    n[0] = most
    return n


def _table(b, tokens, page, gen, dev):
    """Pages of b sequences of up to `tokens`, handed out in no order."""
    per = -(-tokens // page)
    return torch.randperm(b * per, generator=gen, device=dev).view(b, per).to(torch.int32)


def _quantised(x):
    """Rows of the last axis in 8 bits and their scales."""
    top = x.abs().amax(-1, keepdim=True).double().clamp_min(1e-30)
    return (x.double() * 127 / top).round().to(torch.int8), (top / 127).float().squeeze(-1)


def _pool(pages, hk, page, d, gen, dev):
    """A pool of rows and scales as normally distributed states leave it."""
    q = torch.zeros(pages, hk, page, -(-d // 16) * 16, dtype=torch.int8, device=dev)
    s = torch.empty(pages, hk, page, device=dev)
    step = max(1, (1 << 25) // (hk * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn(n, hk, page, d, generator=gen, device=dev)
        q[i:i + n, ..., :d], s[i:i + n] = _quantised(x)
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DT[case["dt"]]

    def rnd(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + mean).to(dt)

    s = {"case": dict(case)}
    if case["op"].startswith("ln"):
        rows, c = case["rows"], case["c"]
        s["x"] = rnd(rows, c, mean=0.3)
        s["weight"] = s["bias"] = None
        if case["affine"]:
            s["weight"] = 1 + 0.1 * torch.randn(c, generator=gen, device=dev)
            s["bias"] = 0.1 * torch.randn(c, generator=gen, device=dev)
        if case["op"] == "ln_train":
            s["dy"] = rnd(rows, c)
        return s
    if case["op"] == "i8":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = rnd(m, k)
        w = torch.randn(n, k, generator=gen, device=dev) * k ** -0.5
        q, s["w_scale"] = _quantised(w)
        # rows of the weights start at multiples of 16 bytes
        s["w"] = torch.zeros(n, -(-k // 16) * 16, dtype=torch.int8, device=dev)[:, :k]
        s["w"].copy_(q)
        s["bias"] = 0.1 * torch.randn(n, generator=gen, device=dev) if case["bias"] else None
        return s
    b, hk, d, page = (case[x] for x in ("b", "hk", "d", "page"))
    if case["op"] == "cache":
        t = case["t"]
        s["table"] = _table(b, case["past"] + t, page, gen, dev)
        pages = s["table"].numel()
        for n in ("k_pool", "v_pool"):
            s[n] = torch.zeros(pages, hk, page, -(-d // 16) * 16, dtype=torch.int8, device=dev)
        for n in ("k_scale", "v_scale"):
            s[n] = torch.zeros(pages, hk, page, device=dev)
        if case["fused_kv"]:
            kv = rnd(b, t, 2, hk, d)
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            s["k"], s["v"] = rnd(b, t, hk, d), rnd(b, t, hk, d)
        s["lens"] = _lens(b, t, gen, dev) if case["ragged"] else None
        s["start"] = torch.randint(0, case["past"] + 1, (b,), generator=gen, device=dev,
                                   dtype=torch.int32)
    else:
        tq, tk, hq = case["tq"], case["tk"], case["hq"]
        s["q"] = rnd(b, tq, hq, d)
        s["table"] = _table(b, tk, page, gen, dev)
        pages = s["table"].numel()
        s["k_pool"], s["k_scale"] = _pool(pages, hk, page, d, gen, dev)
        s["v_pool"], s["v_scale"] = _pool(pages, hk, page, d, gen, dev)
        s["lens"] = _lens(b, tk, gen, dev)
    if own:
        import implicit_gemm_nhwc_amd as igc
        s["cache"] = igc.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], d)
    return s


# ----------------------------------------------------------- plain form
def _plain_ln(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xm = x - mean
    r = torch.rsqrt((xm * xm).mean(1, keepdim=True) + _EPS)
    xh = xm * r
    y = xh if s["weight"] is None else xh * s["weight"] + s["bias"]
    y = y.to(s["x"].dtype)
    if s["case"]["op"] == "ln":
        return y
    dy = s["dy"].float()
    u = dy if s["weight"] is None else dy * s["weight"]
    dx = r * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(y.dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_i8(s):
    q, scale = _quantised(s["x"])
    y = torch.matmul(q.float(), s["w"].float().t().contiguous())
    y = y * scale[:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype), "x_scale": scale}


def _slots(s, t):
    """Page and place of tokens start .. start + t - 1 of every sequence."""
    page = s["case"]["page"]
    pos = s["start"].long()[:, None] + torch.arange(t, device=s["start"].device)
    pos = pos.clamp_max(s["table"].shape[1] * page - 1)
    return s["table"].gather(1, pos // page).long(), pos % page


def _plain_cache(s):
    c = s["case"]
    t, d = c["t"], c["d"]
    pages, place = _slots(s, t)
    keep = torch.ones_like(pages, dtype=torch.bool)
    if s["lens"] is not None:
        keep = torch.arange(t, device=pages.device)[None] < s["lens"][:, None]
    got = {}
    for n in ("k", "v"):
        q, scale = _quantised(s[n])
        at = (pages[keep], slice(None), place[keep])
        s[n + "_pool"][at[0], :, at[2], :d] = q[keep]
        s[n + "_scale"][at[0], :, at[2]] = scale[keep]
        back = s[n + "_pool"][pages, :, place, :d].float() * s[n + "_scale"][pages, :, place, None]
        got[n] = torch.where(keep[:, :, None, None], back, 0.0).to(s[n].dtype)
    return got


def _plain_attn(s):
    c, q = s["case"], s["q"]
    b, tq, hq, d = q.shape
    hk, page = c["hk"], c["page"]
    g, n = hq // hk, s["table"].shape[1] * page
    # [b, pages, hk, page, d] -> [b, hk, n, d]
    k, v = (s[x + "_pool"][s["table"].long()][..., :d].float()
            * s[x + "_scale"][s["table"].long()][..., None] for x in ("k", "v"))
    k, v = (x.permute(0, 2, 1, 3, 4).reshape(b, hk, n, d) for x in (k, v))
    qf = q.float().view(b, tq, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, tq * g, d)
    p = torch.matmul(qf, k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(d))
    last = s["lens"].long()[:, None]
    if c["causal"]:
        last = last - torch.arange(tq - 1, -1, -1, device=q.device)
    last = last.expand(b, tq).repeat_interleave(g, 1)[:, None, :, None]
    p.masked_fill_(torch.arange(n, device=q.device) >= last, -math.inf)
    top = p.amax(3, keepdim=True).clamp_min_(-3e38)
    p.sub_(top).exp_()
    p.div_(p.sum(3, keepdim=True).clamp_min(1e-38))
    o = torch.matmul(p, v)
    return o.view(b, hk, tq, g, d).permute(0, 2, 1, 3, 4).reshape(b, tq, hq, d).to(q.dtype)


# -------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if not own:
        if op.startswith("ln"):
            return _plain_ln(s)
        return {"i8": _plain_i8, "cache": _plain_cache, "attn": _plain_attn}[op](s)
    import implicit_gemm_nhwc_amd as igc
    if op.startswith("ln"):
        y = igc.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS)
        if op == "ln":
            return y
        dx, dw, db = igc.layer_norm_bwd(s["dy"], s["x"], s["weight"], eps=_EPS)
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    if op == "i8":
        q, scale = igc.quantize_rows(s["x"])
        y = igc.linear_i8(q, scale, s["w"], s["w_scale"], bias=s["bias"], dtype=s["x"].dtype)
        return {"y": y, "x_scale": scale}
    if op == "cache":
        igc.kv_cache_write(s["cache"], s["k"], s["v"], s["table"], s["start"], lens=s["lens"])
        k, v = igc.kv_cache_read(s["cache"], s["table"], s["start"], s["case"]["t"],
                                 lens=s["lens"], dtype=s["k"].dtype)
        return {"k": k, "v": v}
    return igc.cache_attention(s["q"], s["cache"], s["table"], s["lens"],
                               causal=s["case"]["causal"])


def work(case):
    op = case["op"]
    if op.startswith("ln"):
        n, c = case["rows"] * case["c"], case["c"]
        if op == "ln":
            return {"bytes": 4 * n + 8 * c, "flops": 8 * n}
        # x and dy once each, y and dx; weight, bias and their gradients
        return {"bytes": 8 * n + 16 * c, "flops": 22 * n}
    if op == "i8":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + 2 * m * n + 4 * (m + n) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * k * n}
    b, hk, d = case["b"], case["hk"], case["d"]
    # ragged lengths leave about a third out
    keep = 2.0 / 3.0 if b > 1 else 1.0
    if op == "cache":
        rows = 2 * b * case["t"] * hk * (keep if case["ragged"] else 1.0)
        # 16-bit rows read, 8-bit rows and scales written and read, 16-bit rows written (all)
        return {"bytes": int(rows * (2 * d + 2 * (d + 4)) + 4 * b * case["t"] * hk * d),
                "flops": int(rows * 6 * d)}
    keys = b * case["tk"] * keep
    return {"bytes": int(4 * b * case["tq"] * case["hq"] * d + keys * hk * 2 * (d + 4)
                         + 4 * b + 4 * keys / case["page"]),
            "flops": int(4 * keys * case["tq"] * case["hq"] * d)}


# ------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "ln_train": _exact_ln, "i8": _exact_i8, "cache": _exact_cache,
            "attn": _exact_attn}[case["op"]](s)


def _exact_ln(s):
    """y from the moments about zero of the shifted row; the gradient as the
    projection of w dy off the constants and off x - mean."""
    x = s["x"].double()
    c = x.shape[1]
    w = torch.ones(c, dtype=torch.float64, device=x.device)
    if s["weight"] is not None:
        w = s["weight"].double()
    centred = x - x.sum(1, keepdim=True) / c
    sd = (centred.square().sum(1, keepdim=True) / c + _EPS).sqrt()
    y = centred / sd * w
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["case"]["op"] == "ln":
        return y
    g = s["dy"].double()
    gw = g * w
    gw = gw - gw.sum(1, keepdim=True) / c
    dx = gw / sd - centred * (gw * centred).sum(1, keepdim=True) / (c * sd ** 3)
    return {"y": y, "dx": dx, "dweight": torch.einsum("rc,rc->c", g, centred / sd),
            "dbias": torch.einsum("rc->c", g)}


def _exact_rows(x):
    """(integers, scales) of 8-bit rows in 64 bits."""
    x = x.double()
    step = x.abs().max(-1).values / 127
    return torch.where(step[..., None] > 0, torch.round(127 * x / (127 * step)[..., None]), 0.0), step


def _exact_i8(s):
    q, step = _exact_rows(s["x"])
    y = torch.mm(q, s["w"].double().t().contiguous())
    y = y * s["w_scale"].double()[None] * step[:, None]
    if s["bias"] is not None:
        y = y + s["bias"].double()[None]
    return {"y": y, "x_scale": step}


def _exact_cache(s):
    got = {}
    for n in ("k", "v"):
        q, step = _exact_rows(s[n])
        got[n] = q * step[..., None]
        if s["lens"] is not None:
            for i, m in enumerate(s["lens"].tolist()):
                got[n][i, m:] = 0
    return got


def _exact_attn(s):
    """Sequence by sequence and key head by key head over its own rows."""
    c, q = s["case"], s["q"]
    b, tq, hq, d = q.shape
    per = hq // c["hk"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for i, m in enumerate(s["lens"].tolist()):
        at = torch.arange(m, device=q.device)
        page, place = s["table"][i, at // c["page"]].long(), at % c["page"]
        for h in range(c["hk"]):
            k, v = (s[x + "_pool"][page, h, place, :d].double()
                    * s[x + "_scale"][page, h, place, None].double() for x in ("k", "v"))
            for t in range(tq):
                n = max(0, m - (tq - 1 - t)) if c["causal"] else m
                if n:
                    z = q[i, t, h * per:(h + 1) * per].double() @ k[:n].t().contiguous()
                    out[i, t, h * per:(h + 1) * per] = torch.softmax(z / d ** 0.5, 1) @ v[:n]
    return out
