"""Cases of the attention operators: cross attention to an encoder's states
(forward, single token, training) and the per-head norm of queries and keys
with the position rotation (forward, single token, training).

The cases are the attention blocks that stand between convolution layers of
an image model (the map's pixels are the queries, a text encoder's states the
keys and values) and the caption decoder that reads an image encoder's states
one token at a time.  With own = False, run() computes the operators from
elementary torch operations in 32 bits; with own = True it makes the calls of
implicit_gemm_nhwc_amd.  exact() has the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-6


# ------------------------------------------------------------------ cases
def _attn(name, op, dt, b, tq, tk, hq, hk, d, mask="none", fused_kv=False):
    """op: "attn" (inference), "attn_train" (forward and backward).  mask:
    "none", "lens" (ragged lengths), "keys" (a byte per key), "both".
    fused_kv: k and v are the halves of one projection's output."""
    c = {"op": op, "dt": dt, "b": b, "tq": tq, "tk": tk, "hq": hq, "hk": hk, "d": d,
         "mask": mask, "fused_kv": fused_kv}
    if name:
        c["name"] = name
    return c


def _norm(name, op, dt, b, tq, tk, hq, hk, d, rot, pos="rows", interleaved=False):
    """op: "norm" (inference), "norm_train".  pos: "rows" (token t is table
    row t) or "given" (table rows by position numbers)."""
    c = {"op": op, "dt": dt, "b": b, "tq": tq, "tk": tk, "hq": hq, "hk": hk, "d": d,
         "rot": rot, "pos": pos, "interleaved": interleaved}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # an 8x8 bottleneck map of one image reading a short prompt: latency
        _attn("attn_small_map", "attn", "fp16", 1, 64, 77, 8, 8, 40, "lens"),
        # a 64x64 map of 256 channels (4 heads of 64) and padded prompts
        _attn("attn_map_prompt", "attn", "bf16", 8, 4096, 77, 4, 4, 64, "keys", True),
        # 56x56 maps and a ragged batch of longer documents, shared key heads
        _attn("attn_map_ragged", "attn", "fp16", 4, 3136, 1333, 16, 4, 64, "both"),
        # the largest: 128x128 maps and 4096 encoder states, heads of 128
        _attn("attn_large", "attn", "bf16", 2, 16384, 4096, 16, 16, 128),
        # caption decoder, one token a sequence over a 28x28 map's states
        _attn("attn_token", "attn", "bf16", 8, 1, 784, 16, 4, 128, "none", True),
        # one token of a few long sequences (many images or pages a sequence)
        _attn("attn_token_long", "attn", "bf16", 4, 1, 65537, 32, 8, 128, "lens"),
        # training at a 28x28 map, batch 32, padded prompts
        _attn("attn_train_prompt", "attn_train", "bf16", 32, 784, 77, 8, 8, 64, "keys"),
        # training with grouped heads and long ragged encoder states
        _attn("attn_train_long", "attn_train", "bf16", 2, 4096, 2048, 16, 8, 128, "lens"),
        # norm and rotation of one decoded token at its position
        _norm("norm_token", "norm", "bf16", 8, 1, 1, 16, 4, 128, 128, "given"),
        # norm and rotation of a 64x64 map's queries and 1024 states' keys
        _norm("norm_map", "norm", "bf16", 16, 4096, 1024, 16, 8, 128, 128),
        # training, small odd map, part of each head rotated, adjacent pairs
        _norm("norm_train_odd", "norm_train", "fp16", 3, 961, 333, 8, 8, 80, 40, "given", True),
        # training at a 56x56 map, batch 32
        _norm("norm_train_map", "norm_train", "bf16", 32, 3136, 333, 8, 8, 64, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_token", "attn_train", "norm", "norm_train"])
    dt = rng.choice(["bf16", "fp16"])
    d = rng.choice([40, 64, 64, 80, 128, 128])
    hk = rng.choice([1, 2, 4, 8, 10])
    hq = hk * rng.choice([1, 1, 2, 4])
    b = _log(rng, 1, 32)
    if op.startswith("norm"):
        rot = rng.choice([d, d, d // 2 // 8 * 8])
        pos, inter = rng.choice(["rows", "given"]), rng.random() < 0.3
        tq, tk = _log(rng, 1, 8192), _log(rng, 1, 8192)
        while b * (tq * hq + tk * hk) * d > 16 * (4096 * 16 + 1024 * 8) * 128:
            b, tq, tk = (b + 1) // 2, (tq * 3 + 3) // 4, (tk * 3 + 3) // 4
        return _norm(None, op, dt, b, tq, tk, hq, hk, d, rot, pos, inter)
    mask = rng.choice(["none", "lens", "keys", "both"])
    fused = rng.random() < 0.5
    if op == "attn_token":
        tk = _log(rng, 33, 65537)
        while b * tk * hk * d > 4 * 65537 * 8 * 128:
            b, tk = (b + 1) // 2, (tk * 3 + 3) // 4
        return _attn(None, "attn", dt, b, rng.choice([1, 1, 1, 2, 3]), tk, hq, hk, d, mask, fused)
    tq, tk = _log(rng, 33, 16384), _log(rng, 9, 4096)
    top = 2 * 16384 * 4096 * 16 * 128 // (4 if op == "attn_train" else 1)
    while b * tq * tk * hq * d > top:
        b, tq = (b + 1) // 2, (tq * 3 + 3) // 4
    return _attn(None, op, dt, b, tq, tk, hq, hk, d, mask, fused)


# ----------------------------------------------------------------- inputs
def _lens(b, tk, gen, dev):
    """Ragged lengths between a third of tk and tk, the first one full."""
    n = torch.randint(max(1, tk // 3), tk + 1, (b,), generator=gen, device=dev,
                      dtype=torch.int32)
    n[0] = tk
    return n


def _key_mask(b, tk, gen, dev):
    """Padded prompts: a prefix of each row is kept, and of that nineteen
    keys in twenty."""
    n = _lens(b, tk, gen, dev)
    keep = torch.arange(tk, device=dev)[None] < n[:, None]
    drop = torch.rand(b, tk, generator=gen, device=dev) < 0.05
    drop[:, 0] = False
    return (keep & ~drop).to(torch.uint8)


def _angles(n, rot, dev):
    """[n, rot] float32: cosines, then sines, of t * 10000^(-2i/rot),
    the angles in 64 bits."""
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
    a = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DT[case["dt"]]
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    s = {"case": dict(case), "q": rnd(b, tq, hq, d)}
    if case["op"].startswith("norm"):
        s["k"] = rnd(b, tk, hk, d)
        for n in ("q", "k"):
            s[n + "_weight"] = 1 + 0.1 * torch.randn(d, generator=gen, device=dev)
        rows = max(tq, tk)
        if case["pos"] == "given":
            rows = max(4096, 2 * rows)
            for n, t in (("q", tq), ("k", tk)):
                first = torch.randint(0, rows - t + 1, (b, 1), generator=gen, device=dev)
                s[n + "_positions"] = (first + torch.arange(t, device=dev)).to(torch.int32)
        else:
            s["q_positions"] = s["k_positions"] = None
        s["table"] = _angles(rows, case["rot"], dev)
        if case["op"] == "norm_train":
            s["dq"], s["dk"] = rnd(b, tq, hq, d), rnd(b, tk, hk, d)
        return s
    if case["fused_kv"]:
        kv = rnd(b, tk, 2, hk, d)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    else:
        s["k"], s["v"] = rnd(b, tk, hk, d), rnd(b, tk, hk, d)
    s["kv_lens"] = _lens(b, tk, gen, dev) if case["mask"] in ("lens", "both") else None
    s["key_mask"] = _key_mask(b, tk, gen, dev) if case["mask"] in ("keys", "both") else None
    if case["op"] == "attn_train":
        s["dout"] = rnd(b, tq, hq, d)
    return s


# ----------------------------------------------------------- plain form
def _valid(s, b, tk, dev):
    ok = torch.ones(b, tk, dtype=torch.bool, device=dev)
    if s["kv_lens"] is not None:
        ok &= torch.arange(tk, device=dev)[None] < s["kv_lens"][:, None]
    if s["key_mask"] is not None:
        ok &= s["key_mask"] != 0
    return ok


def _plain_attn(s, train):
    q, k, v = s["q"], s["k"], s["v"]
    b, tq, hq, d = q.shape
    tk, hk = k.shape[1], k.shape[2]
    g, scale = hq // hk, 1.0 / math.sqrt(d)
    ok = _valid(s, b, tk, q.device)
    # queries of one key head in one product: [b, hk, tq * g, d]
    qf = q.float().view(b, tq, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, tq * g, d)
    rows = ok[:, :, None, None]
    kf = torch.where(rows, k.float(), 0.0).permute(0, 2, 1, 3).contiguous()
    vf = torch.where(rows, v.float(), 0.0).permute(0, 2, 1, 3).contiguous()
    p = torch.matmul(qf, kf.transpose(2, 3).contiguous()).mul_(scale)
    p.masked_fill_(~ok[:, None, None, :], -math.inf)
    top = p.amax(3, keepdim=True).clamp_min_(-3e38)
    p.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    p.div_(total.clamp_min(1e-38))

    def back(x):   # [b, hk, tq * g, n] -> [b, tq, hq, n]
        return x.view(b, hk, tq, g, -1).permute(0, 2, 1, 3, 4).reshape(b, tq, hq, -1)

    of = torch.matmul(p, vf)
    out = back(of).to(q.dtype)
    if not train:
        return out
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    lse = back(lse).squeeze(3).permute(0, 2, 1).contiguous()
    df = s["dout"].float().view(b, tq, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, tq * g, d)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), df)
    ds = torch.matmul(df, vf.transpose(2, 3).contiguous())
    ds.sub_((df * of).sum(3, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, kf).mul_(scale)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), qf).mul_(scale)
    return {"out": out, "lse": lse, "dq": back(dq).to(q.dtype),
            "dk": dk.permute(0, 2, 1, 3).contiguous().to(q.dtype),
            "dv": dv.permute(0, 2, 1, 3).contiguous().to(q.dtype)}


def _turn(x, cos, sin, inter, back=False):
    """The first 2 * cos.shape[-1] values of the last axis rotated."""
    h = cos.shape[-1]
    if back:
        sin = -sin
    if inter:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([t, x[..., 2 * h:]], -1)


def _plain_norm(s, n, train):
    x, w, pos = s[n], s[n + "_weight"], s[n + "_positions"]
    h, inter = s["case"]["rot"] // 2, s["case"]["interleaved"]
    rows = s["table"][:x.shape[1]][None] if pos is None else s["table"][pos.long()]
    cos, sin = rows[:, :, None, :h], rows[:, :, None, h:]
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(3, keepdim=True) + _EPS)
    xh = xf * r
    y = _turn(xh * w, cos, sin, inter).to(x.dtype)
    if not train:
        return y
    g = _turn(s["d" + n].float(), cos, sin, inter, back=True)
    dw = (g * xh).flatten(0, 2).sum(0)
    u = g * w
    dx = r * (u - xh * (u * xh).mean(3, keepdim=True))
    return y, dx.to(x.dtype), dw


# -------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        import implicit_gemm_nhwc_amd as igc
        if op == "attn":
            return igc.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"],
                                       key_mask=s["key_mask"])
        if op == "attn_train":
            out, lse = igc.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"],
                                           key_mask=s["key_mask"], return_lse=True)
            dq, dk, dv = igc.cross_attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse,
                                                 kv_lens=s["kv_lens"], key_mask=s["key_mask"])
            return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
        kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], q_table=s["table"],
                  k_table=s["table"], q_positions=s["q_positions"],
                  k_positions=s["k_positions"], eps=_EPS, interleaved=s["case"]["interleaved"])
        yq, yk = igc.qk_norm_rope(s["q"], s["k"], **kw)
        if op == "norm":
            return {"q": yq, "k": yk}
        dq, dk, dqw, dkw = igc.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **kw)
        return {"q": yq, "k": yk, "dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if op in ("attn", "attn_train"):
        return _plain_attn(s, op == "attn_train")
    if op == "norm":
        return {"q": _plain_norm(s, "q", False), "k": _plain_norm(s, "k", False)}
    (yq, dq, dqw), (yk, dk, dkw) = _plain_norm(s, "q", True), _plain_norm(s, "k", True)
    return {"q": yq, "k": yk, "dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def work(case):
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))
    nq, nk = 2 * b * tq * hq * d, 2 * b * tk * hk * d
    if case["op"].startswith("norm"):
        rows = b * (tq * hq + tk * hk)
        table = 4 * case["rot"] * (max(tq, tk) if case["pos"] == "rows" else b * (tq + tk))
        if case["op"] == "norm":
            return {"bytes": 2 * (nq + nk) + table + 8 * d, "flops": 8 * rows * d}
        return {"bytes": 4 * (nq + nk) + table + 16 * d, "flops": 24 * rows * d}
    # every key counted: ragged lengths leave about a third of it out
    keep = 1.0 if case["mask"] == "none" else 2.0 / 3.0 if b > 1 else 1.0
    small = (4 * b if case["mask"] in ("lens", "both") else 0) + (
        b * tk if case["mask"] in ("keys", "both") else 0)
    pairs = b * hq * tq * tk * keep
    if case["op"] == "attn":
        return {"bytes": int(2 * nq + 2 * nk * keep + small), "flops": int(4 * pairs * d)}
    # forward reads q, k, v and writes out, lse; backward reads dout besides
    # and writes three gradients; its scores are formed again
    return {"bytes": int(4 * nq + 4 * nk * keep + 4 * b * hq * tq + small),
            "flops": int(14 * pairs * d)}


# ------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_attn(s)


def _exact_attn(s):
    """Softmax attention head by head over the gathered valid keys."""
    c = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    train = c["op"] == "attn_train"
    per = c["hq"] // c["hk"]
    f64 = dict(dtype=torch.float64, device=q.device)
    out = torch.zeros(q.shape, **f64)
    lse = torch.full((c["b"], c["hq"], c["tq"]), -math.inf, **f64)
    dq, dk, dv = torch.zeros(q.shape, **f64), torch.zeros(k.shape, **f64), torch.zeros(v.shape, **f64)
    for i in range(c["b"]):
        n = c["tk"] if s["kv_lens"] is None else int(s["kv_lens"][i])
        idx = torch.arange(n, device=q.device)
        if s["key_mask"] is not None:
            idx = idx[s["key_mask"][i, :n] > 0]
        if idx.numel() == 0:
            continue
        for h in range(c["hq"]):
            kk, vv = k[i, idx, h // per].double(), v[i, idx, h // per].double()
            qq = q[i, :, h].double()
            z = (qq @ kk.t()) / c["d"] ** 0.5
            lse[i, h] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[i, h][:, None])
            o = w @ vv
            out[i, :, h] = o
            if train:
                go = s["dout"][i, :, h].double()
                dv[i, idx, h // per] += w.t() @ go
                gz = w * (go @ vv.t() - (go * o).sum(1, keepdim=True)) / c["d"] ** 0.5
                dq[i, :, h] = gz @ kk
                dk[i, idx, h // per] += gz.t() @ qq
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else out


def _exact_norm(s):
    """The rotation as a product of complex numbers; gradients by the chain
    rule through r = (mean x^2 + eps)^(-1/2)."""
    c = s["case"]
    h, got = c["rot"] // 2, {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"].double()
        pos = s[n + "_positions"]
        if pos is None:
            pos = torch.arange(x.shape[1], device=x.device)[None]
        t = s["table"].double()[pos.long()]
        e = torch.complex(t[..., :h], t[..., h:])[:, :, None]

        def spin(u, by):
            u = u.clone()
            lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if c["interleaved"] else (
                slice(0, h), slice(h, 2 * h))
            z = torch.complex(u[..., lo], u[..., hi]) * by
            u[..., lo], u[..., hi] = z.real, z.imag
            return u

        m = x.square().mean(-1, keepdim=True) + _EPS
        got[n] = spin(x / m.sqrt() * w, e)
        if c["op"] == "norm_train":
            gn = spin(s["d" + n].double(), e.conj())
            got["d" + n] = gn * w / m.sqrt() - x * (gn * w * x).sum(-1, keepdim=True) / (
                x.shape[-1] * m ** 1.5)
            got["d" + n + "_weight"] = (gn * x / m.sqrt()).sum((0, 1, 2))
    if c["op"] == "norm":
        return got
    return {k: got[k] for k in ("q", "k", "dq", "dk", "dq_weight", "dk_weight")}
