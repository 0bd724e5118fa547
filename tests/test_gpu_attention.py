"""Cross attention on the GPU against the float64 oracle.

Bounds, element by element, with u = eps / 2 of the element type: each output
is rounded once (u times its value); the probabilities (forward, dv) and ds
(dq, dk) are rounded before their products (u times the sum of magnitudes they
enter); Delta is formed from the rounded out; and everything held in fp32
costs `slop`: the scores' products (D roundings of at most sum |q| |k|), the
exponent (an error of |s| 2^-23 in its argument) and the sums over the keys.
fp16 probabilities below 2^-14 of their scaled range lose bits: 2^-24 of the
sum of magnitudes covers them.
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


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _make(dt, b, tq, tk, hq, hk, d, mask="none", layout="dense", seed=0, amp=1.0):
    gen = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen) * amp

    if layout == "fused":        # k and v halves of one projection
        q = rnd(b, tq, hq, d).to(dt).to(DEV)
        kv = rnd(b, tk, 2, hk, d).to(dt).to(DEV)
        k, v = kv[:, :, 0], kv[:, :, 1]
    elif layout == "heads":      # [batch, head, token, D] storage
        q, k, v = (rnd(b, h, t, d).to(dt).to(DEV).transpose(1, 2)
                   for t, h in ((tq, hq), (tk, hk), (tk, hk)))
    elif layout == "padded":     # rows longer than the heads, an offset start
        q, k, v = (rnd(b, t + 3, h + 1, d + 24).to(dt).to(DEV)[:, 1:t + 1, 1:, 8:8 + d]
                   for t, h in ((tq, hq), (tk, hk), (tk, hk)))
    else:
        q, k, v = (rnd(b, t, h, d).to(dt).to(DEV) for t, h in ((tq, hq), (tk, hk), (tk, hk)))
    go = rnd(b, tq, hq, d).to(dt).to(DEV)
    lens = km = None
    if mask in ("lens", "both"):
        lens = torch.randint(0, tk + 1, (b,), generator=gen, dtype=torch.int32)
        lens[0] = tk
        if b > 1:
            lens[1] = 0
        lens = lens.to(DEV)
    if mask in ("keys", "both"):
        km = (torch.rand(b, tk, generator=gen) < 0.7).to(torch.uint8)
        if b > 2:
            km[2] = 0
        km = km.to(DEV)
    return q, k, v, go, lens, km


def _slop(r, d, tk):
    return 2.0 ** -22 * (r["s_abs"] * (1 + d / 4) + tk / 4 + 16)


def _near(name, got, ref, bound):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - bound
    i = over.argmax() if over.numel() else None
    worst = float(((got - ref).abs() / bound.clamp_min(1e-300)).max()) if over.numel() else 0.0
    _say(f"    {name}: {worst:.3f} of the bound")
    assert i is None or float(over.max()) <= 0, (
        f"{name}: {float(got.flatten()[i])} for {float(ref.flatten()[i])}, "
        f"bound {float(bound.flatten()[i]):.3g}")


def _check(r, dt, tk, out=None, lse=None, grads=None, max_go=0.0, max_v=0.0, scale=None):
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -24 if dt == HF else 2.0 ** -133   # half a step of the smallest numbers
    b, tq, hq, d = r["out"].shape
    scale = d ** -0.5 if scale is None else scale
    slop = _slop(r, d, tk)                                     # [b, hq, tq]
    rows = slop.transpose(1, 2)[..., None]
    few = (2.0 ** -24 if dt == HF else 0.0) * r["v_abs"][:, None]
    ob = u * r["out"].abs() + (1 + u) * ((u + rows) * r["out_abs"] + few) + tiny
    if out is not None:
        _near("out", out, r["out"], ob)
    if lse is not None:
        got = lse.cpu().double()
        empty = torch.isinf(r["lse"])
        assert torch.equal(torch.isinf(got) & (got < 0), empty)
        _near("lse", got.masked_fill(empty, 0), r["lse"].masked_fill(empty, 0),
              slop + 2.0 ** -23 * r["lse"].masked_fill(empty, 0).abs())
    if grads is None:
        return
    dq, dk, dv = grads
    hk = r["dk"].shape[2]
    g = hq // hk
    qb, kb, vb = torch.zeros_like(r["dq"]), torch.zeros_like(r["dk"]), torch.zeros_like(r["dv"])
    # fp16: ds is kept within 2^15 of its bound 2 max|do| max|v|, so its
    # smallest step is 2^-39 of it
    step = 2.0 ** -37 * max_go * max_v * 2 if dt == HF else 0.0
    for (i, h), (idx, p, ds, go, kk, vv, qq) in r["parts"].items():
        s = slop[i, h][:, None]
        dd = (go.abs() * ob[i, :, h]).sum(1, keepdim=True)
        mag = go.abs() @ vv.abs().t() + (go.abs() * r["out_abs"][i, :, h]).sum(1, keepdim=True)
        e = u * ds.abs() + p * dd + s * p * mag + step
        qb[i, :, h] = scale * (e @ kk.abs())
        kb[i, idx, h // g] += scale * (e.t() @ qq.abs())
        vb[i, idx, h // g] += ((u + s) * p + (2.0 ** -38 if dt == HF else 0)).t() @ go.abs()
    more = 1 + u
    _near("dq", dq, r["dq"], u * r["dq"].abs() + more * qb + tiny)
    _near("dk", dk, r["dk"], u * r["dk"].abs() + more * kb + tiny)
    _near("dv", dv, r["dv"], u * r["dv"].abs() + more * vb + tiny)


CASES = [
    # dt, b, tq, tk, hq, hk, d, mask, layout
    (BF, 1, 1, 1, 1, 1, 8, "none", "dense"),
    (HF, 1, 1, 1, 1, 1, 128, "none", "dense"),
    (BF, 2, 1, 33, 4, 4, 64, "none", "dense"),            # one token
    (HF, 3, 1, 257, 8, 2, 128, "both", "fused"),
    (BF, 3, 1, 1000, 8, 1, 40, "lens", "dense"),          # split keys, joined
    (HF, 4, 3, 777, 6, 2, 96, "keys", "heads"),
    (BF, 1, 2, 3000, 64, 4, 80, "none", "padded"),
    (HF, 3, 2, 129, 16, 1, 32, "both", "dense"),          # 32 rows exactly
    (BF, 3, 11, 129, 3, 1, 64, "both", "dense"),          # 33 rows
    (HF, 1, 64, 77, 8, 8, 40, "lens", "dense"),
    (BF, 3, 65, 64, 2, 2, 64, "both", "fused"),
    (HF, 2, 127, 65, 2, 1, 128, "keys", "dense"),
    (BF, 2, 129, 63, 3, 3, 16, "none", "heads"),
    (HF, 3, 130, 31, 6, 2, 72, "both", "padded"),
    (BF, 3, 100, 500, 4, 2, 128, "both", "dense"),
    (HF, 3, 300, 200, 5, 5, 88, "lens", "fused"),
    (BF, 3, 200, 333, 10, 2, 104, "keys", "dense"),
    (HF, 1, 33, 2049, 2, 2, 64, "none", "dense"),         # few rows, many keys: split
    (BF, 1, 2049, 33, 2, 2, 64, "none", "dense"),         # many rows, few keys: split dk, dv
    (HF, 1, 1025, 40, 4, 1, 128, "none", "dense"),
    (BF, 1, 700, 257, 3, 1, 48, "none", "heads"),         # groups not a power of two
    (HF, 2, 96, 256, 7, 1, 24, "keys", "dense"),
    (BF, 2, 500, 130, 2, 2, 112, "keys", "padded"),
    (HF, 2, 257, 300, 2, 2, 120, "keys", "dense"),
    (BF, 3, 40, 70, 2, 2, 56, "both", "dense"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}")
def test_attention_and_gradients(case):
    dt, b, tq, tk, hq, hk, d, mask, layout = case
    _say(f"attention {case}")
    q, k, v, go, lens, km = _make(*case, seed=tq * 7 + tk)
    kw = dict(kv_lens=lens, key_mask=km)
    r = oracle.cross_attention(q, k, v, kv_lens=lens, key_mask=km, dout=go)
    out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
    only = igc.cross_attention(q, k, v, **kw)
    assert torch.equal(out, only)
    _check(r, dt, tk, out, lse)
    grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    _check(r, dt, tk, grads=grads, max_go=float(go.norm(dim=-1).max()),
           max_v=float(v.norm(dim=-1).max()))
    # keys that are not valid have no gradient, rows without keys neither
    for i in range(b):
        ok = oracle.valid_keys(i, tk, lens, km).to(DEV)
        assert (grads[1][i, ~ok] == 0).all() and (grads[2][i, ~ok] == 0).all()
        if not ok.any():
            assert (out[i] == 0).all() and (lse[i] == -math.inf).all() and (grads[0][i] == 0).all()
    # the order of every sum is fixed
    out2, lse2 = igc.cross_attention(q, k, v, return_lse=True, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(grads, igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("scale,amp", [(0.01, 1.0), (1.0, 3.0), (3.0, 0.02)])
def test_attention_scales(dt, scale, amp):
    """Flat and saturated rows, small and large gradients (fp16's range)."""
    for grad in (1e-3, 30.0):
        _say(f"scales {dt} {scale} {amp} {grad}")
        q, k, v, go, lens, km = _make(dt, 2, 70, 150, 4, 2, 64, "keys", seed=5, amp=amp)
        go = go * grad
        kw = dict(kv_lens=lens, key_mask=km, scale=scale)
        r = oracle.cross_attention(q, k, v, dout=go, **kw)
        out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
        _check(r, dt, 150, out, lse, scale=scale)
        grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
        _check(r, dt, 150, grads=grads, max_go=float(go.norm(dim=-1).max()),
               max_v=float(v.norm(dim=-1).max()), scale=scale)


@pytest.mark.parametrize("tq,tk", [(1, 300), (1, 5000), (90, 300), (700, 90)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_masked_places_may_hold_anything(dt, tq, tk):
    """NaN and infinities in keys and values that are not valid change no bit
    of any result."""
    _say(f"masked places {dt} {tq} {tk}")
    q, k, v, go, lens, km = _make(dt, 3, tq, tk, 4, 2, 64, "both", seed=3)
    kw = dict(kv_lens=lens, key_mask=km)
    out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
    grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    k2, v2 = k.clone(), v.clone()
    for i in range(3):
        bad = (~oracle.valid_keys(i, tk, lens, km)).nonzero()[:, 0].to(DEV)
        for n, x in enumerate((math.nan, math.inf, -math.inf, torch.finfo(dt).min)):
            k2[i, bad[n::4]] = x
            v2[i, bad[n::4]] = x if n else math.inf
    out2, lse2 = igc.cross_attention(q, k2, v2, return_lse=True, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(grads, igc.cross_attention_bwd(go, q, k2, v2, out, lse, **kw)):
        assert torch.equal(x, y)


def test_nan_in_a_valid_key_reaches_its_rows():
    q, k, v, _, _, _ = _make(BF, 2, 40, 100, 2, 2, 64)
    v[1, 7] = math.nan
    out = igc.cross_attention(q, k, v)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()
    k[0, 99] = math.nan
    assert torch.isnan(igc.cross_attention(q, k, v)[0]).all()
    assert torch.isnan(igc.cross_attention(q[:, :1], k, v)[0]).all()


def test_lengths_out_of_range_are_clamped():
    q, k, v, _, _, _ = _make(BF, 3, 40, 100, 2, 2, 64)
    lens = torch.tensor([-5, 1 << 30, 100], dtype=torch.int32, device=DEV)
    out, lse = igc.cross_attention(q, k, v, kv_lens=lens, return_lse=True)
    full = igc.cross_attention(q, k, v)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert torch.equal(out[1:], full[1:])


def test_empty_extents():
    for b, tq, tk, h in ((0, 4, 4, 2), (2, 0, 4, 2), (2, 4, 0, 2), (2, 4, 4, 0), (2, 1, 0, 2)):
        q, k, v, go, _, _ = _make(BF, b, tq, tk, h, h, 64)
        out, lse = igc.cross_attention(q, k, v, return_lse=True)
        assert out.shape == q.shape and (out == 0).all() and (lse == -math.inf).all()
        dq, dk, dv = igc.cross_attention_bwd(go, q, k, v, out, lse)
        assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all()
        assert dk.shape == k.shape


def test_shared_states_through_stride_zero():
    """One encoder's states for a whole batch, and a mask for it."""
    q, k, v, go, _, _ = _make(HF, 1, 50, 120, 4, 2, 64)
    q = torch.randn(3, 50, 4, 64, device=DEV).to(HF)
    go = torch.randn(3, 50, 4, 64, device=DEV).to(HF)
    km = (torch.rand(1, 120, device=DEV) < 0.5)
    big = [t.expand(3, *t.shape[1:]) for t in (k, v)]
    args = (q, *big)
    own = (q, *(t.contiguous() for t in big))
    out, lse = igc.cross_attention(*args, key_mask=km.expand(3, 120), return_lse=True)
    out2, lse2 = igc.cross_attention(*own, key_mask=km.repeat(3, 1), return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    g1 = igc.cross_attention_bwd(go, *args, out, lse, key_mask=km.expand(3, 120))
    g2 = igc.cross_attention_bwd(go, *own, out, lse, key_mask=km.repeat(3, 1))
    for x, y in zip(g1, g2):
        assert x.shape[0] == 3 and torch.equal(x, y)


@pytest.mark.parametrize("tq", [1, 40])
def test_offsets_past_32_bits(tq):
    """Token strides that carry the last keys past 4 GiB."""
    tk, step = 34000, 65536
    kbuf = torch.zeros(tk, step, dtype=BF, device=DEV)
    kbuf[:, 64:192] = torch.randn(tk, 128, device=DEV).to(BF)
    k = kbuf[None, :, None, 64:128]
    v = kbuf[None, :, None, 128:192]
    q = torch.randn(1, tq, 1, 64, device=DEV).to(BF)
    go = torch.randn(1, tq, 1, 64, device=DEV).to(BF)
    out, lse = igc.cross_attention(q, k, v, return_lse=True)
    kc, vc = k.contiguous(), v.contiguous()
    out2, lse2 = igc.cross_attention(q, kc, vc, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(igc.cross_attention_bwd(go, q, k, v, out, lse),
                    igc.cross_attention_bwd(go, q, kc, vc, out, lse)):
        assert torch.equal(x, y)
    # and as outputs: dk and dv into the same wide rows
    lib_dk, lib_dv = kbuf[None, :, None, 256:320], kbuf[None, :, None, 320:384]
    dq = torch.empty_like(q)
    rc = igc.cross_attn_bwd(go, q, kc, vc, out, lse, dq, lib_dk, lib_dv)
    assert rc == 1
    assert torch.equal(lib_dk.contiguous(), y_dk(go, q, kc, vc, out, lse))


@pytest.mark.parametrize("tq", [1, 40])
def test_head_major_cache(tq):
    """Keys and values [b, heads, tokens, D] seen as [b, tokens, heads, D],
    with heads further apart than 2^23 elements: the dense cache's bits."""
    tk, d = 70000, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, go = (torch.randn(1, tq, 4, d, device=DEV, generator=gen).to(BF) for _ in range(2))
    kv = torch.randn(2, 1, 2, tk, d, device=DEV, generator=gen).to(BF)
    k, v = kv.transpose(2, 3)
    assert k.stride(2) > 1 << 23
    kc, vc = k.contiguous(), v.contiguous()
    out, lse = igc.cross_attention(q, k, v, return_lse=True)
    want, want_lse = igc.cross_attention(q, kc, vc, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    grads = igc.cross_attention_bwd(go, q, kc, vc, out, lse)
    dkv = torch.full_like(kv, 7.0)
    dk, dv = dkv.transpose(2, 3)
    dq = torch.empty_like(q)
    assert igc.cross_attn_bwd(go, q, k, v, out, lse, dq, dk, dv) == 1
    for x, y in zip((dq, dk, dv), grads):
        assert torch.equal(x, y)


def y_dk(*a):
    return igc.cross_attention_bwd(*a)[1]


@pytest.mark.parametrize("tq,tk", [(1, 700), (60, 90), (400, 50)])
def test_guard_bands(tq, tk):
    """Nothing outside the outputs' elements is written."""
    q, k, v, go, lens, km = _make(BF, 2, tq, tk, 4, 2, 40, "keys")
    ref, lse_ref = igc.cross_attention(q, k, v, key_mask=km, return_lse=True)
    out = torch.full((2, tq + 2, 6, 56), 7.0, dtype=BF, device=DEV)
    lse = torch.full((2 * 4 * tq + 64,), 5.0, device=DEV)
    rc = igc.cross_attn_fwd(q, k, v, out[:, 1:-1, 1:5, 8:48], lse=lse[32:-32].view(2, 4, tq),
                            key_mask=km)
    assert rc == 1
    assert torch.equal(out[:, 1:-1, 1:5, 8:48], ref)
    assert torch.equal(lse[32:-32].view(2, 4, tq), lse_ref)
    out[:, 1:-1, 1:5, 8:48] = 7.0
    assert (out == 7.0).all() and (lse[:32] == 5.0).all() and (lse[-32:] == 5.0).all()
    grads = igc.cross_attention_bwd(go, q, k, v, ref, lse_ref, key_mask=km)
    pads = [torch.full((2, t.shape[1] + 2, t.shape[2] + 2, 56), 7.0, dtype=BF, device=DEV)
            for t in (q, k, v)]
    cut = [p[:, 1:-1, 1:-1, 8:48] for p in pads]
    need = igc.cross_attn_bwd_workspace_bytes(q.shape, k.shape, BF)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    rc = igc.cross_attn_bwd(go, q, k, v, ref, lse_ref, *cut, key_mask=km, workspace=ws[128:-128])
    assert rc == 1
    for c, p, g in zip(cut, pads, grads):
        assert torch.equal(c, g)
        c.fill_(7.0)
        assert (p == 7.0).all()
    assert (ws[:128] == 0x5A).all() and (ws[-128:] == 0x5A).all()


def test_gradients_not_wanted():
    q, k, v, go, _, _ = _make(HF, 2, 300, 90, 4, 2, 64)
    out, lse = igc.cross_attention(q, k, v, return_lse=True)
    dq, dk, dv = igc.cross_attention_bwd(go, q, k, v, out, lse)
    a, b, c = torch.empty_like(dq), torch.empty_like(dk), torch.empty_like(dv)
    assert igc.cross_attn_bwd(go, q, k, v, out, lse, a, None, None) == 1
    assert igc.cross_attn_bwd(go, q, k, v, out, lse, None, b, c) == 1
    assert torch.equal(a, dq) and torch.equal(b, dk) and torch.equal(c, dv)


def test_another_stream_and_given_workspace():
    q, k, v, go, lens, _ = _make(BF, 3, 2, 3000, 8, 2, 128, "lens")
    ref, lse_ref = igc.cross_attention(q, k, v, kv_lens=lens, return_lse=True)
    g_ref = igc.cross_attention_bwd(go, q, k, v, ref, lse_ref, kv_lens=lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out, lse = igc.cross_attention(q, k, v, kv_lens=lens, return_lse=True, stream=stream)
        g = igc.cross_attention_bwd(go, q, k, v, out, lse, kv_lens=lens, stream=stream)
        s.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, lse_ref)
        assert all(torch.equal(x, y) for x, y in zip(g, g_ref))
    need = igc.cross_attn_fwd_workspace_bytes(q.shape, k.shape, BF)
    assert need > 0
    out = torch.empty_like(ref)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert igc.cross_attn_fwd(q, k, v, out, kv_lens=lens, workspace=ws) == 1
    assert torch.equal(out, ref)
    assert igc.cross_attn_fwd(q, k, v, out, kv_lens=lens, workspace=ws[:need // 32 * 16]) == 0
    assert igc.cross_attn_fwd_check(q, k, v, out, kv_lens=lens, workspace=ws[:16]) == 12


def test_captured_into_a_graph():
    """Forward and backward in a graph, replayed with eager work between."""
    q, k, v, go, lens, km = _make(HF, 3, 90, 200, 4, 2, 64, "both")
    kw = dict(kv_lens=lens, key_mask=km)
    igc.cross_attention(q, k, v, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
        grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
        tok = igc.cross_attention(q[:, :1], k, v, **kw)
    for n in range(4):
        for t in (q, k, v, go):
            t.copy_(torch.randn(t.shape, device=DEV) * (n + 1) * 0.5)
        lens.copy_(torch.tensor([200, 50 * n, 3], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        o2, l2 = igc.cross_attention(q, k, v, return_lse=True, **kw)
        g2 = igc.cross_attention_bwd(go, q, k, v, o2, l2, **kw)
        t2 = igc.cross_attention(q[:, :1], k, v, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(tok, t2)
        assert all(torch.equal(x, y) for x, y in zip(grads, g2))


@pytest.mark.parametrize("case", [c for c in CASES if c[2] > 1 or c[3] > 1],
                         ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}")
def test_poisoned_lds(case):
    """The same bits from the build whose kernels fill their LDS with NaN
    first: no read runs ahead of its data."""
    _say(f"poison {case}")
    q, k, v, go, lens, km = _make(*case, seed=11)
    kw = dict(kv_lens=lens, key_mask=km)
    out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
    grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    with igc.using_library(igc.POISON_LIB_PATH):
        out2, lse2 = igc.cross_attention(q, k, v, return_lse=True, **kw)
        grads2 = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(grads, grads2))


def test_binding_refusals():
    q, k, v, go, lens, km = _make(BF, 2, 10, 20, 4, 2, 64, "both")
    bad = [dict(q=q[0]), dict(k=k.half()), dict(v=v[:, :19]), dict(k=k[:1], v=v[:1]),
           dict(q=q.transpose(2, 3)), dict(kv_lens=lens.long()), dict(kv_lens=lens[:1]),
           dict(key_mask=km[:, :10]), dict(key_mask=km.float()), dict(k=k.cpu()),
           dict(q=q.float(), k=k.float(), v=v.float())]
    for kw in bad:
        a = dict(q=q, k=k, v=v)
        a.update({n: kw.pop(n) for n in list(kw) if n in a})
        with pytest.raises(igc.InvalidArgument):
            igc.cross_attention(a["q"], a["k"], a["v"], **kw)
    with pytest.raises(igc.Declined, match="scale"):
        igc.cross_attention(q, k, v, scale=-1.0)
    with pytest.raises(igc.Declined, match="groups"):
        igc.cross_attention(q[:, :, :3], k, v)
    with pytest.raises(igc.Declined, match="head_dim"):
        igc.cross_attention(q[..., :12], k[..., :12], v[..., :12])
    with pytest.raises(igc.Declined, match="dtype"):
        f8 = [t.to(torch.float8_e4m3fn) for t in (q, k, v)]
        igc.cross_attention(*f8)
    with pytest.raises(igc.Declined, match="alignment"):
        igc.cross_attention(torch.zeros(2 * 10 * 4 * 64 + 1, dtype=BF, device=DEV)[1:].view(
            2, 10, 4, 64), k, v)
    out, lse = igc.cross_attention(q, k, v, return_lse=True)
    for a in ((go[:1], out, lse), (go, out[:, :9], lse), (go, out, lse[:, :2]),
              (go, out, lse.double())):
        with pytest.raises(igc.InvalidArgument):
            igc.cross_attention_bwd(a[0], q, k, v, a[1], a[2])
    with pytest.raises(igc.Declined, match="null_pointer"):
        igc.cross_attention_bwd(go, q, k, v, out, None)
