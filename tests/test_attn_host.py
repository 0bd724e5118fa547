"""Host-side gates of the attention operators (CPU only: every call here is
refused, or checked, before any HIP call; fake pointers are never read)."""
import math
import struct

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from implicit_gemm_nhwc_amd import attention as A

Q, K, V, O, LSE, WS, GO, DQ, DK, DV = (0x100000000 * (i + 1) for i in range(10))


def _view(p, t, h, d):
    return dict(data=p, batch=t * h * d, token=h * d, head=d)


def _attn(**kw):
    """Packed igc_cross_attn of a good call with fields replaced: q_token=...,
    k_data=..., scale=..."""
    f = dict(b=2, tq=300, tk=500, hq=8, hk=4, d=64, lse=0, lens=0, mask=0, mask_stride=0,
             scale=0.125, dtype=0, ws=0, ws_bytes=0)
    f.update({k: v for k, v in kw.items() if k in f})
    views = dict(q=_view(Q, f["tq"], f["hq"], f["d"]), k=_view(K, f["tk"], f["hk"], f["d"]),
                 v=_view(V, f["tk"], f["hk"], f["d"]), o=_view(O, f["tq"], f["hq"], f["d"]))
    for k, v in kw.items():
        if "_" in k and k.split("_")[0] in views:
            views[k.split("_")[0]][k.split("_")[1]] = v
    flat = [x for n in "qkvo" for x in views[n].values()]
    return A._ATTN.pack(f["b"], f["tq"], f["tk"], f["hq"], f["hk"], f["d"], *flat, f["lse"],
                        f["lens"], f["mask"], f["mask_stride"], f["scale"], f["dtype"], f["ws"],
                        f["ws_bytes"])


def _grad(views=None, **kw):
    kw.setdefault("lse", LSE)
    g = dict(go=_view(GO, 300, 8, 64), dq=_view(DQ, 300, 8, 64), dk=_view(DK, 500, 4, 64),
             dv=_view(DV, 500, 4, 64))
    for n, v in (views or {}).items():
        g[n].update(v)
    return _attn(**kw) + A._VIEWS.pack(*[x for n in ("go", "dq", "dk", "dv")
                                         for x in g[n].values()])


def _reason(rc):
    return igc.REASONS[rc]


BAD = [
    (dict(dtype=2), "dtype"), (dict(dtype=-1), "dtype"),
    (dict(b=-1), "shape"), (dict(tk=-1), "shape"),
    (dict(hk=3), "groups"), (dict(hk=0), "groups"),
    (dict(d=12), "head_dim"), (dict(d=136), "head_dim"), (dict(d=0), "head_dim"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=math.nan), "scale"),
    (dict(scale=math.inf), "scale"), (dict(scale=1e300), "scale"), (dict(scale=1e-300), "scale"),
    (dict(tk=1 << 31), "size_limit"), (dict(tq=1 << 30, hq=16), "size_limit"),
    (dict(k_token=1 << 23), "size_limit"), (dict(q_head=1 << 24), "size_limit"),
    (dict(q_batch=1 << 40), "size_limit"),
    (dict(q_token=-512), "stride"), (dict(mask=Q + 4096 * 4096, mask_stride=-1), "stride"),
    (dict(q_data=Q + 8), "alignment"), (dict(k_token=260), "alignment"),
    (dict(o_data=O + 2), "alignment"), (dict(lens=WS + 2), "alignment"),
    (dict(lse=LSE + 1), "alignment"),
    (dict(q_data=0), "null_pointer"), (dict(v_data=0), "null_pointer"),
    (dict(o_data=0), "null_pointer"),
    (dict(o_data=Q), "overlap"), (dict(o_data=K + 128), "overlap"), (dict(o_token=0), "overlap"),
    (dict(o_head=56), "overlap"), (dict(o_batch=8), "overlap"),
    (dict(lse=Q + 64), "overlap"), (dict(lse=O + 64), "overlap"), (dict(lens=O + 64), "overlap"),
    (dict(mask=O, mask_stride=500), "overlap"),
]


def test_good_calls_accepted():
    L = igc.lib()
    assert L.cross_attn_fwd_check(_attn()) == 0
    assert L.cross_attn_fwd_check(_attn(lse=LSE, lens=WS, mask=WS + 64, mask_stride=0)) == 0
    assert L.cross_attn_fwd_check(_attn(k_batch=0, v_batch=0)) == 0      # shared states
    assert L.cross_attn_fwd_check(_attn(tk=0, k_data=0, v_data=0)) == 0
    assert L.cross_attn_fwd_check(_attn(b=0, q_data=0, k_data=0, v_data=0, o_data=0)) == 0
    assert L.cross_attn_fwd_check(_attn(dtype=1, d=8)) == 0
    # strides of an axis of one entry say nothing
    assert L.cross_attn_fwd_check(_attn(b=1, q_batch=3, o_batch=-5)) == 0
    assert L.cross_attn_bwd_check(_grad()) == 0
    assert L.cross_attn_bwd_check(_grad(dict(dq=dict(data=0)))) == 0
    assert L.cross_attn_bwd_check(_grad(dict(dk=dict(data=0), dv=dict(data=0)))) == 0


@pytest.mark.parametrize("kw,reason", BAD)
def test_attention_refusals(kw, reason):
    L = igc.lib()
    packed = _attn(**kw)
    assert _reason(L.cross_attn_fwd_check(packed)) == reason
    assert L.cross_attn_fwd(packed, None) == 0


def test_head_major_strides():
    """Keys and values of a long head-major cache have head strides of
    kv_len * D; queries stay within what a tile addresses in 32 bits."""
    L = igc.lib()
    # far above the other buffers of the calls
    far = 1 << 46
    for head, reason in ((1 << 23, 0), (1 << 39, 0), (1 << 40, "size_limit")):
        for n in "kv":
            rc = L.cross_attn_fwd_check(_attn(**{n + "_head": head, n + "_data": far}))
            assert rc == 0 if reason == 0 else _reason(rc) == reason
    for name in ("q_head", "o_head"):
        assert _reason(L.cross_attn_fwd_check(_attn(**{name: 1 << 23}))) == "size_limit"
    # more than an address space holds
    rc = L.cross_attn_fwd_check(_attn(b=1 << 22, k_batch=1 << 39))
    assert _reason(rc) == "size_limit"
    for n in ("dk", "dv"):
        views = {n: dict(data=far, batch=1 << 39, head=1 << 24)}
        assert L.cross_attn_bwd_check(_grad(views)) == 0


def test_attention_workspace_rules():
    L = igc.lib()
    few = dict(b=1, tq=1, tk=20000, hq=8, hk=8)
    need = L.cross_attn_fwd_workspace_bytes(_attn(**few))
    assert need > 0
    assert L.cross_attn_fwd_workspace_bytes(_attn(dtype=2)) == 0
    assert L.cross_attn_fwd_check(_attn(**few, ws=WS, ws_bytes=need)) == 0
    for kw, reason in ((dict(ws=WS, ws_bytes=need - 1), "workspace"),
                       (dict(ws=WS + 4, ws_bytes=need), "alignment"),
                       (dict(ws=O, ws_bytes=need), "overlap"),
                       (dict(ws=K, ws_bytes=need), "overlap")):
        packed = _attn(**few, **kw)
        assert _reason(L.cross_attn_fwd_check(packed)) == reason
        assert L.cross_attn_fwd(packed, None) == 0
    need = L.cross_attn_bwd_workspace_bytes(_grad())
    assert need > 0
    assert L.cross_attn_bwd_check(_grad(ws=WS, ws_bytes=need)) == 0
    for kw, reason in ((dict(ws=WS, ws_bytes=need - 1), "workspace"),
                       (dict(ws=DQ, ws_bytes=need), "overlap"),
                       (dict(ws=GO, ws_bytes=need), "overlap"),
                       (dict(ws=LSE, ws_bytes=need), "overlap")):
        packed = _grad(**kw)
        assert _reason(L.cross_attn_bwd_check(packed)) == reason
        assert L.cross_attn_bwd(packed, None) == 0


@pytest.mark.parametrize("views,kw,reason", [
    ({}, dict(lse=0), "null_pointer"),
    (dict(go=dict(data=0)), {}, "null_pointer"),
    (dict(dk=dict(data=0)), {}, "null_pointer"),
    (dict(dv=dict(data=0)), {}, "null_pointer"),
    (dict(go=dict(data=GO + 8)), {}, "alignment"),
    (dict(dq=dict(token=0)), {}, "overlap"),
    (dict(dq=dict(data=Q)), {}, "overlap"),
    (dict(dk=dict(data=K)), {}, "overlap"),
    (dict(dv=dict(data=GO)), {}, "overlap"),
    (dict(dk=dict(data=LSE)), {}, "overlap"),
    (dict(dv=dict(batch=64)), {}, "overlap"),
    # 64 token strides and the strides over a group's 128 heads pass 2^31 bytes
    (dict(go=dict(token=(1 << 23) - 8, head=(1 << 23) - 8), dq=dict(data=0)), dict(hq=512),
     "size_limit"),
    ({}, dict(scale=-0.1), "scale"),
    ({}, dict(dtype=2), "dtype"),
    ({}, dict(d=20), "head_dim"),
])
def test_attention_gradient_refusals(views, kw, reason):
    L = igc.lib()
    packed = _grad(views, **kw)
    rc = L.cross_attn_bwd_check(packed)
    assert _reason(rc) == reason
    assert L.cross_attn_bwd(packed, None) == 0


def test_null_arguments():
    L = igc.lib()
    for name in ("cross_attn_fwd", "cross_attn_bwd", "qk_norm_rope_fwd", "qk_norm_rope_bwd"):
        assert _reason(getattr(L, name + "_check")(None)) == "null_pointer"
        assert getattr(L, name)(None, None) == 0


W, T, P, DW = (0x2000000000 + (i << 24) for i in range(4))


def _norm(q=None, k=None, d=64, rot=64, inter=0, dtype=0, eps=1e-6, ws=0, ws_bytes=0):
    def part(base, h, over):
        f = dict(b=2, t=100, h=h, x=base, x_b=100 * h * 64, x_t=h * 64, x_h=64, g=base + (1 << 28),
                 g_b=100 * h * 64, g_t=h * 64, g_h=64, o=base + (2 << 28), o_b=100 * h * 64,
                 o_t=h * 64, o_h=64, w=0, dw=0, table=T, rows=128, pos=0, pos_b=0)
        f.update(over or {})
        return list(f.values())
    return A._QK.pack(*part(Q, 8, q), *part(K, 4, k), d, rot, inter, dtype, eps, ws, ws_bytes)


def test_norm_good_calls():
    L = igc.lib()
    assert L.qk_norm_rope_fwd_check(_norm()) == 0
    assert L.qk_norm_rope_bwd_check(_norm()) == 0
    assert L.qk_norm_rope_fwd_check(_norm(q=dict(o=Q))) == 0                 # in place
    assert L.qk_norm_rope_fwd_check(_norm(k=dict(b=0, x=0, o=0, g=0, table=0, rows=0))) == 0
    assert L.qk_norm_rope_fwd_check(_norm(rot=0, q=dict(table=0, rows=0),
                                          k=dict(table=0, rows=0))) == 0
    assert L.qk_norm_rope_fwd_check(_norm(q=dict(rows=1, pos=P))) == 0
    # both parts in place in one buffer of queries and keys
    both = dict(x_t=12 * 64, o_t=12 * 64, x_b=1200 * 64, o_b=1200 * 64)
    assert L.qk_norm_rope_fwd_check(_norm(q=dict(x=Q, o=Q, **both),
                                          k=dict(x=Q + 1024, o=Q + 1024, **both))) == 0
    assert L.qk_norm_rope_bwd_check(_norm(q=dict(o=Q + (1 << 28)))) == 0     # dx over dy


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "dtype"), (dict(d=63), "head_dim"), (dict(d=256), "head_dim"),
    (dict(rot=63), "head_dim"), (dict(rot=66), "head_dim"), (dict(rot=-2), "head_dim"),
    (dict(eps=-1.0), "scale"), (dict(eps=math.nan), "scale"),
    (dict(q=dict(b=-1)), "shape"), (dict(q=dict(rows=99)), "shape"),
    (dict(k=dict(rows=0, pos=P)), "shape"),
    (dict(q=dict(b=1 << 30, t=1 << 30)), "size_limit"),
    (dict(q=dict(x_t=1 << 23)), "size_limit"),
    (dict(q=dict(x=0)), "null_pointer"), (dict(k=dict(o=0)), "null_pointer"),
    (dict(q=dict(table=0)), "null_pointer"),
    (dict(q=dict(x=Q + 2)), "alignment"), (dict(q=dict(w=W + 2)), "alignment"),
    (dict(q=dict(pos=P + 1)), "alignment"), (dict(k=dict(x_h=68)), "alignment"),
    (dict(q=dict(x_h=-64)), "stride"), (dict(q=dict(pos=P, pos_b=-1)), "stride"),
    (dict(q=dict(o=Q + 16)), "overlap"), (dict(q=dict(o=K)), "overlap"),
    (dict(q=dict(o_t=0)), "overlap"), (dict(q=dict(o=T)), "overlap"),
    (dict(k=dict(o=Q + (2 << 28) + 128)), "overlap_outputs"),
])
def test_norm_refusals(kw, reason):
    L = igc.lib()
    packed = _norm(**kw)
    rc = L.qk_norm_rope_fwd_check(packed)
    if reason == "overlap_outputs":
        # two outputs may interleave in one buffer (a fused projection's
        # gradient): their elements are the caller's to keep apart
        assert rc == 0
        return
    assert _reason(rc) == reason
    assert L.qk_norm_rope_fwd(packed, None) == 0


@pytest.mark.parametrize("kw,reason", [
    (dict(q=dict(g=0)), "null_pointer"),
    (dict(q=dict(o=Q)), "overlap"),                       # dx over x
    (dict(q=dict(dw=Q)), "overlap"), (dict(q=dict(dw=DW), k=dict(dw=DW + 4)), "overlap"),
    (dict(q=dict(dw=DW + 2)), "alignment"), (dict(q=dict(dw=W, w=W)), "overlap"),
    (dict(q=dict(dw=DW), ws=WS, ws_bytes=64), "workspace"),
    (dict(q=dict(dw=DW), ws=WS + 8, ws_bytes=1 << 30), "alignment"),
    (dict(q=dict(dw=DW), ws=Q, ws_bytes=1 << 30), "overlap"),
])
def test_norm_gradient_refusals(kw, reason):
    L = igc.lib()
    packed = _norm(**kw)
    assert _reason(L.qk_norm_rope_bwd_check(packed)) == reason
    assert L.qk_norm_rope_bwd(packed, None) == 0


def test_structs_are_the_headers():
    # 8-byte fields throughout: the packed sizes are those of the C structs
    assert A._ATTN.size == 8 * 30 and A._VIEWS.size == 8 * 16
    assert A._QK.size == 8 * (2 * 21 + 7)
    assert struct.calcsize("P") == 8


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 4, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(igc.InvalidArgument):
        igc.cross_attention(q, q, q)
    with pytest.raises(igc.InvalidArgument):
        igc.cross_attention_bwd(q, q, q, q, q, None)
    with pytest.raises(igc.InvalidArgument):
        igc.qk_norm_rope(q)
    with pytest.raises(igc.InvalidArgument):
        igc.qk_norm_rope_bwd(q, None, q)


def test_rope_tables():
    t = igc.rope_table(5, 6, base=100.0, first=3)
    assert t.shape == (5, 6) and t.dtype == torch.float32
    for p in range(5):
        for i in range(3):
            a = (p + 3) * 100.0 ** (-2 * i / 6)
            assert t[p, i].item() == pytest.approx(math.cos(a), abs=1e-7)
            assert t[p, 3 + i].item() == pytest.approx(math.sin(a), abs=1e-7)
    m = igc.rope_table_2d(3, 4, 8, base=100.0)
    one = igc.rope_table(4, 4, base=100.0)
    for y in range(3):
        for x in range(4):
            row = m[y * 4 + x]
            assert torch.equal(row[:2], one[y, :2]) and torch.equal(row[2:4], one[x, :2])
            assert torch.equal(row[4:6], one[y, 2:]) and torch.equal(row[6:], one[x, 2:])
