"""Host-side gates of the decoder block's operators (CPU only: every call here
is refused, or checked, before any HIP call; fake pointers are never read)."""
import math
import os
import struct
import subprocess

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from implicit_gemm_nhwc_amd import decoder as D

X, G, O, W, B, DW, DB, WS, S, T, L0, K, V, KS, VS = (0x100000000 * (i + 1) for i in range(15))


def _reason(rc):
    return igc.REASONS[rc]


# --------------------------------------------------------------- layer norm
def _ln(**kw):
    f = dict(n0=2, n1=30, n2=7, c=96, x=X, x0=30 * 7 * 96, x1=7 * 96, x2=96, g=G, g0=30 * 7 * 96,
             g1=7 * 96, g2=96, o=O, o0=30 * 7 * 96, o1=7 * 96, o2=96, w=W, b=B, dw=0, db=0,
             eps=1e-5, dtype=0, ws=0, ws_bytes=0)
    f.update(kw)
    return D._LN.pack(*f.values())


LN_BAD = [
    (dict(dtype=2), "dtype"), (dict(dtype=-1), "dtype"), (dict(n0=-1), "shape"),
    (dict(c=0), "shape"), (dict(c=-5), "shape"), (dict(c=16385), "size_limit"),
    (dict(n0=1 << 31), "size_limit"), (dict(n0=1 << 20, n1=1 << 20), "size_limit"),
    (dict(n0=1 << 30, n1=1 << 30, n2=1 << 30), "size_limit"),
    # 512 threads a row: 2^23 rows of 16384 are 2^32 threads
    (dict(n0=1 << 23, n1=1, n2=1, c=16384, x0=0, o0=16384), "size_limit"),
    (dict(eps=-1e-9), "scale"), (dict(eps=math.nan), "scale"), (dict(eps=1e39), "scale"),
    (dict(x=0), "null_pointer"), (dict(o=0), "null_pointer"),
    (dict(x=X + 1), "alignment"), (dict(w=W + 2), "alignment"), (dict(b=B + 1), "alignment"),
    (dict(x2=-96), "stride"), (dict(x0=1 << 40), "size_limit"),
    (dict(n0=1 << 18, n1=1, x0=(1 << 39) + 2), "size_limit"),   # 2^57 elements
    (dict(o=X + 2), "overlap"), (dict(o2=95), "overlap"), (dict(o1=96), "overlap"),
    (dict(o=W), "overlap"), (dict(o=B - 64), "overlap"),
]


@pytest.mark.parametrize("kw,reason", LN_BAD)
def test_layer_norm_refusals(kw, reason):
    L = igc.lib()
    packed = _ln(**kw)
    assert _reason(L.layer_norm_fwd_check(packed)) == reason
    assert L.layer_norm_fwd(packed, None) == 0


def test_layer_norm_accepted():
    L = igc.lib()
    for kw in (dict(), dict(o=X), dict(w=0, b=0), dict(x=X + 2, o=O + 6), dict(x0=0),
               dict(n0=0, x=0, o=0, g=0), dict(x2=0), dict(c=1, x2=1, o2=3, x1=7, o1=30),
               dict(n0=1, x0=-4, o0=-4), dict(dtype=1, eps=0.0)):
        assert L.layer_norm_fwd_check(_ln(**kw)) == 0, kw
    for kw in (dict(), dict(o=G), dict(dw=DW, db=DB), dict(dw=DW), dict(b=0, db=DB)):
        assert L.layer_norm_bwd_check(_ln(**kw)) == 0, kw


@pytest.mark.parametrize("kw,reason", [
    (dict(g=0), "null_pointer"), (dict(g=G + 1), "alignment"), (dict(o=X), "overlap"),
    (dict(o=G + 2), "overlap"), (dict(dw=DW + 2), "alignment"), (dict(dw=DW, db=DW + 4), "overlap"),
    (dict(dw=X), "overlap"), (dict(db=G + 64), "overlap"), (dict(db=O), "overlap"),
    (dict(dw=W, db=DB), "overlap"),
    (dict(dw=DW, ws=WS, ws_bytes=16), "workspace"), (dict(dw=DW, ws=WS + 8, ws_bytes=1 << 30), "alignment"),
    (dict(dw=DW, ws=X, ws_bytes=1 << 30), "overlap"), (dict(dw=DW, ws=O, ws_bytes=1 << 30), "overlap"),
    (dict(dw=DW, ws=DW, ws_bytes=1 << 30), "overlap"), (dict(dw=DW, ws=W - 256, ws_bytes=1 << 30), "overlap"),
])
def test_layer_norm_gradient_refusals(kw, reason):
    L = igc.lib()
    packed = _ln(**kw)
    assert _reason(L.layer_norm_bwd_check(packed)) == reason
    assert L.layer_norm_bwd(packed, None) == 0


def test_layer_norm_workspace():
    L = igc.lib()
    assert L.layer_norm_bwd_workspace_bytes(_ln()) == 0
    need = L.layer_norm_bwd_workspace_bytes(_ln(dw=DW))
    assert need > 0 and need % (2 * 96 * 4) == 0
    assert L.layer_norm_bwd_workspace_bytes(_ln(db=DB)) == need
    assert L.layer_norm_bwd_workspace_bytes(_ln(dw=DW, c=0)) == 0
    assert L.layer_norm_bwd_workspace_bytes(_ln(dw=DW, n0=0)) == 0
    assert L.layer_norm_bwd_check(_ln(dw=DW, ws=WS, ws_bytes=need)) == 0
    assert _reason(L.layer_norm_bwd_check(_ln(dw=DW, ws=WS, ws_bytes=need - 1))) == "workspace"
    assert igc.layer_norm_bwd_workspace_bytes((2, 30, 7, 96), torch.bfloat16) == need
    assert igc.layer_norm_bwd_workspace_bytes((420, 96), torch.float16) == need
    assert igc.layer_norm_bwd_workspace_bytes((420, 96), torch.float32) == 0


# ------------------------------------------------------------ rows in 8 bits
def _quant(**kw):
    f = dict(n0=2, n1=30, n2=7, c=100, x=X, x0=30 * 7 * 100, x1=7 * 100, x2=100, q=O,
             q0=30 * 7 * 112, q1=7 * 112, q2=112, s=S, dtype=0)
    f.update(kw)
    return D._QUANT.pack(*f.values())


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "dtype"), (dict(n1=-1), "shape"), (dict(c=0), "shape"),
    (dict(c=131072), "size_limit"), (dict(n0=1 << 31), "size_limit"),
    (dict(n0=1 << 16, n1=1 << 16), "size_limit"), (dict(x=0), "null_pointer"),
    (dict(q=0), "null_pointer"), (dict(s=0), "null_pointer"), (dict(x=X + 1), "alignment"),
    (dict(q=O + 8), "alignment"), (dict(q2=104), "alignment"), (dict(s=S + 2), "alignment"),
    (dict(x1=-1), "stride"), (dict(q2=96, c=97), "overlap"), (dict(q=X), "overlap"),
    (dict(s=X + 400), "overlap"), (dict(s=O), "overlap"),
])
def test_quantize_rows_refusals(kw, reason):
    L = igc.lib()
    packed = _quant(**kw)
    assert _reason(L.quantize_rows_check(packed)) == reason
    assert L.quantize_rows(packed, None) == 0


def test_quantize_rows_accepted():
    L = igc.lib()
    for kw in (dict(), dict(x=X + 2), dict(x0=0), dict(n0=0, x=0, q=0, s=0),
               dict(c=131071, n0=1, n1=1, n2=1)):
        assert L.quantize_rows_check(_quant(**kw)) == 0, kw


# ------------------------------------------------------------ their product
def _lin(**kw):
    f = dict(m=70, n=50, k=100, x=X, x_p=112, w=W, w_p=112, xs=S, ws=S + (1 << 20), b=B, y=O, y_p=50,
             dtype=0)
    f.update(kw)
    return D._LINEAR.pack(*f.values())


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "dtype"), (dict(m=-1), "shape"), (dict(k=-1), "shape"),
    (dict(k=131072), "size_limit"), (dict(m=1 << 31), "size_limit"),
    (dict(x=0), "null_pointer"), (dict(w=0), "null_pointer"), (dict(y=0), "null_pointer"),
    (dict(xs=0), "null_pointer"), (dict(ws=0), "null_pointer"),
    (dict(x=X + 8), "alignment"), (dict(x_p=104), "alignment"), (dict(w_p=100), "alignment"),
    (dict(y=O + 1), "alignment"), (dict(xs=S + 1), "alignment"), (dict(b=B + 2), "alignment"),
    (dict(x_p=-16), "stride"), (dict(y_p=49), "stride"), (dict(w_p=1 << 22), "size_limit"),
    (dict(y_p=1 << 40), "size_limit"),
    (dict(m=(1 << 31) - 1, n=1 << 20, x_p=0, y_p=1 << 20, y=1 << 60), "size_limit"),
    (dict(y=X), "overlap"), (dict(y=W + 64), "overlap"), (dict(y=S), "overlap"),
    (dict(y=B - 2), "overlap"),
])
def test_linear_refusals(kw, reason):
    L = igc.lib()
    packed = _lin(**kw)
    assert _reason(L.linear_i8_check(packed)) == reason
    assert L.linear_i8(packed, None) == 0


def test_linear_accepted():
    L = igc.lib()
    for kw in (dict(), dict(b=0), dict(x_p=0), dict(w_p=0), dict(y=O + 2, y_p=51),
               dict(m=0, x=0, y=0, xs=0), dict(n=0, w=0, y=0, ws=0), dict(k=0, x=0, w=0),
               dict(m=1, y_p=0, x_p=16), dict(k=131071, x_p=131072, w_p=131072)):
        assert L.linear_i8_check(_lin(**kw)) == 0, kw


# ------------------------------------------------------------------ the cache
def _cache(**kw):
    f = dict(k=K, v=V, ks=KS, vs=VS, pages=20, page=32, heads=6, d=72)
    f.update({n: v for n, v in kw.items() if n in f})
    return D._CACHE.pack(*f.values())


def _io(**kw):
    h, d = kw.get("heads", 6), kw.get("d", 72)
    f = dict(b=3, t=50, x=X, x_b=50 * h * d, x_t=h * d, x_h=d, y=G, y_b=50 * h * d, y_t=h * d, y_h=d,
             table=T, stride=9, entries=9, start=S, lens=L0, dtype=0)
    f.update({n: v for n, v in kw.items() if n in f})
    return _cache(**kw) + D._IO.pack(*f.values())


def _pair(h, delta, t=None, b=None):
    """k and v of the same strides, v `delta` elements behind k."""
    t = t or 6 * h
    b = b or 50 * t
    return dict(x_h=h, x_t=t, x_b=b, y_h=h, y_t=t, y_b=b, y=X + 2 * delta)


CACHE_BAD = [
    (dict(page=8), "shape"), (dict(page=24), "shape"), (dict(page=2048), "shape"),
    (dict(pages=-1), "shape"), (dict(heads=-1), "shape"), (dict(d=0), "head_dim"),
    (dict(d=136), "head_dim"), (dict(d=20), "head_dim"), (dict(pages=1 << 31), "size_limit"),
    (dict(pages=(1 << 31) - 1, page=1024), "size_limit"), (dict(k=0), "null_pointer"),
    (dict(vs=0), "null_pointer"), (dict(k=K + 8), "alignment"), (dict(ks=KS + 4), "alignment"),
    (dict(v=K), "overlap"), (dict(vs=KS), "overlap"), (dict(ks=K + 256), "overlap"),
]
IO_BAD = CACHE_BAD + [
    (dict(dtype=2), "dtype"), (dict(b=-1), "shape"), (dict(t=-1), "shape"),
    (dict(entries=-1), "shape"), (dict(b=1 << 31), "size_limit"),
    (dict(b=1 << 30, t=1 << 30), "size_limit"), (dict(b=1 << 20, t=1 << 16), "size_limit"),
    (dict(x=0), "null_pointer"), (dict(y=0), "null_pointer"), (dict(table=0), "null_pointer"),
    (dict(start=0), "null_pointer"), (dict(x=X + 8), "alignment"), (dict(x_t=6 * 72 + 4), "alignment"),
    (dict(table=T + 2), "alignment"), (dict(start=S + 1), "alignment"), (dict(lens=L0 + 2), "alignment"),
    (dict(x_h=-72), "stride"), (dict(stride=-1), "stride"), (dict(stride=1 << 40), "stride"),
    (dict(x=K), "overlap"), (dict(y=KS), "overlap"),
]


@pytest.mark.parametrize("kw,reason", IO_BAD)
@pytest.mark.parametrize("name", ["kv_cache_write", "kv_cache_read"])
def test_cache_refusals(name, kw, reason):
    L = igc.lib()
    packed = _io(**kw)
    assert _reason(getattr(L, name + "_check")(packed)) == reason
    assert getattr(L, name)(packed, None) == 0


def test_cache_refusals_of_one_direction():
    """What a call writes may not be what it reads; outputs may not repeat."""
    L = igc.lib()
    for kw in (dict(table=K + 64), dict(start=VS), dict(lens=V)):
        assert _reason(L.kv_cache_write_check(_io(**kw))) == "overlap"
        assert L.kv_cache_read_check(_io(**kw)) == 0
    for kw in (dict(table=X), dict(start=G + 64), dict(lens=X + 64), dict(x_t=0), dict(y_h=64),
               dict(y=X), dict(y=X + 16), dict(y=X + 6 * 72 * 2), dict(y=X + 144),
               _pair(h=144, delta=64), _pair(h=144, delta=80), _pair(h=72, t=864, delta=424),
               _pair(h=72, t=864, delta=864), _pair(h=72, t=432, b=43200, delta=21608),
               dict(_pair(h=72, t=864, delta=432), y_h=144)):
        assert _reason(L.kv_cache_read_check(_io(**kw))) == "overlap", kw
        assert L.kv_cache_write_check(_io(**kw)) == 0
    # halves of heads' rows, of tokens and of sequences; either first
    for kw in (_pair(h=144, delta=72), _pair(h=72, t=864, delta=432), _pair(h=72, t=880, delta=440),
               _pair(h=72, t=432, b=43200, delta=21600), _pair(h=3600, t=72, b=43200, delta=21600),
               dict(_pair(h=144, delta=72), x=X + 144, y=X), dict(y=X + 3 * 50 * 6 * 72 * 2)):
        assert L.kv_cache_read_check(_io(**kw)) == 0, kw


def test_cache_accepted():
    L = igc.lib()
    for name in ("kv_cache_write_check", "kv_cache_read_check"):
        check = getattr(L, name)
        for kw in (dict(), dict(lens=0), dict(stride=0), dict(b=0, x=0, y=0, table=0, start=0),
                   dict(t=0, x=0, y=0), dict(heads=0, x=0, y=0, k=0, v=0, ks=0, vs=0),
                   dict(pages=0, k=0, v=0, ks=0, vs=0), dict(entries=0, table=0), dict(page=1024)):
            assert check(_io(**kw)) == 0, (name, kw)


# ------------------------------------------------------- attention over it
def _attn(**kw):
    tq, hq, d = kw.get("tq", 3), kw.get("hq", 12), kw.get("d", 72)
    f = dict(b=3, tq=tq, hq=hq, q=X, q_b=tq * hq * d, q_t=hq * d, q_h=d, o=O, o_b=tq * hq * d,
             o_t=hq * d, o_h=d, lse=0, table=T, stride=50, entries=50, lens=L0, causal=1, scale=0.1,
             dtype=0, ws=0, ws_bytes=0)
    f.update({n: v for n, v in kw.items() if n in f})
    return _cache(**kw) + D._CATTN.pack(*f.values())


@pytest.mark.parametrize("kw,reason", CACHE_BAD + [
    (dict(dtype=2), "dtype"), (dict(b=-1), "shape"),
    (dict(entries=-1), "shape"), (dict(heads=5), "groups"), (dict(heads=0), "groups"),
    (dict(scale=0.0), "scale"), (dict(scale=math.nan), "scale"), (dict(scale=1e300), "scale"),
    (dict(scale=1e-40), "scale"), (dict(b=1 << 31), "size_limit"),
    (dict(b=1 << 29), "size_limit"), (dict(tq=1 << 30), "size_limit"),
    (dict(entries=1 << 26), "size_limit"), (dict(b=1 << 21), "size_limit"),
    (dict(q_t=1 << 23), "size_limit"), (dict(q_h=1 << 23), "size_limit"),
    (dict(hq=1536, q_h=(1 << 23) - 8), "size_limit"),
    (dict(q=0), "null_pointer"), (dict(o=0), "null_pointer"), (dict(lens=0), "null_pointer"),
    (dict(table=0), "null_pointer"), (dict(q=X + 8), "alignment"), (dict(lse=S + 2), "alignment"),
    (dict(lens=L0 + 1), "alignment"), (dict(q_b=-72), "stride"), (dict(stride=-2), "stride"),
    (dict(o=X), "overlap"), (dict(o=K), "overlap"), (dict(o_h=64), "overlap"),
    (dict(lse=O), "overlap"), (dict(lse=VS), "overlap"), (dict(o=T), "overlap"),
    (dict(lse=L0), "overlap"), (dict(ws=WS, ws_bytes=16), "workspace"),
    (dict(ws=WS + 8, ws_bytes=1 << 30), "alignment"), (dict(ws=O, ws_bytes=1 << 30), "overlap"),
    (dict(ws=V, ws_bytes=1 << 30), "overlap"), (dict(ws=X, ws_bytes=1 << 30), "overlap"),
])
def test_cache_attention_refusals(kw, reason):
    L = igc.lib()
    packed = _attn(**kw)
    assert _reason(L.cache_attn_fwd_check(packed)) == reason
    assert L.cache_attn_fwd(packed, None) == 0


def test_cache_attention_accepted():
    L = igc.lib()
    for kw in (dict(), dict(lse=S), dict(q_b=0), dict(stride=0), dict(causal=0), dict(entries=0, table=0),
               dict(b=0, q=0, o=0, lens=0, table=0), dict(tq=0, q=0, o=0, lens=0),
               dict(hq=0, q=0, o=0, lens=0), dict(pages=0, k=0, v=0, ks=0, vs=0), dict(d=8),
               dict(entries=(1 << 26) - 129)):
        assert L.cache_attn_fwd_check(_attn(**kw)) == 0, kw


def test_cache_attention_workspace():
    L = igc.lib()
    assert L.cache_attn_fwd_workspace_bytes(_attn(entries=20)) == 0      # 640 tokens: no split
    need = L.cache_attn_fwd_workspace_bytes(_attn())
    assert need > 0 and need % 4 == 0
    assert L.cache_attn_fwd_check(_attn(ws=WS, ws_bytes=need)) == 0
    assert _reason(L.cache_attn_fwd_check(_attn(ws=WS, ws_bytes=need - 4))) == "workspace"
    assert L.cache_attn_fwd_workspace_bytes(_attn(dtype=5)) == 0
    # many sequences fill the card without a split
    assert L.cache_attn_fwd_workspace_bytes(_attn(b=400)) == 0


def test_null_arguments():
    L = igc.lib()
    for name in ("layer_norm_fwd", "layer_norm_bwd", "quantize_rows", "linear_i8", "kv_cache_write",
                 "kv_cache_read", "cache_attn_fwd"):
        assert _reason(getattr(L, name + "_check")(None)) == "null_pointer"
        assert getattr(L, name)(None, None) == 0
    assert L.layer_norm_bwd_workspace_bytes(None) == 0
    assert L.cache_attn_fwd_workspace_bytes(None) == 0


def test_structs_are_the_headers(tmp_path):
    names = ("igc_layer_norm", "igc_quantize_rows", "igc_linear_i8", "igc_kv_cache", "igc_kv_io",
             "igc_cache_attn")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "igemm_decoder.h"\nint main(void) {\n' + "".join(
        f'    printf("%zu\\n", sizeof({n}));\n' for n in names) + "    return 0;\n}\n")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", include, str(src), "-o",
                    str(tmp_path / "sizes")], check=True)
    sizes = [int(x) for x in subprocess.run([str(tmp_path / "sizes")], check=True,
                                            capture_output=True, text=True).stdout.split()]
    c = D._CACHE.size
    assert sizes == [D._LN.size, D._QUANT.size, D._LINEAR.size, c, c + D._IO.size, c + D._CATTN.size]
    assert struct.calcsize("P") == 8


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q = torch.zeros(4, 32, dtype=torch.int8)
    for call in (lambda: igc.layer_norm(x), lambda: igc.layer_norm_bwd(x, x),
                 lambda: igc.quantize_rows(x), lambda: igc.linear_i8(q, x[0], q, x[0]),
                 lambda: igc.KVCache.empty(2, 16, 2, 32, device="cpu"),
                 lambda: igc.kv_cache_read(None, x, x, 1),
                 lambda: igc.kv_cache_write(None, x, x, x, x),
                 lambda: igc.cache_attention(x, None, x, x)):
        with pytest.raises(igc.InvalidArgument):
            call()
