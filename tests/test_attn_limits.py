"""Attention gates and host arithmetic at the limits of their types (CPU only:
no call here reaches a kernel launch)."""
import threading

import pytest

import implicit_gemm_nhwc_amd as igc
from test_attn_host import _attn, _grad, _norm, _reason


def _ends(f, *args):
    """f's result, from a thread of its own, so that a call that does not end
    fails its test instead of hanging the run."""
    got = []
    t = threading.Thread(target=lambda: got.append(f(*args)), daemon=True)
    t.start()
    t.join(20)
    assert got, "the call does not return"
    return got[0]


@pytest.mark.parametrize("hq", [1, 3, 1 << 30, (1 << 30) + 1, (1 << 31) - 1])
def test_groups_of_many_heads(hq):
    """No rows and no keys: nothing is launched, but the group's divisor is
    formed (its shift passes 31 bits above 2^30 heads)."""
    none = dict(data=0)
    packed = _grad(dict(go=none, dq=none, dk=none, dv=none), b=1, tq=0, tk=0, hq=hq, hk=1, lse=0,
                   q_data=0, k_data=0, v_data=0, o_data=0)
    L = igc.lib()
    assert _reason(L.cross_attn_bwd_check(packed)) == "ok"
    assert L.cross_attn_bwd_workspace_bytes(packed) == 0
    assert _ends(L.cross_attn_bwd, packed, None) == 1


# a tensor of which every batch entry is the same (inputs), or small (out)
_SHARED = dict(tq=1, tk=500, hq=1, hk=1, d=8, q_batch=0, k_batch=0, v_batch=0)
FAR = 1 << 60      # above all buffers of the calls


@pytest.mark.parametrize("b,stride,reason", [
    (1 << 30, (1 << 40) - 1, "size_limit"),       # 2^70: passes 64 bits
    ((1 << 24) + 1, 1 << 39, "size_limit"),       # 2^63: a negative product
    ((1 << 25) + 1, 1 << 39, "size_limit"),       # 2^64: the product is 0
    (1 << 20, 1 << 37, "size_limit"),             # 2^57: more than an address space
    (1 << 20, 500, "ok"), (1 << 20, 0, "ok"), (1, (1 << 40) - 1, "ok"),
])
def test_mask_extents(b, stride, reason):
    L = igc.lib()
    packed = _attn(b=b, mask=FAR, mask_stride=stride, **_SHARED)
    assert _reason(L.cross_attn_fwd_check(packed)) == reason
    none = dict(data=0)
    same = dict(batch=0, token=0, head=0)
    packed = _grad(dict(go=same, dq=none, dk=none, dv=none), b=b, mask=FAR, mask_stride=stride,
                   **_SHARED)
    assert _reason(L.cross_attn_bwd_check(packed)) == reason


@pytest.mark.parametrize("b,stride,reason", [
    (1 << 30, (1 << 40) - 1, "size_limit"), ((1 << 24) + 1, 1 << 39, "size_limit"),
    ((1 << 25) + 1, 1 << 39, "size_limit"), (1 << 20, 1 << 37, "size_limit"),
    (1 << 20, 100, "ok"), (1 << 20, 0, "ok"), (1, (1 << 40) - 1, "ok"),
])
def test_position_extents(b, stride, reason):
    L = igc.lib()
    part = dict(b=b, t=1, h=1, x_b=0, g_b=0, o=FAR >> 1, o_b=64, o_t=64, pos=FAR, pos_b=stride)
    none = dict(b=0, x=0, o=0, g=0)
    for packed in (_norm(q=part, k=none), _norm(q=none, k=part)):
        assert _reason(L.qk_norm_rope_fwd_check(packed)) == reason
        assert _reason(L.qk_norm_rope_bwd_check(packed)) == reason


@pytest.mark.parametrize("scale,reason", [
    (3e38, "scale"),       # finite in fp32, but scale * log2(e), which the kernels hold, is not
    (2.36e38, "scale"), (2.35e38, "ok"), (1e-30, "ok"), (9e-31, "scale"),
])
def test_scale_range(scale, reason):
    L = igc.lib()
    assert _reason(L.cross_attn_fwd_check(_attn(scale=scale))) == reason
    assert _reason(L.cross_attn_bwd_check(_grad(scale=scale))) == reason
    if reason != "ok":
        assert L.cross_attn_fwd(_attn(scale=scale), None) == 0


@pytest.mark.parametrize("heads,tq,tk,most", [
    (1, 1, 300, (1 << 23) - 1),     # single tokens: 512 threads a key head
    (16, 1, 1, (1 << 19) - 1),
    (1, 200, 300, (1 << 23) - 1),   # two row tiles of 256 threads
    (1, 64, 77, (1 << 24) - 1),     # few keys
])
def test_threads_of_an_attention_launch(heads, tq, tk, most):
    """A launch of 2^32 threads or more would run only a part of itself."""
    L = igc.lib()
    kw = dict(tq=tq, tk=tk, hq=heads, hk=heads, d=8, k_batch=0, v_batch=0, q_batch=0, o_data=FAR)
    assert _reason(L.cross_attn_fwd_check(_attn(b=most, **kw))) == "ok"
    packed = _attn(b=most + 1, **kw)
    assert _reason(L.cross_attn_fwd_check(packed)) == "size_limit"
    assert L.cross_attn_fwd(packed, None) == 0


@pytest.mark.parametrize("tq,tk,most", [
    (1, 77, (1 << 24) - 1),          # rows in 256 threads, keys in three waves
    (64, 300, (1 << 24) // 3),       # three key tiles of 256 threads
    (1000, 100, (1 << 23) - 1),      # 16 row tiles a head walked: 512 threads
])
def test_threads_of_a_gradient_launch(tq, tk, most):
    L = igc.lib()
    none = dict(data=0)
    views = dict(go=dict(batch=0, token=8, head=8), dq=none, dk=none, dv=none)
    kw = dict(tq=tq, tk=tk, hq=1, hk=1, d=8, k_batch=0, v_batch=0, q_batch=0, o_data=FAR,
              lse=FAR >> 1)
    assert _reason(L.cross_attn_bwd_check(_grad(views, b=most, **kw))) == "ok"
    packed = _grad(views, b=most + 1, **kw)
    assert _reason(L.cross_attn_bwd_check(packed)) == "size_limit"
    assert L.cross_attn_bwd(packed, None) == 0


@pytest.mark.parametrize("d,items", [(8, 64), (64, 32), (128, 16)])
def test_threads_of_a_norm_launch(d, items):
    """items: a workgroup's lane groups (four heads of a token each)."""
    L = igc.lib()
    most = ((1 << 24) - 1) * items
    none = dict(b=0, x=0, o=0, g=0)

    def call(tokens):
        part = dict(b=1, t=tokens, h=4, x_t=4 * d, x_h=d, g_t=4 * d, g_h=d, o_t=4 * d, o_h=d,
                    x=1 << 50, g=1 << 51, o=1 << 52, table=0, rows=0)
        return _norm(q=part, k=none, d=d, rot=0)

    assert _reason(L.qk_norm_rope_fwd_check(call(most))) == "ok"
    assert _reason(L.qk_norm_rope_fwd_check(call(most + 1))) == "size_limit"
    assert L.qk_norm_rope_fwd(call(most + 1), None) == 0
    # backward the workgroups loop
    assert _reason(L.qk_norm_rope_bwd_check(call(most + 1))) == "ok"
