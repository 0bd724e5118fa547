"""Attention gates and host arithmetic at the limits of their types (CPU only:
no call here reaches a kernel launch)."""
import threading

import pytest

import implicit_gemm_nhwc_amd as igc
from test_attn_host import _grad, _reason


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
