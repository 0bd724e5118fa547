"""Forms of the attention kernels that ordinary small calls do not reach."""
import os
import sys

import pytest
import torch

import implicit_gemm_nhwc_amd as igc

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


def _rnd(dt, *shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dt).to(DEV)


@pytest.mark.parametrize("library", ["ordinary", "poisoned"])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d", [8, 40, 64, 96, 104, 128])
def test_no_query_rows(d, dt, library):
    """The sums over no rows are 0, also where the kernel has staged the keys
    in LDS (D above 96), whose place its sums of row groups take."""
    path = igc.LIB_PATH if library == "ordinary" else igc.POISON_LIB_PATH
    for tk in (1, 31, 64, 130, 777):
        _say(f"no rows {d} {dt} {library} {tk}")
        q = torch.empty(3, 0, 4, d, dtype=dt, device=DEV)
        k, v = _rnd(dt, 3, tk, 2, d, seed=1), _rnd(dt, 3, tk, 2, d, seed=2)
        lens = torch.tensor([tk, 0, tk // 2], dtype=torch.int32, device=DEV)
        with igc.using_library(path):
            for kw in ({}, {"kv_lens": lens}):
                out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
                dq, dk, dv = igc.cross_attention_bwd(q, q, k, v, out, lse, **kw)
                assert dq.shape == q.shape and dk.shape == k.shape
                assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d", [40, 64, 128])
def test_no_query_heads(d, dt):
    """Keys that no head reads: no outputs, and gradients of 0."""
    for b, tq, tk, hk in ((2, 5, 77, 3), (1, 200, 300, 1), (2, 0, 64, 2)):
        _say(f"no heads {d} {dt} {b} {tq} {tk} {hk}")
        q = torch.empty(b, tq, 0, d, dtype=dt, device=DEV)
        k, v = _rnd(dt, b, tk, hk, d, seed=1), _rnd(dt, b, tk, hk, d, seed=2)
        out, lse = igc.cross_attention(q, k, v, return_lse=True)
        assert out.shape == q.shape and lse.shape == (b, 0, tq)
        dq, dk, dv = igc.cross_attention_bwd(q, q, k, v, out, lse)
        assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
        assert dk.shape == k.shape and dv.shape == v.shape


def test_many_single_tokens():
    """As many key heads as one launch takes (2^23 - 16 workgroups of eight
    waves), one key each: the output is its value, and so is dv dout."""
    b = (1 << 19) - 1
    gen = torch.Generator(device=DEV).manual_seed(7)
    q, k, v, go = (torch.randn(b, 1, 16, 8, device=DEV, generator=gen).to(BF) for _ in range(4))
    out, lse = igc.cross_attention(q, k, v, return_lse=True)
    assert torch.equal(out, v)
    s = (q.double() * k.double()).sum(-1).transpose(1, 2) * 8 ** -0.5
    assert ((lse.double() - s).abs() <= 2.0 ** -20 * (1 + s.abs())).all()
    dq, dk, dv = igc.cross_attention_bwd(go, q, k, v, out, lse)
    # p differs from 1 by fp32 roundings, which one rounding of dv may show
    assert ((dv.float() - go.float()).abs() <= 2.0 ** -8 * go.float().abs()).all()
    q2, k2 = (torch.cat([t, t[:1]]) for t in (q, k))
    with pytest.raises(igc.Declined, match="size_limit"):
        igc.cross_attention(q2, k2, k2)
