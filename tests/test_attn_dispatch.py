"""Every form of the attention kernels that the plans choose between is
compared with the float64 oracle: the plans' rules, mirrored here and pinned to
the library by its workspace sizes (CPU), say which form a case reaches; the
cases below are those that the ordinary ones leave out (GPU).

The bounds are those of test_gpu_attention.py, over some entries of the batch.
"""
import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from oracle import attention as oracle
from test_gpu_attention import BF, CASES, HF, _check, _make, _say

CUS, FEW, TILE = 256, 128, 64


def _ceil(a, b):
    return -(-a // b)


def _padded(d):
    return next(x for x in (32, 64, 96, 128) if d <= x)


def _short_tiles(bh, rows, slots):
    blocks = _ceil(rows, 32)
    rounds = _ceil(blocks, max(1, slots // bh) * 4)
    return max(1, _ceil(blocks, max(1, rounds) * 4))


def forward(dt, b, tq, tk, hq, hk, d, mask):
    """(form, join, workspace bytes) of a forward call."""
    bh, rows = b * hk, tq * hq // hk
    if rows > 32 and tk <= FEW:
        return ("few keys", dt, _padded(d)), None, 0
    token = rows <= 32
    step = 256 if token else TILE
    groups = bh if token else bh * _ceil(rows, 128)
    steps = _ceil(tk, step)
    n = 1
    if not token:
        n = min(2 * CUS // groups, steps // 3)
    elif steps > 4:
        n = CUS // groups
        if _ceil(steps, max(1, n)) > 16:
            n = 4 * CUS // groups
    per = _ceil(max(1, steps), max(1, n))
    splits = _ceil(max(1, steps), per)
    join = None if splits == 1 else ("few splits" if splits <= 8 else "many splits", dt)
    form = ("token", dt, _padded(d)) if token else (
        "rows", dt, _padded(d), "masked" if mask in ("keys", "both") else "plain")
    return form, join, 0 if splits == 1 else 4 * splits * bh * rows * (d + 2)


def backward(dt, b, tq, tk, hq, hk, d, mask):
    """(forms, workspace bytes) of a gradient call."""
    bh, rows = b * hk, tq * hq // hk
    row64, key64, key32 = _ceil(rows, 64), _ceil(tk, 64), _ceil(tk, 32)
    pad = row64 * 64
    bound = max(1, min(_ceil(4 * CUS, bh), pad // 16, 256))

    def split(want, least, groups, tiles):
        n = max(1, min(want // groups, tiles // least))
        per = _ceil(max(1, tiles), n)
        return _ceil(max(1, tiles), per), per

    waves = max(1, min(4, key32))
    nkv, per = split(CUS, 2, bh * _ceil(key32, waves), row64)
    walk = _ceil(min(per * 64, rows), 64)
    groups = 1 if d <= 96 and walk <= 8 else 2
    nq, _ = split(2 * CUS, 3, bh * _ceil(rows, 128), key64)
    forms = {("dk dv", dt, _padded(d), waves, groups)}
    if tk <= FEW:
        nq = 1
        bound = 4 * _short_tiles(bh, pad, (2 if d <= 64 else 1) * CUS)
        forms.add(("few keys rows", dt, _padded(d)))
    else:
        forms.update({("dq", dt, _padded(d)), ("row pass", dt)})
    if nkv > 1:
        forms.add(("join dk dv", dt))
    if nq > 1:
        forms.add(("join dq", dt))
    part = max(2 * nkv * bh * tk * d if nkv > 1 else 0, nq * bh * rows * d if nq > 1 else 0)
    return forms, 4 * (part + 2 * bh * pad + (2 * bh * bound if dt == HF else 0))


# Walks of more than eight row tiles in one workgroup: two waves a key block,
# for each number of key blocks a workgroup, and groups that do not divide 64.
LONG_WALKS = [
    (dt, b, tq, tk, g * hk, hk, d, mask, layout)
    for dt in (BF, HF)
    for d, b, hk in ((24, 33, 4), (64, 19, 8), (80, 66, 2), (128, 33, 4))
    for tk, tq, g, mask, layout in ((31, 640, 1, "both", "dense"), (64, 201, 3, "keys", "fused"),
                                    (77, 577, 1, "both", "heads"), (125, 300, 2, "lens", "padded"))
] + [
    (BF, 8, 1100, 300, 10, 10, 40, "both", "fused"),     # three key tiles, 18 row tiles
    (HF, 5, 333, 260, 40, 10, 88, "lens", "dense"),
    (HF, 8, 1100, 300, 10, 10, 128, "keys", "fused"),
    (BF, 1, 2200, 1000, 8, 8, 64, "keys", "dense"),
]
# the other forms that the ordinary cases leave out
OTHERS = [
    (BF, 2, 70, 300, 2, 2, 32, "both", "dense"), (HF, 2, 70, 300, 2, 2, 32, "lens", "dense"),
    (HF, 2, 70, 300, 2, 2, 32, "both", "dense"), (HF, 2, 90, 400, 2, 2, 64, "both", "fused"),
    (BF, 2, 90, 400, 2, 2, 88, "none", "fused"), (BF, 2, 90, 400, 2, 2, 96, "keys", "heads"),
    (HF, 2, 90, 400, 2, 2, 96, "both", "heads"), (HF, 2, 90, 400, 2, 2, 128, "none", "heads"),
    (BF, 2, 90, 400, 2, 2, 128, "none", "dense"),
    (BF, 2, 1, 300, 2, 2, 32, "both", "dense"), (BF, 2, 3, 300, 4, 2, 96, "both", "dense"),
    (BF, 2, 3, 300, 4, 2, 128, "both", "dense"), (HF, 2, 3, 300, 4, 2, 64, "both", "dense"),
    (BF, 2, 90, 40, 2, 2, 96, "both", "dense"), (HF, 2, 90, 90, 4, 2, 32, "both", "dense"),
    (BF, 1, 2, 9000, 4, 2, 128, "keys", "dense"), (HF, 1, 2, 9000, 4, 2, 40, "both", "dense"),
    (HF, 1, 40, 9000, 4, 2, 64, "both", "dense"), (BF, 1, 200, 1500, 2, 1, 64, "none", "dense"),
    (BF, 1, 2, 2000, 64, 32, 64, "none", "dense"), (HF, 1, 2, 2000, 64, 32, 64, "both", "dense"),
    (BF, 2, 70, 300, 2, 2, 32, "none", "dense"),
    (BF, 3, 90, 77, 2, 2, 24, "both", "dense"), (BF, 3, 45, 30, 6, 2, 64, "keys", "fused"),
    (BF, 3, 90, 31, 2, 2, 80, "both", "dense"), (BF, 3, 90, 95, 2, 2, 88, "lens", "padded"),
    (HF, 3, 90, 9, 2, 2, 32, "both", "dense"), (HF, 3, 90, 50, 2, 2, 24, "keys", "heads"),
    (HF, 3, 90, 32, 2, 2, 64, "both", "dense"), (HF, 3, 45, 64, 6, 2, 56, "keys", "fused"),
    (HF, 3, 90, 33, 2, 2, 72, "both", "dense"), (HF, 3, 90, 96, 2, 2, 96, "lens", "dense"),
]


def _all_forms():
    forms, joins = set(), set()
    dims = (32, 64, 96, 128)
    for dt in (BF, HF):
        joins.update({("few splits", dt), ("many splits", dt)})
        forms.update({("row pass", dt), ("join dk dv", dt), ("join dq", dt)})
        for d in dims:
            forms.update({("token", dt, d), ("few keys", dt, d), ("rows", dt, d, "masked"),
                          ("rows", dt, d, "plain"), ("few keys rows", dt, d), ("dq", dt, d)})
            for waves in (1, 2, 3, 4):
                forms.update(("dk dv", dt, d, waves, n) for n in ((2,) if d == 128 else (1, 2)))
    return forms | joins


def test_cases_reach_every_form():
    seen = set()
    for case in CASES + LONG_WALKS + OTHERS:
        form, join, _ = forward(*case[:8])
        seen |= {form, join} | backward(*case[:8])[0]
    seen.discard(None)
    assert _all_forms() - seen == set()
    assert seen <= _all_forms()
    for case in LONG_WALKS:
        assert {f[4] for f in backward(*case[:8])[0] if f[0] == "dk dv"} == {2}, case


@pytest.mark.parametrize("case", CASES + LONG_WALKS + OTHERS, ids=str)
def test_plans_are_the_librarys(case):
    """Workspaces hold the number of splits, of padded rows and of bounds."""
    dt, b, tq, tk, hq, hk, d, mask, _ = case
    q, k = (b, tq, hq, d), (b, tk, hk, d)
    assert igc.cross_attn_fwd_workspace_bytes(q, k, dt) == forward(*case[:8])[2]
    assert igc.cross_attn_bwd_workspace_bytes(q, k, dt) == backward(*case[:8])[1]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LONG_WALKS + OTHERS,
                         ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}")
def test_form_against_the_oracle(case):
    dt, b, tq, tk, hq, hk, d, mask, layout = case
    _say(f"form {case}")
    q, k, v, go, lens, km = _make(*case, seed=tq * 5 + tk)
    kw = dict(kv_lens=lens, key_mask=km)
    out, lse = igc.cross_attention(q, k, v, return_lse=True, **kw)
    grads = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    top = dict(max_go=float(go.norm(dim=-1).max()), max_v=float(v.norm(dim=-1).max()))
    # the first entries (full, no keys, no unmasked keys) and the last one
    for i in sorted({0, 1, 2, b - 1} & set(range(b))):
        def cut(*ts):
            return [None if t is None else t[i:i + 1] for t in ts]

        one = dict(zip(("kv_lens", "key_mask"), cut(lens, km)))
        qi, ki, vi, gi = cut(q, k, v, go)
        r = oracle.cross_attention(qi, ki, vi, dout=gi, **one)
        _check(r, dt, tk, *cut(out, lse), grads=cut(*grads), **top)
    again = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    with igc.using_library(igc.POISON_LIB_PATH):
        out2, lse2 = igc.cross_attention(q, k, v, return_lse=True, **kw)
        poisoned = igc.cross_attention_bwd(go, q, k, v, out, lse, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y, z in zip(grads, again, poisoned):
        assert torch.equal(x, y) and torch.equal(x, z)
