"""The norm gradient's workgroups loop over rounds of lane groups where there
are more than run at once: such calls against the float64 oracle (GPU), and
the plan behind them, pinned to the library by its workspace (CPU).  Bounds as
in test_gpu_qk_norm.py, but for the weight gradient the chains of its sum: four
heads a round in a lane, the workgroup's lane groups in order, every 64th
workgroup in order and a tree over 64, one rounding each, after fp32 roundings
of a row's norm (d + 16 of them) and of a turned pair (at most |a| + |b|, which
2 max |g| bounds).  A round counted twice or left out is far outside."""
import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from test_attn_host import _norm, DW
from oracle import attention as oracle
from test_gpu_qk_norm import BF, DEV, HF, _check, _inputs, _rnd

MOST = 3 * 256      # workgroups of both parts together


def _lanes(d):
    return 4 if d <= 32 else 8 if d <= 64 else 16


def plan(b, tq, tk, hq, hk, d):
    """(tiles, workgroups) of the two parts, and which rule gave the rounds."""
    tiles = [-(-b * t * -(-h // 4) // (256 // _lanes(d))) for t, h in ((tq, hq), (tk, hk))]
    rounds, rule = -(-sum(tiles) // MOST), "even"
    if sum(-(-n // rounds) for n in tiles) > MOST:
        rounds, rule = -(-sum(tiles) // (MOST - 1)), "two parts round up"
    return tiles, [-(-n // rounds) for n in tiles], rounds, rule


CASES = [
    # dt, b, tq, tk, hq, hk, d, rot, positions, interleaved, weights
    (BF, 8, 3137, 333, 8, 8, 64, 64, False, False, True),     # uneven parts, three rounds
    (HF, 1, 24608, 24544, 4, 4, 64, 32, True, False, True),   # 769 and 767 tiles
    (HF, 3, 5000, 4099, 9, 3, 40, 40, True, False, True),     # 20-value halves, a head over fours
    (BF, 2, 12345, 77, 5, 1, 80, 40, False, True, True),      # pairs, part of a head
    (BF, 4, 6007, 1, 10, 2, 24, 24, False, False, False),     # halves not of whole chunks, no weight
    (HF, 2, 12289, 3, 4, 4, 128, 128, True, False, True),     # 1537 tiles and one
    (BF, 1, 12272, 16, 4, 1, 128, 0, False, False, True),     # 767 and 1: a single round, full
    (BF, 1, 12288, 16, 4, 1, 128, 0, False, False, True),     # 768 and 1: two
]


def test_cases_take_rounds():
    rounds = [plan(*c[1:7])[2] for c in CASES]
    assert sorted(set(rounds)) == [1, 2, 3] or set(rounds) > {1, 2, 3}
    assert {plan(*c[1:7])[3] for c in CASES} == {"even", "two parts round up"}
    for c in CASES:
        tiles, groups, n, _ = plan(*c[1:7])
        assert sum(groups) <= MOST and all(g * n >= t for g, t in zip(groups, tiles))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_plan_is_the_librarys(case):
    _, b, tq, tk, hq, hk, d = case[:7]
    groups = plan(b, tq, tk, hq, hk, d)[1]
    packed = _norm(q=dict(b=b, t=tq, h=hq, dw=DW), k=dict(b=b, t=tk, h=hk, dw=DW + 4096), d=d, rot=0)
    assert igc.lib().qk_norm_rope_bwd_workspace_bytes(packed) == 4 * sum(groups) * _lanes(d) * 8


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}.{c[7]}")
def test_rounds_against_the_oracle(case):
    print(f"norm rounds {case}", flush=True)
    dt = case[0]
    q, k, gq, gk, kw, one = _inputs(case)
    yq, yk = igc.qk_norm_rope(q, k, **kw)
    dq, dk, dqw, dkw = igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    _check(dt, q, yq, one[0], gq, dq, dqw)
    _check(dt, k, yk, one[1], gk, dk, dkw)
    _, groups, rounds, _ = plan(*case[1:7])
    for x, g, dw, w, blocks in ((q, gq, dqw, one[0], groups[0]), (k, gk, dkw, one[1], groups[1])):
        r = oracle.qk_norm_rope(x, grad=g, **w)
        x64 = x.cpu().double()
        xh = x64 * (x64.square().mean(-1, keepdim=True) + w["eps"]) ** -0.5
        pair = (2 * r["g"].abs().amax(-1, keepdim=True) * xh.abs()).sum((0, 1, 2))
        chain = 4 * rounds + 256 // _lanes(case[6]) + -(-blocks // 64) + 6 + case[6] + 16
        far = (dw.cpu().double() - r["dweight"]).abs()
        bound = chain * 2.0 ** -24 * r["dweight_abs"] + 2.0 ** -23 * pair
        print(f"    dweight: {float((far / bound).max()):.3f} of the bound", flush=True)
        assert (far <= bound).all()
    alone = {n: (None if n.startswith("k_") else v) for n, v in kw.items()}
    again = igc.qk_norm_rope_bwd(gq, None, q, **alone)
    assert torch.equal(again[0], dq)
    _check(dt, q, yq, one[0], gq, again[0], again[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("weight", [False, True])
def test_gradients_of_extreme_rows(dt, weight):
    """Zero rows (eps alone), the largest values, subnormal ones."""
    x = _rnd(1, 6, 2, 64, seed=3).to(dt)
    x[0, 0] = 0
    x[0, 1] = torch.finfo(dt).max / 64 if dt == HF else 1e17
    x[0, 2] *= 1e-6
    x[0, 3, 0, :63] = 0                       # one value alone carries the row
    x[0, 4, 1] = x[0, 4, 1].abs().neg()
    x = x.to(DEV)
    gy = _rnd(1, 6, 2, 64, seed=4).to(dt).to(DEV)
    w = (1 + 0.3 * _rnd(64, seed=5)).to(DEV) if weight else None
    kw = dict(eps=1e-6)
    y = igc.qk_norm_rope(x, q_weight=w, **kw)
    dx, _, dw, _ = igc.qk_norm_rope_bwd(gy, None, x, q_weight=w, **kw)
    _check(dt, x, y, dict(weight=w, **kw), gy, dx, dw)
