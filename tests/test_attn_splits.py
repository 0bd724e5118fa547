"""Ranges of split attention launches near 2^31 keys: the device's arithmetic
(csrc/attn_split.hpp) compiled for the host, over the library's own plans (CPU
only), and the kernels themselves on the GPU."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import implicit_gemm_nhwc_amd as igc

CSRC = os.path.join(os.path.dirname(igc.__file__), "csrc")
LONGEST = (1 << 31) - 4097     # the most keys a call may have
DEV = "cuda:0"


@pytest.fixture(scope="module")
def split_end(tmp_path_factory):
    folder = tmp_path_factory.mktemp("split")
    src, lib = folder / "split.cpp", folder / "split.so"
    src.write_text('#include "attn_split.hpp"\n'
                   'extern "C" int end_of(int b, int s, int e) { return igc::split_end(b, s, e); }\n')
    # -ftrapv: a sum that passes int ends the process instead of wrapping
    subprocess.run(["g++", "-O1", "-ftrapv", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    str(src), "-o", str(lib)], check=True, timeout=60)
    return ctypes.CDLL(str(lib)).end_of


# rows of one key head, keys a step of the kernel that takes them
@pytest.mark.parametrize("tq,step", [(1, 256), (40, 64)])
@pytest.mark.parametrize("tk", [LONGEST, (1 << 31) - 5000, (1 << 31) - (1 << 21), (1 << 30) + 77,
                                100003])
@pytest.mark.parametrize("heads", [1, 4])
def test_splits_cover_all_keys(split_end, tq, step, tk, heads):
    need = igc.cross_attn_fwd_workspace_bytes((1, tq, heads, 8), (1, tk, heads, 8),
                                              torch.bfloat16)
    nsplit, rest = divmod(need, heads * tq * (8 + 2) * 4)
    assert nsplit > 1 and rest == 0
    steps = -(-tk // step)
    # the shortest whole number of steps that so many splits need
    split = -(-steps // nsplit) * step
    if tk >= (1 << 31) - 5000:
        assert nsplit * split >= 1 << 31     # the case that an int sum does not hold
    at = 0
    for sp in range(nsplit):
        assert sp * split < tk
        end = split_end(sp * split, split, tk)
        assert end == min(tk, sp * split + split)
        at = end
    assert at == tk


def test_split_ends(split_end):
    top = (1 << 31) - 1
    for begin, split, end in ((0, top, 0), (0, top, 5), (0, 5, 5), (5, 5, 5), (7, 5, 5),
                              (top - 3, 64, top), (top - 64, 64, top), (top, top, top),
                              (0, 64, 65), (64, 64, 65)):
        got = split_end(begin, split, end)
        assert range(begin, got) == range(begin, min(end, begin + split))


@pytest.mark.gpu
@pytest.mark.parametrize("tq", [1, 40])
def test_last_keys_of_the_longest_caches(tq):
    """Only the last 100 of 2^31 - 5000 keys are valid.  One key's row serves
    all (token stride 0), so the probabilities are 1 / 100 each, the output is
    the value's row, and lse = s + log 100."""
    tk, n, d = (1 << 31) - 5000, 100, 8
    print(f"last keys {tq}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(tq)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)

    q, go, k1, v1 = rnd(1, tq, 1, d), rnd(1, tq, 1, d), rnd(1, 1, 1, d), rnd(1, 1, 1, d)
    k, v = k1.expand(1, tk, 1, d), v1.expand(1, tk, 1, d)
    mask = torch.zeros(1, tk, dtype=torch.uint8, device=DEV)
    mask[0, tk - n:] = 1
    out, lse = igc.cross_attention(q, k, v, key_mask=mask, return_lse=True)
    s = d ** -0.5 * (q[0, :, 0].cpu().double() @ k1[0, 0, 0].cpu().double())
    assert torch.equal(out.cpu(), v1.expand(1, tq, 1, d).cpu())
    # fp32: the scores' products and one logarithm
    assert (lse[0, 0].cpu().double() - s - math.log(n)).abs().max() < 2.0 ** -18
    # the gradient at out = 0: ds_j = p_j dp_j, the same for all keys
    dq = torch.full_like(q, 7.0)
    zero = torch.zeros_like(out)
    assert igc.cross_attn_bwd(go, q, k, v, zero, lse, dq, None, None, key_mask=mask) == 1
    dp = go[0, :, 0].cpu().double() @ v1[0, 0, 0].cpu().double()
    want = d ** -0.5 * dp[:, None] * k1[0, 0, 0].cpu().double()
    # ds and dq are rounded once each, the fp32 steps before are below 2^-12
    assert (dq[0, :, 0].cpu().double() - want).abs().le(
        (2.0 ** -7 + 2.0 ** -12) * want.abs() + 1e-30).all()
