"""The debug build fills the LDS of every kernel that has any: the sources on
the CPU, the norm's kernels (whose LDS other tests do not poison) on the GPU."""
import os
import re

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from test_gpu_qk_norm import CASES, _inputs

CSRC = os.path.join(os.path.dirname(igc.__file__), "csrc")


def _kernels():
    """(file, kernel, body) of every kernel in the sources."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for start in re.finditer(r"__global__.*?(\w+)\(\w+ \w+[^{;]*\)\s*\{", text, re.S):
            depth, at = 1, start.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield name, start.group(1), text[start.end():at]


def test_every_kernel_with_lds_is_poisoned():
    with_lds = [k for k in _kernels() if "__shared__" in k[2]]
    assert len(with_lds) > 12
    for name, kernel, body in with_lds:
        arrays = re.findall(r"__shared__[^;]*?(\w+)\[[^;]*;", body)
        assert arrays, (name, kernel)
        for array in arrays:
            fill = re.search(r"lds_poison<[^;]*\b%s\b" % array, body)
            assert fill, f"{name}: {kernel} does not fill {array}"
            use = re.search(r"\b%s\b" % array, body[fill.end():])
            assert use, (name, kernel, array)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES,
                         ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}.{c[5]}.{c[6]}.{c[7]}")
def test_norm_with_poisoned_lds(case):
    """Outputs, gradients and weight gradients: the ordinary build's bits."""
    print(f"norm poison {case}", flush=True)
    q, k, gq, gk, kw, _ = _inputs(case)
    want = igc.qk_norm_rope(q, k, **kw) + igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    with igc.using_library(igc.POISON_LIB_PATH):
        got = igc.qk_norm_rope(q, k, **kw) + igc.qk_norm_rope_bwd(gq, gk, q, k, **kw)
    for x, y in zip(want, got):
        assert torch.isfinite(y).all() and torch.equal(x, y)
