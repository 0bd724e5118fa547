"""Layer norm, its gradient and the quantising of rows at the ends of the range
of widths that each kernel form takes and at every length of a row's last piece,
against the float64 oracle (bounds: test_gpu_layer_norm.py): rows at any
alignment between NaNs, in place, and under the debug build."""
import os

import pytest
import torch

import implicit_gemm_nhwc_amd as igc
from oracle import decoder as oracle
from test_gpu_layer_norm import _check, _rnd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16

# first and last widths of the forms (lanes a row x pieces of 8 values a lane),
# and every length of the last piece
ENDS = [1, 7, 8, 64, 65, 128, 129, 192, 193, 256, 257, 384, 385, 512, 513, 768, 769, 1024, 1025, 1536,
        1537, 2048, 2049, 4096, 4097, 6144, 6145, 8192, 8193, 12288, 12289, 16384]
TAILS = list(range(9, 16)) + list(range(401, 408)) + list(range(2041, 2048)) + list(range(5001, 5008))


def setup_module(_):
    if not (os.path.exists(igc.LIB_PATH) and os.path.exists(igc.POISON_LIB_PATH)):
        import __graft_entry__
        __graft_entry__.build()


def _between_nans(t, gap, off):
    """t's rows `gap` NaNs apart, `off` behind the storage's start."""
    rows, c = t.shape
    buf = torch.full((off + rows * (c + gap) + 16,), float("nan"), dtype=t.dtype, device=DEV)
    v = buf[off:off + rows * (c + gap)].view(rows, c + gap)[:, :c]
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("c", ENDS + TAILS)
def test_norm(c):
    dt = BF if c % 2 else HF
    rows = 9 if c < 2048 else 3
    x, dy = (_rnd(rows, c, seed=s).to(dt).to(DEV) for s in (1, 2))
    w, b = (1 + 0.3 * _rnd(c, seed=3)).to(DEV), (0.3 * _rnd(c, seed=4)).to(DEV)
    print(f"rows of {c}", flush=True)
    y = igc.layer_norm(x, w, b)
    grads = igc.layer_norm_bwd(dy, x, w)
    _check(x, y, dict(weight=w, bias=b, eps=1e-5), dy, *grads)
    for path in (igc.LIB_PATH, igc.POISON_LIB_PATH):
        with igc.using_library(path):
            xb, xv = _between_nans(x, 3, 1)
            gb, gv = _between_nans(dy, 1, 2)
            assert torch.equal(igc.layer_norm(xv, w, b), y)
            assert all(torch.equal(p, q) for p, q in zip(igc.layer_norm_bwd(gv, xv, w), grads))
            # in place, the NaNs between the rows left as they are
            around = torch.isnan(gb)
            assert igc.layer_norm_grad(gv, xv, gv, weight=w) == 1
            assert torch.equal(gv, grads[0]) and torch.equal(torch.isnan(gb), around)
            around = torch.isnan(xb)
            assert igc.layer_norm_fwd(xv, xv, weight=w, bias=b) == 1
            assert torch.equal(xv, y) and torch.equal(torch.isnan(xb), around)


@pytest.mark.parametrize("c", ENDS + TAILS + [16385, 20001, 32768, 40007])
def test_quantised(c):
    dt = HF if c % 2 else BF
    rows = 9 if c < 2048 else 3
    x = _rnd(rows, c, seed=5).to(dt).to(DEV)
    _, xv = _between_nans(x, 5, 3)
    print(f"rows of {c}", flush=True)
    want, scale = oracle.rows_i8(x)
    pitch = -(-c // 16) * 16 + 16
    for path in (igc.LIB_PATH, igc.POISON_LIB_PATH):
        with igc.using_library(path):
            q, s = igc.quantize_rows(xv)
            assert torch.equal(q.cpu().double(), want) and torch.equal(s.cpu(), scale)
            # bytes between the rows stay
            buf = torch.full((rows, pitch), 99, dtype=torch.int8, device=DEV)
            s2 = torch.empty(rows, device=DEV)
            packed = igc.decoder._QUANT.pack(1, 1, rows, c, xv.data_ptr(), 0, 0, xv.stride(0),
                                             buf.data_ptr(), 0, 0, pitch, s2.data_ptr(),
                                             igc.DTYPE_CODES[dt])
            stream = torch.cuda.current_stream().cuda_stream
            assert igc.lib().quantize_rows(packed, stream) == 1
            assert torch.equal(buf[:, :c], q) and (buf[:, c:] == 99).all() and torch.equal(s2, s)
