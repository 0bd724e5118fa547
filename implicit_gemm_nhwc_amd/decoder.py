"""Binding of the decoder block's operators of include/igemm_decoder.h: layer
norm with its gradient.

Argument marshalling only, as in the package's other calls: every step runs in
the HIP kernels of libigemmconv.so, and there is no fallback.  InvalidArgument
is raised for tensors the C ABI cannot describe, Declined (with the library's
reason) for what its gate refuses.  Results carry no autograd history: a
training program calls the backward entries itself (or from its own
torch.autograd.Function).

  layer_norm_fwd, layer_norm_fwd_check, layer_norm_grad,
  layer_norm_bwd_check, layer_norm_bwd_workspace_bytes
mirror the C entries (layer_norm_grad: layer_norm_bwd; 1 handled, 0 declined,
< 0 HIP error; outputs and workspace given); layer_norm and layer_norm_bwd
allocate their outputs and raise on failure.
"""
import struct

import torch

from . import DTYPE_CODES, InvalidArgument, lib
from .attention import (_current_gpu, _device, _elsewhere, _like, _on, _raise, _raw_stream,
                        _small, _work)

_LN = struct.Struct("@20qdqqq")
_NO_VIEW = (0, 0, 0, 0)
_FORWARD = object()   # in place of a gradient


def _element(t, name):
    """Type code of a bf16 or fp16 tensor."""
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise InvalidArgument(f"{name} dtype {t.dtype} is not bf16 or fp16")
    return DTYPE_CODES[t.dtype]


def _rows(name, t, dtype, device, shape=None):
    """(sizes of the three leading axes, channels) and (pointer, their strides)
    of a tensor [..., C] of one to four axes."""
    if not isinstance(t, torch.Tensor):
        raise InvalidArgument(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise InvalidArgument(f"{name} dtype {t.dtype} differs from {dtype}")
    if t.get_device() != device:
        raise InvalidArgument(f"{name} is on {t.device}, the other tensors on GPU {device}")
    if not 1 <= t.dim() <= 4:
        raise InvalidArgument(f"{name} must have one to four axes (got {tuple(t.shape)})")
    if shape is not None and t.shape != shape:
        raise InvalidArgument(f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise InvalidArgument(f"{name}: the values of a row must be adjacent")
    lead = 4 - t.dim()
    sizes = (1,) * lead + tuple(t.shape)
    return sizes, (t.data_ptr(), *((0,) * lead + t.stride())[:3])


def _channel(name, t, c, device):
    """Pointer of an fp32 tensor of one value a channel (or None)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.shape != (c,):
        raise InvalidArgument(f"{name} must be a tensor of shape {(c,)}")
    return _small(name, t, torch.float32, device)


# --------------------------------------------------------------- layer norm
def _ln_pack(x, out, weight, bias, eps, grad=_FORWARD, dweight=None, dbias=None,
             ws=(0, 0)):
    device = _device(x, "x")
    code = _element(x, "x")
    sizes, xv = _rows("x", x, x.dtype, device)
    _, ov = _rows("out", out, x.dtype, device, x.shape)
    gv = _NO_VIEW
    if grad is not _FORWARD:
        _, gv = _rows("the gradient", grad, x.dtype, device, x.shape)
    c = sizes[3]
    return _LN.pack(*sizes, *xv, *gv, *ov, _channel("weight", weight, c, device),
                    _channel("bias", bias, c, device), _channel("dweight", dweight, c, device),
                    _channel("dbias", dbias, c, device), float(eps), code, *ws), device


def layer_norm_fwd(x, out, *, weight=None, bias=None, eps=1e-5, stream=None) -> int:
    """Enqueue the layer norm of x [..., C] into out (x itself: in place).  1
    handled, 0 declined, < 0 HIP error."""
    packed, device = _ln_pack(x, out, weight, bias, eps)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().layer_norm_fwd(packed, _raw_stream(device))
    return lib().layer_norm_fwd(packed, _raw_stream(device))


def layer_norm_fwd_check(x, out, *, weight=None, bias=None, eps=1e-5) -> int:
    """Host-only gate of layer_norm_fwd: 0 or a decline reason code."""
    return lib().layer_norm_fwd_check(_ln_pack(x, out, weight, bias, eps)[0])


def layer_norm_grad(dy, x, dx, *, weight=None, dweight=None, dbias=None, eps=1e-5,
                    workspace=None, workspace_bytes=0, stream=None) -> int:
    """Enqueue the gradients into dx (dy itself: in place), dweight and dbias
    (fp32 [C], or None: not wanted).  1 handled, 0 declined, < 0 HIP error."""
    device = _device(x, "x")
    packed, _ = _ln_pack(x, dx, weight, None, eps, dy, dweight, dbias,
                         _work(workspace, workspace_bytes, device))
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().layer_norm_bwd(packed, _raw_stream(device))
    return lib().layer_norm_bwd(packed, _raw_stream(device))


def layer_norm_bwd_check(dy, x, dx, *, weight=None, dweight=None, dbias=None, eps=1e-5,
                         workspace=None, workspace_bytes=0) -> int:
    """Host-only gate of layer_norm_grad: 0 or a decline reason code."""
    device = _device(x, "x")
    return lib().layer_norm_bwd_check(
        _ln_pack(x, dx, weight, None, eps, dy, dweight, dbias,
                 _work(workspace, workspace_bytes, device))[0])


def layer_norm_bwd_workspace_bytes(shape, dtype) -> int:
    """Workspace of a layer_norm_grad with a dweight or dbias at x of this
    shape (0 when it would be declined)."""
    sizes = (1,) * (4 - len(shape)) + tuple(shape)
    return lib().layer_norm_bwd_workspace_bytes(
        _LN.pack(*sizes, *(0,) * 14, 16, 16, 1.0, DTYPE_CODES.get(dtype, -1), 0, 0))


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, stream=None):
    """Rows of x [..., C] (one to four axes) less their mean, divided by their
    standard deviation, times weight and plus bias (fp32 [C] or None).  Returns
    a dense tensor like x.  Gradients by layer_norm_bwd (none are recorded for
    autograd)."""
    device = _device(x, "x")
    if _elsewhere(device, stream):
        with _on(device, stream):
            return layer_norm(x, weight, bias, eps=eps)
    out = _like(x)
    packed, _ = _ln_pack(x, out, weight, bias, eps)
    L = lib()
    rc = L.layer_norm_fwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("layer_norm_fwd", rc, L.layer_norm_fwd_check, packed)
    return out


def layer_norm_bwd(dy, x, weight=None, *, eps=1e-5, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm at x, weight and bias from
    dy, dx dense like x, the others fp32 (also for a weight or bias of None,
    which count as ones and zeros)."""
    device = _device(x, "x")
    if _elsewhere(device, stream):
        with _on(device, stream):
            return layer_norm_bwd(dy, x, weight, eps=eps)
    dx = _like(x)
    c = x.shape[-1] if x.dim() else 0
    dw = torch.empty(c, dtype=torch.float32, device=x.device)
    db = torch.empty_like(dw)
    packed, _ = _ln_pack(x, dx, weight, None, eps, dy, dw, db)
    L = lib()
    need = L.layer_norm_bwd_workspace_bytes(packed)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        packed = packed[:-16] + struct.pack("@qq", ws.data_ptr(), need)
    rc = L.layer_norm_bwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("layer_norm_bwd", rc, L.layer_norm_bwd_check, packed)
    return dx, dw, db
