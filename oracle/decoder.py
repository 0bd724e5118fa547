"""Oracle of the decoder block's operators (TEST INFRASTRUCTURE ONLY): the
definitions of include/igemm_decoder.h in float64 on the CPU, sharing no code
with the HIP library.

Pinned in tests/test_decoder_oracle.py by pure-Python loops, finite differences
and torch's automatic differentiation."""
import torch


def _wide(t):
    return t.detach().cpu().double()


def layer_norm(x, *, weight=None, bias=None, eps=1e-5, grad=None):
    """dict of y and, for bounds on rounding, xh and r; with grad = dy also dx,
    dweight and dbias, and what stands behind them."""
    x = _wide(x)
    c = x.shape[-1]
    w = torch.ones(c).double() if weight is None else _wide(weight)
    b = torch.zeros(c).double() if bias is None else _wide(bias)
    d = x - x.mean(-1, keepdim=True)
    r = (d.square().mean(-1, keepdim=True) + eps) ** -0.5
    xh = d * r
    got = {"y": xh * w + b, "xh": xh, "r": r, "w": w, "b": b,
           "a": x.abs().mean(-1, keepdim=True)}
    if grad is not None:
        g = _wide(grad)
        u = g * w
        q = (u * xh).mean(-1, keepdim=True)
        lead = tuple(range(x.dim() - 1))
        got.update(dx=r * (u - u.mean(-1, keepdim=True) - xh * q), u=u, q=q,
                   dweight=(g * xh).sum(lead), dbias=g.sum(lead), g=g)
    return got
