"""Binding of the attention operators of include/igemm_attn.h: cross attention
to an encoder's states, and the per-head norm of queries and keys with the
position rotation, each with its backward pass.

Argument marshalling only, as in the package's convolution calls: every step
runs in the HIP kernels of libigemmconv.so, and there is no fallback.
InvalidArgument is raised for tensors the C ABI cannot describe, Declined
(with the library's reason) for what its gate refuses.

Tensors are [batch, token, head, D], D adjacent, any other strides that are
multiples of 16 bytes; an NHWC map [N, H, W, heads * D] is
map.view(N, H * W, heads, D).

Results carry no autograd history, whatever the inputs require: a training
program calls the backward entries itself (or from its own
torch.autograd.Function).

  cross_attn_fwd, cross_attn_fwd_check, cross_attn_fwd_workspace_bytes,
  cross_attn_bwd, cross_attn_bwd_check, cross_attn_bwd_workspace_bytes,
  qk_norm_rope_fwd, qk_norm_rope_fwd_check,
  qk_norm_rope_bwd, qk_norm_rope_bwd_check, qk_norm_rope_bwd_workspace_bytes
mirror the C entries (1 handled, 0 declined, < 0 HIP error; outputs and
workspace given); cross_attention, cross_attention_bwd, qk_norm_rope and
qk_norm_rope_bwd allocate their outputs and raise on failure; rope_table and rope_table_2d make the
rotation's tables.
"""
import ctypes
import struct

import torch

from . import DTYPE_CODES, REASONS, Declined, InvalidArgument, lib

try:   # the ordinary calls in C++ (csrc/attn_marshal.cpp); without it, all through Python
    from . import _attn_marshal as _fast
except ImportError:
    _fast = None

_ATTN = struct.Struct("@26qdqqq")
_VIEWS = struct.Struct("@16q")   # dout, dq, dk, dv
_QK = struct.Struct("@42q4qdqq")   # two parts of 21 fields
_NO_PART = (0,) * 21
_NO_VIEW = (0, 0, 0, 0)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_gpu = torch._C._cuda_getDevice


def _view(name, t, dtype, device):
    """(pointer, batch, token, head stride) of a [batch, token, head, D] tensor."""
    if not isinstance(t, torch.Tensor):
        raise InvalidArgument(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise InvalidArgument(f"{name} dtype {t.dtype} differs from {dtype}")
    if t.get_device() != device:
        raise InvalidArgument(f"{name} is on {t.device}, the other tensors on GPU {device}")
    if t.dim() != 4:
        raise InvalidArgument(f"{name} must be [batch, token, head, D] (got {tuple(t.shape)})")
    sb, st, sh, sd = t.stride()
    if sd != 1 and t.shape[3] > 1:
        raise InvalidArgument(f"{name}: the D values of a head must be adjacent")
    return t.data_ptr(), sb, st, sh


def _small(name, t, dtype, device):
    """Pointer of a dense side tensor (or None)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise InvalidArgument(f"{name} must be {dtype} (got {t.dtype})")
    if t.get_device() != device:
        raise InvalidArgument(f"{name} is on {t.device}, the other tensors on GPU {device}")
    raise InvalidArgument(f"{name} must be contiguous")


def _device(t, name="q"):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise InvalidArgument(f"{name} must be a GPU tensor")
    return t.get_device()


def _work(ws, nbytes, device):
    """Pointer and bytes of a workspace tensor (or None)."""
    if ws is None:
        return 0, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise InvalidArgument("workspace must be contiguous and on the tensors' GPU")
    have = ws.numel() * ws.element_size()
    if nbytes and have < nbytes:
        raise InvalidArgument(f"workspace holds {have} bytes, workspace_bytes says {nbytes}")
    return ws.data_ptr(), nbytes or have


class _on:
    """Runs the block on the tensors' GPU, and with `stream` (a torch stream
    or a raw handle) as its current one, so that what is allocated inside
    belongs to the stream that uses it."""

    def __init__(self, device, stream):
        self.device = torch.cuda.device(device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        self.stream = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        self.device.__enter__()
        if self.stream is not None:
            self.stream.__enter__()

    def __exit__(self, *err):
        if self.stream is not None:
            self.stream.__exit__(*err)
        self.device.__exit__(*err)


def _elsewhere(device, stream):
    return stream is not None or device != _current_gpu()


def _entries():
    """The current library's entries as attn_marshal.cpp takes them."""
    L = lib()
    try:
        return L.attn_entries
    except AttributeError:
        pass
    L.attn_entries = _fast.bind(*(
        ctypes.cast(getattr(L, n), ctypes.c_void_p).value
        for n in ("cross_attn_fwd", "cross_attn_fwd_workspace_bytes", "cross_attn_bwd",
                  "cross_attn_bwd_workspace_bytes", "qk_norm_rope_fwd", "qk_norm_rope_bwd",
                  "qk_norm_rope_bwd_workspace_bytes")))
    return L.attn_entries


def _raise(name, rc, check, packed):
    if rc == 0:
        reason = check(packed)
        raise Declined(f"{name} declined: {REASONS.get(reason, reason)}")
    raise RuntimeError(f"{name} failed with HIP error {-rc}")


# --------------------------------------------------------- cross attention
def _attn_head(q, k, v, kv_lens, key_mask, scale):
    """Sizes and input views of igc_cross_attn, its side arrays with scale and
    type, and the GPU."""
    device = _device(q)
    dtype = q.dtype
    if dtype not in DTYPE_CODES:
        raise InvalidArgument(f"q dtype {dtype} is not bf16 or fp16")
    views = _view("q", q, dtype, device) + _view("k", k, dtype, device) + _view(
        "v", v, dtype, device)
    b, tq, hq, d = q.shape
    ks = k.shape
    kb, tk, hk, kd = ks
    if kb != b or kd != d or v.shape != ks:
        raise InvalidArgument(f"q {tuple(q.shape)}, k {tuple(ks)} and v {tuple(v.shape)} "
                              "do not belong together")
    np_ = mp = ms = 0
    if kv_lens is not None:
        np_ = _small("kv_lens", kv_lens, torch.int32, device)
        if kv_lens.shape != (b,):
            raise InvalidArgument(f"kv_lens must be {(b,)} (got {tuple(kv_lens.shape)})")
    if key_mask is not None:
        if key_mask.dtype not in (torch.uint8, torch.bool):
            raise InvalidArgument(f"key_mask must be uint8 or bool (got {key_mask.dtype})")
        if key_mask.get_device() != device:
            raise InvalidArgument("key_mask is not on the tensors' GPU")
        if key_mask.shape != (b, tk):
            raise InvalidArgument(f"key_mask must be {(b, tk)} (got {tuple(key_mask.shape)})")
        ms, inner = key_mask.stride()
        if inner != 1 and tk > 1:
            raise InvalidArgument("key_mask: the keys of a batch entry must be adjacent")
        mp = key_mask.data_ptr()
    if scale is None:
        scale = d ** -0.5 if d else 1.0
    return ((b, tq, tk, hq, hk, d) + views,
            (np_, mp, ms, float(scale), DTYPE_CODES[dtype]), device)


def _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale):
    """_attn_head with the caller's out and lse: all but the workspace."""
    head, tail, device = _attn_head(q, k, v, kv_lens, key_mask, scale)
    ov = _view("out", out, q.dtype, device)
    if out.shape != q.shape:
        raise InvalidArgument(f"out must have q's shape {tuple(q.shape)}")
    lp = _small("lse", lse, torch.float32, device)
    if lse is not None and lse.shape != (head[0], head[3], head[1]):
        raise InvalidArgument(f"lse must be {(head[0], head[3], head[1])} "
                              f"(got {tuple(lse.shape)})")
    return head + ov + (lp,) + tail, device


def _like(t):
    """A new dense tensor of t's shape and type."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def cross_attn_fwd(q, k, v, out, *, lse=None, kv_lens=None, key_mask=None, scale=None,
                   workspace=None, workspace_bytes=0, stream=None) -> int:
    """Enqueue cross attention into out (and lse).  1 handled, 0 declined, < 0
    HIP error."""
    head, device = _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale)
    ws = _work(workspace, workspace_bytes, device)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().cross_attn_fwd(_ATTN.pack(*head, *ws), _raw_stream(device))
    return lib().cross_attn_fwd(_ATTN.pack(*head, *ws), _raw_stream(device))


def cross_attn_fwd_check(q, k, v, out, *, lse=None, kv_lens=None, key_mask=None, scale=None,
                         workspace=None, workspace_bytes=0) -> int:
    """Host-only gate of cross_attn_fwd: 0 or a decline reason code."""
    head, device = _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale)
    return lib().cross_attn_fwd_check(_ATTN.pack(*head, *_work(workspace, workspace_bytes, device)))


def cross_attn_fwd_workspace_bytes(q_shape, k_shape, dtype) -> int:
    """Workspace of a call of these shapes (0 when none is needed, or when it
    would be declined)."""
    b, tq, hq, d = q_shape
    _, tk, hk, _ = k_shape
    return lib().cross_attn_fwd_workspace_bytes(
        _ATTN.pack(b, tq, tk, hq, hk, d, *(0,) * 20, 1.0, DTYPE_CODES.get(dtype, -1), 0, 0))


def cross_attention(q, k, v, *, scale=None, kv_lens=None, key_mask=None, return_lse=False,
                    stream=None):
    """Attention of q [b, tq, hq, D] to the encoder's states k, v [b, tk, hk,
    D] (hk dividing hq); scale defaults to 1 / sqrt(D).  kv_lens (int32 [b])
    and key_mask (uint8 or bool [b, tk], nonzero = attend) say which keys are
    valid; a row without one gives 0.  Returns out, dense like q, and with
    return_lse also the fp32 row statistics [b, hq, tq] for
    cross_attention_bwd, which is the way to gradients (none are recorded for
    autograd)."""
    device = _device(q)
    if _fast is not None and stream is None:
        r = _fast.cross_attention(_entries(), q, k, v, scale, kv_lens, key_mask, return_lse,
                                  _raw_stream(device), _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return cross_attention(q, k, v, scale=scale, kv_lens=kv_lens, key_mask=key_mask,
                                   return_lse=return_lse)
    head, tail, _ = _attn_head(q, k, v, kv_lens, key_mask, scale)
    b, tq, _, hq, _, d = head[:6]
    out = _like(q)
    lse = None
    if return_lse:
        lse = torch.empty((b, hq, tq), dtype=torch.float32, device=q.device)
    args = head + (out.data_ptr(), tq * hq * d, hq * d, d,
                   0 if lse is None else lse.data_ptr()) + tail
    L = lib()
    packed = _ATTN.pack(*args, 0, 0)
    need = L.cross_attn_fwd_workspace_bytes(packed)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        packed = _ATTN.pack(*args, ws.data_ptr(), need)
    rc = L.cross_attn_fwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("cross_attn_fwd", rc, L.cross_attn_fwd_check, packed)
    return (out, lse) if return_lse else out


def _grad_views(q, k, v, dout, dq, dk, dv, device):
    views = _view("dout", dout, q.dtype, device)
    if dout.shape != q.shape:
        raise InvalidArgument(f"dout must have q's shape {tuple(q.shape)}")
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            views += _NO_VIEW
            continue
        views += _view(name, t, q.dtype, device)
        if t.shape != like.shape:
            raise InvalidArgument(f"{name} must have {name[1]}'s shape {tuple(like.shape)}")
    return _VIEWS.pack(*views)


def cross_attn_bwd(dout, q, k, v, out, lse, dq, dk, dv, *, kv_lens=None, key_mask=None,
                   scale=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    """Enqueue the gradients into dq, dk, dv (dq, or dk and dv, may be None:
    not wanted).  1 handled, 0 declined, < 0 HIP error."""
    head, device = _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale)
    packed = _ATTN.pack(*head, *_work(workspace, workspace_bytes, device)) + _grad_views(
        q, k, v, dout, dq, dk, dv, device)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().cross_attn_bwd(packed, _raw_stream(device))
    return lib().cross_attn_bwd(packed, _raw_stream(device))


def cross_attn_bwd_check(dout, q, k, v, out, lse, dq, dk, dv, *, kv_lens=None, key_mask=None,
                         scale=None, workspace=None, workspace_bytes=0) -> int:
    """Host-only gate of cross_attn_bwd: 0 or a decline reason code."""
    head, device = _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale)
    return lib().cross_attn_bwd_check(
        _ATTN.pack(*head, *_work(workspace, workspace_bytes, device))
        + _grad_views(q, k, v, dout, dq, dk, dv, device))


def cross_attn_bwd_workspace_bytes(q_shape, k_shape, dtype) -> int:
    """Workspace of a call of these shapes (0 when it would be declined)."""
    b, tq, hq, d = q_shape
    _, tk, hk, _ = k_shape
    return lib().cross_attn_bwd_workspace_bytes(
        _ATTN.pack(b, tq, tk, hq, hk, d, *(0,) * 20, 1.0, DTYPE_CODES.get(dtype, -1), 0, 0)
        + bytes(_VIEWS.size))


def cross_attention_bwd(dout, q, k, v, out, lse, *, scale=None, kv_lens=None, key_mask=None,
                        stream=None):
    """Gradients (dq, dk, dv), dense, of cross_attention at q, k and v from
    dout, with its out and lse (return_lse) and the same scale, kv_lens and
    key_mask.  dk and dv sum over the query heads that share a key head."""
    device = _device(q)
    if _fast is not None and stream is None:
        r = _fast.cross_attention_bwd(_entries(), dout, q, k, v, out, lse, scale, kv_lens,
                                      key_mask, _raw_stream(device), _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return cross_attention_bwd(dout, q, k, v, out, lse, scale=scale, kv_lens=kv_lens,
                                       key_mask=key_mask)
    head, _ = _attn_args(q, k, v, out, lse, kv_lens, key_mask, scale)
    dq, dk, dv = _like(q), _like(k), _like(v)
    views = _grad_views(q, k, v, dout, dq, dk, dv, device)
    L = lib()
    packed = _ATTN.pack(*head, 0, 0) + views
    need = L.cross_attn_bwd_workspace_bytes(packed)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        packed = _ATTN.pack(*head, ws.data_ptr(), need) + views
    rc = L.cross_attn_bwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("cross_attn_bwd", rc, L.cross_attn_bwd_check, packed)
    return dq, dk, dv


# ------------------------------------------- norm of queries and keys, rotation
def _part(n, x, grad, out, dw, weight, table, positions, dtype, device, d):
    """All fields of an igc_qk_part.  out: a tensor to check, or the view of a
    new one; dw: a tensor to check, a pointer or 0."""
    xv = _view(n, x, dtype, device)
    shape = x.shape
    b, t, h, dd = shape
    if dd != d:
        raise InvalidArgument(f"{n} has heads of {dd}, not {d}")
    g = _NO_VIEW
    if grad is not None:
        g = _view(n + "'s gradient", grad, dtype, device)
        if grad.shape != shape:
            raise InvalidArgument(f"d{n} must have {n}'s shape {tuple(shape)}")
    if not isinstance(out, tuple):
        o, out = out, _view(n + "'s output", out, dtype, device)
        if o.shape != shape:
            raise InvalidArgument(f"{n}'s output must have its shape {tuple(shape)}")
    wp = 0
    if weight is not None:
        wp = _small("weight", weight, torch.float32, device)
        if weight.dim() != 1 or len(weight) != d:
            raise InvalidArgument(f"{n}_weight must be {(d,)} (got {tuple(weight.shape)})")
    if isinstance(dw, torch.Tensor):
        if dw.shape != (d,):
            raise InvalidArgument(f"the gradient of {n}_weight must be {(d,)}")
        dw = _small("weight gradient", dw, torch.float32, device)
    pp = ps = 0
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.dim() != 2:
            raise InvalidArgument(f"{n}_positions must be int32 [batch, token] (got "
                                  f"{positions.dtype}, {tuple(positions.shape)})")
        if positions.get_device() != device:
            raise InvalidArgument(f"{n}_positions is not on the tensors' GPU")
        pb, pt = positions.shape
        ps, inner = positions.stride()
        if pb != b or pt != t:
            raise InvalidArgument(f"{n}_positions must be {(b, t)} (got {(pb, pt)})")
        if inner != 1 and t > 1:
            raise InvalidArgument(f"{n}_positions: the tokens of a batch entry must be adjacent")
        pp = positions.data_ptr()
    return (b, t, h, *xv, *g, *out, wp, dw or 0, *table, pp, ps)


def _table(t, name, device):
    """(pointer, rows) of a rotation table and the values it turns."""
    if t is None:
        return (0, 0), 0
    if t.dim() != 2:
        raise InvalidArgument(f"{name} must be [rows, rotated values] (got {tuple(t.shape)})")
    rows, rot = t.shape
    return (_small(name, t, torch.float32, device), rows), rot


_NONE2 = (None, None)


def _qk_pack(q, k, grads, outs, dweights, q_weight, k_weight, q_table, k_table, q_positions,
             k_positions, eps, interleaved, ws=(0, 0)):
    """igc_qk_norm, packed.  grads, outs and dweights: pairs (_part)."""
    first = q if q is not None else k
    device = _device(first, "q" if q is not None else "k")
    dtype = first.dtype
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise InvalidArgument(f"dtype {dtype} is not bf16 or fp16")
    if first.dim() != 4:
        raise InvalidArgument(f"tensors must be [batch, token, head, D] (got "
                              f"{tuple(first.shape)})")
    d = first.shape[3]
    a = b = _NO_PART
    rot = None
    if q is not None:
        table, rot = _table(q_table, "q_table", device)
        a = _part("q", q, grads[0], outs[0], dweights[0], q_weight, table, q_positions, dtype,
                  device, d)
    if k is not None:
        if q is None or k_table is not q_table:
            table, rot_k = _table(k_table, "k_table", device)
            if rot is not None and rot_k != rot:
                raise InvalidArgument("q_table and k_table must rotate the same number of values")
            rot = rot_k
        b = _part("k", k, grads[1], outs[1], dweights[1], k_weight, table, k_positions, dtype,
                  device, d)
    return _QK.pack(*a, *b, d, rot, 1 if interleaved else 0, code, eps, *ws), device


def _dense(t, shape):
    """View of a new dense tensor."""
    _, n, h, d = shape
    return t.data_ptr(), n * h * d, h * d, d


def qk_norm_rope_fwd(q, k, q_out, k_out, *, q_weight=None, k_weight=None, q_table=None,
                     k_table=None, q_positions=None, k_positions=None, eps=1e-6,
                     interleaved=False, stream=None) -> int:
    """Enqueue the norm and rotation of q and k (either may be None) into
    q_out, k_out (q and k themselves: in place).  1 handled, 0 declined, < 0
    HIP error."""
    packed, device = _qk_pack(q, k, _NONE2, (q_out, k_out), _NONE2, q_weight, k_weight, q_table,
                              k_table, q_positions, k_positions, eps, interleaved)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().qk_norm_rope_fwd(packed, _raw_stream(device))
    return lib().qk_norm_rope_fwd(packed, _raw_stream(device))


def qk_norm_rope_fwd_check(q, k, q_out, k_out, *, q_weight=None, k_weight=None, q_table=None,
                           k_table=None, q_positions=None, k_positions=None, eps=1e-6,
                           interleaved=False) -> int:
    """Host-only gate of qk_norm_rope_fwd: 0 or a decline reason code."""
    return lib().qk_norm_rope_fwd_check(
        _qk_pack(q, k, _NONE2, (q_out, k_out), _NONE2, q_weight, k_weight, q_table, k_table,
                 q_positions, k_positions, eps, interleaved)[0])


def qk_norm_rope_bwd_check(dq, dk, q, k, dq_out, dk_out, *, q_weight=None, k_weight=None,
                           dq_weight=None, dk_weight=None, q_table=None, k_table=None,
                           q_positions=None, k_positions=None, eps=1e-6, interleaved=False,
                           workspace=None, workspace_bytes=0) -> int:
    """Host-only gate of qk_norm_rope_bwd: 0 or a decline reason code."""
    device = _device(q if q is not None else k)
    return lib().qk_norm_rope_bwd_check(
        _qk_pack(q, k, (dq, dk), (dq_out, dk_out), (dq_weight, dk_weight), q_weight, k_weight,
                 q_table, k_table, q_positions, k_positions, eps, interleaved,
                 _work(workspace, workspace_bytes, device))[0])


def qk_norm_rope(q, k=None, *, q_weight=None, k_weight=None, q_table=None, k_table=None,
                 q_positions=None, k_positions=None, eps=1e-6, interleaved=False, stream=None):
    """The heads of q [b, tq, hq, D] and k [b', tk, hk, D] divided by their
    root mean square, times the weight (fp32 [D] or None), their first
    table.shape[1] values rotated in pairs by the table row (fp32 {cosines,
    sines}, rope_table) of their position (int32 [b, t] or None: the token's
    number).  Returns the two results, dense; k may be None (then q's result
    alone).  Gradients by qk_norm_rope_bwd (none are recorded for autograd)."""
    device = _device(q)
    if _fast is not None and stream is None:
        r = _fast.qk_norm_rope(_entries(), q, k, q_weight, k_weight, q_table, k_table,
                               q_positions, k_positions, eps, interleaved, _raw_stream(device),
                               _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return qk_norm_rope(q, k, q_weight=q_weight, k_weight=k_weight, q_table=q_table,
                                k_table=k_table, q_positions=q_positions,
                                k_positions=k_positions, eps=eps, interleaved=interleaved)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise InvalidArgument("q and k must be [batch, token, head, D]")
    q_out = _like(q)
    if k is None:
        k_out, outs = None, (_dense(q_out, q.shape), None)
    else:
        k_out = _like(k)
        outs = (_dense(q_out, q.shape), _dense(k_out, k.shape))
    packed, _ = _qk_pack(q, k, _NONE2, outs, _NONE2, q_weight, k_weight, q_table, k_table,
                         q_positions, k_positions, eps, interleaved)
    L = lib()
    rc = L.qk_norm_rope_fwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("qk_norm_rope_fwd", rc, L.qk_norm_rope_fwd_check, packed)
    return q_out if k is None else (q_out, k_out)


def qk_norm_rope_bwd(dq, dk, q, k=None, *, q_weight=None, k_weight=None, q_table=None,
                     k_table=None, q_positions=None, k_positions=None, eps=1e-6,
                     interleaved=False, stream=None):
    """Gradients of qk_norm_rope at its inputs: dq, dk are those of its
    results.  Returns (dq, dk, dq_weight, dk_weight) at q, k and the weights
    (fp32; also for a weight of None, which counts as ones); k may be None
    (its two gradients are then None)."""
    device = _device(q)
    if _fast is not None and stream is None:
        r = _fast.qk_norm_rope_bwd(_entries(), dq, dk, q, k, q_weight, k_weight, q_table, k_table,
                                   q_positions, k_positions, eps, interleaved,
                                   _raw_stream(device), _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return qk_norm_rope_bwd(dq, dk, q, k, q_weight=q_weight, k_weight=k_weight,
                                    q_table=q_table, k_table=k_table, q_positions=q_positions,
                                    k_positions=k_positions, eps=eps, interleaved=interleaved)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise InvalidArgument("q and k must be [batch, token, head, D]")
    d = q.shape[3]
    dqw = torch.empty(d, dtype=torch.float32, device=q.device)
    dq_out = _like(q)
    if k is None:
        dk_out = dkw = None
        outs, dws = (_dense(dq_out, q.shape), None), (dqw.data_ptr(), None)
    else:
        dk_out = _like(k)
        outs = (_dense(dq_out, q.shape), _dense(dk_out, k.shape))
        dkw = torch.empty_like(dqw)
        dws = (dqw.data_ptr(), dkw.data_ptr())
    packed, _ = _qk_pack(q, k, (dq, dk), outs, dws, q_weight, k_weight, q_table, k_table,
                         q_positions, k_positions, eps, interleaved)
    L = lib()
    need = L.qk_norm_rope_bwd_workspace_bytes(packed)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        packed = packed[:-16] + struct.pack("@qq", ws.data_ptr(), need)
    rc = L.qk_norm_rope_bwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("qk_norm_rope_bwd", rc, L.qk_norm_rope_bwd_check, packed)
    return dq_out, dk_out, dqw, dkw


def rope_table(n, rot, *, base=10000.0, first=0, device=None):
    """Table of qk_norm_rope for n positions from `first` on: fp32 [n, rot],
    cosines then sines of position * base^(-2 i / rot), the angles formed in
    64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = (torch.arange(n, dtype=torch.float64) + first)[:, None] * base ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


def rope_table_2d(h, w, rot, *, base=10000.0, device=None):
    """Table for the pixels of an h x w map in NHWC order (rot a multiple of
    4): the first half of the angles from the pixel's row, the second from its
    column, each as rope_table's of rot / 2."""
    i = torch.arange(rot // 4, dtype=torch.float64)
    f = base ** (-4.0 * i / rot)
    r = torch.arange(h, dtype=torch.float64)[:, None, None] * f
    c = torch.arange(w, dtype=torch.float64)[None, :, None] * f
    a = torch.cat([r.expand(h, w, -1), c.expand(h, w, -1)], 2).reshape(h * w, rot // 2)
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)
