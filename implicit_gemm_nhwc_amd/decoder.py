"""Binding of the decoder block's operators of include/igemm_decoder.h: layer
norm with its gradient, rows in 8 bits and their product, the paged cache of
keys and values in 8 bits, and the attention of new tokens over it.

Argument marshalling only, as in the package's other calls: every step runs in
the HIP kernels of libigemmconv.so, and there is no fallback.  InvalidArgument
is raised for tensors the C ABI cannot describe, Declined (with the library's
reason) for what its gate refuses.  Results carry no autograd history: a
training program calls the backward entries itself (or from its own
torch.autograd.Function).

  layer_norm_fwd, layer_norm_fwd_check, layer_norm_grad,
  layer_norm_bwd_check, layer_norm_bwd_workspace_bytes,
  cache_attn_fwd, cache_attn_fwd_check, cache_attn_fwd_workspace_bytes,
  linear_i8_check, kv_cache_write_check
mirror the C entries (layer_norm_grad: layer_norm_bwd; 1 handled, 0 declined,
< 0 HIP error; outputs and workspace given); layer_norm, layer_norm_bwd,
quantize_rows, linear_i8, kv_cache_write, kv_cache_read and cache_attention
allocate their outputs and raise on failure.
"""
import ctypes
import struct

import torch

from . import DTYPE_CODES, InvalidArgument, lib
from .attention import (_current_gpu, _dense, _device, _elsewhere, _like, _on, _raise,
                        _raw_stream, _small, _view, _work)

try:   # the ordinary calls in C++ (csrc/decoder_marshal.cpp); without it, all through Python
    from . import _decoder_marshal as _fast
except ImportError:
    _fast = None

_LN = struct.Struct("@20qdqqq")
_QUANT = struct.Struct("@14q")
_LINEAR = struct.Struct("@13q")
_CACHE = struct.Struct("@8q")
_IO = struct.Struct("@16q")        # after a cache
_CATTN = struct.Struct("@17qdqqq")   # after a cache
_NO_VIEW = (0, 0, 0, 0)
_FORWARD = object()   # in place of a gradient


def _entries():
    """The current library's entries as decoder_marshal.cpp takes them."""
    L = lib()
    try:
        return L.decoder_entries
    except AttributeError:
        pass
    L.decoder_entries = _fast.bind(*(
        ctypes.cast(getattr(L, n), ctypes.c_void_p).value
        for n in ("layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_bytes",
                  "quantize_rows", "linear_i8", "kv_cache_write", "kv_cache_read",
                  "cache_attn_fwd", "cache_attn_fwd_workspace_bytes")))
    return L.decoder_entries


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
    if _fast is not None and stream is None:
        r = _fast.layer_norm(_entries(), x, weight, bias, eps, _raw_stream(device), _current_gpu())
        if r is not None:
            return r
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
    if _fast is not None and stream is None:
        r = _fast.layer_norm_bwd(_entries(), dy, x, weight, eps, _raw_stream(device),
                                 _current_gpu())
        if r is not None:
            return r
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


# ------------------------------------------------------------ rows in 8 bits
def quantize_rows(x, *, stream=None):
    """Rows of x [..., C] (one to four axes) as integers and a scale: m = max
    |x| of the row, scale = m / 127 in fp32, q = 127 x / m rounded to nearest,
    ties to even.  Returns (q int8 [..., C], scale fp32 [...]); q's rows start
    at multiples of 16 bytes, as linear_i8 reads them.  A row with an infinity
    or a NaN has scale NaN, one below 2^-110 scale 0."""
    device = _device(x, "x")
    if _fast is not None and stream is None:
        r = _fast.quantize_rows(_entries(), x, _raw_stream(device), _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return quantize_rows(x)
    code = _element(x, "x")
    sizes, xv = _rows("x", x, x.dtype, device)
    c = sizes[3]
    pitch = -(-c // 16) * 16
    q = torch.empty((*x.shape[:-1], pitch), dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    packed = _QUANT.pack(*sizes, *xv, q.data_ptr(), sizes[1] * sizes[2] * pitch,
                         sizes[2] * pitch, pitch, scale.data_ptr(), code)
    L = lib()
    rc = L.quantize_rows(packed, _raw_stream(device))
    if rc != 1:
        _raise("quantize_rows", rc, L.quantize_rows_check, packed)
    return (q if pitch == c else q[..., :c]), scale


def _matrix(name, t, device):
    """(rows, k, pitch) of an int8 tensor [..., k] whose rows lie one pitch
    apart, k adjacent, with room for the last row's whole 16-byte pieces."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int8 or t.dim() < 1:
        raise InvalidArgument(f"{name} must be an int8 tensor [..., k]")
    if t.get_device() != device:
        raise InvalidArgument(f"{name} is on {t.device}, the other tensors on GPU {device}")
    k = t.shape[-1]
    if t.stride(-1) != 1 and k > 1:
        raise InvalidArgument(f"{name}: the values of a row must be adjacent")
    rows, pitch = 1, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n != 1 and rows:
            if pitch is None:
                pitch = s
            elif s != pitch * rows:
                raise InvalidArgument(f"{name}: its rows must lie one stride apart")
        rows *= n
    if pitch is None:
        pitch = -(-k // 16) * 16
    if rows and k % 16:
        end = t.storage_offset() + (rows - 1) * pitch + -(-k // 16) * 16
        if end > t.untyped_storage().nbytes():
            raise InvalidArgument(f"{name}: the last row's 16-byte pieces end past its storage "
                                  "(quantize_rows leaves room for them)")
    return rows, k, pitch


def _vector(name, t, shape, device):
    """Pointer of a dense fp32 tensor of this shape."""
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        raise InvalidArgument(f"{name} must be a tensor of shape {tuple(shape)}")
    return _small(name, t, torch.float32, device)


def _linear_pack(x, x_scale, w, w_scale, bias, out):
    device = _device(x, "x")
    rows, k, pitch = _matrix("x", x, device)
    n, wk, w_pitch = _matrix("w", w, device)
    if w.dim() != 2 or wk != k:
        raise InvalidArgument(f"w must be [n, {k}] (got {tuple(w.shape)})")
    code = _element(out, "y")
    return _LINEAR.pack(rows, n, k, x.data_ptr(), pitch, w.data_ptr(), w_pitch,
                        _vector("x_scale", x_scale, x.shape[:-1], device),
                        _vector("w_scale", w_scale, (n,), device),
                        0 if bias is None else _vector("bias", bias, (n,), device),
                        out.data_ptr(), n, code)


def linear_i8_check(x, x_scale, w, w_scale, out, *, bias=None) -> int:
    """Host-only gate of linear_i8 into a dense out: 0 or a decline reason
    code."""
    return lib().linear_i8_check(_linear_pack(x, x_scale, w, w_scale, bias, out))


def linear_i8(x, x_scale, w, w_scale, *, bias=None, dtype=torch.bfloat16, stream=None):
    """The product of rows in 8 bits: x int8 [..., k] with x_scale fp32 [...]
    and w int8 [n, k] with w_scale fp32 [n] (quantize_rows of the tokens and of
    the weights) give dtype [..., n]: (x w^T) x_scale w_scale + bias (fp32 [n]
    or None).  The integer sums are exact; x_scale times a sum has to stay below
    2^128 (an x_scale up to 2^96 always does).  Rows start at multiples of 16
    bytes, which their last 16-byte piece may reach past k."""
    device = _device(x, "x")
    if _fast is not None and stream is None:
        r = _fast.linear_i8(_entries(), x, x_scale, w, w_scale, bias, dtype,
                            _raw_stream(device), _current_gpu())
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return linear_i8(x, x_scale, w, w_scale, bias=bias, dtype=dtype)
    if dtype not in (torch.bfloat16, torch.float16):
        raise InvalidArgument(f"dtype {dtype} is not bf16 or fp16")
    n = w.shape[0] if isinstance(w, torch.Tensor) and w.dim() else 0
    if x.dim() < 1:
        raise InvalidArgument("x must be an int8 tensor [..., k]")
    y = torch.empty((*x.shape[:-1], n), dtype=dtype, device=x.device)
    packed = _linear_pack(x, x_scale, w, w_scale, bias, y)
    L = lib()
    rc = L.linear_i8(packed, _raw_stream(device))
    if rc != 1:
        _raise("linear_i8", rc, L.linear_i8_check, packed)
    return y


# ------------------------------------------------------------------ the cache
class KVCache:
    """A pool of pages of keys and values in 8 bits: k, v int8 [pages,
    kv_heads, page_tokens, D rounded up to 16] and k_scale, v_scale fp32
    [pages, kv_heads, page_tokens], all dense.  Sequences reach it through
    tables of page numbers, int32 [batch, entries]; who owns which page is the
    caller's to keep."""

    def __init__(self, k, v, k_scale, v_scale, head_dim):
        device = _device(k, "k")
        if k.dim() != 4 or k.dtype != torch.int8 or not k.is_contiguous():
            raise InvalidArgument("k must be a dense int8 [pages, kv_heads, page_tokens, D]")
        if k.shape[3] != -(-head_dim // 16) * 16:
            raise InvalidArgument(f"k's rows must hold head_dim ({head_dim}) rounded up to 16 "
                                  f"(got {tuple(k.shape)})")
        for name, t, shape, dtype in (("v", v, k.shape, torch.int8),
                                      ("k_scale", k_scale, k.shape[:3], torch.float32),
                                      ("v_scale", v_scale, k.shape[:3], torch.float32)):
            if not isinstance(t, torch.Tensor) or t.shape != shape:
                raise InvalidArgument(f"{name} must be a tensor of shape {tuple(shape)}")
            _small(name, t, dtype, device)
        self._parts = (k, v, k_scale, v_scale)
        self.head_dim = head_dim
        pages, heads, tokens, _ = k.shape
        self.device = device
        self.kv_heads = heads
        self.packed = _CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                  v_scale.data_ptr(), pages, tokens, heads, head_dim)

    @classmethod
    def empty(cls, pages, page_tokens, kv_heads, head_dim, *, device="cuda"):
        """A new pool of zeros."""
        shape = (pages, kv_heads, page_tokens)
        rows = [torch.zeros((*shape, -(-head_dim // 16) * 16), dtype=torch.int8, device=device)
                for _ in range(2)]
        scales = [torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*rows, *scales, head_dim)

    k, v, k_scale, v_scale = (property(lambda self, i=i: self._parts[i]) for i in range(4))


def _pool(cache):
    if not isinstance(cache, KVCache):
        raise InvalidArgument("cache must be a KVCache")
    return cache.device


def _page_table(table, b, device):
    """(pointer, stride, entries) of a table of b rows."""
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32 or table.dim() != 2:
        raise InvalidArgument("table must be an int32 tensor [batch, entries]")
    if table.get_device() != device:
        raise InvalidArgument(f"table is on {table.device}, the cache on GPU {device}")
    if table.shape[0] != b:
        raise InvalidArgument(f"table must have {b} rows (got {tuple(table.shape)})")
    entries = table.shape[1]
    if table.stride(1) != 1 and entries > 1:
        raise InvalidArgument("table: the entries of a sequence must be adjacent")
    return table.data_ptr(), table.stride(0), entries


def _per_sequence(name, t, b, device, optional=False):
    """Pointer of an int32 tensor of one number a sequence."""
    if t is None and optional:
        return 0
    if not isinstance(t, torch.Tensor) or t.shape != (b,):
        raise InvalidArgument(f"{name} must be an int32 tensor of shape {(b,)}")
    return _small(name, t, torch.int32, device)


def _io_pack(cache, kv, kviews, table, start, lens, dtype, device):
    b, t = kv[:2]
    if dtype not in (torch.bfloat16, torch.float16):
        raise InvalidArgument(f"dtype {dtype} is not bf16 or fp16")
    return cache.packed + _IO.pack(b, t, *kviews, *_page_table(table, b, device),
                                   _per_sequence("start", start, b, device),
                                   _per_sequence("lens", lens, b, device, True),
                                   DTYPE_CODES[dtype])


def _write_pack(cache, k, v, table, start, lens):
    device = _pool(cache)
    if not isinstance(k, torch.Tensor):
        raise InvalidArgument("k must be a tensor")
    views = _view("k", k, k.dtype, device) + _view("v", v, k.dtype, device)
    if k.shape != v.shape or k.shape[2] != cache.kv_heads or k.shape[3] != cache.head_dim:
        raise InvalidArgument(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [batch, tokens, "
                              f"{cache.kv_heads}, {cache.head_dim}]")
    return _io_pack(cache, k.shape, views, table, start, lens, k.dtype, device), device


def kv_cache_write_check(cache, k, v, table, start, *, lens=None) -> int:
    """Host-only gate of kv_cache_write: 0 or a decline reason code."""
    return lib().kv_cache_write_check(_write_pack(cache, k, v, table, start, lens)[0])


def kv_cache_write(cache, k, v, table, start, *, lens=None, stream=None):
    """Quantise k and v (bf16 or fp16 [batch, tokens, kv_heads, D], pointers and
    strides multiples of 16 bytes, the values of a head adjacent) into the
    cache: token i < lens[b] (int32 [batch]; None: all) of sequence b goes to
    position start[b] + i (int32 [batch]), which is token p % page_tokens of
    page table[b, p // page_tokens].  Positions past the table and pages
    outside the pool are left out.  The page of a place must not be written
    twice in one call."""
    device = _pool(cache)
    if _fast is not None and stream is None and device == _current_gpu():
        if _fast.kv_cache_write(_entries(), cache.packed, k, v, table, start, lens,
                                _raw_stream(device), device):
            return
    packed, _ = _write_pack(cache, k, v, table, start, lens)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return kv_cache_write(cache, k, v, table, start, lens=lens)
    L = lib()
    rc = L.kv_cache_write(packed, _raw_stream(device))
    if rc != 1:
        _raise("kv_cache_write", rc, L.kv_cache_write_check, packed)


def kv_cache_read(cache, table, start, tokens, *, lens=None, dtype=torch.bfloat16, stream=None):
    """The keys and values that the cache holds at positions start[b] .. start[b]
    + tokens - 1, as dense tensors [batch, tokens, kv_heads, D] of dtype; zeros
    from lens[b] on, NaN where a position or page does not exist."""
    device = _pool(cache)
    if _fast is not None and stream is None and device == _current_gpu():
        r = _fast.kv_cache_read(_entries(), cache.packed, table, start, tokens, lens, dtype,
                                _raw_stream(device), device)
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return kv_cache_read(cache, table, start, tokens, lens=lens, dtype=dtype)
    b = table.shape[0] if isinstance(table, torch.Tensor) and table.dim() else 0
    shape = (b, tokens, cache.kv_heads, cache.head_dim)
    if tokens < 0:
        raise InvalidArgument(f"tokens must not be negative (got {tokens})")
    k = torch.empty(shape, dtype=dtype, device=cache.k.device)
    v = torch.empty_like(k)
    packed = _io_pack(cache, shape, _dense(k, shape) + _dense(v, shape), table, start, lens,
                      dtype, device)
    L = lib()
    rc = L.kv_cache_read(packed, _raw_stream(device))
    if rc != 1:
        _raise("kv_cache_read", rc, L.kv_cache_read_check, packed)
    return k, v


# ------------------------------------------------------- attention over it
def _cattn_pack(q, cache, table, lens, out, lse, causal, scale, ws=(0, 0)):
    """igc_cache_attn, packed.  out: a tensor to check, or the view of a new
    one; lse: a tensor to check, a pointer or None."""
    device = _pool(cache)
    if not isinstance(q, torch.Tensor):
        raise InvalidArgument("q must be a tensor")
    code = _element(q, "q")
    qv = _view("q", q, q.dtype, device)
    b, tq, hq, d = q.shape
    if d != cache.head_dim:
        raise InvalidArgument(f"q has heads of {d}, the cache of {cache.head_dim}")
    if not isinstance(out, tuple):
        o, out = out, _view("out", out, q.dtype, device)
        if o.shape != q.shape:
            raise InvalidArgument(f"out must have q's shape {tuple(q.shape)}")
    if isinstance(lse, torch.Tensor):
        if lse.shape != (b, hq, tq):
            raise InvalidArgument(f"lse must be {(b, hq, tq)} (got {tuple(lse.shape)})")
        lse = _small("lse", lse, torch.float32, device)
    if scale is None:
        scale = d ** -0.5
    return cache.packed + _CATTN.pack(
        b, tq, hq, *qv, *out, lse or 0, *_page_table(table, b, device),
        _per_sequence("lens", lens, b, device), 1 if causal else 0, float(scale), code, *ws)


def cache_attn_fwd(q, cache, table, lens, out, *, lse=None, causal=True, scale=None,
                   workspace=None, workspace_bytes=0, stream=None) -> int:
    """Enqueue the attention over the cache into out (and lse).  1 handled, 0
    declined, < 0 HIP error."""
    device = _pool(cache)
    packed = _cattn_pack(q, cache, table, lens, out, lse, causal, scale,
                         _work(workspace, workspace_bytes, device))
    if _elsewhere(device, stream):
        with _on(device, stream):
            return lib().cache_attn_fwd(packed, _raw_stream(device))
    return lib().cache_attn_fwd(packed, _raw_stream(device))


def cache_attn_fwd_check(q, cache, table, lens, out, *, lse=None, causal=True, scale=None,
                         workspace=None, workspace_bytes=0) -> int:
    """Host-only gate of cache_attn_fwd: 0 or a decline reason code."""
    return lib().cache_attn_fwd_check(
        _cattn_pack(q, cache, table, lens, out, lse, causal, scale,
                    _work(workspace, workspace_bytes, _pool(cache))))


def cache_attn_fwd_workspace_bytes(q_shape, cache, entries, dtype) -> int:
    """Workspace of a call with a table of so many entries a sequence (0 when
    none is needed, or when it would be declined)."""
    b, tq, hq, _ = q_shape
    return lib().cache_attn_fwd_workspace_bytes(
        cache.packed + _CATTN.pack(b, tq, hq, *(0,) * 9, 0, 0, entries, 0, 0, 1.0,
                                   DTYPE_CODES.get(dtype, -1), 0, 0))


def cache_attention(q, cache, table, lens, *, causal=True, scale=None, return_lse=False,
                    stream=None):
    """Attention of new tokens q [batch, tq, hq, D] (kv_heads dividing hq) to
    the lens[b] (int32 [batch]) tokens that sequence b holds in the cache, at
    the places that table (int32 [batch, entries]) gives its positions.  The
    new tokens are the last tq of them (kv_cache_write puts them there first)
    and causal lets token i attend up to its own position only.  scale
    defaults to 1 / sqrt(D).  A row that attends to nothing gives 0, one whose
    scores are all -inf (an infinite query) NaN.  q's pointer and strides are
    multiples of 16 bytes, the values of a head adjacent.  Returns out, dense
    like q, and with return_lse also the fp32 statistics [batch, hq, tq].  No
    gradients: the cache is for inference."""
    device = _pool(cache)
    if _fast is not None and stream is None and device == _current_gpu():
        r = _fast.cache_attention(_entries(), q, cache.packed, table, lens, causal, scale,
                                  return_lse, _raw_stream(device), device)
        if r is not None:
            return r
    if _elsewhere(device, stream):
        with _on(device, stream):
            return cache_attention(q, cache, table, lens, causal=causal, scale=scale,
                                   return_lse=return_lse)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise InvalidArgument("q must be a tensor [batch, token, head, D]")
    out = _like(q)
    lse = None
    if return_lse:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32,
                          device=q.device)
    packed = _cattn_pack(q, cache, table, lens, _dense(out, q.shape),
                         None if lse is None else lse.data_ptr(), causal, scale)
    L = lib()
    need = L.cache_attn_fwd_workspace_bytes(packed)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        packed = packed[:-16] + struct.pack("@qq", ws.data_ptr(), need)
    rc = L.cache_attn_fwd(packed, _raw_stream(device))
    if rc != 1:
        _raise("cache_attn_fwd", rc, L.cache_attn_fwd_check, packed)
    return (out, lse) if return_lse else out
