"""Python binding of an expert layer's operators (``include/dsmem_experts.h``).

Argument marshalling only, like the histogram's binding: ``dsmem_route`` and
``dsmem_route_backward`` choose experts from a router's scores,
``dsmem_group`` orders rows by expert, ``dsmem_grouped_matmul`` (with
``transpose=True`` for the gradient of its rows) and
``dsmem_grouped_matmul_wgrad`` multiply each group with its own matrix,
``dsmem_combine`` and ``dsmem_combine_backward`` bring the rows back to their
tokens, and ``dsmem_grad_clip`` clips gradients by their global norm.

Rows of float inputs are contiguous and may be further apart than their length
(slices of columns); views that repeat rows by a stride of 0, as ``expand``
makes, are refused.

Every call is asynchronous on ``stream`` (default: torch's current stream).
With a ``stream`` given, new outputs belong to it, and inputs are recorded on
it, so their memory is not reused before the call has run; work that produces
the inputs on other streams is the caller's to order.
"""
from __future__ import annotations

import array
import ctypes
import operator

F32, F16, BF16 = 0, 1, 2
_MOST = 2 ** 31 - 1   # of the C entries' 32-bit arguments; ctypes would wrap what lies beyond
_DTYPE = operator.attrgetter("dtype")

_p, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
SIGNATURES = {
    "dsmem_route": [_p, _i32, _i64, _i32, _i64, _i32, _i32, _p, _p, _p],
    "dsmem_route_backward": [_p, _i32, _i64, _i32, _i64, _i32, _i32, _p, _p, _p, _p, _p],
    "dsmem_group": [_p, _i64, _i32, _p, _p, _p, _p],
    "dsmem_grouped_matmul": [_p, _i64, _i64, _p, _i64, _i64, _p, _i32, _p, _i32, _i64, _i32, _i32,
                             _i32, _i32, _p, _i32, _p],
    "dsmem_grouped_matmul_wgrad": [_p, _i64, _p, _i64, _i64, _p, _i32, _p, _i32, _i64, _i32, _i32,
                                   _i32, _p, _i32, _p],
    "dsmem_combine": [_p, _i64, _i64, _p, _p, _i64, _i32, _i32, _i32, _p, _p],
    "dsmem_combine_backward": [_p, _i64, _p, _i64, _p, _p, _p, _i64, _i32, _i32, _i32, _p, _p, _p],
    "dsmem_grad_clip": [_p, _i32, _f32, _p, _p],
    "dsmem_mx4_quantize": [_p, _i32, _i64, _i32, _i64, _p, _p, _p],
    "dsmem_mx4_dequantize": [_p, _p, _i64, _i32, _i32, _p, _p],
    "dsmem_mx4_grouped_matmul": [_p, _p, _i64, _p, _p, _p, _i32, _p, _i32, _i64, _i32, _i32, _p, _i32, _p],
    "dsmem_expert_layer": [_p, _i64, _i32, _i32, _i32, _i32, _p, _i32, _i32, _i64, _i32, _i32, _p, _p, _p,
                           _i32, _p, _p],
}


class _Library:
    """The library's entry points and torch, looked up once."""

    def __getattr__(self, name):
        import torch
        from . import lib
        loaded = lib()
        for fn, args in SIGNATURES.items():
            entry = getattr(loaded, fn)
            entry.argtypes = args
            entry.restype = ctypes.c_int
            self.__dict__[fn] = entry
        self.torch, self.Tensor, self.empty = torch, torch.Tensor, torch.empty
        self.int32, self.float32, self.uint8 = torch.int32, torch.float32, torch.uint8
        self.bfloat16 = torch.bfloat16
        self.device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        return self.__dict__[name]


_lib = _Library()


def _check(rc):
    if rc:
        from . import _check as check
        check(rc)


def _float_tensor(name, t, dims):
    """The type code and device index of a CUDA float tensor of `dims`
    dimensions whose rows are contiguous."""
    if not isinstance(t, _lib.Tensor):
        raise TypeError(f"{name} must be a CUDA float32, float16 or bfloat16 tensor")
    code, index = _lib.codes.get(t.dtype), t.get_device()
    if code is None or index < 0:
        raise TypeError(f"{name} must be a CUDA float32, float16 or bfloat16 tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {t.dim()})")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return code, index


def _like(name, t, dims, code, index):
    """Checks that `t` is such a tensor of the type `code` on device `index`."""
    got = _float_tensor(name, t, dims)
    if got[0] != code:
        raise TypeError(f"{name} has another type than expected (got {t.dtype})")
    if got[1] != index:
        raise ValueError(f"{name} must be on device {index}")


def _out_of_range(**sizes):
    """The error for sizes of which one does not fit a 32-bit argument."""
    name, value = next((n, v) for n, v in sizes.items() if not 0 <= v <= _MOST)
    return ValueError(f"{name} must be in [0, 2^31) (got {value})")


def _row_stride(t, columns):
    """Elements between rows; rows of a single one have no stride of their own."""
    return columns if t.is_contiguous() or t.shape[0] <= 1 else t.stride(0)


def _int_tensor(name, t, count=None, index=None):
    """The device index of a contiguous CUDA int32 tensor of `count` elements."""
    if not isinstance(t, _lib.Tensor) or t.dtype != _lib.int32 or t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA torch.int32 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if count is not None and t.numel() != count:
        raise ValueError(f"{name} must have {count} elements (got {t.numel()})")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}")
    return t.get_device()


def _weights(name, t, shape, index):
    _like(name, t, 2, F32, index)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and of shape {tuple(shape)}")


def _elsewhere(call, device, stream, *args, **options):
    """call(*args, **options) with `device`, and a given `stream`, made current."""
    torch = _lib.torch
    if stream is not None and stream.device != device:
        raise ValueError(f"stream must be on {device}")
    with torch.cuda.device(device):
        if stream is None:
            return call(*args, **options)
        with torch.cuda.stream(stream):
            result = call(*args, **options)
    for t in (*args, *options.values()):
        for each in t if isinstance(t, (list, tuple)) else (t,):
            if isinstance(each, torch.Tensor):
                each.record_stream(stream)
    return result


def _current(index, stream):
    """The current stream's handle, or None where another device or stream is asked for."""
    if stream is not None or index != _lib.device():
        return None
    return _lib.raw_stream(index)


def dsmem_route(logits, top_k: int, renormalize: bool = True, stream=None):
    """Each token's `top_k` experts from its row of `logits` [tokens, experts].

    Returns (ids int32 [tokens, top_k], weights float32 [tokens, top_k]): the
    largest logits, equal ones by lowest index, with their share of the
    softmax over the chosen (`renormalize`) or over all experts.  Logits of
    -inf and NaN are never chosen; missing choices are id -1 with weight 0."""
    dtype, index = _float_tensor("logits", logits, 2)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_route, logits.device, stream, logits, top_k, renormalize)
    tokens, experts = logits.shape
    if experts > _MOST or not 0 <= top_k <= _MOST:
        raise _out_of_range(experts=experts, top_k=top_k)
    shape, device = (tokens, top_k), logits.device
    ids = _lib.empty(shape, dtype=_lib.int32, device=device)
    weights = _lib.empty(shape, dtype=_lib.float32, device=device)
    _check(_lib.dsmem_route(
        logits.data_ptr(), dtype, tokens, experts, _row_stride(logits, experts), int(top_k),
        int(renormalize), ids.data_ptr(), weights.data_ptr(), s))
    return ids, weights


def dsmem_route_backward(logits, ids, weights, grad_weights, renormalize: bool = True, stream=None):
    """Gradient of dsmem_route's weights with respect to `logits` (of its
    type); `ids` and `weights` are the forward call's."""
    dtype, index = _float_tensor("logits", logits, 2)
    tokens, experts = logits.shape
    _int_tensor("ids", ids, None, index)
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    _weights("weights", weights, ids.shape, index)
    _weights("grad_weights", grad_weights, ids.shape, index)
    if experts > _MOST or top_k > _MOST:
        raise _out_of_range(experts=experts, top_k=top_k)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_route_backward, logits.device, stream, logits, ids, weights,
                          grad_weights, renormalize)
    out = _lib.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _check(_lib.dsmem_route_backward(
        logits.data_ptr(), dtype, tokens, experts, _row_stride(logits, experts), top_k,
        int(renormalize), ids.data_ptr(), weights.data_ptr(), grad_weights.data_ptr(),
        out.data_ptr(), s))
    return out


def dsmem_group(keys, num_groups: int, stream=None):
    """Stable order of int32 `keys` by value.  Returns (offsets [num_groups +
    1], order [n], position [n]), int32: group g has the places offsets[g] ..
    offsets[g + 1]; order[p] is the key at place p (-1 behind the last group),
    position[i] the place of key i (-1 for keys outside [0, num_groups))."""
    s = _current(_int_tensor("keys", keys), stream)
    if s is None:
        return _elsewhere(dsmem_group, keys.device, stream, keys, num_groups)
    if not -_MOST <= num_groups <= _MOST:
        raise _out_of_range(num_groups=num_groups)
    n, empty, int32, device = keys.numel(), _lib.empty, _lib.int32, keys.device
    offsets = empty(max(int(num_groups), 0) + 1, dtype=int32, device=device)
    order, position = empty(n, dtype=int32, device=device), empty(n, dtype=int32, device=device)
    _check(_lib.dsmem_group(
        keys.data_ptr(), n, int(num_groups), offsets.data_ptr(), order.data_ptr(),
        position.data_ptr(), s))
    return offsets, order, position


def _out_type(code, dtype, out_dtype):
    """The output's type and its code, for a product's inputs of type `dtype`."""
    if code == F32:
        raise TypeError("grouped products take float16 or bfloat16")
    if out_dtype is None or out_dtype == dtype:
        return dtype, code
    if out_dtype != _lib.float32:
        raise TypeError("out_dtype must be the inputs' type or torch.float32")
    return out_dtype, F32


def dsmem_grouped_matmul(x, weight, offsets, order=None, fan: int = 1, transpose: bool = False,
                         out_dtype=None, stream=None):
    """Row p of the result is x[row(p)] @ weight[g].T (with `transpose`:
    x[row(p)] @ weight[g]) for the group g that holds place p, where row(p) is
    order[p] // fan, or p without `order`.  weight is [groups, outer, inner];
    places of no group give zeros."""
    code, index = _float_tensor("x", x, 2)
    _like("weight", weight, 3, code, index)
    groups, outer, inner = weight.shape
    rows, columns = x.shape
    if max(groups, outer, inner) > _MOST or not -_MOST <= fan <= _MOST:
        raise _out_of_range(groups=groups, outer=outer, inner=inner, fan=fan)
    depth, cols = (outer, inner) if transpose else (inner, outer)
    if columns != depth:
        raise ValueError(f"x must have {depth} columns (got {columns})")
    dtype, out_code = _out_type(code, x.dtype, out_dtype)
    _int_tensor("offsets", offsets, groups + 1, index)
    n, named = rows, None
    if order is not None:
        _int_tensor("order", order, None, index)
        n, named = order.numel(), order.data_ptr()
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_grouped_matmul, x.device, stream, x, weight, offsets, order, fan,
                          transpose, out_dtype)
    out = _lib.empty((n, cols), dtype=dtype, device=x.device)
    between, row = outer * inner, inner
    if not weight.is_contiguous():
        between = weight.stride(0) if groups > 1 else between
        row = weight.stride(1) if outer > 1 else row
    _check(_lib.dsmem_grouped_matmul(
        x.data_ptr(), rows, _row_stride(x, columns), weight.data_ptr(), row, between,
        offsets.data_ptr(), groups, named, int(fan), n, outer, inner, int(transpose), code,
        out.data_ptr(), out_code, s))
    return out


def dsmem_grouped_matmul_wgrad(dy, x, offsets, order=None, fan: int = 1, out_dtype=None,
                               stream=None):
    """Gradient of dsmem_grouped_matmul(x, weight, ...) with respect to its
    weight [groups, outer, inner]: out[g] = sum over the places p of group g of
    dy[p]^T x[row(p)]."""
    code, index = _float_tensor("dy", dy, 2)
    _like("x", x, 2, code, index)
    dtype, out_code = _out_type(code, dy.dtype, out_dtype)
    _int_tensor("offsets", offsets, None, index)
    (n, outer), (rows, inner), groups = dy.shape, x.shape, offsets.numel() - 1
    if max(groups, outer, inner) > _MOST or not -_MOST <= fan <= _MOST:
        raise _out_of_range(groups=groups, outer=outer, inner=inner, fan=fan)
    if order is not None:
        _int_tensor("order", order, n, index)
    elif rows != n:
        raise ValueError(f"x must have {n} rows (got {rows})")
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_grouped_matmul_wgrad, dy.device, stream, dy, x, offsets, order,
                          fan, out_dtype)
    out = _lib.empty((groups, outer, inner), dtype=dtype, device=dy.device)
    _check(_lib.dsmem_grouped_matmul_wgrad(
        dy.data_ptr(), _row_stride(dy, outer), x.data_ptr(), rows, _row_stride(x, inner),
        offsets.data_ptr(), groups, None if order is None else order.data_ptr(), int(fan), n,
        outer, inner, code, out.data_ptr(), out_code, s))
    return out


def dsmem_combine(z, position, weights=None, stream=None):
    """out[t] = sum over j of weights[t, j] * z[position[t, j]] (weights of 1
    when None); positions outside z are dropped."""
    dtype, index = _float_tensor("z", z, 2)
    _int_tensor("position", position, None, index)
    if position.dim() != 2:
        raise ValueError("position must be [tokens, top_k]")
    if weights is not None:
        _weights("weights", weights, position.shape, index)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_combine, z.device, stream, z, position, weights)
    (tokens, top_k), (rows, width) = position.shape, z.shape
    if max(top_k, width) > _MOST:
        raise _out_of_range(top_k=top_k, width=width)
    out = _lib.empty((tokens, width), dtype=z.dtype, device=z.device)
    _check(_lib.dsmem_combine(
        z.data_ptr(), rows, _row_stride(z, width), position.data_ptr(),
        None if weights is None else weights.data_ptr(), tokens, top_k, width, dtype,
        out.data_ptr(), s))
    return out


def dsmem_combine_backward(dy, z, position, order, weights, stream=None):
    """Gradients (dz, dweights) of dsmem_combine; `position` and `order` are
    one dsmem_group call's, `weights` ones for a combination without."""
    dtype, index = _float_tensor("dy", dy, 2)
    _like("z", z, 2, dtype, index)
    _int_tensor("position", position, None, index)
    if position.dim() != 2:
        raise ValueError("position must be [tokens, top_k]")
    _weights("weights", weights, position.shape, index)
    (tokens, top_k), (rows, width) = position.shape, z.shape
    if max(top_k, width) > _MOST:
        raise _out_of_range(top_k=top_k, width=width)
    if dy.shape != (tokens, width):
        raise ValueError(f"dy must be [{tokens}, {width}]")
    if rows != tokens * top_k:
        raise ValueError(f"z must have {tokens * top_k} rows (got {rows})")
    _int_tensor("order", order, rows, index)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_combine_backward, dy.device, stream, dy, z, position, order,
                          weights)
    dz = _lib.empty((rows, width), dtype=z.dtype, device=z.device)
    dweights = _lib.empty((tokens, top_k), dtype=_lib.float32, device=z.device)
    _check(_lib.dsmem_combine_backward(
        dy.data_ptr(), _row_stride(dy, width), z.data_ptr(), _row_stride(z, width),
        position.data_ptr(), order.data_ptr(), weights.data_ptr(), tokens, top_k, width, dtype,
        dz.data_ptr(), dweights.data_ptr(), s))
    return dz, dweights


def _mx4_tensors(name, pair, dims, index=None):
    """The device index of a pair (values, scales) of 4-bit rows, contiguous
    CUDA uint8 tensors whose last dimensions belong together."""
    got = other = -1
    if isinstance(pair, (tuple, list)) and len(pair) == 2:
        values, scales = pair
        if isinstance(values, _lib.Tensor) and isinstance(scales, _lib.Tensor) \
                and values.dtype is scales.dtype is _lib.uint8:
            got, other = values.get_device(), scales.get_device()
    if got < 0 or other < 0:
        raise TypeError(f"{name} must be a pair (values, scales) of CUDA torch.uint8 tensors")
    shape, of_scales = values.shape, scales.shape
    if dims is not None and len(shape) != dims or len(shape) < 1:
        raise ValueError(f"{name}'s values must have {dims or 'some'} dimensions (got {len(shape)})")
    if len(of_scales) != len(shape) or shape[-1] != 16 * of_scales[-1] or shape[-1] % 64 or shape[-1] == 0 \
            or shape[:-1] != of_scales[:-1]:
        raise ValueError(f"{name}'s values and scales must have rows of 64 and 4 bytes for each 128 elements")
    if not values.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if other != got or index is not None and index != got:
        raise ValueError(f"{name} must be on one device" if index is None else f"{name} must be on device {index}")
    return got


def dsmem_mx4_quantize(x, stream=None):
    """Rows of floats [..., columns] to microscaled 4-bit elements: e2m1 values
    with a power-of-two scale of each 32.  Returns (values, scales), uint8 [...,
    64 * q] and [..., 4 * q] for q = ceil(columns / 128); what is behind a row's
    end is zero.  More than one leading dimension must be viewable as one."""
    flat = x
    if isinstance(x, _lib.Tensor) and x.dim() != 2:
        if x.dim() < 1 or x.shape[-1] < 1:
            raise ValueError("x must have rows of one column or more")
        flat = x.view(-1, x.shape[-1])
    dtype, index = _float_tensor("x", flat, 2)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_mx4_quantize, x.device, stream, x)
    rows, columns = flat.shape
    if columns > _MOST:
        raise _out_of_range(columns=columns)
    quads, device = (columns + 127) // 128, x.device
    lead = (rows,) if flat is x else x.shape[:-1]
    values = _lib.empty((*lead, 64 * quads), dtype=_lib.uint8, device=device)
    scales = _lib.empty((*lead, 4 * quads), dtype=_lib.uint8, device=device)
    _check(_lib.dsmem_mx4_quantize(
        flat.data_ptr(), dtype, rows, columns, _row_stride(flat, columns), values.data_ptr(),
        scales.data_ptr(), s))
    return values, scales


def dsmem_mx4_dequantize(values, scales, columns=None, dtype=None, stream=None):
    """The floats that 4-bit rows stand for, [..., columns] (default: all, with
    what pads them), in `dtype` (default torch.float32)."""
    index = _mx4_tensors("values and scales", (values, scales), None)
    most = 2 * values.shape[-1]
    columns = most if columns is None else columns
    if not most - 128 < columns <= most:
        raise ValueError(f"columns must be in ({most - 128}, {most}] (got {columns})")
    dtype = _lib.float32 if dtype is None else dtype
    code = _lib.codes.get(dtype)
    if code is None:
        raise TypeError("dtype must be torch.float32, torch.float16 or torch.bfloat16")
    if columns > _MOST:
        raise _out_of_range(columns=columns)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_mx4_dequantize, values.device, stream, values, scales, columns, dtype)
    out = _lib.empty((*values.shape[:-1], columns), dtype=dtype, device=values.device)
    _check(_lib.dsmem_mx4_dequantize(
        values.data_ptr(), scales.data_ptr(), values.numel() // values.shape[-1], columns, code,
        out.data_ptr(), s))
    return out


def dsmem_mx4_grouped_matmul(x, weight, offsets, order=None, fan: int = 1, out_dtype=None, stream=None):
    """dsmem_grouped_matmul of 4-bit rows with 4-bit matrices: x and weight are
    pairs (values, scales) of dsmem_mx4_quantize, of [rows, inner] and [groups,
    outer, inner].  The result has `out_dtype` (default torch.bfloat16)."""
    index = _mx4_tensors("x", x, 2)
    _mx4_tensors("weight", weight, 3, index)
    (x_values, x_scales), (w_values, w_scales) = x, weight
    (rows, pitch), (groups, outer, w_pitch) = x_values.shape, w_values.shape
    if pitch != w_pitch:
        raise ValueError(f"x and weight must have rows of one length (got {pitch} and {w_pitch} bytes)")
    if max(groups, outer, 2 * pitch) > _MOST or not -_MOST <= fan <= _MOST:
        raise _out_of_range(groups=groups, outer=outer, inner=2 * pitch, fan=fan)
    dtype = _lib.bfloat16 if out_dtype is None else out_dtype
    code = _lib.codes.get(dtype)
    if code is None:
        raise TypeError("out_dtype must be torch.float32, torch.float16 or torch.bfloat16")
    _int_tensor("offsets", offsets, groups + 1, index)
    n, named = rows, None
    if order is not None:
        _int_tensor("order", order, None, index)
        n, named = order.numel(), order.data_ptr()
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_mx4_grouped_matmul, x_values.device, stream, x, weight, offsets, order, fan, dtype)
    out = _lib.empty((n, outer), dtype=dtype, device=x_values.device)
    _check(_lib.dsmem_mx4_grouped_matmul(
        x_values.data_ptr(), x_scales.data_ptr(), rows, w_values.data_ptr(), w_scales.data_ptr(),
        offsets.data_ptr(), groups, named, int(fan), n, outer, 2 * pitch, out.data_ptr(), code, s))
    return out


_ACTIVATIONS = {"relu": 0, "silu": 1}


def _layer_matrices(name, m, shape, code, index):
    """The words of a dsmem_matrices_t for matrices of `shape`, 16-bit ones of
    the type `code` or a pair of 4-bit tensors."""
    if not isinstance(m, (tuple, list)):
        _like(name, m, 3, code, index)
        if m.shape != shape:
            raise ValueError(f"{name} must be of shape {tuple(shape)} (got {tuple(m.shape)})")
        experts, rows, columns = shape
        if m.is_contiguous():
            return m.data_ptr(), 0, columns, rows * columns
        return (m.data_ptr(), 0, m.stride(1) if rows > 1 else columns,
                m.stride(0) if experts > 1 else rows * columns)
    _mx4_tensors(name, m, 3, index)
    values, scales = m
    want = (*shape[:2], (shape[2] + 127) // 128 * 64)
    if values.shape != want:
        raise ValueError(f"{name}'s values must be of shape {want} (got {tuple(values.shape)})")
    return values.data_ptr(), scales.data_ptr(), 0, 0


def dsmem_expert_layer(x, logits, up, down, top_k: int, gate=None, activation: str = "relu",
                       renormalize: bool = True, stream=None):
    """A whole expert layer for up to 64 tokens x [tokens, width], as when
    decoding: with ids and weights those of dsmem_route(logits, top_k,
    renormalize), the sum over each token's experts e of weight * down[e] h, where
    h = act(up[e] x), or act(gate[e] x) * (up[e] x) with a `gate`.

    up and gate are [experts, hidden, width], down [experts, width, hidden]: all
    three tensors of x's type (float16 or bfloat16), or all pairs (values,
    scales) of dsmem_mx4_quantize.  `activation` is "relu" or "silu"."""
    code, index = _float_tensor("x", x, 2)
    if code == F32:
        raise TypeError("x must be a CUDA float16 or bfloat16 tensor")
    logits_code, _ = got = _float_tensor("logits", logits, 2)
    if got[1] != index:
        raise ValueError(f"logits must be on device {index}")
    (tokens, width), experts = x.shape, logits.shape[1]
    if logits.shape[0] != tokens:
        raise ValueError(f"logits must have {tokens} rows (got {logits.shape[0]})")
    kind = _ACTIVATIONS.get(activation)
    if kind is None:
        raise ValueError('activation must be "relu" or "silu"')
    first = up[0] if isinstance(up, (tuple, list)) and up else up
    if not isinstance(first, _lib.Tensor) or first.dim() != 3:
        raise TypeError("up must be a tensor of 3 dimensions or a pair of such (values, scales)")
    hidden = first.shape[1]
    if max(tokens, width, hidden, experts) > _MOST or not 0 <= top_k <= _MOST:
        raise _out_of_range(tokens=tokens, width=width, hidden=hidden, experts=experts, top_k=top_k)
    s = _current(index, stream)
    if s is None:
        return _elsewhere(dsmem_expert_layer, x.device, stream, x, logits, up, down, top_k, gate,
                          activation, renormalize)
    words = array.array("Q", _layer_matrices("up", up, (experts, hidden, width), code, index)
                        + _layer_matrices("down", down, (experts, width, hidden), code, index))
    if gate is not None:
        words.extend(_layer_matrices("gate", gate, (experts, hidden, width), code, index))
    out = _lib.empty((tokens, width), dtype=x.dtype, device=x.device)
    at = words.buffer_info()[0]
    _check(_lib.dsmem_expert_layer(
        x.data_ptr(), _row_stride(x, width), code, tokens, width, hidden, logits.data_ptr(), logits_code,
        experts, _row_stride(logits, experts), int(top_k), int(renormalize), at,
        None if gate is None else at + 64, at + 32, kind, out.data_ptr(), s))
    return out


def dsmem_grad_clip(grads, max_norm: float, out=None, stream=None):
    """Global norm of `grads` (a list of contiguous CUDA tensors), returned as
    a float32 tensor without dimensions; the gradients times min(1, max_norm /
    (norm + 1e-6)) go to `out`, a list of tensors of their types and sizes, or
    in place.  max_norm is positive and finite; the largest float32 gives the
    norm alone."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError("out must have one tensor for each gradient")
    tensor = _lib.Tensor
    types = list(map(_DTYPE, grads))
    codes = list(map(_lib.codes.get, types))
    counts = list(map(tensor.numel, grads))
    devices = set(map(tensor.get_device, grads)) or {_lib.torch.cuda.current_device()}
    if None in codes or -1 in devices:
        raise TypeError("grads must be CUDA float32, float16 or bfloat16 tensors")
    if len(devices) > 1 or not all(map(tensor.is_contiguous, grads)):
        raise ValueError("grads must be contiguous and on one device")
    if out is not grads and (
            list(map(_DTYPE, out)) != types or list(map(tensor.numel, out)) != counts
            or not devices.issuperset(map(tensor.get_device, out))
            or not all(map(tensor.is_contiguous, out))):
        raise ValueError("out must match grads in type, size and device and be contiguous")
    device = _lib.torch.device("cuda", *devices)
    s = _current(device.index, stream)
    if s is None:
        return _elsewhere(dsmem_grad_clip, device, stream, grads, max_norm, out)
    words = array.array("Q", bytes(32 * max(len(grads), 1)))   # entries of dsmem_grad_t
    end = 4 * len(grads)
    words[0:end:4] = array.array("Q", map(tensor.data_ptr, grads))
    words[1:end:4] = array.array("Q", map(tensor.data_ptr, out))
    words[2:end:4] = array.array("Q", counts)
    words[3:end:4] = array.array("Q", codes)
    norm = _lib.empty((), dtype=_lib.float32, device=device)
    _check(_lib.dsmem_grad_clip(
        words.buffer_info()[0], len(grads), float(max_norm), norm.data_ptr(), s))
    return norm
