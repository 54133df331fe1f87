"""Python binding of an expert layer's operators (``include/dsmem_experts.h``).

Argument marshalling only, like the histogram's binding: ``dsmem_route`` and
``dsmem_route_backward`` choose experts from a router's scores,
``dsmem_group`` orders rows by expert, ``dsmem_grouped_matmul`` (with
``transpose=True`` for the gradient of its rows) and
``dsmem_grouped_matmul_wgrad`` multiply each group with its own matrix,
``dsmem_combine`` and ``dsmem_combine_backward`` bring the rows back to their
tokens, and ``dsmem_grad_clip`` clips gradients by their global norm.

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
        self.torch = torch
        self.device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        return self.__dict__[name]


_lib = _Library()


def _check(rc):
    if rc:
        from . import _check as check
        check(rc)


def _float_tensor(name, t, dims, dtype=None):
    """The type code of a CUDA float tensor of `dims` dimensions whose rows
    are contiguous."""
    if not isinstance(t, _lib.torch.Tensor) or not t.is_cuda or t.dtype not in _lib.codes:
        raise TypeError(f"{name} must be a CUDA float32, float16 or bfloat16 tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {t.dim()})")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return _lib.codes[t.dtype]


def _row_stride(t):
    """Elements between rows; rows of a single one have no stride of their own."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _int_tensor(name, t, count, device):
    if not isinstance(t, _lib.torch.Tensor) or t.dtype != _lib.torch.int32 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA torch.int32 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if count is not None and t.numel() != count:
        raise ValueError(f"{name} must have {count} elements (got {t.numel()})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


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
        for each in t if isinstance(t, list) else (t,):
            if isinstance(each, torch.Tensor):
                each.record_stream(stream)
    return result


def _current(device):
    """The current stream's handle, or None when `device` is not the current one."""
    index = device.index
    if index != _lib.device():
        return None
    return _lib.raw_stream(index)


def dsmem_route(logits, top_k: int, renormalize: bool = True, stream=None):
    """Each token's `top_k` experts from its row of `logits` [tokens, experts].

    Returns (ids int32 [tokens, top_k], weights float32 [tokens, top_k]): the
    largest logits, equal ones by lowest index, with their share of the
    softmax over the chosen (`renormalize`) or over all experts.  Logits of
    -inf and NaN are never chosen; missing choices are id -1 with weight 0."""
    dtype = _float_tensor("logits", logits, 2)
    tokens, experts = logits.shape
    s = None if stream is not None else _current(logits.device)
    if s is None:
        return _elsewhere(dsmem_route, logits.device, stream, logits, top_k, renormalize)
    ids = _lib.torch.empty((tokens, top_k), dtype=_lib.torch.int32, device=logits.device)
    weights = _lib.torch.empty((tokens, top_k), dtype=_lib.torch.float32, device=logits.device)
    _check(_lib.dsmem_route(
        logits.data_ptr(), dtype, tokens, experts, _row_stride(logits), int(top_k),
        int(renormalize), ids.data_ptr(), weights.data_ptr(), s))
    return ids, weights


def dsmem_route_backward(logits, ids, weights, grad_weights, renormalize: bool = True, stream=None):
    """Gradient of dsmem_route's weights with respect to `logits` (of its
    type); `ids` and `weights` are the forward call's."""
    dtype = _float_tensor("logits", logits, 2)
    tokens, experts = logits.shape
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    _int_tensor("ids", ids, None, logits.device)
    for name, t in (("weights", weights), ("grad_weights", grad_weights)):
        _float_tensor(name, t, 2, _lib.torch.float32)
        if t.shape != ids.shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and of the shape of ids")
    _same_device(logits.device, weights=weights, grad_weights=grad_weights)
    s = None if stream is not None else _current(logits.device)
    if s is None:
        return _elsewhere(dsmem_route_backward, logits.device, stream, logits, ids, weights,
                          grad_weights, renormalize)
    out = _lib.torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _check(_lib.dsmem_route_backward(
        logits.data_ptr(), dtype, tokens, experts, _row_stride(logits), top_k,
        int(renormalize), ids.data_ptr(), weights.data_ptr(), grad_weights.data_ptr(),
        out.data_ptr(), s))
    return out


def dsmem_group(keys, num_groups: int, stream=None):
    """Stable order of int32 `keys` by value.  Returns (offsets [num_groups +
    1], order [n], position [n]), int32: group g has the places offsets[g] ..
    offsets[g + 1]; order[p] is the key at place p (-1 behind the last group),
    position[i] the place of key i (-1 for keys outside [0, num_groups))."""
    _int_tensor("keys", keys, None, None)
    n = keys.numel()
    s = None if stream is not None else _current(keys.device)
    if s is None:
        return _elsewhere(dsmem_group, keys.device, stream, keys, num_groups)
    torch = _lib.torch
    like = dict(dtype=torch.int32, device=keys.device)
    offsets = torch.empty(max(int(num_groups), 0) + 1, **like)
    order, position = torch.empty(n, **like), torch.empty(n, **like)
    _check(_lib.dsmem_group(
        keys.data_ptr(), n, int(num_groups), offsets.data_ptr(), order.data_ptr(),
        position.data_ptr(), s))
    return offsets, order, position


def _product_types(code, dtype, out_dtype):
    """The output's type and its code, for inputs of the type `dtype`."""
    if code == F32:
        raise TypeError("grouped products take float16 or bfloat16")
    if out_dtype is None or out_dtype == dtype:
        return dtype, code
    if out_dtype != _lib.torch.float32:
        raise TypeError("out_dtype must be the inputs' type or torch.float32")
    return out_dtype, F32


def dsmem_grouped_matmul(x, weight, offsets, order=None, fan: int = 1, transpose: bool = False,
                         out_dtype=None, stream=None):
    """Row p of the result is x[row(p)] @ weight[g].T (with `transpose`:
    x[row(p)] @ weight[g]) for the group g that holds place p, where row(p) is
    order[p] // fan, or p without `order`.  weight is [groups, outer, inner];
    places of no group give zeros."""
    dtype = _float_tensor("x", x, 2)
    _float_tensor("weight", weight, 3, x.dtype)
    groups, outer, inner = weight.shape
    depth, cols = (outer, inner) if transpose else (inner, outer)
    if x.shape[1] != depth:
        raise ValueError(f"x must have {depth} columns (got {x.shape[1]})")
    out_dtype, out_code = _product_types(dtype, x.dtype, out_dtype)
    _int_tensor("offsets", offsets, groups + 1, x.device)
    if order is not None:
        _int_tensor("order", order, None, x.device)
    _same_device(x.device, weight=weight)
    n = x.shape[0] if order is None else order.numel()
    s = None if stream is not None else _current(x.device)
    if s is None:
        return _elsewhere(dsmem_grouped_matmul, x.device, stream, x, weight, offsets, order, fan,
                          transpose, out_dtype)
    out = _lib.torch.empty((n, cols), dtype=out_dtype, device=x.device)
    _check(_lib.dsmem_grouped_matmul(
        x.data_ptr(), x.shape[0], _row_stride(x), weight.data_ptr(), weight.stride(1) if outer
        > 1 else inner, weight.stride(0) if groups > 1 else outer * inner, offsets.data_ptr(),
        groups, None if order is None else order.data_ptr(), int(fan), n, outer, inner,
        int(transpose), dtype, out.data_ptr(), out_code, s))
    return out


def dsmem_grouped_matmul_wgrad(dy, x, offsets, order=None, fan: int = 1, out_dtype=None,
                               stream=None):
    """Gradient of dsmem_grouped_matmul(x, weight, ...) with respect to its
    weight [groups, outer, inner]: out[g] = sum over the places p of group g of
    dy[p]^T x[row(p)]."""
    dtype = _float_tensor("dy", dy, 2)
    _float_tensor("x", x, 2, dy.dtype)
    out_dtype, out_code = _product_types(dtype, dy.dtype, out_dtype)
    _int_tensor("offsets", offsets, None, dy.device)
    n, outer, inner, groups = dy.shape[0], dy.shape[1], x.shape[1], offsets.numel() - 1
    if order is not None:
        _int_tensor("order", order, n, dy.device)
    elif x.shape[0] != n:
        raise ValueError(f"x must have {n} rows (got {x.shape[0]})")
    _same_device(dy.device, x=x)
    s = None if stream is not None else _current(dy.device)
    if s is None:
        return _elsewhere(dsmem_grouped_matmul_wgrad, dy.device, stream, dy, x, offsets, order,
                          fan, out_dtype)
    out = _lib.torch.empty((groups, outer, inner), dtype=out_dtype, device=dy.device)
    _check(_lib.dsmem_grouped_matmul_wgrad(
        dy.data_ptr(), _row_stride(dy), x.data_ptr(), x.shape[0], _row_stride(x),
        offsets.data_ptr(), groups, None if order is None else order.data_ptr(), int(fan), n,
        outer, inner, dtype, out.data_ptr(), out_code, s))
    return out


def _positions(position, weights):
    _int_tensor("position", position, None, None)
    if position.dim() != 2:
        raise ValueError("position must be [tokens, top_k]")
    if weights is not None:
        _float_tensor("weights", weights, 2, _lib.torch.float32)
        if weights.shape != position.shape or not weights.is_contiguous():
            raise ValueError("weights must be contiguous and of the shape of position")


def dsmem_combine(z, position, weights=None, stream=None):
    """out[t] = sum over j of weights[t, j] * z[position[t, j]] (weights of 1
    when None); positions outside z are dropped."""
    dtype = _float_tensor("z", z, 2)
    _positions(position, weights)
    _same_device(z.device, position=position, weights=weights)
    (tokens, top_k), width = position.shape, z.shape[1]
    s = None if stream is not None else _current(z.device)
    if s is None:
        return _elsewhere(dsmem_combine, z.device, stream, z, position, weights)
    out = _lib.torch.empty((tokens, width), dtype=z.dtype, device=z.device)
    _check(_lib.dsmem_combine(
        z.data_ptr(), z.shape[0], _row_stride(z), position.data_ptr(), None if weights is None
        else weights.data_ptr(), tokens, top_k, width, dtype, out.data_ptr(), s))
    return out


def dsmem_combine_backward(dy, z, position, order, weights, stream=None):
    """Gradients (dz, dweights) of dsmem_combine; `position` and `order` are
    one dsmem_group call's."""
    _float_tensor("dy", dy, 2)
    dtype = _float_tensor("z", z, 2, dy.dtype)
    _positions(position, weights)
    if weights is None:
        raise TypeError("weights must be a CUDA float32 tensor")
    (tokens, top_k), width = position.shape, z.shape[1]
    if dy.shape != (tokens, width):
        raise ValueError(f"dy must be [{tokens}, {width}]")
    if z.shape[0] != tokens * top_k:
        raise ValueError(f"z must have {tokens * top_k} rows (got {z.shape[0]})")
    _int_tensor("order", order, tokens * top_k, dy.device)
    _same_device(dy.device, z=z, position=position, weights=weights)
    s = None if stream is not None else _current(dy.device)
    if s is None:
        return _elsewhere(dsmem_combine_backward, dy.device, stream, dy, z, position, order,
                          weights)
    dz = _lib.torch.empty((tokens * top_k, width), dtype=z.dtype, device=z.device)
    dweights = _lib.torch.empty((tokens, top_k), dtype=_lib.torch.float32, device=z.device)
    _check(_lib.dsmem_combine_backward(
        dy.data_ptr(), _row_stride(dy), z.data_ptr(), _row_stride(z), position.data_ptr(),
        order.data_ptr(), weights.data_ptr(), tokens, top_k, width, dtype, dz.data_ptr(),
        dweights.data_ptr(), s))
    return dz, dweights


def dsmem_grad_clip(grads, max_norm: float, out=None, stream=None):
    """Global norm of `grads` (a list of contiguous CUDA tensors), returned as
    a float32 tensor without dimensions; the gradients times min(1, max_norm /
    (norm + 1e-6)) go to `out`, a list of tensors of their types and sizes, or
    in place."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError("out must have one tensor for each gradient")
    torch, tensor = _lib.torch, _lib.torch.Tensor
    device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
    types = list(map(_DTYPE, grads))
    codes = list(map(_lib.codes.get, types))
    counts = list(map(tensor.numel, grads))
    devices = set(map(tensor.get_device, grads))
    if None in codes or -1 in devices:
        raise TypeError("grads must be CUDA float32, float16 or bfloat16 tensors")
    if len(devices) > 1 or not all(map(tensor.is_contiguous, grads)):
        raise ValueError("grads must be contiguous and on one device")
    if out is not grads and (
            list(map(_DTYPE, out)) != types or list(map(tensor.numel, out)) != counts
            or set(map(tensor.get_device, out)) != devices
            or not all(map(tensor.is_contiguous, out))):
        raise ValueError("out must match grads in type, size and device and be contiguous")
    table = array.array("Q", bytes(32 * max(len(grads), 1)))   # entries of dsmem_grad_t
    table[0:4 * len(grads):4] = array.array("Q", map(tensor.data_ptr, grads))
    table[1:4 * len(grads):4] = array.array("Q", map(tensor.data_ptr, out))
    table[2:4 * len(grads):4] = array.array("Q", counts)
    table[3:4 * len(grads):4] = array.array("Q", codes)
    s = None if stream is not None else _current(device)
    if s is None:
        return _elsewhere(dsmem_grad_clip, device, stream, grads, max_norm, out)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _check(_lib.dsmem_grad_clip(
        table.buffer_info()[0], len(grads), float(max_norm), norm.data_ptr(), s))
    return norm
