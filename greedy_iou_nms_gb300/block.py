"""Operators of a transformer block among a detector's candidates, forward and
backward: linear layer with activation and residual, layer normalisation with
the residual stream, and rotary positions on several axes.

The raw entry points carry the names of the C functions (device addresses as
ints, the status code returned); the functions below them work on CUDA
tensors, run on their device's current stream and never synchronise.
greedy_iou_nms_gb300.autograd has the same operators for torch's autograd.
"""
from __future__ import annotations

import ctypes
import decimal
import functools

from . import head
from .head import (NMS_TYPE_F32, _ACTS, _launch, _lib, _like, _raise, _same, _type, _types)

NMS_LAYER_MAX_WIDTH = 16384
NMS_LINEAR_MAX_WIDTH = 1 << 20
NMS_ROTARY_MAX_AXES = 8
NMS_ROTARY_MAX_DIM = 4096
NMS_POSITION_I32 = 16

EXPORTED = ("nms_linear_workspace_size", "nms_linear_run", "nms_linear_grad_workspace_size", "nms_linear_grad_run",
            "nms_layer_norm_run", "nms_layer_norm_workspace_size", "nms_layer_norm_grad_run", "nms_rotary_run")


def declare(lib) -> None:
    """Argument types of the entry points (called once by load())."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    psz = ctypes.POINTER(ctypes.c_size_t)
    for name, args in (
            ("nms_linear_workspace_size", [i32, i64, i32, i32, i32, psz]),
            ("nms_linear_run", [vp, i64, i32, i64, i32, vp, i64, i32, vp, i32, i32, vp, i64, vp, vp, vp, vp, sz, vp]),
            ("nms_linear_grad_workspace_size", [i32, i64, i32, i32, i32, psz]),
            ("nms_linear_grad_run", [vp, i64, vp, i64, i32, i64, i32, vp, i64, i32, vp, i32, vp, vp, vp, vp, vp, sz,
                                     vp]),
            ("nms_layer_norm_run", [vp, i64, vp, i64, i32, i64, i32, vp, vp, i32, f32, vp, vp, vp, vp, vp]),
            ("nms_layer_norm_workspace_size", [i64, i32, psz]),
            ("nms_layer_norm_grad_run", [vp, i64, vp, i64, vp, i64, i32, i64, i32, vp, vp, vp, i32, vp, vp, vp, vp,
                                         sz, vp]),
            ("nms_rotary_run", [vp, i64, i64, i64, i32, i64, i64, i32, i32, vp, i32, i64, i32, vp, i32, i32, i32, vp,
                                i64, i64, i64, vp])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


# ------------------------------------------------------------- raw C entries

@functools.lru_cache(maxsize=4096)
def nms_linear_workspace_size(type: int, rows: int, inner: int, outer: int, aligned: int) -> int:
    out = ctypes.c_size_t(0)
    st = _lib().nms_linear_workspace_size(type, rows, inner, outer, aligned, ctypes.byref(out))
    if st:
        _raise(st, "nms_linear_workspace_size")
    return out.value


def nms_linear_run(x: int, x_row: int, type: int, rows: int, inner: int, weight: int, weight_row: int, outer: int,
                   bias: int, bias_type: int, act: int, residual: int, residual_row: int, y: int, pre: int,
                   dev_status: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().nms_linear_run(x or None, x_row, type, rows, inner, weight or None, weight_row, outer, bias or None,
                                 bias_type, act, residual or None, residual_row, y or None, pre or None,
                                 dev_status or None, workspace or None, workspace_bytes, stream or None)


@functools.lru_cache(maxsize=4096)
def nms_linear_grad_workspace_size(type: int, rows: int, inner: int, outer: int, aligned: int) -> int:
    out = ctypes.c_size_t(0)
    st = _lib().nms_linear_grad_workspace_size(type, rows, inner, outer, aligned, ctypes.byref(out))
    if st:
        _raise(st, "nms_linear_grad_workspace_size")
    return out.value


def nms_linear_grad_run(dy: int, dy_row: int, x: int, x_row: int, type: int, rows: int, inner: int, weight: int,
                        weight_row: int, outer: int, pre: int, act: int, dx: int, dweight: int, dbias: int,
                        dev_status: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().nms_linear_grad_run(dy or None, dy_row, x or None, x_row, type, rows, inner, weight or None,
                                      weight_row, outer, pre or None, act, dx or None, dweight or None, dbias or None,
                                      dev_status or None, workspace or None, workspace_bytes, stream or None)


def nms_layer_norm_run(x: int, x_row: int, residual: int, residual_row: int, type: int, rows: int, width: int,
                       weight: int, bias: int, param_type: int, eps: float, y: int, sum: int, mean: int, rstd: int,
                       stream: int) -> int:
    return _lib().nms_layer_norm_run(x or None, x_row, residual or None, residual_row, type, rows, width,
                                     weight or None, bias or None, param_type, eps, y or None, sum or None,
                                     mean or None, rstd or None, stream or None)


@functools.lru_cache(maxsize=4096)
def nms_layer_norm_workspace_size(rows: int, width: int) -> int:
    out = ctypes.c_size_t(0)
    st = _lib().nms_layer_norm_workspace_size(rows, width, ctypes.byref(out))
    if st:
        _raise(st, "nms_layer_norm_workspace_size")
    return out.value


def nms_layer_norm_grad_run(dy: int, dy_row: int, x: int, x_row: int, dsum: int, dsum_row: int, type: int, rows: int,
                            width: int, mean: int, rstd: int, weight: int, param_type: int, dx: int, dweight: int,
                            dbias: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().nms_layer_norm_grad_run(dy or None, dy_row, x or None, x_row, dsum or None, dsum_row, type, rows,
                                          width, mean or None, rstd or None, weight or None, param_type, dx or None,
                                          dweight or None, dbias or None, workspace or None, workspace_bytes,
                                          stream or None)


def nms_rotary_run(x: int, x_batch: int, x_token: int, x_head: int, type: int, batch: int, tokens: int, heads: int,
                   dim: int, positions: int, position_type: int, sets: int, axes: int, lut: int, pairs: int,
                   halves: int, inverse: int, y: int, y_batch: int, y_token: int, y_head: int, stream: int) -> int:
    return _lib().nms_rotary_run(x or None, x_batch, x_token, x_head, type, batch, tokens, heads, dim,
                                 positions or None, position_type, sets, axes, lut or None, pairs, halves, inverse,
                                 y or None, y_batch, y_token, y_head, stream or None)


# ----------------------------------------------------------- tensor helpers

def _rows(x, where: str):
    """(tensor, stride from row to row, rows, width) of rows [..., width];
    copied only where they do not lie at one stride."""
    shape = x.shape
    if not shape:
        raise ValueError(f"{where}: rows must be [..., width]")
    width, rows = shape[-1], 1
    for n in shape[:-1]:
        rows *= n
    if x.is_contiguous():
        return x, width, rows, width
    stride = x.stride()
    step, span, fits = width, None, width <= 1 or stride[-1] == 1
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if span is None:
            step = s
        elif s != span:
            fits = False
        span = s * n
    return (x, step, rows, width) if fits else (x.contiguous(), width, rows, width)


def _aligned(bytes_each: int, *operands) -> int:
    """Whether (tensor, row stride, width) operands and their rows start at
    multiples of 16 bytes and do not overlap."""
    for t, row, width in operands:
        if t.data_ptr() % 16 or row * bytes_each % 16 or row < width:
            return 0
    return 1


def _weight(x, weight, width: int, where: str):
    """The weight [outer, width] with its elements next to one another."""
    if weight.dim() != 2 or weight.shape[1] != width or weight.dtype is not x.dtype or \
            weight.get_device() != x.get_device():
        raise ValueError(f"{where}: weight must be [outer, inner] of x's type beside x")
    if weight.stride(1) != 1 and width > 1:
        weight = weight.contiguous()
    return weight


def _act(act: str, where: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"{where}: act must be 'none', 'relu', 'silu' or 'gelu'")
    return code


# ------------------------------------------------------------- linear layer

def linear_act(x, weight, bias=None, *, act: str = "none", residual=None, return_pre: bool = False):
    """y = act(x weight^T + bias) + residual.

    x [..., inner] float32, float16 or bfloat16; weight [outer, inner] of x's
    type; bias [outer] float32 or of x's type; act one of none, relu, silu,
    gelu; residual [..., outer] of x's type.  With return_pre also the
    activation's argument like y, which `linear_act_grad` takes.
    """
    where = "linear_act"
    kind = _type(x, where, "x")
    code = _act(act, where)
    torch = head._torch()
    xs, x_row, rows, inner = _rows(x, where)
    weight = _weight(x, weight, inner, where)
    outer, w_row = weight.shape[0], weight.stride(0)
    bias_at, bias_kind = None, NMS_TYPE_F32
    if bias is not None:
        if bias.shape != (outer,) or bias.get_device() != x.get_device() or not bias.is_contiguous() or \
                (bias.dtype is not torch.float32 and bias.dtype is not x.dtype):
            raise ValueError("linear_act: bias must be a contiguous [outer] tensor beside x, float32 or of x's type")
        bias_at, bias_kind = bias.data_ptr(), _types[bias.dtype]
    y = torch.empty((*x.shape[:-1], outer), dtype=x.dtype, device=x.device)
    res_at, res_row = None, 0
    if residual is not None:
        _same(residual, y, where, "residual")
        residual, res_row = _rows(residual, where)[:2]
        res_at = residual.data_ptr()
    pre = torch.empty_like(y) if return_pre else None
    wsb = nms_linear_workspace_size(kind, rows, inner, outer,
                                    _aligned(x.element_size(), (xs, x_row, inner), (weight, w_row, inner)))
    ws = torch.empty(wsb, dtype=torch.uint8, device=x.device) if wsb else None
    st = _launch(x, _lib().nms_linear_run, xs.data_ptr(), x_row, kind, rows, inner, weight.data_ptr(), w_row, outer,
                 bias_at, bias_kind, code, res_at, res_row, y.data_ptr(), pre.data_ptr() if return_pre else None, None,
                 ws.data_ptr() if wsb else None, wsb)
    if st:
        _raise(st, "nms_linear_run")
    return (y, pre) if return_pre else y


def linear_act_grad(dy, x, weight, pre=None, *, act: str = "none", need=(True, True, True)):
    """Gradient of `linear_act`: (dx like x, dweight like weight, dbias float32
    [outer]); the residual's is dy itself.  pre is the forward's (not read
    with act 'none'); need says which of the three are wanted, the others are
    None."""
    where = "linear_act_grad"
    kind = _type(x, where, "x")
    code = _act(act, where)
    torch = head._torch()
    xs, x_row, rows, inner = _rows(x, where)
    weight = _weight(x, weight, inner, where)
    outer, w_row = weight.shape[0], weight.stride(0)
    if dy.shape != (*x.shape[:-1], outer) or dy.dtype is not x.dtype or dy.get_device() != x.get_device():
        raise ValueError("linear_act_grad: dy must be [..., outer] of x's type beside x")
    dys, dy_row = _rows(dy, where)[:2]
    pre_at = None
    if code:
        if pre is None:
            raise ValueError("linear_act_grad: an activation's gradient needs the forward's pre")
        _same(pre, dy, where, "pre")
        pre = pre.contiguous()
        pre_at = pre.data_ptr()
    dx = _like(x) if need[0] else None
    dweight = torch.empty((outer, inner), dtype=x.dtype, device=x.device) if need[1] else None
    dbias = torch.empty(outer, dtype=torch.float32, device=x.device) if need[2] else None
    if not any(need):
        return None, None, None
    wsb = nms_linear_grad_workspace_size(kind, rows, inner, outer, _aligned(x.element_size(), (xs, x_row, inner),
                                                                            (weight, w_row, inner),
                                                                            (dys, dy_row, outer)))
    ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    st = _launch(x, _lib().nms_linear_grad_run, dys.data_ptr(), dy_row, xs.data_ptr(), x_row, kind, rows, inner,
                 weight.data_ptr(), w_row, outer, pre_at, code, *(None if t is None else t.data_ptr()
                                                                  for t in (dx, dweight, dbias)), None, ws.data_ptr(),
                 wsb)
    if st:
        _raise(st, "nms_linear_grad_run")
    return dx, dweight, dbias


# ------------------------------------------------------ layer normalisation

def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, residual=None, return_stats: bool = False):
    """y = layer_norm(x + residual) * weight + bias over the last axis.

    x, residual [..., width] float32, float16 or bfloat16; weight, bias
    [width] float32 or of x's type.  Returns y; with a residual (y, sum), sum
    = x + residual in x's type, the rows that are normalised; with
    return_stats also mean and rstd [...] (float32), which `layer_norm_grad`
    takes.
    """
    where = "layer_norm"
    kind = _type(x, where, "x")
    torch = head._torch()
    xs, x_row, rows, width = _rows(x, where)
    wp, bp, ptype = head._params(x, width, weight, bias, where)
    y, total, res_at, res_row = _like(x), None, None, 0
    if residual is not None:
        _same(residual, x, where, "residual")
        residual, res_row = _rows(residual, where)[:2]
        res_at, total = residual.data_ptr(), _like(x)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    st = _launch(x, _lib().nms_layer_norm_run, xs.data_ptr(), x_row, res_at, res_row, kind, rows, width, wp or None,
                 bp or None, ptype, eps, y.data_ptr(), None if total is None else total.data_ptr(),
                 mean.data_ptr() if return_stats else None, rstd.data_ptr() if return_stats else None)
    if st:
        _raise(st, "nms_layer_norm_run")
    if residual is None:
        return (y, mean, rstd) if return_stats else y
    return (y, total, mean, rstd) if return_stats else (y, total)


def layer_norm_grad(dy, x, mean, rstd, weight=None, *, dsum=None):
    """Gradient of `layer_norm`: (dx, dweight, dbias), dx like x and that of
    the residual too, the parameters' gradients float32 [width].  x holds the
    normalised rows (the forward's sum, with a residual); dsum like x is the
    gradient that reaches the sum by other ways and is added to dx."""
    where = "layer_norm_grad"
    kind = _type(x, where, "x")
    torch = head._torch()
    _same(dy, x, where, "dy")
    xs, x_row, rows, width = _rows(x, where)
    dys, dy_row = _rows(dy, where)[:2]
    wp, _, ptype = head._params(x, width, weight, None, where)
    for s in (mean, rstd):
        if s.shape != x.shape[:-1] or s.dtype is not torch.float32 or s.get_device() != x.get_device() or \
                not s.is_contiguous():
            raise ValueError("layer_norm_grad: mean and rstd must be contiguous float32 [...] tensors beside x")
    sum_at, sum_row = None, 0
    if dsum is not None:
        _same(dsum, x, where, "dsum")
        dsum, sum_row = _rows(dsum, where)[:2]
        sum_at = dsum.data_ptr()
    dx = _like(x)
    dweight = torch.empty(width, dtype=torch.float32, device=x.device)
    dbias = torch.empty_like(dweight)
    wsb = nms_layer_norm_workspace_size(rows, width)
    ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    st = _launch(x, _lib().nms_layer_norm_grad_run, dys.data_ptr(), dy_row, xs.data_ptr(), x_row, sum_at, sum_row,
                 kind, rows, width, mean.data_ptr(), rstd.data_ptr(), wp or None, ptype, dx.data_ptr(),
                 dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(), wsb)
    if st:
        _raise(st, "nms_layer_norm_grad_run")
    return dx, dweight, dbias


# --------------------------------------------------------- rotary positions

_RADIAN = (1 << 128) * 10 ** 50 // 628318530717958647692528676655900576839433879875021  # of a turn, in units of 2^-128


def rotary_lut(*pairs: int, base: float = 10000.0):
    """Table for `rotary`: pairs[a] pairs of elements turn by axis a of the
    positions, pair j of n by base^(-j / n) radians a position.  int64 [2,
    sum(pairs)] on the CPU: fractions of a turn in units of 2^-64, axes."""
    if not pairs or min(pairs) < 0 or sum(pairs) < 1 or len(pairs) > NMS_ROTARY_MAX_AXES or not 1.0 <= base < 1e300:
        raise ValueError("rotary_lut: numbers of pairs by axis (not negative, one pair at least, "
                         f"{NMS_ROTARY_MAX_AXES} axes at most) and a base of 1 or more")
    with decimal.localcontext() as c:
        c.prec = 45
        log = decimal.Decimal(base).ln()
        # Factors from pair to pair, in units of 2^-128.
        factors = [int((-log / n).exp() * (1 << 128)) if n else 0 for n in pairs]
    turns = []
    for n, factor in zip(pairs, factors):
        f = _RADIAN
        for _ in range(n):
            turns.append((f + (1 << 63)) >> 64)
            f = f * factor >> 128
    axes = [a for a, n in enumerate(pairs) for _ in range(n)]
    torch = head._torch()
    return torch.tensor([turns, axes], dtype=torch.int64)


def _rotary(x, positions, lut, halves: bool, inverse: bool, where: str):
    kind = _type(x, where, "x")
    torch = head._torch()
    if x.dim() != 4:
        raise ValueError(f"{where}: x must be [batch, tokens, heads, dim]")
    B, n, H, D = x.shape
    place = x.get_device()
    if positions.dtype is torch.int32:
        position_kind = NMS_POSITION_I32
    elif positions.dtype is torch.float32:
        position_kind = NMS_TYPE_F32
    else:
        position_kind = None
    if position_kind is None or positions.dim() != 3 or positions.shape[0] not in (1, B) or \
            positions.shape[1] != n or positions.get_device() != place:
        raise ValueError(f"{where}: positions must be int32 or float32 [1 or batch, tokens, axes] beside x")
    if lut.dtype is not torch.int64 or lut.dim() != 2 or lut.shape[0] != 2 or lut.get_device() != place or \
            2 * lut.shape[1] > D:
        raise ValueError(f"{where}: lut must be int64 [2, pairs] beside x, of no more pairs than x's vectors have")
    positions, lut = positions.contiguous(), lut.contiguous()
    if D > 1 and x.stride(3) != 1:
        x = x.contiguous()
    y = torch.empty_like(x, memory_format=torch.preserve_format)  # a dense x keeps the order of its axes
    if D > 1 and y.stride(3) != 1:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    st = _launch(x, _lib().nms_rotary_run, x.data_ptr(), x.stride(0), x.stride(1), x.stride(2), kind, B, n, H, D,
                 positions.data_ptr(), position_kind, positions.shape[0], positions.shape[2], lut.data_ptr(),
                 lut.shape[1], int(halves), int(inverse), y.data_ptr(), y.stride(0), y.stride(1), y.stride(2))
    if st:
        _raise(st, "nms_rotary_run")
    return y


def rotary(x, positions, lut, *, halves: bool = True):
    """Rotary positions: x [batch, tokens, heads, dim] (any strides but the
    last; queries and keys of a packed projection are one slice of it) with
    each pair of elements turned by its token's position.

    positions int32 or float32 [1 or batch, tokens, axes] (fractions count, as
    a box's centre in cells); lut from `rotary_lut`, on x's device.  With
    halves pair i is elements i and i + pairs, without it 2 i and 2 i + 1;
    elements behind the pairs are copied.
    """
    return _rotary(x, positions, lut, halves, False, "rotary")


def rotary_grad(dy, positions, lut, *, halves: bool = True):
    """Gradient of `rotary` to x: the incoming gradient turned back."""
    return _rotary(dy, positions, lut, halves, True, "rotary_grad")
