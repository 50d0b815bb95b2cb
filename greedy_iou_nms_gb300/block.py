"""Operators of a transformer block among a detector's candidates, forward and
backward: linear layer with activation and residual, layer normalisation with
the residual stream, and rotary positions on several axes.

The raw entry points carry the names of the C functions (device addresses as
ints, the status code returned); the functions below them work on CUDA
tensors, run on their device's current stream and never synchronise.  Their
operands are checked and handed over in C++ (binding/block_binding.cpp).
greedy_iou_nms_gb300.autograd has the same operators for torch's autograd.
"""
from __future__ import annotations

import ctypes
import decimal
import functools

from . import head
from .head import _ACTS, _lib, _raise

NMS_LAYER_MAX_WIDTH = 16384
NMS_LINEAR_MAX_WIDTH = 1 << 18
NMS_ACT_ROUND_SLOPES = 256
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


# ---------------------------------------------------------- tensor functions

_native_module = None


def _native():
    """The C++ half of the tensor functions: operands' checks, outputs, workspace and the call of the C entry."""
    global _native_module
    if _native_module is None:
        import importlib.machinery
        import importlib.util
        import os

        import torch  # noqa: F401  (the module needs its libraries)

        from ._build import BINDING_LIB
        if not os.path.exists(BINDING_LIB):
            raise RuntimeError(f"the tensor functions are not built at {BINDING_LIB}: call greedy_iou_nms_gb300.build() (with "
                               "a torch for CUDA)")
        lib = _lib()
        loader = importlib.machinery.ExtensionFileLoader("gbblock", BINDING_LIB)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("gbblock", loader))
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTED))
        _native_module = module
    return _native_module


def _act(act: str, where: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"{where}: act must be 'none', 'relu', 'silu' or 'gelu'")
    return code


def linear_act(x, weight, bias=None, *, act: str = "none", residual=None, return_pre: bool = False, status=None):
    """y = act(x weight^T + bias) + residual.

    x [..., inner] float32, float16 or bfloat16; weight [outer, inner] of x's
    type; bias [outer] float32 or of x's type; act one of none, relu, silu,
    gelu; residual [..., outer] of x's type.  With return_pre also the
    activation's argument like y, which `linear_act_grad` takes.

    Every wait of the kernels on the tensor cores is bounded.  One that gives up
    (after seconds, where a calculation takes microseconds: the device is not
    right) leaves NaNs, and NMS_ERR_TIMEOUT in status, one int32 beside x that
    the caller has set to 0, where it is given.
    """
    out = _native().linear_act(x, weight, bias, _act(act, "linear_act"), residual, bool(return_pre), status)
    if type(out) is int:
        _raise(out, "nms_linear_run")
    return out if return_pre else out[0]


def linear_act_grad(dy, x, weight, pre=None, *, act: str = "none", need=(True, True, True), round_slopes: bool = False,
                    status=None):
    """Gradient of `linear_act`: (dx like x, dweight like weight, dbias float32
    [outer]); the residual's is dy itself.  pre is the forward's (not read
    with act 'none'); need says which of the three are wanted, the others are
    None.  round_slopes: dy act'(pre) is rounded to a 16-bit type before the
    products, which then take half as long with silu and gelu and are off by
    that rounding.  status as for `linear_act`."""
    code = _act(act, "linear_act_grad") | (NMS_ACT_ROUND_SLOPES if round_slopes else 0)
    out = _native().linear_act_grad(dy, x, weight, pre, code, status, *need)
    if type(out) is int:
        _raise(out, "nms_linear_grad_run")
    return out


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, residual=None, return_stats: bool = False):
    """y = layer_norm(x + residual) * weight + bias over the last axis.

    x, residual [..., width] float32, float16 or bfloat16; weight, bias
    [width] float32 or of x's type.  Returns y; with a residual (y, sum), sum
    = x + residual in x's type, the rows that are normalised; with
    return_stats also mean and rstd [...] (float32), which `layer_norm_grad`
    takes.
    """
    out = _native().layer_norm(x, weight, bias, eps, residual, bool(return_stats))
    if type(out) is int:
        _raise(out, "nms_layer_norm_run")
    return out if len(out) > 1 else out[0]


def layer_norm_grad(dy, x, mean, rstd, weight=None, *, dsum=None):
    """Gradient of `layer_norm`: (dx, dweight, dbias), dx like x and that of
    the residual too, the parameters' gradients float32 [width].  x holds the
    normalised rows (the forward's sum, with a residual); dsum like x is the
    gradient that reaches the sum by other ways and is added to dx."""
    out = _native().layer_norm_grad(dy, x, mean, rstd, weight, dsum)
    if type(out) is int:
        _raise(out, "nms_layer_norm_grad_run")
    return out


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


def _rotary(x, positions, lut, halves: bool, inverse: bool):
    out = _native().rotary(x, positions, lut, bool(halves), inverse)
    if type(out) is int:
        _raise(out, "nms_rotary_run")
    return out[0]


def rotary(x, positions, lut, *, halves: bool = True):
    """Rotary positions: x [batch, tokens, heads, dim] (any strides but the
    last; queries and keys of a packed projection are one slice of it) with
    each pair of elements turned by its token's position.

    positions int32 or float32 [1 or batch, tokens, axes] (fractions count, as
    a box's centre in cells); lut from `rotary_lut`, on x's device.  With
    halves pair i is elements i and i + pairs, without it 2 i and 2 i + 1;
    elements behind the pairs are copied.
    """
    return _rotary(x, positions, lut, halves, False)


def rotary_grad(dy, positions, lut, *, halves: bool = True):
    """Gradient of `rotary` to x: the incoming gradient turned back."""
    return _rotary(dy, positions, lut, halves, True)
