"""Operators of a trainable detection head, forward and backward: group
normalisation with activation and dropout on channels-last maps, dropout from
a counter-based generator, and attention weights with a learned bias by
buckets of relative position.

The raw entry points carry the names of the C functions (device addresses as
ints, the status code returned); the functions below them work on CUDA
tensors, run on their device's current stream and never synchronise.
greedy_iou_nms_gb300.autograd has the same operators for torch's autograd.
"""
from __future__ import annotations

import bisect
import ctypes
import functools

NMS_TYPE_F32 = 0
NMS_TYPE_F16 = 1
NMS_TYPE_BF16 = 2
NMS_ACT_NONE = 0  # nms_group_norm_run activations
NMS_ACT_RELU = 1
NMS_ACT_SILU = 2
NMS_ACT_GELU = 3
NMS_NORM_MAX_CHANNELS = 16384
NMS_NORM_MAX_BATCH = 1 << 20
NMS_NORM_MAX_PIXELS = 1 << 28
NMS_RELATION_MAX_BUCKETS = 1024
NMS_RELATION_MAX_HEADS = 4096
NMS_RELATION_MAX_AXES = 4
NMS_RELATION_MAX_REACH = 1 << 20

EXPORTED = ("nms_dropout_run", "nms_group_norm_workspace_size", "nms_group_norm_run", "nms_group_norm_grad_run",
            "nms_relation_buckets_run", "nms_relation_softmax_run", "nms_relation_grad_workspace_size",
            "nms_relation_softmax_grad_run")

_ACTS = {"none": NMS_ACT_NONE, "relu": NMS_ACT_RELU, "silu": NMS_ACT_SILU, "gelu": NMS_ACT_GELU}


def declare(lib) -> None:
    """Argument types of the entry points (called once by load())."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    f64, u64, psz = ctypes.c_double, ctypes.c_uint64, ctypes.POINTER(ctypes.c_size_t)
    for name, args in (
            ("nms_dropout_run", [vp, vp, i32, i64, f64, u64, u64, vp, vp]),
            ("nms_group_norm_workspace_size", [i64, i64, i32, i32, psz]),
            ("nms_group_norm_run", [vp, i64, i64, i32, i64, i64, i32, i32, vp, vp, i32, f32, i32, f64, u64, u64,
                                    vp, vp, vp, vp, sz, vp]),
            ("nms_group_norm_grad_run", [vp, i64, i64, vp, i64, i64, i32, i64, i64, i32, i32, vp, vp, vp, vp, i32,
                                         i32, f64, u64, u64, vp, vp, vp, vp, sz, vp]),
            ("nms_relation_buckets_run", [vp, i64, vp, i64, i64, i64, i32, vp, i32, vp, vp]),
            ("nms_relation_softmax_run", [vp, i32, i64, i32, i64, i64, vp, i64, vp, i32, vp, f32, vp, vp]),
            ("nms_relation_grad_workspace_size", [i64, i32, i64, i64, i32, psz]),
            ("nms_relation_softmax_grad_run", [vp, vp, i32, i64, i32, i64, i64, vp, i64, i32, vp, f32, vp, vp, vp,
                                               sz, vp])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import load
        _loaded = load()
    return _loaded


def _raise(code: int, where: str):
    from . import NmsError
    raise NmsError(code, where)


# ------------------------------------------------------------- raw C entries

def nms_dropout_run(x: int, residual: int, type: int, n: int, drop_p: float, seed: int, offset: int, y: int,
                    stream: int) -> int:
    return _lib().nms_dropout_run(x or None, residual or None, type, n, drop_p, seed, offset, y or None,
                                  stream or None)


@functools.lru_cache(maxsize=4096)
def nms_group_norm_workspace_size(batch: int, pixels: int, channels: int, groups: int) -> int:
    out = ctypes.c_size_t(0)
    st = _lib().nms_group_norm_workspace_size(batch, pixels, channels, groups, ctypes.byref(out))
    if st:
        _raise(st, "nms_group_norm_workspace_size")
    return out.value


def nms_group_norm_run(x: int, x_image: int, x_pixel: int, type: int, batch: int, pixels: int, channels: int,
                       groups: int, weight: int, bias: int, param_type: int, eps: float, act: int, drop_p: float,
                       seed: int, offset: int, y: int, mean: int, rstd: int, workspace: int, workspace_bytes: int,
                       stream: int) -> int:
    return _lib().nms_group_norm_run(x or None, x_image, x_pixel, type, batch, pixels, channels, groups,
                                     weight or None, bias or None, param_type, eps, act, drop_p, seed, offset,
                                     y or None, mean or None, rstd or None, workspace or None, workspace_bytes,
                                     stream or None)


def nms_group_norm_grad_run(dy: int, dy_image: int, dy_pixel: int, x: int, x_image: int, x_pixel: int, type: int,
                            batch: int, pixels: int, channels: int, groups: int, mean: int, rstd: int, weight: int,
                            bias: int, param_type: int, act: int, drop_p: float, seed: int, offset: int, dx: int,
                            dweight: int, dbias: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().nms_group_norm_grad_run(dy or None, dy_image, dy_pixel, x or None, x_image, x_pixel, type, batch,
                                          pixels, channels, groups, mean or None, rstd or None, weight or None,
                                          bias or None, param_type, act, drop_p, seed, offset, dx or None,
                                          dweight or None, dbias or None, workspace or None, workspace_bytes,
                                          stream or None)


def nms_relation_buckets_run(q_pos: int, q_sets: int, k_pos: int, k_sets: int, queries: int, keys: int, axes: int,
                             lut: int, reach: int, buckets: int, stream: int) -> int:
    return _lib().nms_relation_buckets_run(q_pos or None, q_sets, k_pos or None, k_sets, queries, keys, axes,
                                           lut or None, reach, buckets or None, stream or None)


def nms_relation_softmax_run(scores: int, type: int, batch: int, heads: int, queries: int, keys: int, buckets: int,
                             sets: int, table: int, num_buckets: int, key_mask: int, scale: float, probs: int,
                             stream: int) -> int:
    return _lib().nms_relation_softmax_run(scores or None, type, batch, heads, queries, keys, buckets or None, sets,
                                           table or None, num_buckets, key_mask or None, scale, probs or None,
                                           stream or None)


@functools.lru_cache(maxsize=4096)
def nms_relation_grad_workspace_size(batch: int, heads: int, queries: int, keys: int, num_buckets: int) -> int:
    out = ctypes.c_size_t(0)
    st = _lib().nms_relation_grad_workspace_size(batch, heads, queries, keys, num_buckets, ctypes.byref(out))
    if st:
        _raise(st, "nms_relation_grad_workspace_size")
    return out.value


def nms_relation_softmax_grad_run(dprobs: int, probs: int, type: int, batch: int, heads: int, queries: int,
                                  keys: int, buckets: int, sets: int, num_buckets: int, key_mask: int, scale: float,
                                  dscores: int, dtable: int, workspace: int, workspace_bytes: int,
                                  stream: int) -> int:
    return _lib().nms_relation_softmax_grad_run(dprobs or None, probs or None, type, batch, heads, queries, keys,
                                                buckets or None, sets, num_buckets, key_mask or None, scale,
                                                dscores or None, dtable or None, workspace or None, workspace_bytes,
                                                stream or None)


# ----------------------------------------------------------- tensor helpers

_torch_module = None
_types = {}
_raw_stream = None


def _torch():
    global _torch_module, _raw_stream
    if _torch_module is None:
        import torch
        _types.update({torch.float32: NMS_TYPE_F32, torch.float16: NMS_TYPE_F16, torch.bfloat16: NMS_TYPE_BF16})
        # The current stream's handle without a Stream object around it, where this torch has that.
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch_module = torch
    return _torch_module


def _type(x, where: str, name: str) -> int:
    _torch()
    t = _types.get(x.dtype)
    if t is None or not x.is_cuda:
        raise ValueError(f"{where}: {name} must be a float32, float16 or bfloat16 CUDA tensor")
    return t


def _stream(x) -> int:
    if _raw_stream is not None:
        return _raw_stream(x.get_device())
    return _torch().cuda.current_stream(x.device).cuda_stream


def _launch(x, entry, *args) -> int:
    """entry(*args, the current stream of x's device), that device current:
    a launch goes to the current one."""
    cuda, at = _torch().cuda, x.get_device()
    if cuda.current_device() == at:
        return entry(*args, _stream(x))
    with cuda.device(at):
        return entry(*args, _stream(x))


def _like(x):
    """An uninitialised contiguous tensor of x's shape and type."""
    if x.is_contiguous():
        return _torch_module.empty_like(x)
    return _torch_module.empty_like(x, memory_format=_torch_module.contiguous_format)


def _same(x, like, where: str, name: str) -> None:
    if x.shape != like.shape or x.dtype is not like.dtype or x.get_device() != like.get_device():
        raise ValueError(f"{where}: {name} must have the shape, type and device of the other operand")


def _drop_numbers(p: float, seed: int, offset: int, where: str) -> None:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"{where}: p must lie in [0, 1]")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError(f"{where}: seed and offset must be integers of 64 bits, not negative")


def _map(x, where: str):
    """(tensor, image stride, pixel stride, batch, pixels, channels) of a
    channels-last map [batch, ..., channels]; copied only where its pixels do
    not lie at one stride."""
    shape = x.shape
    if len(shape) < 2:
        raise ValueError(f"{where}: the map must be [batch, ..., channels]")
    batch, channels, pixels = shape[0], shape[-1], 1
    for n in shape[1:-1]:
        pixels *= n
    if x.is_contiguous():
        return x, channels * pixels, channels, batch, pixels, channels
    # One pixel stride: the last pixel axis of more than one entry sets it and
    # each axis before it spans the axes after it.
    stride = x.stride()
    step, span, fits = channels, None, channels <= 1 or stride[-1] == 1
    for n, s in zip(reversed(shape[1:-1]), reversed(stride[1:-1])):
        if n == 1:
            continue
        if span is None:
            step = s
            fits = fits and s >= channels
        elif s != span:
            fits = False
        span = s * n
    if not fits:
        return x.contiguous(), channels * pixels, channels, batch, pixels, channels
    return x, stride[0] if batch > 1 else 0, step, batch, pixels, channels


def _params(x, channels: int, weight, bias, where: str):
    """Addresses of weight and bias and their type."""
    kind = None
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        t = p.dtype
        if p.dim() != 1 or p.shape[0] != channels or p.get_device() != x.get_device() or not p.is_contiguous() or \
                (t is not _torch_module.float32 and t is not x.dtype) or (kind is not None and t is not kind):
            raise ValueError(f"{where}: {name} must be a contiguous [channels] tensor beside x, float32 or of x's "
                             "type, weight and bias alike")
        kind = t
    return (0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
            NMS_TYPE_F32 if kind is None else _types[kind])


def group_norm_act(x, groups: int, weight=None, bias=None, *, eps: float = 1e-5, act: str = "none", p: float = 0.0,
                   seed: int = 0, offset: int = 0, return_stats: bool = False):
    """y = dropout(act(group_norm(x) * weight + bias)) of a channels-last map.

    x [batch, ..., channels] float32, float16 or bfloat16 (a torch
    channels_last tensor [N, C, H, W] is such a map as x.permute(0, 2, 3, 1));
    weight, bias [channels] float32 or of x's type; act one of none, relu,
    silu, gelu.  Dropout with probability p by (seed, offset) and the
    element's index, as `dropout`.  With return_stats also mean and rstd
    [batch, groups] (float32), which `group_norm_act_grad` takes.
    """
    kind = _type(x, "group_norm_act", "x")
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("group_norm_act: act must be 'none', 'relu', 'silu' or 'gelu'")
    _drop_numbers(p, seed, offset, "group_norm_act")
    torch = _torch_module
    xs, image, pixel, batch, pixels, channels = _map(x, "group_norm_act")
    wp, bp, ptype = _params(x, channels, weight, bias, "group_norm_act")
    wsb = nms_group_norm_workspace_size(batch, pixels, channels, groups)
    y, mean, rstd = _like(x), None, None
    if return_stats:
        mean = torch.empty((batch, groups), dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    st = _launch(x, _lib().nms_group_norm_run, xs.data_ptr(), image, pixel, kind, batch, pixels, channels, groups, wp,
                 bp, ptype, eps, code, p, seed, offset, y.data_ptr(), mean.data_ptr() if return_stats else None,
                 rstd.data_ptr() if return_stats else None, ws.data_ptr(), wsb)
    if st:
        _raise(st, "nms_group_norm_run")
    return (y, mean, rstd) if return_stats else y


def group_norm_act_grad(dy, x, mean, rstd, groups: int, weight=None, bias=None, *, act: str = "none",
                        p: float = 0.0, seed: int = 0, offset: int = 0):
    """Gradient of `group_norm_act`: (dx, dweight, dbias), dx like x, the
    parameters' gradients float32 [channels].  mean and rstd, the parameters
    and the dropout numbers are the forward's."""
    where = "group_norm_act_grad"
    kind = _type(x, where, "x")
    _same(dy, x, where, "dy")
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("group_norm_act_grad: act must be 'none', 'relu', 'silu' or 'gelu'")
    _drop_numbers(p, seed, offset, where)
    torch = _torch_module
    xs, image, pixel, batch, pixels, channels = _map(x, where)
    dys, dimage, dpixel = _map(dy, where)[:3]
    wp, bp, ptype = _params(x, channels, weight, bias, where)
    for s in (mean, rstd):
        if s.shape != (batch, groups) or s.dtype is not torch.float32 or s.get_device() != x.get_device() or \
                not s.is_contiguous():
            raise ValueError("group_norm_act_grad: mean and rstd must be contiguous float32 [batch, groups] tensors "
                             "beside x")
    wsb = nms_group_norm_workspace_size(batch, pixels, channels, groups)
    dx = _like(x)
    dweight = torch.empty(channels, dtype=torch.float32, device=x.device)
    dbias = torch.empty_like(dweight)
    ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    st = _launch(x, _lib().nms_group_norm_grad_run, dys.data_ptr(), dimage, dpixel, xs.data_ptr(), image, pixel, kind,
                 batch, pixels, channels, groups, mean.data_ptr(), rstd.data_ptr(), wp, bp, ptype, code, p, seed,
                 offset, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(), wsb)
    if st:
        _raise(st, "nms_group_norm_grad_run")
    return dx, dweight, dbias


def dropout(x, p: float, seed: int, offset: int = 0, *, residual=None):
    """residual + x * mask / keep (no residual: the product alone), the mask a
    function of (seed, offset, element index): the same numbers give the same
    mask.  keep = 1 - p, rounded to a 65536th."""
    kind = _type(x, "dropout", "x")
    _drop_numbers(p, seed, offset, "dropout")
    if residual is not None:
        _same(residual, x, "dropout", "residual")
        residual = residual.contiguous()
    x = x.contiguous()
    y = _torch_module.empty_like(x)
    st = _launch(x, _lib().nms_dropout_run, x.data_ptr(), None if residual is None else residual.data_ptr(), kind,
                 x.numel(), p, seed, offset, y.data_ptr())
    if st:
        _raise(st, "nms_dropout_run")
    return y


def dropout_grad(dy, p: float, seed: int, offset: int = 0):
    """Gradient of `dropout` to x: the same mask on the incoming gradient (the
    residual's gradient is dy itself)."""
    return dropout(dy, p, seed, offset)


def relation_lut_log(num_buckets: int, max_distance: int, *, ahead: str = "mirror"):
    """Table for `relation_buckets` of one axis in logarithmic buckets:
    distances below half the buckets have one each, longer ones up to
    max_distance share the rest evenly over their logarithm, still longer ones
    the last.  ahead says what becomes of a key ahead of its query: 'mirror'
    (as far behind; num_buckets in all), 'own' (buckets of its own, num_buckets
    to each side, 2 * num_buckets in all) or 'mask'.  int32 [1, 2 * max_distance
    + 1], on the CPU."""
    if num_buckets < 2 or max_distance < num_buckets // 2 or ahead not in ("mirror", "own", "mask"):
        raise ValueError("relation_lut_log: num_buckets >= 2, max_distance >= num_buckets // 2, ahead one of "
                         "'mirror', 'own', 'mask'")
    exact = num_buckets // 2
    span = num_buckets - exact
    # The first distance of bucket exact + k: (d / exact)^span >= (max_distance / exact)^k, settled in whole numbers (a
    # logarithm's rounding puts distances on a boundary into the bucket before).
    firsts = []
    for k in range(1, span):
        least = max_distance ** k * exact ** (span - k)
        d = max(exact, int(exact * (max_distance / exact) ** (k / span)))
        while d ** span < least:
            d += 1
        while d > exact and (d - 1) ** span >= least:
            d -= 1
        firsts.append(d)
    parts = [d if d < exact else exact + bisect.bisect_right(firsts, d) for d in range(max_distance + 1)]
    front = {"mirror": parts, "own": [num_buckets + b for b in parts], "mask": [-1] * len(parts)}[ahead]
    return _torch().tensor([parts[:0:-1] + [parts[0]] + front[1:]], dtype=_torch().int32)


def relation_lut_cells(reach_rows: int, reach_columns: int):
    """Table for `relation_buckets` of (row, column) cells: a bucket for each
    offset within the reaches, (2 * reach_rows + 1) * (2 * reach_columns + 1)
    in all; offsets beyond take the edge's.  int32 [2, 2 * reach + 1] with reach
    the larger one, on the CPU."""
    torch = _torch()
    reach = max(reach_rows, reach_columns)
    at = torch.arange(-reach, reach + 1, dtype=torch.int32)
    rows = (at.clamp(-reach_rows, reach_rows) + reach_rows) * (2 * reach_columns + 1)
    return torch.stack([rows, at.clamp(-reach_columns, reach_columns) + reach_columns]).to(torch.int32)


def relation_buckets(q_pos, k_pos, lut):
    """Bucket of every (query, key) pair by relative position: int16 [sets,
    queries, keys] from int32 CUDA tensors q_pos [sets or 1, queries, axes],
    k_pos [sets or 1, keys, axes] and lut [axes, 2 * reach + 1] (see
    `relation_lut_log`, `relation_lut_cells`); -1 masks the pair."""
    torch = _torch()
    if not (q_pos.dtype is k_pos.dtype is lut.dtype is torch.int32 and q_pos.is_cuda and
            q_pos.get_device() == k_pos.get_device() == lut.get_device()):
        raise ValueError("relation_buckets: q_pos, k_pos and lut must be int32 tensors on one CUDA device")
    if q_pos.dim() != 3 or k_pos.dim() != 3 or lut.dim() != 2:
        raise ValueError("relation_buckets: positions must be [sets, length, axes] and lut [axes, 2 * reach + 1]")
    (qs, Q, axes), (ks, K, k_axes), (l_axes, width) = q_pos.shape, k_pos.shape, lut.shape
    if axes != k_axes or axes != l_axes or width % 2 == 0:
        raise ValueError("relation_buckets: lut must be [axes, 2 * reach + 1] with the positions' axes")
    if qs != ks and qs != 1 and ks != 1:
        raise ValueError("relation_buckets: q_pos and k_pos must have as many sets, or one of them one")
    q_pos, k_pos, lut = q_pos.contiguous(), k_pos.contiguous(), lut.contiguous()
    out = torch.empty((ks if qs == 1 else qs, Q, K), dtype=torch.int16, device=q_pos.device)
    st = _launch(q_pos, _lib().nms_relation_buckets_run, q_pos.data_ptr(), qs, k_pos.data_ptr(), ks, Q, K, axes,
                 lut.data_ptr(), width // 2, out.data_ptr())
    if st:
        _raise(st, "nms_relation_buckets_run")
    return out


def _relation(scores, buckets, key_mask, where: str):
    torch = _torch_module
    if scores.dim() != 4:
        raise ValueError(f"{where}: scores must be [batch, heads, queries, keys]")
    B, H, Q, K = scores.shape
    place = scores.get_device()
    if buckets.dtype is not torch.int16 or buckets.get_device() != place or buckets.dim() != 3:
        raise ValueError(f"{where}: buckets must be int16 [1 or batch, queries, keys] beside the scores")
    sets, queries, keys = buckets.shape
    if sets not in (1, B) or queries != Q or keys != K:
        raise ValueError(f"{where}: buckets must be int16 [1 or batch, queries, keys] beside the scores")
    mask = None
    if key_mask is not None:
        if key_mask.shape != (B, K) or key_mask.dtype not in (torch.bool, torch.uint8) or \
                key_mask.get_device() != place:
            raise ValueError(f"{where}: key_mask must be bool or uint8 [batch, keys] beside the scores")
        key_mask = key_mask.contiguous()
        mask = key_mask.data_ptr()
    return B, H, Q, K, buckets.contiguous(), sets, key_mask, mask


def relation_softmax(scores, table, buckets, *, scale: float = 1.0, key_mask=None):
    """Attention weights with a learned bias: softmax over the valid keys of
    scale * scores + table[buckets, head].

    scores [batch, heads, queries, keys]; table [num_buckets, heads]; buckets
    from `relation_buckets` (one map, or one for each image); key_mask bool
    [batch, keys], true where a key takes part.  A masked pair's weight is 0,
    a row without valid pairs is all 0.  Returns weights like scores.
    """
    where = "relation_softmax"
    kind = _type(scores, where, "scores")
    torch = _torch_module
    B, H, Q, K, buckets, sets, key_mask, mask = _relation(scores, buckets, key_mask, where)
    if table.dim() != 2 or table.shape[1] != H or table.get_device() != scores.get_device():
        raise ValueError("relation_softmax: table must be [num_buckets, heads] beside the scores")
    if table.dtype is not torch.float32:
        table = table.to(torch.float32)
    table, scores = table.contiguous(), scores.contiguous()
    out = torch.empty_like(scores)
    st = _launch(scores, _lib().nms_relation_softmax_run, scores.data_ptr(), kind, B, H, Q, K, buckets.data_ptr(),
                 sets, table.data_ptr(), table.shape[0], mask, scale, out.data_ptr())
    if st:
        _raise(st, "nms_relation_softmax_run")
    return out


def relation_softmax_grad(dprobs, probs, buckets, num_buckets: int, *, scale: float = 1.0, key_mask=None):
    """Gradient of `relation_softmax`: (dscores like probs, dtable float32
    [num_buckets, heads]) from the incoming gradient and the forward's
    weights, map, scale and mask."""
    where = "relation_softmax_grad"
    kind = _type(probs, where, "probs")
    torch = _torch_module
    _same(dprobs, probs, where, "dprobs")
    B, H, Q, K, buckets, sets, key_mask, mask = _relation(probs, buckets, key_mask, where)
    dprobs, probs = dprobs.contiguous(), probs.contiguous()
    wsb = nms_relation_grad_workspace_size(B, H, Q, K, num_buckets)
    ws = torch.empty(wsb, dtype=torch.uint8, device=probs.device)
    ds = torch.empty_like(probs)
    dtable = torch.empty((num_buckets, H), dtype=torch.float32, device=probs.device)
    st = _launch(probs, _lib().nms_relation_softmax_grad_run, dprobs.data_ptr(), probs.data_ptr(), kind, B, H, Q, K,
                 buckets.data_ptr(), sets, num_buckets, mask, scale, ds.data_ptr(), dtable.data_ptr(), ws.data_ptr(),
                 wsb)
    if st:
        _raise(st, "nms_relation_softmax_grad_run")
    return ds, dtable
