"""Binding of the routed-experts operators (C ABI in include/mxmoe.h): what
stands around the experts' grouped products.

    route / route_bwd       scores, the choice of top experts, their weights
    dispatch                the choice -> group sizes, offsets and row maps
    gather_quantize         token rows into expert order, quantized on the way
                            (MXFP8 for mx, blocks of 128 for b128)
    combine / combine_bwd   weighted sum of a token's expert rows

Gradients: combine_bwd gives the weights' (route_bwd takes it to the logits),
gather_quantize with weights the experts' rows', combine without weights that of
the gathered rows. A slot is a token's j-th choice: slot t * top + j.

Conventions as in b128 and lm: checked arguments, outputs allocated with torch
unless given in `out`, torch's current stream, no fallback.
"""

import ctypes

import torch

from . import b128, lm, mx
from .lm import _BF, _F32, _NONE, _addr, _codes, _done, _format, _launch, _matrix, _out, _rows, _whole, padded_rows
from .mx import MXError, _want

MAX_EXPERTS, MAX_TOP, MAX_GROUPS = 1024, 16, 16
_I32T = torch.int32
_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}

_P, _I64, _I32, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
_SIGS = {
    "mx_route": ([_P, _INT, _I64, _I64, _I32, _P, _INT, _I32, _I32, _INT, _I32, _INT, _F, _P, _P, _P], _INT),
    "mx_route_bwd": ([_P, _INT, _I64, _I64, _I32, _INT, _P, _I32, _INT, _F, _P, _P, _P], _INT),
    "mx_dispatch_work": ([_I64, _I32], _I64),
    "mx_dispatch": ([_P, _I64, _I32, _I32, _I64] + [_P] * 6, _INT),
    "mx_gather_quantize": ([_P, _I64, _I64, _I64, _P, _I32, _P, _I64, _INT, _INT] + [_P] * 5, _INT),
    "mx_b128_gather_quantize": ([_P, _I64, _I64, _I64, _P, _I32, _P, _I64, _INT] + [_P] * 5, _INT),
    "mx_combine": ([_P, _I64, _I64, _P, _P, _P, _I64, _I64, _I32, _I64, _P, _P], _INT),
    "mx_combine_bwd": ([_P, _I64, _P, _I64, _I64, _P, _I64, _I32, _I64, _P, _P], _INT),
}
EXPORTS = tuple(_SIGS)

_lib = None


def lib():
    """libmxfp8.so with the operators of this module bound."""
    global _lib
    if _lib is None:
        L = b128.lib()
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


_host = None


def host():
    global _host
    if _host is None:
        lib()
        _host = b128.host()
    return _host


def _choice(v, name, table):
    try:
        return table[v]
    except (KeyError, TypeError):
        raise MXError(f"{name}: {v!r}, expected {' or '.join(map(repr, table))}") from None


def _logits(x, top, scale):
    T, E = shape = _matrix(x, "x", (_BF, _F32))
    ld = _rows(x, "x", x.dtype, shape)
    if not 1 <= E <= MAX_EXPERTS:
        raise MXError(f"x: {E} experts, expected 1 to {MAX_EXPERTS}")
    if not 1 <= top <= min(MAX_TOP, E):
        raise MXError(f"top: {top}, expected 1 to {min(MAX_TOP, E)}")
    if not abs(scale) < float("inf"):
        raise MXError(f"scale: {scale}, expected a finite number")
    return T, E, ld


def route(x, top, bias=None, score="softmax", groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0,
          out=None):
    """The `top` experts of each token and their weights.

    x: logits, bf16 or float32 [T, E], rows may be strided, -infinity rules an
    expert out; bias: float32 [E], added to the scores for the choice only.
    score: "softmax" or "sigmoid". groups > 1: only the top_groups groups (of
    E / groups consecutive experts) with the largest sum of their two best
    choice values (group_score "top2") or best value ("max") stay. renorm: the
    weights are divided by their sum; then times scale. Returns a dict with weights (float32 [T, top]) and
    idx (int32 [T, top]) in descending order, ties to the lower index; -1 and 0 where no expert is left."""
    if out is None:
        res = _done((_host or host()).route(x, top, bias, score, groups, top_groups, group_score, renorm, scale), "mx_route")
        if res is not None:
            return res
    sc, gsc = _choice(score, "score", _SCORES), _choice(group_score, "group_score", _GROUP_SCORES)
    T, E, ld = _logits(x, top, scale)
    if not 1 <= groups <= MAX_GROUPS or E % groups:
        raise MXError(f"groups: {groups}, expected a divisor of {E}, at most {MAX_GROUPS}")
    if not 1 <= top_groups <= groups:
        raise MXError(f"top_groups: {top_groups}, expected 1 to {groups}")
    if bias is not None:
        _whole(bias, "bias", _F32, (E,))
    given, out, dev = out, dict(out or {}), x.device
    w, idx = _out(out, "weights", (T, top), _F32, dev), _out(out, "idx", (T, top), _I32T, dev)
    lib()
    _launch("mx_route", given, (x, bias), (x.data_ptr(), mx._DT[x.dtype], ld, T, E, _addr(bias), sc, groups, top_groups,
                                           gsc, top, int(bool(renorm)), scale, w, idx))
    return out


def route_bwd(x, idx, dweights, score="softmax", renorm=True, scale=1.0, out=None):
    """Gradient of route's weights with respect to x: idx is the forward's,
    dweights float32 [T, top]. Choices whose score is 0 as a float32 have no part.
    Returns [T, E] of x's type."""
    if out is None:
        res = _done((_host or host()).route_bwd(x, idx, dweights, score, renorm, scale), "mx_route_bwd")
        if res is not None:
            return res
    sc = _choice(score, "score", _SCORES)
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2:
        raise MXError("idx: expected an int32 tensor [T, top]")
    top = idx.shape[1]
    T, E, ld = _logits(x, top, scale)
    _whole(idx, "idx", _I32T, (T, top))
    _whole(dweights, "dweights", _F32, (T, top))
    if out is None:
        out = torch.empty((T, E), dtype=x.dtype, device=x.device)
    else:
        _whole(out, "out", x.dtype, (T, E))
    lib()
    _launch("mx_route_bwd", None, (x, idx, dweights, out),
            (x.data_ptr(), mx._DT[x.dtype], ld, T, E, sc, idx.data_ptr(), top, int(bool(renorm)), scale,
             dweights.data_ptr(), out.data_ptr()))
    return out


def capacity(slots, experts, multiple=128):
    """Rows that hold any choice of `slots` slots, a multiple of `multiple`."""
    return (slots + min(experts, slots) * (multiple - 1) + multiple - 1) // multiple * multiple


def dispatch(idx, experts, multiple=128, cap=None, out=None):
    """Rows in expert order for the chosen experts idx (int32 [T, top]; an
    entry outside [0, experts) gets no row). Returns int32 tensors: sizes and
    offs [experts] (slots of each expert; ends of the groups, padded to
    `multiple` rows, as the grouped products take them), src [cap] (the slot
    of each row, -1 for padding) and pos (the row of each slot, -1 if none, of
    idx's shape). cap: rows of the expert-ordered tensors, by default
    capacity(...)."""
    if out is None:
        res = _done((_host or host()).dispatch(idx, experts, multiple, cap), "mx_dispatch")
        if res is not None:
            return res
    _want(idx, "idx", _I32T)
    slots = idx.numel()
    if not 1 <= experts <= MAX_EXPERTS:
        raise MXError(f"experts: {experts}, expected 1 to {MAX_EXPERTS}")
    if not 1 <= multiple <= 1024:
        raise MXError(f"multiple: {multiple}, expected 1 to 1024")
    least = slots + min(experts, slots) * (multiple - 1)
    if cap is None:
        cap = capacity(slots, experts, multiple)
    elif cap < least:
        raise MXError(f"cap: {cap} rows, needs at least {least}")
    given, out, dev = out, dict(out or {}), idx.device
    p = [_out(out, k, shape, _I32T, dev)
         for k, shape in (("sizes", (experts,)), ("offs", (experts,)), ("src", (cap,)), ("pos", tuple(idx.shape)))]
    n = lib().mx_dispatch_work(slots, experts)
    work = torch.empty(n, dtype=_I32T, device=dev) if n else None
    _launch("mx_dispatch", given, (idx,), (idx.data_ptr(), slots, experts, multiple, cap, *p, _addr(work)))
    return out


def gather_quantize(x, src, top, weights=None, fmt="mxfp8", mode="rceil", layout="k128", colwise=False, out=None):
    """Row r = x[src[r] // top] (zeros where src[r] < 0), or with weights
    (float32, one a slot) bf16(weights[src[r]] * x[src[r] // top]), quantized.

    x: bf16 [T, C], rows may be strided; src: int32 [rows] (dispatch's). fmt
    "mxfp8" with mode "rceil" / "floor" and a scale layout, or "b128" with mode
    "f32" / "rceil". Returns q_row / s_row and, with colwise, q_col / s_col over
    the rows padded to the block step, as mx.quantize or b128.quantize."""
    if out is None:
        res = _done((_host or host()).gather_quantize(x, src, top, weights, fmt, mode, layout, colwise),
                    "mx_gather_quantize")
        if res is not None:
            return res
    if fmt not in ("mxfp8", "b128"):
        raise MXError(f"fmt: {fmt!r}, expected 'mxfp8' or 'b128'")
    blocks = fmt == "b128"
    if blocks:
        if layout != "k128":
            raise MXError("layout: blocks of 128 have one layout")
        m = b128.mode_of(mode)
    else:
        m, lay = _format(mode, layout)
    T, C = shape = _matrix(x, "x")
    ld = _rows(x, "x", _BF, shape)
    lm._blocks("columns", C, layout)
    _want(src, "src", _I32T)
    if top < 1:
        raise MXError(f"top: {top}, expected at least 1")
    if weights is not None:
        _want(weights, "weights", _F32, T * top)
    rows = src.numel()
    given, out, dev = out, dict(out or {}), x.device
    pair = b128.take_pair if blocks else lambda o, q, s, R, C_, d: _codes(o, q, s, R, C_, layout, d)
    row = pair(out, "q_row", "s_row", rows, C, dev)
    col = pair(out, "q_col", "s_col", C, padded_rows(rows, layout), dev) if colwise else _NONE
    lib()
    _launch("mx_b128_gather_quantize" if blocks else "mx_gather_quantize", given, (x, src, weights),
            (x.data_ptr(), ld, T, C, src.data_ptr(), top, _addr(weights), rows, m, *(() if blocks else (lay,)), *row, *col))
    return out


def _slots(pos, T):
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2 or pos.shape[1] < 1:
        raise MXError("pos: expected an int32 tensor [T, top]")
    _whole(pos, "pos", _I32T, (T if T is not None else pos.shape[0], pos.shape[1]))
    return pos.shape


def combine(y, pos, weights=None, r=None, out=None):
    """out_t = r_t + sum_j weights_tj * y[pos_tj] (weights None: ones; r None:
    nothing added): y bf16 [rows, C], C a multiple of 8, pos int32 [T, top],
    weights float32 [T, top], r bf16 [T, C]. An entry of pos outside y's rows has no
    part. Returns bf16 [T, C]."""
    if out is None:
        res = _done((_host or host()).combine(y, pos, weights, r), "mx_combine")
        if res is not None:
            return res
    R, C = shape = _matrix(y, "y")
    ld = _rows(y, "y", _BF, shape)
    T, top = _slots(pos, None)
    if weights is not None:
        _whole(weights, "weights", _F32, (T, top))
    ld_r = 0 if r is None else _rows(r, "r", _BF, (T, C))
    if C < 8 or C % 8:
        raise MXError(f"columns: {C}, expected a positive multiple of 8")
    if out is None:
        out = torch.empty((T, C), dtype=_BF, device=y.device)
    else:
        _whole(out, "out", _BF, (T, C))
    lib()
    _launch("mx_combine", None, (y, pos, weights, r, out),
            (y.data_ptr(), ld, R, pos.data_ptr(), _addr(weights), _addr(r), ld_r, T, top, C, out.data_ptr()))
    return out


def combine_bwd(dout, y, pos, out=None):
    """Gradient of combine's weights: float32 [T, top] of <dout_t, y[pos_tj]>,
    0 where pos is outside y's rows."""
    if out is None:
        res = _done((_host or host()).combine_bwd(dout, y, pos), "mx_combine_bwd")
        if res is not None:
            return res
    R, C = shape = _matrix(y, "y")
    ld = _rows(y, "y", _BF, shape)
    T, top = _slots(pos, None)
    ld_d = _rows(dout, "dout", _BF, (T, C))
    if C < 8 or C % 8:
        raise MXError(f"columns: {C}, expected a positive multiple of 8")
    if out is None:
        out = torch.empty((T, top), dtype=_F32, device=y.device)
    else:
        _whole(out, "out", _F32, (T, top))
    lib()
    _launch("mx_combine_bwd", None, (dout, y, pos, out),
            (dout.data_ptr(), ld_d, y.data_ptr(), ld, R, pos.data_ptr(), T, top, C, out.data_ptr()))
    return out
