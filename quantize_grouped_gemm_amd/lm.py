"""Binding of the layer-boundary operators (C ABI in include/mxlm.h): what an
MXFP8 transformer runs between its GEMMs.

    add_rmsnorm_quant / add_rmsnorm_bwd     residual addition, RMS norm, MXFP8
    swiglu_ckpt_fwd / swiglu_ckpt_bwd       SwiGLU with an 8-bit checkpoint
    token_logprobs / token_logprobs_bwd     scoring of given tokens; the loss

Like the functions of mx: arguments are checked against the sizes that go with
them, outputs are allocated with torch unless given in `out`, the library is
called on torch's current stream, and there is no fallback. Codes and scales
are uint8 tensors under the keys q_row / s_row, q_col / s_col, q_ck / s_ck in
the layouts of mx.quantize. The number of rows T is free; column-wise codes
cover padded_rows(T, layout) rows, the ones past T being zeros, so they feed
mx.scaled_mm as they are.
"""

import ctypes

import torch

from . import mx
from .mx import MXError, _check, _device, _flag, _ptr, _stream, _u8, _want, _want_rows, scale_shape

IGNORE_INDEX = -100
MAX_COLS = 16384      # longest row of the norm
MAX_TOP = 64

_P, _I64, _I32, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
_SIGS = {
    "mx_add_rmsnorm_quant": ([_P, _I64, _P, _I64, _P, _I64, _I64, _F, _INT, _INT] + [_P] * 9, _INT),
    "mx_add_rmsnorm_bwd_work": ([_I64, _I64], _I64),
    "mx_add_rmsnorm_bwd": ([_P, _I64, _P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _INT, _INT] + [_P] * 8, _INT),
    "mx_swiglu_ckpt_fwd": ([_P, _P, _I64, _I64, _I64, _INT, _INT] + [_P] * 7, _INT),
    "mx_swiglu_ckpt_bwd": ([_P, _I64, _P, _P, _I64, _I64, _INT, _INT] + [_P] * 5, _INT),
    "mx_token_logprobs_work": ([_I64, _I64, _I32], _I64),
    "mx_token_logprobs": ([_P, _INT, _I64, _I64, _I64, _P, _I64, _F, _I32] + [_P] * 8, _INT),
    "mx_token_logprobs_bwd": ([_P, _INT, _I64, _I64, _I64, _P, _I64] + [_P] * 4 + [_F, _INT, _INT] + [_P] * 6, _INT),
}
EXPORTS = tuple(_SIGS)

_lib = None


def lib():
    """libmxfp8.so with the operators of this module bound."""
    global _lib
    if _lib is None:
        L = mx.lib()
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def padded_rows(T, layout="k128"):
    """Rows that column-wise codes of T rows cover."""
    step = 128 if layout == "k128" else 32
    return (T + step - 1) // step * step


def _format(mode, layout):
    if mode not in mx._MODES:
        raise MXError(f"mode: {mode!r}, expected 'rceil' or 'floor'")
    if layout not in mx._LAYOUTS:
        raise MXError(f"layout: {layout!r}, expected 'k128' or 'plain'")
    return mx._MODES[mode], mx._LAYOUTS[layout]


def _matrix(t, name, dtypes=(torch.bfloat16,)):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes:
        raise MXError(f"{name}: expected a 2-D tensor of {', '.join(str(d) for d in dtypes)}")
    return t.shape


def _ld(t):
    """Row stride; that of a single row does not matter."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _codes(out, keys, R, C, layout, dev):
    """The codes [R, C] and scales under keys = ("q_..", "s_.."), taken from
    `out` or allocated."""
    q, s = keys
    shape = scale_shape(R, C, layout)
    if out.get(q) is None:
        out[q] = _u8((R, C), dev)
    else:
        _want(out[q], q, torch.uint8, R * C)
    if out.get(s) is None:
        out[s] = _u8(shape, dev)
    else:
        _want(out[s], s, torch.uint8, R * C // 32)


def _tensor(out, key, shape, dtype, dev):
    if out.get(key) is None:
        out[key] = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _want(out[key], key, dtype, shape=shape)
    return out[key]


_ROW, _COL, _CK = ("q_row", "s_row"), ("q_col", "s_col"), ("q_ck", "s_ck")


def _blocks(name, n, layout):
    step = 128 if layout == "k128" else 32
    if n <= 0 or n % step:
        raise MXError(f"{name}: {n}, expected a positive multiple of {step}")


def _norm_width(C, layout):
    _blocks("columns", C, layout)
    if C > MAX_COLS:
        raise MXError(f"columns: {C}, at most {MAX_COLS}")


def add_rmsnorm_quant(x, w, r=None, eps=1e-6, mode="rceil", layout="k128", colwise=False, checkpoint=False, out=None):
    """s = bf16(x + r) (s = x without r), y = bf16(s * rstd * w) with
    rstd = (mean s^2 + eps)^(-1/2), and y in MXFP8.

    x, r: bf16 [T, C], rows may be strided; w: float32 [C]. Returns a dict
    with sum (with r; bf16), rstd (float32 [T]), q_row / s_row, with colwise
    q_col / s_col [C, padded_rows(T)], and with checkpoint q_ck / s_ck, the
    row-wise MXFP8 copy of s that add_rmsnorm_bwd takes in its place."""
    m, lay = _format(mode, layout)
    T, C = _matrix(x, "x")
    _want_rows(x, "x", torch.bfloat16, (T, C))
    if r is not None:
        _want_rows(r, "r", torch.bfloat16, (T, C))
    _want(w, "w", torch.float32, shape=(C,))
    _norm_width(C, layout)
    dev = x.device
    out = dict(out or {})
    if r is not None:
        _tensor(out, "sum", (T, C), torch.bfloat16, dev)
    _tensor(out, "rstd", (T,), torch.float32, dev)
    _codes(out, _ROW, T, C, layout, dev)
    if colwise:
        _codes(out, _COL, C, padded_rows(T, layout), layout, dev)
    if checkpoint:
        _codes(out, _CK, T, C, layout, dev)
    _device(x, w, r, *out.values())
    col = (_ptr(out["q_col"]), _ptr(out["s_col"])) if colwise else (None, None)
    ck = (_ptr(out["q_ck"]), _ptr(out["s_ck"])) if checkpoint else (None, None)
    st = lib().mx_add_rmsnorm_quant(_ptr(x), _ld(x), _ptr(r), 0 if r is None else _ld(r), _ptr(w), T, C, eps, m, lay,
                                    None if r is None else _ptr(out["sum"]), _ptr(out["rstd"]), _ptr(out["q_row"]),
                                    _ptr(out["s_row"]), *col, *ck, _stream(dev))
    _check(st, "mx_add_rmsnorm_quant")
    return out


def add_rmsnorm_bwd(dy, w, rstd, x=None, checkpoint=None, dsum=None, mode="rceil", layout="k128", rowwise=True,
                    colwise=False, out=None, work=None):
    """Gradient of add_rmsnorm_quant: dy bf16 [T, C] is the gradient of y,
    dsum (bf16 or None) the one that reaches s past the norm.

    s comes from x (bf16: the forward's sum, or its x without r) or from
    checkpoint = (q_ck, s_ck). Returns a dict with dx (bf16: the gradient of x
    and of r), dw (float32 [C]) and MXFP8 copies of dx: q_row / s_row and, with
    colwise, q_col / s_col. work: optional float32 scratch of bwd_work(T, C)
    elements."""
    m, lay = _format(mode, layout)
    T, C = _matrix(dy, "dy")
    _want_rows(dy, "dy", torch.bfloat16, (T, C))
    _want(w, "w", torch.float32, shape=(C,))
    _want(rstd, "rstd", torch.float32, shape=(T,))
    _norm_width(C, layout)
    if (x is None) == (checkpoint is None):
        raise MXError("give exactly one of x and checkpoint")
    q_ck = s_ck = None
    if x is not None:
        _want_rows(x, "x", torch.bfloat16, (T, C))
    else:
        q_ck, s_ck = checkpoint
        _want(q_ck, "q_ck", torch.uint8, shape=(T, C))
        _want(s_ck, "s_ck", torch.uint8, shape=scale_shape(T, C, layout))
    if dsum is not None:
        _want_rows(dsum, "dsum", torch.bfloat16, (T, C))
    dev = dy.device
    out = dict(out or {})
    _tensor(out, "dx", (T, C), torch.bfloat16, dev)
    _tensor(out, "dw", (C,), torch.float32, dev)
    if rowwise:
        _codes(out, _ROW, T, C, layout, dev)
    if colwise:
        _codes(out, _COL, C, padded_rows(T, layout), layout, dev)
    n = bwd_work(T, C)
    if work is None:
        work = torch.empty((n,), dtype=torch.float32, device=dev)
    else:
        _want(work, "work", torch.float32)
        if work.numel() < n:
            raise MXError(f"work: {work.numel()} elements, needs {n}")
    _device(dy, w, rstd, x, q_ck, s_ck, dsum, work, *out.values())
    row = (_ptr(out["q_row"]), _ptr(out["s_row"])) if rowwise else (None, None)
    col = (_ptr(out["q_col"]), _ptr(out["s_col"])) if colwise else (None, None)
    st = lib().mx_add_rmsnorm_bwd(_ptr(dy), _ld(dy), _ptr(w), _ptr(rstd), _ptr(x), 0 if x is None else _ld(x),
                                  _ptr(q_ck), _ptr(s_ck), _ptr(dsum), 0 if dsum is None else _ld(dsum), T, C, m, lay,
                                  _ptr(out["dx"]), _ptr(out["dw"]), *row, *col, _ptr(work), _stream(dev))
    _check(st, "mx_add_rmsnorm_bwd")
    return out


def bwd_work(T, C):
    """float32 elements of scratch that add_rmsnorm_bwd needs."""
    return lib().mx_add_rmsnorm_bwd_work(T, C)


def swiglu_ckpt_fwd(a, b, mode="rceil", layout="k128", out=None):
    """h = silu(a) * b for bf16 [T, H] views sharing a row stride (the halves
    of the w13 output). Returns q_row / s_row and q_col / s_col of h, and
    q_ck / s_ck, the row-wise MXFP8 copy of [a | b] [T, 2H] that
    swiglu_ckpt_bwd takes: the bf16 input need not be kept."""
    m, lay = _format(mode, layout)
    T, H = _matrix(a, "a")
    _want_rows(a, "a", torch.bfloat16, (T, H))
    _want_rows(b, "b", torch.bfloat16, (T, H))
    if _ld(a) != _ld(b):
        raise MXError("a and b must share a row stride")
    _blocks("hidden", H, layout)
    dev = a.device
    out = dict(out or {})
    _codes(out, _ROW, T, H, layout, dev)
    _codes(out, _COL, H, padded_rows(T, layout), layout, dev)
    _codes(out, _CK, T, 2 * H, layout, dev)
    _device(a, b, *out.values())
    st = lib().mx_swiglu_ckpt_fwd(_ptr(a), _ptr(b), _ld(a), T, H, m, lay, _ptr(out["q_row"]), _ptr(out["s_row"]),
                                  _ptr(out["q_col"]), _ptr(out["s_col"]), _ptr(out["q_ck"]), _ptr(out["s_ck"]),
                                  _stream(dev))
    _check(st, "mx_swiglu_ckpt_fwd")
    return out


def swiglu_ckpt_bwd(dh, q_ck, s_ck, mode="rceil", layout="k128", out=None):
    """Gradient of swiglu_ckpt_fwd from its checkpoint: dh bf16 [T, H] gives
    [dA | dB] [T, 2H] as q_row / s_row and q_col / s_col."""
    m, lay = _format(mode, layout)
    T, H = _matrix(dh, "dh")
    _want_rows(dh, "dh", torch.bfloat16, (T, H))
    _blocks("hidden", H, layout)
    _want(q_ck, "q_ck", torch.uint8, shape=(T, 2 * H))
    _want(s_ck, "s_ck", torch.uint8, shape=scale_shape(T, 2 * H, layout))
    dev = dh.device
    out = dict(out or {})
    _codes(out, _ROW, T, 2 * H, layout, dev)
    _codes(out, _COL, 2 * H, padded_rows(T, layout), layout, dev)
    _device(dh, q_ck, s_ck, *out.values())
    st = lib().mx_swiglu_ckpt_bwd(_ptr(dh), _ld(dh), _ptr(q_ck), _ptr(s_ck), T, H, m, lay, _ptr(out["q_row"]),
                                  _ptr(out["s_row"]), _ptr(out["q_col"]), _ptr(out["s_col"]), _stream(dev))
    _check(st, "mx_swiglu_ckpt_bwd")
    return out


def _logits(x, targets, scale):
    T, V = _matrix(x, "x", (torch.bfloat16, torch.float32))
    _want_rows(x, "x", x.dtype, (T, V))
    if V < 1:
        raise MXError("x: empty vocabulary")
    _want(targets, "targets", torch.int64, shape=(T,))
    if not 1e-6 <= scale <= 1e6:
        raise MXError(f"scale: {scale}, expected a number in [1e-6, 1e6]")
    return T, V


def token_logprobs(x, targets, scale=1.0, top=0, ignore_index=IGNORE_INDEX, out=None, dev_err=None):
    """Log probabilities of the given tokens under softmax(scale * x).

    x: bf16 or float32 [T, V], any V, rows may be strided; targets: int64 [T],
    ignore_index for a row that is not scored. Returns a dict of float32
    tensors: logp [T] (0 where not scored), entropy [T], stats [T, 2] (the row
    maximum and log sum exp of the scaled differences from it) and, with
    top > 0, top_logp [T, top] and top_idx (int32), the largest logits in
    descending order, ties to the lower index. Entries of -infinity are ruled
    out. dev_err: optional int32 device flag word; bit 3 reports a target
    outside the vocabulary (treated as not scored)."""
    T, V = _logits(x, targets, scale)
    if not 0 <= top <= min(MAX_TOP, V):
        raise MXError(f"top: {top}, expected 0 to {min(MAX_TOP, V)}")
    dev = x.device
    out = dict(out or {})
    f32 = torch.float32
    _tensor(out, "logp", (T,), f32, dev)
    _tensor(out, "entropy", (T,), f32, dev)
    _tensor(out, "stats", (T, 2), f32, dev)
    if top:
        _tensor(out, "top_logp", (T, top), f32, dev)
        _tensor(out, "top_idx", (T, top), torch.int32, dev)
    n = lib().mx_token_logprobs_work(T, V, top)
    work = _u8((n,), dev) if n else None
    _device(x, targets, _flag(dev_err), *out.values())
    alt = (_ptr(out["top_logp"]), _ptr(out["top_idx"])) if top else (None, None)
    st = lib().mx_token_logprobs(_ptr(x), mx._DT[x.dtype], _ld(x), T, V, _ptr(targets), ignore_index, scale, top,
                                 _ptr(out["logp"]), _ptr(out["entropy"]), _ptr(out["stats"]), *alt, _ptr(work),
                                 _ptr(dev_err), _stream(dev))
    _check(st, "mx_token_logprobs")
    return out


def token_logprobs_bwd(x, targets, stats, entropy, dlogp=None, dent=None, scale=1.0, mode="rceil", layout="k128",
                       ignore_index=IGNORE_INDEX, out=None, dev_err=None):
    """Gradient of token_logprobs with respect to x, in MXFP8 both ways.

    stats and entropy are the forward's; dlogp, dent: float32 [T], the
    gradients of logp and entropy (None: zero). Returns q_row / s_row
    [T, V_pad] and q_col / s_col [V_pad, padded_rows(T)], with V_pad = V
    rounded up to the layout's block step (128 or 32) and zeros past V."""
    m, lay = _format(mode, layout)
    T, V = _logits(x, targets, scale)
    _want(stats, "stats", torch.float32, shape=(T, 2))
    _want(entropy, "entropy", torch.float32, shape=(T,))
    for t, name in ((dlogp, "dlogp"), (dent, "dent")):
        if t is not None:
            _want(t, name, torch.float32, shape=(T,))
    dev = x.device
    out = dict(out or {})
    Vp = padded_rows(V, layout)
    _codes(out, _ROW, T, Vp, layout, dev)
    _codes(out, _COL, Vp, padded_rows(T, layout), layout, dev)
    _device(x, targets, stats, entropy, dlogp, dent, _flag(dev_err), *out.values())
    st = lib().mx_token_logprobs_bwd(_ptr(x), mx._DT[x.dtype], _ld(x), T, V, _ptr(targets), ignore_index, _ptr(stats),
                                     _ptr(entropy), _ptr(dlogp), _ptr(dent), scale, m, lay, _ptr(out["q_row"]),
                                     _ptr(out["s_row"]), _ptr(out["q_col"]), _ptr(out["s_col"]), _ptr(dev_err),
                                     _stream(dev))
    _check(st, "mx_token_logprobs_bwd")
    return out
