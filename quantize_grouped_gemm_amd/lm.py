"""Binding of the layer-boundary operators (C ABI in include/mxlm.h): what an
MXFP8 transformer runs between its GEMMs.

    add_rmsnorm_quant / add_rmsnorm_bwd     residual addition, RMS norm, MXFP8
    swiglu_ckpt_fwd / swiglu_ckpt_bwd       SwiGLU with an 8-bit checkpoint
    token_logprobs / token_logprobs_bwd     scoring of given tokens; the loss

Like the functions of mx: arguments are checked against the sizes that go with
them, outputs are allocated with torch unless given in `out`, the library is
called on torch's current stream, and there is no fallback. Calls without
given outputs go through _lmhost (C++), which takes 4 to 10 us of host time
where the steps below take 11 to 21; its checks are these in short, and what it
does not take as it is (given outputs, arguments to refuse) comes back and is
checked here, with a message. Without a built _lmhost.so such calls are refused.
It allocates what belongs together at once: codes and their scales, and the
outputs of token_logprobs, are slices of one allocation, so keeping or saving one
of them keeps the memory of all (outputs made here have one each).

Codes and scales are uint8 tensors under the keys q_row / s_row, q_col / s_col,
q_ck / s_ck in the layouts of mx.quantize. The number of rows T is free;
column-wise codes cover padded_rows(T, layout) rows, the ones past T being zeros,
so they feed mx.scaled_mm as they are.
"""

import ctypes

import torch

from . import mx
from .mx import MXError, _check, _flag, _want, _want_rows, scale_shape

IGNORE_INDEX = -100
MAX_COLS = 16384      # longest row of the norm
MAX_TOP = 64

_NONE = (None, None)

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
_host = None


def host():
    """The C++ host path (loaded once, with the library it calls)."""
    global _host
    if _host is None:
        lib()
        try:
            from . import _lmhost
        except ImportError as e:
            raise MXError(f"_lmhost.so: {e}; build it with python -m quantize_grouped_gemm_amd.build") from None
        _host = _lmhost
    return _host


def _done(res, name):
    """The outputs of a call through _lmhost, or None if it was left to the
    checks here; raises if the library refused it."""
    if res.__class__ is int:
        _check(res, name)
    return res


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


# The operators run for a few microseconds on small inputs, so the checks are
# written to cost little where they pass: one comparison each, and the
# functions of mx, which find out what is wrong, only where one fails.

_U8, _BF, _F32, _I32T = torch.uint8, torch.bfloat16, torch.float32, torch.int32
_empty = torch.empty


def _format(mode, layout):
    try:
        return mx._MODES[mode], mx._LAYOUTS[layout]
    except (KeyError, TypeError):
        if mode not in mx._MODES:
            raise MXError(f"mode: {mode!r}, expected 'rceil' or 'floor'") from None
        raise MXError(f"layout: {layout!r}, expected 'k128' or 'plain'") from None


def _matrix(t, name, dtypes=(_BF,)):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes:
        raise MXError(f"{name}: expected a 2-D tensor of {', '.join(str(d) for d in dtypes)}")
    return t.shape


def _rows(t, name, dtype, shape):
    """Checks a matrix of contiguous rows; returns its row stride (strides that
    no second row or column makes use of do not matter)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        _want_rows(t, name, dtype, shape)
    R, C = shape
    ld, one = t.stride()
    if (C > 1 and one != 1) or (R > 1 and ld < C):
        _want_rows(t, name, dtype, shape)
    return ld if R > 1 else C


def _whole(t, name, dtype, shape):
    """Checks a contiguous tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _want(t, name, dtype, shape=shape)


def _out(out, key, shape, dtype, dev):
    """The output under `key`, taken from `out` or allocated; its address."""
    t = out.get(key)
    if t is None:
        t = out[key] = _empty(*shape, dtype=dtype, device=dev)
    else:
        _whole(t, key, dtype, shape)
    return t.data_ptr()


def _codes(out, q, s, R, C, layout, dev):
    """The codes [R, C] and scales under the keys q and s; their addresses.
    Given ones may have any shape of the right size."""
    if out.get(q) is None:
        out[q] = _empty(R, C, dtype=_U8, device=dev)
    else:
        _want(out[q], q, _U8, R * C)
    if out.get(s) is None:
        if layout == "k128":
            out[s] = _empty(C // 128, R, 4, dtype=_U8, device=dev)
        else:
            out[s] = _empty(R, C // 32, dtype=_U8, device=dev)
    else:
        _want(out[s], s, _U8, R * C // 32)
    return out[q].data_ptr(), out[s].data_ptr()


def _launch(name, given, tensors, args):
    """Checks that every tensor is on the current device and calls the library
    on torch's current stream. `given`: outputs that the caller passed."""
    idx = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != idx:
            mx._device(*tensors)
    if given:
        mx._device(tensors[0], *[t for t in given.values() if isinstance(t, torch.Tensor)])
    if idx < 0 or idx != torch.cuda.current_device():
        mx._device(*tensors)
    _check(getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(idx)), name)


def _addr(t):
    return None if t is None else t.data_ptr()


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
    if out is None:
        res = _done((_host or host()).add_rmsnorm_quant(x, w, r, eps, mode, layout, colwise, checkpoint),
                    "mx_add_rmsnorm_quant")
        if res is not None:
            return res
    m, lay = _format(mode, layout)
    T, C = shape = _matrix(x, "x")
    ld = _rows(x, "x", _BF, shape)
    ld_r = 0 if r is None else _rows(r, "r", _BF, shape)
    _whole(w, "w", _F32, (C,))
    _norm_width(C, layout)
    given, out, dev = out, dict(out or {}), x.device
    total = None if r is None else _out(out, "sum", shape, _BF, dev)
    rstd = _out(out, "rstd", (T,), _F32, dev)
    row = _codes(out, "q_row", "s_row", T, C, layout, dev)
    col = _codes(out, "q_col", "s_col", C, padded_rows(T, layout), layout, dev) if colwise else _NONE
    ck = _codes(out, "q_ck", "s_ck", T, C, layout, dev) if checkpoint else _NONE
    _launch("mx_add_rmsnorm_quant", given, (x, w, r),
            (x.data_ptr(), ld, _addr(r), ld_r, w.data_ptr(), T, C, eps, m, lay, total, rstd, *row, *col, *ck))
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
    if out is None and work is None:
        q_ck, s_ck = _NONE if checkpoint is None else checkpoint
        res = _done((_host or host()).add_rmsnorm_bwd(dy, w, rstd, x, q_ck, s_ck, dsum, mode, layout, rowwise, colwise),
                    "mx_add_rmsnorm_bwd")
        if res is not None:
            return res
    m, lay = _format(mode, layout)
    T, C = shape = _matrix(dy, "dy")
    ld = _rows(dy, "dy", _BF, shape)
    _whole(w, "w", _F32, (C,))
    _whole(rstd, "rstd", _F32, (T,))
    _norm_width(C, layout)
    if (x is None) == (checkpoint is None):
        raise MXError("give exactly one of x and checkpoint")
    ld_x, q_ck, s_ck = 0, None, None
    if x is not None:
        ld_x = _rows(x, "x", _BF, shape)
    else:
        q_ck, s_ck = checkpoint
        _whole(q_ck, "q_ck", _U8, shape)
        _whole(s_ck, "s_ck", _U8, scale_shape(T, C, layout))
    ld_s = 0 if dsum is None else _rows(dsum, "dsum", _BF, shape)
    given, out, dev = out, dict(out or {}), dy.device
    dx = _out(out, "dx", shape, _BF, dev)
    dw = _out(out, "dw", (C,), _F32, dev)
    row = _codes(out, "q_row", "s_row", T, C, layout, dev) if rowwise else _NONE
    col = _codes(out, "q_col", "s_col", C, padded_rows(T, layout), layout, dev) if colwise else _NONE
    n = bwd_work(T, C)
    if work is None:
        work = _empty(n, dtype=_F32, device=dev)
    else:
        _want(work, "work", _F32)
        if work.numel() < n:
            raise MXError(f"work: {work.numel()} elements, needs {n}")
    _launch("mx_add_rmsnorm_bwd", given, (dy, w, rstd, x, q_ck, s_ck, dsum, work),
            (dy.data_ptr(), ld, w.data_ptr(), rstd.data_ptr(), _addr(x), ld_x, _addr(q_ck), _addr(s_ck), _addr(dsum),
             ld_s, T, C, m, lay, dx, dw, *row, *col, work.data_ptr()))
    return out


def bwd_work(T, C):
    """float32 elements of scratch that add_rmsnorm_bwd needs."""
    return lib().mx_add_rmsnorm_bwd_work(T, C)


def swiglu_ckpt_fwd(a, b, mode="rceil", layout="k128", out=None):
    """h = silu(a) * b for bf16 [T, H] views sharing a row stride (the halves
    of the w13 output). Returns q_row / s_row and q_col / s_col of h, and
    q_ck / s_ck, the row-wise MXFP8 copy of [a | b] [T, 2H] that
    swiglu_ckpt_bwd takes: the bf16 input need not be kept."""
    if out is None:
        res = _done((_host or host()).swiglu_ckpt_fwd(a, b, mode, layout), "mx_swiglu_ckpt_fwd")
        if res is not None:
            return res
    m, lay = _format(mode, layout)
    T, H = shape = _matrix(a, "a")
    ld = _rows(a, "a", _BF, shape)
    if _rows(b, "b", _BF, shape) != ld:
        raise MXError("a and b must share a row stride")
    _blocks("hidden", H, layout)
    given, out, dev = out, dict(out or {}), a.device
    row = _codes(out, "q_row", "s_row", T, H, layout, dev)
    col = _codes(out, "q_col", "s_col", H, padded_rows(T, layout), layout, dev)
    ck = _codes(out, "q_ck", "s_ck", T, 2 * H, layout, dev)
    _launch("mx_swiglu_ckpt_fwd", given, (a, b), (a.data_ptr(), b.data_ptr(), ld, T, H, m, lay, *row, *col, *ck))
    return out


def swiglu_ckpt_bwd(dh, q_ck, s_ck, mode="rceil", layout="k128", out=None):
    """Gradient of swiglu_ckpt_fwd from its checkpoint: dh bf16 [T, H] gives
    [dA | dB] [T, 2H] as q_row / s_row and q_col / s_col."""
    if out is None:
        res = _done((_host or host()).swiglu_ckpt_bwd(dh, q_ck, s_ck, mode, layout), "mx_swiglu_ckpt_bwd")
        if res is not None:
            return res
    m, lay = _format(mode, layout)
    T, H = shape = _matrix(dh, "dh")
    ld = _rows(dh, "dh", _BF, shape)
    _blocks("hidden", H, layout)
    _whole(q_ck, "q_ck", _U8, (T, 2 * H))
    _whole(s_ck, "s_ck", _U8, scale_shape(T, 2 * H, layout))
    given, out, dev = out, dict(out or {}), dh.device
    row = _codes(out, "q_row", "s_row", T, 2 * H, layout, dev)
    col = _codes(out, "q_col", "s_col", 2 * H, padded_rows(T, layout), layout, dev)
    _launch("mx_swiglu_ckpt_bwd", given, (dh, q_ck, s_ck),
            (dh.data_ptr(), ld, q_ck.data_ptr(), s_ck.data_ptr(), T, H, m, lay, *row, *col))
    return out


def _logits(x, targets, scale):
    T, V = shape = _matrix(x, "x", (_BF, _F32))
    ld = _rows(x, "x", x.dtype, shape)
    if V < 1:
        raise MXError("x: empty vocabulary")
    _whole(targets, "targets", torch.int64, (T,))
    if not 1e-6 <= scale <= 1e6:
        raise MXError(f"scale: {scale}, expected a number in [1e-6, 1e6]")
    return T, V, ld


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
    if out is None and dev_err is None:
        res = _done((_host or host()).token_logprobs(x, targets, scale, top, ignore_index), "mx_token_logprobs")
        if res is not None:
            return res
    T, V, ld = _logits(x, targets, scale)
    if not 0 <= top <= min(MAX_TOP, V):
        raise MXError(f"top: {top}, expected 0 to {min(MAX_TOP, V)}")
    given, out, dev = out, dict(out or {}), x.device
    logp = _out(out, "logp", (T,), _F32, dev)
    entropy = _out(out, "entropy", (T,), _F32, dev)
    stats = _out(out, "stats", (T, 2), _F32, dev)
    alt = (_out(out, "top_logp", (T, top), _F32, dev), _out(out, "top_idx", (T, top), _I32T, dev)) if top else _NONE
    n = lib().mx_token_logprobs_work(T, V, top)
    work = _empty(n, dtype=_U8, device=dev) if n else None
    _launch("mx_token_logprobs", given, (x, targets, _flag(dev_err)),
            (x.data_ptr(), mx._DT[x.dtype], ld, T, V, targets.data_ptr(), ignore_index, scale, top, logp, entropy, stats,
             *alt, _addr(work), _addr(dev_err)))
    return out


def token_logprobs_bwd(x, targets, stats, entropy, dlogp=None, dent=None, scale=1.0, mode="rceil", layout="k128",
                       ignore_index=IGNORE_INDEX, out=None, dev_err=None):
    """Gradient of token_logprobs with respect to x, in MXFP8 both ways.

    stats and entropy are the forward's; dlogp, dent: float32 [T], the
    gradients of logp and entropy (None: zero). Returns q_row / s_row
    [T, V_pad] and q_col / s_col [V_pad, padded_rows(T)], with V_pad = V
    rounded up to the layout's block step (128 or 32) and zeros past V."""
    if out is None and dev_err is None:
        res = _done((_host or host()).token_logprobs_bwd(x, targets, stats, entropy, dlogp, dent, scale, mode, layout,
                                                         ignore_index), "mx_token_logprobs_bwd")
        if res is not None:
            return res
    m, lay = _format(mode, layout)
    T, V, ld = _logits(x, targets, scale)
    _whole(stats, "stats", _F32, (T, 2))
    _whole(entropy, "entropy", _F32, (T,))
    if dlogp is not None:
        _whole(dlogp, "dlogp", _F32, (T,))
    if dent is not None:
        _whole(dent, "dent", _F32, (T,))
    given, out, dev = out, dict(out or {}), x.device
    Vp = padded_rows(V, layout)
    row = _codes(out, "q_row", "s_row", T, Vp, layout, dev)
    col = _codes(out, "q_col", "s_col", Vp, padded_rows(T, layout), layout, dev)
    _launch("mx_token_logprobs_bwd", given, (x, targets, stats, entropy, dlogp, dent, _flag(dev_err)),
            (x.data_ptr(), mx._DT[x.dtype], ld, T, V, targets.data_ptr(), ignore_index, stats.data_ptr(),
             entropy.data_ptr(), _addr(dlogp), _addr(dent), scale, m, lay, *row, *col, _addr(dev_err)))
    return out
