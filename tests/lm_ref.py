"""The layer-boundary operators in float64 on the CPU, from their definitions
(torch), and the tolerances of their MXFP8 outputs.

A quantized output is checked two ways against the float64 value v it stands
for (before any rounding):
  * every element: with E the kernel's scale exponent, v is clipped to
    448 * 2^E (FLOOR scales saturate), and the stored value may be off by the
    bf16 rounding (2^-8 |v|), the E4M3 rounding (2^-4 |v|, or half a subnormal
    step 2^-10 * 2^E) and a float32 evaluation error F32 * mag, where mag is
    |v| or, for a sum that can cancel, the sum of its terms' magnitudes. The
    scale byte itself has to be the rule's for a block maximum within that
    evaluation error of the exact one.
  * all elements: the codes are those of bf16(v) except where v lies so close
    to a bf16 rounding border that float32 arithmetic decides it, and that
    border is also one of E4M3's: at an evaluation error of 2^-22 a share of
    2 * 2^-22 / 2^-8 of the bf16 values flips and 1 in 16 of those moves a
    code, 8e-6 in all; 1e-4 leaves room for the elements that cancel.
"""

import numpy as np
import torch

from oracle import mx as O

F64 = torch.float64
F32 = 2.0 ** -19     # relative error of a float32 evaluation of a few dozen roundings


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def pad_rows(v, step):
    n = (v.shape[0] + step - 1) // step * step
    return torch.cat([v, v.new_zeros(n - v.shape[0], v.shape[1])]) if n != v.shape[0] else v


# ---------------------------------------------------------------- formulas

def norm_fwd(s, w, eps):
    """s float64 [T, C] (the bf16 sum) -> rstd, y."""
    rstd = (s.square().mean(-1) + eps) ** -0.5
    return rstd, s * rstd[:, None] * w


def norm_bwd(dy, w, rstd, s, dsum):
    xh = s * rstd[:, None]
    g = dy * w
    dx = (g - xh * (g * xh).mean(-1, keepdim=True)) * rstd[:, None] + (0 if dsum is None else dsum)
    return dx, (dy * xh).sum(0)


def swiglu(a, b):
    return a * torch.sigmoid(a) * b


def swiglu_bwd(dh, a, b):
    s = torch.sigmoid(a)
    return torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], 1)


def logprob_fwd(x, t, scale, ignore=-100):
    """x float64 [T, V]: m, ls, logp, entropy."""
    m = x.amax(-1)
    d = (x - m[:, None]) * scale
    e = torch.where(x == -torch.inf, 0.0, torch.exp(d))
    s = e.sum(-1)
    ls = torch.log(s)
    empty = m == -torch.inf
    ls = torch.where(empty, -torch.inf, ls)
    ent = torch.where(empty, 0.0, ls - torch.where(e > 0, e * d, 0.0).sum(-1) / s)
    ok = (t != ignore) & (t >= 0) & (t < x.shape[1])
    dt = d.gather(1, torch.where(ok, t, 0)[:, None])[:, 0]
    logp = torch.where(ok, torch.where(empty, -torch.inf, dt - ls), 0.0)
    return m, ls, logp, ent


def logprob_bwd(x, t, m, ls, ent, dlogp, dent, scale, ignore=-100):
    empty = (m == -torch.inf)[:, None]
    lp = torch.where(empty, 0.0, (x - m[:, None]) * scale - ls[:, None])
    p = torch.where(empty | (x == -torch.inf), 0.0, torch.exp(lp))
    ok = (t != ignore) & (t >= 0) & (t < x.shape[1])
    g = torch.where(ok, dlogp, 0.0)[:, None]
    onehot = torch.zeros_like(x).scatter_(1, torch.where(ok, t, 0)[:, None], ok.to(F64)[:, None])
    grad = g * (onehot - p) - torch.where(p > 0, p * dent[:, None] * (lp + ent[:, None]), 0.0)
    return torch.where(empty, 0.0, grad * scale)


# ---------------------------------------------------------------- checks

def plain_scales(s):
    a = s.detach().cpu().numpy()
    return np.ascontiguousarray(np.moveaxis(a, -3, -2).reshape(a.shape[1], 4 * a.shape[0])) if a.ndim == 3 else a


def check_codes(q, s, v, mode, what, mag=None):
    """q, s: the kernel's codes and scales; v float64 [R, C], the value they
    stand for; mag: see above."""
    assert tuple(q.shape) == tuple(v.shape), f"{what}: {tuple(q.shape)} vs {tuple(v.shape)}"
    if v.numel() == 0:
        return
    v = v.numpy()
    err = F32 * (np.abs(v) if mag is None else np.maximum(mag.numpy(), np.abs(v)))
    q = q.detach().cpu().numpy()
    s = plain_scales(s)
    amax = np.abs(v).reshape(v.shape[0], -1, 32).max(-1)
    rule = lambda a: O.quantize(np.repeat(a[..., None], 32, -1).reshape(v.shape), mode)[1].astype(np.int64)
    bf = lambda a: O.bf16_to_f64(O.f64_to_bf16(a))
    eblk = err.reshape(v.shape[0], -1, 32).max(-1)
    lo, hi = rule(bf(np.maximum(amax - eblk, 0))), rule(bf(amax + eblk))
    assert np.all((s >= lo) & (s <= hi)), f"{what}: {int(((s < lo) | (s > hi)).sum())} scale bytes off"
    E = np.repeat(s.astype(np.int64) - 127, 32, axis=-1).astype(np.float64)
    got = O.dequantize(q, s)
    lim = 448 * np.exp2(E)
    tol = np.abs(v) * (2.0 ** -4 + 2.0 ** -8) + 2 * err + 2.0 ** -10 * np.exp2(E)
    bad = np.abs(got - np.clip(v, -lim, lim)) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values beyond their rounding"
    qr, sr = O.quantize(bf(v), mode)
    diff = int((O.dequantize(qr, sr) != got).sum())
    assert diff <= 4 + 1e-4 * v.size, f"{what}: {diff} of {v.size} values are another code"


def check_dual(out, v, mode, layout, what, row=True, col=True, mag=None):
    step = 128 if layout == "k128" else 32
    if row:
        check_codes(out["q_row"], out["s_row"], v, mode, what + " row", mag)
    if col:
        mc = None if mag is None else pad_rows(mag, step).t().contiguous()
        check_codes(out["q_col"], out["s_col"], pad_rows(v, step).t().contiguous(), mode, what + " col", mc)
