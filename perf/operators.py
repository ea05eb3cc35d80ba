"""The layer-boundary operators as measured workloads: their inputs, their
plain form in elementary torch operations, and their values in 64 bits.

Three families, each forward and backward:
  norm      residual addition + RMS norm + MXFP8 output, and its gradient
            (optionally from an 8-bit checkpoint of the residual stream),
            with the input gradient quantized for the GEMMs behind it
  swiglu    SwiGLU + dual MXFP8 quantization that keeps an 8-bit checkpoint
            of its input, and the gradient taken from that checkpoint
  logprob   log probabilities of given tokens with entropy and top
            alternatives, and the gradient of the logits in MXFP8

`own = False` computes the plain form, `own = True` calls
quantize_grouped_gemm_amd.lm. E4M3 codes and E8M0 scales are returned as
float8 tensors, i.e. as the numbers that they stand for.
"""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100          # the target of a token that is not scored
EPS = 1e-6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decoded token entering an MLP block: latency only
        dict(name="norm_fwd_token", op="norm_fwd", T=1, C=4096, residual=True, col=False, ckpt=False, mode="rceil",
             layout="k128"),
        # the residual stream of a full training batch before the routed experts, kept in 8 bits for the backward
        dict(name="norm_fwd_train", op="norm_fwd", T=16384, C=5120, residual=True, col=True, ckpt=True, mode="rceil",
             layout="k128"),
        # a ragged micro-batch (rows no multiple of any tile) of a wide model, stream kept in bf16
        dict(name="norm_bwd_ragged", op="norm_bwd", T=1000, C=7168, residual=True, col=True, ckpt=False, mode="floor",
             layout="k128"),
        # the dense training batch, from the 8-bit checkpoint
        dict(name="norm_bwd_train", op="norm_bwd", T=8192, C=4096, residual=True, col=True, ckpt=True, mode="rceil",
             layout="k128"),
        # one fine-grained expert's share of a small batch
        dict(name="swiglu_fwd_small", op="swiglu_fwd", T=130, H=2048, mode="rceil", layout="k128"),
        # the dense MLP of a training batch
        dict(name="swiglu_fwd_train", op="swiglu_fwd", T=8192, H=14336, mode="rceil", layout="k128"),
        # a ragged share of routed tokens at an expert's hidden size
        dict(name="swiglu_bwd_ragged", op="swiglu_bwd", T=1000, H=8192, mode="floor", layout="k128"),
        dict(name="swiglu_bwd_train", op="swiglu_bwd", T=8192, H=14336, mode="rceil", layout="k128"),
        # scoring one sampled token with its 20 best alternatives
        dict(name="logprob_fwd_token", op="logprob_fwd", T=1, V=131072, top=20, dtype="bf16", scale=1.0, masked=False),
        # scoring a batch of sampled sequences under a temperature, 5 alternatives each
        dict(name="logprob_fwd_batch", op="logprob_fwd", T=4096, V=131072, top=5, dtype="bf16", scale=0.8,
             masked=False),
        # an odd vocabulary in float32, part of it masked out
        dict(name="logprob_bwd_odd", op="logprob_bwd", T=333, V=50001, dtype="f32", scale=1.0, masked=True,
             mode="rceil", layout="k128"),
        # the loss gradient of a training batch, straight into the head's two gradient GEMMs
        dict(name="logprob_bwd_train", op="logprob_bwd", T=4096, V=131072, dtype="bf16", scale=1.0, masked=False,
             mode="rceil", layout="k128"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "swiglu_fwd", "swiglu_bwd", "logprob_fwd", "logprob_bwd"])
    mode, layout = rng.choice(["rceil", "floor"]), rng.choice(["k128", "k128", "plain"])
    step = 128 if layout == "k128" else 32
    if op.startswith("norm"):
        C = step * max(1, _log_int(rng, 256, 8192) // step)
        T = _log_int(rng, 1, min(16384, 80_000_000 // C))
        return dict(op=op, T=T, C=C, residual=rng.random() < 0.75, col=rng.random() < 0.75, ckpt=rng.random() < 0.5,
                    mode=mode, layout=layout)
    if op.startswith("swiglu"):
        H = step * max(1, _log_int(rng, 256, 14336) // step)
        T = _log_int(rng, 1, min(16384, 115_000_000 // H))
        return dict(op=op, T=T, H=H, mode=mode, layout=layout)
    V = _log_int(rng, 1000, 131072)
    T = _log_int(rng, 1, min(8192, 260_000_000 // V))
    case = dict(op=op, T=T, V=V, dtype=rng.choice(["bf16", "f32"]), scale=rng.choice([1.0, 0.7, 1.25]),
                masked=rng.random() < 0.3)
    if op == "logprob_fwd":
        return dict(case, top=rng.choice([0, 1, 5, 20, 64]))
    return dict(case, mode=mode, layout=layout)


def _up(n, m):
    return (n + m - 1) // m * m


def _step(case):
    return 128 if case["layout"] == "k128" else 32


def work(case):
    """Each input read once, each output written once; one 8-bit tensor is
    1 + 1/32 bytes a value."""
    op, T = case["op"], case["T"]
    q = 1 + 1 / 32
    if op == "norm_fwd":
        n = T * case["C"]
        col = _up(T, _step(case)) * case["C"] if case["col"] else 0
        b = n * (2 + (4 if case["residual"] else 0) + q + (q if case["ckpt"] else 0)) + q * col + 4 * case["C"] + 4 * T
        return {"bytes": b, "flops": 6 * n}
    if op == "norm_bwd":
        n = T * case["C"]
        col = _up(T, _step(case)) * case["C"] if case["col"] else 0
        b = n * (2 + (q if case["ckpt"] else 2) + (2 if case["residual"] else 0) + 2 + q) + q * col + 8 * case["C"]
        return {"bytes": b + 4 * T, "flops": 12 * n}
    if op == "swiglu_fwd":
        n, c = T * case["H"], _up(T, _step(case)) * case["H"]
        return {"bytes": n * (4 + 2 * q + q) + q * c, "flops": 8 * n}
    if op == "swiglu_bwd":
        n, c = T * case["H"], _up(T, _step(case)) * case["H"]
        return {"bytes": n * (2 + 2 * q + 2 * q) + 2 * q * c, "flops": 14 * n}
    n = T * case["V"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "logprob_fwd":
        return {"bytes": n * e + T * (8 + 4 + 4 + 8 + 8 * case["top"]), "flops": 5 * n}
    s = _step(case)
    vp = _up(case["V"], s)
    return {"bytes": n * e + q * T * vp + q * _up(T, s) * vp + 28 * T, "flops": 8 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, std, g, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _stream_like(T, C, g):
    """A residual stream: unit variance with a few strong channels."""
    gain = torch.ones(C, device="cuda")
    gain[torch.randint(0, C, (max(1, C // 512),), generator=g, device="cuda")] = 20.0
    return (torch.randn((T, C), generator=g, device="cuda") * gain).to(BF16)


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    st = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        C = case["C"]
        st["w"] = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
        x = _stream_like(T, C, g)
        if op == "norm_fwd":
            st["x"] = x
            st["r"] = _randn((T, C), 0.5, g) if case["residual"] else None
            return st
        st["dy"] = _randn((T, C), 1e-2, g)
        st["dsum"] = _randn((T, C), 1e-2, g) if case["residual"] else None
        st["rstd"] = torch.rsqrt(x.double().square().mean(-1) + EPS).float()
        if case["ckpt"]:
            st["x"] = None
            st["q_ck"], st["s_ck"] = _plain_quant(x, case["mode"], case["layout"])
        else:
            st["x"], st["q_ck"], st["s_ck"] = x, None, None
        return st
    if op in ("swiglu_fwd", "swiglu_bwd"):
        z = _randn((T, 2 * case["H"]), 1.5, g)
        if op == "swiglu_fwd":
            st["z"] = z
            return st
        st["dh"] = _randn((T, case["H"]), 1e-2, g)
        st["q_ck"], st["s_ck"] = _plain_quant(z, case["mode"], case["layout"])
        return st
    V = case["V"]
    x = _randn((T, V), 2.5, g, BF16 if case["dtype"] == "bf16" else F32)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    x.scatter_add_(1, tgt[:, None], torch.full((T, 1), 6.0, device="cuda", dtype=x.dtype))
    if case["masked"]:      # tokens that a grammar or a mask rules out, never the given one
        keep = x.gather(1, tgt[:, None])
        x[:, V // 3:V // 2] = -math.inf
        x.scatter_(1, tgt[:, None], keep)
    tgt[torch.rand(T, generator=g, device="cuda") < 0.1] = IGNORE
    st["x"], st["t"] = x, tgt
    if op == "logprob_bwd":
        f = _plain_logprob_fwd({"case": dict(case, top=0), "x": x, "t": tgt})
        st["stats"], st["entropy"] = f["stats"], f["entropy"]
        st["dlogp"] = torch.randn(T, generator=g, device="cuda") / T
        st["dent"] = 1e-2 * torch.randn(T, generator=g, device="cuda") / T
    return st


# --------------------------------------------------------------------------
# Plain form: elementary operations in float32
# --------------------------------------------------------------------------

def _plain_quant(v, mode, layout):
    """MXFP8 of a bf16 matrix along its rows: codes and scales (uint8). The
    scale exponent comes from the block maximum's bits, the codes from a cast
    of the scaled values."""
    R, C = v.shape
    b = v.float().reshape(R, C // 32, 32)
    bits = b.abs().amax(-1).contiguous().view(torch.int32)
    e = (bits >> 23) - 127 - 8
    if mode == "rceil":
        e = e + ((bits & 0x7FFFFF) > 0x600000).int()
    e = e.clamp(min=-127)
    inv = ((127 - e) << 23).view(F32)
    q = (b * inv[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).reshape(R, C)
    s = (e + 127).to(torch.uint8)
    if layout == "k128":
        s = s.reshape(R, C // 128, 4).permute(1, 0, 2).contiguous()
    return q, s


def _plain_dequant(q, s, layout):
    R, C = q.shape
    if layout == "k128":
        s = s.permute(1, 0, 2).reshape(R, C // 32)
    return (q.view(torch.float8_e4m3fn).float().reshape(R, C // 32, 32)
            * s.view(torch.float8_e8m0fnu).float()[..., None]).reshape(R, C)


def _rows_up(v, n):
    return v if v.shape[0] == n else torch.cat([v, v.new_zeros(n - v.shape[0], v.shape[1])])


def _plain_dual(v, case, row=True, col=True):
    """Both directions of a bf16 matrix; the column-wise one over its rows
    filled up with zeros to the block step."""
    out = {}
    if row:
        out["q_row"], out["s_row"] = _plain_quant(v, case["mode"], case["layout"])
    if col:
        vt = _rows_up(v, _up(v.shape[0], _step(case))).t().contiguous()
        out["q_col"], out["s_col"] = _plain_quant(vt, case["mode"], case["layout"])
    return out


def _plain_norm_fwd(st):
    case, out = st["case"], {}
    x = st["x"]
    if st["r"] is not None:
        x = (x.float() + st["r"].float()).to(BF16)
        out["sum"] = x
    xf = x.float()
    rstd = 1.0 / torch.sqrt(xf.square().mean(-1) + EPS)
    y = (xf * rstd[:, None] * st["w"]).to(BF16)
    out["rstd"] = rstd
    out.update(_plain_dual(y, case, True, case["col"]))
    if case["ckpt"]:
        out["q_ck"], out["s_ck"] = _plain_quant(x, case["mode"], case["layout"])
    return out


def _plain_norm_bwd(st):
    case = st["case"]
    x = _plain_dequant(st["q_ck"], st["s_ck"], case["layout"]) if case["ckpt"] else st["x"].float()
    xh = x * st["rstd"][:, None]
    dy = st["dy"].float()
    g = dy * st["w"]
    c = (g * xh).mean(-1, keepdim=True)
    dx = (g - xh * c) * st["rstd"][:, None]
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    dx = dx.to(BF16)
    out = {"dx": dx, "dw": (dy * xh).sum(0)}
    out.update(_plain_dual(dx, case, True, case["col"]))
    return out


def _plain_swiglu_fwd(st):
    case = st["case"]
    z = st["z"].float()
    a, b = z[:, :case["H"]], z[:, case["H"]:]
    h = (a / (1.0 + torch.exp(-a)) * b).to(BF16)
    out = _plain_dual(h, case)
    out["q_ck"], out["s_ck"] = _plain_quant(st["z"], case["mode"], case["layout"])
    return out


def _plain_swiglu_bwd(st):
    case = st["case"]
    z = _plain_dequant(st["q_ck"], st["s_ck"], case["layout"])
    a, b = z[:, :case["H"]], z[:, case["H"]:]
    dh = st["dh"].float()
    s = 1.0 / (1.0 + torch.exp(-a))
    dz = torch.cat([dh * b * s * (1.0 + a * (1.0 - s)), dh * a * s], 1).to(BF16)
    return _plain_dual(dz, case)


def _plain_logprob_fwd(st):
    case, t = st["case"], st["t"]
    x = st["x"].float()
    m = x.amax(-1)
    d = (x - m[:, None]) * case["scale"]
    e = torch.exp(d)
    s = e.sum(-1)
    ls = torch.log(s)
    ent = ls - torch.where(e > 0, e * d, 0.0).sum(-1) / s
    scored = t != IGNORE
    dt = d.gather(1, t.clamp(min=0)[:, None])[:, 0]
    out = {"logp": torch.where(scored, dt - ls, 0.0), "entropy": ent, "stats": torch.stack([m, ls], 1)}
    if case["top"]:
        # one whole-number key a value, larger for a larger value, then for a lower index
        u = x.contiguous().view(torch.int32).to(torch.int64)
        u = torch.where(u < 0, -(u & 0x7FFFFFFF), u)
        key = (u << 32) + (0x7FFFFFFF - torch.arange(x.shape[1], device=x.device))
        idx = key.topk(case["top"], -1, True, True).indices
        out["top_logp"] = d.gather(1, idx) - ls[:, None]
        out["top_idx"] = idx.int()
    return out


def _plain_logprob_bwd(st):
    case, t = st["case"], st["t"]
    x = st["x"].float()
    lp = (x - st["stats"][:, :1]) * case["scale"] - st["stats"][:, 1:]
    p = torch.exp(lp)
    scored = t != IGNORE
    g = torch.where(scored, st["dlogp"], 0.0)[:, None]
    grad = -p * (g + st["dent"][:, None] * (lp + st["entropy"][:, None]))
    grad = torch.where(p > 0, grad, 0.0)
    grad.scatter_add_(1, t.clamp(min=0)[:, None], g)
    grad = (grad * case["scale"]).to(BF16)
    V = x.shape[1]
    vp = _up(V, _step(case))
    if vp != V:
        grad = torch.cat([grad, grad.new_zeros(grad.shape[0], vp - V)], 1)
    return _plain_dual(grad, case)


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "swiglu_fwd": _plain_swiglu_fwd,
          "swiglu_bwd": _plain_swiglu_bwd, "logprob_fwd": _plain_logprob_fwd, "logprob_bwd": _plain_logprob_bwd}


# --------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------

def _own(st):
    from quantize_grouped_gemm_amd import lm

    case = st["case"]
    op = case["op"]
    if op.startswith("logprob"):
        if op == "logprob_fwd":
            return lm.token_logprobs(st["x"], st["t"], scale=case["scale"], top=case["top"])
        return lm.token_logprobs_bwd(st["x"], st["t"], st["stats"], st["entropy"], st["dlogp"], st["dent"],
                                     scale=case["scale"], mode=case["mode"], layout=case["layout"])
    kw = dict(mode=case["mode"], layout=case["layout"])
    if op == "norm_fwd":
        return lm.add_rmsnorm_quant(st["x"], st["w"], st["r"], eps=EPS, colwise=case["col"], checkpoint=case["ckpt"],
                                    **kw)
    if op == "norm_bwd":
        ck = (st["q_ck"], st["s_ck"]) if case["ckpt"] else None
        return lm.add_rmsnorm_bwd(st["dy"], st["w"], st["rstd"], x=st["x"], checkpoint=ck, dsum=st["dsum"],
                                  rowwise=True, colwise=case["col"], **kw)
    if op == "swiglu_fwd":
        H = case["H"]
        return lm.swiglu_ckpt_fwd(st["z"][:, :H], st["z"][:, H:], **kw)
    return lm.swiglu_ckpt_bwd(st["dh"], st["q_ck"], st["s_ck"], **kw)


def run(st):
    out = _own(st) if own else _PLAIN[st["case"]["op"]](st)
    return {k: v.view(torch.float8_e4m3fn) if k.startswith("q_") else v.view(torch.float8_e8m0fnu)
            if k.startswith("s_") else v for k, v in out.items()}


# --------------------------------------------------------------------------
# Values in 64 bits, from the definitions
# --------------------------------------------------------------------------

def _round(v, digits, emin):
    """Nearest number of `digits` binary digits (exponent at least emin), ties to even."""
    step = _pow2((torch.frexp(v)[1] - 1).clamp(min=emin) - (digits - 1))
    return torch.round(v / step) * step


def _bf(v):
    return _round(v, 8, -126)


def _pow2(e):
    """2^e exactly, from the bits of a float64 (exp2 and ldexp on the GPU are off by an ulp)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx64(v, case):
    """(code values, scale values) of a float64 matrix of bf16 numbers."""
    R, C = v.shape
    b = v.reshape(R, C // 32, 32)
    m = b.abs().amax(-1)
    e = torch.frexp(m)[1] - 9                 # 2^(e+8) <= m < 2^(e+9)
    if case["mode"] == "rceil":               # the smallest e with m <= 448 * 2^e
        e = torch.where(m > 448 * _pow2(e), e + 1, e)
    e = torch.where(m > 0, e, -127).clamp(min=-127)
    s = _pow2(e)
    q = _round(b / s[..., None], 4, -6).clamp(-448, 448).reshape(R, C)
    if case["layout"] == "k128":
        s = s.reshape(R, C // 128, 4).transpose(0, 1).contiguous()
    return q, s


def _dual64(v, case, col=True):
    out = {}
    out["q_row"], out["s_row"] = _mx64(v, case)
    if col:
        full = v.new_zeros(_up(v.shape[0], _step(case)), v.shape[1])
        full[:v.shape[0]] = v
        out["q_col"], out["s_col"] = _mx64(full.t().contiguous(), case)
    return out


def _value64(q, s, case):
    """The matrix that stored codes and scales stand for."""
    c = torch.arange(256, device=q.device)
    e, f = (c >> 3) & 15, (c & 7).double()
    val = torch.where(e > 0, (8 + f) * _pow2(e - 10), f * 2.0 ** -9) * torch.where(c > 127, -1.0, 1.0)
    if case["layout"] == "k128":
        s = s.transpose(0, 1).reshape(q.shape[0], -1)
    return val[q.long()] * _pow2(s.int() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = st["x"].double()
        out = {}
        if st["r"] is not None:
            x = _bf(x + st["r"].double())
            out["sum"] = x
        out["rstd"] = (torch.linalg.vector_norm(x, dim=1) ** 2 / case["C"] + EPS) ** -0.5
        out.update(_dual64(_bf(x * (out["rstd"][:, None] * st["w"].double())), case, case["col"]))
        if case["ckpt"]:
            out["q_ck"], out["s_ck"] = _mx64(x, case)
        return out
    if op == "norm_bwd":
        x = _value64(st["q_ck"], st["s_ck"], case) if case["ckpt"] else st["x"].double()
        r, w, dy = st["rstd"].double()[:, None], st["w"].double(), st["dy"].double()
        # y_i = w_i x_i r, dr/dx_j = -r^3 x_j / C
        dr = (dy * w * x).sum(1, keepdim=True)
        dx = dy * w * r - x * (r ** 3 * dr / case["C"])
        if st["dsum"] is not None:
            dx = dx + st["dsum"].double()
        dx = _bf(dx)
        return {"dx": dx, "dw": (dy * (x * r)).sum(0), **_dual64(dx, case, case["col"])}
    if op.startswith("swiglu"):
        H = case["H"]
        z = st["z"].double() if op == "swiglu_fwd" else _value64(st["q_ck"], st["s_ck"], case)
        a, b = z[:, :H], z[:, H:]
        sig = torch.sigmoid(a)
        if op == "swiglu_fwd":
            out = _dual64(_bf(a * sig * b), case)
            out["q_ck"], out["s_ck"] = _mx64(z, case)
            return out
        dh = st["dh"].double()
        return _dual64(_bf(torch.cat([dh * b * (sig + a * sig * torch.sigmoid(-a)), dh * (a * sig)], 1)), case)
    x, t = st["x"].double(), st["t"]
    scored = t != IGNORE
    at = torch.where(scored, t, 0)[:, None]
    if op == "logprob_fwd":
        lse = torch.logsumexp(x * case["scale"], 1)
        lp = x * case["scale"] - lse[:, None]
        out = {"logp": lp.gather(1, at)[:, 0] * scored, "entropy": torch.special.entr(lp.exp()).sum(1)}
        m = x.max(1).values
        out["stats"] = torch.stack([m, lse - m * case["scale"]], 1)
        if case["top"]:
            order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            out["top_logp"], out["top_idx"] = lp.gather(1, order), order.int()
        return out
    m, ls = st["stats"].double().unbind(1)
    lp = x * case["scale"] - (m * case["scale"] + ls)[:, None]
    p = lp.exp()
    d = torch.zeros_like(x).scatter_(1, at, scored.double()[:, None]) - p
    d = d * (st["dlogp"].double() * scored)[:, None]
    d += (torch.special.entr(p) - p * st["entropy"].double()[:, None]) * st["dent"].double()[:, None]
    d = _bf(d * case["scale"])
    full = d.new_zeros(d.shape[0], _up(d.shape[1], _step(case)))
    full[:, :d.shape[1]] = d
    return _dual64(full, case)
