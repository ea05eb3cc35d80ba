"""Residual addition + RMS norm + MXFP8 output and its gradient on the GPU,
against the float64 formulas (lm_ref), and bit for bit against the library's
own quantizer where the bf16 tensor that was quantized is known."""

import pytest
import torch

import lm_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import lm, mx, synth

pytestmark = pytest.mark.gpu
F64, BF = torch.float64, torch.bfloat16

# T, C, layout: one row and none, tile and block edges, every row shape of
# the kernels (columns below and above 512, 2048, 4096, 6144 and 8192)
SHAPES = [(0, 128, "k128"), (1, 128, "k128"), (1, 4096, "k128"), (31, 32, "plain"), (33, 544, "plain"),
          (130, 2080, "plain"), (257, 640, "k128"), (129, 5120, "k128"), (40, 7168, "k128"), (17, 8192, "k128"),
          (34, 16384, "k128"), (1000, 384, "k128")]


def _rows(T, C, std, g, pad=0):
    """bf16 [T, C] on the GPU whose rows are C + pad apart, and its float64 copy."""
    t = synth.normal_bf16((T, C + pad), std, g).to(dev())[:, :C]
    return t, t.cpu().to(F64)


def _eq(a, b, what):
    assert torch.equal(a, b), f"{what}: {int((a != b).sum())} of {a.numel()} differ"


def _mx_rows(v, mode, layout):
    return mx.quantize(v, mode, True, False, layout)


def _mx_cols(v, mode, layout):
    p = lm.padded_rows(v.shape[0], layout)
    full = torch.zeros((p, v.shape[1]), dtype=BF, device=v.device)
    full[:v.shape[0]] = v
    return mx.quantize(full, mode, False, True, layout)


@pytest.mark.parametrize("variant", ["plain_norm", "residual", "residual_ckpt_col", "col", "ckpt"])
@pytest.mark.parametrize("T,C,layout", SHAPES)
def test_norm_fwd(gpu, T, C, layout, variant):
    mode = "floor" if (T + C // 32) % 2 else "rceil"
    res, col, ck = "residual" in variant, "col" in variant, "ckpt" in variant
    print(f"T={T} C={C} {layout} {mode} {variant}", flush=True)
    g = synth.generator(T * 31 + C)
    x, x64 = _rows(T, C, 1.0, g, pad=8 * (T % 3))
    r, r64 = _rows(T, C, 0.5, g, pad=8 * (T % 2)) if res else (None, None)
    w = 1 + 0.1 * torch.randn(C, generator=g)
    out = lm.add_rmsnorm_quant(x, w.to(dev()), r, eps=1e-6, mode=mode, layout=layout, colwise=col, checkpoint=ck)
    assert ("sum" in out) == res and ("q_col" in out) == col and ("q_ck" in out) == ck
    s = (x.float() + r.float()).to(BF) if res else x.contiguous()
    if res:
        _eq(out["sum"], s, "sum")
    s64 = s.cpu().to(F64)
    rstd, y = R.norm_fwd(s64, w.to(F64), 1e-6)
    # a thread's 16 squares in float32 (half of their 16 roundings after the root), the rest in float64
    assert torch.all((out["rstd"].cpu().to(F64) / rstd - 1).abs() <= 10 * 2.0 ** -24)
    R.check_dual(out, y, mode, layout, "y", True, col)
    # y formed from the kernel's own statistic by the same steps: rstd = h + l
    # with h its upper 8 bits, then fma(s h, w, (s l) w); the sum in float64
    # holds the fused product exactly
    h = (out["rstd"].view(torch.int32) & -65536).view(torch.float32)[:, None]
    lo = ((s.float() * (out["rstd"][:, None] - h)) * w.to(dev())).to(F64)
    yk = ((s.float() * h).to(F64) * w.to(dev()).to(F64) + lo).float().to(BF)
    if T:
        ref = _mx_rows(yk, mode, layout)
        _eq(out["q_row"], ref["q_row"], "q_row")
        _eq(out["s_row"], ref["s_row"], "s_row")
        if col:
            ref = _mx_cols(yk, mode, layout)
            _eq(out["q_col"], ref["q_col"], "q_col")
            _eq(out["s_col"], ref["s_col"], "s_col")
        if ck:
            ref = _mx_rows(s, mode, layout)
            _eq(out["q_ck"], ref["q_row"], "q_ck")
            _eq(out["s_ck"], ref["s_row"], "s_ck")


@pytest.mark.parametrize("variant", ["x", "x_dsum_col", "ckpt", "ckpt_dsum_col", "x_norow"])
@pytest.mark.parametrize("T,C,layout", SHAPES)
def test_norm_bwd(gpu, T, C, layout, variant):
    mode = "floor" if (T + C // 32) % 2 else "rceil"
    ck, col, res = "ckpt" in variant, "col" in variant, "dsum" in variant
    row = "norow" not in variant
    print(f"T={T} C={C} {layout} {mode} {variant}", flush=True)
    g = synth.generator(T * 37 + C)
    x, x64 = _rows(T, C, 1.0, g, pad=8 * (T % 3))
    dy, dy64 = _rows(T, C, 1e-2, g, pad=8 * (T % 2))
    ds, ds64 = _rows(T, C, 1e-2, g) if res else (None, None)
    w = 1 + 0.1 * torch.randn(C, generator=g)
    rstd, _ = R.norm_fwd(x64, w.to(F64), 1e-6)
    rstd = rstd.float()
    kw = dict(x=x)
    if ck:
        q = lm.add_rmsnorm_quant(x, w.to(dev()), mode=mode, layout=layout, checkpoint=True)
        kw = dict(checkpoint=(q["q_ck"], q["s_ck"]))
        x64 = torch.from_numpy(R.O.dequantize(q["q_ck"].cpu().numpy(), R.plain_scales(q["s_ck"]))) if T else x64
    out = lm.add_rmsnorm_bwd(dy, w.to(dev()), rstd.to(dev()), dsum=ds, mode=mode, layout=layout, rowwise=row,
                             colwise=col, **kw)
    rs = rstd.to(F64)
    dx, dw = R.norm_bwd(dy64, w.to(F64), rs, x64, ds64)
    xh = x64 * rs[:, None]
    gw = (dy64 * w.to(F64)).abs()
    mag = (gw + xh.abs() * (gw * xh.abs()).mean(-1, keepdim=True)) * rs[:, None]
    if res:
        mag = mag + ds64.abs()
    got = out["dx"].cpu().to(F64)
    assert torch.all((got - dx).abs() <= 2.0 ** -8 * dx.abs() + 2 * R.F32 * mag)
    # dw: partial sums of up to 16 rows, then up to 32 sequential parts and a tree of 32
    assert torch.all((out["dw"].cpu().to(F64) - dw).abs() <= 96 * 2.0 ** -24 * (dy64 * xh).abs().sum(0) + 1e-30)
    R.check_dual(out, dx, mode, layout, "dx", row, col, mag)
    if T and row:
        ref = _mx_rows(out["dx"], mode, layout)
        _eq(out["q_row"], ref["q_row"], "q_row")
        _eq(out["s_row"], ref["s_row"], "s_row")
    if T and col:
        ref = _mx_cols(out["dx"], mode, layout)
        _eq(out["q_col"], ref["q_col"], "q_col")
        _eq(out["s_col"], ref["s_col"], "s_col")


def test_norm_repeats_bit_for_bit(gpu):
    """The sums run in a fixed order: the same call gives the same bits."""
    g = synth.generator(5)
    x, _ = _rows(999, 1536, 1.0, g)
    dy, _ = _rows(999, 1536, 1e-2, g)
    w = torch.ones(1536, device=dev())
    f = lm.add_rmsnorm_quant(x, w)
    a = lm.add_rmsnorm_bwd(dy, w, f["rstd"], x=x, colwise=True)
    for _ in range(3):
        b = lm.add_rmsnorm_bwd(dy, w, f["rstd"], x=x, colwise=True)
        for k in a:
            _eq(a[k], b[k], k)


def test_norm_special_rows(gpu):
    """A zero row (eps only), a row of subnormals, a row with a NaN and one
    with an infinity: the bad rows stay bad and the others are untouched."""
    T, C = 64, 256
    g = synth.generator(6)
    x, _ = _rows(T, C, 1.0, g)
    w = torch.ones(C, device=dev())
    clean = lm.add_rmsnorm_quant(x, w, layout="plain")
    y = x.clone()
    y[3] = 0
    y[5] = 1e-39
    y[7, 9] = float("nan")
    y[11, 200] = float("inf")
    out = lm.add_rmsnorm_quant(y, w, layout="plain", colwise=True, checkpoint=True)
    keep = [i for i in range(T) if i not in (3, 5, 7, 11)]
    for k in ("q_row", "s_row"):
        _eq(out[k][keep], clean[k][keep], k)
    assert not out["q_row"][3].any() and abs(out["rstd"][3].item() - 1e3) < 1e-2
    assert torch.isfinite(out["rstd"][5])
    assert torch.isnan(out["rstd"][7]) and (out["s_row"][7] == 255).all()
    assert out["rstd"][11].item() == 0 and out["s_row"][11, 200 // 32] == 255
    assert out["s_ck"][7, 0] == 255 and (out["s_ck"][7, 1:] < 255).all()
