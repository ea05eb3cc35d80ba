"""SwiGLU with an 8-bit checkpoint on the GPU: against the float64 formulas,
and bit for bit against the library's own quantizer and dequantizer."""

import pytest
import torch

import lm_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import lm, mx, synth

pytestmark = pytest.mark.gpu
F64, BF = torch.float64, torch.bfloat16

SHAPES = [(0, 128, "k128"), (1, 32, "plain"), (1, 128, "k128"), (31, 160, "plain"), (33, 96, "plain"),
          (127, 384, "k128"), (128, 256, "k128"), (129, 2048, "k128"), (300, 1056, "plain"), (513, 640, "k128")]


def _z(T, H, seed, pad):
    t = synth.normal_bf16((T, 2 * H + pad), 1.5, synth.generator(seed)).to(dev())
    return t, t[:, :H], t[:, H:2 * H]


@pytest.mark.parametrize("mode", ["rceil", "floor"])
@pytest.mark.parametrize("T,H,layout", SHAPES)
def test_swiglu_ckpt(gpu, T, H, layout, mode):
    print(f"T={T} H={H} {layout} {mode}", flush=True)
    z, a, b = _z(T, H, T + 7 * H, pad=8 * (T % 3))
    out = lm.swiglu_ckpt_fwd(a, b, mode, layout)
    assert out["q_ck"].shape == (T, 2 * H) and out["q_col"].shape == (H, lm.padded_rows(T, layout))
    R.check_dual(out, R.swiglu(a.cpu().to(F64), b.cpu().to(F64)), mode, layout, "h")
    if T:
        ref = mx.quantize(z[:, :2 * H], mode, True, False, layout)
        assert torch.equal(out["q_ck"], ref["q_row"]) and torch.equal(out["s_ck"], ref["s_row"])
    dh = synth.normal_bf16((T, H + 16), 1e-2, synth.generator(T)).to(dev())[:, :H]
    got = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"], mode, layout)
    z64 = torch.from_numpy(R.O.dequantize(out["q_ck"].cpu().numpy(), R.plain_scales(out["s_ck"]))) if T else \
        torch.zeros((0, 2 * H), dtype=F64)
    d64, a64, b64 = dh.cpu().to(F64), z64[:, :H], z64[:, H:]
    s = torch.sigmoid(a64)
    mag = torch.cat([(d64 * b64 * s).abs() * (1 + a64.abs() * (1 - s)), (d64 * a64 * s).abs()], 1)
    R.check_dual(got, R.swiglu_bwd(d64, a64, b64), mode, layout, "dz", mag=mag)


@pytest.mark.parametrize("T,H", [(256, 384), (128, 2048)])
def test_agrees_with_the_bf16_operators(gpu, T, H):
    """Where the row count suits them, the operators without a checkpoint give
    the same bytes: forward on z, backward on the checkpoint's values (E4M3
    values are bf16 values)."""
    z, a, b = _z(T, H, 3, 0)
    out = lm.swiglu_ckpt_fwd(a, b)
    ref = mx.swiglu_quant_fwd(a, b)
    for k in ("q_row", "s_row", "q_col", "s_col"):
        assert torch.equal(out[k], ref[k]), k
    zq = mx.dequantize(out["q_ck"], out["s_ck"], BF)
    dh = synth.normal_bf16((T, H), 1e-2, synth.generator(4)).to(dev())
    got = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"])
    ref = mx.swiglu_quant_bwd(dh, zq[:, :H], zq[:, H:])
    for k in ("q_row", "s_row", "q_col", "s_col"):
        assert torch.equal(got[k], ref[k]), k


@pytest.mark.parametrize("T,H,layout", [(8192, 384, "k128"), (8200, 160, "plain"), (9001, 128, "k128")])
def test_tile_orders_agree(gpu, T, H, layout):
    """From 8192 rows on the tiles are walked in another order: the same bytes
    as from shorter calls over the same rows (multiples of the block step)."""
    z, a, b = _z(T, H, 17, 0)
    dh = synth.normal_bf16((T, H), 1e-2, synth.generator(18)).to(dev())
    out = lm.swiglu_ckpt_fwd(a, b, layout=layout)
    got = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"], layout=layout)
    for r0 in range(0, T, 4096):
        r1 = min(r0 + 4096, T)
        part = lm.swiglu_ckpt_fwd(a[r0:r1], b[r0:r1], layout=layout)
        pb = lm.swiglu_ckpt_bwd(dh[r0:r1], part["q_ck"], part["s_ck"], layout=layout)
        cols = slice(r0, r0 + lm.padded_rows(r1 - r0, layout))
        for whole, piece, keys in ((out, part, ("row", "ck")), (got, pb, ("row",))):
            for k in keys:
                assert torch.equal(whole["q_" + k][r0:r1], piece["q_" + k]), (k, r0)
            assert torch.equal(whole["q_col"][:, cols], piece["q_col"]), r0
            if layout == "plain":
                assert torch.equal(whole["s_row"][r0:r1], piece["s_row"])
                assert torch.equal(whole["s_col"][:, cols.start // 32:cols.stop // 32], piece["s_col"])
            else:
                assert torch.equal(whole["s_row"][:, r0:r1], piece["s_row"])
                assert torch.equal(whole["s_col"][cols.start // 128:cols.stop // 128], piece["s_col"])


def test_special_values(gpu):
    """Zero halves give zeros, a NaN block stays a NaN block and reaches only
    its own gradients, every scale byte is read back."""
    T, H = 32, 128
    z, a, b = _z(T, H, 9, 0)
    z[0] = 0
    z[4, 5] = float("nan")
    out = lm.swiglu_ckpt_fwd(a, b, layout="plain")
    assert not out["q_row"][0].any() and not out["q_ck"][0].any()
    assert out["s_ck"][4, 0] == 255 and (out["s_ck"][4, 1:] != 255).all()
    dh = torch.ones((T, H), dtype=BF, device=dev())
    got = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"], layout="plain")
    assert (got["s_row"][4] == 255).nonzero().flatten().tolist() == [0, H // 32]
    assert (got["s_row"][5] != 255).all()
    # every scale byte: dB = dh a sigmoid(a) with b = 0
    q = torch.zeros((256, 64), dtype=torch.uint8, device=dev())
    q[:, :32] = 0x38     # 1.0
    s = torch.arange(256, dtype=torch.uint8, device=dev())[:, None].repeat(1, 2)
    one = torch.ones((256, 32), dtype=BF, device=dev())
    got = lm.swiglu_ckpt_bwd(one, q, s, layout="plain")
    av = torch.pow(2.0, torch.arange(255, dtype=F64) - 127)
    v = av * torch.sigmoid(av)
    R.check_codes(got["q_row"][:255, 32:], got["s_row"][:255, 1:], v[:, None].repeat(1, 32).clamp(max=2.0 ** 127),
                  "rceil", "dB")
    assert got["s_row"][255, 1] == 255


def test_every_code_under_every_scale(gpu):
    """The checkpoint's values for all 256 codes under all scale bytes: the
    gradient from it equals the one from the dequantized bf16 tensor (exact for
    scales whose values bf16 holds: E from -117 to 119). A NaN that arithmetic
    produced has no defined sign: that bit is left out where the value is NaN."""
    E = torch.arange(10, 247)
    q = torch.arange(256, dtype=torch.uint8).repeat(E.numel(), 2).to(dev())          # a: all codes, b: all codes
    s = E.to(torch.uint8)[:, None].repeat(1, 16).to(dev())
    dh = torch.full((E.numel(), 256), 2.0 ** -60, dtype=BF, device=dev())
    got = lm.swiglu_ckpt_bwd(dh, q, s, layout="plain")
    z = mx.dequantize(q, s, BF)
    T = lm.padded_rows(E.numel(), "plain")
    zp = torch.zeros((T, 512), dtype=BF, device=dev())
    zp[:E.numel()] = z
    dp = torch.zeros((T, 256), dtype=BF, device=dev())
    dp[:E.numel()] = dh
    ref = mx.swiglu_quant_bwd(dp, zp[:, :256], zp[:, 256:], layout="plain")
    assert torch.equal(got["s_row"], ref["s_row"][:E.numel()])
    sign = torch.isnan(z[:, :256] + z[:, 256:]).to(torch.uint8).repeat(1, 2) * 0x80
    assert torch.equal(got["q_row"] | sign, ref["q_row"][:E.numel()] | sign)
