"""Rows weighted into bf16's subnormal range are rounded once there too: the float32
product's own error is then below what float32 can hold."""

import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import moe, mx, synth

pytestmark = pytest.mark.gpu
F64, BF, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32


def _near_borders(top):
    """x [64, 128] of size 2^-100 and a weight a row that takes column 1 next to the middle of two subnormal bf16 values
    of size 2^top, from either side."""
    x = (synth.normal_bf16((64, 128), 1.0, synth.generator(21)).to(F64) * 2.0 ** -100).to(BF)
    g = torch.Generator().manual_seed(22)
    x[:, 1] = ((128 + 2 * torch.randint(0, 64, (64,), generator=g) + 1).to(F64) * 2.0 ** -107).to(BF)     # odd, 8 bits
    v = x[:, 1].to(F64)
    steps = torch.randint(2 ** (133 + top), 2 ** (134 + top), (64,), generator=g).to(F64)
    mid = (steps + 0.5) * 2.0 ** -133
    w = (mid / v).float()
    side = torch.arange(64) % 5 - 2                                       # two steps of the weight to either side
    w = (w.view(I32) + side.to(I32)).view(F32)
    assert int((w.to(F64) * v != mid).sum()) > 40
    return x, w


@pytest.mark.parametrize("top", [-130, -128, -127])
def test_one_rounding(gpu, top):
    x, w = _near_borders(top)
    src = torch.arange(64, dtype=I32)
    rows = R.gather(x, src, 1, w)
    twice = (x.float() * w[:, None]).to(BF)
    assert int((twice != rows).sum()) > 5      # what two roundings would give
    for col in (False, True):
        got = moe.gather_quantize(x.to(dev()), src.to(dev()), 1, w.to(dev()), colwise=col)
        ref = mx.quantize(rows.to(dev()), "rceil", True, False)
        for k, v in ref.items():
            assert torch.equal(got[k], v), f"{k}: {int((got[k] != v).sum())} differ"
    # what the codes stand for: every value of these rows is a multiple of 2^-133 that E4M3 holds to 4 bits
    q = mx.dequantize(got["q_row"], got["s_row"]).cpu().to(F64)
    off = (q - rows.to(F64)).abs()
    assert torch.all(off <= 2.0 ** -4 * rows.to(F64).abs() + 2.0 ** -137)
