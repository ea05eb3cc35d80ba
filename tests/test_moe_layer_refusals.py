"""Calls of MoELayer that its operators alone would let through: they are refused before
anything runs."""

import pytest
import torch

from _helpers import dev
from quantize_grouped_gemm_amd import moe_layer, mx

BF, F32 = torch.bfloat16, torch.float32


def z(*shape, dtype=BF, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


def raises(fn, *args, match, **kw):
    with pytest.raises(mx.MXError, match=match):
        fn(*args, **kw)


@pytest.mark.parametrize("recipe", ["mxfp8", "b128"])
def test_weights(recipe):
    make = lambda a, b, top=2: moe_layer.MoELayer(a, b, top, recipe)
    raises(make, z(4, 256, 128), z(128, 128), match="w2")
    raises(make, z(4, 256, 128).float(), z(4, 128, 128), match="w13")
    raises(make, z(4, 128, 128), z(4, 128, 128), match="w13")
    raises(make, z(3, 256, 128), z(4, 128, 128), match="w13")
    raises(make, z(4, 256, 256), z(4, 128, 128), match="w13")
    raises(make, z(4, 288, 128), z(4, 128, 144), match="multiples of 128")
    raises(make, z(4, 256, 144), z(4, 144, 128), match="multiples of 128")
    raises(make, z(4, 256, 128), z(4, 128, 128), match="cuda")
    layer = object.__new__(moe_layer.MoELayer)
    layer.E, layer.D, layer.H, layer.recipe = 4, 128, 128, recipe
    raises(layer.set_weights, z(5, 256, 128), z(5, 128, 128), match="w2")


def _calls(layer, d):
    f = layer.forward
    x, logits = z(5, 128, device=d), z(5, 4, dtype=F32, device=d)
    raises(f, x, logits[:4], match="logits")
    raises(f, x[:4], logits, match="logits")
    raises(f, x, z(5, 5, dtype=F32, device=d), match="logits")
    raises(f, x, z(5, 3, dtype=F32, device=d), match="logits")
    raises(f, z(5, 256, device=d), logits, match="x: ")
    raises(f, x.float(), logits, match="x: ")
    raises(f, x, logits, z(4, 128, device=d), match="r: ")
    raises(f, x, logits, z(5, 128, dtype=F32, device=d), match="r: ")
    raises(layer.backward, {"xq": {"q_row": x}, "x": x}, x, match="train=True")


@pytest.mark.parametrize("recipe", ["mxfp8", "b128"])
def test_calls(recipe):
    layer = object.__new__(moe_layer.MoELayer)
    layer.E, layer.D, layer.H, layer.top, layer.recipe, layer.bias, layer.routing = 4, 128, 128, 2, recipe, None, {}
    _calls(layer, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("recipe", ["mxfp8", "b128"])
def test_calls_on_the_device(gpu, recipe):
    d = dev()
    layer = moe_layer.MoELayer(z(4, 256, 128, device=d), z(4, 128, 128, device=d), 2, recipe)
    _calls(layer, d)
    x, logits = z(5, 128, device=d), z(5, 4, dtype=F32, device=d)
    out, c = layer.forward(x, logits)
    raises(layer.backward, c, x, match="train=True")
    out, c = layer.forward(x, logits, train=True)
    raises(layer.backward, c, z(6, 128, device=d), match="dout")
    assert set(layer.backward(c, x)) == {"dx", "dlogits", "dw13", "dw2"}
