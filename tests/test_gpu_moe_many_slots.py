"""Dispatch of more than 2^20 slots: its waves then hold more rounds of 64 slots than
stay in their registers, and read the rest from memory once to count and once to place."""

import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import moe

pytestmark = pytest.mark.gpu
I32 = torch.int32


# 2^20 + 1 slots (the first wave to hold more than 512), a ragged last chunk and wave, more than twice as many, one choice
@pytest.mark.parametrize("T,top,E,multiple", [((1 << 20) + 1, 1, 3, 128), (140001, 8, 64, 128), (140001, 8, 1000, 1),
                                              (300007, 8, 17, 16)])
def test_dispatch(gpu, T, top, E, multiple):
    print(f"T={T} top={top} E={E} multiple={multiple}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    # popular and rare experts, slots without one, and entries outside
    p = torch.exp(1.5 * torch.randn(E, generator=g))
    idx = torch.multinomial(p, T * top, replacement=True, generator=g).view(T, top).to(I32)
    idx[::37, 0] = -1
    idx[5::1001, top - 1] = E
    idx[T - 1, 0] = E - 1
    idx[7, 0], idx[T - 2, top - 1] = 2 ** 31 - 1, -2 ** 31
    cap = moe.capacity(T * top, E, multiple)
    got, ref = moe.dispatch(idx.to(dev()), E, multiple), R.dispatch(idx, E, multiple, cap)
    for k, v in ref.items():
        assert torch.equal(got[k].cpu(), v), f"{k}: {int((got[k].cpu() != v).sum())} of {v.numel()} differ"
