"""Routing with 16 lanes a token at its edges. Experts up to 256 take 16 lanes from 4097
tokens on (up to 16 experts always), and 64 lanes below; the two have exchanges and
group joins of their own, so what test_gpu_moe_route checks with few tokens is checked
here with many."""

import pytest
import torch

import moe_ref as R
import test_gpu_moe_route as few
from _helpers import dev
from quantize_grouped_gemm_amd import moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T = 4100


# every register count (1 to 16), experts that end inside a lane, and one expert more than 16 lanes take
@pytest.mark.parametrize("E,top", [(8, 2), (17, 3), (24, 4), (33, 2), (64, 6), (100, 3), (128, 8), (160, 6), (240, 16), (255, 6),
                                   (256, 8), (257, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route(gpu, E, top, dtype):
    few.test_route(gpu, T, E, top, dtype)


@pytest.mark.parametrize("E,top", [(8, 2), (24, 4), (33, 2), (100, 3), (200, 16), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd(gpu, E, top, score):
    few.test_route_bwd(gpu, T + 1, E, top, score)


@pytest.mark.parametrize("E,top,groups,top_groups", [(256, 8, 8, 3), (256, 6, 2, 1), (256, 8, 16, 7), (128, 8, 2, 1), (64, 4, 16, 5),
                                                     (30, 4, 15, 4), (48, 3, 6, 4), (96, 6, 3, 2), (160, 6, 8, 3), (240, 5, 10, 3)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups(gpu, E, top, groups, top_groups, group_score):
    few.test_route_groups(gpu, T + 2, E, top, groups, top_groups, group_score)


def test_ties(gpu):
    few.test_ties_go_to_the_lower_index(gpu, T)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_little_left(gpu, score):
    few.test_rows_with_little_left(gpu, score, T)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinity(gpu, score):
    few.test_nan_and_infinity(gpu, score, T)


def test_both_lane_counts_give_the_same(gpu):
    """The same rows among many and alone: equal choices, and equal weights (the sums differ by float64 roundings)."""
    for E, groups in ((256, 8), (100, 4), (20, 1)):
        x, g = few._logits(T, E, F32, E)
        x[torch.rand(x.shape, generator=g) < 0.2] = -float("inf")
        for score in ("softmax", "sigmoid"):
            kw = dict(score=score, groups=groups, top_groups=max(1, groups // 2))
            many, alone = moe.route(x.to(dev()), 4, **kw), moe.route(x[-600:].contiguous().to(dev()), 4, **kw)
            assert torch.equal(many["idx"][-600:], alone["idx"])
            assert torch.allclose(many["weights"][-600:], alone["weights"], rtol=2.0 ** -23, atol=0)
            ref = R.route(x[-600:], 4, **kw)[1]
            assert torch.equal(alone["idx"].cpu(), ref)
