"""Routing and its gradient on the GPU against the float64 formulas (moe_ref):
the choice exactly, weights to the roundings that they have."""

import numpy as np
import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import moe

pytestmark = pytest.mark.gpu
F64, BF, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32
INF = float("inf")

# s rounded to float32 (its share of the sum too), then the weight: three halves of an ulp
W_TOL = 3 * 2.0 ** -24 * (1 + 2.0 ** -20)


def _check(x, top, bias=None, **kw):
    out = moe.route(x.to(dev()), top, None if bias is None else bias.to(dev()), **kw)
    w, idx = R.route(x, top, bias, **kw)
    assert out["weights"].dtype is F32 and out["idx"].dtype is I32
    got = out["idx"].cpu()
    assert torch.equal(got, idx), f"{int((got != idx).sum())} of {idx.numel()} choices differ"
    g = out["weights"].cpu().to(F64)
    nan = torch.isnan(w)
    assert torch.equal(torch.isnan(g), nan)
    assert torch.all(((g - w).abs() <= W_TOL * w.abs() + 2.0 ** -149)[~nan])
    return out


def _logits(T, E, dtype, seed, std=1.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E + pad), generator=g) * std).to(dtype)[:, :E], g


# every register count with 64 lanes a token (with 16, of more than 16 experts: MANY below and
# test_gpu_moe_lanes), rows of any alignment, one expert and one token
SHAPES = [(0, 8, 2), (1, 1, 1), (1, 256, 8), (3, 5, 3), (7, 16, 4), (33, 33, 5), (100, 64, 6), (65, 128, 8), (50, 160, 6),
          (17, 200, 16), (9, 257, 8), (5, 512, 10), (4, 1000, 16), (6, 1024, 8), (2049, 24, 4), (2100, 33, 2),
          (2500, 100, 3), (2064, 256, 8), (2050, 255, 6)]


@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route(gpu, T, E, top, dtype):
    print(f"T={T} E={E} top={top} {dtype}", flush=True)
    for seed, (score, renorm, scale, with_bias) in enumerate([("softmax", True, 1.0, False), ("sigmoid", True, 2.5, True),
                                                              ("softmax", False, 0.5, True), ("sigmoid", False, 1.0, False)]):
        x, g = _logits(T, E, dtype, 100 * E + seed, pad=seed)
        bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
        _check(x, top, bias, score=score, renorm=renorm, scale=scale)


# groups whose experts fill whole lanes and share them (1 to 16 lanes a group), groups that straddle lanes, groups of one
GROUPS = [(70, 256, 8, 8, 4), (2100, 256, 8, 8, 3), (40, 64, 4, 16, 5), (40, 160, 6, 8, 3), (40, 96, 6, 3, 2),
          (40, 30, 4, 5, 2), (2100, 30, 4, 15, 4), (10, 16, 2, 16, 3), (33, 1024, 16, 2, 1), (33, 1024, 8, 16, 7),
          (33, 48, 3, 4, 1), (2100, 48, 3, 6, 4), (2100, 128, 8, 2, 1), (21, 512, 4, 4, 4), (2100, 240, 5, 10, 3)]


@pytest.mark.parametrize("T,E,top,groups,top_groups", GROUPS)
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_groups(gpu, T, E, top, groups, top_groups, group_score):
    print(f"T={T} E={E} top={top} groups={groups}/{top_groups} {group_score}", flush=True)
    for score in ("softmax", "sigmoid"):
        x, g = _logits(T, E, F32, E + groups)
        x[torch.rand(x.shape, generator=g) < 0.3] = -INF     # groups with one expert or none left
        bias = 0.2 * torch.randn(E, generator=g)
        _check(x, top, bias, score=score, groups=groups, top_groups=top_groups, group_score=group_score)


@pytest.mark.parametrize("T", [40, 2100])
def test_ties_go_to_the_lower_index(gpu, T):
    """Few distinct logits: equal experts and equal groups everywhere; scores that saturate to 1."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(0, 3, (T, 64), generator=g).to(BF)
    for score in ("softmax", "sigmoid"):
        _check(x, 12, score=score)
        _check(x, 12, score=score, groups=8, top_groups=3, group_score="max")
        _check(x, 12, torch.zeros(64), score=score, groups=8, top_groups=3)
    _check(torch.randint(20, 60, (T, 64), generator=g).to(F32), 12, score="sigmoid")
    _check(torch.zeros((T, 64)), 12, score="softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [12, 2100])
def test_rows_with_little_left(gpu, score, T):
    """No expert, one, and fewer than asked for; by the logits and by the bias; the type's lowest value is a value."""
    x, g = _logits(T, 24, F32, 6)
    x[0::4] = -INF
    x[1::4, 1:] = -INF
    x[2::4, 3:] = -INF
    out = _check(x, 6, score=score)
    assert torch.all(out["idx"][0::4] == -1) and torch.all(out["weights"][0::4] == 0)
    bias = torch.zeros(24)
    bias[5:] = -INF
    _check(x, 6, bias, score=score, groups=4, top_groups=2)
    low = torch.full((T, 24), torch.finfo(F32).min)
    low[:, 7] = 0
    _check(low, 6, score=score)
    _check(low.to(BF), 6, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [10, 2100])
def test_nan_and_infinity(gpu, score, T):
    x, g = _logits(T, 40, F32, 7)
    x[0, 3] = float("nan")
    x[1, 4] = INF
    x[2] = float("nan")
    x[3, 5], x[3, 6] = float("nan"), -INF
    x[4, 5:9] = INF
    x[5] = INF
    out = moe.route(x.to(dev()), 4, score=score)
    idx, w = out["idx"].cpu(), out["weights"].cpu()
    for t in range(6):      # distinct experts in range whatever the row holds
        assert len(set(idx[t].tolist())) == 4 and int(idx[t].min()) >= 0 and int(idx[t].max()) < 40
    if score == "softmax":
        assert torch.all(torch.isnan(w[:6]))
    else:
        assert torch.all(torch.isnan(w[0])) and idx[0, 0] == 3
        assert not torch.isnan(w[1]).any() and idx[1, 0] == 4
        assert idx[4].tolist() == [5, 6, 7, 8] and idx[5].tolist() == [0, 1, 2, 3]
    wr, ir = R.route(x[6:], 4, score=score)
    assert torch.equal(idx[6:], ir) and torch.allclose(w[6:].to(F64), wr, rtol=W_TOL, atol=0)
    dw = torch.ones((T, 4), device=dev())
    dx = moe.route_bwd(x.to(dev()), out["idx"], dw, score=score).cpu()
    assert torch.isfinite(dx[6:]).all()


def test_scores_decide_next_to_each_other(gpu):
    """Logits one float32 step apart: their scores round to the same float32 or to neighbours, never the wrong way."""
    g = torch.Generator().manual_seed(8)
    base = torch.randn(300, generator=g)
    x = base[:, None] + torch.arange(-8, 8)[None] * (2.0 ** -24 * base.abs()[:, None])
    x = x[:, torch.randperm(16, generator=g)].float().contiguous()
    for score in ("softmax", "sigmoid"):
        _check(x, 8, score=score)
        _check(x, 8, torch.full((16,), 0.25), score=score)


@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd(gpu, T, E, top, score):
    print(f"T={T} E={E} top={top} {score}", flush=True)
    for renorm, dtype in ((True, F32), (False, F32), (True, BF)):
        x, g = _logits(T, E, dtype, 7 * E + T, pad=T % 3)
        x[torch.rand(x.shape, generator=g) < 0.2] = -INF
        dw = torch.randn((T, top), generator=g)
        _, idx = R.route(x, top, score=score)
        if T > 2:
            idx[1] = idx[1, 0]             # the same expert more than once
            idx[2, top // 2] = E + 5       # an entry outside has no part
        got = moe.route_bwd(x.to(dev()), idx.to(dev()), dw.to(dev()), score=score, renorm=renorm, scale=1.5)
        assert got.dtype is dtype and got.shape == (T, E)
        ref = R.route_bwd(x, idx, dw, score, renorm, 1.5)
        # float64 inside: one rounding to float32 (and one to bf16), and what cancels in float64
        tol = 2.0 ** -24 * ref.abs() + (2.0 ** -8 * ref.abs() if dtype is BF else 0) + 1e-13
        off = (got.cpu().to(F64) - ref).abs()
        assert torch.all(off <= tol * (1 + 2.0 ** -6)), float(off.max())


def test_gradient_of_a_sure_choice(gpu):
    """Renormalised weights of one expert do not depend on its logit, and nearly sure ones keep their digits."""
    x = torch.tensor([[30.0, 0.0, -5.0, 1.0], [12.0, -12.0, 0.0, 0.0]])
    idx = torch.tensor([[0, 1], [0, 3]], dtype=I32)
    dw = torch.tensor([[1.0, -2.0], [0.5, 0.25]])
    for score in ("softmax", "sigmoid"):
        got = moe.route_bwd(x.to(dev()), idx.to(dev()), dw.to(dev()), score=score).cpu().to(F64)
        ref = R.route_bwd(x, idx, dw, score)
        assert torch.allclose(got, ref, rtol=2.0 ** -22, atol=1e-15), (got, ref)
        one = moe.route_bwd(x.to(dev()), idx[:, :1].contiguous().to(dev()), dw[:, :1].contiguous().to(dev()), score=score)
        assert float(one.abs().max()) <= 1e-15


def test_repeated_and_on_a_side_stream(gpu):
    x, _ = _logits(3000, 256, BF, 9)
    xd = x.to(dev())
    first = moe.route(xd, 8, score="sigmoid", groups=8, top_groups=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = moe.route(xd, 8, score="sigmoid", groups=8, top_groups=4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first["idx"], again["idx"]) and torch.equal(first["weights"], again["weights"])


# 16 lanes a token from 4097 tokens on: every register count, groups on whole lanes and across them
MANY = [(4100, 24, 4, 3, 2), (4097, 33, 2, 1, 1), (4101, 64, 6, 8, 3), (4100, 100, 3, 4, 2), (4100, 128, 8, 2, 1),
        (8200, 256, 8, 8, 4), (8197, 255, 6, 5, 3), (8193, 160, 6, 8, 3), (8200, 240, 16, 1, 1)]


@pytest.mark.parametrize("T,E,top,groups,top_groups", MANY)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(gpu, T, E, top, groups, top_groups, score):
    print(f"T={T} E={E} top={top} groups={groups}/{top_groups} {score}", flush=True)
    for dtype in (F32, BF):
        x, g = _logits(T, E, dtype, E + T, pad=T % 3)
        x[torch.rand(x.shape, generator=g) < 0.2] = -INF
        x[5] = -INF
        bias = 0.1 * torch.randn(E, generator=g)
        out = _check(x, top, bias, score=score, groups=groups, top_groups=top_groups)
        dw = torch.randn((T, top), generator=g)
        got = moe.route_bwd(x.to(dev()), out["idx"], dw.to(dev()), score=score)
        ref = R.route_bwd(x, out["idx"].cpu(), dw, score)
        tol = 2.0 ** -24 * ref.abs() + (2.0 ** -8 * ref.abs() if dtype is BF else 0) + 1e-13
        assert torch.all((got.cpu().to(F64) - ref).abs() <= tol * (1 + 2.0 ** -6))
