"""The routing gradient where chosen scores are 0 as float32: the forward's weights
are 0 there whatever the logits, so the gradient has no part from them."""

import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import moe

F64, BF, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32
INF = float("inf")
# scores of 0 as float32: sigmoid(x) and, next to a logit of 0, softmax(x) below 2^-150
LOW = [-120.0, -800.0, -1e4, torch.finfo(F32).min, -INF]


def _there(x, idx, score):
    """idx without the entries whose score is 0 as a float32."""
    s = R.scores(x.to(F64), score).float()
    ok = (idx >= 0) & (idx < x.shape[1])
    si = s.gather(1, torch.where(ok, idx, torch.zeros_like(idx)).long())
    return torch.where(ok & (si == 0), torch.full_like(idx, -1), idx)


def _rows(score, E, dtype):
    """Rows of logits and the experts chosen of them: all of the chosen low, one of them not, scores that float32
    holds as subnormal numbers, and ordinary ones."""
    g = torch.Generator().manual_seed(11)
    x, idx = [], []
    for low in LOW:
        for rest in (low, 0.0):
            row = torch.full((E,), rest)
            row[:4] = low
            if score == "softmax":
                row[E - 1] = 0.0
            x.append(row)
            idx.append([0, 1, 2, 3])
        one = row.clone()
        one[2] = 0.5
        x.append(one)
        idx.append([0, 1, 2, 3])
    sub = torch.zeros(E)
    sub[:4] = torch.tensor([-100.0, -101.0, -100.5, -130.0])
    x += [sub, torch.randn(E, generator=g), torch.full((E,), -INF)]
    idx += [[0, 1, 2, 3], [1, 1, 3, E + 2], [-1, -1, -1, -1]]
    return torch.stack(x).to(dtype), torch.tensor(idx, dtype=I32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_formula_against_differences(score, renorm):
    x, idx = _rows(score, 9, F64)
    keep = torch.isfinite(x).all(1) & (x.abs().amax(1) < 1e6)
    x, idx = x[keep], idx[keep]
    dw = torch.randn(idx.shape, generator=torch.Generator().manual_seed(3), dtype=F64)

    def weights(v):
        return (R.route_weights(v, _there(v, idx, score), score, renorm, 2.5) * dw).sum()

    got = R.route_bwd(x, _there(x, idx, score), dw, score, renorm, 2.5)
    ref, h = torch.zeros_like(x), 1e-6
    for i in range(x.numel()):
        d = torch.zeros(x.numel(), dtype=F64)
        d[i] = h
        ref.view(-1)[i] = (weights(x + d.view_as(x)) - weights(x - d.view_as(x))) / (2 * h)
    assert torch.allclose(got, ref, rtol=1e-6, atol=1e-8)


# both lane counts a token (16 lanes: few experts, or more than 4096 rows), experts that fill the lanes and do not
@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(18, 16), (18, 9), (18, 40), (18, 256), (18, 1000), (4100, 40), (4104, 256)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradient_follows_the_forward(gpu, T, E, score, dtype):
    x, idx = _rows(score, E, dtype)
    n = -(-T // x.shape[0])
    x, idx = x.repeat(n, 1)[:T], idx.repeat(n, 1)[:T]
    g = torch.Generator().manual_seed(T + E)
    for renorm in (True, False):
        for size in (1.0, 1e6):
            dw = size * torch.randn((T, 4), generator=g)
            got = moe.route_bwd(x.to(dev()), idx.to(dev()), dw.to(dev()), score=score, renorm=renorm, scale=1.5).cpu().to(F64)
            there = _there(x, idx, score)
            ref = R.route_bwd(x, there, dw, score, renorm, 1.5)
            # float64 inside, some ten roundings and an exponential off by 2^-50 of terms up to 1.5 |dw|, then one
            # rounding to float32 (and one to bf16)
            tol = (2.0 ** -24 + (2.0 ** -8 if dtype is BF else 0)) * ref.abs() * (1 + 2.0 ** -6)
            tol = tol + 2.0 ** -45 * float(dw.abs().max()) + 2.0 ** -149
            assert torch.isfinite(got).all()
            off = (got - ref).abs()
            assert torch.all(off <= tol), (renorm, size, int((off > tol).any(1).nonzero()[0]), float(off.max()))
            if renorm:
                none = (there < 0).all(1)
                assert int(none.sum()) >= T // 2 and torch.all(got[none] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 4100])
def test_forward_of_low_logits(gpu, T):
    """The weights that the gradient belongs to: 0 where every score is 0, and a choice of value 0 like any other."""
    for low in LOW[:-1]:
        x = torch.full((T, 24), low)
        out = moe.route(x.to(dev()), 4, score="sigmoid")
        assert torch.all(out["weights"] == 0) and out["idx"].cpu().tolist() == [[0, 1, 2, 3]] * T
        dw = torch.tensor([1.0, -1.0, 2.0, 0.5]).expand(T, 4).contiguous()
        assert torch.all(moe.route_bwd(x.to(dev()), out["idx"], dw.to(dev()), score="sigmoid") == 0)
