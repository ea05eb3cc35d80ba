"""Token log probabilities and their gradient where values are out of the
ordinary: rows of NaN, logits of large magnitude, rows with one token left,
targets predicted almost surely, gradients of any size.

Tolerances of the sums are those of test_gpu_lm_logprob (its docstring derives
them)."""

import math

import pytest
import torch

import lm_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import lm
from test_gpu_lm_logprob import _check_fwd

pytestmark = pytest.mark.gpu
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [64, 5000, 32000, 131072])
def test_alternatives_of_rows_with_nan(gpu, V, dtype):
    """Rows of NaN, whole or with a few other entries (fewer than alternatives;
    finite, masked, infinite), in whole rows and in rows split over workgroups:
    every result is NaN, and the alternatives are distinct tokens of the
    vocabulary, NaN first."""
    top = 20
    few = [3, V // 2, V - 1]
    rows = [torch.full((V,), NAN) for _ in range(7)]
    rows[1][few] = torch.tensor([1.0, -2.0, 3.0])
    rows[2][few] = -INF
    rows[3][: V // 2] = -INF
    rows[4] = torch.full((V,), -INF)
    rows[4][V - 5] = NAN
    rows[5] = torch.linspace(-3, 3, V)
    rows[5][V // 3] = NAN
    rows[6][few] = torch.tensor([INF, 0.0, -INF])
    x = torch.stack(rows).to(dtype).to(dev())
    t = torch.full((len(rows),), 3).to(dev())
    print(f"V={V} {dtype}", flush=True)
    out = lm.token_logprobs(x, t, top=top)
    for k in ("logp", "entropy", "top_logp"):
        assert torch.isnan(out[k]).all(), k
    idx = out["top_idx"].cpu().long()
    assert ((idx >= 0) & (idx < V)).all()
    nan = torch.isnan(x).cpu()
    for r in range(len(rows)):
        want = min(top, int(nan[r].sum()))
        assert idx[r].unique().numel() == top, r
        assert idx[r][:want].tolist() == nan[r].nonzero().flatten()[:want].tolist(), r
