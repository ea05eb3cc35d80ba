"""Strides of operands with one row or one column: whatever torch reports for a
dimension of size one, the operators take the matrix."""

import pytest
import torch

from _helpers import dev
from quantize_grouped_gemm_amd import lm, mx

U8, BF, F32, I64 = torch.uint8, torch.bfloat16, torch.float32, torch.int64


def _row(C, device, dtype=BF):
    """[1, C] with strides (1, 1), contiguous as torch sees it."""
    t = torch.linspace(-2, 2, C).to(dtype).to(device)[:, None].t()
    assert t.shape == (1, C) and t.stride() == (1, 1) and t.is_contiguous()
    return t


def _column(T, device, dtype=BF):
    """[T, 1] with strides (1, T)."""
    t = torch.linspace(-2, 2, T).to(dtype).to(device)[None].t()
    assert t.shape == (T, 1) and t.stride() == (1, T)
    return t


def _calls(device):
    C = 256
    x, w, rstd = _row(C, device), torch.ones(C, device=device), torch.ones(1, device=device)
    t1, tn = torch.zeros(1, dtype=I64, device=device), torch.zeros(5, dtype=I64, device=device)
    q, s = torch.full((1, 2 * C), 0x38, dtype=U8, device=device), torch.full((4, 1, 4), 127, dtype=U8, device=device)
    st1, e1 = torch.zeros((1, 2), device=device), torch.zeros(1, device=device)
    st5, e5 = torch.zeros((5, 2), device=device), torch.zeros(5, device=device)
    return [("norm", lambda v, **k: lm.add_rmsnorm_quant(v, w, v, colwise=True, **k), x),
            ("norm_bwd", lambda v, **k: lm.add_rmsnorm_bwd(v, w, rstd, x=v, dsum=v, **k), x),
            ("swiglu", lambda v, **k: lm.swiglu_ckpt_fwd(v, v, **k), x),
            ("swiglu_bwd", lambda v, **k: lm.swiglu_ckpt_bwd(v, q, s, **k), x),
            ("logprobs", lambda v, **k: lm.token_logprobs(v, t1, top=3, **k), x),
            ("logprobs_bwd", lambda v, **k: lm.token_logprobs_bwd(v, t1, st1, e1, e1 + 1, **k), x),
            ("one_token", lambda v, **k: lm.token_logprobs(v, tn, top=1, **k), _column(5, device)),
            ("one_token_bwd", lambda v, **k: lm.token_logprobs_bwd(v, tn, st5, e5, e5 + 1, **k), _column(5, device))]


@pytest.mark.parametrize("i", range(8))
def test_accepted_up_to_the_device(i):
    """On the CPU every check passes up to the one of the device."""
    _, call, v = _calls("cpu")[i]
    with pytest.raises(mx.MXError, match="cuda"):
        call(v)


def test_strides_that_matter_are_still_refused():
    w = torch.ones(256)
    for bad in (torch.zeros((256, 2), dtype=BF).t(), torch.zeros((1, 256), dtype=BF).expand(2, 256),
                torch.zeros((1, 512), dtype=BF)[:, ::2]):
        with pytest.raises(mx.MXError, match="contiguous rows"):
            lm.add_rmsnorm_quant(bad, w)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(8))
def test_same_results_as_from_a_copy(gpu, i):
    """Both paths of the binding (with outputs allocated and with given ones)."""
    name, call, v = _calls(dev())[i]
    ref = call(torch.empty(v.shape, dtype=v.dtype, device=v.device).copy_(v))
    for got in (call(v), call(v, out={})):
        assert got.keys() == ref.keys()
        for k in ref:
            assert torch.equal(got[k], ref[k]), (name, k)
