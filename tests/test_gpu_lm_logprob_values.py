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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [9001, 131072])
def test_logits_of_large_magnitude(gpu, V, dtype):
    """Finite masks of -1e10 and -5e29 over runs of tokens and over whole rows,
    common offsets of any size, one entry far above ordinary ones that rise from
    tile to tile: differences of logits decide, not their size."""
    top = 20
    g = torch.Generator().manual_seed(V)
    base = torch.randn(V, generator=g)
    i = torch.arange(V)
    run = (i >= V // 8) & (i < V - V // 4)

    def masked(m, at):
        return torch.where(at, torch.tensor(m), base)

    rising = base + 22.0 * (i // 2048).float().clamp(max=3)
    spike = rising.clone()
    spike[V - 2] = 6e28
    step = 2.0 ** 10 * (torch.arange(V) % 5).float()
    rows = [masked(-1e10, run), masked(-1e10, ~run), torch.full((V,), -1e10), masked(-5e29, run), torch.full((V,), -5e29),
            spike, rising, masked(-3e9, i != 7), masked(-1e9, run), torch.full((V,), 7e9), -1e10 + step, 2.0 ** 34 + step,
            2.0 ** 70 * (1 + (i % 7).float()), torch.full((V,), -1.7e8) + step, base + 9e7]
    x = torch.stack(rows).to(dtype).to(dev())
    t = torch.full((len(rows),), 7).to(dev())
    t[1::2] = V - 3
    print(f"V={V} {dtype}", flush=True)
    _check_fwd(lm.token_logprobs(x, t, scale=0.7, top=top), x, t, float(torch.tensor(0.7)), top)
    _check_fwd(lm.token_logprobs(x, t, top=top), x, t, 1.0, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [700, 9001, 100003])
def test_rows_with_one_token_left(gpu, V, dtype):
    """The only token left has probability 1: log probability and entropy are
    exactly 0, wherever it stands and whatever its logit is; next to tokens that
    are all but impossible, no log probability is above 0 and no entropy below."""
    T = 300
    g = torch.Generator().manual_seed(V)
    x = torch.full((T, V), -INF)
    t = torch.randint(0, V, (T,), generator=g)
    x[torch.arange(T), t] = 12.0 * torch.randn(T, generator=g)
    for rows in (T, 100):                     # 100: rows that long are split over workgroups
        for scale in (1.0, 0.83):
            xd, td = x[:rows].to(dtype).to(dev()), t[:rows].to(dev())
            out = lm.token_logprobs(xd, td, scale=scale, top=2)
            for k in ("logp", "entropy"):
                assert not out[k].any(), (k, int((out[k] != 0).sum()))
            assert not out["stats"][:, 1].any() and not out["top_logp"][:, 0].any()
            # others from 15 to 40 below
            near = torch.where(x[:rows] == -INF, 15.0 + 25.0 * torch.rand((rows, V), generator=g), 0.0)
            near = (x[:rows].amax(-1, keepdim=True) - near / scale).to(dtype).to(dev())
            out = lm.token_logprobs(near, td, scale=scale, top=2)
            assert (out["logp"] <= 0).all() and (out["entropy"] >= 0).all() and (out["stats"][:, 1] >= 0).all()
            assert (out["top_logp"] <= 0).all()


def _sure_rows(T, V, dtype, scale, lo, hi, seed):
    """Rows whose target holds all but e^-lo .. e^-hi of the probability, in
    random places; on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, V), generator=g) / scale
    t = torch.randint(0, V, (T,), generator=g)
    rest = torch.logsumexp(x.to(F64) * scale, -1)
    x[torch.arange(T), t] = ((rest + torch.linspace(lo, hi, T).to(F64)) / scale).float()
    return x.to(dtype).to(dev()), t.to(dev())


def _other_codes(out, grad, mode):
    """How many of the values that out's row-wise codes stand for are not those
    of bf16(grad) quantized."""
    qr, sr = R.O.quantize(R.O.bf16_to_f64(R.O.f64_to_bf16(grad.numpy())), mode)
    got = R.O.dequantize(out["q_row"].cpu().numpy(), R.plain_scales(out["s_row"]))
    return R.O.dequantize(qr, sr) != got


def _gradient(x, t, f, dlogp, dent, scale):
    x64, tc = x.cpu().to(F64), t.cpu()
    m, ls = f["stats"].cpu().to(F64).unbind(1)
    return R.logprob_bwd(x64, tc, m, ls, f["entropy"].cpu().to(F64), dlogp.to(F64), dent.to(F64), scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1.0, 0.8, 0.9])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_sure_targets(gpu, dtype, scale, entropy):
    """1 - p of a target that holds all but 3e-4 to 6e-6 of the probability does
    not lose its digits. The gradient at the target is off by some 8 roundings of
    float32, 2^-21 of itself; an E4M3 border lies within that for 2 * 2^-21 in
    2^-4 of the values, 2^-16, and as often for the borders that bf16 moves: of
    2048 rows 0.06 are expected to change a code, and 3 are allowed. (The target
    is the largest value of its block, and a moved scale moves the block's other
    codes only where they are rounded away.)"""
    T, V = 2048, 256
    scale = float(torch.tensor(scale))
    x, t = _sure_rows(T, V, dtype, scale, 8.1, 12.0, 5)
    f = lm.token_logprobs(x, t, scale=scale)
    g = torch.Generator().manual_seed(9)
    dlogp = (0.5 + torch.rand(T, generator=g)) / T
    dent = 0.05 * torch.rand(T, generator=g) / T if entropy else torch.zeros(T)
    out = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], dlogp.to(dev()), dent.to(dev()) if entropy else None,
                                scale=scale, layout="plain")
    other = torch.from_numpy(_other_codes(out, _gradient(x, t, f, dlogp, dent, scale), "rceil"))
    at = other[torch.arange(T), t.cpu()]
    print(f"{dtype} scale={scale} entropy={entropy}: {int(at.sum())} of {T} targets, {int(other.sum())} of all", flush=True)
    assert int(at.sum()) <= 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offset", [0.0, 40.0, -300.0])
def test_entropy_gradient_of_sure_rows(gpu, dtype, offset):
    """Rows that only the entropy reaches (target ignored) and whose best token
    holds all but 3e-4 to 6e-6 of the probability: l + H there is a few times
    1e-4, far below the logits it is formed from. It is off by some 4 roundings
    of itself and p by 2^-20: 2^-15 of the values change a code, of 2048 rows
    0.1; 3 are allowed."""
    T, V = 2048, 256
    x, t = _sure_rows(T, V, F32, 1.0, 8.1, 12.0, 6)
    x = (x + offset).to(dtype)
    best = x.amax(-1, keepdim=True)
    x = torch.where(x == best, best, torch.minimum(x, best - 6))     # one best token, whatever the type rounds
    f = lm.token_logprobs(x, torch.full_like(t, -100))
    dent = (0.5 + torch.rand(T, generator=torch.Generator().manual_seed(3))) / T
    out = lm.token_logprobs_bwd(x, torch.full_like(t, -100), f["stats"], f["entropy"], None, dent.to(dev()), layout="plain")
    grad = _gradient(x, torch.full_like(t, -100), f, torch.zeros(T), dent, 1.0)
    other = torch.from_numpy(_other_codes(out, grad, "rceil"))
    at = other[torch.arange(T), x.argmax(-1).cpu()]
    print(f"{dtype} offset={offset}: {int(at.sum())} of {T} best tokens, {int(other.sum())} of all", flush=True)
    assert int(at.sum()) <= 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["dlogp", "dent", "both"])
def test_gradients_of_any_size(gpu, dtype, which):
    """Incoming gradients from 1e-28 to 1e30 (in turn by row) keep their digits,
    masked tokens stay exactly 0, and rows next to each other do not meet."""
    T, V = 130, 1000
    g = torch.Generator().manual_seed(11)
    x = torch.randn((T, V), generator=g) * 2.5
    t = torch.randint(0, V, (T,), generator=g)
    x[:, V // 3:V // 2] = -INF
    x[torch.arange(T), t] = 3.0
    x, t = x.to(dtype).to(dev()), t.to(dev())
    f = lm.token_logprobs(x, t)
    size = 10.0 ** (-28 + 58 * (torch.randperm(T, generator=g).to(F64) / (T - 1)))
    dlogp, dent = ((size * (1 + torch.rand(T, generator=g))).float() for _ in range(2))
    if which == "dlogp":
        dent = torch.zeros(T)
    if which == "dent":
        dlogp = torch.zeros(T)
    out = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], dlogp.to(dev()), dent.to(dev()), layout="plain")
    x64, tc = x.cpu().to(F64), t.cpu()
    m, ls = f["stats"].cpu().to(F64).unbind(1)
    ent = f["entropy"].cpu().to(F64)
    grad = _gradient(x, t, f, dlogp, dent, 1.0)
    lp = torch.where(x64 == -INF, 0.0, x64 - m[:, None] - ls[:, None])
    p = torch.where(x64 == -INF, 0.0, lp.exp())
    mag = p * (dlogp.abs()[:, None] + dent.abs()[:, None] * (lp.abs() + ent.abs()[:, None]))
    mag[torch.arange(T), tc] += dlogp.abs()
    Vp = lm.padded_rows(V, "plain")
    pad = lambda v: torch.cat([v, v.new_zeros(T, Vp - V)], 1)
    R.check_codes(out["q_row"], out["s_row"], pad(grad), "rceil", which, pad(mag))
    gone = torch.nn.functional.pad(x == -INF, (0, Vp - V), value=True)
    gone[torch.arange(T), t] = False
    assert not (out["q_row"] & 0x7F)[gone].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", [(300, 30001), (300, 131072), (100, 131072)])
@pytest.mark.parametrize("lo,hi", [(7.0, 9.0), (2.0, 4.0)])
def test_scoring_of_sure_rows(gpu, T, V, dtype, lo, hi):
    """Rows whose target holds all but e^-lo .. e^-hi of the probability. S, between
    1 and 2, passes at most 32 roundings within a tile, 32 over a thread's tiles and 10
    where threads are joined, each at most 2^-24 and of either sign: sqrt(74) 2^-24 =
    5e-7 root mean square, and as much in ls. A holds the best token's term times at
    most 8.5: roundings up to 2^-21, 4.1e-6 in A / S, 2.9e-6 in the entropy times ln 2,
    next to those of ls."""
    x, t = _sure_rows(T, V, dtype, 1.0, lo, hi, V)
    out = lm.token_logprobs(x, t)
    x64 = x.cpu().to(F64)
    _, ls, logp, ent = R.logprob_fwd(x64, t.cpu(), 1.0)
    rms = {k: float((got.cpu().to(F64) - want).square().mean().sqrt())
           for k, got, want in (("ls", out["stats"][:, 1], ls), ("logp", out["logp"], logp), ("entropy", out["entropy"], ent))}
    print(f"T={T} V={V} {dtype} {lo}: {rms}", flush=True)
    assert rms["ls"] <= 5.2e-7 and rms["logp"] <= 5.2e-7 and rms["entropy"] <= 3.0e-6
