"""Dispatch, the gathered quantization and combine on the GPU: maps exactly,
gathered codes bit for bit, sums to the roundings that they have."""

import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import b128, moe, mx, synth

pytestmark = pytest.mark.gpu
F64, BF, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32


def _same(got, ref, what=""):
    for k, v in ref.items():
        g = got[k].cpu()
        v = v.cpu()
        if v.dtype is F32:
            assert torch.equal(torch.isnan(g), torch.isnan(v)), f"{what} {k}"
            g, v = torch.nan_to_num(g), torch.nan_to_num(v)
        assert g.shape == v.shape and torch.equal(g, v), f"{what} {k}: {int((g != v).sum())} of {v.numel()} differ"


def _choice(T, top, E, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.exp(skew * torch.randn(E, generator=g))
    return torch.multinomial(p.expand(max(T, 1), E), min(top, E), generator=g)[:T].to(I32)


# one workgroup (up to 4096 slots) and several chunks, one expert, experts without tokens, one token, none
PLANS = [(0, 2, 8, 128), (1, 1, 1, 128), (1, 8, 256, 1), (13, 8, 256, 1), (100, 2, 8, 16), (1000, 8, 40, 128),
         (1024, 8, 256, 1), (1025, 8, 256, 128), (1500, 6, 1000, 4), (5000, 2, 1024, 1), (20000, 8, 64, 128),
         (33333, 1, 3, 128), (70000, 4, 17, 7), (262144, 1, 130, 128)]


@pytest.mark.parametrize("T,top,E,multiple", PLANS)
def test_dispatch(gpu, T, top, E, multiple):
    print(f"T={T} top={top} E={E} multiple={multiple}", flush=True)
    idx = _choice(T, top, E, T + E, skew=1.5)
    cap = moe.capacity(idx.numel(), E, multiple)
    _same(moe.dispatch(idx.to(dev()), E, multiple), R.dispatch(idx, E, multiple, cap))


@pytest.mark.parametrize("T", [50, 4000])
def test_dispatch_odd_choices(gpu, T):
    """Slots without an expert, experts outside, one expert for everything, a capacity beyond the least."""
    E = 12
    idx = _choice(T, 4, E, 1)
    idx[::3, 1] = -1
    idx[1::5, 2] = E
    idx[2::7, 3] = 2 ** 31 - 1
    idx[5] = -2 ** 31
    cap = moe.capacity(T * 4, E) + 333
    got = moe.dispatch(idx.to(dev()), E, cap=cap)
    _same(got, R.dispatch(idx, E, 128, cap))
    none = torch.full_like(idx, -1)
    _same(moe.dispatch(none.to(dev()), E, cap=cap), R.dispatch(none, E, 128, cap))
    one = torch.full_like(idx, 7)
    _same(moe.dispatch(one.to(dev()), E, 1), R.dispatch(one, E, 1, T * 4))


def test_dispatch_is_stable_over_runs_and_buffers(gpu):
    idx = _choice(9000, 4, 300, 3).to(dev())
    first = moe.dispatch(idx, 300)
    out = {k: torch.full_like(v, 77) for k, v in first.items()}
    again = moe.dispatch(idx, 300, out=out)
    for k in first:
        assert again[k] is out[k] and torch.equal(first[k], again[k]), k


# ---------------------------------------------------------------- gather + quantize

GATHERS = [(5, 2, 4, 1, 128), (1, 8, 64, 1, 512), (33, 4, 8, 128, 640), (130, 6, 16, 128, 256), (200, 1, 3, 128, 1152)]


def _rows(T, C, pad, seed):
    g = synth.generator(seed)
    x = synth.normal_bf16((T, C + pad), 1.0, g)[:, :C]
    return x, g


@pytest.mark.parametrize("T,top,E,multiple,C", GATHERS)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("fmt,mode,layout", [("mxfp8", "rceil", "k128"), ("mxfp8", "floor", "plain"), ("b128", "f32", "k128"),
                                             ("b128", "rceil", "k128")])
def test_gather_quantize(gpu, T, top, E, multiple, C, weighted, fmt, mode, layout):
    print(f"T={T} top={top} E={E} multiple={multiple} C={C} {fmt} {mode} {layout} weighted={weighted}", flush=True)
    x, g = _rows(T, C, 8 * (T % 3), T + C)
    idx = _choice(T, top, E, T)
    if T > 4:
        idx[3, 0] = -1
    plan = R.dispatch(idx, E, multiple, moe.capacity(idx.numel(), E, multiple))
    w = torch.rand((T, idx.shape[1]), generator=g) * 2 if weighted else None
    rows = R.gather(x, plan["src"], idx.shape[1], w)
    xd = torch.empty((T, C + 8 * (T % 3)), dtype=BF, device=dev())[:, :C]
    xd.copy_(x)
    for col in (False, True):
        got = moe.gather_quantize(xd, plan["src"].to(dev()), idx.shape[1], None if w is None else w.to(dev()), fmt=fmt, mode=mode,
                                  layout=layout, colwise=col)
        if fmt == "b128":
            ref = R.quant_dual(rows, mode, col)
        else:
            ref = mx.quantize(rows.to(dev()), mode, True, False, layout)
            if col:
                n = (len(rows) + 127) // 128 * 128 if layout == "k128" else (len(rows) + 31) // 32 * 32
                full = torch.zeros((n, C), dtype=BF)
                full[:len(rows)] = rows
                ref.update(mx.quantize(full.to(dev()), mode, False, True, layout))
        assert set(got) == set(ref)
        _same(got, ref, f"col={col}")


def test_weighted_rows_are_rounded_once(gpu):
    """Weights whose float32 product lies on a bf16 border that the exact product does not."""
    g = torch.Generator().manual_seed(11)
    x = synth.normal_bf16((64, 128), 1.0, synth.generator(12))
    x[:, 0] = 448.0                                # a block maximum that keeps the other codes fine
    w = torch.rand(64, generator=g) + 0.5
    # for each row, a weight that takes its column 1 next to the middle of two bf16 values
    v = x[:, 1].to(F64)
    near = R.round_bf16(v * w).to(F64)
    mid = near + torch.sign(near) * torch.ldexp(torch.ones_like(near), torch.frexp(near)[1] - 9)     # half a bf16 step
    w = (mid / v).float()
    src = torch.arange(64, dtype=I32)
    rows = R.gather(x, src, 1, w)
    assert int(((x.float() * w[:, None]).to(BF) != rows).sum()) > 0     # two roundings differ somewhere
    got = moe.gather_quantize(x.to(dev()), src.to(dev()), 1, w.to(dev()), fmt="b128", mode="f32", colwise=True)
    _same(got, R.quant_dual(rows, "f32"))


@pytest.mark.parametrize("fmt,mode", [("mxfp8", "rceil"), ("b128", "f32")])
def test_gather_leaves_nan_in_its_rows(gpu, fmt, mode):
    """NaN and infinity reach their own blocks, padding rows are zeros, maps that point past x give zeros."""
    x, _ = _rows(9, 256, 0, 3)
    x[2, 5], x[4, 200] = float("nan"), float("inf")
    src = torch.tensor([0, -1, 2, 3, 4, 12, 8, 7, -5], dtype=I32)
    rows = R.gather(x, torch.where(src > 8, torch.full_like(src, -1), src), 1)
    got = moe.gather_quantize(x.to(dev()), src.to(dev()), 1, fmt=fmt, mode=mode, colwise=True)
    full = torch.zeros((128, 256), dtype=BF)
    full[:9] = rows
    if fmt == "b128":
        ref = R.quant_dual(rows, mode)
    else:
        ref = mx.quantize(rows.to(dev()), mode)
        ref.update(mx.quantize(full.to(dev()), mode, False, True))
    _same(got, ref)


# ---------------------------------------------------------------- combine

COMBINES = [(1, 1, 8, 4), (5, 2, 64, 40), (13, 8, 7168, 120), (33, 3, 520, 100), (70, 9, 1000, 640), (3, 20, 5120, 70),
            (256, 8, 2048, 2100), (50, 4, 5128, 90), (9, 1, 2056, 30), (21, 3, 6152, 64)]


@pytest.mark.parametrize("T,top,C,rows", COMBINES)
def test_combine(gpu, T, top, C, rows):
    print(f"T={T} top={top} C={C} rows={rows}", flush=True)
    pad = 8 * (T % 2)
    y, g = _rows(rows, C, pad, T + C)
    r, _ = _rows(T, C, pad, T + C + 1)
    pos = torch.randint(0, rows, (T, top), generator=g).to(I32)      # rows used twice and not at all
    pos[T // 2, 0] = -1
    pos[0, top - 1] = rows + 3
    w = torch.randn((T, top), generator=g)
    ok = (pos >= 0) & (pos < rows)
    yd, rd = (torch.empty((len(t), C + pad), dtype=BF, device=dev())[:, :C].copy_(t) for t in (y, r))
    terms = torch.where(ok[..., None], y.to(F64)[pos.clamp(0, rows - 1).long()], torch.zeros((), dtype=F64))
    for weights, res in ((w, r), (w, None), (None, r), (None, None)):
        t = terms * (weights.to(F64)[..., None] if weights is not None else 1)
        ref = t.sum(1) + (0 if res is None else res.to(F64))
        mag = t.abs().sum(1) + (0 if res is None else res.to(F64).abs())
        got = moe.combine(yd, pos.to(dev()), None if weights is None else weights.to(dev()), None if res is None else rd)
        off = (got.cpu().to(F64) - ref).abs()
        tol = (top + 1) * 2.0 ** -24 * mag + 2.0 ** -8 * ref.abs()
        assert torch.all(off <= tol * (1 + 2.0 ** -6)), float((off / tol.clamp(min=1e-300)).max())
    dout, _ = _rows(T, C, pad, 5)
    dd = torch.empty((T, C + pad), dtype=BF, device=dev())[:, :C].copy_(dout)
    t = terms * dout.to(F64)[:, None]
    got = moe.combine_bwd(dd, yd, pos.to(dev())).cpu()
    assert torch.all(got[~ok] == 0)
    # a thread's chain of 8 products per 2048 columns, then 8 joins
    tol = (8 * (C // 2048 + 1) + 8) * 2.0 ** -24 * t.abs().sum(-1)
    assert torch.all((got.to(F64) - t.sum(-1)).abs() <= tol)


def test_masked_rows_do_not_reach_the_sum(gpu):
    """NaN in rows that no slot points to stays there; a token without rows gets its residual or zeros."""
    y = torch.full((6, 64), float("nan"), dtype=BF)
    y[2] = 1.0
    pos = torch.tensor([[2, -1], [-1, -1], [2, 2]], dtype=I32)
    w = torch.tensor([[0.5, float("nan")], [1.0, 1.0], [0.25, 0.5]])
    out = moe.combine(y.to(dev()), pos.to(dev()), w.to(dev())).cpu()
    assert out[:, 0].tolist() == [0.5, 0.0, 0.75]
    d = moe.combine_bwd(torch.ones((3, 64), dtype=BF, device=dev()), y.to(dev()), pos.to(dev())).cpu()
    assert d.tolist() == [[64.0, 0.0], [0.0, 0.0], [64.0, 64.0]]


def test_empty_calls(gpu):
    y = torch.empty((0, 64), dtype=BF, device=dev())
    pos = torch.zeros((3, 2), dtype=I32, device=dev())
    assert torch.all(moe.combine(y, pos) == 0) and moe.combine(y, pos[:0]).shape == (0, 64)
    assert torch.all(moe.combine_bwd(torch.ones((3, 64), dtype=BF, device=dev()), y, pos) == 0)
    x = torch.empty((0, 128), dtype=BF, device=dev())
    got = moe.gather_quantize(x, torch.full((5,), -1, dtype=I32, device=dev()), 2, fmt="b128", mode="f32", colwise=True)
    assert torch.all(got["q_row"] == 0) and torch.all(got["q_col"] == 0)
    got = moe.gather_quantize(x, torch.empty((0,), dtype=I32, device=dev()), 2)
    assert got["q_row"].shape == (0, 128)
    assert b128.quantize(x, colwise=True)["s_col"].shape == (0, 128)
