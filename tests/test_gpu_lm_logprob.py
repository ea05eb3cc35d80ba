"""Token log probabilities and their gradient on the GPU, against the float64
formulas.

The row sums S = sum e_j and A = sum e_j d_j are float32 sums of V terms, at
most V / 256 + 8 of them one after the other; e_j itself is off by the
exponential's ulp and half an ulp of its argument (below 40 where it counts):
ERR(V) = (V / 256 + 64) 2^-24 bounds the relative error of S and of A's terms.
ls = ln S is then off by ERR + 2^-23 |ls|, logp by that plus 2^-23 of its own
terms, and the entropy by ERR (1 + 2 E|d|)."""

import pytest
import torch

import lm_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import lm, mx

pytestmark = pytest.mark.gpu
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32

# T, V, top, dtype
FWD = [(0, 100, 5, BF), (1, 1, 1, F32), (1, 7, 7, BF), (3, 64, 64, BF), (5, 1000, 20, F32), (33, 2049, 5, BF),
       (2, 50001, 64, F32), (7, 50001, 20, BF), (1, 131072, 20, BF), (1, 131071, 64, BF), (130, 4097, 1, F32),
       (257, 1111, 0, BF), (600, 9000, 5, BF), (1500, 2500, 20, F32), (1100, 333, 64, BF), (4, 262147, 33, BF)]


def _logits(T, V, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, V + pad), generator=g) * 2.5).to(dtype)
    t = torch.randint(0, V, (T,), generator=g)
    if T > 2:
        t[2] = -100
    return x.to(dev())[:, :V], t.to(dev())


def _check_fwd(out, x, t, scale, top, what=""):
    x64, t = x.cpu().to(F64), t.cpu()
    T, V = x64.shape
    m, ls, logp, ent = R.logprob_fwd(x64, t, scale)
    err = (V / 256 + 64) * 2.0 ** -24
    fin = m > -torch.inf
    got = {k: v.cpu().to(F64) for k, v in out.items()}
    assert torch.equal(got["stats"][:, 0], m), what
    d_ls = err + 2.0 ** -23 * ls.abs()
    assert torch.all(((got["stats"][:, 1] - ls).abs() <= d_ls) | ~fin), what
    assert torch.equal(got["stats"][:, 1][~fin], ls[~fin]), what
    dif = (got["logp"] - logp).abs()
    assert torch.all((dif <= d_ls + 2.0 ** -22 * (logp.abs() + ls.abs())) | (got["logp"] == logp)), what
    md = torch.where(fin, (ls - ent).abs(), 0.0)    # E|d|
    assert torch.all((got["entropy"] - ent).abs() <= torch.where(fin, err * (1 + 2 * md) + 2.0 ** -22 * (ls.abs() + md), 0.0)), what
    if top:
        order = torch.sort(x64, dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(out["top_idx"].cpu().long(), order), what
        lt = (x64.gather(1, order) - torch.where(fin, m, 0.0)[:, None]) * scale - torch.where(fin, ls, 0.0)[:, None]
        gl = got["top_logp"]
        assert torch.all(((gl - lt).abs() <= d_ls[:, None] + 2.0 ** -22 * (lt.abs() + ls.abs()[:, None])) | (gl == lt)), what


@pytest.mark.parametrize("T,V,top,dtype", FWD)
def test_fwd(gpu, T, V, top, dtype):
    scale = [1.0, 0.7, 1.25][V % 3]
    x, t = _logits(T, V, dtype, T + V, pad=(T + V) % 4)
    print(f"T={T} V={V} top={top} {dtype} scale={scale}", flush=True)
    out = lm.token_logprobs(x, t, scale=scale, top=top)
    _check_fwd(out, x, t, scale, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [300, 9001, 131072])
def test_fwd_ties_and_masks(gpu, V, dtype):
    """Rows that test the order and the masks: all equal, zeros of both signs,
    descending, ascending, the best values next to each other, the best values
    in one thread's share, part masked, all but few masked (fewer left than
    alternatives), all masked, masked by the lowest finite value, all at the
    lowest finite value, huge values."""
    top = 20
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    base = torch.randn(V, generator=g)
    i = torch.arange(V)
    share = base.clone()
    share[(i // 8) % 256 == 3] += 50.0
    few = torch.full((V,), -torch.inf)
    few[torch.tensor([V - 1, 5, V // 2])] = torch.tensor([1.0, 2.0, 2.0])
    lowmask = torch.where(i % 3 == 0, base, torch.tensor(low))
    part = torch.where(i % 3 == 1, base, torch.tensor(-torch.inf))
    block = base.clone()
    block[100:140] += 30.0
    rows = [torch.zeros(V), torch.where(i % 2 == 0, -0.0, 0.0), -i.float() / V, i.float() / V, block, share, part, few,
            torch.full((V,), -torch.inf), lowmask, torch.full((V,), low), base * 1e34, base * 1e-30,
            torch.where(i == V - 1, 80.0, -80.0)]
    x = torch.stack(rows).to(dtype).to(dev())
    t = torch.full((len(rows),), 5).to(dev())
    print(f"V={V} {dtype}", flush=True)
    out = lm.token_logprobs(x, t, top=top)
    x64 = x.cpu().to(F64)
    huge = 11        # differences beyond float32's useful range: one token holds everything
    keep = [r for r in range(len(rows)) if r != huge]
    _check_fwd({k: v[keep] for k, v in out.items()}, x[keep], t[keep], 1.0, top)
    order = torch.sort(x64[huge], descending=True, stable=True).indices[:top]
    assert torch.equal(out["top_idx"][huge].cpu().long(), order)
    assert out["stats"][huge, 1].item() == 0 and out["entropy"][huge].item() == 0
    empty = 8
    assert out["entropy"][empty].item() == 0 and out["logp"][empty].item() == -torch.inf
    assert out["top_idx"][empty].tolist() == list(range(top))


def test_fwd_bad_values(gpu):
    """A NaN or +infinity makes its row NaN (indices stay in range) and leaves
    the others alone; a target outside the vocabulary is reported and not
    scored."""
    x, t = _logits(6, 5000, BF, 1)
    ref = lm.token_logprobs(x, t, top=5)
    y = x.clone()
    y[1, 4000] = float("nan")
    y[3, 17] = float("inf")
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out = lm.token_logprobs(y, t, top=5, dev_err=err)
    for r in (0, 2, 4, 5):
        for k in out:
            assert torch.equal(out[k][r], ref[k][r]), (r, k)
    for r in (1, 3):
        assert torch.isnan(out["logp"][r]) and torch.isnan(out["entropy"][r]) and torch.isnan(out["stats"][r, 1])
        assert ((out["top_idx"][r] >= 0) & (out["top_idx"][r] < 5000)).all()
    assert err.item() == 0
    t2 = t.clone()
    t2[4], t2[5] = 5000, -3
    out = lm.token_logprobs(x, t2, dev_err=err)
    assert err.item() == 8 and out["logp"][4].item() == 0 and out["logp"][5].item() == 0
    assert torch.equal(out["entropy"], ref["entropy"])
    q = lm.token_logprobs_bwd(y, t, out["stats"], out["entropy"], dlogp=torch.ones(6, device=dev()), layout="plain")
    ok = lm.token_logprobs_bwd(x, t, out["stats"], out["entropy"], dlogp=torch.ones(6, device=dev()), layout="plain")
    assert torch.equal(q["q_row"][0], ok["q_row"][0])


BWD = [(0, 100, BF, "plain"), (1, 1, F32, "plain"), (1, 1000, BF, "k128"), (33, 129, BF, "plain"),
       (130, 1025, F32, "k128"), (128, 4096, BF, "k128"), (257, 5001, BF, "k128"), (40, 20000, F32, "plain")]


@pytest.mark.parametrize("mode", ["rceil", "floor"])
@pytest.mark.parametrize("T,V,dtype,layout", BWD)
def test_bwd(gpu, T, V, dtype, layout, mode):
    scale = [1.0, 0.7, 1.25][V % 3]
    x, t = _logits(T, V, dtype, 3 * T + V, pad=(T + V) % 4)
    print(f"T={T} V={V} {dtype} {layout} {mode}", flush=True)
    if T > 5 and V > 4:
        x[4, V // 3:V // 2] = -torch.inf
        x[5] = -torch.inf
    f = lm.token_logprobs(x, t, scale=scale)
    g = torch.Generator().manual_seed(T)
    dlogp, dent = torch.randn(T, generator=g) / max(T, 1), 1e-2 * torch.randn(T, generator=g) / max(T, 1)
    out = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], dlogp.to(dev()), dent.to(dev()), scale=scale, mode=mode,
                                layout=layout)
    Vp = lm.padded_rows(V, layout)
    assert out["q_row"].shape == (T, Vp) and out["q_col"].shape == (Vp, lm.padded_rows(T, layout))
    x64, tc = x.cpu().to(F64), t.cpu()
    m, ls = f["stats"].cpu().to(F64).unbind(1)
    ent = f["entropy"].cpu().to(F64)
    grad = R.logprob_bwd(x64, tc, m, ls, ent, dlogp.to(F64), dent.to(F64), scale)
    empty = (m == -torch.inf)[:, None]
    lp = torch.where(empty | (x64 == -torch.inf), 0.0, (x64 - m[:, None]) * scale - ls[:, None])
    p = torch.where(empty | (x64 == -torch.inf), 0.0, torch.exp(lp))
    mag = scale * p * (dlogp.abs()[:, None] + dent.abs()[:, None] * (lp.abs() + ent.abs()[:, None]))
    hit = torch.zeros_like(x64)
    ok = tc != -100
    hit[ok, tc[ok]] = 1.0
    mag = mag + hit * scale * dlogp.abs()[:, None].to(F64)
    pad = lambda v: torch.cat([v, v.new_zeros(T, Vp - V)], 1)
    R.check_dual(out, pad(grad), mode, layout, "grad", mag=pad(mag))


@pytest.mark.parametrize("which", ["dlogp", "dent", "neither"])
def test_bwd_missing_gradients_are_zero(gpu, which):
    x, t = _logits(37, 777, BF, 8)
    f = lm.token_logprobs(x, t)
    z = torch.zeros(37, device=dev())
    g = torch.linspace(-1, 1, 37, device=dev())
    kw = {"dlogp": dict(dlogp=g), "dent": dict(dent=g), "neither": {}}[which]
    full = dict(dlogp=z, dent=z)
    full.update(kw)
    a = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], **kw)
    b = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], **full)
    da, db = (mx.dequantize(o["q_row"], o["s_row"]) for o in (a, b))
    assert torch.equal(da, db)


def test_strided_and_unaligned_rows(gpu):
    """A vocabulary slice starting at an odd column equals its copy."""
    x, t = _logits(19, 3001, BF, 10)
    v = x[:, 7:2500]
    t = t.clamp(max=2492)
    a, b = lm.token_logprobs(v, t, top=9), lm.token_logprobs(v.contiguous(), t, top=9)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    ga = lm.token_logprobs_bwd(v, t, a["stats"], a["entropy"], dlogp=torch.ones(19, device=dev()))
    gb = lm.token_logprobs_bwd(v.contiguous(), t, a["stats"], a["entropy"], dlogp=torch.ones(19, device=dev()))
    for k in ga:
        assert torch.equal(ga[k], gb[k]), k


def test_bwd_tile_orders_agree(gpu):
    """A large aligned gradient walks its tiles in another order: the same
    bytes as from calls over 2048 of its rows."""
    T, V = 4100, 49152
    g = torch.Generator(device=dev()).manual_seed(0)
    x = (torch.randn((T, V), generator=g, device=dev()) * 2.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device=dev())
    f = lm.token_logprobs(x, t)
    dl, de = torch.randn(T, generator=g, device=dev()) / T, torch.randn(T, generator=g, device=dev()) / T
    out = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], dl, de)
    for r0 in range(0, T, 2048):
        r = slice(r0, min(r0 + 2048, T))
        part = lm.token_logprobs_bwd(x[r], t[r], f["stats"][r], f["entropy"][r], dl[r], de[r])
        n = part["q_col"].shape[1]
        assert torch.equal(out["q_row"][r], part["q_row"]) and torch.equal(out["s_row"][:, r], part["s_row"])
        assert torch.equal(out["q_col"][:, r0:r0 + n], part["q_col"])
        assert torch.equal(out["s_col"][r0 // 128:(r0 + n) // 128], part["s_col"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1.0, 1e-3, 40.0])
def test_bwd_masks_and_magnitudes(gpu, dtype, scale):
    """Rows masked by the lowest finite value, all at it (uniform), with a large
    common offset, with one token far above the rest, and all masked, next to
    ordinary rows in the same tile."""
    V = 1001
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(4)
    base = torch.randn(V, generator=g)
    i = torch.arange(V)
    spike = base.clone()
    spike[17] = 300.0
    rows = [base, torch.where(i % 3 == 0, base, torch.tensor(low)), torch.full((V,), low), base + 1000.0, base - 5000.0,
            spike, torch.full((V,), -torch.inf), torch.where(i % 2 == 0, base, torch.tensor(-torch.inf)), base * 1e-20]
    x = torch.stack(rows).to(dtype)
    T = len(rows)
    t = torch.full((T,), 18)
    f = lm.token_logprobs(x.to(dev()), t.to(dev()), scale=scale)
    dl, de = torch.linspace(-1, 1, T) + 0.05, torch.linspace(0.5, -0.5, T) + 0.01
    out = lm.token_logprobs_bwd(x.to(dev()), t.to(dev()), f["stats"], f["entropy"], dl.to(dev()), de.to(dev()), scale=scale,
                                layout="plain")
    x64 = x.to(F64)
    m, ls = f["stats"].cpu().to(F64).unbind(1)
    ent = f["entropy"].cpu().to(F64)
    grad = R.logprob_bwd(x64, t, m, ls, ent, dl.to(F64), de.to(F64), scale)
    empty = (m == -torch.inf)[:, None]
    lp = torch.where(empty | (x64 == -torch.inf), 0.0, (x64 - m[:, None]) * scale - ls[:, None])
    p = torch.where(empty | (x64 == -torch.inf), 0.0, torch.exp(lp))
    # an entry's own size bounds what its float32 difference from m can lose
    size = torch.where(p > 0, 1 + scale * (x64.clamp(min=-1e30).abs() + torch.where(empty[:, 0], 0.0, m).abs()[:, None]) / 64,
                       1.0)
    size[2] = 1.0    # its differences are exact zeros
    mag = scale * p * size * (dl.abs()[:, None] + de.abs()[:, None] * (1 + lp.abs() + ent.abs()[:, None]))
    mag[:, 18] += scale * dl.abs()
    Vp = lm.padded_rows(V, "plain")
    pad = lambda v: torch.cat([v, v.new_zeros(T, Vp - V)], 1)
    R.check_dual(out, pad(grad), "rceil", "plain", "grad", mag=pad(mag))


@pytest.mark.parametrize("T,V,top,dtype", [(128, 70000, 9, BF), (129, 70000, 9, BF), (100, 65536, 5, F32), (9, 65537, 64, BF),
                                           (2, 200003, 64, F32), (257, 32768, 3, BF), (256, 32768, 3, BF)])
def test_fwd_around_the_launch_rules(gpu, T, V, top, dtype):
    """Both sides of the limits where rows are split and workgroups widened."""
    x, t = _logits(T, V, dtype, V - T)
    print(f"T={T} V={V} top={top} {dtype}", flush=True)
    _check_fwd(lm.token_logprobs(x, t, top=top), x, t, 1.0, top)


@pytest.mark.parametrize("T,V", [(16, 131072), (140, 70001)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fill", ["infinity", "lowest"])
def test_fwd_allowed_sets(gpu, T, V, dtype, fill):
    """Masks that leave 1 to 20000 tokens of a large vocabulary, scattered or next to
    each other, in whole rows and in rows split over workgroups: alternatives
    beyond them are the first masked tokens."""
    top = 20
    g = torch.Generator().manual_seed(T)
    low = -torch.inf if fill == "infinity" else torch.finfo(dtype).min
    counts = [1, 2, 19, 20, 21, 64, 300, 600, 1088, 1089, 5000, 20000]
    x = torch.full((T, V), low)
    t = torch.zeros(T, dtype=torch.int64)
    for r in range(T):
        n = counts[r % len(counts)]
        at = torch.randperm(V, generator=g)[:n] if r % 2 else V // 3 + torch.arange(n)
        x[r, at] = 2.5 * torch.randn(n, generator=g)
        t[r] = at[0]
    print(f"T={T} V={V} {dtype} {fill}", flush=True)
    x = x.to(dtype).to(dev())
    t = t.to(dev())
    _check_fwd(lm.token_logprobs(x, t, top=top), x, t, 1.0, top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_fwd_targets_of_split_rows(gpu, dtype):
    """Targets at the borders of a split row's segments, not scored ones, and
    ones outside the vocabulary."""
    V = 131072
    at = [0, 8191, 8192, V // 2 - 1, V // 2, V - 1, -100, 7]
    x, _ = _logits(len(at), V, dtype, 3)
    t = torch.tensor(at).to(dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    _check_fwd(lm.token_logprobs(x, t, top=3, dev_err=err), x, t, 1.0, 3)
    assert err.item() == 0
    t[7] = V
    out = lm.token_logprobs(x, t, dev_err=err)
    assert err.item() == 8 and out["logp"][7].item() == 0 and out["logp"][6].item() == 0
