"""The variants of the layer-boundary operators that large calls take: groups of
several rows in the norm's backward, tiles and rows in plain order, logits and
codes that go past the caches. Where rows do not depend on each other, results are
compared bit for bit with calls over slices of rows, which stay below those limits
(the other test files check them against the 64-bit formulas)."""

import pytest
import torch

import lm_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import lm, synth
from test_gpu_lm_norm import _eq, _mx_cols, _mx_rows, _rows

pytestmark = pytest.mark.gpu
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32

# T, C, layout; rows of a group in the backward. Below and above 8M elements, one
# and two chunks a thread, one and several rows at a time in a workgroup, last
# groups that are not full
NORM = [(1001, 7168, "k128"), (9001, 1024, "k128"), (601, 16384, "k128"), (2101, 4128, "plain"), (8203, 480, "plain")]


@pytest.mark.parametrize("T,C,layout", NORM)
def test_norm_fwd(gpu, T, C, layout):
    print(f"T={T} C={C} {layout}", flush=True)
    g = synth.generator(T + C)
    x, _ = _rows(T, C, 1.0, g, pad=8)
    r, _ = _rows(T, C, 0.5, g)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(dev())
    out = lm.add_rmsnorm_quant(x, w, r, layout=layout, colwise=True, checkpoint=True)
    for i in range(0, T, 256):
        rows = slice(i, min(i + 256, T))
        part = lm.add_rmsnorm_quant(x[rows], w, r[rows], layout=layout, checkpoint=True)
        for k in ("sum", "rstd", "q_row", "q_ck"):
            _eq(out[k][rows], part[k], (k, i))
        for k in ("s_row", "s_ck"):
            _eq(out[k][:, rows] if layout == "k128" else out[k][rows], part[k], (k, i))
    # y as the kernel forms it (see test_norm_fwd of the smaller shapes)
    s, rstd = out["sum"].float(), out["rstd"][:, None]
    h = (rstd.view(torch.int32) & -65536).view(F32)
    y = ((s * h).to(F64) * w.to(F64) + ((s * (rstd - h)) * w).to(F64)).float().to(BF)
    ref = _mx_cols(y, "rceil", layout)
    _eq(out["q_col"], ref["q_col"], "q_col")
    _eq(out["s_col"], ref["s_col"], "s_col")


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("T,C,layout", NORM)
def test_norm_bwd(gpu, T, C, layout, ckpt):
    print(f"T={T} C={C} {layout} ckpt={ckpt}", flush=True)
    g = synth.generator(T * 3 + C)
    x, _ = _rows(T, C, 1.0, g, pad=8)
    dy, dy64 = _rows(T, C, 1e-2, g)
    ds, _ = _rows(T, C, 1e-2, g, pad=16)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(dev())
    f = lm.add_rmsnorm_quant(x, w, layout=layout, checkpoint=True)

    def call(rows, whole):
        src = dict(x=x[rows])
        if ckpt:
            s = f["s_ck"][:, rows] if layout == "k128" else f["s_ck"][rows]
            src = dict(checkpoint=(f["q_ck"][rows], s.contiguous()))
        return lm.add_rmsnorm_bwd(dy[rows], w, f["rstd"][rows], dsum=ds[rows], layout=layout, colwise=whole, **src)

    out, again = call(slice(0, T), True), call(slice(0, T), True)
    for k in out:
        _eq(out[k], again[k], k)
    for i in range(0, T, 128):       # one row a group
        rows = slice(i, min(i + 128, T))
        _eq(out["dx"][rows], call(rows, False)["dx"], ("dx", i))
    ref = _mx_rows(out["dx"], "rceil", layout)
    _eq(out["q_row"], ref["q_row"], "q_row")
    _eq(out["s_row"], ref["s_row"], "s_row")
    ref = _mx_cols(out["dx"], "rceil", layout)
    _eq(out["q_col"], ref["q_col"], "q_col")
    _eq(out["s_col"], ref["s_col"], "s_col")
    # dw: up to 16 rows in turn, then a thread's parts (at most 4096 / 256 in each of 4 sums), 2 joins of
    # those and 64 threads in turn: at most 98 roundings of the sum of magnitudes
    s64 = x.cpu().to(F64)
    if ckpt:
        s64 = torch.from_numpy(R.O.dequantize(f["q_ck"].cpu().numpy(), R.plain_scales(f["s_ck"])))
    t = dy64 * (s64 * f["rstd"].cpu().to(F64)[:, None])
    assert torch.all((out["dw"].cpu().to(F64) - t.sum(0)).abs() <= 100 * 2.0 ** -24 * t.abs().sum(0))


# above 2^28 codes: aligned rows, the same in bands of tiles, rows that start at odd elements
GRAD = [(2200, 131072, BF), (2200, 131072, F32), (4224, 65536, BF), (2700, 100001, BF), (2700, 100001, F32)]


@pytest.mark.parametrize("T,V,dtype", GRAD)
def test_loss_gradient(gpu, T, V, dtype):
    print(f"T={T} V={V} {dtype}", flush=True)
    g = torch.Generator(device=dev()).manual_seed(V)
    x = (torch.randn((T, V), generator=g, device=dev()) * 2.5).to(dtype)
    t = torch.randint(0, V, (T,), generator=g, device=dev())
    f = lm.token_logprobs(x, t)
    dl, de = torch.randn(T, generator=g, device=dev()) / T, torch.randn(T, generator=g, device=dev()) / T
    out = lm.token_logprobs_bwd(x, t, f["stats"], f["entropy"], dl, de)
    for r0 in range(0, T, 1024):
        r = slice(r0, min(r0 + 1024, T))
        part = lm.token_logprobs_bwd(x[r], t[r], f["stats"][r], f["entropy"][r], dl[r], de[r])
        n = part["q_col"].shape[1]
        assert torch.equal(out["q_row"][r], part["q_row"]) and torch.equal(out["s_row"][:, r], part["s_row"])
        assert torch.equal(out["q_col"][:, r0:r0 + n], part["q_col"])
        assert torch.equal(out["s_col"][r0 // 128:(r0 + n) // 128], part["s_col"])


@pytest.mark.parametrize("T,V,dtype", [(1100, 131072, BF), (600, 131072, F32), (2700, 50001, BF), (1400, 50001, F32)])
@pytest.mark.parametrize("top", [0, 20])
def test_scoring(gpu, T, V, dtype, top):
    """More than 256 MB of logits."""
    print(f"T={T} V={V} {dtype} top={top}", flush=True)
    g = torch.Generator(device=dev()).manual_seed(V + T)
    x = (torch.randn((T, V), generator=g, device=dev()) * 2.5).to(dtype)
    t = torch.randint(0, V, (T,), generator=g, device=dev())
    t[::7] = -100
    out = lm.token_logprobs(x, t, scale=0.9, top=top)
    n = (T + 1) // 2                 # above 256 rows: the same workgroups
    for r in (slice(0, n), slice(n, T)):
        part = lm.token_logprobs(x[r], t[r], scale=0.9, top=top)
        for k in out:
            assert torch.equal(out[k][r], part[k]), k


def _normal(shape, std, g):
    return torch.empty(shape, dtype=BF, device=dev()).normal_(0, std, generator=g)


@pytest.mark.parametrize("T,C", [(140032, 16384)])
def test_norm_past_32_bits(gpu, T, C):
    """More than 2^31 elements: the last rows equal a call of their own."""
    g = torch.Generator(device=dev()).manual_seed(1)
    x, w = _normal((T, C), 1.0, g), torch.ones(C, device=dev())
    out = lm.add_rmsnorm_quant(x, w, colwise=True, checkpoint=True)
    bwd = lm.add_rmsnorm_bwd(x, w, out["rstd"], checkpoint=(out["q_ck"], out["s_ck"]), colwise=True)
    r0 = T - 640
    part = lm.add_rmsnorm_quant(x[r0:], w, colwise=True, checkpoint=True)
    pb = lm.add_rmsnorm_bwd(x[r0:], w, part["rstd"], checkpoint=(part["q_ck"], part["s_ck"]), colwise=True)
    for whole, piece, rows, codes in ((out, part, ("rstd",), ("q_row", "q_ck")), (bwd, pb, ("dx",), ("q_row",))):
        for k in rows + codes:
            _eq(whole[k][r0:], piece[k], k)
        for k in codes:
            s = k.replace("q_", "s_")
            _eq(whole[s][:, r0:], piece[s], s)
        _eq(whole["q_col"][:, r0:], piece["q_col"], "q_col")
        _eq(whole["s_col"][r0 // 128:], piece["s_col"], "s_col")


@pytest.mark.parametrize("T,H", [(70016, 16384)])
def test_swiglu_past_32_bits(gpu, T, H):
    g = torch.Generator(device=dev()).manual_seed(2)
    z, dh = _normal((T, 2 * H), 1.5, g), _normal((T, H), 1e-2, g)
    out = lm.swiglu_ckpt_fwd(z[:, :H], z[:, H:])
    bwd = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"])
    r0 = T - 640
    part = lm.swiglu_ckpt_fwd(z[r0:, :H], z[r0:, H:])
    pb = lm.swiglu_ckpt_bwd(dh[r0:], part["q_ck"], part["s_ck"])
    for whole, piece, codes in ((out, part, ("q_row", "q_ck")), (bwd, pb, ("q_row",))):
        for k in codes:
            s = k.replace("q_", "s_")
            _eq(whole[k][r0:], piece[k], k)
            _eq(whole[s][:, r0:], piece[s], s)
        _eq(whole["q_col"][:, r0:], piece["q_col"], "q_col")
        _eq(whole["s_col"][r0 // 128:], piece["s_col"], "s_col")


@pytest.mark.parametrize("T,V,pad", [(17024, 131072, 0), (17024, 130001, 4)])
def test_logits_past_32_bits(gpu, T, V, pad):
    """Aligned rows, and rows of an odd vocabulary further apart."""
    g = torch.Generator(device=dev()).manual_seed(3)
    x = _normal((T, V + pad), 2.5, g)[:, :V]
    t = torch.randint(0, V, (T,), generator=g, device=dev())
    dl = torch.randn(T, generator=g, device=dev()) / T
    out = lm.token_logprobs(x, t, top=5)
    bwd = lm.token_logprobs_bwd(x, t, out["stats"], out["entropy"], dl, dl)
    r0 = T - 640
    part = lm.token_logprobs(x[r0:], t[r0:], top=5)
    pb = lm.token_logprobs_bwd(x[r0:], t[r0:], part["stats"], part["entropy"], dl[r0:], dl[r0:])
    for k in out:
        _eq(out[k][r0:], part[k], k)
    _eq(bwd["q_row"][r0:], pb["q_row"], "q_row")
    _eq(bwd["s_row"][:, r0:], pb["s_row"], "s_row")
    _eq(bwd["q_col"][:, r0:], pb["q_col"], "q_col")
    _eq(bwd["s_col"][r0 // 128:], pb["s_col"], "s_col")


@pytest.mark.parametrize("T,H,layout", [(8300, 8320, "k128"), (9001, 7712, "plain")])
def test_swiglu_tile_orders(gpu, T, H, layout):
    """More than 4096 tiles of long rows: the backward walks them in another order."""
    g = torch.Generator(device=dev()).manual_seed(4)
    z, dh = _normal((T, 2 * H), 1.5, g), _normal((T, H), 1e-2, g)
    out = lm.swiglu_ckpt_fwd(z[:, :H], z[:, H:], layout=layout)
    bwd = lm.swiglu_ckpt_bwd(dh, out["q_ck"], out["s_ck"], layout=layout)
    for r0 in range(0, T, 4096):
        r1 = min(r0 + 4096, T)
        part = lm.swiglu_ckpt_fwd(z[r0:r1, :H], z[r0:r1, H:], layout=layout)
        pb = lm.swiglu_ckpt_bwd(dh[r0:r1], part["q_ck"], part["s_ck"], layout=layout)
        cols = slice(r0, r0 + lm.padded_rows(r1 - r0, layout))
        for whole, piece, codes in ((out, part, ("q_row", "q_ck")), (bwd, pb, ("q_row",))):
            for k in codes:
                s = k.replace("q_", "s_")
                _eq(whole[k][r0:r1], piece[k], (k, r0))
                _eq(whole[s][:, r0:r1] if layout == "k128" else whole[s][r0:r1], piece[s], (s, r0))
            _eq(whole["q_col"][:, cols], piece["q_col"], ("q_col", r0))
            step = 128 if layout == "k128" else 32
            blocks = slice(cols.start // step, cols.stop // step)
            _eq(whole["s_col"][blocks] if layout == "k128" else whole["s_col"][:, blocks], piece["s_col"], ("s_col", r0))
