"""Quantizers whose codes go past the caches (results of more than 100 Mi codes) against
the variant that keeps them there: the same call on a part of the rows, small enough for
the other variant, which the other tests compare with the definition; the last rows are
compared with the definition here too."""

import pytest
import torch

import moe_ref as R
from _helpers import dev
from quantize_grouped_gemm_amd import b128, moe

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
STREAM = 100 << 20


def _same(got, ref, what=""):
    assert got.shape == ref.shape and torch.equal(got, ref), f"{what}: {int((got != ref).sum())} of {ref.numel()} differ"


def _x(T, C, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randn((T, C), generator=g, device=dev()).to(BF)


@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("fmt,mode,layout", [("mxfp8", "rceil", "k128"), ("mxfp8", "floor", "plain"), ("b128", "f32", "k128"),
                                             ("b128", "rceil", "k128")])
def test_gather(gpu, fmt, mode, layout, weighted, col):
    T, C, top, part = 7000, 7168, 4, 1280
    x = _x(T, C, 1)
    g = torch.Generator(device=dev()).manual_seed(2)
    idx = torch.randint(0, 9, (T, top), generator=g, device=dev(), dtype=I32)
    src = moe.dispatch(idx, 9, cap=T * top + 1287)["src"]         # ends in rows without a slot, and inside a tile
    w = torch.rand((T, top), generator=g, device=dev()) + 0.1 if weighted else None
    rows = src.numel()
    assert rows * C > STREAM > part * C
    kw = dict(fmt=fmt, mode=mode, layout=layout, colwise=col)
    got = moe.gather_quantize(x, src, top, w, **kw)
    mid, last = (rows // 2) // 128 * 128, (rows - part) // 128 * 128
    for lo, hi in ((0, part), (mid, mid + part), (last, rows)):
        ref = moe.gather_quantize(x, src[lo:hi].clone(), top, w, **kw)
        k128 = layout == "k128"
        _same(got["q_row"][lo:hi], ref["q_row"], "q_row")
        _same(got["s_row"][:, lo:hi] if k128 else got["s_row"][lo:hi], ref["s_row"], "s_row")
        if col:
            n = ref["q_col"].shape[1]
            _same(got["q_col"][:, lo:lo + n], ref["q_col"], "q_col")
            step = 128 if k128 else 32
            _same(got["s_col"][lo // step:(lo + n) // step] if k128 else got["s_col"][:, lo // step:(lo + n) // step],
                  ref["s_col"], "s_col")
    if fmt == "b128":
        tail = slice(rows - 1408, rows - 1280)
        plain = R.gather(x.cpu(), src[tail].cpu(), top, None if w is None else w.cpu())
        q, s = R.quant_rows(plain, mode)
        _same(got["q_row"][tail].cpu(), q, "q_row by definition")
        _same(got["s_row"][:, tail].cpu(), s, "s_row by definition")


@pytest.mark.parametrize("mode", ["f32", "rceil"])
@pytest.mark.parametrize("row,col", [(True, False), (False, True), (True, True)])
def test_quantize(gpu, mode, row, col):
    T, C, part = 15001, 7168, 1177
    x = _x(T, C, 3)
    assert T * C > STREAM > part * C
    got = b128.quantize(x, mode, row, col)
    lo = T - part
    assert lo % 128 == 0
    ref = b128.quantize(x[lo:].clone(), mode, row, col)
    if row:
        _same(got["q_row"][lo:], ref["q_row"], "q_row")
        _same(got["s_row"][:, lo:], ref["s_row"], "s_row")
        q, s = R.quant_rows(x[-70:].cpu(), mode)
        _same(got["q_row"][-70:].cpu(), q, "q_row by definition")
        _same(got["s_row"][:, -70:].cpu(), s, "s_row by definition")
    if col:
        _same(got["q_col"][:, lo:], ref["q_col"], "q_col")
        _same(got["s_col"][lo // 128:], ref["s_col"], "s_col")


@pytest.mark.parametrize("mode", ["f32", "rceil"])
def test_quantize_weight(gpu, mode):
    w = torch.stack([_x(4080, 7184, 5 + e) * 0.02 for e in range(4)])
    assert w.numel() > STREAM > w[0].numel()
    got = b128.quantize_weight(w, mode)
    for e in (0, 3):
        ref = b128.quantize_weight(w[e].clone(), mode)
        for k, v in ref.items():
            _same(got[k][e], v, k)
    q, s = R.quant_weight(w[3, 3968:].cpu(), mode)
    _same(got["q"][3, 3968:].cpu(), q, "q by definition")
    _same(got["s"][3, :, 31:].cpu(), s, "s by definition")
