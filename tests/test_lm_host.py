"""Layer-boundary operators without a GPU: the reference formulas' gradients
against central differences, the header against the binding, and every refusal
(binding and C ABI) before any device work."""

import ctypes
import os
import re

import pytest
import torch

import lm_ref as R
from quantize_grouped_gemm_amd import lm, mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U8, BF, F32, I64 = torch.uint8, torch.bfloat16, torch.float32, torch.int64
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(mx.LIB_PATH):
        from quantize_grouped_gemm_amd import build
        build.build()


# ---------------------------------------------------------------- gradients of the formulas

def _differences(f, x, h=1e-6):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view_as(x)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return g


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    s, w, dy, ds = (torch.randn(n, generator=g, dtype=F64) for n in ((3, 32), (32,), (3, 32), (3, 32)))
    f = lambda s_, w_: (R.norm_fwd(s_, w_, 1e-6)[1] * dy).sum() + (s_ * ds).sum()
    dx, dw = R.norm_bwd(dy, w, R.norm_fwd(s, w, 1e-6)[0], s, ds)
    # rstd also holds eps, which the gradient's mean does not see: 1e-6 of it
    assert torch.allclose(dx, _differences(lambda v: f(v, w), s), rtol=1e-5, atol=1e-6)
    assert torch.allclose(dw, _differences(lambda v: f(s, v), w), rtol=1e-6, atol=1e-7)


def test_swiglu_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    a, b, dh = (torch.randn((2, 8), generator=g, dtype=F64) for _ in range(3))
    dz = R.swiglu_bwd(dh, a, b)
    assert torch.allclose(dz[:, :8], _differences(lambda v: (R.swiglu(v, b) * dh).sum(), a), rtol=1e-6, atol=1e-8)
    assert torch.allclose(dz[:, 8:], _differences(lambda v: (R.swiglu(a, v) * dh).sum(), b), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logprob_gradient_against_differences(scale):
    g = torch.Generator().manual_seed(2)
    x = torch.randn((4, 9), generator=g, dtype=F64)
    t = torch.tensor([3, -100, 8, 0])
    dlogp, dent = torch.randn(4, generator=g, dtype=F64), torch.randn(4, generator=g, dtype=F64)

    def f(v):
        _, _, lp, ent = R.logprob_fwd(v, t, scale)
        return (lp * dlogp).sum() + (ent * dent).sum()

    m, ls, _, ent = R.logprob_fwd(x, t, scale)
    got = R.logprob_bwd(x, t, m, ls, ent, dlogp, dent, scale)
    assert torch.allclose(got, _differences(f, x), rtol=1e-6, atol=1e-8)


# ---------------------------------------------------------------- binding and header

def test_header_symbols_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxlm.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mx_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(lm.EXPORTS)
    L = lm.lib()
    for n in names:
        assert hasattr(L, n), n


def raises(fn, *args, match, **kw):
    with pytest.raises(mx.MXError, match=match):
        fn(*args, **kw)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_norm_refusals():
    T, C = 5, 256
    x, w, f = z(T, C), z(C, dtype=F32), lm.add_rmsnorm_quant
    raises(f, x.float(), w, match="x: expected")
    raises(f, z(C, T).t(), w, match="contiguous rows")
    raises(f, x, w.to(BF), match="w: dtype")
    raises(f, x, z(C + 1, dtype=F32), match="w: shape")
    raises(f, x, w, z(T, C + 128), match="r: shape")
    raises(f, z(T, 96), z(96, dtype=F32), match="multiple of 128")
    raises(f, z(T, 48), z(48, dtype=F32), layout="plain", match="multiple of 32")
    raises(f, z(1, 16512), z(16512, dtype=F32), match="at most")
    raises(f, x, w, mode="nearest", match="mode")
    raises(f, x, w, layout="k64", match="layout")
    raises(f, x, w, out={"rstd": z(T + 1, dtype=F32)}, match="rstd: shape")
    raises(f, x, w, colwise=True, out={"q_col": z(C, T, dtype=U8)}, match="q_col: ")
    raises(f, x, w, x, out={"sum": z(T, C, dtype=F32)}, match="sum: dtype")
    raises(f, x, w, match="cuda")
    raises(f, z(T, C + 8)[:, :C], w, match="cuda")
    b, rstd = lm.add_rmsnorm_bwd, z(T, dtype=F32)
    ck = (z(T, C, dtype=U8), z(C // 128, T, 4, dtype=U8))
    raises(b, x, w, rstd, match="exactly one")
    raises(b, x, w, rstd, x=x, checkpoint=ck, match="exactly one")
    raises(b, x, w, z(T + 1, dtype=F32), x=x, match="rstd: shape")
    raises(b, x, w, rstd, checkpoint=(ck[0], z(T, C // 32, dtype=U8)), match="s_ck: shape")
    raises(b, x, w, rstd, checkpoint=(z(T, C), ck[1]), match="q_ck: dtype")
    raises(b, x, w, rstd, x=x, dsum=z(T + 1, C), match="dsum: shape")
    raises(b, x, w, rstd, x=x, work=z(8, dtype=F32), match="work: 8 elements")
    raises(b, x, w, rstd, x=x, match="cuda")


def test_swiglu_refusals():
    T, H = 7, 128
    zz = z(T, 2 * H)
    raises(lm.swiglu_ckpt_fwd, zz[:, :H], z(T, H), match="row stride")
    raises(lm.swiglu_ckpt_fwd, zz[:, :H], zz[:, H:H + 96], match="b: shape")
    raises(lm.swiglu_ckpt_fwd, zz[:, :96], zz[:, H:H + 96], match="multiple of 128")
    raises(lm.swiglu_ckpt_fwd, zz[:, :H], zz[:, H:], out={"q_ck": z(T, H, dtype=U8)}, match="q_ck: ")
    raises(lm.swiglu_ckpt_fwd, zz[:, :H], zz[:, H:], match="cuda")
    q, s = z(T, 2 * H, dtype=U8), z(2 * H // 128, T, 4, dtype=U8)
    raises(lm.swiglu_ckpt_bwd, z(T, H), z(T, H, dtype=U8), s, match="q_ck: shape")
    raises(lm.swiglu_ckpt_bwd, z(T, H), q, z(T, 2 * H // 32, dtype=U8), match="s_ck: shape")
    raises(lm.swiglu_ckpt_bwd, z(T, H).float(), q, s, match="dh: expected")
    raises(lm.swiglu_ckpt_bwd, z(T, H), q, s, match="cuda")


def test_logprob_refusals():
    T, V = 6, 101
    x, t = z(T, V), z(T, dtype=I64)
    f = lm.token_logprobs
    raises(f, x.half(), t, match="x: expected")
    raises(f, x, t.int(), match="targets: dtype")
    raises(f, x, z(T + 1, dtype=I64), match="targets: shape")
    raises(f, x, t, top=65, match="top")
    raises(f, z(T, 3), t, top=4, match="top")
    raises(f, x, t, top=-1, match="top")
    raises(f, x, t, scale=0.0, match="scale")
    raises(f, x, t, scale=float("nan"), match="scale")
    raises(f, z(T, 0), t, match="empty")
    raises(f, z(V, T).t(), t, match="contiguous rows")
    raises(f, x, t, dev_err=z(1, dtype=I64), match="dev_err: dtype")
    raises(f, x, t, top=2, out={"top_idx": z(T, 2, dtype=I64)}, match="top_idx: dtype")
    raises(f, x, t, match="cuda")
    b = lm.token_logprobs_bwd
    st, e = z(T, 2, dtype=F32), z(T, dtype=F32)
    raises(b, x, t, z(T, dtype=F32), e, match="stats: shape")
    raises(b, x, t, st, e, dlogp=z(T), match="dlogp: dtype")
    raises(b, x, t, st, e, out={"q_row": z(T, V, dtype=U8)}, match="q_row: ")
    raises(b, x, t, st, e, match="cuda")


def test_abi_refusals():
    L = lm.lib()
    p, odd = ctypes.c_void_p(16), ctypes.c_void_p(18)   # never dereferenced

    def fwd(x=p, ld=128, r=None, w=p, rows=4, cols=128, eps=1e-6, mode=0, layout=1, sum_=None, rstd=p, q=p, s=p,
            qc=None, sc=None, qk=None, sk=None):
        return L.mx_add_rmsnorm_quant(x, ld, r, ld, w, rows, cols, eps, mode, layout, sum_, rstd, q, s, qc, sc, qk,
                                      sk, None)

    assert fwd(mode=2) == 4 and fwd(layout=3) == 4 and fwd(eps=-1.0) == 4 and fwd(eps=float("inf")) == 4
    assert fwd(rows=-1) == 2 and fwd(rows=65535 * 128 + 1) == 2 and fwd(cols=96) == 2 and fwd(cols=16512) == 2
    assert fwd(x=None) == 1 and fwd(w=None) == 1 and fwd(q=None) == 1 and fwd(r=p) == 1 and fwd(qc=p) == 1
    assert fwd(x=odd) == 3 and fwd(ld=64) == 3 and fwd(ld=132) == 3 and fwd(w=odd) == 3 and fwd(s=odd) == 3
    assert fwd(rows=0) == 0

    # more than 2^21 tiles, row strides above 2^26
    assert fwd(rows=65535 * 128, cols=16384, ld=16384) == 2 and b"tiles" in L.mx_last_error()
    assert fwd(ld=(1 << 26) + 8) == 2
    assert L.mx_token_logprobs_bwd(p, 0, 1 << 26, 4, 1 << 26, p, -100, p, p, p, p, 1.0, 0, 1, p, p, p, p, None, None) == 2
    assert L.mx_token_logprobs_bwd(p, 0, 1 << 20, 1 << 20, 1 << 20, p, -100, p, p, p, p, 1.0, 0, 1, p, p, p, p, None,
                                   None) == 2

    def bwd(x=p, qk=None, sk=None, dw=p, work=p, dx=p, cols=128, rows=4):
        return L.mx_add_rmsnorm_bwd(p, 128, p, p, x, 128, qk, sk, None, 0, rows, cols, 0, 1, dx, dw, p, p, None, None,
                                    work, None)

    assert bwd(x=None) == 1 and bwd(qk=p, sk=p) == 1 and bwd(x=None, qk=p) == 1 and bwd(dw=None) == 1
    assert bwd(work=None) == 1 and bwd(dx=odd) == 3 and bwd(cols=64) == 2
    assert L.mx_add_rmsnorm_bwd_work(0, 128) == 0 and L.mx_add_rmsnorm_bwd_work(1, 128) >= 128

    assert L.mx_swiglu_ckpt_fwd(p, p, 256, 5, 96, 0, 1, p, p, p, p, p, p, None) == 2
    assert L.mx_swiglu_ckpt_fwd(p, p, 256, 5, 128, 0, 1, p, p, p, p, None, p, None) == 1
    assert L.mx_swiglu_ckpt_fwd(p, odd, 256, 5, 128, 0, 1, p, p, p, p, p, p, None) == 3
    assert L.mx_swiglu_ckpt_bwd(p, 64, p, p, 5, 128, 0, 1, p, p, p, p, None) == 3
    assert L.mx_swiglu_ckpt_bwd(None, 128, p, p, 5, 128, 0, 1, p, p, p, p, None) == 1

    def lp(x=p, dt=0, ld=100, rows=4, vocab=100, t=p, scale=1.0, top=0, tl=None, ti=None, stats=p):
        return L.mx_token_logprobs(x, dt, ld, rows, vocab, t, -100, scale, top, p, p, stats, tl, ti, p, None, None)

    assert lp(dt=2) == 4 and lp(scale=0.0) == 4 and lp(scale=1e7) == 4 and lp(vocab=0) == 2
    assert lp(vocab=2 ** 31, ld=2 ** 31) == 2 and lp(ld=99) == 3 and lp(top=65) == 2 and lp(top=101) == 2
    assert lp(top=5) == 1 and lp(x=None) == 1 and lp(t=None) == 1 and lp(x=odd, dt=1) == 3
    assert lp(stats=ctypes.c_void_p(20)) == 3 and lp(rows=0) == 0
    assert L.mx_token_logprobs_work(0, 1000, 5) == 0

    def lb(layout=1, mode=0, q=p, stats=p):
        return L.mx_token_logprobs_bwd(p, 0, 100, 4, 100, p, -100, stats, p, p, p, 1.0, mode, layout, q, p, p, p, None,
                                       None)

    assert lb(layout=2) == 4 and lb(mode=5) == 4 and lb(q=None) == 1 and lb(q=odd) == 3 and lb(stats=None) == 1
    if not torch.cuda.is_available():
        assert fwd() == 5 and bwd() == 5 and lp() == 5 and lb() == 5 and L.mx_last_error()


@pytest.mark.parametrize("dt,limit", [(0, 1 << 26), (1, 1 << 25)])
def test_logit_gradient_strides_are_bounded_in_bytes(dt, limit):
    L, p = lm.lib(), ctypes.c_void_p(16)

    def status(ld, vocab=1000):
        return L.mx_token_logprobs_bwd(p, dt, ld, 4, vocab, p, -100, p, p, p, p, 1.0, 0, 1, p, p, p, p, None, None)

    assert status(limit + 8) == 2 and status(limit, limit) == 2
    if not torch.cuda.is_available():
        assert status(limit) == 5 and status(limit, limit - 128) == 5
