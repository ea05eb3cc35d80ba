"""The operators together: one block with head and loss (lm_block), against the
same block unquantized in float64 with autograd; the operators under HIP graph
capture, on a side stream, and with given outputs.

Tolerance of the composed step: an E4M3 operand carries a relative noise of
2^-4 / sqrt(3) * 0.74 = 2.7% (rounding uniform in a binade), so a GEMM adds
2 * 0.027^2 of its result's power and a checkpoint 0.027^2. A gradient that
has passed k such operands has an SQNR of about 31.5 - 10 log10(k) dB; 4 dB are
left for what the softmax and the norms do with the noise they receive."""

import math

import pytest
import torch

from _helpers import dev
from quantize_grouped_gemm_amd import lm, lm_block, mx, synth

pytestmark = pytest.mark.gpu
F64, BF = torch.float64, torch.bfloat16


def _block(T, D, H, V, seed):
    g = synth.generator(seed)
    n = synth.normal_bf16
    w = dict(w13=n((2 * H, D), D ** -0.5, g), w2=n((D, H), H ** -0.5, g), head=n((V, D), D ** -0.5, g))
    norm1, norm2 = (1 + 0.1 * torch.randn(D, generator=g) for _ in range(2))
    x, r = n((T, D), 1.0, g), n((T, D), 0.5, g)
    t = torch.randint(0, V, (T,), generator=g)
    if T > 3:
        t[3] = -100
    return w, norm1, norm2, x, r, t


def _sqnr(ref, got):
    got = got.detach().cpu().to(F64)
    return 10 * math.log10(float(ref.square().sum() / (ref - got).square().sum()))


@pytest.mark.parametrize("T,D,H,V", [(200, 256, 384, 1000), (33, 128, 256, 515)])
def test_block_step(gpu, T, D, H, V):
    w, norm1, norm2, x, r, t = _block(T, D, H, V, T)
    g = torch.Generator().manual_seed(1)
    dlogp, dent = -torch.rand(T, generator=g) / T, 0.1 * torch.rand(T, generator=g) / T
    # unquantized, float64
    lv = {k: v.to(F64).requires_grad_() for k, v in w.items()}
    n1, n2 = norm1.to(F64).requires_grad_(), norm2.to(F64).requires_grad_()
    s = (x.to(F64) + r.to(F64)).requires_grad_()
    norm = lambda v, k: v * (v.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * k
    z = norm(s, n1) @ lv["w13"].T
    y = (z[:, :H] * torch.sigmoid(z[:, :H]) * z[:, H:]) @ lv["w2"].T
    lp = torch.log_softmax(norm(y + s, n2) @ lv["head"].T, -1)
    ok = t != -100
    logp = torch.where(ok, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    ent = -(lp.exp() * lp).sum(-1)
    ((logp * dlogp.to(F64)).sum() + (ent * dent.to(F64)).sum()).backward()

    d = dev()
    blk = lm_block.LMBlock(norm1.to(d), w["w13"].to(d), w["w2"].to(d), norm2.to(d), w["head"].to(d))
    f, grads = blk.step(x.to(d), r.to(d), t.to(d), dlogp.to(d), dent.to(d))
    ref = {"dx": s.grad, "dw13": lv["w13"].grad, "dw2": lv["w2"].grad, "dhead": lv["head"].grad, "dnorm1": n1.grad,
           "dnorm2": n2.grad}
    # operands passed: logits 6 forward; dlogits 6 + 1; then 1 + 1 a GEMM and 1 a checkpoint
    passed = {"dhead": 8, "dnorm2": 9, "dw2": 12, "dx": 16, "dw13": 15, "dnorm1": 16}
    got = {k: _sqnr(ref[k], grads[k]) for k in ref}
    print({k: round(v, 1) for k, v in got.items()}, "logp", round(_sqnr(logp.detach(), f["logp"]), 1), flush=True)
    for k, n in passed.items():
        assert got[k] > 31.5 - 10 * math.log10(n) - 4, k
    # the noise of the logits (6 operands of 2.7%, logits of about unit size) moves a log probability by 2 * 0.07
    assert (f["logp"].cpu().to(F64) - logp.detach()).abs().max() < 6 * 0.14
    # scoring sees the same forward
    sc = blk.score(x.to(d), r.to(d), t.to(d), top=5)
    assert torch.equal(sc["logp"], f["logp"]) and sc["top_idx"].shape == (T, 5)


def test_score_one_token(gpu):
    """Scoring one token equals its row of a batch."""
    w, norm1, norm2, x, r, t = _block(64, 256, 128, 777, 5)
    d = dev()
    blk = lm_block.LMBlock(norm1.to(d), w["w13"].to(d), w["w2"].to(d), norm2.to(d), w["head"].to(d))
    x, r, t = x.to(d), r.to(d), t.to(d)
    many, one = blk.score(x, r, t, top=3), blk.score(x[9:10], r[9:10], t[9:10], top=3)
    for k in many:
        assert torch.equal(many[k][9:10], one[k]), k


def test_graph_replays_the_step(gpu):
    """The step's operators captured once with given outputs, replayed on new
    inputs with eager work between the replays."""
    T, C, H, V = 77, 256, 128, 5000
    d = dev()
    g = synth.generator(2)

    def inputs(i):
        g = synth.generator(100 + i)
        n = synth.normal_bf16
        return [n(s, 1.0, g).to(d) for s in ((T, C), (T, C), (T, 2 * H), (T, H), (T, V))]

    w = torch.ones(C, device=d)
    t = torch.randint(0, V, (T,), device=d)
    dl = torch.randn(T, device=d)
    work = torch.empty(lm.bwd_work(T, C), device=d)

    def chain(v, o=None):
        o = o or {}
        x, r, z, dh, lg = v
        a = lm.add_rmsnorm_quant(x, w, r, colwise=True, checkpoint=True, out=o.get("a"))
        b = lm.add_rmsnorm_bwd(r, w, a["rstd"], checkpoint=(a["q_ck"], a["s_ck"]), dsum=x, colwise=True, out=o.get("b"),
                               work=work)
        c = lm.swiglu_ckpt_fwd(z[:, :H], z[:, H:], out=o.get("c"))
        e = lm.swiglu_ckpt_bwd(dh, c["q_ck"], c["s_ck"], out=o.get("e"))
        f = lm.token_logprobs(lg, t, top=7, out=o.get("f"))
        h = lm.token_logprobs_bwd(lg, t, f["stats"], f["entropy"], dl, dl, out=o.get("h"))
        return {"a": a, "b": b, "c": c, "e": e, "f": f, "h": h}

    bufs = inputs(0)
    outs = chain(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(bufs, outs)
    for i in range(1, 5):
        new = inputs(i)
        for b, n in zip(bufs, new):
            b.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref = chain(new)
        torch.cuda.synchronize()
        for k in ref:
            for name in ref[k]:
                assert torch.equal(outs[k][name], ref[k][name]), (i, k, name)


def test_side_stream(gpu):
    """Calls go to the current stream: made on a side stream behind the work
    that fills their inputs, they see those inputs."""
    d = dev()
    x = torch.zeros((512, 4096), dtype=BF, device=d)
    w = torch.ones(4096, device=d)
    src = synth.normal_bf16((512, 4096), 1.0, synth.generator(3)).to(d)
    lg = torch.zeros((64, 50001), dtype=BF, device=d)
    lsrc = synth.normal_bf16((64, 50001), 2.0, synth.generator(4)).to(d)
    t = torch.arange(64, device=d)
    want, lwant = lm.add_rmsnorm_quant(src, w, colwise=True), lm.token_logprobs(lsrc, t, top=4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x.copy_(src)
        lg.copy_(lsrc)
        got, lgot = lm.add_rmsnorm_quant(x, w, colwise=True), lm.token_logprobs(lg, t, top=4)
    s.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k]), k
    for k in lwant:
        assert torch.equal(lwant[k], lgot[k]), k


def test_given_outputs_are_used_and_nothing_past_them_is_written(gpu):
    """Outputs inside larger buffers: the bytes around them stay."""
    d = dev()
    T, C = 45, 416
    x = synth.normal_bf16((T, C), 1.0, synth.generator(6)).to(d)
    w = torch.ones(C, device=d)
    ref = lm.add_rmsnorm_quant(x, w, x, layout="plain", colwise=True, checkpoint=True)
    bufs, out = {}, {}
    for k, v in ref.items():
        n = v.numel() * v.element_size()
        bufs[k] = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=d)
        out[k] = bufs[k][256:256 + n].view(v.dtype).view(v.shape)
    got = lm.add_rmsnorm_quant(x, w, x, layout="plain", colwise=True, checkpoint=True, out=out)
    for k, v in ref.items():
        assert got[k].data_ptr() == out[k].data_ptr() and torch.equal(got[k], v), k
        n = v.numel() * v.element_size()
        assert (bufs[k][:256] == 0xA5).all() and (bufs[k][256 + n:] == 0xA5).all(), k
    V = 1003
    lg = synth.normal_bf16((T, V), 2.0, synth.generator(7)).to(d)
    t = torch.arange(T, device=d)
    for ref, call in ((lm.token_logprobs(lg, t, top=9), lambda o: lm.token_logprobs(lg, t, top=9, out=o)),):
        bufs, out = {}, {}
        for k, v in ref.items():
            n = v.numel() * v.element_size()
            bufs[k] = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=d)
            out[k] = bufs[k][256:256 + n].view(v.dtype).view(v.shape)
        call(out)
        for k, v in ref.items():
            n = v.numel() * v.element_size()
            assert torch.equal(out[k], v), k
            assert (bufs[k][:256] == 0xA5).all() and (bufs[k][256 + n:] == 0xA5).all(), k
