"""The last block of an MXFP8 language model with its head and loss, composed
from the GEMMs (mx) and the layer-boundary operators (lm): training step and
scoring. Nothing between two GEMMs is done outside a fused operator, and what
the backward needs is kept in 8 bits.

  forward   s  = x + r;  n = norm(s)            add_rmsnorm_quant (s kept in 8 bits)
            z  = n w13^T                        scaled_mm
            h  = silu(z_a) z_b                  swiglu_ckpt_fwd   (z kept in 8 bits)
            y  = h w2^T                         scaled_mm
            s2 = y + s; n2 = norm(s2)           add_rmsnorm_quant (s2 kept in 8 bits)
            logits = n2 head^T                  scaled_mm
            log probabilities, entropy          token_logprobs
  backward  dlogits                             token_logprobs_bwd
            dn2 = dlogits head, dhead           scaled_mm x 2
            ds2 (= dy, gradient of s)           add_rmsnorm_bwd
            dh = dy w2, dw2                     scaled_mm x 2
            dz                                  swiglu_ckpt_bwd
            dn = dz w13, dw13                   scaled_mm x 2
            ds (= dx = dr)                      add_rmsnorm_bwd   (joins ds2)

The number of tokens is free, and so is the vocabulary: the head's weight is
padded with zero rows to a multiple of 128 and the loss reads the logits' first
V columns.
"""

import torch

from . import lm, mx


class LMBlock:
    """MXFP8 weights of the block: w13 bf16 [2H, D] (gate rows first), w2
    [D, H], head [V, D]; norm1, norm2 float32 [D]. D and H are multiples of
    128."""

    def __init__(self, norm1, w13, w2, norm2, head, mode="rceil", eps=1e-6):
        self.norm1, self.norm2, self.mode, self.eps = norm1, norm2, mode, eps
        self.H, self.D, self.V = w2.shape[1], w2.shape[0], head.shape[0]
        self.Vp = lm.padded_rows(self.V)
        full = torch.zeros((self.Vp, self.D), dtype=torch.bfloat16, device=head.device)
        full[:self.V] = head
        self.q13 = mx.quantize(w13, mode, True, True)
        self.q2 = mx.quantize(w2, mode, True, True)
        self.qv = mx.quantize(full, mode, True, True)

    def _forward(self, x, r, train):
        n1 = lm.add_rmsnorm_quant(x, self.norm1, r, self.eps, self.mode, colwise=train, checkpoint=train)
        z = mx.scaled_mm(n1["q_row"], n1["s_row"], self.q13["q_row"], self.q13["s_row"])
        h = lm.swiglu_ckpt_fwd(z[:, :self.H], z[:, self.H:], self.mode)
        y = mx.scaled_mm(h["q_row"], h["s_row"], self.q2["q_row"], self.q2["s_row"])
        n2 = lm.add_rmsnorm_quant(y, self.norm2, n1["sum"], self.eps, self.mode, colwise=train, checkpoint=train)
        logits = mx.scaled_mm(n2["q_row"], n2["s_row"], self.qv["q_row"], self.qv["s_row"])
        return n1, h, n2, logits[:, :self.V]

    def score(self, x, r, targets, scale=1.0, top=0):
        """Log probabilities, entropy and alternatives of the given tokens
        (lm.token_logprobs) for the stream x + r, bf16 [T, D]."""
        return lm.token_logprobs(self._forward(x, r, False)[3], targets, scale=scale, top=top)

    def step(self, x, r, targets, dlogp, dent=None, scale=1.0):
        """Forward and backward for the objective sum(dlogp * logp) +
        sum(dent * entropy): returns (token_logprobs' dict, gradients), the
        latter dx (bf16, of x and of r), dw13, dw2, dhead, dnorm1, dnorm2
        (float32)."""
        m, f32 = self.mode, torch.float32
        n1, h, n2, logits = self._forward(x, r, True)
        f = lm.token_logprobs(logits, targets, scale=scale)
        g = lm.token_logprobs_bwd(logits, targets, f["stats"], f["entropy"], dlogp, dent, scale=scale, mode=m)
        dn2 = mx.scaled_mm(g["q_row"], g["s_row"], self.qv["q_col"], self.qv["s_col"])
        dhead = mx.scaled_mm(g["q_col"], g["s_col"], n2["q_col"], n2["s_col"], f32)
        b2 = lm.add_rmsnorm_bwd(dn2, self.norm2, n2["rstd"], checkpoint=(n2["q_ck"], n2["s_ck"]), mode=m, colwise=True)
        dh = mx.scaled_mm(b2["q_row"], b2["s_row"], self.q2["q_col"], self.q2["s_col"])
        dw2 = mx.scaled_mm(b2["q_col"], b2["s_col"], h["q_col"], h["s_col"], f32)
        dz = lm.swiglu_ckpt_bwd(dh, h["q_ck"], h["s_ck"], m)
        dn = mx.scaled_mm(dz["q_row"], dz["s_row"], self.q13["q_col"], self.q13["s_col"])
        dw13 = mx.scaled_mm(dz["q_col"], dz["s_col"], n1["q_col"], n1["s_col"], f32)
        b1 = lm.add_rmsnorm_bwd(dn, self.norm1, n1["rstd"], checkpoint=(n1["q_ck"], n1["s_ck"]), dsum=b2["dx"], mode=m,
                                rowwise=False)
        return f, {"dx": b1["dx"], "dw13": dw13, "dw2": dw2, "dhead": dhead[:self.V], "dnorm1": b1["dw"],
                   "dnorm2": b2["dw"]}
