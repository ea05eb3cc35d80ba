"""A routed-experts SwiGLU layer composed from the routing operators (moe), the
experts' grouped products (mx or b128) and the fused SwiGLU (mx): forward,
training step, and the form for a few tokens. The router's logits come from the
caller (its projection is a GEMM of any kind) and their gradient goes back there.

  forward   weights, idx = route(logits)           scores, top experts
            sizes, offs, src, pos                  dispatch
            rows in expert order, quantized        gather_quantize
            z = rows w13[e]^T                      grouped product
            h = silu(z_a) z_b                      swiglu
            y = h w2[e]^T                          grouped product
            out_t = r_t + sum_j weights_tj y_pos   combine
  backward  dweights, dlogits                      combine_bwd, route_bwd
            dy rows = weight * dout, quantized     gather_quantize
            dh = dy w2[e], dw2[e] = dy^T h         grouped products
            dz                                     swiglu backward
            dx rows = dz w13[e], dw13[e]           grouped products
            dx_t = sum of its rows                 combine

Two recipes for the experts: "mxfp8" (blocks of 32, E8M0 scales) and "b128"
(float32 scales of 1 x 128 and 128 x 128), whose SwiGLU goes through bf16. Groups
are padded to 128 rows where columns are quantized or mx multiplies; b128 alone
needs no padding to run forward, so a few tokens cost the rows that they have.
"""

import torch

from . import b128, moe, mx
from .lm import _matrix, _rows

_RECIPES = ("mxfp8", "b128")


class MoELayer:
    """Experts' weights w13 bf16 [E, 2H, D] (gate rows first), w2 [E, D, H]; D and
    H multiples of 128. `routing`: the keyword arguments of moe.route (score,
    groups, top_groups, group_score, renorm, scale). bias: float32 [E] or None, the
    balance term of the choice (may be changed between calls)."""

    def __init__(self, w13, w2, top, recipe="mxfp8", bias=None, **routing):
        if recipe not in _RECIPES:
            raise mx.MXError(f"recipe: {recipe!r}, expected 'mxfp8' or 'b128'")
        if not isinstance(w2, torch.Tensor) or w2.dim() != 3:
            raise mx.MXError("w2: expected a tensor [E, D, H]")
        self.E, self.D, self.H = w2.shape
        if self.D % 128 or self.H % 128:
            raise mx.MXError(f"w2: D ({self.D}) and H ({self.H}) must be multiples of 128")
        self.top, self.recipe, self.bias, self.routing = top, recipe, bias, routing
        self.set_weights(w13, w2)

    def set_weights(self, w13, w2):
        """Quantizes the experts' weights (once an optimizer step)."""
        for w, name, shape in ((w2, "w2", (self.E, self.D, self.H)), (w13, "w13", (self.E, 2 * self.H, self.D))):
            if not isinstance(w, torch.Tensor) or w.dtype is not torch.bfloat16 or w.shape != shape:
                raise mx.MXError(f"{name}: expected a bf16 tensor of shape {shape}")
        if self.recipe == "b128":
            self.q13, self.q2 = b128.quantize_weight(w13), b128.quantize_weight(w2)
        else:
            self.q13, self.q2 = mx.quantize(w13, "rceil", True, True), mx.quantize(w2, "rceil", True, True)

    def _grouped(self, a, q, offs, transposed=False, out=None):
        if self.recipe == "b128":
            return b128.grouped_mm(a["q_row"], a["s_row"], q["q_t" if transposed else "q"],
                                   q["s_t" if transposed else "s"], offs, out=out)
        d = "col" if transposed else "row"
        return mx.grouped_mm_fwd(a["q_row"], a["s_row"], q["q_" + d], q["s_" + d], offs, out=out)

    def _wgrad(self, g, x, offs):
        if g["q_col"].shape[1] == 0:      # no token
            return torch.zeros((self.E, g["q_col"].shape[0], x["q_col"].shape[0]), device=offs.device)
        f = b128.grouped_mm_wgrad if self.recipe == "b128" else mx.grouped_mm_wgrad
        return f(g["q_col"], g["s_col"], x["q_col"], x["s_col"], offs)

    def _gather(self, x, src, weights=None, train=False):
        mode = "f32" if self.recipe == "b128" else "rceil"
        return moe.gather_quantize(x, src, self.top, weights, fmt=self.recipe, mode=mode, colwise=train)

    def forward(self, x, logits, r=None, train=False):
        """x bf16 [T, D], logits bf16 or float32 [T, E], r bf16 [T, D] or None
        (added to the output). Returns (out bf16 [T, D], what backward takes)."""
        T = _matrix(x, "x")[0]
        _rows(x, "x", torch.bfloat16, (T, self.D))
        # a token without logits or without x, or an expert without weights, would drop out unseen
        if _matrix(logits, "logits", (torch.bfloat16, torch.float32)) != (T, self.E):
            raise mx.MXError(f"logits: shape {tuple(logits.shape)}, expected {(T, self.E)}")
        if r is not None:
            _rows(r, "r", torch.bfloat16, (T, self.D))
        f = moe.route(logits, self.top, bias=self.bias, **self.routing)
        plan = moe.dispatch(f["idx"], self.E, multiple=128 if train or self.recipe == "mxfp8" else 1)
        xq = self._gather(x, plan["src"], train=train)
        cap, H = plan["src"].numel(), self.H
        z = torch.empty((cap + -cap % 128, 2 * H), dtype=torch.bfloat16, device=x.device)
        z[cap:].zero_()
        self._grouped(xq, self.q13, plan["offs"], out=z[:cap])
        a, b = z[:, :H], z[:, H:]
        if self.recipe == "b128":
            h = mx.swiglu_quant_fwd(a, b, want_h=True)["h"][:cap]
            hq = b128.quantize(h, colwise=train)
        else:
            hq = mx.swiglu_quant_fwd(a, b)
        y = self._grouped(hq, self.q2, plan["offs"])
        out = moe.combine(y, plan["pos"], f["weights"], r)
        return out, dict(f, **plan, x=x, logits=logits, xq=xq, z=z, hq=hq, y=y)

    def backward(self, c, dout):
        """Gradients for dout bf16 [T, D], c from forward(train=True): a dict with
        dx (bf16; r's gradient is dout itself), dlogits (of the logits' type), dw13 and dw2
        (float32)."""
        if "q_col" not in c["xq"]:
            raise mx.MXError("backward: c comes from a forward without train=True")
        _rows(dout, "dout", torch.bfloat16, c["x"].shape)
        H, offs = self.H, c["offs"]
        kw = {k: v for k, v in self.routing.items() if k in ("score", "renorm", "scale")}
        dlogits = moe.route_bwd(c["logits"], c["idx"], moe.combine_bwd(dout, c["y"], c["pos"]), **kw)
        dyq = self._gather(dout, c["src"], c["weights"], train=True)
        dh = self._grouped(dyq, self.q2, offs, transposed=True)
        dw2 = self._wgrad(dyq, c["hq"], offs)
        a, b = c["z"][:, :H], c["z"][:, H:]
        if self.recipe == "b128":
            dzq = b128.quantize(mx.swiglu_quant_bwd(dh, a, b, want_dab=True)["dab"], colwise=True)
        else:
            dzq = mx.swiglu_quant_bwd(dh, a, b)
        dx = moe.combine(self._grouped(dzq, self.q13, offs, transposed=True), c["pos"])
        return {"dx": dx, "dlogits": dlogits, "dw13": self._wgrad(dzq, c["xq"], offs), "dw2": dw2}
