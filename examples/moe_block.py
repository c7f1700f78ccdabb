"""A Mixture-of-Experts block around the routed experts, from the library's calls.

    n            = norm_pre(r)                                     norm that opens the block
    logits       = n Wr^T                                          router (a plain product)
    ids, w       = route_topk(logits)                              top-k, counts, balance loss
    y_routed     = moe_forward("mxfp4", n, ids, w, ...)            routed experts
    y_shared     = fp8_linear(swiglu(fp8_linear(n)))               shared expert, FP8 with 128-value scales
    r', n'       = norm_post(r, y_routed + y_shared, gate, alpha)  sandwich norm, gate, residual scale, next block's norm

`forward` serves (any number of tokens, one for a decode step); `train_step` adds the gradients of what such a block
trains beside frozen routed experts: its norms, its gate, the shared expert and, through the balance loss, the router.

    python examples/moe_block.py [--tokens 64] [--hidden 512] [--experts 16] [--top-k 4] [--inter 256]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_mixture_experts_moe_gb300 import binding as qb  # noqa: E402
from quantized_mixture_experts_moe_gb300 import inputs as gen  # noqa: E402

EPS = 1e-6


class MoeBlock:
    def __init__(self, H=512, I=256, E=16, k=4, seed=0, device="cuda"):
        self.H, self.I, self.E, self.k = H, I, E, k
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device=device) * scale

        # norms, column gate, router and shared expert: fp32 masters
        self.w_in, self.w_out, self.w_next = (1 + normal(H, scale=0.1) for _ in range(3))
        self.gate = 1 + normal(1, H, scale=0.1)
        self.alpha = 0.5
        self.router = normal(E, H, scale=H ** -0.5)
        self.w1, self.w2 = normal(2 * I, H, scale=H ** -0.5), normal(H, I, scale=I ** -0.5)
        self.quantise()
        # routed experts: MXFP4 weights, packed once
        weights = gen.make_all(gen.custom("block", "mxfp4", 1, H, E, k, I, seed=seed))
        self.experts = qb.prepack_mxfp4(*(torch.from_numpy(weights[n]).to(device) for n in ("w1", "w1_s", "w2", "w2_s")), H, I)

    def quantise(self):
        """The shared expert's FP8 codes and scales, from its masters (again after each update of them)."""
        self.w1_q, self.w1_s, self.w1t_q = qb.fp8_quant_blocks(self.w1, transposed=True)
        self.w2_q, self.w2_s, self.w2t_q = qb.fp8_quant_blocks(self.w2, transposed=True)

    def routed(self, n, ids, w):
        out, _ = qb.moe_forward("mxfp4", n.view(torch.int16), ids, w, *self.experts, I=self.I, E=self.E)
        return out.view(torch.bfloat16)

    def forward(self, r, n=None, mask=None, coef=None):
        """r [T, H] bf16 stream; n: its norm, where the block before gave it; mask: tokens to route.  Returns (r', n', what
        train_step needs)."""
        rstd_in = None
        if n is None:
            n, rstd_in = qb.norm_pre(r, self.w_in, eps=EPS)
        logits = n.float() @ self.router.t()
        route = qb.route_topk(logits, self.k, mask=mask, coef=coef)
        h = qb.fp8_linear(n, self.w1_q, self.w1_s)
        a = (torch.nn.functional.silu(h[:, :self.I].float()) * h[:, self.I:].float()).bfloat16()
        y = self.routed(n, route.ids, route.w) + qb.fp8_linear(a, self.w2_q, self.w2_s)
        out, n_next, rstd, rstd_next = qb.norm_post(r, y, w=self.w_out, gate=self.gate, alpha=self.alpha, w_next=self.w_next, eps=EPS)
        return out, n_next, dict(r=r, n=n, rstd_in=rstd_in, logits=logits, route=route, h=h, a=a, y=y, out=out, rstd=rstd, rstd_next=rstd_next)

    def train_step(self, r, dout, dn_next, coef=0.01, mask=None):
        """Loss gradients for dout (of r') and dn_next (of n'); the routed experts and their weights w are held fixed."""
        out, n_next, s = self.forward(r, mask=mask, coef=coef)
        dr, dy, dw_out, dgate, dw_next = qb.norm_post_backward(dout, s["y"], w=self.w_out, rstd=s["rstd"], gate=self.gate, alpha=self.alpha,
                                                               dn=dn_next, out=out, w_next=self.w_next, rstd_next=s["rstd_next"])
        da, dw2 = qb.fp8_linear_backward(dy, s["a"], self.w2t_q, self.w2_s)
        h1, h2 = s["h"][:, :self.I].float(), s["h"][:, self.I:].float()
        sig = torch.sigmoid(h1)
        da = da.float()
        dh = torch.cat([da * h2 * sig * (1 + h1 * (1 - sig)), da * h1 * sig], 1).bfloat16()
        dn, dw1 = qb.fp8_linear_backward(dh, s["n"], self.w1t_q, self.w1_s)
        one = torch.ones(1, device=r.device)
        dlogits = qb.route_topk_backward(s["logits"], s["route"], dloss=one)
        dn = (dn.float() + dlogits @ self.router).bfloat16()
        dx, dw_in = qb.norm_pre_backward(dn, r, s["rstd_in"], self.w_in, dres=dr)
        return dx, dict(w_in=dw_in, w_out=dw_out, w_next=dw_next, gate=dgate, router=dlogits.t() @ s["n"].float(), w1=dw1, w2=dw2), s["route"]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--inter", type=int, default=256)
    a = ap.parse_args()
    block = MoeBlock(a.hidden, a.inter, a.experts, a.top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    out, n_next, s = block.forward(r, coef=0.01)
    print(f"prefill of {a.tokens} tokens: |r'| {out.float().norm().item():.4f}, balance loss {s['route'].loss.item():.6f}, "
          f"pairs per expert {s['route'].counts[:-1].tolist()}")
    out1, n1, _ = block.forward(r[:1])
    print(f"decode of one token: {'the same row' if torch.allclose(out1.float(), out[:1].float(), rtol=2e-2, atol=2e-2) else 'ANOTHER row'}")
    dout, dn_next = ((0.1 * torch.randn(r.shape, generator=g, device="cuda")).bfloat16() for _ in range(2))
    dx, grads, _ = block.train_step(r, dout, dn_next)
    print("gradients: dx %.4f, " % dx.float().norm().item() + ", ".join(f"{n} {t.float().norm().item():.4f}" for n, t in grads.items()))
    assert int(qb.status_word("cuda").item()) == 0


if __name__ == "__main__":
    main()
