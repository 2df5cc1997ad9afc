"""Training steps of one pre-norm Mixture-of-Experts block on the library's operators.

    stream = x + r                                layer_norm_fwd (residual add and norm in one pass)
    y      = layer_norm(stream)
    s, ids = top-K of softmax(y Wr)               router_fwd, with the balance and z losses per packed sequence
    h      = y W1_e, a = SiLU(gate) * up          glu_fwd: the activation, and gate/up saved in 8 bits
    out    = stream + sum_k s_k a W2_e

and back: moe_bwd from the 8-bit checkpoint (dx, dW1, dW2, ds), router_bwd and balance_bwd for the router's logits,
layer_norm_bwd with the skip connection's gradient added.  The expert and router products of the forward are plain
torch matrix products.

    python examples/train_block.py [--steps 20] [--tokens 2048]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_routing_gb300 as mb  # noqa: E402

MODE, RENORM, EPS = mb.ROUTER_TOPK_OVER_SOFTMAX, True, 1e-5


class Block:
    """Weights of the block and one training step's forward and backward."""

    def __init__(self, H, I, E, K, block_size=128, alpha=0.01, beta=0.001, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        self.H, self.I, self.E, self.K, self.B = H, I, E, K, block_size
        self.alpha, self.beta = alpha, beta
        self.gamma, self.beta_norm = torch.ones(H, device=device), torch.zeros(H, device=device)
        self.Wr = rand(H, E) * H ** -0.5
        self.W1 = (rand(E, H, 2 * I) * H ** -0.5).to(torch.bfloat16)
        self.W2 = (rand(E, I, H) * I ** -0.5).to(torch.bfloat16)

    def forward(self, x, residual, seg_offsets):
        """x, residual bf16 [T, H]; seg_offsets int32 [num_seq + 1] of the packed sequences.  Returns the stream
        behind the block, the two router losses and what the backward needs."""
        n = mb.layer_norm_fwd(x, self.gamma, self.beta_norm, eps=EPS, residual=residual)
        y = n["y"]
        logits = y.float() @ self.Wr
        route = mb.router_fwd(MODE, logits, self.K, renorm=RENORM, seg_offsets=seg_offsets, alpha=self.alpha,
                              beta=self.beta)
        meta = mb.route_meta(route["ids"], self.E, self.B)
        ends = meta["expert_offsets"].tolist()
        rows = ends[-1]                                     # routed slots; padding tokens have none
        token = meta["x_gather_idx"][:rows].long()
        grouped = y[token]
        split = [slice(ends[e], ends[e + 1]) for e in range(self.E)]
        h = torch.cat([grouped[s] @ self.W1[e] for e, s in enumerate(split)])
        act = mb.glu_fwd(h, meta, self.B)                   # h itself is not kept
        down = torch.cat([act["a"][s] @ self.W2[e] for e, s in enumerate(split)])
        s = route["scores"].flatten()[meta["s_scatter_idx"][:rows].long()]
        out = n["sum"].float().index_add(0, token, s[:, None] * down.float()).to(torch.bfloat16)
        saved = dict(norm=n, logits=logits, route=route, ckpt_q=act["ckpt_q"], ckpt_sf=act["ckpt_sf"], seg=seg_offsets)
        return out, route["loss"], saved

    def backward(self, dout, saved):
        """dout bf16 [T, H]: gradient of the stream behind the block.  Returns the gradients of the stream in front
        (of x and of the residual alike) and of the weights; the router losses' gradient is in them."""
        n, logits, route, seg = (saved[k] for k in ("norm", "logits", "route", "seg"))
        y = n["y"]
        g = mb.moe_bwd(x=y, dout=dout, s=route["scores"], ids=route["ids"], E=self.E, I=self.I, block_size=self.B,
                       ckpt_q=saved["ckpt_q"], ckpt_sf=saved["ckpt_sf"], W1=self.W1, W2=self.W2)
        dlogits = mb.router_bwd(MODE, route["ids"], g["ds"], self.E, logits=logits, scores=route["scores"], renorm=RENORM)
        dlogits = mb.balance_bwd(logits, route["lse"], route["counts"], self.K, seg_offsets=seg, alpha=self.alpha,
                                 beta=self.beta, add=dlogits)
        dy = (g["dx"].float() + dlogits @ self.Wr.t()).to(torch.bfloat16)
        d = mb.layer_norm_bwd(dy, n["sum"], self.gamma, n["mean"], n["rstd"], dres=dout)
        return dict(stream=d["dx"], gamma=d["dgamma"], beta=d["dbeta"], Wr=y.float().t() @ dlogits, W1=g["dW1"],
                    W2=g["dW2"], status=g["status"], dlogits=dlogits)

    def update(self, grads, lr):
        for name, w in (("gamma", self.gamma), ("beta", self.beta_norm), ("Wr", self.Wr), ("W1", self.W1), ("W2", self.W2)):
            w -= (lr * grads[name].float()).to(w.dtype)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    T, H = a.tokens, 512
    block = Block(H=H, I=256, E=16, K=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, target = (torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    seg = torch.tensor([0, T // 3, T // 3 + T // 2, T - 8], dtype=torch.int32, device="cuda")   # 8 padding tokens
    for step in range(a.steps):
        out, aux, saved = block.forward(x, r, seg)
        diff = out.float() - target.float()
        grads = block.backward((diff / T).to(torch.bfloat16), saved)
        block.update(grads, lr=0.02)
        if step % 5 == 0 or step == a.steps - 1:
            assert int(grads["status"].item()) == 0 and int(saved["route"]["status"].item()) == 0
            print(f"step {step:3d}  loss {0.5 * diff.square().sum().item() / T:10.4f}  balance {aux[0].item():.5f}  z {aux[1].item():.5f}")


if __name__ == "__main__":
    main()
