"""Training steps of a small language model of balanced MoE blocks.

    python examples/block_step.py [--steps 40]

Each block routes its tokens with sigmoid scores, groups of experts and a bias
for balance, adds a shared expert that every token passes, and stands between
two norms: one after it, with a gate for every token, and one before the next
block, in one pass over the residual stream.  The bias is moved after every
step by the loads of the experts.  Data and optimiser are those of
``train_step.py``.
"""

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dropless_moe_block_gb300 as dm  # noqa: E402

EPS = 1e-5


class BlockLanguageModel:
    """Weights, gradients and buffers of T tokens through `layers` blocks of
    width d: E routed experts of width F in `groups` groups, k per token, and a
    shared one of width S, under a V-word head.  `scale` is the residual
    stream's, `gates` [layers, T] what each token's blocks are weighed with."""

    def __init__(self, T, d, V, layers=2, E=16, F=128, k=4, groups=4, top_groups=2, S=256, scale=1.0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf = torch.bfloat16

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(bf)

        self.T, self.d, self.V, self.layers, self.scale = T, d, V, layers, scale
        routing = {"scores": "sigmoid", "groups": groups, "top_groups": top_groups}
        self.blocks = [dm.DMoELayer(T, d, E, F, k, "swiglu", True, balanced=routing) for _ in range(layers)]
        self.shared = [dm.SharedExpert(T, d, S) for _ in range(layers)]
        p = {"embedding": normal(V, d, std=1.0), "head": normal(V, d, std=d ** -0.5)}
        f32 = {}  # weights kept in fp32
        for l in range(layers):
            p |= {f"gate{l}": normal(E, d, std=d ** -0.5), f"w1_{l}": normal(d, E * F, std=d ** -0.5),
                  f"w3_{l}": normal(d, E * F, std=d ** -0.5), f"w2_{l}": normal(E * F, d, std=F ** -0.5),
                  f"s1_{l}": normal(d, S, std=d ** -0.5), f"s2_{l}": normal(S, d, std=S ** -0.5)}
            f32 |= {f"sb1_{l}": torch.zeros(S, device="cuda"), f"sb2_{l}": torch.zeros(d, device="cuda")}
        for l in range(layers + 1):
            f32[f"pre{l}"] = torch.ones(d, device="cuda")
        for l in range(layers):
            f32[f"post{l}"] = torch.ones(d, device="cuda")
        self.p = p | f32
        self.g = {"embedding": torch.zeros(V, d, device="cuda"), "head": torch.empty_like(p["head"])}
        for l, (b, s) in enumerate(zip(self.blocks, self.shared)):
            self.g |= {f"w1_{l}": b.dW1, f"w3_{l}": b.dW3, f"w2_{l}": b.dW2, f"gate{l}": torch.empty(E, d, device="cuda"),
                       f"s1_{l}": s.dW1, f"s2_{l}": s.dW2, f"sb1_{l}": s.db1, f"sb2_{l}": s.db2}
        for n in f32:
            if n.startswith("p"):
                self.g[n] = torch.empty(d, device="cuda")
        rows = lambda: torch.empty(T, d, device="cuda", dtype=bf)  # noqa: E731
        col = lambda: torch.empty(T, device="cuda")  # noqa: E731
        self.h = [rows() for _ in range(layers + 1)]  # the residual stream before each block, and at the end
        self.y = [rows() for _ in range(layers + 1)]  # what the norms before the blocks and the head give
        self.rstd_h, self.rstd_u = [col() for _ in range(layers + 1)], [col() for _ in range(layers)]
        self.dh, self.du, self.dy = [rows(), rows()], rows(), rows()
        self.d_gates = torch.empty(layers, T, device="cuda")
        self.loss, self.lse, self.norm = col(), col(), torch.empty(1, device="cuda")
        ws = max(dm.linear_cross_entropy_workspace_size(T, d, V), dm.add_rms_norm_backward_workspace_size(T, d),
                 dm.sandwich_norm_backward_workspace_size(T, d))
        self.ws = torch.empty(ws, device="cuda", dtype=torch.uint8)
        self.grads = dm.GradList(self.g.values())  # clipped in place

    def forward_backward(self, tokens, targets, gates):
        """Per-token losses (0 where a target is -100); the gradients of their
        mean are in self.g and self.d_gates."""
        p, L = self.p, self.layers
        self.h[0] = p["embedding"][tokens]
        dm.add_rms_norm(self.h[0], None, p["pre0"], EPS, None, self.y[0], rstd=self.rstd_h[0])
        for l, (b, s) in enumerate(zip(self.blocks, self.shared)):
            routed = b.forward(self.y[l], None, p[f"w1_{l}"], p[f"w2_{l}"], p[f"w3_{l}"], w_gate=p[f"gate{l}"])
            u = s.forward(self.y[l], p[f"s1_{l}"], p[f"s2_{l}"], p[f"sb1_{l}"], p[f"sb2_{l}"], residual=routed)
            dm.sandwich_norm(u, self.h[l], p[f"post{l}"], p[f"pre{l + 1}"], EPS, self.h[l + 1], self.y[l + 1],
                             gate=gates[l], scale=self.scale, rstd_u=self.rstd_u[l], rstd_h=self.rstd_h[l + 1])
        dm.linear_cross_entropy(self.y[L], p["head"], targets, self.loss, self.lse, self.ws, dx=self.dy,
                                dw=self.g["head"])
        dy, dh = self.dy, None
        for l in reversed(range(L)):
            b, s = self.blocks[l], self.shared[l]
            out = self.dh[l % 2]
            dm.sandwich_norm_backward(dy, s.y, self.h[l + 1], p[f"post{l}"], p[f"pre{l + 1}"], self.rstd_u[l],
                                      self.rstd_h[l + 1], self.du, out, self.g[f"post{l}"], self.g[f"pre{l + 1}"],
                                      self.ws, dh=dh, gate=gates[l], d_gate=self.d_gates[l], scale=self.scale)
            dh = out
            dy = s.backward(self.du, self.y[l], p[f"s1_{l}"], p[f"s2_{l}"])
            dy.add_(b.backward(self.du, self.y[l], p[f"w1_{l}"], p[f"w2_{l}"], p[f"w3_{l}"]))
            dy.addmm_(b.d_logits.to(dy.dtype), p[f"gate{l}"])
            torch.mm(b.d_logits.t(), self.y[l].float(), out=self.g[f"gate{l}"])
        dx = self.du
        dm.add_rms_norm_backward(dy, self.h[0], p["pre0"], self.rstd_h[0], dx, self.g["pre0"], self.ws, dh=dh)
        self.g["embedding"].zero_().index_add_(0, tokens, dx.float())
        return self.loss

    def step(self, tokens, targets, gates, lr=0.5, max_norm=1.0, rate=1e-3):
        """One SGD step, and one of the routers' biases; the mean loss before it
        and the gradients' global norm."""
        loss = self.forward_backward(tokens, targets, gates)
        dm.clip_grad_norm(self.grads, max_norm, self.norm)
        for n, w in self.p.items():
            w.add_(self.g[n].to(w.dtype), alpha=-lr)
        for b in self.blocks:
            b.balance(rate)
        return loss.sum() / (targets != -100).sum().clamp(min=1), self.norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--words", type=int, default=1009)
    a = ap.parse_args()
    torch.manual_seed(1)
    model = BlockLanguageModel(a.tokens, a.width, a.words)
    follow = torch.randperm(a.words, device="cuda")
    gates = torch.ones(model.layers, a.tokens, device="cuda")
    for i in range(a.steps):
        tokens = torch.randint(0, a.words, (a.tokens,), device="cuda")
        loss, norm = model.step(tokens, follow[tokens].to(torch.int32), gates)
        if i % 5 == 0 or i + 1 == a.steps:
            load = model.blocks[0].tokens_per_expert
            print(f"step {i:3d}  loss {float(loss):.4f}  gradient norm {float(norm):.3f}  "
                  f"loads of the first block's experts {int(load.min())} to {int(load.max())}")
    err = dm.get_error()
    if err:
        raise SystemExit(f"device error word {err:#x}")


if __name__ == "__main__":
    main()
