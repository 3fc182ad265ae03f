"""Training steps of a small MoE language model with the package's operators.

    python examples/train_step.py [--steps 40]

Each of the model's layers is a residual addition + RMS norm, a linear gate
and a dropless MoE block; a last norm feeds the vocabulary head, whose loss
and gradients come from ``linear_cross_entropy``.  After the backward pass all
gradients are clipped to a global norm, and plain SGD updates the weights.
The data is synthetic: the next word is a fixed permutation of the last one,
so the loss falls from ln(V) within a few steps.
"""

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dropless_moe_block_gb300 as dm  # noqa: E402

EPS = 1e-5


class MoELanguageModel:
    """Weights, gradients and buffers of T tokens through `layers` MoE blocks of
    width d (E experts of width F, k per token) under a V-word head."""

    def __init__(self, T, d, V, layers=2, E=8, F=256, k=2, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf = torch.bfloat16

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(bf)

        self.T, self.d, self.V, self.layers, self.k = T, d, V, layers, k
        self.blocks = [dm.DMoELayer(T, d, E, F, k, "swiglu", True) for _ in range(layers)]
        p = {"embedding": normal(V, d, std=1.0), "head": normal(V, d, std=d ** -0.5),
             "norm_out": torch.ones(d, device="cuda", dtype=bf)}
        for l in range(layers):
            p[f"norm{l}"] = torch.ones(d, device="cuda", dtype=bf)
            p[f"gate{l}"] = normal(E, d, std=d ** -0.5)
            p[f"w1_{l}"] = normal(d, E * F, std=d ** -0.5)
            p[f"w3_{l}"] = normal(d, E * F, std=d ** -0.5)
            p[f"w2_{l}"] = normal(E * F, d, std=F ** -0.5)
        self.p = p
        # gradients: the blocks hold their own, the norms' are fp32
        self.g = {"embedding": torch.zeros(V, d, device="cuda"), "head": torch.empty_like(p["head"])}
        for l, b in enumerate(self.blocks):
            self.g |= {f"w1_{l}": b.dW1, f"w3_{l}": b.dW3, f"w2_{l}": b.dW2,
                       f"gate{l}": torch.empty(E, d, device="cuda")}
        for n in [f"norm{l}" for l in range(layers)] + ["norm_out"]:
            self.g[n] = torch.empty(d, device="cuda")
        rows = lambda: torch.empty(T, d, device="cuda", dtype=bf)  # noqa: E731
        self.h = [rows() for _ in range(layers + 1)]  # the residual stream at each norm
        self.y = [rows() for _ in range(layers + 1)]  # what the norms give
        self.rstd = [torch.empty(T, device="cuda") for _ in range(layers + 1)]
        self.dh = [rows() for _ in range(2)]          # the stream's gradient, by turns
        self.dy = rows()
        self.loss, self.lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        self.norm = torch.empty(1, device="cuda")
        ws = max(dm.linear_cross_entropy_workspace_size(T, d, V), dm.add_rms_norm_backward_workspace_size(T, d))
        self.ws = torch.empty(ws, device="cuda", dtype=torch.uint8)
        self.grads = dm.GradList(self.g.values())  # clipped in place

    def forward_backward(self, tokens, targets):
        """Per-token losses (0 where a target is -100); the gradients of their
        mean are in self.g."""
        p, L = self.p, self.layers
        x, stream = p["embedding"][tokens], None
        for l, b in enumerate(self.blocks):
            dm.add_rms_norm(x, stream, p[f"norm{l}"], EPS, self.h[l] if stream is not None else None, self.y[l],
                            rstd=self.rstd[l])
            if stream is None:
                self.h[l] = x  # nothing was added yet
            stream = self.h[l]
            x = b.forward(self.y[l], None, p[f"w1_{l}"], p[f"w2_{l}"], p[f"w3_{l}"], w_gate=p[f"gate{l}"])
        dm.add_rms_norm(x, stream, p["norm_out"], EPS, self.h[L], self.y[L], rstd=self.rstd[L])
        dm.linear_cross_entropy(self.y[L], p["head"], targets, self.loss, self.lse, self.ws, dx=self.dy,
                                dw=self.g["head"])

        dh = self.dh[0]
        dm.add_rms_norm_backward(self.dy, self.h[L], p["norm_out"], self.rstd[L], dh, self.g["norm_out"], self.ws)
        for l in reversed(range(L)):
            b = self.blocks[l]
            # dh is the gradient of the block's output and of the stream beside it
            dy = b.backward(dh, self.y[l], p[f"w1_{l}"], p[f"w2_{l}"], p[f"w3_{l}"])
            dy = torch.addmm(dy, b.d_logits.to(dy.dtype), p[f"gate{l}"])
            torch.mm(b.d_logits.t(), self.y[l].float(), out=self.g[f"gate{l}"])
            out = self.dh[1] if dh is self.dh[0] else self.dh[0]
            dm.add_rms_norm_backward(dy, self.h[l], p[f"norm{l}"], self.rstd[l], out, self.g[f"norm{l}"], self.ws,
                                     dh=dh)
            dh = out
        self.g["embedding"].zero_().index_add_(0, tokens, dh.float())
        return self.loss

    def step(self, tokens, targets, lr=0.5, max_norm=1.0):
        """One SGD step; the mean loss before it and the gradients' global norm."""
        loss = self.forward_backward(tokens, targets)
        dm.clip_grad_norm(self.grads, max_norm, self.norm)
        for n, w in self.p.items():
            w.add_(self.g[n].to(w.dtype), alpha=-lr)
        return loss.sum() / (targets != -100).sum().clamp(min=1), self.norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--words", type=int, default=1009)
    a = ap.parse_args()
    torch.manual_seed(1)
    model = MoELanguageModel(a.tokens, a.width, a.words)
    follow = torch.randperm(a.words, device="cuda")
    for i in range(a.steps):
        tokens = torch.randint(0, a.words, (a.tokens,), device="cuda")
        loss, norm = model.step(tokens, follow[tokens].to(torch.int32))
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i:3d}  loss {float(loss):.4f}  gradient norm {float(norm):.3f}")
    err = dm.get_error()
    if err:
        raise SystemExit(f"device error word {err:#x}")


if __name__ == "__main__":
    main()
