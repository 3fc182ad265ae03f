"""The example's training step: its gradients against autograd of the same
model in plain fp32 torch, and the loss it reaches."""

import importlib.util
import os

import pytest
import torch

from helpers import RMS_CHAIN, TOL_CHAIN

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dropless_moe_block_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.dm.get_error(clear=True)
    return m


def plain_loss(m, p, tokens, targets, eps):
    """The model in fp32, with the experts the package's router chose."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * w

    h = p["embedding"][tokens]
    for l, b in enumerate(m.blocks):
        y = norm(h, p[f"norm{l}"])
        probs = torch.softmax(y @ p[f"gate{l}"].t(), 1)
        chosen = b.expert_idx.long()
        w = probs.gather(1, chosen)
        w = w / w.sum(1, keepdim=True)
        F = p[f"w1_{l}"].shape[1] // probs.shape[1]
        out = torch.zeros_like(h)
        for e in range(probs.shape[1]):
            c = slice(e * F, (e + 1) * F)
            a = torch.nn.functional.silu(y @ p[f"w1_{l}"][:, c]) * (y @ p[f"w3_{l}"][:, c])
            out = out + (a @ p[f"w2_{l}"][c]) * (w * (chosen == e)).sum(1, keepdim=True)
        h = h + out
    logits = norm(h, p["norm_out"]) @ p["head"].t()
    return torch.nn.functional.cross_entropy(logits, targets.long(), ignore_index=-100)


def test_gradients_of_a_step(ex):
    T, d, V = 300, 128, 513
    m = ex.MoELanguageModel(T, d, V, layers=2, E=4, F=128, k=2, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    targets[::7] = -100
    loss = m.forward_backward(tokens, targets)
    p = {n: w.float().requires_grad_(True) for n, w in m.p.items()}
    want = plain_loss(m, p, tokens, targets, ex.EPS)
    want.backward()
    got = float(loss.sum() / (targets != -100).sum())
    # every operator between the embedding and the loss rounds its output to
    # bf16 once: the chain's bound, as for a layer's outputs
    want = float(want.detach())
    assert abs(got - want) <= TOL_CHAIN * want
    assert ex.dm.get_error() == 0
    for n, w in p.items():
        a, b = m.g[n].float(), w.grad
        rms = float((a - b).square().mean().sqrt() / b.square().mean().sqrt())
        # two layers, each with three roundings on the way forth and back: the
        # one-block chain's bound for the head, twice it further down
        assert rms <= (RMS_CHAIN if n in ("head", "norm_out") else 2 * RMS_CHAIN), f"{n}: rms {rms:.3e}"


def test_loss_falls(ex):
    T, d, V = 1024, 256, 257
    m = ex.MoELanguageModel(T, d, V, layers=2, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    follow = torch.randperm(V, generator=g, device="cuda")
    losses = []
    for _ in range(30):
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        loss, norm = m.step(tokens, follow[tokens].to(torch.int32))
        losses.append(float(loss))
    assert ex.dm.get_error() == 0
    assert losses[0] > 5.0 and losses[-1] < 0.5 * losses[0], losses
