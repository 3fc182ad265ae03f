"""The balanced block's training step: its gradients against autograd of the same model in plain fp32 torch; the layer with a
balanced router and the shared expert by themselves."""

import importlib.util
import os

import pytest
import torch

from helpers import RMS_CHAIN, TOL_CHAIN

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dropless_moe_block_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("block_step", os.path.join(ROOT, "examples", "block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.dm.get_error(clear=True)
    return m


def plain_loss(m, p, tokens, targets, gates, eps):
    """The model in fp32, with the experts the package's routers chose."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * w

    h = p["embedding"][tokens]
    for l, b in enumerate(m.blocks):
        y = norm(h, p[f"pre{l}"])
        scores = torch.sigmoid(y @ p[f"gate{l}"].t())
        chosen = b.expert_idx.long()
        w = scores.gather(1, chosen)
        w = w / w.sum(1, keepdim=True)
        E = scores.shape[1]
        F = p[f"w1_{l}"].shape[1] // E
        out = torch.nn.functional.gelu(y @ p[f"s1_{l}"] + p[f"sb1_{l}"]) @ p[f"s2_{l}"] + p[f"sb2_{l}"]
        for e in range(E):
            c = slice(e * F, (e + 1) * F)
            a = torch.nn.functional.silu(y @ p[f"w1_{l}"][:, c]) * (y @ p[f"w3_{l}"][:, c])
            out = out + (a @ p[f"w2_{l}"][c]) * (w * (chosen == e)).sum(1, keepdim=True)
        h = m.scale * h + gates[l][:, None] * norm(out, p[f"post{l}"])
    logits = norm(h, p[f"pre{m.layers}"]) @ p["head"].t()
    return torch.nn.functional.cross_entropy(logits, targets.long(), ignore_index=-100)


@pytest.mark.gpu
def test_gradients_of_a_step(ex):
    T, d, V = 300, 128, 513
    m = ex.BlockLanguageModel(T, d, V, layers=2, E=8, F=128, k=3, groups=4, top_groups=2, S=136, scale=0.9, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    for n, w in m.p.items():  # weights that are not all ones, biases that are not zeros
        if w.dim() == 1:
            w.add_(torch.randn(w.shape, generator=g, device="cuda"), alpha=0.1)
    for b in m.blocks:
        b.route_bias.copy_(torch.randn(8, generator=g, device="cuda") * 0.05)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    targets[::7] = -100
    gates = torch.sigmoid(torch.randn(2, T, generator=g, device="cuda"))
    loss = m.forward_backward(tokens, targets, gates)
    p = {n: w.float().requires_grad_(True) for n, w in m.p.items()}
    free = gates.clone().requires_grad_(True)
    want = plain_loss(m, p, tokens, targets, free, ex.EPS)
    want.backward()
    got = float(loss.sum() / (targets != -100).sum())
    want = float(want.detach())
    # every operator between the embedding and the loss rounds its output to
    # bf16 once: the chain's bound, as for a layer's outputs
    assert abs(got - want) <= TOL_CHAIN * want
    assert ex.dm.get_error() == 0
    pairs = {n: (m.g[n].float(), w.grad) for n, w in p.items()} | {"gates": (m.d_gates, free.grad)}
    for n, (a, b) in pairs.items():
        rms = float((a - b).square().mean().sqrt() / b.square().mean().sqrt())
        # two blocks, each with four roundings on the way forth and back (experts,
        # shared expert, norms, stream): the one-block chain's bound for the
        # head, twice it further down
        assert rms <= (RMS_CHAIN if n in ("head", "pre2") else 2 * RMS_CHAIN), f"{n}: rms {rms:.3e}"
    # the same bits once more: every sum runs in a fixed order
    kept = {n: t.clone() for n, t in m.g.items() if n != "embedding"}
    m.forward_backward(tokens, targets, gates)
    for n, t in kept.items():
        assert torch.equal(m.g[n], t), n


@pytest.mark.gpu
def test_steps_run_and_balance(ex):
    T, d, V = 512, 128, 257
    m = ex.BlockLanguageModel(T, d, V, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    gates = torch.ones(2, T, device="cuda")
    for _ in range(3):
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        before = [b.route_bias.clone() for b in m.blocks]
        loss, norm = m.step(tokens, tokens.to(torch.int32), gates)
        assert bool(torch.isfinite(loss)) and bool(torch.isfinite(norm).all())
        for b, was in zip(m.blocks, before):
            load = b.tokens_per_expert.double()
            assert torch.equal(b.route_bias, was + 1e-3 * torch.sign(load.mean() - load).float())
    assert ex.dm.get_error() == 0


@pytest.mark.gpu
def test_balanced_layer_in_a_graph(ex):
    """A captured step of a layer that routes with a bias, replayed after the bias has moved."""
    dm = ex.dm
    T, d, E, F, k = 256, 128, 8, 128, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    bf = torch.bfloat16
    x, dy = (torch.randn(T, d, generator=g, device="cuda").to(bf) for _ in range(2))
    logits = torch.randn(T, E, generator=g, device="cuda")
    w1, w2 = ((torch.randn(*s, generator=g, device="cuda") * 0.1).to(bf) for s in ((d, E * F), (E * F, d)))
    routing = {"scores": "sigmoid", "groups": 4, "top_groups": 2, "scale": 1.5}
    a, b = (dm.DMoELayer(T, d, E, F, k, "gelu", True, balanced=routing) for _ in range(2))
    graph, launches = a.capture(x, logits, w1, w2, dy=dy, concurrent=True)
    for bias in (0.0, 0.3):
        for layer in (a, b):
            layer.route_bias.copy_(torch.linspace(-bias, bias, E, device="cuda"))
        graph.replay()
        b.forward(x, logits, w1, w2)
        b.backward(dy, x, w1, w2)
        for n in ("expert_idx", "gate_w", "y", "dx", "dW1", "dW2", "d_logits"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert dm.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("T,d,F", [(1, 64, 256), (70, 128, 520), (600, 256, 1032)])
def test_shared_expert(ex, T, d, F, act):
    dm = ex.dm
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    x, res, dy = r(T, d), r(T, d), r(T, d)
    w1, w2, b1, b2 = r(d, F, std=d ** -0.5), r(F, d, std=F ** -0.5), r(F), r(d)
    s = dm.SharedExpert(T, d, F, act)
    y = s.forward(x, w1, w2, b1, b2, residual=res)
    dx = s.backward(dy, x, w1, w2)
    p = [t.double().requires_grad_(True) for t in (x, w1, w2, b1, b2)]
    f = torch.nn.functional.gelu if act == "gelu" else torch.nn.functional.silu
    ref = f(p[0] @ p[1] + p[3]) @ p[2] + p[4] + res.double()
    ref.backward(dy.double())
    for n, a, b in (("y", y, ref.detach()), ("dx", dx, p[0].grad), ("dW1", s.dW1, p[1].grad), ("dW2", s.dW2, p[2].grad),
                    ("db1", s.db1, p[3].grad), ("db2", s.db2, p[4].grad)):
        a = a.double()
        # roundings between two products (the activation or its factor, dz, the
        # output): three half steps of bf16 of a chain, as of a layer's
        assert float((a - b).abs().max()) <= TOL_CHAIN * float(b.abs().max()), n
        assert float((a - b).norm()) <= RMS_CHAIN * float(b.norm()), n
    assert dm.get_error() == 0


def test_layer_refuses_other_fronts_and_names():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as dm
    with pytest.raises(ValueError, match="separate"):
        dm.DMoELayer(64, 128, 4, 128, 1, device="cpu", front="fused", balanced={})
    with pytest.raises(ValueError, match="unknown bias"):
        dm.DMoELayer(64, 128, 4, 128, 1, device="cpu", balanced={"bias": 1})
    layer = dm.DMoELayer(64, 128, 4, 128, 1, device="cpu")
    with pytest.raises(ValueError, match="bias"):
        layer.balance(0.1)
    names = [n for n, _ in dm.DMoELayer(64, 128, 4, 128, 1, device="cpu", balanced={}).forward_calls(
        None, None, None, None, w_gate=object())]
    assert names[:3] == ["gate_route_topk", "route_balanced", "permute_pad"]
    with pytest.raises(ValueError):
        dm.SharedExpert(4, 64, 64, "relu", device="cpu")
