"""The block's operators where test_block_ops.py does not take them: products cut along K with all that
follows the sums, outputs that lie over what their call reads, and the edges of what the operators allow.

Sums of products are made exact, where that helps: whole numbers times a power of two, whose sums fp32 holds however they are
ordered or cut, so that what follows them is compared without a sum's error.
"""

import ctypes
import math

import pytest
import torch

import test_block_ops as ops
from test_block_ops import (BF, F32, I32, U16, U32, clean, close, dm, empty, randn, ref_act, ref_route, ref_sandwich_backward,  # noqa: F401
                            ref_scores, check_backward, route, weights, workspace)


def whole(seed, *shape, most=2, unit=1.0, dtype=BF):
    """Whole numbers from -most to most, times unit (a power of two)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randint(-most, most + 1, shape, generator=g, device="cuda").double() * unit).to(dtype)


def launches(dm, f):
    n = dm.launch_count()
    f()
    return dm.launch_count() - n


# --------------------------------------------------------------- dense linear

# Forward products that a pair of CTAs sums in parts, one part a range of K, and a second launch joins.
CUT = [(1, 26960, 8), (7, 16392, 72), (130, 12296, 1032), (509, 15168, 1208), (2051, 8200, 264), (4300, 8200, 264)]
# Forward products of whole sums in pairs of CTAs: tiles 256 and 512 columns wide.
WHOLE = [(2560, 512, 4096), (1031, 1000, 5128), (2303, 6152, 4096)]


def exact_case(M, K, N, act, bias, residual):
    x, w = whole(1, M, K), whole(2, K, N, unit=2.0 ** -6)
    b = None if bias is None else whole(3, N, unit=0.25, dtype=bias)
    r = whole(4, M, N, most=9, unit=0.125) if residual else None
    z = x.double() @ w.double()  # exact: |z| 2^6 < 4 K < 2^24
    if b is not None:
        z = z + b.double()
    return x, w, b, r, z


def check_exact(got, z, act, r, what, deriv=None):
    y, f = ref_act(z, act)
    if r is not None:
        y = y + r.double()
    if act == "none":
        assert torch.equal(got, y.to(F32).to(BF)), what  # (y is exact in fp32: one rounding)
        return
    # Phi is known to 1.5e-7, sigmoid to a few ulp, and what is added rounds once more
    ea = 4e-7 * (1 + z.abs())
    close(got, y, U16 * y.abs() + ea + 4 * U32 * (y.abs() + 4), what)
    if deriv is not None:
        close(deriv, f, U16 * f.abs() + ea, what + ": deriv")


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", CUT)
@pytest.mark.parametrize("act,bias,residual", [("none", None, False), ("none", BF, True), ("gelu", F32, True),
                                               ("silu", BF, False), ("silu", F32, True)])
def test_linear_cut_along_its_sum(dm, M, K, N, act, bias, residual):
    x, w, b, r, z = exact_case(M, K, N, act, bias, residual)
    y, f = empty(M, N), None if act == "none" else empty(M, N)
    ws, guard = workspace(dm.linear_workspace_size(M, K, N))
    # a later rule of the cuts that takes these sizes elsewhere has to name others here
    assert launches(dm, lambda: dm.linear(x, w, y, ws, bias=b, act=act, deriv=f, residual=r)) == 2
    check_exact(y, z, act, r, "y", f)
    assert bool((guard == 0x5a).all())
    if r is not None:  # onto the residual, and rows of wider tensors
        kept = r.clone()
        dm.linear(x, w, r, ws, bias=b, act=act, residual=r)
        assert torch.equal(r, y)
        wide = empty(M, K + N + 16)
        wide[:, 8:8 + K], wide[:, 16 + K:] = x, kept
        y.fill_(777.0)
        dm.linear(wide[:, 8:8 + K], w, y, ws, bias=b, act=act, residual=wide[:, 16 + K:])
        assert torch.equal(r, y)


@pytest.mark.gpu
def test_linear_workspace_of_cut_products_serves_fewer_rows(dm):
    K, N = 15168, 1208
    n = dm.linear_workspace_size(509, K, N)
    ws, guard = workspace(n)
    w = whole(2, K, N, unit=2.0 ** -6)
    cut = 0
    for M in (509, 400, 300, 257, 200, 130, 65, 3):
        assert dm.linear_workspace_size(M, K, N) <= n
        x, y = whole(M, M, K), empty(M, N)
        cut += launches(dm, lambda: dm.linear(x, w, y, ws)) == 2
        assert torch.equal(y, (x.double() @ w.double()).to(F32).to(BF)), M
    assert cut >= 3
    assert bool((guard == 0x5a).all())
    with pytest.raises(dm.DmoeError):  # too small for the parts' sums, which are not written then
        x, y = whole(1, 509, K), empty(509, N)
        dm.linear(x, w, y, ws[:1 << 16])
    assert bool((y == 777.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", WHOLE)
@pytest.mark.parametrize("act,bias", [("none", BF), ("gelu", F32), ("silu", None)])
def test_linear_of_pairs_onto_its_residual(dm, M, K, N, act, bias):
    """y over the residual, which the same tiles read: the result of the call that keeps them apart."""
    x, w, b, r, z = exact_case(M, K, N, act, bias, True)
    y = empty(M, N)
    ws, _ = workspace(dm.linear_workspace_size(M, K, N))
    assert launches(dm, lambda: dm.linear(x, w, y, ws, bias=b, act=act, residual=r)) == 1
    check_exact(y, z, act, r, "y")
    for _ in range(3):  # not once by chance
        onto = r.clone()
        dm.linear(x, w, onto, ws, bias=b, act=act, residual=onto)
        assert torch.equal(onto, y)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(2560, 4096, 512), (1031, 5128, 1000), (130, 1032, 12296), (1, 8, 26960), (2051, 264, 8200)])
def test_linear_backward_onto_its_factor(dm, M, K, N):
    """dx over factor, in whole tiles and behind sums that were cut."""
    dy, w, f = whole(1, M, N), whole(2, K, N, unit=2.0 ** -6), whole(3, M, K, most=9, unit=0.125)
    ws, guard = workspace(dm.linear_backward_workspace_size(M, K, N))
    want = ((dy.double() @ w.double().t()) * f.double()).to(F32).to(BF)  # below 2^24 units of 2^-9: exact before its rounding
    dx = empty(M, K)
    dm.linear_backward(dy, None, w, dx, None, ws, factor=f)
    assert torch.equal(dx, want)
    for _ in range(3):
        onto = f.clone()
        dm.linear_backward(dy, None, w, onto, None, ws, factor=onto)
        assert torch.equal(onto, want)
    assert bool((guard == 0x5a).all())


def test_linear_widths_end_at_2_to_the_20_without_gpu():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    L, most = m.lib(), 1 << 20
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(9)]
    for K, N in ((most + 8, 64), (64, most + 8)):
        assert m.linear_workspace_size(4, K, N) == 0 and m.linear_backward_workspace_size(4, K, N) == 0
        # x, ldx, w, bias, f32, act, residual, ldr, M, K, N, y, deriv, ws, ws_bytes
        assert L.dmoe_linear(p[0], K, p[1], None, 0, 0, None, 0, 4, K, N, p[2], None, p[3], 1 << 30, None) == 1
        # dy, lddy, deriv, x, ldx, w, factor, M, K, N, dx, dw, f32, dbias, ws, ws_bytes
        assert L.dmoe_linear_backward(p[0], N, None, p[1], K, p[2], None, 4, K, N, p[3], p[4], 0, None, p[5], 1 << 30, None) == 1
    for K, N in ((most, 64), (64, most)):
        assert m.linear_workspace_size(4, K, N) > 0 and m.linear_backward_workspace_size(4, K, N) > 0


# -------------------------------------------------------------------- routing

@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(8300, 64, 4, 1, 1), (8193, 64, 8, 2, 1), (8200, 128, 3, 4, 2), (8195, 256, 8, 8, 4),
                                                     (8192, 256, 8, 1, 1), (50, 64, 1, 1, 1), (70, 256, 1, 8, 2), (3000, 96, 5, 4, 2)])
def test_route_with_experts_ruled_out_and_forced(dm, T, E, k, groups, top_groups, scores):
    """A bias of minus infinity or NaN rules an expert out, one of plus infinity forces it: alone, together, and where they leave fewer
    experts than are chosen."""
    size = E // groups
    logits = randn(1, T, E, dtype=F32)
    logits[3::50, size - 1:] = -math.inf  # few experts left
    logits[7::60] = -math.inf             # none
    for out, forced in (([2], []), ([0, 1, E - 1], []), ([5], [3]), ([], [1, E - 2]), (list(range(4, E)), [0])):
        bias = randn(2, E, scale=0.02, dtype=F32)
        bias[out] = -math.inf
        bias[out[1:2]] = math.nan
        bias[forced] = math.inf
        idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=top_groups)
        ri, rw = ref_route(logits, bias, k, scores, groups, top_groups, True, 1.0)
        assert torch.equal(idx.long(), ri), (out, forced)
        close(w, rw, 400 * U32 * rw + 2.0 ** -126, "gate_w")


def c_of(logits, bias, scores):
    """What experts are chosen by, in 64 bits."""
    z = clean(logits)
    c = ref_scores(z, scores) + bias.double()
    return torch.where((z == -math.inf) | torch.isnan(c), torch.full_like(c, -math.inf), c)


def check_choice(logits, bias, idx, w, k, scores, groups, top_groups):
    """A choice whose candidates lie as close as 64-bit roundings: not the reference's order, but its values, and the weights of the
    very choice.  A 64-bit score is off by some 1e-16 of values below 1, a softmax's by 1e-15."""
    T, E = logits.shape
    i, c = idx.long(), c_of(logits, bias, scores)
    assert int(i.min()) >= 0 and int(i.max()) < E
    assert bool((i.sort(1).values.diff(dim=1) > 0).all())  # distinct
    got = c.gather(1, i)
    assert float(got.diff(dim=1).max()) < 1e-14  # descending
    settled = torch.ones(T, dtype=torch.bool, device="cuda")
    if top_groups < groups:
        worth = c.view(T, groups, -1).topk(2, 2).values.sum(2)
        order = worth.sort(dim=1, descending=True).values
        least = order[:, top_groups - 1:top_groups]
        assert bool((worth.gather(1, i // (E // groups)) >= least - 4e-14).all())  # of groups that may stay
        settled = (least - order[:, top_groups:top_groups + 1])[:, 0] > 4e-14
    ri, _ = ref_route(logits, bias, k, scores, groups, top_groups, True, 1.0)
    assert float((got - c.gather(1, ri)).abs()[settled].max()) < 1e-14
    s = ref_scores(clean(logits), scores).gather(1, i)
    close(w, s / s.sum(1, keepdim=True), 400 * U32 * s / s.sum(1, keepdim=True), "gate_w")
    return int(settled.sum())


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,groups,top_groups", [(300, 1, 1), (300, 8, 3), (8300, 1, 1), (8300, 8, 3)])
def test_route_of_rows_that_the_bias_levels(dm, scores, T, groups, top_groups):
    """Choices within fp32's step of one another in every row: all of them are the 64 bits' to make."""
    E, k = 256, 8
    row = randn(1, 1, E, dtype=F32)
    bias = (0.5 - ref_scores(row.double(), scores)[0]).to(F32)
    logits = row + randn(2, T, E, scale=1e-7, dtype=F32)
    c = c_of(logits, bias, scores)
    assert float((c.amax(1) - c.amin(1)).max()) < 1e-6
    idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=top_groups)
    assert check_choice(logits, bias, idx, w, k, scores, groups, top_groups) > T // 2


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(9000, 96, 6, 4, 2), (9000, 160, 8, 5, 3), (6000, 512, 8, 16, 4), (6000, 512, 8, 1, 1),
                                                     (4000, 1024, 33, 32, 5)])
def test_route_of_several_tokens_a_warp(dm, T, E, k, groups, top_groups, scores):
    """Warps that walk from token to token, with the groups' scores of one where the last one's were."""
    ops.test_route(dm, T, E, k, groups, top_groups, scores, True, True)


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", [(5, 8, 1, 4), (300, 96, 3, 4), (40, 64, 1, 2), (9000, 256, 8, 8), (9000, 64, 8, 2)])
def test_route_by_groups_whose_worth_passes_fp32(dm, T, E, k, groups, scores):
    """Two biases near fp32's end: their sums are infinite in fp32, and different in 64 bits."""
    size = E // groups
    logits = randn(1, T, E, dtype=F32)
    for sums in ((2e38, 3e38), (3e38, 2e38), (-2e38, -1.9e38), (-3e38, 3e38)):
        bias = torch.full((E,), sums[0], device="cuda")
        bias[size:2 * size] = sums[1]
        idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=1)
        ri, rw = ref_route(logits, bias, k, scores, groups, 1, True, 1.0)
        assert torch.equal(idx.long(), ri), sums
        close(w, rw, 400 * U32 * rw + 2.0 ** -126, "gate_w")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(600, 64), (600, 40), (8200, 64)])
def test_renormalised_sigmoids_far_from_one_another(dm, T, E):
    """Chosen sigmoids whose quotients fp32 holds while the smaller ones themselves are below what it holds in full."""
    k = 6
    logits = torch.full((T, E), -500.0, device="cuda")
    top = torch.linspace(-29.9, 3.0, T, device="cuda")
    logits[:, :k] = top[:, None] - torch.tensor([0.0, 30.0, 55.0, 62.0, 70.0, 80.0], device="cuda")
    idx, w = route(dm, logits, k, scores="sigmoid")
    ri, rw = ref_route(logits, None, k, "sigmoid", 1, 1, True, 1.0)
    assert torch.equal(idx.long(), ri)
    # exponentials of arguments without a rounding (2 ulp; twice the root's), a sum and a quotient
    close(w, rw, 40 * U32 * rw + 2.0 ** -126, "gate_w")
    d = randn(1, T, k, dtype=F32)
    dl = empty(T, E, dtype=F32)
    dm.route_balanced_backward(logits, idx, d, dl, scores="sigmoid")
    ref = ops.ref_route_backward(logits, ri, d, "sigmoid", True, 1.0)
    size = torch.zeros(T, E, device="cuda", dtype=torch.float64).scatter_(1, ri, rw * 2 * d.double().abs().amax(1, keepdim=True))
    close(dl, ref, 100 * U32 * size + 2.0 ** -126, "d_logits")


def test_route_refuses_outputs_over_its_inputs_without_gpu():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    L = m.lib()
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(5)]
    # logits, bias, T, E, k, scores, groups, top_groups, renormalize, scale, expert_idx, gate_w
    assert L.dmoe_route_balanced(p[0], p[1], 4, 8, 8, 1, 1, 1, 1, 1.0, p[2], p[0], None) == 1
    # logits, expert_idx, d_gate, T, E, k, scores, renormalize, scale, d_logits
    assert L.dmoe_route_balanced_backward(p[0], p[1], p[2], 4, 8, 8, 1, 1, 1.0, p[0], None) == 1
    assert L.dmoe_route_balanced_backward(p[0], p[1], p[2], 4, 8, 8, 1, 1, 1.0, p[2], None) == 1


@pytest.mark.gpu
def test_route_refuses_outputs_over_its_inputs(dm):
    """With as many choices as experts the weights have the logits' shape, and the gradients one another's."""
    T, E = 64, 8
    logits, idx, w = randn(1, T, E, dtype=F32), empty(T, E, dtype=I32), empty(T, E, dtype=F32)
    kept = logits.clone()
    with pytest.raises(ValueError, match="gate_w must not overlap logits"):
        dm.route_balanced(logits, E, idx, logits)
    both = empty(T * E + T * 2 - 4, dtype=F32)
    with pytest.raises(ValueError, match="gate_w must not overlap logits"):
        dm.route_balanced(both[:T * E].view(T, E), 2, idx.view(-1)[:2 * T].view(T, 2), both[T * E - 4:].view(T, 2))
    dm.route_balanced(logits, E, idx, w)
    d = randn(2, T, E, dtype=F32)
    for over in (d, logits):
        with pytest.raises(ValueError, match="d_logits must not overlap"):
            dm.route_balanced_backward(logits, idx, d, over)
    assert torch.equal(logits, kept)


# ----------------------------------------------------- norms around the block

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2])
def test_gradient_of_a_gate_a_row_needs_no_workspace(dm, T):
    """One row's gate is a gate of T rows, too: its gradient is written by the row, with no sums to bring together."""
    d = 264
    dy, u, h = randn(1, T, d), randn(2, T, d), randn(3, T, d, scale=3.0)
    a, b = weights(False, d)
    gate = torch.sigmoid(randn(9, T, dtype=F32))
    ru = torch.rsqrt(u.float().square().mean(1) + 1e-5)
    rh = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    got = {"du": empty(T, d), "dx": empty(T, d), "gate": empty(T, dtype=F32)}
    dm.sandwich_norm_backward(dy, u, h, a, b, ru, rh, got["du"], got["dx"], None, None, None, gate=gate, d_gate=got["gate"])
    ref, size = ref_sandwich_backward(dy, u, h, a, b, ru, rh, None, gate, 1.0)
    check_backward(got, ref, size, T)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(1000, 8200), (500, 12808), (700, 16384)])
@pytest.mark.parametrize("kind,wf32,scale,stream", [("row", True, 0.7, True), ("one", False, 1.0, False)])
def test_sandwich_norm_of_many_wide_rows(dm, T, d, kind, wf32, scale, stream):
    """Four vectors a thread, several rows a block: its ring filled again and again, of one stage at 16384 columns."""
    ops.test_sandwich_norm(dm, T, d, kind, wf32, scale)
    ops.test_sandwich_norm_backward(dm, T, d, kind, wf32, scale, stream)


# ------------------------------------------------------ a block's other parts

@pytest.mark.gpu
@pytest.mark.parametrize("has1,has2", [(False, False), (True, False), (False, True), (True, True)])
def test_shared_expert_makes_the_gradients_of_biases_it_has(dm, has1, has2):
    """One launch less for every bias that is not there, the other gradients bit for bit the same, and what was in db1 and db2 left
    there."""
    T, d, F = 70, 128, 520
    x, dy = randn(1, T, d), randn(2, T, d)
    w1, w2 = randn(3, d, F, scale=d ** -0.5), randn(4, F, d, scale=F ** -0.5)
    full, s = dm.SharedExpert(T, d, F), dm.SharedExpert(T, d, F)
    zero1, zero2 = torch.zeros(F, device="cuda"), torch.zeros(d, device="cuda")
    y = full.forward(x, w1, w2, zero1, zero2)
    n = launches(dm, lambda: full.backward(dy, x, w1, w2))
    assert float(s.db1.abs().sum() + s.db2.abs().sum()) == 0.0
    s.db1.fill_(7.0), s.db2.fill_(7.0)
    assert torch.equal(s.forward(x, w1, w2, zero1 if has1 else None, zero2 if has2 else None), y)
    assert launches(dm, lambda: s.backward(dy, x, w1, w2)) == n - (not has1) - (not has2)
    for name in ("dx", "dW1", "dW2"):
        assert torch.equal(getattr(s, name), getattr(full, name)), name
    assert torch.equal(s.db1, full.db1) if has1 else bool((s.db1 == 7.0).all())
    assert torch.equal(s.db2, full.db2) if has2 else bool((s.db2 == 7.0).all())


def test_layers_own_gate_and_its_limit(monkeypatch):
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    big = m.DMoELayer(64, 128, 320, 128, 2, device="cpu", balanced={})
    with pytest.raises(ValueError, match="256 experts, not 320"):
        big.forward_calls(None, None, None, None, w_gate=object())
    assert [n for n, _ in big.forward_calls(None, None, None, None)][:2] == ["route_balanced", "permute_pad"]
    # a balanced layer's gate makes logits: it chooses no more than it has to
    seen = []
    monkeypatch.setattr(m, "gate_route_topk", lambda x, w, k, renorm, logits, idx, gate: seen.append((k, idx.shape, gate.shape)))
    for balanced, k in (({}, 1), (None, 6)):
        layer = m.DMoELayer(64, 128, 16, 128, 6, device="cpu", balanced=balanced)
        dict(layer.forward_calls(None, None, None, None, w_gate=object()))["gate_route_topk"]()
        assert seen.pop() == (k, (64, k), (64, k))


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(8, 3), (64, 8)])
def test_balanced_layer_with_its_own_gate(dm, E, k):
    """The choice, weights and output of the same layer given the logits that the gate made."""
    T, d, F = 300, 128, 128
    x, wg = randn(1, T, d), randn(2, E, d, scale=d ** -0.5)
    w1, w2 = randn(3, d, E * F, scale=d ** -0.5), randn(4, E * F, d, scale=F ** -0.5)
    own, given = (dm.DMoELayer(T, d, E, F, k, "gelu", True, balanced={"scores": "sigmoid", "groups": 4, "top_groups": 2}) for _ in "ab")
    for layer in (own, given):
        layer.route_bias.copy_(torch.linspace(-0.2, 0.2, E, device="cuda"))
    own.forward(x, None, w1, w2, w_gate=wg)
    z = x.double() @ wg.double().t()
    close(own.gate_logits, z, 2 * d * U32 * (x.double().abs() @ wg.double().abs().t()), "logits")
    given.forward(x, own.gate_logits.clone(), w1, w2)
    for name in ("expert_idx", "gate_w", "tokens_per_expert", "y"):
        assert torch.equal(getattr(own, name), getattr(given, name)), name
