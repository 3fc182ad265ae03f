"""Balanced routing, the norms around a block and the dense linear layer,
against 64-bit references.

References are computed here, in float64, from the definitions in
``include/dmoe.h``.  Tolerances follow from the number formats: U16 = 2^-8 is
half a step of bf16, U32 = 2^-24 half a step of fp32, relative, and a sum of n
products in any order is off by at most about n U32 times the sum of their
magnitudes.
"""

import ctypes
import math

import pytest
import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -24
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    m.get_error(clear=True)
    yield m
    assert m.get_error(clear=True) == 0


def randn(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64) * scale).to(dtype)


def empty(*shape, dtype=BF):
    """Filled with a value that no result holds."""
    if dtype in (I32, U8):
        return torch.full(shape, 77, device="cuda", dtype=dtype)
    return torch.full(shape, 777.0, device="cuda", dtype=F32).to(dtype)


def workspace(n):
    """Bytes with a guard behind them."""
    t = torch.full((n + 256,), 0x5a, device="cuda", dtype=U8)
    return t[:max(n, 16)], t[max(n, 16):]


def close(got, ref, tol, what):
    got = got.detach().double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float(((got - ref).abs() - tol).max()):.3e} over its tolerance")


# -------------------------------------------------------------------- routing

def clean(logits):
    z = logits.double()
    return torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z.clamp(max=torch.finfo(F32).max))


def ref_scores(z, scores):
    if scores == "sigmoid":
        return torch.sigmoid(z)
    m = z.amax(1, keepdim=True)
    e = torch.where(z == -math.inf, torch.zeros_like(z), torch.exp(z - m))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def ref_route(logits, bias, k, scores, groups, top_groups, renorm, scale):
    z = clean(logits)
    T, E = z.shape
    s = ref_scores(z, scores)
    c = s if bias is None else s + bias.double()
    c = torch.where((z == -math.inf) | torch.isnan(c), torch.full_like(c, -math.inf), c)
    order = z if bias is None else c
    key = order.clone()
    left = torch.ones_like(z, dtype=torch.bool)
    if top_groups < groups:
        top = c.view(T, groups, E // groups).topk(min(2, E // groups), 2).values
        worth = torch.where(top[..., -1] == -math.inf, top[..., 0], top.sum(2))
        best = worth.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=z.device).scatter_(1, best, True)
        left = kept.repeat_interleave(E // groups, 1)
    # those of other groups behind all: by two stable sorts
    by_key = key.sort(dim=1, descending=True, stable=True).indices
    away = (~left).gather(1, by_key).int()
    idx = by_key.gather(1, away.sort(dim=1, stable=True).indices)[:, :k]
    if renorm:
        zc = z.gather(1, idx)
        ls = torch.nn.functional.logsigmoid(zc) if scores == "sigmoid" else zc
        top = ls.amax(1, keepdim=True)
        e = torch.where(ls == -math.inf, torch.zeros_like(ls), torch.exp(ls - top))
        w = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = s.gather(1, idx)
    return idx, w * scale


def ref_route_backward(logits, idx, d_gate, scores, renorm, scale):
    z = clean(logits).requires_grad_()
    zc = z.gather(1, idx)
    if renorm:
        w = torch.softmax(torch.nn.functional.logsigmoid(zc) if scores == "sigmoid" else zc, 1)
    else:
        w = torch.sigmoid(zc) if scores == "sigmoid" else torch.softmax(z, 1).gather(1, idx)
    (w * d_gate.double() * scale).sum().backward()
    return z.grad


def route(dm, logits, k, **kw):
    T = logits.shape[0]
    idx, w = empty(T, k, dtype=I32), empty(T, k, dtype=F32)
    dm.route_balanced(logits, k, idx, w, **kw)
    return idx, w


ROUTES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (5, 8, 2, 1, 1), (9, 31, 31, 1, 1), (130, 64, 1, 1, 1), (77, 66, 5, 3, 2),
    (1000, 256, 8, 8, 4), (513, 96, 6, 32, 5), (64, 40, 12, 20, 7), (33, 160, 6, 5, 1), (257, 512, 40, 16, 3),
    (17, 1024, 9, 1, 1), (12, 1024, 64, 32, 2), (11, 24, 3, 24, 5), (2049, 128, 8, 2, 1), (6, 7, 7, 7, 7),
    # four tokens a warp: one expert each, or many tokens
    (1, 64, 1, 1, 1), (7, 128, 1, 4, 2), (130, 256, 1, 8, 8), (33, 128, 1, 2, 1), (50, 256, 1, 2, 1), (8193, 64, 8, 2, 1),
    (8195, 128, 5, 4, 3), (9001, 256, 8, 8, 4), (8192, 256, 7, 4, 1), (8194, 256, 8, 1, 1), (8200, 64, 6, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,groups,top_groups", ROUTES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,renorm", [(False, False), (False, True), (True, False), (True, True)])
def test_route(dm, T, E, k, groups, top_groups, scores, biased, renorm):
    logits = randn(T + E, T, E, scale=1.5, dtype=F32)
    bias = randn(E, E, scale=0.05 if scores == "sigmoid" else 0.3 / E, dtype=F32) if biased else None
    kw = dict(scores=scores, groups=groups, top_groups=top_groups, scale=2.5)
    idx, w = route(dm, logits, k, bias=bias, renormalize=renorm, **kw)
    ri, rw = ref_route(logits, bias, k, scores, groups, top_groups, renorm, 2.5)
    assert torch.equal(idx.long(), ri)
    # expf (2 ulp), its argument's rounding (|z| up to 12), a sum of up to E, quotient, scale
    e = (2 * 12 + E / 32 + k + 16) * U32
    close(w, rw, 2 * e * rw, "gate_w")
    d_gate = randn(3, T, k, dtype=F32)
    dl = empty(T, E, dtype=F32)
    dm.route_balanced_backward(logits, idx, d_gate, dl, scores=scores, renormalize=renorm, scale=2.5)
    rd = ref_route_backward(logits, ri, d_gate, scores, renorm, 2.5)
    # a weight times differences of what arrives
    size = 2.5 * ref_scores(clean(logits), scores) * 2 * d_gate.double().abs().sum(1, keepdim=True)
    if renorm:
        size = torch.full_like(size, 0.0).scatter_(1, ri, rw * 2 * d_gate.double().abs().amax(1, keepdim=True))
    close(dl, rd, 4 * e * size + 1e-30, "d_logits")


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
def test_route_where_32_bits_cannot_tell(dm, scores, groups, top_groups):
    """A bias that levels one row's choices to within an ulp: 64 bits decide."""
    T, E, k = 300, 256, 8
    row = randn(1, 1, E, dtype=F32)
    level = ref_scores(row.double(), scores)[0]
    bias = (0.5 - level).to(F32)
    logits = row.repeat(T, 1)
    logits += randn(2, T, E, scale=1e-7, dtype=F32)
    idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=top_groups)
    ri, rw = ref_route(logits, bias, k, scores, groups, top_groups, True, 1.0)
    c = ref_scores(logits.double(), scores) + bias.double()
    assert float((c.amax(1) - c.amin(1)).max()) < 1e-6
    # candidates whose 64-bit values lie within a few of their own roundings may
    # come in either order: their values must then agree that closely
    got, want = c.gather(1, idx.long()), c.gather(1, ri)
    if groups == 1:
        assert float((got - want).abs().max()) < 1e-14
    assert float((idx.long() != ri).any(1).double().mean()) < 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,biased", [(1, 1, False), (1, 1, True), (8, 3, True), (8, 3, False)])
def test_route_of_many_tokens_with_open_orders(dm, scores, groups, top_groups, biased):
    """A batch large enough for four tokens a warp, in which rows with ties, masks and extremes lie between usual ones."""
    T, E, k = 8300, 256, 8
    logits = randn(1, T, E, dtype=F32)
    bias = randn(2, E, scale=0.02, dtype=F32) if biased else None
    logits[::7] = 0.0                                             # padding
    logits[3::11] = (torch.arange(E, device="cuda") % 5).float()  # ties all over
    logits[5::13, 9:] = -math.inf                                 # few experts left, one of them twice
    logits[6::17, ::2] = -math.inf
    logits[8::19] = math.nan
    logits[9::23] *= 1e20
    if biased:
        logits[2::29] = torch.logit(((0.5 - bias).double()).clamp(1e-3, 1 - 1e-3)).to(F32)  # sigmoids level with the bias
    idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=top_groups)
    ri, rw = ref_route(logits, bias, k, scores, groups, top_groups, True, 1.0)
    same = (idx.long() == ri).all(1)
    level = torch.zeros(T, dtype=torch.bool, device="cuda")
    if biased:
        level[2::29] = True
    # everywhere but in the levelled rows, whose 64-bit values differ by their own roundings
    assert bool(same[~level].all())
    assert float(same[level].double().mean()) > 0.9 if biased else True
    close(w[same], rw[same], 400 * U32 * rw[same] + 2.0 ** -126, "gate_w")


@pytest.mark.gpu
def test_route_ties_go_to_the_lower_expert(dm):
    T, E = 40, 64
    logits = torch.zeros(T, E, device="cuda")
    logits[1::2] = (torch.arange(E, device="cuda") % 4).float()
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.25, device="cuda")):
        for scores in ("softmax", "sigmoid"):
            for groups, top in ((1, 1), (16, 5)):
                idx, w = route(dm, logits, 6, bias=bias, scores=scores, groups=groups, top_groups=top)
                ri, rw = ref_route(logits, bias, 6, scores, groups, top, True, 1.0)
                assert torch.equal(idx.long(), ri)
                close(w, rw, 64 * U32 * rw, "gate_w")
    assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_route_masked_and_extreme_logits(dm, scores, renorm, biased, groups, top_groups):
    E, k = 16, 6
    top = torch.finfo(F32).max
    inf = math.inf
    # (a bias of plus infinity forces its expert, one of minus infinity or NaN rules it out)
    rows = [[-inf] * E, [float("nan")] * E, [0.0] + [-inf] * 15, [-inf] * 14 + [1.0, 2.0], [-top] * E,
            [top] * 3 + [-top] * 13, [inf] + [1.0] * 15, [float("nan"), 3.0] * 8, [-200.0 - i for i in range(E)],
            [-100.0 + 3 * i for i in range(E)], [300.0 - i for i in range(E)], [-0.0, 0.0] * 8,
            [-inf, -3.0, -inf, 2.0] * 4]
    logits = torch.tensor(rows, device="cuda")
    bias = torch.tensor([0.01 * (i % 5) for i in range(E)], device="cuda") if biased else None
    if biased:
        bias[3], bias[7], bias[9] = -inf, float("nan"), inf
    idx, w = route(dm, logits, k, bias=bias, scores=scores, groups=groups, top_groups=top_groups, renormalize=renorm)
    ri, rw = ref_route(logits, bias, k, scores, groups, top_groups, renorm, 1.0)
    assert torch.equal(idx.long(), ri)
    # the argument of an exponential of up to 300 is rounded, too
    close(w, rw, 400 * U32 * rw + 2.0 ** -126, "gate_w")
    dl = empty(len(rows), E, dtype=F32)
    dm.route_balanced_backward(logits, idx, torch.ones_like(w), dl, scores=scores, renormalize=renorm)
    assert bool(torch.isfinite(dl).all())
    assert float(dl[0].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(dm, scores, renorm):
    T, E, k = 6, 32, 4
    logits = randn(5, T, E, dtype=F32)
    idx, _ = route(dm, logits, k, scores=scores, renormalize=renorm)
    d = randn(6, T, k, dtype=F32)
    dl = empty(T, E, dtype=F32)
    dm.route_balanced_backward(logits, idx, d, dl, scores=scores, renormalize=renorm)
    z, i = logits.double(), idx.long()

    def f(z):
        s = ref_scores(z, scores).gather(1, i)
        return (d.double() * (s / s.sum(1, keepdim=True) if renorm else s)).sum(1)

    for e in range(E):
        step = torch.zeros_like(z)
        step[:, e] = 1e-5
        num = (f(z + step) - f(z - step)) / 2e-5
        close(dl[:, e], num, 1e-6, f"expert {e}")


@pytest.mark.gpu
def test_route_in_a_graph_on_another_stream_and_nothing(dm):
    logits = randn(1, 100, 64, dtype=F32)
    bias = randn(2, 64, scale=0.01, dtype=F32)
    idx, w = empty(100, 4, dtype=I32), empty(100, 4, dtype=F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dm.route_balanced(logits, 4, idx, w, bias=bias, scores="sigmoid", groups=4, top_groups=2)
    s.synchronize()
    want = idx.clone(), w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dm.route_balanced(logits, 4, idx, w, bias=bias, scores="sigmoid", groups=4, top_groups=2)
    idx.fill_(7), w.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    e = torch.empty(0, 64, device="cuda")
    dm.route_balanced(e, 4, empty(0, 4, dtype=I32), empty(0, 4, dtype=F32))
    dm.route_balanced_backward(e, empty(0, 4, dtype=I32), empty(0, 4, dtype=F32), e)


@pytest.mark.gpu
def test_route_backward_reports_an_expert_out_of_range(dm):
    logits = randn(1, 3, 8, dtype=F32)
    idx = torch.tensor([[0, 1], [8, 2], [-1, 3]], dtype=I32, device="cuda")
    dl = empty(3, 8, dtype=F32)
    dm.route_balanced_backward(logits, idx, torch.ones(3, 2, device="cuda"), dl, scores="sigmoid", renormalize=False)
    assert dm.get_error(clear=True) == (5 << 8 | 5)
    assert bool((dl[1] != 0).nonzero().view(-1).tolist() == [2]) and bool((dl[2] != 0).nonzero().view(-1).tolist() == [3])


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 5, 64, 1000])
def test_balance_bias(dm, E):
    load = torch.randint(0, 50, (E,), device="cuda", dtype=I32)
    bias = randn(1, E, dtype=F32)
    want = bias + 0.001 * torch.sign(load.double().mean() - load.double()).to(F32)
    dm.balance_bias(bias, load, 0.001)
    assert torch.equal(bias, want)


# ----------------------------------------------------- norms around the block

SIZES = [(1, 8), (3, 24), (5, 136), (17, 520), (130, 1000), (7, 3584), (2, 4096), (5, 4104), (3, 8200), (2, 16384),
         (1030, 256), (700, 2056)]


def gate_of(kind, T):
    return None if kind == "none" else torch.sigmoid(randn(9, T if kind == "row" else 1, dtype=F32))


def ref_sandwich(u, x, a, b, gate, scale, eps):
    g = torch.ones(1, device="cuda", dtype=torch.float64) if gate is None else gate.double()
    ud, a, b = u.double(), a.double(), b.double()
    ru = 1.0 / torch.sqrt((ud * ud).mean(1) + eps)
    n = ud * (ru * g)[:, None] * a
    return ru, scale * x.double() + n, abs(scale) * x.double().abs() + n.abs()


def weights(wf32, d):
    dt = F32 if wf32 else BF
    return randn(3, d, scale=0.3, dtype=dt) + 1, randn(4, d, scale=0.3, dtype=dt) + 1


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("kind,wf32,scale", [("none", False, 1.0), ("row", True, 0.7), ("one", False, -0.5)])
def test_sandwich_norm(dm, T, d, kind, wf32, scale):
    eps = 1e-5
    u, x = randn(1, T, d, scale=0.5), randn(2, T, d, scale=3.0)
    a, b = weights(wf32, d)
    gate = gate_of(kind, T)
    h, y, ru, rh = empty(T, d), empty(T, d), empty(T, dtype=F32), empty(T, dtype=F32)
    dm.sandwich_norm(u, x, a, b, eps, h, y, gate=gate, scale=scale, rstd_u=ru, rstd_h=rh)
    rr, hr, size = ref_sandwich(u, x, a, b, gate, scale, eps)
    e = 80 * U32  # a thread's up to 32 squares, shuffles and warps, mean and root
    close(ru, rr, e * rr, "rstd_u")
    close(h, hr, U16 * hr.abs() + 2 * e * size, "h")
    hd = h.double()  # the norm reads the kept value
    rhr = 1.0 / torch.sqrt((hd * hd).mean(1) + eps)
    yr = hd * rhr[:, None] * b.double()
    close(rh, rhr, e * rhr, "rstd_h")
    close(y, yr, (U16 + 2 * e) * yr.abs(), "y")


def ref_sandwich_backward(dy, u, h, a, b, ru, rh, dh, gate, scale):
    dy, u, h, a, b = (t.double() for t in (dy, u, h, a, b))
    ru, rh = ru.double()[:, None], rh.double()[:, None]
    dh = torch.zeros_like(u) if dh is None else dh.double()
    g = torch.ones(1, 1, device="cuda", dtype=torch.float64) if gate is None else gate.double()[:, None]
    gy = dy * b
    dH = dh + rh * (gy - h * rh ** 2 * (gy * h).mean(1, keepdim=True))
    SH = dh.abs() + rh * (gy.abs() + h.abs() * rh ** 2 * (gy * h).abs().mean(1, keepdim=True))
    along, S_along = ru * (a * dH * u).sum(1, keepdim=True), ru * (a.abs() * SH * u.abs()).sum(1, keepdim=True)
    du = g * ru * (a * dH - u * ru * along / u.shape[1])
    S_du = g * ru * (a.abs() * SH + u.abs() * ru * S_along / u.shape[1])
    ref = {"du": du, "dx": scale * dH, "da": (g * ru * dH * u).sum(0), "db": (rh * dy * h).sum(0)}
    size = {"du": S_du, "dx": abs(scale) * SH, "da": (g * ru * SH * u.abs()).sum(0), "db": (rh * dy * h).abs().sum(0)}
    if gate is not None:
        one = gate.shape[0] == 1
        ref["gate"] = along.sum().view(1) if one else along.view(-1)
        size["gate"] = S_along.sum().view(1) if one else S_along.view(-1)
    return ref, size


def check_backward(got, ref, size, T):
    e = 120 * U32  # three sums of a row, as above, and their combination
    for n in ("du", "dx"):
        close(got[n], ref[n], U16 * ref[n].abs() + e * size[n], n)
    for n in ("da", "db", "gate"):
        if n in ref and got.get(n) is not None:
            close(got[n], ref[n], (e + T * U32) * size[n], n)


WIDTHS = [512, 520, 1024, 1032, 1536, 1544, 2048, 2056, 2560, 2568, 3064, 3080, 4096, 4104, 5120, 5128, 6144, 6152, 8192]


@pytest.mark.gpu
@pytest.mark.parametrize("d", WIDTHS)
def test_sandwich_norm_on_both_sides_of_every_width(dm, d):
    for T, kind, wf32, scale in ((9, "row", False, 0.7), (160, "one", True, 1.0)):
        test_sandwich_norm(dm, T, d, kind, wf32, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", SIZES + [(3001, 72)])
@pytest.mark.parametrize("kind,wf32,scale,stream", [("none", False, 1.0, True), ("row", True, 0.7, False),
                                                    ("one", False, -0.5, True)])
def test_sandwich_norm_backward(dm, T, d, kind, wf32, scale, stream):
    dy, u, h = randn(1, T, d), randn(2, T, d, scale=0.5), randn(5, T, d, scale=3.0)
    dh = randn(6, T, d) if stream else None
    a, b = weights(wf32, d)
    gate = gate_of(kind, T)
    ru = torch.rsqrt(u.float().square().mean(1) + 1e-5)
    rh = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    got = {"du": empty(T, d), "dx": empty(T, d), "da": empty(d, dtype=F32), "db": empty(d, dtype=F32)}
    if gate is not None:
        got["gate"] = empty(gate.shape[0], dtype=F32)
    ws, guard = workspace(dm.sandwich_norm_backward_workspace_size(T, d))
    dm.sandwich_norm_backward(dy, u, h, a, b, ru, rh, got["du"], got["dx"], got["da"], got["db"], ws, dh=dh, gate=gate,
                              d_gate=got.get("gate"), scale=scale)
    ref, size = ref_sandwich_backward(dy, u, h, a, b, ru, rh, dh, gate, scale)
    check_backward(got, ref, size, T)
    assert bool((guard == 0x5a).all())
    again = {n: t.clone() for n, t in got.items()}
    dm.sandwich_norm_backward(dy, u, h, a, b, ru, rh, got["du"], got["dx"], got["da"], got["db"], ws, dh=dh, gate=gate,
                              d_gate=got.get("gate"), scale=scale)
    for n in got:
        assert torch.equal(got[n], again[n]), n  # the same sums in the same order


@pytest.mark.gpu
@pytest.mark.parametrize("d", WIDTHS)
def test_sandwich_norm_backward_on_both_sides_of_every_width(dm, d):
    for T, kind, wf32, scale, stream in ((9, "row", False, 0.7, True), (1600, "one", True, 1.0, False)):
        test_sandwich_norm_backward(dm, T, d, kind, wf32, scale, stream)


@pytest.mark.gpu
def test_sandwich_norm_against_differences(dm):
    """The backward against differences of the 64-bit forward (its h unrounded)."""
    T, d, eps, scale = 4, 40, 1e-5, 0.8
    u, x, dy, dh = randn(1, T, d), randn(2, T, d), randn(3, T, d), randn(4, T, d)
    a, b = weights(True, d)
    gate = gate_of("row", T)

    def f(u, x, a, b, gate):
        ru = 1.0 / torch.sqrt((u * u).mean(1) + eps)
        h = scale * x + u * (ru * gate)[:, None] * a
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * b
        return float((dy.double() * y + dh.double() * h).sum())

    p = [t.double() for t in (u, x, a, b, gate)]
    h, y = empty(T, d), empty(T, d)
    ru, rh = empty(T, dtype=F32), empty(T, dtype=F32)
    dm.sandwich_norm(u, x, a, b, eps, h, y, gate=gate, scale=scale, rstd_u=ru, rstd_h=rh)
    out = [empty(T, d), empty(T, d), empty(d, dtype=F32), empty(d, dtype=F32), empty(T, dtype=F32)]
    ws, _ = workspace(dm.sandwich_norm_backward_workspace_size(T, d))
    dm.sandwich_norm_backward(dy, u, h, a, b, ru, rh, *out[:4], ws, dh=dh, gate=gate, d_gate=out[4], scale=scale)
    for i, o in enumerate(out):
        for at in ([(0, 0), (1, 7), (3, 39)] if o.dim() == 2 else [(0,), (3,)]):
            q = [t.clone() for t in p]
            q[i][at] += 1e-5
            r = [t.clone() for t in p]
            r[i][at] -= 1e-5
            num = (f(*q) - f(*r)) / 2e-5
            # h is kept in bf16: every element of a row's gradient moves by up to
            # U16 of the row's terms; those of d elements and a few rows
            assert abs(float(o[at]) - num) <= 8 * U16 * max(1.0, abs(num)) * 2, (i, at)


@pytest.mark.gpu
def test_sandwich_norm_strides_in_place_and_other_stream(dm):
    T, d = 33, 264
    a, b = weights(False, d)
    u, x = randn(1, T, d), randn(2, T, d)
    h, y = empty(T, d), empty(T, d)
    dm.sandwich_norm(u, x, a, b, 1e-5, h, y)
    wide = empty(T, 3 * d)
    wide[:, d:2 * d], wide[:, 2 * d:] = u, x
    u2, x2 = wide[:, d:2 * d], wide[:, 2 * d:]
    h2, y2 = empty(T, d), empty(T, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dm.sandwich_norm(u2, x2, a, b, 1e-5, h2, y2)
    s.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)
    u3, x3 = u.clone(), x.clone()
    dm.sandwich_norm(u3, x3, a, b, 1e-5, x3, u3)  # h over the stream, y over the block's output
    assert torch.equal(h, x3) and torch.equal(y, u3)
    # backward: dy, u and dh as slices, and in place
    ru = torch.rsqrt(u.float().square().mean(1) + 1e-5)
    rh = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    dy, dh = randn(3, T, d), randn(4, T, d)
    ws, _ = workspace(dm.sandwich_norm_backward_workspace_size(T, d))
    du, dx, da, db = empty(T, d), empty(T, d), empty(d, dtype=F32), empty(d, dtype=F32)
    dm.sandwich_norm_backward(dy, u, h, a, b, ru, rh, du, dx, da, db, ws, dh=dh)
    wide[:, :d], wide[:, d:2 * d], wide[:, 2 * d:] = dy, u, dh
    du2, dx2, da2, db2 = empty(T, d), empty(T, d), empty(d, dtype=F32), empty(d, dtype=F32)
    dm.sandwich_norm_backward(wide[:, :d], wide[:, d:2 * d], h, a, b, ru, rh, du2, dx2, da2, db2, ws, dh=wide[:, 2 * d:])
    assert all(torch.equal(p, q) for p, q in ((du, du2), (dx, dx2), (da, da2), (db, db2)))
    dy3, dh3 = dy.clone(), dh.clone()
    dm.sandwich_norm_backward(dy3, u, h, a, b, ru, rh, dy3, dh3, None, None, None, dh=dh3)
    assert torch.equal(du, dy3) and torch.equal(dx, dh3)


@pytest.mark.gpu
def test_sandwich_norm_non_finite_rows_stay_apart_and_no_rows(dm):
    T, d = 9, 512
    a, b = weights(False, d)
    u, x = randn(1, T, d), randn(2, T, d)
    u[3, 5], x[6, 100] = math.inf, math.nan
    h, y = empty(T, d), empty(T, d)
    dm.sandwich_norm(u, x, a, b, 1e-5, h, y)
    ok = [i for i in range(T) if i not in (3, 6)]
    assert bool(torch.isfinite(y[ok]).all()) and not bool(torch.isfinite(y[3]).all())
    zero = torch.zeros(2, d, device="cuda", dtype=BF)
    dm.sandwich_norm(zero, zero, a, b, 1e-5, h[:2], y[:2])
    assert float(y[:2].abs().max()) == 0.0
    e = torch.empty(0, d, device="cuda", dtype=BF)
    f = torch.empty(0, device="cuda")
    dm.sandwich_norm(e, e, a, b, 1e-5, e.clone(), e.clone())
    da, db, dg = empty(d, dtype=F32), empty(d, dtype=F32), empty(1, dtype=F32)
    ws, _ = workspace(dm.sandwich_norm_backward_workspace_size(0, d))
    dm.sandwich_norm_backward(e, e, e, a, b, f, f, e.clone(), e.clone(), da, db, ws, gate=torch.ones(1, device="cuda"),
                              d_gate=dg)
    assert float(da.abs().sum() + db.abs().sum() + dg.abs().sum()) == 0.0


# --------------------------------------------------------------- dense linear

def ref_act(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


def check_linear(dm, M, K, N, act, bias, residual, x=None):
    x = randn(1, M, K) if x is None else x
    w = randn(2, K, N, scale=K ** -0.5)
    b = None if bias is None else randn(3, N, scale=0.3, dtype=bias)
    r = randn(4, M, N) if residual else None
    y = empty(M, N)
    f = None if act == "none" else empty(M, N)
    ws, guard = workspace(dm.linear_workspace_size(M, K, N))
    dm.linear(x, w, y, ws, bias=b, act=act, deriv=f, residual=r)
    z = x.double() @ w.double()
    S = x.double().abs() @ w.double().abs()
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    yr, fr = ref_act(z, act)
    if r is not None:
        yr = yr + r.double()
    # fp32 sums of K products, where the tensor cores truncate; the second
    # derivatives stay below 0.8; Phi is known to 1.5e-7, sigmoid to a few ulp
    ez = 2 * (K + 8) * U32 * S
    ea = 0.0 if act == "none" else 4e-7 * (1 + z.abs())
    close(y, yr, U16 * yr.abs() + 1.2 * ez + ea + 4 * U32 * (yr.abs() + 4), "y")
    if f is not None:
        close(f, fr, U16 * fr.abs() + 0.8 * ez + ea, "deriv")
    assert bool((guard == 0x5a).all())


LINEAR = [(1, 8, 8), (1, 4096, 1024), (7, 72, 136), (16, 2048, 520), (3, 8200, 1000), (17, 4104, 2056), (33, 2048, 1032),
          (64, 4096, 4096), (65, 4096, 264), (128, 520, 264), (130, 1032, 2056), (257, 64, 1000),
          (600, 264, 8), (1000, 8, 600), (513, 4096, 512), (2560, 512, 4096), (1031, 1000, 5128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("act,bias,residual", [("none", None, False), ("none", BF, True), ("gelu", F32, False),
                                               ("silu", BF, True)])
def test_linear(dm, M, K, N, act, bias, residual):
    check_linear(dm, M, K, N, act, bias, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(200, 264, 8192), (600, 512, 2048), (1000, 520, 2056), (2000, 512, 2048), (5999, 72, 520)])
@pytest.mark.parametrize("act,bias,residual", [("none", BF, True), ("gelu", F32, True)])
def test_linear_of_many_small_tiles(dm, M, K, N, act, bias, residual):
    check_linear(dm, M, K, N, act, bias, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("kept,f32", [(False, False), (True, True)])
def test_linear_backward(dm, M, K, N, kept, f32):
    dy, x, w = randn(1, M, N), randn(2, M, K), randn(3, K, N, scale=K ** -0.5)
    deriv = randn(4, M, N, scale=0.5) if kept else None
    factor = randn(5, M, K, scale=0.5) if kept else None
    dx, dw, db = empty(M, K), empty(K, N, dtype=F32 if f32 else BF), empty(N, dtype=F32)
    ws, guard = workspace(dm.linear_backward_workspace_size(M, K, N))
    dm.linear_backward(dy, x, w, dx, dw, ws, deriv=deriv, dbias=db, factor=factor)
    prod = dy.double() * (1.0 if deriv is None else deriv.double())
    dz = prod.to(F32).to(BF).double()  # products of bf16 values are exact in fp32: dz has these bits
    f = 1.0 if factor is None else factor.double()
    ref, S = (dz @ w.double().t()) * f, (dz.abs() @ w.double().abs().t()) * (1.0 if factor is None else f.abs())
    close(dx, ref, U16 * ref.abs() + 2 * (N + 8) * U32 * S, "dx")
    ref, S = x.double().t() @ dz, x.double().abs().t() @ dz.abs()
    close(dw, ref, (0 if f32 else U16) * ref.abs() + 2 * (M + 8) * U32 * S, "dw")
    close(db, prod.sum(0), (M + 8) * U32 * prod.abs().sum(0), "dbias")
    assert bool((guard == 0x5a).all())
    # one at a time, with the same results
    for want in ("dx", "dw", "db"):
        o = {"dx": torch.empty_like(dx), "dw": torch.empty_like(dw), "db": torch.empty_like(db)}
        dm.linear_backward(dy, x if want == "dw" else None, w, o["dx"] if want == "dx" else None,
                           o["dw"] if want == "dw" else None, ws, deriv=deriv, dbias=o["db"] if want == "db" else None,
                           factor=factor if want == "dx" else None)
        if want == "db":
            assert torch.equal(o["db"], db)
        else:  # alone they may be cut otherwise, which only changes the order of fp32 sums
            got, both = o[want].double(), {"dx": dx, "dw": dw}[want].double()
            assert float((got - both).norm()) <= 2 * U16 * float(both.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(8, 264, 4104), (64, 512, 2048), (64, 2048, 136), (129, 136, 4096), (300, 1000, 1000),
                                   (200, 64, 64), (512, 2048, 512), (1023, 72, 520), (260, 72, 8200)])
@pytest.mark.parametrize("kept,f32", [(False, True), (True, False)])
def test_linear_backward_of_small_products(dm, M, K, N, kept, f32):
    """One of the two sums much shorter than the other, and blocks of rows and of columns that are not whole."""
    test_linear_backward(dm, M, K, N, kept, f32)


@pytest.mark.gpu
def test_linear_against_differences(dm):
    M, K, N = 6, 24, 16
    for act in ("gelu", "silu"):
        x, w, b, dy = randn(1, M, K), randn(2, K, N, scale=K ** -0.5), randn(3, N, dtype=F32), randn(4, M, N)
        y, f = empty(M, N), empty(M, N)
        ws, _ = workspace(max(dm.linear_workspace_size(M, K, N), dm.linear_backward_workspace_size(M, K, N)))
        dm.linear(x, w, y, ws, bias=b, act=act, deriv=f)
        out = [empty(M, K), empty(K, N, dtype=F32), empty(N, dtype=F32)]
        dm.linear_backward(dy, x, w, out[0], out[1], ws, deriv=f, dbias=out[2])
        p = [t.double() for t in (x, w, b)]

        def loss(x, w, b):
            return float((dy.double() * ref_act(x @ w + b, act)[0]).sum())

        for i, o in enumerate(out):
            for at in ([(0, 0), (5, 7)] if o.dim() == 2 else [(0,), (15,)]):
                q, r = [t.clone() for t in p], [t.clone() for t in p]
                q[i][at] += 1e-5
                r[i][at] -= 1e-5
                num = (loss(*q) - loss(*r)) / 2e-5
                # deriv, dz and dx are rounded to bf16: three half steps of up to 24 terms of about 1
                assert abs(float(o[at]) - num) <= 3 * U16 * 12, (act, i, at)


@pytest.mark.gpu
def test_linear_strides_in_place_graph_and_no_rows(dm):
    M, K, N = 70, 264, 520
    x, w, r = randn(1, M, K), randn(2, K, N, scale=K ** -0.5), randn(3, M, N)
    ws, _ = workspace(max(dm.linear_workspace_size(M, K, N), dm.linear_backward_workspace_size(M, K, N)))
    y = empty(M, N)
    dm.linear(x, w, y, ws, residual=r)
    wide = randn(9, M, K + N + 8)
    wide[:, 8:8 + K], wide[:, 8 + K:] = x, r
    y2 = empty(M, N)
    dm.linear(wide[:, 8:8 + K], w, y2, ws, residual=wide[:, 8 + K:])
    assert torch.equal(y, y2)
    r3 = r.clone()
    dm.linear(x, w, r3, ws, residual=r3)
    assert torch.equal(y, r3)
    g = torch.cuda.CUDAGraph()
    y4 = empty(M, N)
    with torch.cuda.graph(g):
        dm.linear(x, w, y4, ws, residual=r)
    g.replay()
    assert torch.equal(y, y4)
    x.copy_(randn(5, M, K))
    g.replay()
    dm.linear(x, w, y, ws, residual=r)
    assert torch.equal(y, y4)
    # backward of slices, dx over its factor
    dy, f = randn(6, M, N), randn(7, M, K)
    dx, dw = empty(M, K), empty(K, N)
    dm.linear_backward(dy, x, w, dx, dw, ws, factor=f)
    wide[:, 8:8 + K], wide[:, 8 + K:] = x, dy
    dw2 = empty(K, N)
    dm.linear_backward(wide[:, 8 + K:], wide[:, 8:8 + K], w, f, dw2, ws, factor=f)
    assert torch.equal(dx, f) and torch.equal(dw, dw2)
    e = torch.empty(0, K, device="cuda", dtype=BF)
    z = torch.empty(0, N, device="cuda", dtype=BF)
    dm.linear(e, w, z, ws)
    db = empty(N, dtype=F32)
    dm.linear_backward(z, e, w, e.clone(), dw, ws, dbias=db)
    assert float(dw.abs().sum()) == 0.0 and float(db.abs().sum()) == 0.0


@pytest.mark.gpu
def test_linear_workspace_of_the_longest_serves_the_shorter(dm):
    K, N = 4096, 512
    ws, guard = workspace(dm.linear_workspace_size(512, K, N))
    w = randn(2, K, N, scale=K ** -0.5)
    for M in (1, 9, 64, 129, 200, 257, 384, 512):
        assert dm.linear_workspace_size(M, K, N) <= ws.numel()
        x, y = randn(M, M, K), empty(M, N)
        dm.linear(x, w, y, ws)
        ref = x.double() @ w.double()
        S = x.double().abs() @ w.double().abs()
        close(y, ref, U16 * ref.abs() + 2 * (K + 8) * U32 * S, f"y of {M}")
    assert bool((guard == 0x5a).all())


@pytest.mark.gpu
def test_linear_rows_that_are_not_finite_stay_apart(dm):
    M, K, N = 200, 136, 264
    x, w = randn(1, M, K), randn(2, K, N)
    x[7, 3], x[150, 0] = math.nan, math.inf
    y = empty(M, N)
    ws, _ = workspace(dm.linear_workspace_size(M, K, N))
    dm.linear(x, w, y, ws)
    ok = torch.ones(M, dtype=torch.bool, device="cuda")
    ok[7] = ok[150] = False
    assert bool(torch.isfinite(y[ok]).all()) and not bool(torch.isfinite(y[~ok]).any())


# ------------------------------------------------------------------- refusals

def test_refusals_without_gpu():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    L = m.lib()
    p, odd, s = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002), None
    nan = float("nan")

    def refused(f, args, changes):
        for at, bad in changes:
            a = list(args)
            a[at] = bad
            assert f(*a) == 1, (f.__name__, at, bad)

    # logits, bias, T, E, k, scores, groups, top_groups, renormalize, scale, expert_idx, gate_w
    refused(L.dmoe_route_balanced, [p, p, 4, 64, 8, 1, 8, 4, 1, 1.0, p, p, s],
            [(0, None), (0, odd), (1, odd), (2, -1), (3, 0), (3, 1025), (3, 65), (4, 0), (4, 33), (5, 2), (5, -1), (6, 0),
             (6, 64), (6, 7), (7, 0), (7, 9), (9, nan), (9, math.inf), (10, None), (10, odd), (11, None), (11, odd)])
    # logits, expert_idx, d_gate, T, E, k, scores, renormalize, scale, d_logits
    refused(L.dmoe_route_balanced_backward, [p, p, p, 4, 64, 8, 1, 1, 1.0, p, s],
            [(0, None), (1, None), (2, None), (9, None), (0, odd), (1, odd), (2, odd), (9, odd), (3, -1), (4, 0),
             (4, 1025), (5, 0), (5, 65), (6, 2), (8, nan)])
    refused(L.dmoe_balance_bias, [p, p, 64, 0.1, s], [(0, None), (1, None), (0, odd), (1, odd), (2, 0), (2, 1025), (3, nan)])
    # u, ldu, residual, ldr, w_post, w_pre, f32, gate, gate_rows, scale, eps, T, d, h, y, rstd_u, rstd_h
    q = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]
    refused(L.dmoe_sandwich_norm, [q[0], 64, q[1], 64, q[2], q[3], 0, q[4], 4, 1.0, 1e-5, 4, 64, q[5], q[6], q[7], q[8], s],
            [(0, None), (2, None), (4, None), (5, None), (13, None), (14, None), (14, q[5]), (0, odd), (2, odd), (4, odd),
             (5, odd), (7, odd), (13, odd), (14, odd), (15, odd), (16, odd), (1, 56), (1, 68), (3, 56), (3, 68), (8, 3),
             (8, 0), (10, -1.0), (10, nan), (11, -1), (12, 0), (12, 60), (12, 16392)])
    assert L.dmoe_sandwich_norm(q[0], 72, q[1], 64, q[2], q[3], 0, None, 0, 1.0, 1e-5, 4, 64, q[0], q[6], None, None, s) == 1
    # dy, lddy, u, ldu, h, w_post, w_pre, f32, gate, gate_rows, scale, rstd_u, rstd_h, dh, lddh, T, d, du, dx, dw_post,
    # dw_pre, d_gate, ws, ws_bytes
    args = [q[0], 64, q[1], 64, q[2], q[3], q[3], 0, q[4], 4, 1.0, q[5], q[5], q[6], 64, 4, 64, q[7], q[8], q[9], q[9], q[10],
            q[11], 1 << 24, s]
    refused(L.dmoe_sandwich_norm_backward, args,
            [(i, None) for i in (0, 2, 4, 5, 6, 11, 12, 17, 18)] + [(i, odd) for i in (0, 2, 4, 5, 6, 8, 11, 12, 13, 17, 18,
                                                                                      19, 20, 21, 22)]
            + [(8, None), (18, q[7]), (1, 56), (3, 68), (14, 60), (9, 3), (15, -1), (16, 12), (16, 16392)])
    a = list(args)
    a[14], a[18] = 72, q[6]  # over rows of another pitch
    assert L.dmoe_sandwich_norm_backward(*a) == 1
    # x, ldx, w, bias, f32, act, residual, ldr, M, K, N, y, deriv, ws, ws_bytes
    refused(L.dmoe_linear, [q[0], 64, q[1], q[2], 0, 1, q[3], 128, 4, 64, 128, q[4], q[5], q[6], 1 << 30, s],
            [(0, None), (2, None), (11, None), (0, odd), (2, odd), (3, odd), (6, odd), (11, odd), (12, odd), (13, odd),
             (1, 56), (1, 68), (7, 120), (7, 132), (5, 3), (5, -1), (5, 0), (8, -1), (9, 4), (9, 60), (10, 0), (10, 100),
             (11, q[0]), (11, q[1]), (11, q[5])])
    # dy, lddy, deriv, x, ldx, w, factor, M, K, N, dx, dw, f32, dbias, ws, ws_bytes
    refused(L.dmoe_linear_backward, [q[0], 128, q[1], q[2], 64, q[3], q[4], 4, 64, 128, q[5], q[6], 0, q[7], q[8], 1 << 30, s],
            [(0, None), (3, None), (5, None), (10, None), (0, odd), (2, odd), (3, odd), (5, odd), (6, odd), (10, odd),
             (11, odd), (13, odd), (14, odd), (1, 120), (1, 132), (4, 56), (4, 68), (7, -1), (8, 60), (9, 4), (10, q[0]),
             (10, q[3]), (10, q[6]), (11, q[2])])


def test_sizes_without_gpu():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    last = 0
    for M in (0, 1, 7, 8, 100, 300, 4096, 100000):  # never falls with the rows
        n = m.linear_workspace_size(M, 4096, 1024)
        assert last <= n <= 40 << 20
        last = n
    assert m.linear_workspace_size(4, 12, 64) == 0 and m.linear_backward_workspace_size(4, 64, 12) == 0
    last = 0
    for M in (0, 1, 300, 4096):
        n = m.linear_backward_workspace_size(M, 4096, 1024)
        assert last <= n
        last = n


def test_binding_refuses_what_lies_on_the_host():
    import dropless_moe_block_gb300 as m
    x = torch.zeros(4, 64, dtype=BF)
    f = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.route_balanced(f, 2, torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        m.sandwich_norm(x, x, x[0], x[0], 1e-5, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        m.linear(x, torch.zeros(64, 64, dtype=BF), x, torch.zeros(16, dtype=U8))


@pytest.mark.gpu
def test_binding_refusals(dm):
    lg = randn(1, 4, 64, dtype=F32)
    idx, w = empty(4, 2, dtype=I32), empty(4, 2, dtype=F32)
    with pytest.raises(ValueError, match="scores"):
        dm.route_balanced(lg, 2, idx, w, scores="relu")
    with pytest.raises(ValueError, match="bias"):
        dm.route_balanced(lg, 2, idx, w, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(dm.DmoeError):
        dm.route_balanced(lg, 2, idx, w, groups=3)
    x, h, y = randn(1, 4, 64), empty(4, 64), empty(4, 64)
    a = randn(2, 64)
    with pytest.raises(ValueError, match="gate"):
        dm.sandwich_norm(x, x, a, a, 1e-5, h, y, gate=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError, match="same type"):
        dm.sandwich_norm(x, x, a, a.float(), 1e-5, h, y)
    with pytest.raises(ValueError, match="overlap"):
        dm.sandwich_norm(x, x, a, a, 1e-5, h, h)
    both = empty(5, 64)
    with pytest.raises(ValueError, match="overlap"):
        dm.sandwich_norm(both[:4], x, a, a, 1e-5, both[1:], y)
    wm = randn(3, 64, 128)
    o, ws = empty(4, 128), empty(1 << 16, dtype=U8)
    with pytest.raises(ValueError, match="act"):
        dm.linear(x, wm, o, ws, act="tanh")
    with pytest.raises(ValueError, match="deriv"):
        dm.linear(x, wm, o, ws, deriv=empty(4, 128))
    with pytest.raises(ValueError, match="overlap"):
        dm.linear(x, wm, wm[:4], ws)
    with pytest.raises(ValueError, match="overlap"):
        dm.linear_backward(o, x, wm, x, None, ws)
    with pytest.raises(ValueError, match="factor"):
        dm.linear_backward(o, x, wm, None, None, ws, factor=x)


# ------------------------------------------- what a caller may do besides

@pytest.mark.gpu
def test_rows_behind_the_last_stay_as_they_were(dm):
    def tail(*shape, dtype=BF):
        whole = empty(shape[0] + 9, *shape[1:], dtype=dtype)
        return whole, whole[:shape[0]]

    kept = []
    for M, K, N in ((7, 264, 520), (130, 264, 520), (1000, 4096, 136)):
        x, w = randn(1, M, K), randn(2, K, N, scale=K ** -0.5)
        ws, _ = workspace(max(dm.linear_workspace_size(M, K, N), dm.linear_backward_workspace_size(M, K, N)))
        (a, y), (b, f), (c, dx) = tail(M, N), tail(M, N), tail(M, K)
        dm.linear(x, w, y, ws, act="gelu", deriv=f)
        dm.linear_backward(y, x, w, dx, None, ws, deriv=f)
        kept += [(a, M), (b, M), (c, M)]
    for T, d in ((5, 64), (130, 4104)):
        u, x, w = randn(1, T, d), randn(2, T, d), randn(3, d)
        (a, h), (b, y), (c, du), (e, dx) = tail(T, d), tail(T, d), tail(T, d), tail(T, d)
        (f, ru), (g, rh) = tail(T, dtype=F32), tail(T, dtype=F32)
        dm.sandwich_norm(u, x, w, w, 1e-5, h, y, rstd_u=ru, rstd_h=rh)
        dm.sandwich_norm_backward(y, u, h, w, w, ru, rh, du, dx, None, None, None)
        kept += [(t, T) for t in (a, b, c, e, f, g)]
    for T, E, k in ((5, 64, 1), (8193, 64, 8), (77, 40, 3)):
        (a, idx), (b, gw), (c, dl) = tail(T, k, dtype=I32), tail(T, k, dtype=F32), tail(T, E, dtype=F32)
        lg = randn(1, T, E, dtype=F32)
        dm.route_balanced(lg, k, idx, gw)
        dm.route_balanced_backward(lg, idx, gw, dl)
        kept += [(a, T), (b, T), (c, T)]
    for t, n in kept:
        rest = t[n:]
        assert torch.equal(rest, torch.full_like(rest, 77 if t.dtype is I32 else 777.0))


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_route_of_rows_at_odd_places(dm, shift):
    T, E, k = 8200, 64, 4
    flat = randn(1, T * E + 4, dtype=F32)
    bias = randn(2, E + 4, scale=0.02, dtype=F32)[shift:shift + E]
    logits = flat[shift:shift + T * E].view(T, E)
    idx, w = route(dm, logits, k, bias=bias, scores="sigmoid")
    idx2, w2 = route(dm, logits.clone(), k, bias=bias.clone(), scores="sigmoid")
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    d = randn(3, T, k, dtype=F32)
    out = empty(T * E + 4, dtype=F32)
    dl, dl2 = out[shift:shift + T * E].view(T, E), empty(T, E, dtype=F32)
    dm.route_balanced_backward(logits, idx, d, dl, scores="sigmoid")
    dm.route_balanced_backward(logits, idx, d, dl2, scores="sigmoid")
    assert torch.equal(dl, dl2)


@pytest.mark.gpu
def test_two_calls_at_once(dm):
    """Calls on two streams with workspaces of their own, and two graphs replayed side by side."""
    M, K, N = 600, 1032, 2056
    w = randn(2, K, N, scale=K ** -0.5)
    sets = []
    for i in range(2):
        x, dy = randn(10 + i, M, K), randn(20 + i, M, N)
        ws, _ = workspace(max(dm.linear_workspace_size(M, K, N), dm.linear_backward_workspace_size(M, K, N)))
        sets.append((x, dy, ws, empty(M, N), empty(M, N), empty(M, K), empty(K, N), empty(N, dtype=F32)))

    def run(s):
        x, dy, ws, y, f, dx, dw, db = s
        dm.linear(x, w, y, ws, act="silu", deriv=f)
        dm.linear_backward(dy, x, w, dx, dw, ws, deriv=f, dbias=db)

    want = []
    for s in sets:
        run(s)
        want.append([t.clone() for t in s[3:]])
        for t in s[3:]:
            t.fill_(1.0)
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                run(s)
    torch.cuda.synchronize()
    for s, ref in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(s[3:], ref))
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(s)
        graphs.append(g)
        for t in s[3:]:
            t.fill_(1.0)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, ref in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(s[3:], ref))


@pytest.mark.gpu
def test_long_rows_of_many_tokens(dm):
    """Offsets beyond 32 bits: [70000, 32768] outputs hold 2.3e9 elements."""
    M, K, N = 70000, 64, 32768
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    w = (torch.randn(K, N, generator=g, device="cuda") * K ** -0.5).to(BF)
    r = torch.empty(M, N, device="cuda", dtype=BF)
    r.zero_()
    y = torch.empty(M, N, device="cuda", dtype=BF)
    ws, _ = workspace(dm.linear_workspace_size(M, K, N))
    dm.linear(x, w, y, ws, act="gelu", deriv=r)
    for rows in (slice(0, 3), slice(65534, 65539), slice(M - 3, M)):
        z = x[rows].double() @ w.double()
        ref, df = ref_act(z, "gelu")
        S = x[rows].double().abs() @ w.double().abs()
        tol = 2 * (K + 8) * U32 * S + 4e-7 * (1 + z.abs())
        close(y[rows], ref, U16 * ref.abs() + 1.2 * tol, "y")
        close(r[rows], df, U16 * df.abs() + tol, "deriv")
    del y
    # the norms over the same elements: 140000 rows of 16384
    u = r.view(140000, 16384)
    h, o = torch.empty_like(u), torch.empty_like(u)
    ones = torch.ones(16384, device="cuda", dtype=BF)
    dm.sandwich_norm(u, u, ones, ones, 1e-5, h, o)
    for i in (0, 131072, 139999):
        ref = u[i].double() * (1 + 1 / torch.sqrt(u[i].double().square().mean() + 1e-5))
        close(h[i], ref, (U16 + 200 * U32) * ref.abs(), "h")
