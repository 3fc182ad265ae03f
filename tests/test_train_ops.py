"""The operators beside the layer in a training step, against 64-bit references.

Reference values are computed here, in float64, from the definitions in
``include/dmoe.h``.  Tolerances follow from the number formats: U16 = 2^-8 is
one rounding to bf16 (8 significant bits: half a unit in the last place,
relative), U32 = 2^-24
one rounding to fp32, and a sum of n products in any order is off by at most
about n U32 times the sum of their magnitudes.
"""

import ctypes
import math

import numpy as np
import pytest
import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -24


def _dm():
    from dropless_moe_block_gb300 import build
    build.build()
    import dropless_moe_block_gb300 as m
    return m


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m = _dm()
    m.get_error(clear=True)
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen(seed), dtype=torch.float64) * scale).to(dtype)


def cuda(t):
    return t.cuda()


def empty(*shape, dtype):
    """Filled with a value that no result holds."""
    return torch.full(shape, 777.0, device="cuda", dtype=torch.float32).to(dtype)


def close(got, ref, tol, what):
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float(((got - ref).abs() - tol).max()):.3e} over its tolerance")


# ------------------------------------------------------------------ references

def ref_norm(x, res, w, eps):
    h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    hd = h.double()
    r = 1.0 / torch.sqrt((hd * hd).mean(1) + eps)
    return h, r, hd * r[:, None] * w.double()


def ref_norm_backward(dy, h, w, r, dh):
    dy, h, w, r = dy.double(), h.double(), w.double(), r.double()[:, None]
    u = dy * w
    m = (u * h).mean(1, keepdim=True) * r * r
    dx = r * (u - h * m) + (0.0 if dh is None else dh.double())
    size = r * (u.abs() + (h * m).abs()) + (0.0 if dh is None else dh.double().abs())
    terms = dy * h * r
    return dx, size, terms.sum(0), terms.abs().sum(0)


def ref_loss(x, w, t, ignore, d_loss=None):
    """loss, lse, G, its softmax part |g| exp(l - lse), and the logits in 64 bits."""
    l = x.double() @ w.double().t()
    lse = torch.logsumexp(l, 1)
    V = w.shape[0]
    ok = (t >= 0) & (t < V) & (t != ignore)
    at = torch.where(ok, t, torch.zeros_like(t)).long()
    loss = torch.where(ok, lse - l.gather(1, at[:, None]).view(-1), torch.zeros_like(lse))
    g = (d_loss.double() if d_loss is not None else torch.full_like(lse, 1.0 / max(1, int(ok.sum())))) * ok
    G = torch.exp(l - lse[:, None]) * g[:, None]
    G[~ok] = 0.0
    P = G.abs()
    G.scatter_add_(1, at[:, None], -g[:, None])
    return loss, lse, G, P, l


def logit_error(x, w, d):
    """How far an fp32-accumulated logit may be off, per row (the largest over the vocabulary)."""
    return 2 * (d + 8) * U32 * (x.double().abs() @ w.double().abs().t()).amax(1)


# ------------------------------------------------------------- norm (GPU tests)

NORM_SIZES = [(1, 8), (3, 24), (5, 136), (17, 520), (130, 1000), (7, 3584), (2, 4096), (3, 8200), (2, 16392),
              (1, 32768), (1030, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("residual,wf32", [(True, False), (False, True)])
def test_norm_forward(dm, T, d, residual, wf32):
    eps = 1e-5
    x = randn(1, T, d)
    res = randn(2, T, d, scale=3.0) if residual else None
    w = randn(3, d, scale=0.3, dtype=torch.float32 if wf32 else torch.bfloat16) + 1
    h, rstd = empty(T, d, dtype=torch.bfloat16), empty(T, dtype=torch.float32)
    y = empty(T, d, dtype=torch.bfloat16)
    q, s = empty(T, d, dtype=torch.float8_e4m3fn), empty(T, -(-d // 128), dtype=torch.float32)
    dm.add_rms_norm(cuda(x), None if res is None else cuda(res), cuda(w), eps, h, y, rstd=rstd, q=q, q_scale=s)
    hr, rr, yr = ref_norm(x, res, w, eps)
    assert torch.equal(h.cpu().view(torch.int16), hr.view(torch.int16))
    # a thread adds up to 32 squares, then 5 shuffles and 32 warps; the mean
    # and the reciprocal root add a few roundings more
    e = 80 * U32
    close(rstd, rr, e * rr, "rstd")
    close(y, yr, (U16 + 2 * e) * yr.abs(), "y")
    n = -(-d // 128)
    pad = torch.zeros(T, n * 128, dtype=torch.float64)
    pad[:, :d] = yr
    top = pad.view(T, n, 128).abs().amax(2)
    close(s, top / 448, 2 * e * top / 448, "q_scale")
    back = q.cpu().double() * s.cpu().double().repeat_interleave(128, 1)[:, :d]
    unit = (top / 448).repeat_interleave(128, 1)[:, :d]
    # e4m3: 3 bits of fraction (half a unit is 2^-4 of the value), below 2^-6 steps of 2^-9
    close(back, yr, torch.maximum(2.0 ** -4 * yr.abs(), 2.0 ** -10 * unit) * 1.01, "8-bit rows")


@pytest.mark.gpu
def test_norm_zero_rows_and_only_8_bits(dm):
    T, d = 4, 264
    x = torch.zeros(T, d, dtype=torch.bfloat16)
    x[2, 130:140] = 1.0  # only the second group of row 2 is not zero
    q, s = empty(T, d, dtype=torch.float8_e4m3fn), empty(T, 3, dtype=torch.float32)
    w = torch.ones(d, dtype=torch.bfloat16)
    dm.add_rms_norm(cuda(x), None, cuda(w), 1e-6, None, None, q=q, q_scale=s)
    assert dm.get_error() == 0
    s, q = s.cpu(), q.cpu().float()
    _, _, y = ref_norm(x, None, w, 1e-6)
    assert torch.equal(s[[0, 1, 3]], torch.ones(3, 3)) and s[2, 0] == 1 and s[2, 2] == 1
    assert abs(float(s[2, 1]) - float(y[2, 135]) / 448) <= 1e-5 * float(y[2, 135]) / 448
    assert torch.equal(q != 0, x.float() != 0) and float(q[2, 135]) == 448.0


@pytest.mark.gpu
def test_norm_strides_in_place_and_other_stream(dm):
    T, d, eps = 37, 200, 1e-5
    big = cuda(randn(4, T, 3 * d))
    x, res = big[:, :d], big[:, 2 * d:]
    w = cuda(randn(5, d) + 1)
    h, y = empty(T, d, dtype=torch.bfloat16), empty(T, d, dtype=torch.bfloat16)
    dm.add_rms_norm(x, res, w, eps, h, y)
    xc, rc = x.contiguous(), res.contiguous()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    dm.add_rms_norm(xc, rc, w, eps, rc, xc, stream=stream)  # h over the residual, y over x
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(rc, h) and torch.equal(xc, y)


@pytest.mark.gpu
def test_norm_non_finite_rows_stay_apart(dm):
    T, d = 3, 64
    x = randn(6, T, d)
    x[0, 5], x[1, 6] = math.nan, math.inf
    w = torch.ones(d, dtype=torch.bfloat16)
    y = empty(T, d, dtype=torch.bfloat16)
    dm.add_rms_norm(cuda(x), None, cuda(w), 1e-5, None, y)
    y = y.cpu().float()
    assert torch.isnan(y[0]).all() and math.isnan(float(y[1, 6])) and float(y[1, :6].abs().max()) == 0.0
    _, _, yr = ref_norm(x[2:], None, w, 1e-5)
    close(y[2:], yr, (U16 + 160 * U32) * yr.abs(), "the finite row")


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", NORM_SIZES + [(3001, 72), (700, 2056)])
@pytest.mark.parametrize("stream_grad,wf32", [(True, False), (False, True)])
def test_norm_backward(dm, T, d, stream_grad, wf32):
    h, dy = randn(11, T, d, scale=2.0), randn(12, T, d)
    dh = randn(13, T, d) if stream_grad else None
    w = randn(14, d, scale=0.3, dtype=torch.float32 if wf32 else torch.bfloat16) + 1
    r = (1.0 / torch.sqrt((h.double() ** 2).mean(1) + 1e-5)).float()
    dx, dw = empty(T, d, dtype=torch.bfloat16), empty(d, dtype=torch.float32)
    ws = torch.empty(dm.add_rms_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    args = (cuda(dy), cuda(h), cuda(w), cuda(r))
    dhc = None if dh is None else cuda(dh)
    dm.add_rms_norm_backward(*args, dx, dw, ws, dh=dhc)
    ref, size, dwr, dws = ref_norm_backward(dy, h, w, r, dh)
    close(dx, ref, U16 * ref.abs() + 100 * U32 * size, "dx")
    close(dw, dwr, (T + 8) * U32 * dws + 1e-30, "dw")
    # without dw; over dy; the same bits again
    dx2 = args[0].clone()
    dm.add_rms_norm_backward(dx2, *args[1:], dx2, None, None, dh=dhc)
    assert torch.equal(dx2, dx)
    dw2 = empty(d, dtype=torch.float32)
    dm.add_rms_norm_backward(*args, dx, dw2, ws, dh=dhc)
    assert torch.equal(dw, dw2)


@pytest.mark.gpu
def test_norm_backward_strides_and_no_rows(dm):
    T, d = 19, 96
    big = cuda(randn(15, T, 2 * d))
    h, w, r = cuda(randn(16, T, d)), cuda(randn(17, d)), torch.rand(T, device="cuda") + 0.5
    ws = torch.empty(dm.add_rms_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    outs = []
    for dy, dh in ((big[:, :d], big[:, d:]), (big[:, :d].contiguous(), big[:, d:].contiguous())):
        dx, dw = empty(T, d, dtype=torch.bfloat16), empty(d, dtype=torch.float32)
        dm.add_rms_norm_backward(dy, h, w, r, dx, dw, ws, dh=dh)
        outs.append((dx, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    dw = empty(d, dtype=torch.float32)
    none = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    dm.add_rms_norm_backward(none, none, w, torch.empty(0, device="cuda"), none, dw, ws)
    assert float(dw.abs().max()) == 0.0


def directional(f, at, v, step):
    return (f(at + step * v) - f(at - step * v)) / (2 * step)


@pytest.mark.gpu
def test_norm_backward_against_differences(dm):
    """<dx, v> and <dw, v> against central differences of the 64-bit forward."""
    T, d, eps = 6, 48, 1e-3
    h, dy, w = randn(21, T, d), randn(22, T, d), randn(23, d, dtype=torch.float32) + 1
    r = (1.0 / torch.sqrt((h.double() ** 2).mean(1) + eps)).float()
    dx, dw = empty(T, d, dtype=torch.bfloat16), empty(d, dtype=torch.float32)
    ws = torch.empty(dm.add_rms_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    dm.add_rms_norm_backward(cuda(dy), cuda(h), cuda(w), cuda(r), dx, dw, ws)

    def value(hd, wd):
        return float((dy.double() * hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps) * wd).sum())

    v, u = randn(24, T, d, dtype=torch.float64), randn(25, d, dtype=torch.float64)
    got = dx.cpu().double() * v
    want = directional(lambda a: value(a, w.double()), h.double(), v, 1e-5)
    assert abs(float(got.sum()) - want) <= 2 * U16 * float(got.abs().sum())
    got = dw.cpu().double() * u
    want = directional(lambda a: value(h.double(), a), w.double(), u, 1e-5)
    assert abs(float(got.sum()) - want) <= 1e-5 * float(got.abs().sum())


# ------------------------------------------------------------- loss (GPU tests)

LOSS_SIZES = [(1, 1, 8), (1, 2, 8), (5, 7, 16), (3, 129, 72), (33, 1009, 256), (130, 300, 64), (257, 513, 136),
              (300, 1024, 520), (513, 2050, 64), (64, 5003, 1032),
              # enough tiles for the widest ones, several a unit, a narrow last column
              (300, 38900, 1032), (2, 6000, 1288),
              # the last counts of the few-token form, and the first beyond it
              (8, 130, 1096), (4, 65, 24), (9, 130, 1096)]


def run_loss(dm, x, w, t, dx=True, dw=torch.bfloat16, **kw):
    T, d = x.shape
    V = w.shape[0]
    out = dict(loss=empty(T, dtype=torch.float32), lse=empty(T, dtype=torch.float32),
               dx=empty(T, d, dtype=torch.bfloat16) if dx else None,
               dw=empty(V, d, dtype=dw) if dw is not None else None)
    n = dm.linear_cross_entropy_workspace_size(T, d, V, grad=dx or dw is not None,
                                               dw_dtype=dw or torch.bfloat16, piece=kw.get("piece", 0))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever something is not written first
    dm.linear_cross_entropy(x, w, t, out["loss"], out["lse"], ws, dx=out["dx"], dw=out["dw"], **kw)
    return out


def check_loss(out, x, w, t, ignore=-100, d_loss=None, base=None):
    T, d = x.shape
    loss, lse, G, P, l = ref_loss(x, w, t, ignore, d_loss)
    # exp2's argument and value, the sums over a group and over the groups, the
    # logarithm: a few 1e-7 of the terms, at most 1e-6 of the exponent's size
    e = logit_error(x, w, d) + 4e-6 + 2e-7 * l.abs().amax(1)
    close(out["lse"], lse, e, "lse")
    close(out["loss"], loss, 2 * e, "loss")
    # the exponentials and G are each rounded to bf16 once; an error of the
    # logit or of lse is one of the softmax part, whatever cancels in G
    off = 2.05 * U16 * G.abs() + 2 * e[:, None] * P
    if out["dx"] is not None:
        ref = G @ w.double()
        close(out["dx"], ref, U16 * ref.abs() + (off + w.shape[0] * U32 * G.abs()) @ w.double().abs() + 1e-30, "dx")
    if out["dw"] is not None:
        ref = G.t() @ x.double()
        f32 = out["dw"].dtype == torch.float32
        tol = (off + (T + 8) * U32 * G.abs()).t() @ x.double().abs()
        total = ref if base is None else ref + base.double()
        close(out["dw"], total, (U32 if f32 else U16) * total.abs() + tol + 1e-30, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,d", LOSS_SIZES)
def test_loss_and_gradients(dm, T, V, d):
    x, w = randn(31, T, d), randn(32, V, d, scale=2.0 / math.sqrt(d))
    t = torch.randint(0, V, (T,), generator=gen(33), dtype=torch.int32)
    if T > 4:
        t[::5] = -100
    xs, wsd, ts = cuda(x), cuda(w), cuda(t)
    out = run_loss(dm, xs, wsd, ts)
    assert dm.get_error() == 0
    check_loss(out, x, w, t)
    again = run_loss(dm, xs, wsd, ts)
    for k in out:
        assert torch.equal(out[k], again[k]), f"{k} differs between two runs"
    alone = run_loss(dm, xs, wsd, ts, dx=False, dw=None)
    assert torch.equal(alone["loss"], out["loss"]) and torch.equal(alone["lse"], out["lse"])


@pytest.mark.gpu
def test_loss_one_gradient_at_a_time_on_another_stream(dm):
    T, V, d = 300, 900, 264
    x, w = randn(56, T, d), randn(57, V, d, scale=0.2)
    t = torch.randint(0, V, (T,), generator=gen(58), dtype=torch.int32)
    xs, wsd, ts = cuda(x), cuda(w), cuda(t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a = run_loss(dm, xs, wsd, ts, dw=None)
        b = run_loss(dm, xs, wsd, ts, dx=False)
    c = run_loss(dm, xs, wsd, ts, dw=None, stream=torch.cuda.current_stream())
    stream.synchronize()
    check_loss(a, x, w, t)
    check_loss(b, x, w, t)
    assert torch.equal(a["dx"], c["dx"]) and torch.equal(a["loss"], b["loss"])


@pytest.mark.gpu
def test_loss_in_a_graph(dm):
    """Captured and replayed with other inputs in the same places."""
    T, V, d = 70, 300, 72
    x, w = randn(70, T, d), randn(71, V, d, scale=0.2)
    t = torch.randint(0, V, (T,), generator=gen(72), dtype=torch.int32)
    xs, wsd, ts = cuda(x), cuda(w), cuda(t)
    out = run_loss(dm, xs, wsd, ts)
    ws = torch.empty(dm.linear_cross_entropy_workspace_size(T, d, V), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        dm.linear_cross_entropy(xs, wsd, ts, out["loss"], out["lse"], ws, dx=out["dx"], dw=out["dw"])
    x = randn(73, T, d)
    t = torch.full((T,), 5, dtype=torch.int32)
    xs.copy_(x)
    ts.copy_(t)
    graph.replay()
    check_loss(out, x, w, t)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [700, 517])  # the last piece of 517 has 5 tokens
def test_loss_in_pieces(dm, dtype, T):
    V, d = 391, 88
    x, w = randn(34, T, d), randn(35, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(36), dtype=torch.int32)
    t[200:500] = -1  # a whole piece without a target that counts
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=dtype, piece=256, ignore_index=-1)
    check_loss(out, x, w, t, ignore=-1)
    whole = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=dtype, ignore_index=-1)
    assert torch.equal(out["loss"], whole["loss"])
    check_loss(whole, x, w, t, ignore=-1)


@pytest.mark.gpu
def test_loss_arriving_gradient_and_accumulation(dm):
    T, V, d = 90, 500, 40
    x, w = randn(37, T, d), randn(38, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(39), dtype=torch.int32)
    t[3] = 7  # ignore_index may be a word
    g = randn(40, T, dtype=torch.float32)
    g[5] = 0.0
    base = randn(41, V, d, dtype=torch.float32)
    out = dict(loss=empty(T, dtype=torch.float32), lse=empty(T, dtype=torch.float32),
               dx=empty(T, d, dtype=torch.bfloat16), dw=cuda(base.clone()))
    n = dm.linear_cross_entropy_workspace_size(T, d, V, dw_dtype=torch.float32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dm.linear_cross_entropy(cuda(x), cuda(w), cuda(t), out["loss"], out["lse"], ws, dx=out["dx"], dw=out["dw"],
                            d_loss=cuda(g), ignore_index=7, accumulate=True)
    check_loss(out, x, w, t, ignore=7, d_loss=g, base=base)
    assert float(out["dx"][5].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0.0, 150.0, -150.0])
def test_loss_of_large_logits(dm, shift):
    """Rows whose logits leave the range where no reference is subtracted: all
    of them far above or below zero, or single ones."""
    T, V, d = 40, 700, 16
    x, w = torch.zeros(T, d), torch.zeros(V, d)
    x[:, 0] = 1.0
    w[:, 0] = shift + torch.randint(-8, 8, (V,), generator=gen(42)).float()  # exact in bf16 up to 256
    w[300, 0] += 90.0  # one group far above the others
    w[690, 0] -= 100.0
    x[7], x[8, 0] = 0.0, -1.0
    x[9, 0] = 0.0
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=gen(43), dtype=torch.int32)
    t[:3] = torch.tensor([300, 690, 5])
    check_loss(run_loss(dm, cuda(x), cuda(w), cuda(t)), x, w, t)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [150.0, -150.0])
def test_loss_of_large_logits_of_few_tokens(dm, shift):
    """The same where dw has its few-token form."""
    T, V, d = 6, 700, 16
    x, w = torch.zeros(T, d), torch.zeros(V, d)
    x[:, 0] = torch.tensor([1.0, -1.0, 0.0, 1.0, 0.5, 1.0])
    x[:, 1] = 1.0
    w[:, 0] = shift + torch.randint(-8, 8, (V,), generator=gen(74)).float()
    w[300, 0] += 90.0
    w[640:, 0] -= 100.0
    w[:, 1] = torch.randint(-2, 3, (V,), generator=gen(75)).float()
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    t = torch.tensor([300, 690, 5, -100, 44, 45], dtype=torch.int32)
    check_loss(run_loss(dm, cuda(x), cuda(w), cuda(t)), x, w, t)


@pytest.mark.gpu
def test_loss_without_targets_that_count(dm):
    T, V, d = 70, 200, 24
    x, w = randn(44, T, d), randn(45, V, d)
    x[3] = math.inf  # an ignored row may hold anything
    t = torch.full((T,), -100, dtype=torch.int32)
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=None)
    assert float(out["loss"].abs().max()) == 0.0 and float(out["dx"].float().abs().max()) == 0.0
    x[3] = 0
    out = run_loss(dm, cuda(x), cuda(w), cuda(t))
    assert float(out["dw"].float().abs().max()) == 0.0
    assert dm.get_error() == 0


@pytest.mark.gpu
def test_loss_reports_a_target_out_of_range(dm):
    T, V, d = 9, 50, 16
    x, w = randn(46, T, d), randn(47, V, d)
    t = torch.randint(0, V, (T,), generator=gen(48), dtype=torch.int32)
    t[2], t[4] = V, -7
    out = run_loss(dm, cuda(x), cuda(w), cuda(t))
    assert dm.get_error(clear=True) == (7 << 8) | 5
    check_loss(out, x, w, t)  # as if they were ignored


@pytest.mark.gpu
def test_loss_one_word_for_all(dm):
    """Every target the same word: its row of dw sums all tokens."""
    T, V, d = 600, 300, 64
    x, w = randn(49, T, d), randn(50, V, d, scale=0.2)
    t = torch.full((T,), 131, dtype=torch.int32)
    check_loss(run_loss(dm, cuda(x), cuda(w), cuda(t)), x, w, t)


@pytest.mark.gpu
def test_loss_no_tokens(dm):
    V, d = 30, 16
    w = cuda(randn(51, V, d))
    x = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    out = run_loss(dm, x, w, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert float(out["dw"].float().abs().max()) == 0.0


@pytest.mark.gpu
def test_loss_against_differences(dm):
    T, V, d = 20, 60, 24
    x, w = randn(52, T, d), randn(53, V, d, scale=0.4)
    t = torch.randint(0, V, (T,), generator=gen(54), dtype=torch.int32)
    t[4] = -100
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=torch.float32)
    n = int((t >= 0).sum())

    def value(xd, wd):
        l = xd @ wd.t()
        lse = torch.logsumexp(l, 1)
        ok = t >= 0
        return float(((lse - l.gather(1, t.clamp(min=0).long()[:, None]).view(-1)) * ok).sum()) / n

    for name, at, f in (("dx", x.double(), lambda a: value(a, w.double())),
                        ("dw", w.double(), lambda a: value(x.double(), a))):
        v = randn(55, *at.shape, dtype=torch.float64)
        got = out[name].cpu().double() * v
        want = directional(f, at, v, 1e-5)
        # G's two roundings and the output's, per term
        assert abs(float(got.sum()) - want) <= 4 * U16 * float(got.abs().sum()), name


# ------------------------------------------------------------- clip (GPU tests)

def clip_case(seed, sizes, kinds, offsets):
    """Tensors of the given sizes that begin `offset` elements into their storage."""
    out = []
    for i, (n, k, o) in enumerate(zip(sizes, kinds, offsets)):
        out.append(cuda(randn(seed + i, n + o, dtype=k))[o:])
    return out


SIZES = [1, 0, 7, 8, 8191, 8192, 8193, 100003, 3, 0]
KINDS = [torch.bfloat16, torch.float32, torch.float32, torch.bfloat16, torch.bfloat16, torch.float32, torch.bfloat16,
         torch.bfloat16, torch.float32, torch.bfloat16]


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("limit", [0.37, 1e9])
def test_clip(dm, shift, limit):
    gs = clip_case(60, SIZES, KINDS, [(i + shift) % 5 for i in range(len(SIZES))])
    outs = clip_case(90, SIZES, KINDS, [(i * shift) % 7 for i in range(len(SIZES))])
    norm = empty(1, dtype=torch.float32)
    before = [g.clone() for g in gs]
    dm.clip_grad_norm(dm.GradList(gs, outs), limit, norm)
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in before))
    c = min(1.0, limit / (total + 1e-6))
    # a thread adds at most 32 vectors' squares in fp32
    assert abs(float(norm) - total) <= 2 * 8 * 33 * U32 * total
    for g, o, k in zip(before, outs, KINDS):
        ref = g.cpu().double() * c
        close(o, ref, ((U16 if k == torch.bfloat16 else 4 * U32) + 600 * U32) * ref.abs(), "clipped")
    for g, b in zip(gs, before):
        assert torch.equal(g, b)
    dm.clip_grad_norm(dm.GradList(gs), limit, norm)  # in place
    for g, o in zip(gs, outs):
        assert torch.equal(g, o)


@pytest.mark.gpu
def test_clip_many_tensors_and_same_bits(dm):
    sizes = [1 + (i * 7919) % 3001 for i in range(300)]
    gs = clip_case(200, sizes, [torch.bfloat16] * 300, [i % 9 for i in range(300)])
    outs = [torch.empty_like(g) for g in gs]
    lst = dm.GradList(gs, outs)
    n1, n2 = empty(1, dtype=torch.float32), empty(1, dtype=torch.float32)
    dm.clip_grad_norm(lst, 1.0, n1)
    first = [o.clone() for o in outs]
    dm.clip_grad_norm(lst, 1.0, n2)
    assert torch.equal(n1, n2) and all(torch.equal(a, b) for a, b in zip(first, outs))
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
    assert abs(float(n1) - total) <= 600 * U32 * total


@pytest.mark.gpu
def test_clip_norms_that_are_not_finite(dm):
    g = cuda(randn(61, 1000))
    norm = empty(1, dtype=torch.float32)
    out = torch.empty_like(g)
    g[17] = math.inf
    dm.clip_grad_norm(dm.GradList([g], [out]), 1.0, norm)
    assert math.isinf(float(norm)) and math.isnan(float(out[17])) and float(out[:17].float().abs().max()) == 0.0
    g[17] = math.nan
    dm.clip_grad_norm(dm.GradList([g], [out]), 1.0, norm)
    assert math.isnan(float(norm)) and bool(torch.isnan(out.float()).all())


@pytest.mark.gpu
def test_clip_of_zeros_and_of_nothing(dm):
    g = torch.zeros(100, device="cuda")
    norm = empty(1, dtype=torch.float32)
    dm.clip_grad_norm(dm.GradList([g]), 1.0, norm)
    assert float(norm) == 0.0 and float(g.abs().max()) == 0.0
    norm.fill_(5)
    dm.clip_grad_norm(dm.GradList([]), 1.0, norm)
    assert float(norm) == 0.0
    g.fill_(2.0)
    dm.clip_grad_norm(dm.GradList([g]), 0.0, norm)
    assert float(norm) == 20.0 and float(g.abs().max()) == 0.0


# -------------------------------------------------------------------- refusals

def test_refusals_without_gpu():
    """Host-side checks of the C entry points: an error status, nothing launched."""
    L = _dm().lib()
    p, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
    f = ctypes.c_float(1e-5)

    def norm(x=p, ldx=64, res=p, ldr=64, w=p, eps=f, T=4, d=64, h=p, y=p, rstd=p, q=None, s=None):
        return L.dmoe_add_rms_norm(x, ldx, res, ldr, w, 0, eps, T, d, h, y, rstd, q, s, None)

    assert norm(T=0) == 0
    for bad in (dict(d=60), dict(d=0), dict(d=32776, ldx=32776, ldr=32776), dict(x=None), dict(w=None), dict(h=None),
                dict(y=None), dict(q=p), dict(ldx=56), dict(ldr=68), dict(x=odd), dict(T=-1),
                dict(eps=ctypes.c_float(-1.0)), dict(eps=ctypes.c_float(math.nan))):
        assert norm(**bad) == 1, bad

    def back(dy=p, ld=64, T=4, d=64, rstd=p, dx=p, dw=p, ws=p, n=1 << 24):
        return L.dmoe_add_rms_norm_backward(dy, ld, p, p, 0, rstd, p, 64, T, d, dx, dw, ws, n, None)

    for bad in (dict(dy=None), dict(ld=60), dict(d=12), dict(rstd=None), dict(dx=None), dict(T=-2), dict(ws=odd)):
        assert back(**bad) == 1, bad

    def loss(x=p, w=p, t=p, T=4, d=64, V=100, out=p, dx=p, dw=p, f32=0, acc=0, piece=0, ws=p, n=1 << 40):
        return L.dmoe_linear_cross_entropy(x, w, t, T, d, V, -100, None, out, None, dx, dw, f32, acc, piece, ws, n, None)

    for bad in (dict(x=None), dict(w=None), dict(t=None), dict(out=None), dict(ws=None), dict(d=60), dict(V=0),
                dict(V=(1 << 24) + 1), dict(acc=1), dict(acc=1, f32=1, dw=None), dict(piece=-1), dict(x=odd),
                dict(dw=odd), dict(n=1000), dict(ws=ctypes.c_void_p(0x1010))):
        assert loss(**bad) == 1, bad

    def clip(g=p, n=1, chunks=1, top=1.0, eps=1e-6, norm=p, ws=p, nws=1 << 20):
        return L.dmoe_clip_grad_norm(g, n, chunks, top, eps, norm, ws, nws, None)

    for bad in (dict(g=None), dict(n=0), dict(n=-1), dict(chunks=-1), dict(top=-1.0), dict(top=math.nan),
                dict(eps=-1.0), dict(norm=None), dict(ws=None), dict(nws=8)):
        assert clip(**bad) == 1, bad
    if not torch.cuda.is_available():  # well-formed calls fail cleanly
        assert norm() in (2, 3) and back() in (2, 3) and loss() in (2, 3) and clip() in (2, 3)


def test_workspace_sizes_and_chunks():
    L = _dm().lib()
    size = L.dmoe_linear_cross_entropy_workspace_size
    assert size(100, 60, 10, 1, 0, 0) == 0  # d not a multiple of 8
    small, grad = size(2048, 64, 32000, 0, 0, 0), size(2048, 64, 32000, 1, 0, 0)
    # the loss alone: 8 bytes a token and 64 words, a fraction of the logits
    assert 2048 * 500 * 8 <= small < 2048 * 501 * 8 and grad - small >= 2048 * 32000 * 2
    # bounded by the piece, plus the fp32 sum of a bf16 dw over several pieces
    assert size(1 << 20, 64, 32000, 1, 1, 4096) == size(4096, 64, 32000, 1, 1, 4096)
    assert size(8192, 64, 32000, 1, 0, 4096) - size(8192, 64, 32000, 1, 1, 4096) == 32000 * 64 * 4
    c = L.dmoe_grad_chunks
    assert [c(0x1000, n, 0) for n in (0, 1, 8192, 8193)] == [0, 1, 1, 2]
    assert c(0x1002, 8192, 0) == 2 and c(0x100c, 8190, 1) == 2 and c(0x100c, 8189, 1) == 1


def test_binding_refuses_wrong_tensors():
    m = _dm()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.add_rms_norm(x, None, w, 1e-5, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        m.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4), None, torch.zeros(8))
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        m.GradList([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="outputs"):
        m.GradList([torch.zeros(4)], [])


@pytest.mark.gpu
def test_binding_refuses_on_the_device(dm):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="weight"):
        dm.add_rms_norm(x, None, w.half(), 1e-5, None, y)
    with pytest.raises(ValueError, match="h is required"):
        dm.add_rms_norm(x, x, w, 1e-5, None, y)
    with pytest.raises(ValueError, match="multiple of 8"):
        dm.add_rms_norm(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64], None, w, 1e-5, None, y)
    with pytest.raises(ValueError, match="q_scale"):
        dm.add_rms_norm(x, None, w, 1e-5, None, y, q=torch.empty(4, 64, dtype=torch.float8_e4m3fn, device="cuda"))
    with pytest.raises(dm.DmoeError):
        dm.add_rms_norm(x, None, w, -1.0, None, y)
    t, l = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(dm.DmoeError):
        dm.linear_cross_entropy(x, x, t, l, None, ws)
    with pytest.raises(ValueError, match="targets"):
        dm.linear_cross_entropy(x, x, t.long(), l, None, ws)
    with pytest.raises(ValueError, match="contiguous"):
        dm.GradList([torch.zeros(4, 4, device="cuda").t()])
