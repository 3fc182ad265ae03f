"""Edges of the operators beside the layer: what stands in rows that do not count, buffers used for other
lengths, masked words, streams, aliases, and the sizes at which the loss changes its launches.

References and the units U16 (one rounding to bf16) and U32 (one to fp32) are those of test_train_ops.py.
"""

import ctypes
import math

import pytest
import torch

from test_train_ops import (U16, U32, _dm, check_loss, close, cuda, dm, empty, gen, logit_error, randn,  # noqa: F401
                            ref_loss, run_loss)


def bounds(x, w, t, d_loss=None, again=0):
    """G, and dx and dw with their bounds (dw in fp32).  Of G only the part that is not the target's passes through
    bf16: once as an exponential (once more where a row's groups are brought to one reference: again = 1), for dw
    once as a multiple of x.  An error e of a logit or of lse is one of the softmax's part, 2 e P; sums add their
    terms' roundings to fp32."""
    T, d = x.shape
    V = w.shape[0]
    _, _, G, P, l = ref_loss(x, w, t, -100, d_loss)
    e = (logit_error(x, w, d) + 4e-6 + 2e-7 * l.abs().amax(1))[:, None]
    ok = t >= 0
    soft = P.clone()
    soft.scatter_(1, torch.where(ok, t, torch.zeros_like(t)).long()[:, None], torch.where(ok[:, None], 0.0, soft[:, :1]))
    a, b = x.double(), w.double()
    dx, dw = G @ b, G.t() @ a
    r = 1.02 * U16 * soft
    tx = U16 * dx.abs() + ((1 + again) * r + 2 * e * P + (V + 8) * U32 * G.abs()) @ b.abs() + 1e-30
    tw = U32 * dw.abs() + ((2 + again) * r + 2 * e * P + (T + 8) * U32 * G.abs()).t() @ a.abs() + 1e-30
    return G, dx, dw, tx, tw


# ------------------------------------------------ rows that do not count

def replaced(out, key, rows, value):
    """out with `value` where the rows of out[key] say nothing."""
    t = out[key].clone()
    t[rows] = value
    return {**out, key: t}


def hold_anything(x, rows):
    """x with rows of an infinity, of NaN and of both."""
    x = x.clone()
    for i, r in enumerate(rows):
        x[r, i % x.shape[1]] = (math.inf, math.nan, -math.inf)[i % 3]
        if i % 3 == 2:
            x[r] = math.nan
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,piece", [(1, 0), (2, 0), (4, 0), (6, 0), (8, 0), (9, 0), (70, 0), (517, 256)])
def test_rows_that_do_not_count_may_hold_anything(dm, T, piece, dtype):
    """The last piece of 517 tokens has 5."""
    V, d = 391, 88
    rows = [T - 1] if T < 6 else [1, 3, T - 1]
    x, w = randn(101, T, d), randn(102, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(103), dtype=torch.int32)
    t[rows] = -100
    out = run_loss(dm, cuda(hold_anything(x, rows)), cuda(w), cuda(t), dw=dtype, piece=piece)
    assert dm.get_error() == 0
    x[rows] = 0  # their gradients are zero whatever they hold
    check_loss(replaced(out, "lse", rows, math.log(V)), x, w, t)
    assert float(out["dx"][rows].float().abs().max()) == 0.0
    if T == 1:
        assert float(out["dw"].float().abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 70, 4100])
def test_rows_of_no_weight_may_hold_anything(dm, T):
    """d_loss 0 at a target that is a word.  From 4096 tokens on the words'
    tokens are added one by one, 70 go by sums of runs."""
    V, d = 300, 64
    rows = [1, 3, T - 1]
    x, w = randn(104, T, d), randn(105, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(106), dtype=torch.int32)
    t[3] = t[1]
    g = randn(107, T, dtype=torch.float32)
    g[rows] = 0.0
    if T == 4100:  # a word of one token, which is such a row
        t[t == 17] = 18
        t[3] = 17
    out = run_loss(dm, cuda(hold_anything(x, rows)), cuda(w), cuda(t), dw=torch.float32, d_loss=cuda(g))
    x[rows] = 0
    out = replaced(out, "lse", rows, math.log(V))
    check_loss(replaced(out, "loss", rows, math.log(V)), x, w, t, d_loss=g)
    assert float(out["dx"][rows].float().abs().max()) == 0.0


# ---------------------------------------------------------- masked words

@pytest.mark.gpu
@pytest.mark.parametrize("T,V,d", [(5, 700, 16), (40, 700, 16), (300, 38900, 1032)])
@pytest.mark.parametrize("level", [0.0, -100.0, 100.0])
def test_words_masked_by_the_lowest_value(dm, T, V, d, level):
    """A column of x that is 1 and of w that is the type's lowest value takes words out of the softmax: single ones,
    and whole groups of 64.  The last size has 512-wide tiles."""
    lowest = torch.finfo(torch.bfloat16).min
    x, w = randn(111, T, d), randn(112, V, d, scale=0.5 / math.sqrt(d))
    x[:, 0], w[:, 0] = 1.0, 0.0
    x[:, 1], w[:, 1] = 1.0, level
    masked = torch.zeros(V, dtype=torch.bool)
    masked[64:192] = masked[3] = masked[V - 5:] = masked[400:470] = True
    keep = ~masked
    words = keep.nonzero().view(-1)
    t = words[torch.randint(0, len(words), (T,), generator=gen(113))]
    w[masked, 0] = lowest
    out = run_loss(dm, cuda(x), cuda(w), cuda(t.int()))
    assert dm.get_error() == 0
    assert float(out["dw"][cuda(masked)].float().abs().max()) == 0.0
    w, t = w[keep], (keep.cumsum(0) - 1)[t].int()
    check_loss({**out, "dx": None, "dw": None}, x, w, t)
    _, dx, dw, tx, tw = bounds(x, w, t, again=1)
    close(out["dx"], dx, tx, "dx")
    close(out["dw"][cuda(keep)], dw, tw + U16 * dw.abs(), "dw")


@pytest.mark.gpu
def test_a_word_masked_in_by_the_highest_value(dm):
    """A logit of 3e38: certain, and the others' loss as large as it."""
    T, V, d = 9, 200, 16
    x, w = torch.zeros(T, d, dtype=torch.bfloat16), torch.zeros(V, d, dtype=torch.bfloat16)
    x[:, 0], w[130, 0] = 1.0, torch.finfo(torch.bfloat16).max
    t = torch.full((T,), 130, dtype=torch.int32)
    t[4] = 7
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dx=False, dw=None)
    top = float(w[130, 0])
    lse, loss = out["lse"].cpu().double(), out["loss"].cpu().double()
    assert float((lse - top).abs().max()) <= 4 * U32 * top
    assert abs(float(loss[4]) - top) <= 8 * U32 * top and float(loss[t == 130].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("level", [0.0, -100.0, -150.0, 100.0])
def test_words_masked_by_minus_infinity(dm, level):
    """The loss alone (dx multiplies what is in w, the infinities too)."""
    T, V, d = 40, 700, 16
    x, w = randn(114, T, d), randn(115, V, d, scale=0.1)
    x[:, 0], w[:, 0] = 1.0, 0.0
    x[:, 1], w[:, 1] = 1.0, level
    masked = torch.zeros(V, dtype=torch.bool)
    masked[64:192] = masked[3] = masked[400:470] = True
    keep = ~masked
    words = keep.nonzero().view(-1)
    t = words[torch.randint(0, len(words), (T,), generator=gen(116))]
    w[masked, 0] = -math.inf
    out = run_loss(dm, cuda(x), cuda(w), cuda(t.int()), dx=False, dw=None)
    check_loss(out, x, w[keep], (keep.cumsum(0) - 1)[t].int())


# ------------------------------------------- one workspace, other lengths

SPACES = [(2048, 32000, 0), (4096, 32000, 0), (4096, 128000, 0), (512, 32000, 0), (64, 500, 0), (256, 1009, 0),
          (1032, 41031, 1024), (8192, 2000, 0)]


@pytest.mark.parametrize("d,V,piece", SPACES)
@pytest.mark.parametrize("grad,f32", [(0, 0), (1, 0), (1, 1)])
def test_workspace_never_shrinks_with_more_tokens(d, V, piece, grad, f32):
    size = _dm().lib().dmoe_linear_cross_entropy_workspace_size
    lengths = sorted(set(range(0, 700)) | set(range(700, 9001, 13)) | {8191, 8192, 8193, 8447, 8448, 16384, 20001})
    sizes = [size(T, d, V, grad, f32, piece) for T in lengths]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("d,V,piece", SPACES)
def test_a_longer_batchs_workspace_is_taken(d, V, piece):
    """Every shorter call gets past the checks of its arguments; a call that asks for fewer outputs does, too."""
    if torch.cuda.is_available():
        pytest.skip("without a device: the calls that are taken must not run")
    L = _dm().lib()
    p = ctypes.c_void_p(0x1000)
    longest = 8192 + 4096
    for f32 in (0, 1):
        n = L.dmoe_linear_cross_entropy_workspace_size(longest, d, V, 1, f32, piece)
        for T in [*range(1, 400, 7), *range(400, longest + 1, 97), 238, 2561, 3555, 3584, 6912, 7440, 7921, longest]:
            for dx, dw in ((p, p), (p, None), (None, p), (None, None)):
                assert L.dmoe_linear_cross_entropy(p, p, p, T, d, V, -100, None, p, None, dx, dw, f32, 0, piece, p, n,
                                                   None) in (2, 3), (T, dx, dw)


@pytest.mark.gpu
def test_loss_in_a_longer_batchs_workspace(dm):
    """The same bits in a workspace made for 1024 tokens as in one of the call's own length."""
    V, d = 9001, 1032
    ws = torch.empty(dm.linear_cross_entropy_workspace_size(1024, d, V), dtype=torch.uint8, device="cuda")
    w = cuda(randn(121, V, d, scale=0.05))
    for T in (5, 13, 238, 300, 513, 1024):
        x = cuda(randn(122, T, d))
        t = cuda(torch.randint(0, V, (T,), generator=gen(123), dtype=torch.int32))
        own = run_loss(dm, x, w, t)
        out = {k: torch.empty_like(v) for k, v in own.items()}
        ws.fill_(255)
        dm.linear_cross_entropy(x, w, t, out["loss"], out["lse"], ws, dx=out["dx"], dw=out["dw"])
        for k in out:
            assert torch.equal(out[k], own[k]), (T, k)


# ------------------------------------------------------- rows in 8 bits

@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(64, 512), (33, 1000), (9, 3584), (5, 8200), (2, 16392)])
def test_8_bit_rows_are_the_quotients_rounded_once(dm, T, d):
    """Given the kernel's own rstd, y in fp32 is two products, the scale one quotient and a value one more: each of
    them, rounded as IEEE says, gives the bits."""
    x = randn(131, T, d, scale=3.0)
    w = randn(132, d, scale=0.3, dtype=torch.float32) + 1
    rstd = empty(T, dtype=torch.float32)
    q, s = empty(T, d, dtype=torch.float8_e4m3fn), empty(T, -(-d // 128), dtype=torch.float32)
    dm.add_rms_norm(cuda(x), None, cuda(w), 1e-5, None, None, rstd=rstd, q=q, q_scale=s)
    y = x.float() * rstd.cpu()[:, None] * w
    n = -(-d // 128)
    pad = torch.zeros(T, n * 128)
    pad[:, :d] = y
    scale = pad.view(T, n, 128).abs().amax(2) / 448.0
    assert torch.equal(s.cpu(), scale)
    want = (y / scale.repeat_interleave(128, 1)[:, :d]).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.gpu
def test_8_bit_rows_of_a_group_with_an_infinity(dm):
    """A value past fp32: its group's scale is infinite, the others of the group are 0, other groups as ever."""
    T, d = 3, 384
    x = randn(133, T, d).abs() + 0.5
    w = torch.ones(d)
    w[140] = 3e38
    q, s = empty(T, d, dtype=torch.float8_e4m3fn), empty(T, 3, dtype=torch.float32)
    x[1] = 0
    x[2, 140] = 50.0
    x[0, 140] = 50.0
    dm.add_rms_norm(cuda(x), None, cuda(w), 1e-5, None, None, q=q, q_scale=s)
    q, s = q.cpu().float(), s.cpu()
    assert torch.equal(torch.isinf(s), torch.tensor([[False, True, False], [False] * 3, [False, True, False]]))
    assert torch.equal(s[1], torch.ones(3)) and float(q[1].abs().max()) == 0.0
    for t in (0, 2):
        assert math.isnan(float(q[t, 140])) and float(q[t, 128:140].abs().max()) == 0.0
        assert float(q[t, :128].max()) == 448.0 and float(q[t, 256:].max()) == 448.0


# ---------------------------------------------------------------- clipping

@pytest.mark.gpu
def test_clip_where_the_factor_is_no_quotient(dm):
    """No limit (an infinite one) never scales; a norm of 0 with eps 0 leaves the zeros alone."""
    norm = empty(1, dtype=torch.float32)
    g = torch.zeros(100, device="cuda")
    dm.clip_grad_norm(dm.GradList([g]), 0.0, norm, eps=0.0)
    assert float(norm) == 0.0 and float(g.abs().max()) == 0.0
    g = cuda(randn(141, 1000))
    before = g.clone()
    dm.clip_grad_norm(dm.GradList([g]), math.inf, norm)
    assert torch.equal(g, before) and math.isfinite(float(norm))
    g[17] = math.inf
    before = g.clone()
    out = torch.empty_like(g)
    dm.clip_grad_norm(dm.GradList([g], [out]), math.inf, norm)
    assert math.isinf(float(norm)) and torch.equal(out, before)


@pytest.mark.gpu
def test_clip_on_another_stream_than_the_lists(dm):
    """A list is ready when it is built, whatever its stream has still to do: its scratch comes from memory that
    held something else, its stream is busy, and the clipping goes to a stream that waits for nothing."""
    sizes = [5000, 70000, 3, 8192]
    gs = [cuda(randn(151 + i, n)) for i, n in enumerate(sizes)]
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
    outs = [torch.empty_like(g) for g in gs]
    norm = empty(1, dtype=torch.float32)
    torch.cuda.synchronize()
    for _ in range(3):
        dirty = [torch.full((1 << 14,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del dirty
        busy, other = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(busy):
            grads = dm.GradList(gs, outs)
            assert busy.query()  # nothing of the building is left to run
        norm.fill_(777.0)
        torch.cuda.synchronize()
        dm.clip_grad_norm(grads, 1.0, norm, stream=other)
        other.synchronize()
        assert abs(float(norm) - total) <= 600 * U32 * total


@pytest.mark.gpu
def test_a_lists_scratch_outlives_its_use_on_another_stream(dm):
    """The list goes while its clipping still waits in another stream; what is allocated next must not get its memory."""
    g = cuda(randn(161, 100000))
    out, norm = torch.empty_like(g), empty(1, dtype=torch.float32)
    total = math.sqrt(float((g.double() ** 2).sum()))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    grads = dm.GradList([g], [out])
    places = {grads.table.data_ptr(), grads.ws.data_ptr()}
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)  # some 10 ms
        dm.clip_grad_norm(grads, 1.0, norm)
    del grads
    fresh = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (40, 512, 1 << 14, 16400) for _ in range(4)]
    assert not places & {f.data_ptr() for f in fresh}
    other.synchronize()
    assert abs(float(norm) - total) <= 600 * U32 * total


def test_gradients_that_overlap_are_refused():
    """Two outputs in one place, or an output over another tensor's gradient, would be scaled twice or half."""
    m = _dm()
    check = m._check_disjoint
    check([(64, 32), (0, 64), (96, 0), (96, 8)], [(64, 32), (0, 64), (96, 0), (96, 8)])  # in place
    check([(0, 64), (0, 64), (32, 64)], [(100, 64), (164, 64), (300, 64)])  # read twice, written apart
    check([(0, 64), (64, 64)], [(128, 64), (192, 64)])
    for ins, outs in (([(0, 64), (0, 64)], [(0, 64), (0, 64)]),        # the same gradient twice, in place
                      ([(0, 64), (100, 64)], [(200, 64), (232, 64)]),  # outputs over each other
                      ([(0, 64), (100, 64)], [(100, 64), (200, 64)]),  # over another's gradient
                      ([(0, 64)], [(32, 64)]),                         # over its own, moved
                      ([(0, 64), (256, 8)], [(0, 64), (60, 8)])):
        with pytest.raises(ValueError, match="overlap"):
            check(ins, outs)


@pytest.mark.gpu
def test_a_gradient_listed_twice_is_refused(dm):
    g, h = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        dm.GradList([g, h, g])
    with pytest.raises(ValueError, match="overlap"):
        dm.GradList([g, h], [h, torch.empty_like(h)])
    norm = empty(1, dtype=torch.float32)
    a, b = torch.empty_like(g), torch.empty_like(g)
    dm.clip_grad_norm(dm.GradList([g, g], [a, b]), 1e9, norm)  # read twice, written apart
    assert torch.equal(a, g) and torch.equal(b, g) and abs(float(norm) - math.sqrt(200)) <= 8 * U32 * 15


# ----------------------------------------------------------------- aliases

def test_rows_written_over_rows_of_another_pitch_are_refused():
    """A block would write over rows that others have not read.  Host-side: an error status, nothing launched."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: not where a device could be given them")
    L = _dm().lib()
    x, r, w, h, y, q, s = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(7))

    def norm(ldx=64, ldr=64, T=4, h=h, y=y):
        return L.dmoe_add_rms_norm(x, ldx, r, ldr, w, 0, ctypes.c_float(1e-5), T, 64, h, y, None, q, s, None)

    def back(lddy=64, lddh=64, T=4, dx=h):
        return L.dmoe_add_rms_norm_backward(x, lddy, y, w, 0, q, r, lddh, T, 64, dx, None, None, 0, None)

    bad = [norm(ldx=128, h=x), norm(ldr=128, h=r), norm(ldx=128, y=x), norm(ldr=128, y=r), back(lddy=128, dx=x),
           back(lddh=128, dx=r)]
    assert bad == [1] * len(bad), bad
    # the same pitch, or one row: an error only because there is no device
    good = [norm(), norm(ldx=128, ldr=72), norm(h=x), norm(h=r), norm(y=x), norm(h=r, y=x), norm(y=r),
            norm(T=1, ldx=128, h=x), back(dx=x), back(dx=r), back(lddy=128), back(T=1, lddy=128, dx=x)]
    assert all(g in (2, 3) for g in good), good


@pytest.mark.gpu
def test_outputs_that_overlap_what_is_read_are_refused(dm):
    T, V, d = 12, 40, 64
    buf = torch.zeros(4 * T + 2 * V, d, dtype=torch.bfloat16, device="cuda")
    x, w = buf[:T], buf[T:T + V]
    t = torch.zeros(T, dtype=torch.int32, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)

    def loss(**kw):
        return run_loss_into(dm, x, w, t, **kw)

    for kw in (dict(dx=x, dw=dw), dict(dx=buf[1:T + 1], dw=dw), dict(dx=buf[1:T + 1]), dict(dx=w[:T]), dict(dw=w),
               dict(dx=dx, dw=buf[:V]), dict(dx=buf[T + V:2 * T + V], dw=buf[T + V + 4:T + 2 * V + 4])):
        with pytest.raises(ValueError, match="overlap"):
            loss(**kw)
    one = randn(165, T, d).cuda()
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        dm.add_rms_norm(one, one, ones, 1e-5, dx, dx)


def run_loss_into(dm, x, w, t, dx=None, dw=None):
    loss = torch.empty(len(t), device="cuda")
    ws = torch.empty(dm.linear_cross_entropy_workspace_size(*x.shape, len(w)), dtype=torch.uint8, device="cuda")
    dm.linear_cross_entropy(x, w, t, loss, None, ws, dx=dx, dw=dw)
    return loss


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 300])
def test_dx_over_x_where_no_dw_is_asked_for(dm, T):
    V, d = 700, 72
    x, w = randn(166, T, d), randn(167, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(168), dtype=torch.int32)
    own = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=None)
    xs = cuda(x)
    loss = run_loss_into(dm, xs, cuda(w), cuda(t), dx=xs)
    assert torch.equal(xs, own["dx"]) and torch.equal(loss, own["loss"])


@pytest.mark.gpu
def test_lanes_that_differ_in_the_first_half_of_a_wide_tile(dm):
    """512-wide tiles whose first 256 words hold some rows' targets, and logits past the references' range in some
    rows only: the second half is loaded by whole warps all the same."""
    T, V, d = 300, 38900, 1032
    x, w = randn(201, T, d), randn(202, V, d, scale=0.5 / math.sqrt(d))
    x[:, 0], w[:, 0] = 0.0, 0.0
    x[::3, 0] = 1.0
    w[0:64, 0], w[512 * 20 + 70:512 * 20 + 100, 0] = 90.0, -120.0
    t = torch.randint(0, V, (T,), generator=gen(203))
    t[::2] = t[::2] // 512 * 512 + t[::2] % 256
    t[::2].clamp_(max=V - 1)
    out = run_loss(dm, cuda(x), cuda(w), cuda(t.int()))
    check_loss({**out, "dx": None, "dw": None}, x, w, t.int())
    _, dx, dw, tx, tw = bounds(x, w, t, again=1)
    close(out["dx"], dx, tx, "dx")
    close(out["dw"], dw, tw + U16 * dw.abs(), "dw")


# ------------------------------------- sizes at which the launches change

def skewed(seed, T, V):
    """Word frequencies like Zipf's, some runs of one word, and words of exactly 1 to 6, 32, 33 and 64 tokens."""
    u = torch.rand(T, generator=gen(seed), dtype=torch.float64)
    t = (torch.exp(u * math.log(V / 2)) - 1.0).long() + V // 2
    at = 0
    for i, n in enumerate((1, 2, 3, 4, 5, 6, 32, 33, 64, 4, 4, 4, 5, 5)):
        t[at:at + n] = i
        at += n
    t = t[torch.randperm(T, generator=gen(seed + 1))].clamp(max=V - 1)
    t[torch.randperm(T, generator=gen(seed + 2))[:T // 10]] = -100
    return t.int()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,d", [(2048, 300, 64), (2049, 300, 64), (4095, 1009, 72), (4096, 1009, 72), (4500, 5003, 72),
                                   (4109, 300, 264)])
def test_loss_of_many_tokens(dm, T, V, d):
    """Above 2048 tokens the row statistics take 32 rows a block and the targets are sorted in several chunks, from
    4096 on the words of up to 4 tokens are added one by one, and more than 16 pair rows make two groups of tiles."""
    x, w, t = randn(171, T, d), randn(172, V, d, scale=2.0 / math.sqrt(d)), skewed(173, T, V)
    out = run_loss(dm, cuda(x), cuda(w), cuda(t))
    assert dm.get_error() == 0
    check_loss(out, x, w, t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,piece", [(700, 256), (517, 256), (8, 0)])
def test_accumulation_over_pieces(dm, T, piece):
    V, d = 391, 88
    x, w = randn(174, T, d), randn(175, V, d, scale=0.3)
    t = torch.randint(0, V, (T,), generator=gen(176), dtype=torch.int32)
    t[::6] = -100
    g, base = randn(177, T, dtype=torch.float32), randn(178, V, d, dtype=torch.float32)
    n = dm.linear_cross_entropy_workspace_size(T, d, V, dw_dtype=torch.float32, piece=piece)
    out = dict(loss=empty(T, dtype=torch.float32), lse=empty(T, dtype=torch.float32), dx=empty(T, d, dtype=torch.bfloat16),
               dw=cuda(base.clone()))
    dm.linear_cross_entropy(cuda(x), cuda(w), cuda(t), out["loss"], out["lse"],
                            torch.full((n,), 255, dtype=torch.uint8, device="cuda"), dx=out["dx"], dw=out["dw"],
                            d_loss=cuda(g), accumulate=True, piece=piece)
    check_loss(out, x, w, t, d_loss=g, base=base)


# ------------------------------------------- where 16 bits are rounded to

def tight_case(T, V, d):
    x, w = randn(181, T, d), randn(182, V, d, scale=0.5 / math.sqrt(d))
    t = torch.randint(0, V, (T,), generator=gen(183), dtype=torch.int32)
    t[::5] = -100
    return x, w, t


def test_the_targets_part_in_16_bits_would_be_seen():
    """The bound is one that G rounded to bf16 as a whole would break (planted in the reference, no kernel)."""
    x, w, t = tight_case(60, 1009, 64)
    G, _, dw, _, tw = bounds(x, w, t)
    rounded = G.float().to(torch.bfloat16).double().t() @ x.double()
    assert bool(((rounded - dw).abs() > tw).any())


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,d", [(60, 1009, 64), (7, 1009, 64), (300, 5003, 136), (4100, 5003, 64)])
def test_the_targets_part_keeps_32_bits(dm, T, V, d):
    x, w, t = tight_case(T, V, d)
    _, dx, dw, tx, tw = bounds(x, w, t)
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dw=torch.float32)
    close(out["dx"], dx, tx, "dx")
    close(out["dw"], dw, tw, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [512, 4096, 8192])
def test_logits_of_sparse_rows(dm, d):
    """Rows of which a few columns are not zero, with logits that are exact in fp32: they come out within the mean
    that is given back for the tensor cores' truncation, (d / 16) 2^-26 of a logit (and a few roundings)."""
    T, V = 24, 130
    x, w = torch.zeros(T, d), torch.zeros(V, d)
    cols = torch.randperm(d, generator=gen(191))[:3]
    for i, c in enumerate(cols):
        x[:, c] = torch.randint(-8, 9, (T,), generator=gen(192 + i)).float()
        w[:, c] = torch.randint(-8, 9, (V,), generator=gen(195 + i)).float()
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=gen(198), dtype=torch.int32)
    loss, lse, _, _, l = ref_loss(x, w, t, -100)
    out = run_loss(dm, cuda(x), cuda(w), cuda(t), dx=False, dw=None)
    top = l.abs().amax(1)
    # besides: exp2's argument (two roundings of up to 1.45 top) and value, the sum and the logarithm
    e = ((d / 16) * 2.0 ** -26 + 8 * U32) * top + 4e-6
    close(out["lse"], lse, e, "lse")
    close(out["loss"], loss, 2 * e, "loss")


@pytest.mark.gpu
def test_clip_in_a_graph(dm):
    """Captured on a stream that the list has not seen, replayed with other gradients, and the list dropped."""
    g = cuda(randn(211, 70000))
    out, norm = torch.empty_like(g), empty(1, dtype=torch.float32)
    grads = dm.GradList([g], [out])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        dm.clip_grad_norm(grads, 1.0, norm)
    for seed in (212, 213):
        g.copy_(randn(seed, 70000))
        graph.replay()
        total = math.sqrt(float((g.double() ** 2).sum()))
        assert abs(float(norm) - total) <= 600 * U32 * total
        ref = g.cpu().double() / (total + 1e-6)
        close(out, ref, (U16 + 600 * U32) * ref.abs(), "clipped")
    del graph, grads
    torch.cuda.synchronize()
