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
