"""Cases of the operators that turn a dropless MoE layer into a block of a model.

Three operators and their gradients, each in its plain form (elementary torch
operations in 32 bits, choices between experts in 64) and as the calls a user
makes of this package:

  route            choice of experts by softmax or sigmoid scores, a bias for
                   balance, groups, top-k, renormalised and scaled weights
  route_backward   gradient of the weights with respect to the logits
  norm             the norm after a block, its gate, the scaled residual
                   stream and the norm before the next block
  norm_backward    its gradient
  linear           a dense product with bias, activation and residual: the two
                   halves of a shared expert
  linear_backward  its gradient
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5  # of the norms


# ---------------------------------------------------------------------- cases

def _route(T, E, k, scores, groups=1, top_groups=1, bias=True, renorm=True, scale=1.0):
    return {"T": T, "E": E, "k": k, "scores": scores, "groups": groups, "top_groups": top_groups, "bias": bias,
            "renorm": renorm, "scale": scale}


def listed():
    return [
        # one generated token among 256 experts in 8 groups: the smallest call, where latency counts
        {"name": "route 1x256", "op": "route", **_route(1, 256, 8, "sigmoid", 8, 4, scale=2.5)},
        # the MoE-XS layer's batch: one expert a token, softmax scores, balanced by the bias alone
        {"name": "route 8192x64", "op": "route", **_route(8192, 64, 1, "softmax", renorm=False)},
        # a long ragged batch over many small experts in groups
        {"name": "route 16381x256", "op": "route", **_route(16381, 256, 8, "sigmoid", 8, 4, scale=2.5)},
        # the fine-grained layer's experts, a ragged batch
        {"name": "route_backward 4095x64", "op": "route_backward", **_route(4095, 64, 8, "softmax")},
        # many small experts, a long batch
        {"name": "route_backward 16384x256", "op": "route_backward", **_route(16384, 256, 8, "sigmoid", 8, 4, scale=2.5)},
        # one generated token's row between two blocks of a 4096-wide model
        {"name": "norm 1x4096", "op": "norm", "T": 1, "d": 4096, "gate": "none", "scale": 1.0},
        # the Mixtral-shaped layer's batch, every token with a gate of its own
        {"name": "norm 8192x4096", "op": "norm", "T": 8192, "d": 4096, "gate": "row", "scale": 0.7},
        # the MoE-XS layer's width, a ragged batch, one learned gate for all tokens: short rows
        {"name": "norm_backward 8191x512", "op": "norm_backward", "T": 8191, "d": 512, "gate": "one", "scale": 1.0},
        # the Mixtral-shaped layer's batch
        {"name": "norm_backward 8192x4096", "op": "norm_backward", "T": 8192, "d": 4096, "gate": "row", "scale": 0.7},
        # one generated token through the second half of a shared expert, onto what the routed ones gave
        {"name": "linear 1x14336x4096", "op": "linear", "M": 1, "K": 14336, "N": 4096, "act": "none", "bias": True,
         "residual": True},
        # a training batch through its first half, the derivative kept: the largest
        {"name": "linear 8192x4096x14336", "op": "linear", "M": 8192, "K": 4096, "N": 14336, "act": "gelu", "bias": True,
         "residual": False},
        # the gradients of a half of the fine-grained layer's width, a ragged batch
        {"name": "linear_backward 4093x3584x10240", "op": "linear_backward", "M": 4093, "K": 3584, "N": 10240,
         "act": "silu", "bias": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, even over the logarithm."""
    n = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
    return max(lo, min(hi, n))


MOST_LINEAR = 8192 * 4096 * 14336


def draw(rng):
    op = rng.choice(("route", "route_backward", "norm", "norm_backward", "linear", "linear_backward"))
    if op in ("route", "route_backward"):
        groups = rng.choice((1, 1, 2, 3, 4, 8, 16))
        each = _log(rng, 2, 512 // groups)
        E = groups * each
        top = rng.randint(1, groups)
        k = rng.randint(1, min(top * each, 12))
        return {"op": op, **_route(_log(rng, 1, 16384), E, k, rng.choice(("softmax", "sigmoid")), groups, top,
                                   rng.random() < 0.8, rng.random() < 0.7, rng.choice((1.0, 2.5)))}
    if op in ("norm", "norm_backward"):
        return {"op": op, "T": _log(rng, 1, 16384), "d": _log(rng, 64, 8192, 8),
                "gate": rng.choice(("none", "row", "one")), "scale": rng.choice((1.0, 0.7))}
    K, N = _log(rng, 64, 14336, 8), _log(rng, 64, 14336, 8)
    most = MOST_LINEAR // (K * N) // (1 if op == "linear" else 2)
    c = {"op": op, "M": _log(rng, 1, min(8192, most)), "K": K, "N": N, "act": rng.choice(("none", "gelu", "silu")),
         "bias": rng.random() < 0.7}
    if op == "linear":
        c["residual"] = rng.random() < 0.5
    return c


def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "route":
            return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
        return {"bytes": 8 * T * E + 8 * T * k, "flops": 8 * T * E}
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        gate = {"none": 0, "row": T, "one": 1}[case["gate"]]
        if op == "norm":
            return {"bytes": 8 * T * d + 4 * d + 8 * T + 4 * gate, "flops": 10 * T * d}
        return {"bytes": 12 * T * d + 12 * d + 8 * T + 8 * gate, "flops": 24 * T * d}
    M, K, N = case["M"], case["K"], case["N"]
    keeps = case["act"] != "none"
    bias = N if case["bias"] else 0
    if op == "linear":
        return {"bytes": 2 * (M * K + K * N + M * N * (1 + keeps + case["residual"]) + bias), "flops": 2 * M * K * N}
    return {"bytes": 2 * (2 * M * K + 2 * K * N + M * N * (1 + keeps)) + 4 * bias, "flops": 4 * M * K * N}


# -------------------------------------------------------------------- prepare

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, device=DEV, dtype=dtype)


def _package():
    import dropless_moe_block_gb300 as dm
    return dm


def _inputs(case, seed):
    """The operator's inputs alone, from the seed."""
    op, g = case["op"], _gen(seed)
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        s = {"logits": _randn(g, T, E, dtype=torch.float32), "bias": None}
        if case["bias"]:  # what a few thousand steps of its update leave, a small part of the scores
            s["bias"] = _randn(g, E, scale=0.02 if case["scores"] == "sigmoid" else 0.5 / E, dtype=torch.float32)
        if op == "route_backward":
            s["expert_idx"] = _choose(s["logits"], s["bias"], case).to(torch.int32)
            s["d_gate"] = _randn(g, T, k, dtype=torch.float32)
        return s
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        s = {"w_post": (1.0 + _randn(g, d, scale=0.1, dtype=torch.float32)).to(torch.bfloat16),
             "w_pre": (1.0 + _randn(g, d, scale=0.1, dtype=torch.float32)).to(torch.bfloat16), "gate": None}
        if case["gate"] != "none":
            s["gate"] = torch.sigmoid(_randn(g, T if case["gate"] == "row" else 1, dtype=torch.float32))
        # a block's output, and a residual stream, which grows along the depth
        s["u"] = _randn(g, T, d, scale=0.5)
        if op == "norm":
            s["x"] = _randn(g, T, d, scale=3.0)
            return s
        s["h"], s["dy"], s["dh"] = _randn(g, T, d, scale=3.0), _randn(g, T, d), _randn(g, T, d)
        s["rstd_u"] = torch.rsqrt(s["u"].float().square().mean(1) + EPS)
        s["rstd_h"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s = {"x": _randn(g, M, K), "w": _randn(g, K, N, scale=K ** -0.5), "bias": None}
    if op == "linear":
        if case["bias"]:
            s["bias"] = _randn(g, N, scale=0.1)
        s["residual"] = _randn(g, M, N) if case["residual"] else None
    else:
        s["dy"], s["deriv"] = _randn(g, M, N), None
        if case["act"] != "none":  # what the forward pass kept
            s["deriv"] = _act(_randn(g, M, N, dtype=torch.float32), case["act"])[1].to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op, f32 = case["op"], torch.float32
    if op == "route":
        T, k = case["T"], case["k"]
        s["expert_idx"], s["gate_w"] = _empty(T, k, dtype=torch.int32), _empty(T, k, dtype=f32)
    elif op == "route_backward":
        s["d_logits"] = _empty(case["T"], case["E"], dtype=f32)
    elif op == "norm":
        T, d = case["T"], case["d"]
        s["h"], s["y"] = _empty(T, d), _empty(T, d)
        s["rstd_u"], s["rstd_h"] = _empty(T, dtype=f32), _empty(T, dtype=f32)
    elif op == "norm_backward":
        T, d = case["T"], case["d"]
        s["du"], s["dx"] = _empty(T, d), _empty(T, d)
        s["dw_post"], s["dw_pre"] = _empty(d, dtype=f32), _empty(d, dtype=f32)
        s["d_gate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    elif op == "linear":
        s["y"] = _empty(case["M"], case["N"])
        s["deriv"] = None if case["act"] == "none" else _empty(case["M"], case["N"])
    else:
        s["dx"], s["dw"] = _empty(case["M"], case["K"]), _empty(case["K"], case["N"])
        s["db"] = _empty(case["N"], dtype=f32) if case["bias"] else None
    if own:  # the workspaces that a program makes once
        dm = _package()
        n = 0
        if op == "norm_backward":
            n = dm.sandwich_norm_backward_workspace_size(case["T"], case["d"])
        elif op == "linear":
            n = dm.linear_workspace_size(case["M"], case["K"], case["N"])
        elif op == "linear_backward":
            n = dm.linear_backward_workspace_size(case["M"], case["K"], case["N"])
        s["ws"] = _empty(max(n, 16), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------ run

def _run_own(s):
    dm, case = _package(), s["case"]
    op = case["op"]
    if op == "route":
        dm.route_balanced(s["logits"], case["k"], s["expert_idx"], s["gate_w"], bias=s["bias"], scores=case["scores"],
                          groups=case["groups"], top_groups=case["top_groups"], renormalize=case["renorm"],
                          scale=case["scale"])
        return {"expert_idx": s["expert_idx"], "gate_w": s["gate_w"]}
    if op == "route_backward":
        dm.route_balanced_backward(s["logits"], s["expert_idx"], s["d_gate"], s["d_logits"], scores=case["scores"],
                                   renormalize=case["renorm"], scale=case["scale"])
        return {"d_logits": s["d_logits"]}
    if op == "norm":
        dm.sandwich_norm(s["u"], s["x"], s["w_post"], s["w_pre"], EPS, s["h"], s["y"], gate=s["gate"],
                         scale=case["scale"], rstd_u=s["rstd_u"], rstd_h=s["rstd_h"])
        return {"h": s["h"], "y": s["y"], "rstd_u": s["rstd_u"], "rstd_h": s["rstd_h"]}
    if op == "norm_backward":
        dm.sandwich_norm_backward(s["dy"], s["u"], s["h"], s["w_post"], s["w_pre"], s["rstd_u"], s["rstd_h"], s["du"],
                                  s["dx"], s["dw_post"], s["dw_pre"], s["ws"], dh=s["dh"], gate=s["gate"],
                                  d_gate=s["d_gate"], scale=case["scale"])
        out = {"du": s["du"], "dx": s["dx"], "dw_post": s["dw_post"], "dw_pre": s["dw_pre"]}
        return out if s["gate"] is None else {**out, "d_gate": s["d_gate"]}
    if op == "linear":
        dm.linear(s["x"], s["w"], s["y"], s["ws"], bias=s["bias"], act=case["act"], deriv=s["deriv"],
                  residual=s["residual"])
        return {"y": s["y"]} if s["deriv"] is None else {"y": s["y"], "deriv": s["deriv"]}
    dm.linear_backward(s["dy"], s["x"], s["w"], s["dx"], s["dw"], s["ws"], dbias=s["db"], deriv=s["deriv"])
    out = {"dx": s["dx"], "dw": s["dw"]}
    return out if s["db"] is None else {**out, "db": s["db"]}


def _scores(z, case):
    return torch.sigmoid(z) if case["scores"] == "sigmoid" else torch.softmax(z, 1)


def _choose(logits, bias, case):
    """The chosen experts, best first, ties to the lower one.  Choices are
    between values that may lie close to one another: in 64 bits, and without
    a bias on the logits themselves, whose order the scores keep."""
    T, E = logits.shape
    z = logits.double()
    if bias is None:
        c = z
    else:
        c = _scores(z, case) + bias.double()
    G = case["groups"]
    if case["top_groups"] < G:
        of = c if bias is not None else _scores(z, case)
        worth = of.view(T, G, E // G).topk(min(2, E // G), dim=2).values.sum(2)
        best = worth.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, best, True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]


def _act(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, None
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    p = torch.sigmoid(z)
    return z * p, p * (1.0 + z * (1.0 - p))


def _run_plain(s):
    case = s["case"]
    op, bf = case["op"], torch.bfloat16
    if op == "route":
        idx = _choose(s["logits"], s["bias"], case)
        w = _scores(s["logits"], case).gather(1, idx)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"expert_idx": idx.to(torch.int32), "gate_w": w * case["scale"]}
    if op == "route_backward":
        idx, p = s["expert_idx"].long(), _scores(s["logits"], case)
        w, d = p.gather(1, idx), s["d_gate"] * case["scale"]
        if case["renorm"]:
            total = w.sum(1, keepdim=True)
            d = (d - (d * w).sum(1, keepdim=True) / total) / total
        dp = torch.zeros_like(p).scatter_(1, idx, d)
        if case["scores"] == "sigmoid":
            return {"d_logits": dp * p * (1.0 - p)}
        return {"d_logits": p * (dp - (dp * p).sum(1, keepdim=True))}
    if op == "norm":
        u = s["u"].float()
        rstd_u = torch.rsqrt(u.square().mean(1) + EPS)
        n = u * rstd_u[:, None] * s["w_post"].float()
        if s["gate"] is not None:
            n = n * s["gate"][:, None]
        h = (case["scale"] * s["x"].float() + n).to(bf)  # the stream is kept in 16 bits
        hf = h.float()
        rstd_h = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd_h[:, None] * s["w_pre"].float()
        return {"h": h, "y": y.to(bf), "rstd_u": rstd_u, "rstd_h": rstd_h}
    if op == "norm_backward":
        u, h, dy = s["u"].float(), s["h"].float(), s["dy"].float()
        ru, rh = s["rstd_u"][:, None], s["rstd_h"][:, None]
        g = dy * s["w_pre"].float()
        dH = s["dh"].float() + rh * (g - h * (rh * rh * (g * h).mean(1, keepdim=True)))
        n = u * ru
        v = dH * s["w_post"].float()
        along = v * n
        gate = 1.0 if s["gate"] is None else s["gate"][:, None]
        du = ru * gate * (v - n * along.mean(1, keepdim=True))
        out = {"du": du.to(bf), "dx": (case["scale"] * dH).to(bf), "dw_post": (gate * dH * n).sum(0),
               "dw_pre": (dy * h * rh).sum(0)}
        if s["gate"] is not None:
            out["d_gate"] = along.sum(1) if case["gate"] == "row" else along.sum().view(1)
        return out
    if op == "linear":
        z = s["x"].float() @ s["w"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y, deriv = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(bf)} if deriv is None else {"y": y.to(bf), "deriv": deriv.to(bf)}
    dz = s["dy"].float()
    if s["deriv"] is not None:
        dz = dz * s["deriv"].float()
    out = {"dx": (dz @ s["w"].float().t()).to(bf), "dw": (s["x"].float().t() @ dz).to(bf)}
    return {**out, "db": dz.sum(0)} if case["bias"] else out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """What run returns, from the definitions in 64 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("route", "route_backward"):
        z = s["logits"].double()
        T, E = z.shape
        if case["scores"] == "softmax":
            p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        else:
            p = 1.0 / (1.0 + torch.exp(-z))
        if op == "route":
            # rounds of taking the best of what is left
            c = p.clone() if s["bias"] is None else p + s["bias"].double()
            left = torch.ones(T, E, dtype=torch.bool, device=DEV)
            size = E // case["groups"]
            if case["top_groups"] < case["groups"]:
                per = c.view(T, case["groups"], size)
                first = per.max(2).values
                worth = first
                if size > 1:
                    rest = per.clone()
                    rest.scatter_(2, per.argmax(2, keepdim=True), -math.inf)
                    worth = first + rest.max(2).values
                for _ in range(case["groups"] - case["top_groups"]):  # the worst goes, of equal ones the last
                    drop = case["groups"] - 1 - worth.flip(1).argmin(1)
                    worth[torch.arange(T, device=DEV), drop] = math.inf
                left &= ~torch.isinf(worth).repeat_interleave(size, 1)
            order = c if s["bias"] is not None else z.clone()
            order = torch.where(left, order, torch.full_like(order, -math.inf))
            idx = torch.empty(T, case["k"], dtype=torch.int64, device=DEV)
            for j in range(case["k"]):
                best = order.max(1, keepdim=True).values
                idx[:, j] = (order == best).int().argmax(1)
                order.scatter_(1, idx[:, j:j + 1], -math.inf)
            w = torch.stack([p[torch.arange(T, device=DEV), idx[:, j]] for j in range(case["k"])], 1)
            if case["renorm"]:
                w = w / w.sum(1)[:, None]
            return {"expert_idx": idx.to(torch.int32), "gate_w": case["scale"] * w}
        # the Jacobian of the weights, row by row of the chosen experts
        idx, d = s["expert_idx"].long(), s["d_gate"].double()
        G = torch.zeros_like(p).scatter_(1, idx, d)
        on = torch.zeros_like(p).scatter_(1, idx, 1.0)
        slope = p if case["scores"] == "softmax" else p * (1.0 - p)  # of a score by its own logit, up to softmax's sum
        if case["renorm"]:
            total = (on * p).sum(1, keepdim=True)
            w = on * p / total
            mean = (w * G).sum(1, keepdim=True)
            return {"d_logits": case["scale"] * on * slope / total * (G - mean)}
        if case["scores"] == "sigmoid":
            return {"d_logits": case["scale"] * G * slope}
        return {"d_logits": case["scale"] * p * (G - torch.einsum("te,te->t", G, p)[:, None])}
    if op in ("norm", "norm_backward"):
        u, d = s["u"].double(), case["d"]
        a, b = s["w_post"].double(), s["w_pre"].double()
        gate = torch.ones(1, dtype=torch.float64, device=DEV) if s["gate"] is None else s["gate"].double()
        if op == "norm":
            ru = 1.0 / torch.sqrt((u * u).sum(1) / d + EPS)
            h = (case["scale"] * s["x"].double() + torch.einsum("td,t,d->td", u, ru * gate, a)).to(torch.bfloat16)
            hd = h.double()
            rh = 1.0 / torch.sqrt((hd * hd).sum(1) / d + EPS)
            return {"h": hd, "y": torch.einsum("td,t,d->td", hd, rh, b), "rstd_u": ru, "rstd_h": rh}
        ru, rh = s["rstd_u"].double()[:, None], s["rstd_h"].double()[:, None]
        nu, nh = u * ru, s["h"].double() * rh  # the normalised rows
        gy = s["dy"].double() * b
        dH = s["dh"].double() + (gy - nh * ((gy * nh).sum(1, keepdim=True) / d)) * rh
        gn = dH * a * gate[:, None]
        out = {"du": (gn - nu * ((gn * nu).sum(1, keepdim=True) / d)) * ru, "dx": case["scale"] * dH,
               "dw_post": torch.einsum("td,td->d", dH * gate[:, None], nu),
               "dw_pre": torch.einsum("td,td->d", s["dy"].double(), nh)}
        if s["gate"] is not None:
            rows = torch.einsum("td,td,d->t", dH, nu, a)
            out["d_gate"] = rows if case["gate"] == "row" else rows.sum().view(1)
        return out
    M, K, N = case["M"], case["K"], case["N"]
    x, w = s["x"].double(), s["w"].double()
    if op == "linear":
        z = torch.mm(x, w)
        if s["bias"] is not None:
            z += s["bias"].double()
        deriv = None
        if case["act"] == "gelu":
            phi = 0.5 * torch.erfc(-z / math.sqrt(2.0))
            y, deriv = z * phi, phi + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
        elif case["act"] == "silu":
            q = 1.0 / (1.0 + torch.exp(-z))
            y, deriv = z * q, q + z * q * (1.0 - q)
        else:
            y = z
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y} if deriv is None else {"y": y, "deriv": deriv}
    dz = s["dy"].double() if s["deriv"] is None else s["dy"].double() * s["deriv"].double()
    out = {"dx": torch.mm(dz, w.t()), "dw": torch.mm(x.t(), dz)}
    return {**out, "db": torch.einsum("mn->n", dz)} if case["bias"] else out
