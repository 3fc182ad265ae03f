"""Cases of the operators that stand beside a dropless MoE layer in a training step.

Three operators, each in its plain form (elementary torch operations in 32
bits) and as the calls a user makes of this package:

  norm           residual addition + root-mean-square norm, bf16 or 8-bit rows
  norm_backward  its gradient
  loss           the vocabulary head's softmax cross entropy, alone
  loss_grad      the same with the gradients of the rows and of the head
  clip           the global norm of many gradients, and their clipping
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 128      # columns that share a scale in the 8-bit rows
E4M3_MAX = 448.0
EPS = 1e-5       # of the norm
CLIP_EPS = 1e-6  # added to the gradients' norm
IGNORE = -100


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one token's row through a 4096-wide layer's norm: the smallest call, where latency counts
        {"name": "norm 1x4096", "op": "norm", "T": 1, "d": 4096, "bits8": False},
        # the Mixtral-shaped layer's batch
        {"name": "norm 8192x4096", "op": "norm", "T": 8192, "d": 4096, "bits8": False},
        # the fine-grained layer's width, a ragged batch, rows in 8 bits beside nothing else
        {"name": "norm8 4093x3584", "op": "norm", "T": 4093, "d": 3584, "bits8": True},
        # the MoE-XS layer's batch: short rows
        {"name": "norm_backward 8192x512", "op": "norm_backward", "T": 8192, "d": 512},
        # a long ragged batch of wide rows
        {"name": "norm_backward 16381x4096", "op": "norm_backward", "T": 16381, "d": 4096},
        # evaluation: losses of a batch over a large vocabulary, nothing kept
        {"name": "loss 2047x4096x128000", "op": "loss", "T": 2047, "d": 4096, "V": 128000, "ignored": 0.0},
        # the tiny layer's batch with a small odd vocabulary: latency
        {"name": "loss_grad 512x256x1009", "op": "loss_grad", "T": 512, "d": 256, "V": 1009, "ignored": 0.0},
        # the MoE-XS layer's batch under a 32000-word head: a short reduction for the logits
        {"name": "loss_grad 8192x512x32000", "op": "loss_grad", "T": 8192, "d": 512, "V": 32000, "ignored": 0.1},
        # the Mixtral-shaped layer's batch under a 32000-word head, an eighth of it prompt that does not count
        {"name": "loss_grad 8192x4096x32000", "op": "loss_grad", "T": 8192, "d": 4096, "V": 32000, "ignored": 0.125},
        # a large odd vocabulary over the fine-grained layer's width, a ragged batch: the largest
        {"name": "loss_grad 4095x3584x128003", "op": "loss_grad", "T": 4095, "d": 3584, "V": 128003, "ignored": 0.0},
        # the small parameters of a deep model (norm weights, gates): many tensors, at odd places of one bucket
        {"name": "clip 400 small", "op": "clip", "tensors": 400, "largest": 40000, "f32": True},
        # the weight gradients of one Mixtral-shaped layer: d x 8 F three times
        {"name": "clip 3x4096x114688", "op": "clip", "tensors": 3, "largest": 4096 * 114688, "f32": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, even over the logarithm (3072, a size of no workload here, left out)."""
    n = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
    n = max(lo, min(hi, n))
    return n + step if n == 3072 else n


MOST_LOSS = 4095 * 3584 * 128003


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "loss", "loss_grad", "loss_grad", "clip"))
    if op in ("norm", "norm_backward"):
        c = {"op": op, "T": _log(rng, 1, 16384), "d": _log(rng, 64, 8192, 8)}
        if op == "norm":
            c["bits8"] = rng.random() < 0.4
        return c
    if op == "clip":
        n = _log(rng, 1, 500)
        return {"op": op, "tensors": n, "largest": _log(rng, 1000, (1 << 30) // n), "f32": rng.random() < 0.5}
    d, V = _log(rng, 64, 4096, 8), _log(rng, 500, 130000)
    T = _log(rng, 1, min(8192, MOST_LOSS // (d * V)))
    return {"op": op, "T": T, "d": d, "V": V, "ignored": rng.choice((0.0, 0.1, 0.5))}


def _sizes(case):
    """Element counts of a clip case's tensors: the largest, then smaller ones down to single elements, mixed."""
    n, top = case["tensors"], case["largest"]
    if n <= 3:
        return [top] * n
    return [max(1, int(top * ((i * 37) % n + 1) ** 3 / n ** 3)) for i in range(n)]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["d"]
        out = 1 + 4 / GROUP if case["bits8"] else 2
        return {"bytes": n * (2 + 2 + 2 + out) + 2 * case["d"] + 4 * case["T"], "flops": 6 * n}
    if op == "norm_backward":
        n = case["T"] * case["d"]
        return {"bytes": n * 8 + 6 * case["d"] + 4 * case["T"], "flops": 10 * n}
    if op == "clip":
        n = sum(_sizes(case))
        small = n // 2 if case["f32"] else 0  # about half of a mixed set's elements are 32-bit
        return {"bytes": 4 * n + 4 * small, "flops": 3 * n}
    T, d, V = case["T"], case["d"], case["V"]
    io = 2 * T * d + 2 * V * d
    if op == "loss":
        return {"bytes": io + 12 * T, "flops": 2 * T * V * d}
    return {"bytes": 2 * io + 12 * T, "flops": 6 * T * V * d}


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
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        s = {"w": 1.0 + _randn(g, d, scale=0.1, dtype=torch.float32)}
        s["w"] = s["w"].to(torch.bfloat16)
        if op == "norm":
            # a residual stream grows along the depth: wider than what is added to it
            s["x"], s["res"] = _randn(g, T, d), _randn(g, T, d, scale=3.0)
        else:
            s["h"], s["dy"], s["dh"] = _randn(g, T, d, scale=3.0), _randn(g, T, d), _randn(g, T, d)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        return s
    if op == "clip":
        sizes = _sizes(case)
        kinds = [torch.float32 if case["f32"] and i % 2 else torch.bfloat16 for i in range(len(sizes))]
        s = {"views": [None] * len(sizes), "flat": {}, "out": {}}
        for dt in (torch.bfloat16, torch.float32):
            mine = [i for i in range(len(sizes)) if kinds[i] == dt]
            if mine:
                # one bucket a type; the tensors are its pieces, so most begin at odd places
                flat = _empty(sum(sizes[i] for i in mine), dtype=dt)
                step = 1 << 28
                for a in range(0, flat.numel(), step):
                    b = min(flat.numel(), a + step)
                    flat[a:b] = _randn(g, b - a, scale=2e-3, dtype=dt)
                s["flat"][str(dt)[6:]] = flat
                out = torch.zeros_like(flat)
                s["out"][str(dt)[6:]] = out
                at = 0
                for i in mine:
                    s["views"][i] = (flat[at:at + sizes[i]], out[at:at + sizes[i]])
                    at += sizes[i]
        n = sum(sizes)
        s["max_norm"] = 0.3 * 2e-3 * math.sqrt(n)  # about 0.3 of the norm: clipping happens
        return s
    T, d, V = case["T"], case["d"], case["V"]
    # rows as they come out of the final norm, a head whose logits spread over several units
    s = {"x": _randn(g, T, d), "w": _randn(g, V, d, scale=2.0 / math.sqrt(d))}
    # words come with Zipf-like frequencies
    u = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1).to(torch.int32)
    drop = torch.rand(T, generator=g, device=DEV) < case["ignored"]
    s["targets"] = torch.where(drop, torch.full_like(t, IGNORE), t)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "norm":
        T, d = case["T"], case["d"]
        s["h"], s["rstd"] = _empty(T, d), _empty(T, dtype=torch.float32)
        if case["bits8"]:
            s["q"] = _empty(T, d, dtype=torch.float8_e4m3fn)
            s["q_scale"] = _empty(T, -(-d // GROUP), dtype=torch.float32)
        else:
            s["y"] = _empty(T, d)
    elif op == "norm_backward":
        s["dx"], s["dw"] = _empty(case["T"], case["d"]), _empty(case["d"], dtype=torch.float32)
    elif op == "clip":
        s["norm"] = _empty(1, dtype=torch.float32)
    else:
        T, d, V = case["T"], case["d"], case["V"]
        s["loss"], s["lse"] = _empty(T, dtype=torch.float32), _empty(T, dtype=torch.float32)
        if op == "loss_grad":
            s["dx"], s["dw"] = _empty(T, d), _empty(V, d)
    if own:  # the workspaces and the table of tensors that a program makes once
        dm = _package()
        if op == "norm_backward":
            s["ws"] = _empty(dm.add_rms_norm_backward_workspace_size(case["T"], case["d"]), dtype=torch.uint8)
        elif op == "clip":
            s["grads"] = dm.GradList([a for a, _ in s["views"]], [b for _, b in s["views"]])
        elif op in ("loss", "loss_grad"):
            n = dm.linear_cross_entropy_workspace_size(case["T"], case["d"], case["V"], grad=op == "loss_grad")
            s["ws"] = _empty(n, dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------ run

def _run_own(s):
    dm, case = _package(), s["case"]
    op = case["op"]
    if op == "norm":
        if case["bits8"]:
            dm.add_rms_norm(s["x"], s["res"], s["w"], EPS, s["h"], None, rstd=s["rstd"], q=s["q"], q_scale=s["q_scale"])
            return {"h": s["h"], "rstd": s["rstd"], "q": s["q"], "q_scale": s["q_scale"]}
        dm.add_rms_norm(s["x"], s["res"], s["w"], EPS, s["h"], s["y"], rstd=s["rstd"])
        return {"h": s["h"], "rstd": s["rstd"], "y": s["y"]}
    if op == "norm_backward":
        dm.add_rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], s["dw"], s["ws"], dh=s["dh"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "clip":
        dm.clip_grad_norm(s["grads"], s["max_norm"], s["norm"], eps=CLIP_EPS)
        return {"norm": s["norm"], "out": s["out"]}
    if op == "loss":
        dm.linear_cross_entropy(s["x"], s["w"], s["targets"], s["loss"], s["lse"], s["ws"], ignore_index=IGNORE)
        return {"loss": s["loss"], "lse": s["lse"]}
    dm.linear_cross_entropy(s["x"], s["w"], s["targets"], s["loss"], s["lse"], s["ws"], dx=s["dx"], dw=s["dw"],
                            ignore_index=IGNORE)
    return {"loss": s["loss"], "lse": s["lse"], "dx": s["dx"], "dw": s["dw"]}


def _quantise(y):
    """Rows in 8 bits: groups of 128 columns, scale = largest magnitude / 448 (1 for a group of zeros)."""
    T, d = y.shape
    n = -(-d // GROUP)
    z = torch.zeros(T, n * GROUP, device=y.device, dtype=y.dtype)
    z[:, :d] = y
    z = z.view(T, n, GROUP)
    top = z.abs().amax(2)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return (z / scale[:, :, None]).view(T, n * GROUP)[:, :d], scale


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)  # the stream is kept in 16 bits
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd[:, None] * s["w"].float()
        if case["bits8"]:
            q, scale = _quantise(y)
            return {"h": h, "rstd": rstd, "q": q.to(torch.float8_e4m3fn), "q_scale": scale}
        return {"h": h, "rstd": rstd, "y": y.to(torch.bfloat16)}
    if op == "norm_backward":
        h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        u = dy * s["w"].float()
        dx = s["dh"].float() + r * (u - h * (r * r * (u * h).mean(1, keepdim=True)))
        return {"dx": dx.to(torch.bfloat16), "dw": (dy * h * r).sum(0)}
    if op == "clip":
        total = sum(f.float().square().sum() for f in s["flat"].values())
        norm = torch.sqrt(total)
        c = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
        return {"norm": norm.view(1), "out": {k: (f.float() * c).to(f.dtype) for k, f in s["flat"].items()}}
    x, w, t = s["x"].float(), s["w"].float(), s["targets"].long()
    counts = t != IGNORE
    at = torch.where(counts, t, torch.zeros_like(t))
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    sums = p.sum(1, keepdim=True)
    lse = (top + torch.log(sums)).view(-1)
    loss = torch.where(counts, lse - logits.gather(1, at[:, None]).view(-1), torch.zeros_like(lse))
    if op == "loss":
        return {"loss": loss, "lse": lse}
    g = counts.float() / counts.sum().clamp(min=1)
    p.mul_((g[:, None] / sums))
    p.scatter_add_(1, at[:, None], -g[:, None])
    return {"loss": loss, "lse": lse, "dx": (p @ w).to(torch.bfloat16), "dw": (p.t() @ x).to(torch.bfloat16)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """What run returns, from the definitions in 64 bits.  8-bit rows: the
    values before they are rounded to 8 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        h = (s["x"].double() + s["res"].double()).to(torch.bfloat16)
        hd = h.double()
        rstd = 1.0 / torch.sqrt((hd * hd).sum(1) / case["d"] + EPS)
        y = torch.einsum("td,t,d->td", hd, rstd, s["w"].double())
        if not case["bits8"]:
            return {"h": h.double(), "rstd": rstd, "y": y}
        n = -(-case["d"] // GROUP)
        scale = torch.stack([y[:, i * GROUP:(i + 1) * GROUP].abs().max(1).values for i in range(n)], 1) / E4M3_MAX
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        return {"h": h.double(), "rstd": rstd, "q": y / scale.repeat_interleave(GROUP, 1)[:, :case["d"]],
                "q_scale": scale}
    if op == "norm_backward":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
        n = h * r[:, None]  # the normalised rows
        gn = dy * w
        along = (gn * n).sum(1) / case["d"]
        return {"dx": s["dh"].double() + (gn - n * along[:, None]) * r[:, None], "dw": torch.einsum("td,td->d", dy, n)}
    if op == "clip":
        step = 1 << 27
        total = 0.0
        for f in s["flat"].values():
            for a in range(0, f.numel(), step):
                v = f[a:a + step].double()
                total += float(torch.dot(v, v))
        norm = math.sqrt(total)
        c = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor([norm], dtype=torch.float64),
                "out": {k: f.double().mul_(c) for k, f in s["flat"].items()}}
    T, d, V = case["T"], case["d"], case["V"]
    if (2 if op == "loss" else 6) * T * V * d > 16e12:  # about 20 seconds of 64-bit products
        return None
    t = s["targets"].long()
    keep = t >= 0
    n = max(1, int(keep.sum()))
    w = s["w"].double()
    loss, lse = torch.zeros(T, dtype=torch.float64, device=DEV), torch.empty(T, dtype=torch.float64, device=DEV)
    dx = torch.zeros(T, d, dtype=torch.float64, device=DEV) if op == "loss_grad" else None
    dw = torch.zeros(V, d, dtype=torch.float64, device=DEV) if op == "loss_grad" else None
    for a in range(0, T, 1024):  # in blocks of rows
        x = s["x"][a:a + 1024].double()
        l = torch.mm(x, w.t())
        lse[a:a + 1024] = torch.logsumexp(l, 1)
        k = keep[a:a + 1024].nonzero().view(-1)
        tk = t[a:a + 1024][k]
        loss[a + k] = lse[a + k] - l[k, tk]
        if dx is not None:
            G = torch.zeros_like(l)
            G[k] = torch.softmax(l[k], 1) / n
            G[k, tk] -= 1.0 / n
            dx[a:a + 1024] = torch.mm(G, w)
            dw.addmm_(G.t(), x)
    if dx is None:
        return {"loss": loss, "lse": lse}
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
