"""The operators that score and train the end of a model: layer_norm_rows, cross_entropy_rows and distill_rows with
their gradients, their cases and plain forms.

The final norm of hidden rows, the head's product and a loss over the whole vocabulary: the cross entropy of given
tokens (a prompt's log-probabilities, or a training step) or the distillation from a teacher's top logits (a draft
head that learns from what the sampler reports), then the way back to the hidden rows, the head and the norm.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MOST = 1024 * 248320 * 2048      # rows x vocabulary x width of the largest loss


def listed():
    return [
        # one request's next token: the last hidden row, with the residual's addition
        dict(name="norm one row", op="norm", T=1, H=4096, type="bf16", residual=True, bias=True),
        # prompts of a full batch inside a layer
        dict(name="norm prompts", op="norm", T=8192, H=8192, type="bf16", residual=True, bias=True),
        # a ragged width in 32 bits, the way back
        dict(name="norm grad odd f32", op="norm_grad", T=1021, H=5003, type="f32", residual=False, bias=True),
        # the way back of a full batch, a gradient that goes around the norm joining it
        dict(name="norm grad prompts", op="norm_grad", T=8192, H=8192, type="bf16", residual=True, bias=True),
        # the log-probability of one token, a small head
        dict(name="score one row", op="cross_entropy", T=1, V=32000, H=1024, skip=0.0),
        # a token of each of 64 slots, the large head
        dict(name="score 64 slots", op="cross_entropy", T=64, V=248320, H=2048, skip=0.0),
        # ragged prompts of several requests, a quarter of the rows not asked for, an odd vocabulary
        dict(name="score prompts", op="cross_entropy", T=4099, V=151001, H=1024, skip=0.25),
        # a step on a few rows with the large head: loss and both gradients
        dict(name="step few rows", op="cross_entropy_grad", T=96, V=248320, H=2048, skip=0.0),
        # a full training step: the rows of the questions left out
        dict(name="step", op="cross_entropy_grad", T=4096, V=32000, H=4096, skip=0.125),
        # how far a draft head is from its teacher, on a verify window of eight slots; an odd vocabulary
        dict(name="distill window", op="distill", T=40, V=151001, H=1024, K=20, skip=0.1, temperature=1.0),
        # a draft head's step from the 20 alternatives that the sampler reports, a small head
        dict(name="distill step", op="distill_grad", T=2048, V=32000, H=2048, K=20, skip=0.1, temperature=1.0),
        # the same with the large head, 64 alternatives and a temperature
        dict(name="distill step large", op="distill_grad", T=1024, V=248320, H=2048, K=64, skip=0.1, temperature=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "cross_entropy", "cross_entropy_grad", "distill", "distill_grad"))
    if op in ("norm", "norm_grad"):
        H = _log(rng, 64, 8192)
        kind = rng.choice(("bf16", "f32"))
        T = min(_log(rng, 1, 8192), 8192 * 8192 // H)
        return dict(op=op, T=T if kind == "bf16" else max(1, T // 2), H=H, type=kind, residual=rng.random() < 0.6, bias=rng.random() < 0.7)
    V, H = _log(rng, 1000, 248320), 8 * _log(rng, 32, 512)
    T = max(1, min(_log(rng, 1, 4099), MOST // (V * H)))
    c = dict(op=op, T=T, V=V, H=H, skip=rng.choice((0.0, 0.1, 0.25, 0.5)))
    if op.startswith("distill"):
        c["K"] = rng.choice((1, 5, 8, 20, 37, 64))
        c["temperature"] = rng.choice((1.0, 0.7, 2.0))
    return c


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, to=torch.float32, by=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(by).to(to)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    T, H = case["T"], case["H"]
    if case["op"] in ("norm", "norm_grad"):
        t = TYPES[case["type"]]
        s["x"] = normal(T, H, to=t)
        s["x"][:, :: 97] *= 20  # a few channels of a hidden row are far larger than the others
        s["w"] = (1 + normal(H, by=0.2)).to(t)
        s["b"] = normal(H, to=t, by=0.1) if case["bias"] else None
        s["r"] = normal(T, H, to=t, by=2.0) if case["residual"] else None
        s["eps"] = 1e-5
        if case["op"] == "norm_grad":  # r is the gradient that goes around the norm
            s["dy"] = normal(T, H, to=t, by=0.1)
            x = s["x"].double()
            mean = x.mean(1, keepdim=True)
            s["mean"], s["rstd"] = mean[:, 0].float(), ((x - mean).square().mean(1) + s["eps"]).rsqrt().float()
        return s
    V, n = case["V"], max(1, case["T"] - int(case["T"] * case["skip"]))
    s["w"] = torch.randn(V, H, generator=g, device="cuda", dtype=torch.bfloat16).mul_(2 * H ** -0.5)  # logits of about +-2 ...
    ids = torch.randint(0, V, (T, case.get("K", 1)), generator=g, device="cuda", dtype=torch.int32)
    s["x"] = (normal(T, H) + uniform(T, 1, lo=0.0, hi=4.0) * s["w"][ids[:, 0].long()].float()).to(torch.bfloat16)  # ... and up to +16 for the token
    out = torch.randperm(T, generator=g, device="cuda")[n:]  # rows that nobody asks for
    s["ids"], s["teacher"], s["temperature"] = ids, None, case.get("temperature", 1.0)
    if case["op"].startswith("distill"):
        K = case["K"]
        s["teacher"] = torch.sort(normal(T, K, by=3.0) + 8.0, dim=1, descending=True).values
        have = torch.where(uniform(T, 1) < 0.2, uniform(T, 1, lo=1.0, hi=K + 1.0).int(), K)  # some rows have fewer alternatives
        s["ids"] = torch.where(torch.arange(K, device="cuda") < have, ids, -1)
        s["teacher"][uniform(T, K) < 0.02] = -math.inf  # a teacher that rules a token out
    s["ids"][out] = -1
    if s["teacher"] is None:
        s["ids"] = s["ids"][:, 0].contiguous()
    s["g"] = torch.full((T,), 1.0 / n, device="cuda")  # of the mean over the rows asked for
    return s


# ------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        import request_token_sampling_gb300 as G
        if s["op"] == "norm":
            o = G.layer_norm_rows(s["x"], s["w"], bias=s["b"], residual=s["r"], eps=s["eps"])
            return {k: o[k] for k in ("y", "mean", "rstd", "residual") if k in o}
        if s["op"] == "norm_grad":
            o = G.layer_norm_grad(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dresidual=s["r"], bias=s["bias"])
            return {k: o[k] for k in ("dx", "dweight", "dbias") if k in o}
        if s["teacher"] is None:
            o = G.cross_entropy_rows(s["x"], s["w"], s["ids"])
            if s["op"] == "cross_entropy_grad":
                o = dict(o, **G.cross_entropy_grad(s["x"], s["w"], s["ids"], o["lse"], s["g"]))
        else:
            o = G.distill_rows(s["x"], s["w"], s["ids"], s["teacher"], temperature=s["temperature"])
            if s["op"] == "distill_grad":
                o = dict(o, **G.distill_grad(s["x"], s["w"], s["ids"], s["teacher"], o["lse"], s["g"], temperature=s["temperature"]))
        return {k: o[k] for k in ("loss", "lse", "dx", "dw") if k in o}
    return {"norm": _norm, "norm_grad": _norm_grad}.get(s["op"], _loss)(s)


def _norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean = h.mean(1, keepdim=True)
    d = h - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    o = {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["r"] is not None:
        o["residual"] = h.to(s["x"].dtype)
    return o


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    v = (s["x"].float() - s["mean"][:, None]) * rstd
    a = dy * s["w"].float()
    dx = (a - a.mean(1, keepdim=True) - v * (a * v).mean(1, keepdim=True)) * rstd
    if s["r"] is not None:
        dx = dx + s["r"].float()
    o = {"dx": dx.to(s["x"].dtype), "dweight": (dy * v).sum(0).to(s["w"].dtype)}
    if s["bias"]:
        o["dbias"] = dy.sum(0).to(s["w"].dtype)
    return o


def _loss(s):
    """A cross entropy is the distillation from a teacher that knows one token alone."""
    t = s["temperature"]
    x, w = s["x"].float(), s["w"].float()
    ids = s["ids"].reshape(x.shape[0], -1)
    teacher = torch.zeros(ids.shape, device=x.device) if s["teacher"] is None else s["teacher"] / t
    there = (ids >= 0) & (teacher != -math.inf)
    teacher = torch.where(there, teacher, torch.full_like(teacher, -math.inf))
    asked = there.any(1, keepdim=True)
    logq = torch.log_softmax(torch.where(asked, teacher, torch.zeros_like(teacher)), 1)
    q = torch.where(asked, torch.exp(logq), torch.zeros_like(logq))
    at = ids.clamp_min(0).long()
    z = x @ w.T / t
    lse = torch.logsumexp(z, 1, keepdim=True)
    each = torch.where(q > 0, q * (logq - (z.gather(1, at) - lse)), torch.zeros_like(q))
    nothing = torch.zeros_like(lse)
    o = {"loss": torch.where(asked, t * t * each.sum(1, keepdim=True), nothing)[:, 0], "lse": torch.where(asked, lse, nothing)[:, 0]}
    if s["op"].endswith("_grad"):
        d = torch.exp(z - lse).scatter_add_(1, at, -q) * torch.where(asked, t * s["g"][:, None], nothing)
        o["dx"], o["dw"] = (d @ w).to(s["x"].dtype), (d.T @ x).to(s["w"].dtype)
    return o


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, H = case["T"], case["H"]
    if case["op"] in ("norm", "norm_grad"):
        size = {"f32": 4, "bf16": 2}[case["type"]]
        if case["op"] == "norm":
            return {"bytes": T * H * size * (2 + 2 * case["residual"]) + 8 * T + H * size * (1 + case["bias"]), "flops": 8 * T * H}
        return {"bytes": T * H * size * (3 + case["residual"]) + 8 * T + H * size * (2 + case["bias"]), "flops": 13 * T * H}
    V, K = case["V"], case.get("K", 1)
    n = max(1, T - int(T * case["skip"]))
    grad = case["op"].endswith("_grad")
    read = 2 * H * (V + n) + 4 * T * K * (2 if "K" in case else 1) + 8 * T
    # the logits, and on the way back the two products of their gradient (that they are not kept, and so are taken again, is the form's choice)
    return {"bytes": read + grad * (2 * H * (V + T) + 4 * T), "flops": (2 + 4 * grad) * n * V * H}


# ------------------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    T, H = x.shape
    if case["op"] == "norm":
        h = x if s["r"] is None else x + s["r"].double()
        var, mean = torch.var_mean(h, dim=1, correction=0)
        y = s["w"].double() * ((h - mean.unsqueeze(1)) / (var + s["eps"]).sqrt().unsqueeze(1))
        o = {"y": y if s["b"] is None else y + s["b"].double(), "mean": mean, "rstd": 1 / (var + s["eps"]).sqrt()}
        return o if s["r"] is None else o | {"residual": h}
    if case["op"] == "norm_grad":
        # y = u / n with u = (x - mean) and n = sqrt(|u|^2 / H + eps): dx is what is left of a / n without its mean and its part along u
        var, mean = torch.var_mean(x, dim=1, correction=0)
        u, n = x - mean.unsqueeze(1), (var + s["eps"]).sqrt().unsqueeze(1)
        dy = s["dy"].double()
        a = dy * s["w"].double()
        dx = (a - a.sum(1, keepdim=True) / H) / n - u * ((a * u).sum(1, keepdim=True) / (H * n ** 3))
        o = {"dx": dx if s["r"] is None else dx + s["r"].double(), "dweight": torch.einsum("th,th->h", dy, u / n)}
        return o | {"dbias": dy.sum(0)} if s["bias"] else o
    w, t = s["w"].double(), float(s["temperature"])
    p = torch.mm(x, w.t()).div_(t)
    top = p.amax(1, keepdim=True)
    lse = (p - top).exp_().sum(1).log().add(top[:, 0])
    q = torch.zeros_like(p)  # the teacher's probabilities over the whole vocabulary
    loss = torch.zeros(T, dtype=torch.float64, device=x.device)
    asked = torch.zeros(T, dtype=torch.bool, device=x.device)
    ids = s["ids"].view(T, -1).cpu()
    gone = torch.zeros_like(ids, dtype=torch.bool) if s["teacher"] is None else s["teacher"].cpu() == -math.inf
    for r in range(T):
        have = [j for j in range(ids.shape[1]) if ids[r, j] >= 0 and not gone[r, j]]
        if not have:
            continue
        asked[r] = True
        at = ids[r, have].long().to(x.device)
        l = torch.zeros(len(have), dtype=torch.float64, device=x.device) if s["teacher"] is None else s["teacher"][r, have].double() / t
        mine = torch.softmax(l, 0)
        some = mine > 0
        loss[r] = t * t * (mine[some] * (mine[some].log() - p[r, at[some]] + lse[r])).sum()
        q[r].index_add_(0, at, mine)
    o = {"loss": loss, "lse": torch.where(asked, lse, 0.0)}
    if case["op"].endswith("_grad"):
        d = p.sub_(lse.unsqueeze(1)).exp_().sub_(q).mul_((t * s["g"].double() * asked).unsqueeze(1))
        o["dx"], o["dw"] = d.mm(w), d.t().mm(x)
    return o
