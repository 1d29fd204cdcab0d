"""The operators around the sampler: norm_rows, project_rows and draw_rows, their cases and plain forms.

A decode step ends in: the final norm of the hidden rows (with the residual's addition, in 8 bits where the
head's weights are), the head's product with each request's low-rank adapter, and the draw of a token per row
from random numbers that the caller brings.  The same projection runs over whole prompts.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
SCALE_MIN = 2.0 ** -100
ONE = 2.0 ** 43          # the whole number that a weight of 1 stands for
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": F8}


def listed():
    return [
        # one request's next token: the last hidden row, for an 8-bit head
        dict(name="norm one row", op="norm", T=1, H=4096, type="bf16", residual=True, y=False, f8=True),
        # 64 slots decode at once
        dict(name="norm 64 slots", op="norm", T=64, H=5120, type="bf16", residual=True, y=False, f8=True),
        # a ragged width in 32 bits, nothing to add, both outputs (an adapter that reads the unrounded row)
        dict(name="norm odd f32", op="norm", T=1021, H=5003, type="f32", residual=False, y=True, f8=True),
        # prompts of a full batch inside a layer
        dict(name="norm prompts", op="norm", T=8192, H=8192, type="bf16", residual=True, y=True, f8=False),
        # one request, a small head (V = 32,000)
        dict(name="head one row", op="project", T=1, N=32000, K=1024, type="bf16", S=1, R=16, prompts=False),
        # eight slots with eight adapters, the large head (V = 248,320)
        dict(name="head 8 slots", op="project", T=8, N=248320, K=2048, type="bf16", S=8, R=16, prompts=False),
        # 64 slots, 32 adapters, the large head in 8 bits
        dict(name="head 64 slots f8", op="project", T=64, N=248320, K=2048, type="f8", S=32, R=32, prompts=False),
        # ragged prompts of several requests through a layer's projection
        dict(name="prompts", op="project", T=4099, N=4096, K=4096, type="bf16", S=8, R=64, prompts=True),
        # one row, V = 32,000: latency
        dict(name="draw one row", op="draw", B=1, V=32000, type="f32", keys="cut"),
        # a verify window of the large vocabulary
        dict(name="draw window", op="draw", B=5, V=248320, type="f32", keys="cut"),
        # 64 rows, each request its own keys: greedy, temperature alone, wide top_k, narrow top_p; bf16 has heavy ties
        dict(name="draw 64 mixed", op="draw", B=64, V=248320, type="bf16", keys="mixed"),
        # a ragged vocabulary, temperature alone (top_k, top_p and min_p off)
        dict(name="draw odd wide", op="draw", B=19, V=151001, type="f32", keys="off"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "project", "draw"))
    if op == "norm":
        H = _log(rng, 64, 8192)
        c = dict(op=op, T=min(_log(rng, 1, 8192), 8192 * 8192 // H), H=H, type=rng.choice(("bf16", "f32")),
                 residual=rng.random() < 0.7, y=rng.random() < 0.5, f8=rng.random() < 0.6)
        c["y"] = c["y"] or not c["f8"]
        if c["type"] == "f32":
            c["T"] = max(1, c["T"] // 2)
        return c
    if op == "project":
        prompts = rng.random() < 0.4
        kind = rng.choice(("bf16", "f8"))
        if prompts:
            return dict(op=op, T=_log(rng, 129, 4099), N=_log(rng, 512, 4096), K=16 * _log(rng, 32, 256), type=kind,
                        S=_log(rng, 1, 16), R=rng.choice((16, 32, 48, 64)), prompts=True)
        K = 16 * _log(rng, 32, 256)
        N = min(_log(rng, 1000, 248320), 248320 * 2048 // K)
        return dict(op=op, T=_log(rng, 1, 128), N=N, K=K, type=kind, S=_log(rng, 1, 64), R=rng.choice((16, 32, 48, 64)),
                    prompts=False)
    return dict(op=op, B=_log(rng, 1, 64), V=_log(rng, 1000, 248320), type=rng.choice(("bf16", "f32")),
                keys=rng.choice(("cut", "mixed", "off")))


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, to=torch.float32, by=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16 if to == torch.bfloat16 else torch.float32).mul_(by).to(to)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = dict(case)
    if case["op"] == "norm":
        t = TYPES[case["type"]]
        s["x"] = normal(case["T"], case["H"], to=t)
        s["x"][:, :: 97] *= 20  # a few channels of a hidden row are far larger than the others
        s["r"] = normal(case["T"], case["H"], to=t, by=2.0) if case["residual"] else None
        s["w"] = (1 + normal(case["H"], by=0.2)).to(t)
        s["eps"] = 1e-6
    elif case["op"] == "project":
        T, N, K, S, R = (case[k] for k in "TNKSR")
        s["sx"] = s["sw"] = None
        if case["type"] == "f8":
            s["x"] = normal(T, K, by=100.0).clamp_(-F8_MAX, F8_MAX).to(F8)
            s["w"] = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16).mul_(100).clamp_(-F8_MAX, F8_MAX).to(F8)
            s["sx"], s["sw"] = uniform(T, lo=0.005, hi=0.03), uniform(N, lo=1e-4, hi=4e-4)
        else:
            s["x"], s["w"] = normal(T, K, to=torch.bfloat16), normal(N, K, to=torch.bfloat16, by=K ** -0.5)
        s["a"], s["b"] = normal(S, R, K, to=torch.bfloat16, by=K ** -0.5), normal(S, N, R, to=torch.bfloat16, by=R ** -0.5)
        s["g"] = uniform(S, lo=0.25, hi=1.0)
        if case["prompts"]:  # whole prompts of one request after another, an adapter or none for each
            ends = torch.sort(whole(0, T, max(1, T // 400))).values.long()
            of = whole(-1, S, ends.numel() + 1)
            s["of"] = of[torch.searchsorted(ends, torch.arange(T, device="cuda"), right=True)].contiguous()
        else:
            s["of"] = torch.where(uniform(T) < 0.1, whole(-1, 0, T), whole(0, S, T))
    else:
        B, V, t = case["B"], case["V"], TYPES[case["type"]]
        ld = -(-V // 8) * 8  # rows start on 16 bytes
        x = normal(B, ld, by=3.0)
        at = torch.randint(0, V, (B, 4), generator=g, device="cuda")
        x.scatter_(1, at, uniform(B, 4, lo=8.0, hi=15.0))
        s["l"] = x.to(t)[:, :V]
        s["u"] = uniform(B)
        if case["keys"] == "off":
            s["t"], s["k"], s["p"], s["m"] = uniform(B, lo=0.7, hi=1.3), whole(0, 1, B), uniform(B, lo=1.0, hi=1.0), uniform(B, lo=0.0, hi=0.0)
        else:
            s["t"], s["k"] = uniform(B, lo=0.5, hi=1.2), whole(20, 200, B)
            s["p"], s["m"] = uniform(B, lo=0.8, hi=0.99), uniform(B, lo=0.0, hi=0.1)
            if case["keys"] == "mixed":
                s["t"] = torch.where(uniform(B) < 0.2, torch.zeros(B, device="cuda"), s["t"])
                s["k"] = torch.where(uniform(B) < 0.4, torch.zeros_like(s["k"]), torch.where(uniform(B) < 0.2, whole(200, max(201, V // 4), B), s["k"]))
                s["p"] = torch.where(uniform(B) < 0.4, torch.ones(B, device="cuda"), s["p"])
                s["m"] = torch.where(uniform(B) < 0.5, torch.zeros(B, device="cuda"), s["m"])
    return s


# ------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        import request_token_sampling_gb300 as G
        if s["op"] == "norm":
            o = G.norm_rows(s["x"], s["w"], residual=s["r"], eps=s["eps"], y=s["y"], f8=s["f8"])
            return {k: o[k] for k in ("y", "q", "scale", "residual") if k in o}
        if s["op"] == "project":
            return {"y": G.project_rows(s["x"], s["w"], x_scale=s["sx"], w_scale=s["sw"], a=s["a"], b=s["b"],
                                        row_adapter=s["of"], adapter_scale=s["g"])}
        o = G.draw_rows(s["l"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
        return {"ids": o["ids"], "lps": o["lps"]}
    return {"norm": _norm, "project": _project, "draw": _draw}[s["op"]](s)


def _norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["w"].float()
    o = {}
    if s["y"]:
        o["y"] = y.to(s["x"].dtype)
    if s["f8"]:
        scale = (y.abs().amax(1) / F8_MAX).clamp_min(SCALE_MIN)
        o["q"], o["scale"] = (y / scale[:, None]).to(F8), scale
    if s["r"] is not None:
        o["residual"] = h.to(s["x"].dtype)
    return o


def _project(s):
    S, R, K = s["a"].shape
    x = s["x"].float()
    y = x @ s["w"].float().T
    if s["sx"] is not None:
        x = x * s["sx"][:, None]
        y = y * s["sx"][:, None] * s["sw"]
    h = (x @ s["a"].float().reshape(S * R, K).T).reshape(-1, S, R) * s["g"][:, None]
    mine = s["of"][:, None] == torch.arange(S, device=x.device)
    h = torch.where(mine[:, :, None], h, torch.zeros_like(h))
    y = y + h.reshape(-1, S * R) @ s["b"].float().permute(0, 2, 1).reshape(S * R, -1)
    return {"y": y.to(torch.bfloat16)}


def _share(of, total):
    """floor(of * total / 2^24) of whole numbers below 2^25 and 2^62."""
    return of * (total >> 24) + ((of * (total & 0xFFFFFF)) >> 24)


def _draw(s):
    x = s["l"].float() + 0.0
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    V = x.shape[1]
    top = x.amax(1, keepdim=True)
    d = torch.where(x == top, torch.zeros_like(x), x - top)
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    ds, rank = d.gather(1, order), torch.arange(V, device=x.device)
    k, p, m, t = s["k"][:, None], s["p"][:, None], s["m"][:, None], s["t"][:, None]
    keep = ((k <= 0) | (rank < k)) & ((m <= 0) | (xs >= top + torch.log(m)))
    keep = (keep | (rank == 0)) & (xs > -math.inf)
    none = torch.zeros_like(order)
    w = torch.where(keep, (torch.exp(ds) * ONE).to(torch.int64), none)
    c = torch.cumsum(w, 1)
    P = (p.clamp(0.0, 1.0) * 2.0 ** 24).to(torch.int64)
    keep = keep & ((p >= 1) | (c - w < _share(P, c[:, -1:])) | (rank == 0))
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    dt = torch.where(d == 0, d, d * (1 / t))
    w = torch.where(kept, (torch.exp(dt) * ONE).to(torch.int64), none)
    c = torch.cumsum(w, 1)
    U = (s["u"].clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 24).to(torch.int64)[:, None]
    ids = (c <= _share(U, c[:, -1:])).sum(1, keepdim=True).clamp_max(V - 1)
    lps = dt.gather(1, ids) - torch.log(c[:, -1:].float() * (1 / ONE))
    greedy = ~(t > 0)
    ids = torch.where(greedy, order[:, :1], ids)
    lps = torch.where(greedy, torch.zeros_like(lps), lps)
    empty = top == -math.inf
    ids = torch.where(empty, torch.full_like(ids, -1), ids)
    lps = torch.where(empty, torch.full_like(lps, math.nan), lps)
    return {"ids": ids[:, 0].to(torch.int32), "lps": lps[:, 0]}


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2, "f8": 1}[case["type"]]
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        each = size * (1 + 2 * case["residual"] + case["y"]) + case["f8"]
        return {"bytes": T * H * each + 4 * T * case["f8"] + H * size, "flops": 6 * T * H}
    if case["op"] == "project":
        T, N, K, S, R = (case[k] for k in "TNKSR")
        used = min(S, T)
        return {"bytes": size * K * (N + T) + 2 * T * N + 2 * used * R * (K + N), "flops": 2 * T * N * K + 2 * T * R * (K + N)}
    return {"bytes": case["B"] * case["V"] * size, "flops": 10 * case["B"] * case["V"]}


# ------------------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
        y = s["w"].double() * h / (h.square().sum(1, keepdim=True) / case["H"] + s["eps"]).sqrt()
        o = {"y": y} if case["y"] else {}
        if case["f8"]:
            o["scale"] = y.abs().max(1).values.div(F8_MAX).clamp(min=SCALE_MIN)
            o["q"] = y / o["scale"].unsqueeze(1)
        return o | ({"residual": h} if s["r"] is not None else {})
    if case["op"] == "project":
        x = s["x"].double() if s["sx"] is None else s["x"].double() * s["sx"].double().unsqueeze(1)
        y = torch.empty(case["T"], case["N"], dtype=torch.float64, device=x.device)
        for n in range(0, case["N"], 16384):
            w = s["w"][n:n + 16384].double()
            y[:, n:n + 16384] = x @ (w if s["sw"] is None else w * s["sw"][n:n + 16384].double().unsqueeze(1)).t()
        for c in range(case["S"]):
            rows = (s["of"] == c).nonzero().flatten()
            y[rows] += s["g"][c].double() * ((x[rows] @ s["a"][c].double().t()) @ s["b"][c].double().t())
        return {"y": y}
    lps = []
    for b in range(case["B"]):
        x = s["l"][b].double()
        v, at = torch.sort(x, descending=True, stable=True)
        k, p, m, t = (float(s[n][b]) for n in "kpmt")
        n = min(int(k), case["V"]) if k > 0 else case["V"]
        if m > 0:
            n = max(1, min(n, int((v >= v[0] + math.log(m)).sum())))
        if p < 1:
            c = torch.softmax(v[:n], 0).cumsum(0)
            n = max(1, min(n, int((c < p).sum()) + 1))
        if not t > 0:
            lps.append(0.0)
            continue
        ids = torch.sort(at[:n]).values
        l = torch.log_softmax(x[ids] / t, 0)
        j = min(int((l.exp().cumsum(0) <= float(s["u"][b])).sum()), n - 1)
        lps.append(float(l[j]))
    return {"ids": None, "lps": torch.tensor(lps, dtype=torch.float64)}
