"""The operators around the sampler against plain implementations of their formulas in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24          # unit rounding of 32-bit sums
HALF = 2.0 ** -8        # of a rounding to bfloat16, which holds 8 bits: half of its step of 2^-7, relative


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    import request_token_sampling_gb300 as G
    return G


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------ norm_rows
def check_norm(x, w, r, eps, o):
    """y, q, scale and residual of one call against the formula."""
    H = x.shape[1]
    h32 = x.float() + r.float() if r is not None else x.float()
    if r is not None:
        assert torch.equal(o["residual"].view(torch.int32 if x.dtype == F32 else torch.int16),
                           h32.to(x.dtype).view(torch.int32 if x.dtype == F32 else torch.int16))
    h = x.double() + (r.double() if r is not None else 0)
    y = h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.double()
    # a thread adds at most H/32 squares one after another (relative error H/32 U, half of it under the root), the
    # rest is a tree; h, the root and two products round once each; the root's function has up to 2 ulp
    near = (H / 64 + 10) * U
    if "y" in o:
        half = 0.0 if x.dtype == F32 else HALF
        tiny = 2.0 ** -126 if x.dtype == F32 else 2.0 ** -133   # results below the normal range round to its step
        assert ((o["y"].double() - y).abs() <= y.abs() * (near + half * (1 + near)) + tiny).all()
    if "q" in o:
        scale = (y.abs().amax(1) / 448).clamp(min=2.0 ** -100)
        assert ((o["scale"].double() - scale).abs() <= scale * (near + 2 * U)).all()
        v = y / o["scale"].double()[:, None]
        step = torch.where(v.abs() < 2.0 ** -6, torch.full_like(v, 2.0 ** -10), v.abs() * 2.0 ** -4)
        assert ((o["q"].double() - v).abs() <= step + v.abs() * (near + 4 * U)).all()
        assert (o["q"].float().abs().amax(1)[scale > 2.0 ** -100] == 448).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (5, 127), (2, 1000), (33, 1024), (7, 2049), (130, 4096),
                                 (2, 5003), (1, 8192), (3, 16392), (2, 131072)])
def test_norm(G, dtype, T, H):
    g = _gen(T * 1000 + H)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    x[:, ::17] *= 30
    r = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    for res in (None, r):
        for kw in (dict(y=True), dict(y=False, f8=True), dict(y=True, f8=True)):
            check_norm(x, w, res, 1e-6, G.norm_rows(x, w, residual=res, eps=1e-6, **kw))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H", [96, 511, 4096])
def test_norm_strides_and_offsets(G, dtype, H):
    """Rows inside wider ones, starting on no more than their element's alignment; the gaps stay as they are."""
    g = _gen(H)
    for off, gap in ((0, 8), (1, 3), (8, 1), (3, 5)):
        def wide(fill):
            t = torch.full((5, H + gap + off), fill, dtype=dtype, device="cuda")
            return t, t[:, off:off + H]
        x = wide(0.0)[1]
        x.copy_(torch.randn(5, H, generator=g, device="cuda"))
        r = wide(0.0)[1]
        r.copy_(torch.randn(5, H, generator=g, device="cuda"))
        wv = torch.ones(H + 1, dtype=dtype, device="cuda")[off % 2:H + off % 2]
        ybuf, y = wide(-7.0)
        qbuf = torch.full((5, H + gap + off), -7.0, device="cuda").to(F8)
        q = qbuf[:, off:off + H]
        rbuf, ro = wide(-7.0)
        out = dict(y=y, q=q, scale=torch.empty(5, device="cuda"), residual=ro)
        check_norm(x, wv, r, 1e-5, G.norm_rows(x, wv, residual=r, eps=1e-5, f8=True, out=out))
        for buf in (ybuf, qbuf.float(), rbuf):
            edge = torch.cat([buf[:, :off], buf[:, off + H:]], 1).float()
            assert (edge == -7.0).all()


def test_norm_in_place_and_empty(G):
    g = _gen(5)
    x = torch.randn(9, 1030, generator=g, device="cuda").to(BF)
    r = torch.randn(9, 1030, generator=g, device="cuda").to(BF)
    w = torch.ones(1030, dtype=BF, device="cuda")
    want = G.norm_rows(x, w, residual=r)
    r2, x2 = r.clone(), x.clone()
    got = G.norm_rows(x, w, residual=r2, out=dict(residual=r2))
    assert torch.equal(got["y"], want["y"]) and torch.equal(r2, want["residual"])
    got = G.norm_rows(x2, w, residual=r, out=dict(residual=x2))
    assert torch.equal(got["y"], want["y"]) and torch.equal(x2, want["residual"])
    o = G.norm_rows(x[:0], w, residual=r[:0], f8=True)
    assert o["y"].shape == (0, 1030) and o["scale"].numel() == 0


def test_norm_zero_tiny_and_broken_rows(G):
    """A row of zeros, one whose outputs are far below 1, a NaN and an infinity: each within its row."""
    H = 640
    x = torch.randn(6, H, generator=_gen(6), device="cuda")
    x[1] = 0
    x[2] *= 1e-30
    x[3, 5] = math.nan
    x[4, H - 1] = math.inf
    w = torch.ones(H, device="cuda")
    o = G.norm_rows(x, w, eps=1e-6, f8=True)
    good = [0, 1, 2, 5]
    check_norm(x[good], w, None, 1e-6, {k: v[good] for k, v in o.items()})
    assert (o["y"][1] == 0).all() and (o["q"][1].float() == 0).all() and o["scale"][1] == 2.0 ** -100
    assert o["y"][3].isnan().all() and o["scale"][3].isnan() and o["q"][3].float().isnan().all()
    # inf * rsqrt(inf) is inf * 0
    assert o["y"][4, H - 1].isnan() and (o["y"][4, :H - 1] == 0).all() and o["scale"][4].isnan()


# ------------------------------------------------------------------------------ project_rows
def project_case(T, N, K, S, R, kind, seed, of=None):
    g = _gen(seed)
    s = dict(x_scale=None, w_scale=None)
    if kind == "f8":
        s["x"] = (torch.randn(T, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
        s["w"] = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
        s["x_scale"] = torch.rand(T, generator=g, device="cuda") * 0.02 + 0.005
        s["w_scale"] = torch.rand(N, generator=g, device="cuda") * 3e-4 + 1e-4
    else:
        s["x"] = torch.randn(T, K, generator=g, device="cuda").to(BF)
        s["w"] = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(BF)
    if S:
        s["a"] = (torch.randn(S, R, K, generator=g, device="cuda") * K ** -0.5).to(BF)
        s["b"] = (torch.randn(S, N, R, generator=g, device="cuda") * R ** -0.5).to(BF)
        s["adapter_scale"] = torch.rand(S, generator=g, device="cuda") + 0.25
        s["row_adapter"] = torch.randint(-1, S, (T,), generator=g, device="cuda", dtype=torch.int32) if of is None else \
            torch.tensor(of, dtype=torch.int32, device="cuda")
    return s


def check_project(s, y):
    """Against the formula.  A sum of n products in 32 bits in any order is off by at most n U of the products'
    magnitudes; the adapter's inner row and the output round to bfloat16 once each."""
    K = s["x"].shape[1]
    x = s["x"].double() * (1 if s["x_scale"] is None else s["x_scale"].double()[:, None])
    w = s["w"].double() * (1 if s["w_scale"] is None else s["w_scale"].double()[:, None])
    want, off = x @ w.T, (K + 4) * U * (x.abs() @ w.abs().T)
    if "a" in s:
        S, R = s["a"].shape[:2]
        for c in range(S):
            rows = (s["row_adapter"] == c).nonzero().flatten()
            a, b, g = s["a"][c].double(), s["b"][c].double(), s["adapter_scale"][c].double()
            h, hb = g * (x[rows] @ a.T), g * (x[rows].abs() @ a.abs().T)
            want[rows] += h @ b.T
            off[rows] += (HALF * h.abs() + (K + 4) * U * hb) @ b.abs().T + (R + 4) * U * (h.abs() @ b.abs().T)
    assert y.shape == want.shape and y.dtype == BF
    bad = (y.double() - want).abs() > off + (want.abs() + off) * HALF
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("T,N,K,S,R", [
    (1, 1, 16, 1, 16), (1, 128, 64, 1, 16), (1, 1000, 1024, 2, 32), (3, 129, 80, 4, 48), (8, 4099, 512, 8, 16),
    (16, 300, 2048, 16, 64), (17, 77, 272, 64, 16), (64, 2000, 1040, 32, 32), (65, 515, 336, 5, 64), (128, 640, 528, 128, 16),
    (129, 257, 144, 3, 96), (200, 1000, 4096, 200, 16), (300, 384, 256, 1, 128), (513, 700, 768, 7, 256), (1000, 130, 32, 2, 64),
])
def test_project(G, kind, T, N, K, S, R):
    s = project_case(T, N, K, S, R, kind, T * 7 + N)
    check_project(s, G.project_rows(**s))
    assert G.tail_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("T", [1, 5, 32, 100, 260])
def test_project_without_adapters(G, kind, T):
    s = project_case(T, 520, 1056, 0, 0, kind, T)
    y = G.project_rows(**s)
    check_project(s, y)
    none = project_case(T, 520, 1056, 3, 32, kind, T, of=[(-1, 3, 99, -5)[i % 4] for i in range(T)])
    none.update({k: s[k] for k in ("x", "w", "x_scale", "w_scale")})
    assert torch.equal(G.project_rows(**none), y)      # ids outside 0..S-1 are no adapter


@pytest.mark.parametrize("T", [2, 40, 400])
def test_project_whole_prompts(G, T):
    """Runs of rows with one adapter, as prompts one after another are."""
    of = [(-1, 2, 2, 0, 1)[min(4, i * 5 // T)] for i in range(T)]
    s = project_case(T, 1030, 640, 3, 64, "bf16", T, of=of)
    check_project(s, G.project_rows(**s))


@pytest.mark.parametrize("T,N,K,S,R", [(2100, 4100, 1096, 5, 64), (1027, 8200, 520, 300, 16), (3000, 2304, 2048, 2, 48),
                                       (600, 20000, 264, 9, 128), (4099, 1281, 160, 1, 32)])
def test_project_many_rows(G, T, N, K, S, R):
    """Calls that take the tiles of two SMs: adapters at random, in runs, and none."""
    s = project_case(T, N, K, S, R, "bf16", T)
    check_project(s, G.project_rows(**s))
    runs = project_case(T, N, K, S, R, "bf16", T, of=[(i * 7 // T) % (S + 1) - 1 for i in range(T)])
    check_project(runs, G.project_rows(**runs))
    bare = {k: v for k, v in s.items() if k in ("x", "w", "x_scale", "w_scale")}
    check_project(bare, G.project_rows(**bare))
    assert G.tail_errors() == 0


def test_project_many_rows_with_a_broken_adapter(G):
    """NaN and infinities in one adapter of a tile: the other rows stay right (their sums may be taken again, in
    another order), its own are not finite where the formula says so."""
    T, N, K, S, R = 1500, 3000, 128, 3, 16
    of = [(0, 1, 2, -1)[i % 4] if i < 700 else 2 for i in range(T)]
    s = project_case(T, N, K, S, R, "bf16", 1, of=of)
    b = s["b"].clone()
    b[1, 3, 5], b[1, 1300, 0], b[1, 2999, 15] = math.inf, math.nan, -math.inf
    broken = G.project_rows(**dict(s, b=b))
    mine = torch.tensor(of, device="cuda") == 1
    hit = torch.zeros(N, dtype=torch.bool, device="cuda")
    hit[[3, 1300, 2999]] = True
    assert (~broken[mine][:, hit].isfinite()).all()
    fixed = broken.clone()
    fixed[mine.nonzero(), hit.nonzero().T] = G.project_rows(**s)[mine.nonzero(), hit.nonzero().T]
    check_project(s, fixed)
    x = s["x"].clone()
    x[2, 9] = math.nan
    broken = G.project_rows(**dict(s, x=x))
    rest = torch.arange(T, device="cuda") != 2
    assert broken[2].isnan().all() and torch.equal(broken[rest], G.project_rows(**s)[rest])
    assert G.tail_errors() == 0


def test_project_strides(G):
    g = _gen(3)
    s = project_case(19, 333, 320, 3, 16, "bf16", 3)
    y = G.project_rows(**s)
    for gap in (8, 24):
        xb = torch.full((19, 320 + gap), math.nan, dtype=BF, device="cuda")
        wb = torch.full((333, 320 + gap), math.nan, dtype=BF, device="cuda")
        xb[:, :320], wb[:, :320] = s["x"], s["w"]
        yb = torch.full((19, 333 + gap + 1), -7.0, dtype=BF, device="cuda")
        G.project_rows(**dict(s, x=xb[:, :320], w=wb[:, :320]), out=yb[:, 1:334])
        assert torch.equal(yb[:, 1:334], y)
        assert (yb[:, 0] == -7).all() and (yb[:, 334:] == -7).all()
    assert G.project_rows(**dict(s, x=s["x"][:0], row_adapter=s["row_adapter"][:0])).shape == (0, 333)


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("T", [4, 48, 150])
def test_project_broken_adapter_stays_with_its_rows(G, kind, T):
    """NaN and infinities in one adapter's matrices: the rows of the others are what they were, bit for bit, and
    its own rows are not finite where the formula says so."""
    of = [(0, 1, 2, -1)[i % 4] for i in range(T)]
    s = project_case(T, 700, 256, 3, 16, kind, T, of=of)
    y = G.project_rows(**s)
    b = s["b"].clone()
    b[1, 3, 5], b[1, 130, 0], b[1, 699, 15] = math.inf, math.nan, -math.inf
    broken = G.project_rows(**dict(s, b=b))
    mine = torch.tensor(of, device="cuda") == 1
    assert torch.equal(broken[~mine], y[~mine])
    hit = torch.zeros(700, dtype=torch.bool, device="cuda")
    hit[[3, 130, 699]] = True
    assert (~broken[mine][:, hit].isfinite()).all() and torch.equal(broken[mine][:, ~hit], y[mine][:, ~hit])
    a = s["a"].clone()
    a[1, 2, 7] = math.nan
    broken = G.project_rows(**dict(s, a=a))
    assert torch.equal(broken[~mine], y[~mine]) and broken[mine].isnan().all()
    x = s["x"].clone().float()
    x[2, 9] = math.nan
    broken = G.project_rows(**dict(s, x=x.to(s["x"].dtype)))
    rest = torch.arange(T, device="cuda") != 2
    assert torch.equal(broken[rest], y[rest]) and broken[2].isnan().all()


def test_project_repeats(G):
    """The same call gives the same bits, and rows do not depend on which other rows a call has."""
    for T in (1, 30, 300):
        s = project_case(T, 2050, 1024, 4, 32, "bf16", 11)
        y = G.project_rows(**s)
        for _ in range(3):
            assert torch.equal(G.project_rows(**s), y)


# ------------------------------------------------------------------------------ draw_rows
def draw_one(x, u, t, k, p, m):
    """(id, log-probability, the ids that a boundary within rounding would give too) by the formula in 64 bits."""
    x = x.double()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    V = int((x > -math.inf).sum())
    if V == 0:
        return -1, math.nan, {-1}
    v, at = torch.sort(x + 0.0, descending=True, stable=True)
    v, at = v[:V], at[:V]
    if not t > 0:
        return int(at[0]), 0.0, {int(at[0])}
    d = torch.where(v == v[0], torch.zeros_like(v), v - v[0])
    n = min(k, V) if k > 0 else V
    if not m <= 0:
        thr = torch.tensor(float(v[0]), dtype=F32) + torch.log(torch.tensor(m, dtype=F32))
        n = max(1, min(n, int((v >= float(thr)).sum())))
    sizes = {n}
    if not p >= 1:
        w = d[:n].exp()
        c = w.cumsum(0) / w.sum()
        eps = 2 * U + 4 * U * (1 + float((w * d[:n].abs()).nan_to_num(0.0).sum() / w.sum()))
        n = max(1, int((c < p).sum()) + 1) if p > 0 else 1
        n = min(n, c.numel())
        sizes = {n} | {q for q in (n - 1, n + 1) if 1 <= q <= c.numel() and abs(float(c[min(n, q) - 1]) - p) <= eps}
    first, ok = None, set()
    for n in [n] + sorted(sizes - {n}):
        ids, back = torch.sort(at[:n])
        dt = d[:n][back] / t
        dt = torch.where(d[:n][back] == 0, torch.zeros_like(dt), dt)
        w = dt.exp()
        c = w.cumsum(0) / w.sum()
        # the ratio rounds twice (2 U of it each), the exponential once more; u acts in steps of 2^-24
        eps = 2 * U + 4 * U * (1 + float((w * dt.abs()).nan_to_num(0.0).sum() / w.sum()))
        j = min(int((c <= u).sum()), n - 1)
        if first is None:
            first = int(ids[j]), float(dt[j] - w.sum().log())
        lo, hi = int((c <= u - eps).sum()), int((c <= u + eps).sum())
        ok |= {int(i) for i in ids[lo:min(hi, n - 1) + 1]}
    return first[0], first[1], ok


def check_draw(G, x, u, t=None, k=None, p=None, m=None, V=None):
    B = x.shape[0]
    f = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    o = G.draw_rows(x, f(u, F32), f(t, F32), f(k, torch.int32), f(p, F32), f(m, F32), V=V)
    ids, lps = o["ids"].tolist(), o["lps"].tolist()
    r32 = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
    exact = 0
    for b in range(B):
        row = x[b, :V] if V is not None else x[b]
        i, lp, ok = draw_one(row, r32(u[b]), r32(t[b]) if t else 1.0, k[b] if k else 0, r32(p[b]) if p else 1.0,
                             r32(m[b]) if m else 0.0)
        assert ids[b] in ok, (b, ids[b], i, ok)
        exact += ids[b] == i
        if ids[b] == i:
            # two roundings of the distance, the logarithm's and the sum's
            assert (math.isnan(lp) and math.isnan(lps[b])) or abs(lps[b] - lp) <= 1e-6 + 8 * U * abs(lp), (b, lps[b], lp)
    assert exact >= B - max(1, B // 16)
    return o


def logits(B, V, dtype, seed, spread=3.0, spikes=3):
    g = _gen(seed)
    ld = -(-V // 8) * 8
    x = torch.full((B, ld), math.nan, device="cuda")
    x[:, :V] = torch.randn(B, V, generator=g, device="cuda") * spread
    if spikes:
        x.scatter_(1, torch.randint(0, V, (B, spikes), generator=g, device="cuda"),
                   torch.rand(B, spikes, generator=g, device="cuda") * 7 + 8)
    return x.to(dtype)[:, :V]


def keys(B, V, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda: torch.rand(1, generator=g).item()  # noqa: E731
    t = [(0.0, 0.3 + r(), 1.0, 0.7 + r())[b % 4] for b in range(B)]
    k = [(0, 20, 1 + int(r() * V), 0, 64 + int(r() * 200), 1)[b % 6] for b in range(B)]
    p = [(1.0, 0.9 + r() * 0.1, r(), 1.0, 0.95)[b % 5] for b in range(B)]
    m = [(0.0, 0.05, 0.0, r() * 1e-4, 0.2, 0.0, 1e-7)[b % 7] for b in range(B)]
    return [r() for _ in range(B)], t, k, p, m


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 1000, 1025, 4099, 32000, 65537, 151001, 248320])
def test_draw(G, dtype, V):
    B = 70 if V < 5000 else 25
    for spread, spikes in ((3.0, 3), (0.5, 0)):
        check_draw(G, logits(B, V, dtype, V, spread, spikes if V > 10 else 0), *keys(B, V, V))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [5, 1000, 40007])
def test_draw_each_cut_alone(G, dtype, V):
    B = 24
    x = logits(B, V, dtype, V + 1, 2.0)
    u = torch.rand(B, generator=torch.Generator().manual_seed(V)).tolist()
    check_draw(G, x, u)
    check_draw(G, x, u, t=[0.1 + 0.2 * b for b in range(B)])
    check_draw(G, x, u, k=[b + 1 for b in range(B)])
    check_draw(G, x, u, k=[V - 1 - b % 3 for b in range(B)])
    check_draw(G, x, u, k=[-b for b in range(B)])
    check_draw(G, x, u, p=[b / B for b in range(B)])
    check_draw(G, x, u, p=[1.0 - 10.0 ** -(b / 3) for b in range(B)])
    check_draw(G, x, u, m=[b / B for b in range(B)])
    check_draw(G, x, u, m=[10.0 ** -(b / 2) for b in range(B)])


def test_draw_ties(G):
    """Rows of one value, of two, and of a few: a cut inside equal logits keeps the lowest indices."""
    for dtype in (F32, BF):
        for V in (9, 3001, 50000):
            B = 12
            x = torch.zeros(B, -(-V // 8) * 8, dtype=dtype, device="cuda")[:, :V]
            x[4:8] = (torch.arange(V, device="cuda") % 2).to(dtype)
            x[8:] = (torch.arange(V, device="cuda") % 5).to(dtype)
            u = [(b + 0.5) / B for b in range(B)]
            check_draw(G, x, u)
            check_draw(G, x, u, k=[1 + b % 7 for b in range(B)])
            check_draw(G, x, u, p=[0.25] * B)
            check_draw(G, x, u, t=[0.5 + b / 4 for b in range(B)], k=[V // 2] * B, p=[0.77] * B, m=[0.01] * B)
    x = torch.zeros(1, 8, device="cuda")
    x[0, ::2] = -0.0      # equal to 0.0: the lowest index comes first all the same
    assert G.draw_rows(x, torch.zeros(1, device="cuda"), top_k=torch.ones(1, dtype=torch.int32, device="cuda"))["ids"].item() == 0


def test_draw_masked_rows(G):
    """-inf, NaN, the type's lowest value and +inf; rows with one entry left and with none."""
    for dtype in (F32, BF):
        V, B = 3000, 10
        x = logits(B, V, dtype, 9)
        x[0] = -math.inf
        x[1] = math.nan
        x[2] = -math.inf
        x[2, 1234] = -5.0
        x[3, : V - 2] = torch.finfo(dtype).min
        x[4] = torch.finfo(dtype).min
        x[5, 7] = math.nan
        x[5, 8:900] = -math.inf
        x[6, 77] = math.inf
        x[6, 2077] = math.inf
        x[7] = torch.finfo(dtype).max
        x[8, ::3] = math.nan
        x[8, 1::3] = -math.inf
        x[9, 1:] = math.nan
        u = [0.999, 0.5, 0.3, 0.7, 0.9, 0.6, 0.75, 0.2, 0.99, 0.4]
        check_draw(G, x, u)
        check_draw(G, x, u, t=[0.7] * B, k=[2] * B, p=[0.9] * B, m=[0.05] * B)
        check_draw(G, x, u, t=[0.0] * B)
        check_draw(G, x, u, k=[2500] * B, p=[0.999] * B)
        o = G.draw_rows(x, torch.tensor(u, device="cuda"))
        assert o["ids"][:3].tolist() == [-1, -1, 1234] and o["lps"][2] == 0 and o["lps"][:2].isnan().all()


def test_draw_odd_keys(G):
    """Keys and random numbers outside their usual range."""
    nan, inf = math.nan, math.inf
    x = logits(8, 1000, F32, 4)
    head = x.argmax(1).tolist()
    t = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    u = torch.full((8,), 0.5, device="cuda")
    ids = lambda **kw: G.draw_rows(x, kw.pop("u", u), **kw)["ids"].tolist()  # noqa: E731
    assert ids(temperature=t(0.0, -1.0, nan, -inf, 1e-45, 1e-30, -0.0, 1e-38)) == head
    assert ids(top_p=t(0.0, -1.0, nan, -inf, 1e-30, 0.0, 0.0, 0.0)) == head
    assert ids(min_p=t(1.0, 2.0, inf, nan, 1e30, 1.5, 1.0, 1.0)) == head
    low = [int(torch.nonzero(x[b] > -inf)[0]) for b in range(8)]
    assert ids(u=t(-1.0, -inf, nan, 0.0, -0.0, 0.0, 0.0, 0.0), temperature=torch.full((8,), 1e30, device="cuda")) == low
    assert ids(u=t(1.0, 2.0, inf, 1.0, 1.0, 1.0, 1.0, 1.0), temperature=torch.full((8,), inf, device="cuda")) == [999] * 8
    off = ids()
    assert ids(top_p=t(1.0, 2.0, inf, 1.0, 1.0, 1.0, 1.0, 1.0), min_p=t(0.0, -1.0, -inf, 0.0, 0.0, 0.0, 0.0, 0.0),
               top_k=torch.tensor([0, -1, 1000, 1001, 2 ** 31 - 1, -2 ** 31, 0, 0], dtype=torch.int32, device="cuda")) == off


def test_draw_whole_range_of_random_numbers(G):
    """Random numbers in equal steps through one row draw every id as often as its probability says."""
    p = torch.tensor([0.5, 0.25, 0.125, 0.0625, 0.0625], device="cuda")
    B = 1 << 12
    x = torch.full((B, 8), -math.inf, device="cuda")
    x[:, :5] = p.log()
    ids = G.draw_rows(x, (torch.arange(B, device="cuda") + 0.5) / B)["ids"]
    assert torch.bincount(ids, minlength=5).tolist() == [B // 2, B // 4, B // 8, B // 16, B // 16]


def test_draw_narrower_than_its_rows(G):
    x = logits(6, 4000, BF, 2)
    check_draw(G, x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], V=777)
    assert G.draw_rows(x[:0], torch.zeros(0, device="cuda"))["ids"].numel() == 0


def test_draw_agrees_with_the_sampler_on_the_cut(G):
    """What is left with u swept over [0, 1) is the sampler's top_k list cut by min_p and top_p."""
    x = logits(1, 5000, F32, 21)
    B = 4096
    u = (torch.arange(B, device="cuda") + 0.5) / B
    one = lambda v, dt=F32: torch.full((B,), v, dtype=dt, device="cuda")  # noqa: E731
    got = set(G.draw_rows(x.expand(B, 5000).contiguous(), u, one(50.0), one(20, torch.int32), one(0.97), one(0.01))["ids"].tolist())
    with G.Sampler(device=0, max_slots=1, max_vocab=5000, max_rows=1) as s:
        s.set_slot(0, dict(temperature=50.0, top_k=20, top_p=0.97, min_p=0.01, seed=1))
        o = s.sample(x.contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), debug=True)
        kept = o["topk_ids"][0, :int(o["kept"][0, 1])].tolist()
    assert got == set(kept)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_draw_many_rows_and_the_largest_vocabulary(G, dtype):
    """More rows than run at once (long ones go first) and a row of 2^19 logits."""
    check_draw(G, logits(700, 1000, dtype, 5), *keys(700, 1000, 5))
    check_draw(G, logits(5, 524288, dtype, 6), *keys(5, 524288, 6))
    B = 2500
    x = logits(B, 64, dtype, 7)
    u = torch.rand(B, generator=torch.Generator().manual_seed(7)).tolist()
    check_draw(G, x, u, k=[1 + b % 70 for b in range(B)], p=[0.5 + 0.5 * (b % 3) for b in range(B)])


@pytest.mark.parametrize("spread", [0.01, 1.0, 30.0])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_draw_wide_cuts(G, dtype, spread):
    """Cuts that leave thousands: flat rows, steep ones, cuts near either end."""
    V, B = 60000, 12
    x = logits(B, V, dtype, 31, spread, 0)
    u = [(b + 0.5) / B for b in range(B)]
    check_draw(G, x, u, k=[1000, 2000, 5000, 20000, 40000, 55000, 59000, 59999, 3000, 700, 30000, 10000])
    check_draw(G, x, u, p=[0.1, 0.3, 0.5, 0.7, 0.8, 0.9, 0.95, 0.99, 0.999, 0.9999, 0.6, 0.2])
    check_draw(G, x, u, k=[50000, 30000] * 6, p=[0.9, 0.5, 0.99] * 4, m=[0.0, 1e-3, 1e-6, 0.0] * 3)


# ------------------------------------------------------------------------------ together
def test_on_another_stream_and_in_a_graph(G):
    """The three calls in a row, on a side stream and replayed from a graph, give what they give on their own."""
    g = _gen(8)
    T, H, N, S, R = 12, 512, 3000, 4, 16
    s = project_case(T, N, H, S, R, "f8", 8)
    x, r = torch.randn(T, H, generator=g, device="cuda").to(BF), torch.randn(T, H, generator=g, device="cuda").to(BF)
    w, u = torch.ones(H, dtype=BF, device="cuda"), torch.rand(T, generator=g, device="cuda")

    def step():
        n = G.norm_rows(x, w, residual=r, y=False, f8=True)
        y = torch.empty(T, N, dtype=BF, device="cuda")
        G.project_rows(**dict(s, x=n["q"], x_scale=n["scale"]), out=y)
        return y, G.draw_rows(y, u, temperature=torch.full((T,), 0.8, device="cuda"))

    y, o = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, o2 = step()
    side.synchronize()
    assert torch.equal(y2, y) and torch.equal(o2["ids"], o["ids"]) and torch.equal(o2["lps"], o["lps"])
    named = G.norm_rows(x, w, residual=r, f8=True, stream=side)
    side.synchronize()
    assert torch.equal(named["q"].view(torch.uint8), G.norm_rows(x, w, residual=r, f8=True)["q"].view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, o3 = step()
    for _ in range(2):
        y3.zero_()
        o3["ids"].fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and torch.equal(o3["ids"], o["ids"])
    assert G.tail_errors() == 0


def test_after_a_sampling_call_that_waits_for_nothing(G):
    """The sampler's own-outputs calls do not wait for what is before them; what follows them still does."""
    x = logits(4, 30000, F32, 77)
    big = torch.empty(1 << 26, device="cuda")
    h, w = torch.randn(4, 512, device="cuda").to(BF), torch.ones(512, dtype=BF, device="cuda")
    y = G.norm_rows(h, w)["y"]
    flags = G.STRATA_FLAG_PDL | G.STRATA_FLAG_EARLY_LOAD | G.STRATA_FLAG_OWN_OUTPUTS
    slot, pos = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with G.Sampler(device=0, max_slots=1, max_vocab=30000, max_rows=4) as s:
        s.set_slot(0, dict(temperature=0.7, seed=3))
        torch.cuda.synchronize()
        for i in range(20):
            late = torch.zeros_like(h)
            big.normal_()
            late.copy_(h)                       # behind the long fill
            s.sample(x, slot, pos, flags=flags)
            assert torch.equal(G.norm_rows(late, w)["y"], y), i


def test_the_example_runs_the_tail(G):
    """The decode example: a captured step gives the tokens of the uncaptured one; slot 0 is greedy."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_tail.py")
    spec = importlib.util.spec_from_file_location("decode_tail", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    ids, lps = mod.decode(6, 4096, 512, 5)
    again, lps2 = mod.decode(6, 4096, 512, 5, graph=False)
    assert torch.equal(ids, again) and torch.equal(lps, lps2)
    assert ((ids >= 0) & (ids < 4096)).all() and (lps <= 0).all() and (lps[:, 0] == 0).all()
    assert len({tuple(c.tolist()) for c in ids.T}) > 1
