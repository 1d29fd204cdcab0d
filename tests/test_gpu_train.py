"""The operators that score and train the end of a model against plain implementations of their formulas in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24          # unit rounding of 32-bit sums
HALF = 2.0 ** -8        # of a rounding to bfloat16: half of its step of 2^-7, relative
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -126}


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    import request_token_sampling_gb300 as G
    return G


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, by=1.0, to=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(to)


def near(got, want, off):
    """|got - want| <= off, elementwise; NaN where NaN is wanted."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    assert torch.equal(got.isnan(), want.isnan())
    ok = ((got - want).abs() <= off) | want.isnan() | (got == want)
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} off by up to {float(((got - want).abs() / off).nan_to_num(0).max()):.3g} times what they may"


# ------------------------------------------------------------------------------ layer_norm_rows
def check_layer_norm(x, w, b, r, eps, o):
    H = x.shape[1]
    h = x.double() + (r.double() if r is not None else 0)
    half = HALF if x.dtype == BF else 0.0
    if r is not None:
        near(o["residual"], h, h.abs() * (U + half) + TINY[x.dtype])
    mean = h.mean(1, keepdim=True)
    d = h - mean
    rstd = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    # a thread adds H/32 values one after another at most, the rest is a tree; h itself is rounded once
    sums = (H / 32 + 12) * U
    off_mean = h.abs().mean(1, keepdim=True) * sums
    # the squares' sum, and the mean's error in it (first order: cancels but for H off_mean^2)
    off_rstd = rstd * (sums / 2 + 4 * U) + rstd ** 3 * (off_mean ** 2 + 2 * U * h.abs().amax(1, keepdim=True) * d.abs().mean(1, keepdim=True))
    near(o["mean"][:, None], mean, off_mean + TINY[F32])
    near(o["rstd"][:, None], rstd, off_rstd)
    v = d * rstd
    y = v * w.double() + (b.double() if b is not None else 0)
    off = w.double().abs() * (rstd * (off_mean + 2 * U * h.abs()) + d.abs() * off_rstd + 4 * U * v.abs()) + 2 * U * y.abs()
    near(o["y"], y, off * (1 + half) + half * y.abs() + TINY[x.dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (5, 127), (2, 1000), (33, 1024), (7, 2049), (130, 4096), (400, 520),
                                 (2, 5003), (1, 8192), (310, 8192), (3, 16392), (2, 131072)])
def test_layer_norm(G, dtype, T, H):
    g = _gen(T * 1000 + H)
    x = _normal(g, T, H, to=dtype)
    x[:, ::17] *= 30
    r, w, b = _normal(g, T, H, to=dtype), (1 + _normal(g, H, by=0.3)).to(dtype), _normal(g, H, to=dtype)
    for res in (None, r):
        for bias in (None, b):
            check_layer_norm(x, w, bias, res, 1e-5, G.layer_norm_rows(x, w, bias=bias, residual=res, eps=1e-5))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H", [96, 511, 4096])
def test_layer_norm_strides_offsets_and_gaps(G, dtype, H):
    """Rows inside wider ones, on no more than their element's alignment; the gaps stay as they are.  Both directions."""
    g = _gen(H)
    for off, gap in ((0, 8), (1, 3), (8, 1), (3, 5)):
        def wide(fill=None):
            t = torch.full((5, H + gap + off), -7.0, dtype=dtype, device="cuda")
            if fill is not None:
                t[:, off:off + H] = fill
            return t, t[:, off:off + H]
        x, r = wide(_normal(g, 5, H))[1], wide(_normal(g, 5, H))[1]
        w = torch.cat([x.new_ones(off % 2), 1 + _normal(g, H, by=0.3).to(dtype)])[off % 2:]
        (ybuf, y), (rbuf, ro) = wide(), wide()
        o = G.layer_norm_rows(x, w, bias=w, residual=r, out=dict(y=y, residual=ro))
        check_layer_norm(x, w, w, r, 1e-5, o)
        (dbuf, dx), dy = wide(), wide(_normal(g, 5, H))[1]
        check_layer_norm_grad(dy, ro, w, o["mean"], o["rstd"], r, G.layer_norm_grad(dy, ro, w, o["mean"], o["rstd"], dresidual=r, out=dict(dx=dx)))
        for buf in (ybuf, rbuf, dbuf):
            assert (torch.cat([buf[:, :off], buf[:, off + H:]], 1).float() == -7.0).all()


def test_layer_norm_far_from_zero(G):
    """Rows whose mean is a thousand times their spread: a variance from sums of squares would lose all of it."""
    x = _normal(_gen(3), 64, 1024) + 1000.0
    w = torch.ones(1024, device="cuda")
    check_layer_norm(x, w, None, None, 1e-5, G.layer_norm_rows(x, w))


def test_layer_norm_constant_broken_empty_and_in_place(G):
    H = 640
    x = _normal(_gen(6), 6, H)
    x[1] = 3.0
    x[3, 5] = math.nan
    x[4, H - 1] = math.inf
    w, b = torch.ones(H, device="cuda"), torch.full((H,), 0.5, device="cuda")
    o = G.layer_norm_rows(x, w, bias=b, eps=1e-6)
    good = [0, 1, 2, 5]
    check_layer_norm(x[good], w, b, None, 1e-6, {k: v[good] for k, v in o.items()})
    assert o["y"][3].isnan().all() and o["y"][4].isnan().all()
    assert (o["y"][1] == 0.5).all()
    e = G.layer_norm_rows(x[:0], w)
    assert e["y"].shape == (0, H) and e["mean"].numel() == 0
    z = x[good].to(BF)
    r = z.flip(0).contiguous()
    want = G.layer_norm_rows(z, w.to(BF), residual=r)
    r2, z2 = r.clone(), z.clone()
    got = G.layer_norm_rows(z, w.to(BF), residual=r2, out=dict(residual=r2))
    assert torch.equal(got["y"], want["y"]) and torch.equal(r2, want["residual"])
    got = G.layer_norm_rows(z2, w.to(BF), residual=r, out=dict(residual=z2))
    assert torch.equal(got["y"], want["y"]) and torch.equal(z2, want["residual"])
    # the statistics alone, and y alone
    s = G.layer_norm_rows(z, w.to(BF), y=False)
    assert set(s) == {"mean", "rstd"}
    assert set(G.layer_norm_rows(z, w.to(BF), stats=False)) == {"y"}


# ------------------------------------------------------------------------------ layer_norm_grad
def check_layer_norm_grad(dy, x, w, mean, rstd, r, o):
    T, H = x.shape
    half = HALF if x.dtype == BF else 0.0
    d, s = dy.double(), rstd.double()[:, None]
    v = (x.double() - mean.double()[:, None]) * s
    a = d * w.double()
    ma, mav = a.mean(1, keepdim=True), (a * v).mean(1, keepdim=True)
    dx = s * (a - ma - v * mav)
    sums = (H / 32 + 12) * U
    off = s * (a.abs().mean(1, keepdim=True) * sums + v.abs() * (a * v).abs().mean(1, keepdim=True) * (sums + 4 * U)
               + 6 * U * (a.abs() + ma.abs() + (v * mav).abs()))
    if r is not None:
        dx = dx + r.double()
        off = off + 2 * U * r.double().abs()
    if "dx" in o:
        near(o["dx"], dx, off * (1 + half) + (half + U) * dx.abs() + TINY[x.dtype])
    for key, each in (("dweight", d * v), ("dbias", d)):
        if key in o:  # T values one after another at most, each with three roundings
            want = each.sum(0)
            near(o[key], want, (T + 6) * U * each.abs().sum(0) * (1 + half) + half * want.abs() + TINY[x.dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (9, 127), (700, 96), (5000, 24), (2, 1000), (33, 1024), (7, 2049), (650, 513),
                                 (130, 4096), (1, 8192), (310, 5003), (310, 8192), (3, 8200), (18, 9001), (2, 131072)])
def test_layer_norm_grad(G, dtype, T, H):
    g = _gen(T * 1000 + H)
    x, dy, r = (_normal(g, T, H, to=dtype) for _ in range(3))
    x[:, ::17] *= 30
    w = (1 + _normal(g, H, by=0.3)).to(dtype)
    o = G.layer_norm_rows(x, w)
    for res in (None, r):
        check_layer_norm_grad(dy, x, w, o["mean"], o["rstd"], res, G.layer_norm_grad(dy, x, w, o["mean"], o["rstd"], dresidual=res))
    p = G.layer_norm_grad(dy, x, w, o["mean"], o["rstd"], dx=False, bias=False)
    assert set(p) == {"dweight"}
    check_layer_norm_grad(dy, x, w, o["mean"], o["rstd"], None, p)
    p = G.layer_norm_grad(dy, x, w, o["mean"], o["rstd"], dweight=False, bias=False)
    assert set(p) == {"dx"}
    check_layer_norm_grad(dy, x, w, o["mean"], o["rstd"], None, p)
    for over in ("dy", "x", "r"):  # in place
        t = dict(dy=dy.clone(), x=x.clone(), r=r.clone())
        p = G.layer_norm_grad(t["dy"], t["x"], w, o["mean"], o["rstd"], dresidual=t["r"], out=dict(dx=t[over]))
        check_layer_norm_grad(dy, x, w, o["mean"], o["rstd"], r, p)


def test_layer_norm_grad_against_differences(G):
    """In 32 bits: (f(x + e u) - f(x - e u)) / 2e for f = sum of y c, along random directions of x, weight and bias."""
    g = _gen(8)
    T, H = 6, 96
    x, c, w, b = _normal(g, T, H), _normal(g, T, H), 1 + _normal(g, H, by=0.2), _normal(g, H)
    o = G.layer_norm_rows(x, w, bias=b)
    d = G.layer_norm_grad(c, x, w, o["mean"], o["rstd"])

    def f(x, w, b):
        x, w, b = x.double(), w.double(), b.double()
        m = x.mean(1, keepdim=True)
        return (((x - m) / ((x - m).square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * c.double()).sum()

    e = 1e-5
    for key, at in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        u = _normal(g, *d[key].shape).double()
        args = [x.double(), w.double(), b.double()]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + e * u, args[at] - e * u
        # the differences' own error: e^2 of the third derivative, and 2^-52 f / e
        assert abs(float((f(*up) - f(*down)) / (2 * e) - (d[key].double() * u).sum())) < 1e-4 * float(d[key].double().norm() * u.norm())


def test_layer_norm_grad_without_rows(G):
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    out = dict(dweight=torch.full((64,), 9.0, dtype=BF, device="cuda"), dbias=torch.full((64,), 9.0, dtype=BF, device="cuda"))
    o = G.layer_norm_grad(x, x, torch.ones(64, dtype=BF, device="cuda"), s, s, out=out)
    assert (o["dweight"] == 0).all() and (o["dbias"] == 0).all() and o["dx"].shape == (0, 64)


# ------------------------------------------------------------------------------ losses
def loss_case(T, V, H, seed, K=0, skip=0.2):
    g = _gen(seed)
    w = _normal(g, V, H, by=2 * H ** -0.5, to=BF)
    ids = torch.randint(0, V, (T, max(K, 1)), generator=g, device="cuda", dtype=torch.int32)
    x = (_normal(g, T, H) + 2 * torch.rand(T, 1, generator=g, device="cuda") * w[ids[:, 0].long()].float()).to(BF)
    teacher = None
    if K:
        teacher = _normal(g, T, K, by=3.0)
        have = torch.rand(T, K, generator=g, device="cuda") > 0.1
        ids = torch.where(have, ids, -1)
        teacher[torch.rand(T, K, generator=g, device="cuda") < 0.05] = -math.inf
    ids[torch.rand(T, generator=g, device="cuda") < skip] = -100
    return x, w, ids if K else ids[:, 0].contiguous(), teacher


class Exact:
    """Loss, lse and gradients in 64 bits, and how far 32-bit sums may be off them."""

    def __init__(self, x, w, ids, teacher=None, s=1.0):
        self.x, self.w, self.s = x.double(), w.double(), float(s)
        T, H = x.shape
        V = w.shape[0]
        ids = ids.view(T, -1)
        there = ids >= 0
        if teacher is not None:
            there = there & (teacher != -math.inf)
        self.asked = there.any(1)
        self.beyond = (there & (ids >= V)).any(1)
        l = torch.where(there, (teacher.double() if teacher is not None else torch.zeros(ids.shape, device=x.device).double()) / s,
                        torch.full(ids.shape, -math.inf, device=x.device, dtype=torch.float64))
        l[~self.asked] = 0.0
        logq = torch.log_softmax(l, 1)
        q = logq.exp() * there
        at = ids.clamp(0, V - 1).long()
        self.asked = self.asked & ~self.beyond
        clean = torch.where(self.asked[:, None], self.x, torch.zeros_like(self.x))
        z = clean @ self.w.T / s
        self.lse = torch.where(self.asked, torch.logsumexp(z, 1), 0.0)
        zk = z.gather(1, at)
        each = torch.where(q > 0, q * (logq - zk + self.lse[:, None]), 0.0)
        self.loss = torch.where(self.asked, s * s * each.sum(1), 0.0)
        self.p = torch.exp(z - self.lse[:, None]) * self.asked[:, None]
        self.q = torch.zeros_like(z).scatter_add_(1, at, q) * self.asked[:, None]
        # the tensor cores add 16 products at a time to a 32-bit sum, which may be cut off instead of rounded; a tile's ids
        # are 256 terms at most, in chunks of 32; exponents have one rounding of their own size
        size = (clean.abs() @ self.w.abs().T) / s
        off_z = size * (H / 16 + 16) * 2 * U + (z.abs() + self.lse.abs()[:, None] + 1) * 4 * U
        self.off_z = off_z
        self.off_lse = off_z.amax(1) + (V / 256 + 300) * U + (self.lse.abs() + 1) * 4 * U
        self.off_loss = s * s * ((q * (off_z.gather(1, at) + self.off_lse[:, None])).sum(1)
                                 + (each.abs() + q * (logq.abs().nan_to_num(0, 0, 0) + zk.abs() + self.lse.abs()[:, None] + 4) * 8).sum(1) * U * 4)
        self.loss[self.beyond] = math.nan
        self.lse[self.beyond] = math.nan
        self.clean = clean

    def check_rows(self, o):
        near(o["lse"], self.lse, self.off_lse)
        near(o["loss"], self.loss, self.off_loss)

    def check_grad(self, o, g):
        T, V = self.p.shape
        g = torch.where(self.asked, g.double(), 0.0)[:, None] * self.s
        d = self.p - self.q
        off_lse = self.off_lse.nan_to_num(0)[:, None]
        off_d = self.p * (self.off_z + off_lse + 2.0 ** -20) + self.q * 8 * U + d.abs() * HALF
        if "dx" in o:
            dx = (d * g) @ self.w
            off = (g.abs() * off_d) @ self.w.abs() + (g * d).abs() @ self.w.abs() * (V / 16 + 32) * 2 * U
            near(o["dx"], dx, off * (1 + HALF) + dx.abs() * (HALF + 4 * U) + TINY[BF])
        if "dw" in o:
            dw = (d * g).T @ self.clean
            same = (g[self.asked] == g[self.asked][:1]).all() if self.asked.any() else True
            scaled = U if same else HALF
            off = (g.abs() * (off_d + d.abs() * scaled)).T @ self.clean.abs() * (1 + HALF) + (g * d).abs().T @ self.clean.abs() * (T / 16 + 32) * 2 * U
            near(o["dw"], dw, off * (1 + HALF) + dw.abs() * (HALF + 4 * U) + TINY[BF])


SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 7, 72), (5, 257, 136), (64, 5003, 128), (128, 300, 520), (129, 255, 64), (129, 1, 8), (200, 256, 264),
          (300, 1031, 72), (515, 2100, 40), (1000, 513, 1024), (1300, 300, 64), (27, 4001, 1176), (40, 1000, 4104)]


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_cross_entropy(G, T, V, H):
    x, w, ids, _ = loss_case(T, V, H, T + V + H)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    for g in (torch.full((T,), 1 / 3, device="cuda"), _normal(_gen(1), T)):
        e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)


@pytest.mark.parametrize("s", [1.0, 2.5])
@pytest.mark.parametrize("T,V,H,K", [(1, 1, 8, 1), (1, 1000, 64, 20), (3, 7, 72, 128), (64, 5003, 128, 33), (129, 255, 64, 5), (300, 1031, 72, 64),
                                     (515, 2100, 40, 1)])
def test_distill(G, T, V, H, K, s):
    x, w, ids, teacher = loss_case(T, V, H, T + V + H + K, K)
    e = Exact(x, w, ids, teacher, s)
    o = G.distill_rows(x, w, ids, teacher, temperature=s)
    e.check_rows(o)
    for g in (torch.full((T,), 1 / 3, device="cuda"), _normal(_gen(1), T)):
        e.check_grad(G.distill_grad(x, w, ids, teacher, o["lse"], g, temperature=s), g)


@pytest.mark.parametrize("T,V,H", [(2049, 140001, 16), (8300, 515, 24)])
def test_pieces_of_the_vocabulary_and_slabs_of_rows(G, T, V, H):
    """More logits than a piece of their differences holds, more rows than a slab of the tiles' sums."""
    x, w, ids, _ = loss_case(T, V, H, 5)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    g = torch.full((T,), 1 / T, device="cuda")
    e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)
