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


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,H", [(617, 513), (700, 1135), (1300, 2049), (650, 5003), (640, 8191), (620, 8192), (1000, 24), (2600, 97), (1301, 301), (900, 512)])
def test_layer_norm_of_many_rows(G, dtype, T, H):
    """Rows that start anywhere, in all tensors the same way and not; both directions."""
    g = _gen(T + H)
    w, b = (1 + _normal(g, H, by=0.3)).to(dtype), _normal(g, H, to=dtype)
    for offs in ((0, 0, 0), (1, 1, 1), (0, 1, 3)):
        x, r, dy = (torch.cat([_normal(g, T, H, to=dtype).view(-1), w.new_zeros(8)]).roll(o)[o:o + T * H].view(T, H) for o in offs)
        x[:, ::29] *= 20
        o = G.layer_norm_rows(x, w, bias=b, residual=r)
        check_layer_norm(x, w, b, r, 1e-5, o)
        check_layer_norm(x, w, None, None, 1e-5, G.layer_norm_rows(x, w))
        n = G.layer_norm_rows(x, w)
        check_layer_norm_grad(dy, x, w, n["mean"], n["rstd"], r, G.layer_norm_grad(dy, x, w, n["mean"], n["rstd"], dresidual=r))
        check_layer_norm_grad(dy, x, w, n["mean"], n["rstd"], None, G.layer_norm_grad(dy, x, w, n["mean"], n["rstd"]))
        again = G.layer_norm_grad(dy, x, w, n["mean"], n["rstd"], dresidual=r, out=dict(dx=dy.clone() if offs[2] == 0 else torch.empty_like(x)))
        check_layer_norm_grad(dy, x, w, n["mean"], n["rstd"], r, again)


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


# ------------------------------------------------------------------------------ where losses can go wrong
@pytest.mark.parametrize("T", [20, 300])
def test_rows_left_out_may_hold_anything(G, T):
    """NaN and infinities in rows without an id reach nothing; all rows left out is zeros; an id beyond the vocabulary is NaN
    for its row alone, and no gradient."""
    x, w, ids, _ = loss_case(T, 700, 72, T)
    ids[3], ids[7] = 700, 2 ** 31 - 1
    ids[5] = -1
    x[ids < 0] = math.nan
    x[5, 3] = math.inf
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    assert o["loss"][3].isnan() and o["lse"][7].isnan() and (o["loss"][ids < 0] == 0).all() and (o["lse"][ids < 0] == 0).all()
    g = torch.ones(T, device="cuda")
    d = G.cross_entropy_grad(x, w, ids, o["lse"], g)
    e.check_grad(d, g)
    assert (d["dx"][ids < 0] == 0).all() and (d["dx"][3] == 0).all()
    g[::2] = 0.0  # rows without weight take no part either, whatever their lse
    lse = o["lse"].clone()
    lse[::2] = math.nan
    d = G.cross_entropy_grad(x, w, ids, lse, g)
    e.check_grad(d, g)
    assert (d["dx"][::2] == 0).all()
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    o = G.cross_entropy_rows(x, w, none)
    assert (o["loss"] == 0).all() and (o["lse"] == 0).all()
    out = dict(dx=torch.full((T, 72), 5.0, device="cuda").to(BF), dw=torch.full((700, 72), 5.0, device="cuda").to(BF))
    d = G.cross_entropy_grad(x, w, none, o["lse"], torch.ones(T, device="cuda"), out=out)
    assert (d["dx"] == 0).all() and (d["dw"] == 0).all()
    empty = G.cross_entropy_grad(x[:0], w, none[:0], o["lse"][:0], o["lse"][:0], out=dict(dw=torch.full((700, 72), 5.0, device="cuda").to(BF)))
    assert (empty["dw"] == 0).all() and empty["dx"].shape == (0, 72)
    assert G.cross_entropy_rows(x[:0], w, none[:0])["loss"].numel() == 0


@pytest.mark.parametrize("T", [20, 300])
def test_a_broken_row_keeps_to_itself(G, T):
    """A NaN in a row that takes part: its loss, lse and dx, and what the formula makes of dw; no other row's."""
    x, w, ids, _ = loss_case(T, 600, 64, T, skip=0.0)
    x[4, 9] = math.nan
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    assert o["loss"][4].isnan() and o["lse"][4].isnan()
    rest = torch.arange(T, device="cuda") != 4
    near(o["loss"][rest], e.loss[rest], e.off_loss[rest])
    g = torch.ones(T, device="cuda")
    d = G.cross_entropy_grad(x, w, ids, o["lse"], g)
    assert d["dx"][4].isnan().all() and not d["dx"][rest].isnan().any() and d["dw"].isnan().all()
    r = Exact(x[rest], w, ids[rest])
    d = G.cross_entropy_grad(x[rest].contiguous(), w, ids[rest].contiguous(), o["lse"][rest].contiguous(), g[rest])
    r.check_grad(d, g[rest])


def test_infinite_logits(G):
    """A logit of -inf has no part in the sum; one of +inf makes lse infinite, as log of a sum with it is."""
    w = torch.zeros(300, 8, device="cuda").to(BF)
    x = torch.zeros(3, 8, device="cuda").to(BF)
    x[:, 0] = 1.0
    w[:, 0] = 1.0
    w[7, 0], w[200, 0] = -math.inf, 2.0
    ids = torch.tensor([200, 7, 3], dtype=torch.int32, device="cuda")
    o = G.cross_entropy_rows(x, w, ids)
    lse = math.log(298 * math.e + math.exp(2.0))
    near(o["lse"], torch.full((3,), lse, device="cuda"), torch.full((3,), 1e-5, device="cuda"))
    near(o["loss"], torch.tensor([lse - 2.0, math.inf, lse - 1.0], device="cuda"), torch.full((3,), 1e-5, device="cuda"))
    w[9, 0] = math.inf
    assert (G.cross_entropy_rows(x, w, ids)["lse"] == math.inf).all()


def test_large_logits(G):
    """Logits of thousands: the sum of exponentials is about the largest."""
    x, w, ids, _ = loss_case(150, 1000, 64, 3)
    x = (x.float() * 300).to(BF)
    e = Exact(x, w, ids)
    assert float(e.lse.abs().max()) > 2000
    e.check_rows(G.cross_entropy_rows(x, w, ids))


@pytest.mark.parametrize("T", [33, 260])
def test_the_same_id_twice_and_few_tokens(G, T):
    """A teacher that names a token several times, rows with one token, with none, with all -inf, and of one only probability."""
    x, w, ids, teacher = loss_case(T, 500, 64, T, K=40)
    ids[1, :] = 17
    ids[2, 1:] = -1
    ids[2, 0] = 499
    ids[3] = -1
    teacher[4] = -math.inf
    ids[6, 5] = 500
    ids[8, ::2] = ids[8, 1::2]
    teacher[9] = 200.0 * torch.arange(40, device="cuda")  # all but one underflow
    e = Exact(x, w, ids, teacher, 0.7)
    o = G.distill_rows(x, w, ids, teacher, temperature=0.7)
    e.check_rows(o)
    assert o["loss"][3] == 0 and o["loss"][4] == 0
    assert bool(o["loss"][6].isnan()) == (float(teacher[6, 5]) > -math.inf)  # an id beyond the vocabulary, if it is there at all
    g = torch.ones(T, device="cuda")
    e.check_grad(G.distill_grad(x, w, ids, teacher, o["lse"], g, temperature=0.7), g)


@pytest.mark.parametrize("T", [33, 260])
def test_a_teachers_id_beyond_the_vocabulary(G, T):
    """It makes its row's loss and lse NaN and takes the row out of the gradients; one that the teacher rules out is not there."""
    x, w, ids, teacher = loss_case(T, 500, 64, T + 1, K=7, skip=0.0)
    ids[5, 2], teacher[5, 2] = 500, 1.0
    ids[6, 3], teacher[6, 3] = 2 ** 31 - 1, -math.inf
    e = Exact(x, w, ids, teacher)
    o = G.distill_rows(x, w, ids, teacher)
    e.check_rows(o)
    assert o["loss"][5].isnan() and o["lse"][5].isnan() and not o["loss"][6].isnan()
    g = torch.ones(T, device="cuda")
    d = G.distill_grad(x, w, ids, teacher, o["lse"], g)
    e.check_grad(d, g)
    assert (d["dx"][5] == 0).all()


@pytest.mark.parametrize("T", [40, 300])
def test_strides_gaps_and_parts_of_the_outputs(G, T):
    """Rows inside wider tensors; the gaps stay as they are; dx alone, dw alone; dw on 16 bytes and no more."""
    V, H = 333, 72
    x, w, ids, _ = loss_case(T, V, H, 9)
    for gap, off in ((8, 0), (24, 8), (56, 16)):
        def wide(n, fill=None):
            t = torch.full((n, H + gap), -7.0, device="cuda").to(BF)
            if fill is not None:
                t[:, off:off + H] = fill
            return t, t[:, off:off + H]
        xs, ws = wide(T, x)[1], wide(V, w)[1]
        e = Exact(x, w, ids)
        o = G.cross_entropy_rows(xs, ws, ids)
        e.check_rows(o)
        g = _normal(_gen(2), T)
        (xb, dx), (wb, dw) = wide(T), wide(V)
        full = G.cross_entropy_grad(xs, ws, ids, o["lse"], g, out=dict(dx=dx, dw=dw))
        e.check_grad(full, g)
        for buf in (xb, wb):
            assert (torch.cat([buf[:, :off], buf[:, off + H:]], 1).float() == -7.0).all()
        a = G.cross_entropy_grad(xs, ws, ids, o["lse"], g, dw=False)
        b = G.cross_entropy_grad(xs, ws, ids, o["lse"], g, dx=False)
        assert set(a) == {"dx"} and set(b) == {"dw"}
        assert torch.equal(a["dx"], dx) and torch.equal(b["dw"], dw)


@pytest.mark.parametrize("T,V,H", [(1, 1000, 64), (96, 5000, 264), (700, 3000, 136)])
def test_the_same_call_gives_the_same_bits(G, T, V, H):
    x, w, ids, teacher = loss_case(T, V, H, 4, K=20)
    g = _normal(_gen(2), T)

    def call():
        o = G.distill_rows(x, w, ids, teacher)
        return dict(o, **G.distill_grad(x, w, ids, teacher, o["lse"], g))

    first = call()
    for _ in range(5):
        again = call()
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("T", [40, 300])
def test_loss_gradients_against_differences(G, T):
    """(f(x + e u) - f(x - e u)) / 2e of f = sum of g loss in 64 bits, along random directions of the rows and of the head."""
    x, w, ids, teacher = loss_case(T, 300, 64, 6, K=8)
    g, s = torch.rand(T, device="cuda", generator=_gen(3)) + 0.5, 1.5
    o = G.distill_rows(x, w, ids, teacher, temperature=s)
    d = G.distill_grad(x, w, ids, teacher, o["lse"], g, temperature=s)

    def f(xx, ww):
        return (Exact(xx, ww, ids, teacher, s).loss * g.double()).sum()

    step = 1e-5
    for key, at in (("dx", 0), ("dw", 1)):
        u = _normal(_gen(7 + at), *d[key].shape).double()
        args = [x.double(), w.double()]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + step * u, args[at] - step * u
        want = float((f(*up) - f(*down)) / (2 * step))
        got = float((d[key].double() * u).sum())
        # each element of the gradient may be off by a rounding of dz and one of its own
        assert abs(want - got) < 3 * HALF * float(d[key].double().norm() * u.norm()) / math.sqrt(u.numel()) + 1e-6 * abs(want) + 3 * HALF * float(d[key].double().norm())


# ------------------------------------------------------------------------------ streams, graphs, neighbours
def _step(G, x, r, ids, w, nw, nb, g, out=None):
    n = G.layer_norm_rows(x, nw, bias=nb, residual=r)
    o = G.cross_entropy_rows(n["y"], w, ids)
    d = G.cross_entropy_grad(n["y"], w, ids, o["lse"], g)
    e = G.layer_norm_grad(d["dx"], n["residual"], nw, n["mean"], n["rstd"])
    return dict(loss=o["loss"], dw=d["dw"], y=n["y"], **e)


def _step_case(T, V, H, seed):
    g = _gen(seed)
    x, w, ids, _ = loss_case(T, V, H, seed)
    return dict(x=x, r=_normal(g, T, H, to=BF), ids=ids, w=w, nw=(1 + _normal(g, H, by=0.2)).to(BF), nb=_normal(g, H, by=0.1, to=BF),
                g=torch.full((T,), 1.0 / T, device="cuda"))


@pytest.mark.parametrize("T", [60, 400])
def test_a_step_of_the_end_of_a_model(G, T):
    """Norm, head, loss and back to the norm's input, against the whole in 64 bits by automatic differentiation."""
    c = _step_case(T, 900, 136, T)
    o = _step(G, **c)
    leaf = {k: c[k].double().requires_grad_() for k in ("x", "w", "nw", "nb")}
    h = leaf["x"] + c["r"].double()
    v = (h - h.mean(1, keepdim=True)) / (h.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    z = (v * leaf["nw"] + leaf["nb"]) @ leaf["w"].T
    ok = c["ids"] >= 0
    loss = (torch.logsumexp(z, 1) - z.gather(1, c["ids"].clamp(min=0).long()[:, None])[:, 0]) * ok
    (loss * c["g"].double()).sum().backward()
    # y is rounded before the head, dz and the gradient of y before what follows: a few roundings of the norms
    for got, want in ((o["loss"], loss), (o["dw"], leaf["w"].grad), (o["dx"], leaf["x"].grad), (o["dweight"], leaf["nw"].grad), (o["dbias"], leaf["nb"].grad)):
        assert float((got.double() - want).norm()) <= 4 * HALF * float(want.norm())


def test_on_another_stream(G):
    c, side = _step_case(200, 600, 72, 1), torch.cuda.Stream()
    want = _step(G, **c)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = _step(G, **c)
    side.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    o = G.cross_entropy_rows(want["y"], c["w"], c["ids"], stream=side)
    d = G.cross_entropy_grad(want["y"], c["w"], c["ids"], o["lse"], c["g"], stream=side)
    n = G.layer_norm_rows(c["x"], c["nw"], bias=c["nb"], residual=c["r"], stream=side)
    side.synchronize()
    assert torch.equal(o["loss"], want["loss"]) and torch.equal(d["dw"], want["dw"]) and torch.equal(n["y"], want["y"])


def test_two_streams_at_once(G):
    """Calls on two streams have workspaces of their own and do not disturb one another."""
    cases = [_step_case(T, 4000, 136, T) for T in (90, 500)]
    want = [_step(G, **c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_step(G, **cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert all(torch.equal(want[i][k], o[k]) for k in o)
    assert G.tail_errors() == 0


@pytest.mark.parametrize("T", [60, 400])
def test_captured_and_replayed(G, T):
    """A captured step follows its inputs from replay to replay, rows that are left out among them."""
    c = _step_case(T, 900, 72, 2)
    _step(G, **c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(G, **c)
    for seed in (3, 4):
        n = _step_case(T, 900, 72, seed)
        for k in c:
            c[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        want = _step(G, **n)
        assert all(torch.equal(want[k], out[k]) for k in want)


def test_a_teacher_from_the_sampler(G):
    """What ``Sampler.logprobs`` reports of a teacher's rows goes to the distillation of a student as it is."""
    V, H, T, K = 5000, 128, 48, 20
    x, w, _, _ = loss_case(T, V, H, 8)
    logits = G.project_rows(x, w)
    with G.Sampler(device=0, max_slots=T, max_vocab=V, max_rows=T) as s:
        top = s.logprobs(logits, top_n=K)
        torch.cuda.synchronize()
    student = (w.float() + 0.02 * _normal(_gen(1), V, H)).to(BF)
    ids, teacher = top["top_ids"], top["top_lps"]
    o = G.distill_rows(x, student, ids, teacher)
    e = Exact(x, student, ids, teacher)
    e.check_rows(o)
    g = torch.full((T,), 1 / T, device="cuda")
    e.check_grad(G.distill_grad(x, student, ids, teacher, o["lse"], g), g)
    same = G.distill_rows(x, w, ids, teacher)["loss"]
    assert (same < o["loss"]).float().mean() > 0.5 and (same > -1e-4).all()


def test_between_other_operators_of_a_stream(G):
    """Norm, projection, losses and draws behind one another, each set up while the one before runs: the same as one by one."""
    g = _gen(12)
    T, V, H = 64, 3000, 264
    x, w, ids, _ = loss_case(T, V, H, 12)
    nw = torch.ones(H, device="cuda").to(BF)
    u = torch.rand(T, generator=g, device="cuda")

    def chain(wait):
        out = []
        for _ in range(6):
            n = G.norm_rows(x, nw)["y"]
            wait()
            l = G.project_rows(n, w)
            wait()
            o = G.cross_entropy_rows(n, w, ids)
            wait()
            i = G.draw_rows(l, u)["ids"]
            wait()
            d = G.cross_entropy_grad(n, w, i, o["lse"], u)
            wait()
            out += [n, l, o["loss"], i, d["dx"], d["dw"]]
        return out

    want = chain(torch.cuda.synchronize)
    got = chain(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_the_c_names_write_into_the_callers_tensors(G):
    T, V, H = 30, 400, 64
    x, w, ids, teacher = loss_case(T, V, H, 15, K=6)
    one = ids[:, 0].contiguous()
    g = torch.ones(T, device="cuda")
    f = lambda *shape, t=F32: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    ws = lambda K, grad: f(G.strata_loss_workspace(T, V, H, K, grad), t=torch.uint8)  # noqa: E731
    loss, lse, dx, dw = f(T), f(T), f(T, H, t=BF), f(V, H, t=BF)
    G.strata_cross_entropy_rows(x, w, one, loss, lse, ws(0, False))
    G.strata_cross_entropy_grad(x, w, one, lse, g, dx, dw, ws(0, True))
    o = G.cross_entropy_rows(x, w, one)
    d = G.cross_entropy_grad(x, w, one, o["lse"], g)
    assert torch.equal(loss, o["loss"]) and torch.equal(lse, o["lse"]) and torch.equal(dx, d["dx"]) and torch.equal(dw, d["dw"])
    G.strata_distill_rows(x, w, ids, teacher, 2.0, loss, lse, ws(6, False))
    G.strata_distill_grad(x, w, ids, teacher, 2.0, lse, g, dx, dw, ws(6, True))
    o = G.distill_rows(x, w, ids, teacher, temperature=2.0)
    d = G.distill_grad(x, w, ids, teacher, o["lse"], g, temperature=2.0)
    assert torch.equal(loss, o["loss"]) and torch.equal(lse, o["lse"]) and torch.equal(dx, d["dx"]) and torch.equal(dw, d["dw"])
    mean, rstd, y, nw = f(T), f(T), f(T, H, t=BF), torch.ones(H, device="cuda").to(BF)
    G.strata_layer_norm_rows(x, nw, y=y, mean=mean, rstd=rstd)
    n = G.layer_norm_rows(x, nw)
    assert torch.equal(y, n["y"]) and torch.equal(mean, n["mean"]) and torch.equal(rstd, n["rstd"])
    dn, db = f(H, t=BF), f(H, t=BF)
    G.strata_layer_norm_grad(y, x, nw, mean, rstd, dx=dx, dweight=dn, dbias=db, workspace=f(G.strata_layer_norm_workspace(T, H), t=torch.uint8))
    d = G.layer_norm_grad(y, x, nw, mean, rstd)
    assert torch.equal(dx, d["dx"]) and torch.equal(dn, d["dweight"]) and torch.equal(db, d["dbias"])


def test_refusals_on_tensors(G):
    x, w, ids, teacher = loss_case(8, 100, 64, 1, K=4)
    one, lse = ids[:, 0].contiguous(), torch.zeros(8, device="cuda")
    for call in (lambda: G.cross_entropy_rows(x[:, :60], w[:, :60], one), lambda: G.cross_entropy_rows(x, w[:, 8:], one),
                 lambda: G.cross_entropy_rows(x, w, one[:4]), lambda: G.cross_entropy_rows(x.t(), w, one),
                 lambda: G.distill_rows(x, w, ids, teacher[:, :3]), lambda: G.distill_rows(x, w, ids, teacher, temperature=0.0),
                 lambda: G.cross_entropy_grad(x, w, one, lse[:3], lse), lambda: G.cross_entropy_grad(x, w, one, lse, lse, dx=False, dw=False),
                 lambda: G.layer_norm_grad(x, x, x[0], lse, lse[:2]), lambda: G.layer_norm_rows(x, x[0, :60])):
        with pytest.raises((ValueError, G.StrataError)):
            call()
    for call in (lambda: G.cross_entropy_rows(x, w, one.long()), lambda: G.cross_entropy_rows(x, w.float(), one),
                 lambda: G.distill_rows(x, w, ids, teacher.to(BF)), lambda: G.layer_norm_rows(x, x[0].float())):
        with pytest.raises(TypeError):
            call()
    assert G.tail_errors() == 0


@pytest.mark.parametrize("T,V,H", [(129, 20000, 256), (700, 5000, 512), (1024, 20000, 264), (260, 100000, 128), (2000, 40000, 512), (600, 70000, 1024)])
def test_tiles_of_one_sm_and_of_two(G, T, V, H):
    """Sizes on both sides of the choices between tiles, and between the rows themselves and a copy of them."""
    x, w, ids, _ = loss_case(T, V, H, 21, skip=0.3)
    x[ids < 0] = math.nan
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    g = torch.full((T,), 1 / T, device="cuda")
    e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)


@pytest.mark.parametrize("T", [5, 200])
def test_the_largest_id_is_beyond_the_vocabulary_too(G, T):
    x, w, ids, teacher = loss_case(T, 90, 64, T, K=3, skip=0.0)
    ids[2, 1], teacher[2, 1] = 2 ** 31 - 1, 0.5
    ids[3, :] = 2 ** 31 - 1
    teacher[3] = 0.0
    e = Exact(x, w, ids, teacher)
    o = G.distill_rows(x, w, ids, teacher)
    e.check_rows(o)
    assert o["loss"][2].isnan() and o["lse"][3].isnan()
    d = G.distill_grad(x, w, ids, teacher, o["lse"], torch.ones(T, device="cuda"))
    e.check_grad(d, torch.ones(T, device="cuda"))


def test_an_infinite_logit_beside_large_ones(G):
    """lse is infinite whatever else there is, in its tile and in others."""
    w = torch.zeros(2000, 8, device="cuda").to(BF)
    w[:, 0] = 150.0
    w[1500, 0] = math.inf
    x = torch.zeros(2, 8, device="cuda").to(BF)
    x[:, 0] = torch.tensor([1.0, 20.0])
    o = G.cross_entropy_rows(x, w, torch.tensor([3, 1500], dtype=torch.int32, device="cuda"))
    assert (o["lse"] == math.inf).all() and o["loss"][0] == math.inf and o["loss"][1].isnan()


@pytest.mark.parametrize("T,V,H", [(3, 200, 32768), (2, 524288, 16), (131072, 300, 8), (140, 70, 32768)])
def test_the_largest_sizes(G, T, V, H):
    x, w, ids, _ = loss_case(T, V, H, 2)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    g = torch.full((T,), 1 / T, device="cuda")
    e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)


@pytest.mark.parametrize("T", [50, 300])
def test_scales_of_any_size_and_sign(G, T):
    """One negative scale for all rows, scales that differ by 2^60, an infinite and a NaN one beside others."""
    x, w, ids, _ = loss_case(T, 400, 64, T + 3, skip=0.0)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    for g in (torch.full((T,), -3e-5, device="cuda"), 2.0 ** torch.linspace(-40, 20, T, device="cuda") * torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)):
        e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)
    for bad in (math.nan, math.inf):
        g = torch.ones(T, device="cuda")
        g[7] = bad
        d = G.cross_entropy_grad(x, w, ids, o["lse"], g)
        rest = torch.arange(T, device="cuda") != 7
        want = G.cross_entropy_grad(x, w, ids, o["lse"], torch.ones(T, device="cuda"))["dx"]
        assert torch.equal(d["dx"][rest], want[rest]) and not d["dx"][7].isfinite().any()
        assert not d["dw"][ids[7].long()].isfinite().any()


@pytest.mark.parametrize("T,V,H", [(1, 2000, 64), (100, 5000, 128), (400, 3000, 64)])
def test_losses_near_zero_keep_their_digits(G, T, V, H):
    """Rows that are all but sure of their token: the loss is log(1 + the sum over the other ids of exp(z - z of the id)), to whose
    terms an error of z is a relative one."""
    x, w, ids, _ = loss_case(T, V, H, 31, skip=0.0)
    x = (x.float() + 8 * w[ids.long()].float()).to(BF)
    e = Exact(x, w, ids)
    z = x.double() @ w.double().T
    at = ids.long()[:, None]
    others = (z - z.gather(1, at)).exp().scatter_(1, at, 0.0).sum(1)
    want = torch.log1p(others)
    assert float(want.min()) < 1e-6
    o = G.cross_entropy_rows(x, w, ids)
    near(o["loss"], want, want * (2 * e.off_z.amax(1) + (V / 256 + 316) * U))
    e.check_rows(o)


def test_outputs_that_share_an_allocation_are_apart(G):
    """Small outputs of a call lie in one allocation: each is whole, contiguous and does not touch another's elements, also with
    some of them given, and large ones beside."""
    g = _gen(40)
    for T, H in ((1, 8), (3, 40), (9, 256), (40, 4096), (5000, 8)):
        x, w, b, r = _normal(g, T, H, to=BF), (1 + _normal(g, H, by=0.2)).to(BF), _normal(g, H, to=BF), _normal(g, T, H, to=BF)
        mine = torch.full((T,), -1.0, device="cuda")
        for out in ({}, dict(mean=mine), dict(y=torch.empty_like(x), rstd=None)):
            o = G.layer_norm_rows(x, w, bias=b, residual=r, out=dict(out))
            check_layer_norm(x, w, b, r, 1e-5, o)
            assert all(v.is_contiguous() and v.data_ptr() % 16 == 0 for v in o.values())
            spans = sorted((v.data_ptr(), v.data_ptr() + v.numel() * v.element_size()) for v in o.values())
            assert all(a[1] <= c[0] for a, c in zip(spans, spans[1:]))
        assert (mine != -1).any()
        d = G.layer_norm_grad(r, x, w, o["mean"], o["rstd"])
        check_layer_norm_grad(r, x, w, o["mean"], o["rstd"], None, d)
        given = torch.empty(H, dtype=BF, device="cuda")
        e = G.layer_norm_grad(r, x, w, o["mean"], o["rstd"], dweight=False, bias=False, out=dict(dweight=given))
        assert torch.equal(given, d["dweight"]) and set(e) == {"dx", "dweight"}
        spans = sorted((v.data_ptr(), v.data_ptr() + v.numel() * v.element_size()) for v in d.values())
        assert all(a[1] <= c[0] for a, c in zip(spans, spans[1:]))


@pytest.mark.parametrize("T,V,H", [(40000, 70, 72), (20000, 300, 264), (4100, 90, 4096)])
def test_dx_of_many_rows_in_one_part(G, T, V, H):
    """Enough tiles of dx that the sum over the ids is not cut: written straight to the rows that take part, any distance apart."""
    x, w, ids, _ = loss_case(T, V, H, 17, skip=0.4)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    g = _normal(_gen(5), T)
    buf = torch.full((T, H + 24), -7.0, device="cuda").to(BF)
    d = G.cross_entropy_grad(x, w, ids, o["lse"], g, dw=False, out=dict(dx=buf[:, 8:8 + H]))
    e.check_grad(d, g)
    assert (torch.cat([buf[:, :8], buf[:, 8 + H:]], 1).float() == -7.0).all()


@pytest.mark.parametrize("T,V,H,K", [(5, 777, 64, 0), (17, 3001, 1096, 5), (100, 513, 72, 0), (128, 300, 520, 3), (130, 1000, 64, 0), (700, 2100, 1096, 2),
                                     (1500, 130, 264, 0), (20000, 300, 72, 0)])
def test_what_the_workspace_held_before_does_not_matter(G, T, V, H, K):
    """A workspace full of NaN patterns, and outputs full of them: everything that is read has been written by the call."""
    x, w, ids, teacher = loss_case(T, V, H, T + K, K=K, skip=0.4)
    e = Exact(x, w, ids, teacher)
    g = _normal(_gen(1), T)
    f = lambda *shape, t=F32: torch.full(shape, math.nan, device="cuda").to(t)  # noqa: E731
    ws = lambda grad: torch.full((G.strata_loss_workspace(T, V, H, K, grad),), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    loss, lse, dx, dw = f(T), f(T), f(T, H, t=BF), f(V, H, t=BF)
    for scale in (g, torch.full_like(g, 0.25)):
        if K:
            G.strata_distill_rows(x, w, ids, teacher, 1.0, loss, lse, ws(False))
            G.strata_distill_grad(x, w, ids, teacher, 1.0, lse, scale, dx, dw, ws(True))
        else:
            G.strata_cross_entropy_rows(x, w, ids, loss, lse, ws(False))
            G.strata_cross_entropy_grad(x, w, ids, lse, scale, dx, dw, ws(True))
        e.check_rows(dict(loss=loss, lse=lse))
        e.check_grad(dict(dx=dx, dw=dw), scale)
    o = G.layer_norm_rows(x, w[0])
    y, mean, rstd, dn, db = f(T, H, t=BF), f(T), f(T), f(H, t=BF), f(H, t=BF)
    G.strata_layer_norm_rows(x, w[0], y=y, mean=mean, rstd=rstd)
    assert torch.equal(y, o["y"]) and torch.equal(rstd, o["rstd"])
    wn = torch.full((G.strata_layer_norm_workspace(T, H),), 255, dtype=torch.uint8, device="cuda")
    G.strata_layer_norm_grad(y, x, w[0], mean, rstd, dx=dx, dweight=dn, dbias=db, workspace=wn)
    check_layer_norm_grad(y, x, w[0], mean, rstd, None, dict(dx=dx, dweight=dn, dbias=db))


@pytest.mark.parametrize("T,V,H,K", [(1, 9, 8, 0), (17, 3001, 1096, 5), (100, 513, 72, 0), (130, 1000, 64, 128), (700, 2100, 1096, 2), (1500, 130, 264, 0),
                                     (2049, 140001, 16, 0)])
def test_nothing_is_written_behind_the_workspace_and_the_outputs(G, T, V, H, K):
    x, w, ids, teacher = loss_case(T, V, H, T + K, K=K, skip=0.1)
    g = torch.ones(T, device="cuda")
    guards = []

    def guarded(n, t):
        size = n * torch.empty(0, dtype=t).element_size()
        buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        guards.append(buf[size:])
        return buf[:size].view(t)

    loss, lse, dx, dw = guarded(T, F32), guarded(T, F32), guarded(T * H, BF).view(T, H), guarded(V * H, BF).view(V, H)
    ws, wg = (guarded(G.strata_loss_workspace(T, V, H, K, grad), torch.uint8) for grad in (False, True))
    if K:
        G.strata_distill_rows(x, w, ids, teacher, 1.0, loss, lse, ws)
        G.strata_distill_grad(x, w, ids, teacher, 1.0, lse, g, dx, dw, wg)
    else:
        G.strata_cross_entropy_rows(x, w, ids, loss, lse, ws)
        G.strata_cross_entropy_grad(x, w, ids, lse, g, dx, dw, wg)
    mean, rstd, y, dn, db = guarded(T, F32), guarded(T, F32), guarded(T * H, BF).view(T, H), guarded(H, BF), guarded(H, BF)
    wn = guarded(G.strata_layer_norm_workspace(T, H), torch.uint8)
    G.strata_layer_norm_rows(x, w[0], y=y, mean=mean, rstd=rstd)
    G.strata_layer_norm_grad(y, x, w[0], mean, rstd, dx=dx, dweight=dn, dbias=db, workspace=wn)
    torch.cuda.synchronize()
    assert all((b == 0xA5).all() for b in guards)


@pytest.mark.parametrize("T,V,H", [(1, 1310, 2056), (3, 2100, 8192), (33, 517, 4104), (128, 700, 2080), (9, 300, 32768), (130, 300, 32768)])
def test_sums_of_wide_rows(G, T, V, H):
    """Of products above 0 every partial sum is below the whole.  The tensor cores cut two times for 16 products (aligning them, and
    the sum), each time at most 2^-23 of what is there, and 64 such steps at most follow one another before sums are added up,
    rounded, at 2^-24: in all (128 + H / 2048) 2^-23 of z.  The rest of lse: scale * z and its way back, the maximum's
    rounding and the sum's, 8 * 2^-24 of it."""
    g = _gen(T + V + H)
    x = (0.5 + torch.rand(T, H, generator=g, device="cuda")).to(BF)
    w = ((0.5 + torch.rand(V, H, generator=g, device="cuda")) * (60.0 / H)).to(BF)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    o = G.cross_entropy_rows(x, w, ids)
    z = x.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    bound = (128 + H / 2048) * 2.0**-23 * z.amax(1) + 8 * 2.0**-24 * want
    assert bool(((o["lse"].double() - want).abs() <= bound).all())
