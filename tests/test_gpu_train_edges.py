"""Calls of the operators that score and train the end of a model at the edges of what they take."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_train import BF, F32, HALF, TINY, U, Exact, G, _gen, _normal, loss_case, near  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ rows that are sure of their token
def sure_case(T, V, H, seed):
    """Logits of the rows' own tokens from 16 to 32 among others of about +-2: 1 - p from about 1e-3 down to 1e-10."""
    g = _gen(seed)
    w = _normal(g, V, H, by=2 * H ** -0.5, to=BF)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    own = 4 + 4 * torch.rand(T, 1, generator=g, device="cuda")
    return (_normal(g, T, H) + own * w[ids.long()].float()).to(BF), w, ids


def check_sure(e, d, steps):
    """dz of a row's token is p - q, of which little is left: its error is that of z - lse, which is the rounding of lse where both calls
    took the same z: `steps` roundings of it, at 2^-24 each.  An error that z has in both moves the other ids' shares, by as much
    of themselves.  Then one rounding of dz to bfloat16, and the products' 32-bit sums and results as everywhere."""
    T, V = e.p.shape
    z_off = 2 * e.off_z.amax(1, keepdim=True)
    lse_off = steps * U * (e.lse.abs()[:, None] + 1)
    # p - q without the loss of digits: of the ids but a row's own p itself, of its own what the others leave of 1
    top = e.q.argmax(1, keepdim=True)
    rest = e.p.clone().scatter_(1, top, 0.0)
    left = e.q.clone().scatter_(1, top, 0.0).sum(1, keepdim=True) - rest.sum(1, keepdim=True)
    want = (rest - e.q).scatter_(1, top, left)
    off_d = (want.abs() * (z_off + HALF) + (e.p + e.q) * lse_off + rest * 2.0 ** -20) * (1 + HALF)
    dx, dw = want @ e.w * e.s, want.T @ e.clean * e.s
    near(d["dx"], dx, (off_d + want.abs() * (V / 16 + 32) * 2 * U) @ e.w.abs() * e.s * (1 + HALF) + dx.abs() * (HALF + 4 * U) + TINY[BF])
    near(d["dw"], dw, (off_d + want.abs() * (T / 16 + 32) * 2 * U).T @ e.clean.abs() * e.s * (1 + HALF) + dw.abs() * (HALF + 4 * U) + TINY[BF])


SURE = [(3, 1000, 520), (100, 1000, 2048), (100, 1000, 2056), (17, 600, 8192), (128, 500, 4096), (300, 1000, 1024), (300, 1000, 1032), (300, 1000, 4096),
        (700, 2100, 2056), (140, 300, 32768)]


@pytest.mark.parametrize("T,V,H", SURE)
def test_the_gradients_of_sure_rows(G, T, V, H):
    """The way back takes the logits that the way there took, bit for bit: lse is the sum's with one rounding, expm1 adds none of its size."""
    x, w, ids = sure_case(T, V, H, T + H)
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    check_sure(e, G.cross_entropy_grad(x, w, ids, o["lse"], torch.ones(T, device="cuda")), 3)


@pytest.mark.parametrize("s", [1.0, 0.5])
@pytest.mark.parametrize("T,V,H", [(100, 1000, 2048), (17, 600, 8192), (300, 1000, 1032), (300, 1000, 4096)])
def test_the_gradients_of_a_student_as_sure_as_its_teacher(G, T, V, H, s):
    """lse is a maximum in steps of log2 e / s and back, and the log of a sum: five roundings; z / s, q and 1 - q have three more."""
    x, w, one = sure_case(T, V, H, T + H + 1)
    ids = torch.stack([one, (one + 1) % V, (one + 7) % V], 1).contiguous()
    teacher = torch.tensor([30.0, 12.0, -4.0], device="cuda").repeat(T, 1)
    e = Exact(x, w, ids, teacher, s)
    o = G.distill_rows(x, w, ids, teacher, temperature=s)
    check_sure(e, G.distill_grad(x, w, ids, teacher, o["lse"], torch.ones(T, device="cuda"), temperature=s), 8)


# ------------------------------------------------------------------------------ a teacher's largest and smallest values
@pytest.mark.parametrize("s", [1.0, 0.7, 0.001, 1000.0])
@pytest.mark.parametrize("T", [9, 200])
def test_a_teachers_values_at_the_types_ends(G, T, s):
    """Finite values are there, whatever the temperature: the lowest one beside others has no share, all of them the same are equal shares."""
    x, w, ids, teacher = loss_case(T, 500, 64, T, K=6, skip=0.0)
    ids = torch.randint(0, 500, (T, 6), generator=_gen(T), device="cuda", dtype=torch.int32)
    teacher[teacher == -math.inf] = 0.0
    low, high = torch.finfo(F32).min, torch.finfo(F32).max
    teacher[0] = low
    teacher[1, 1:] = low
    teacher[2] = high
    teacher[3, ::2] = high
    teacher[4] = low
    teacher[4, 2:] = -math.inf
    teacher[5] = low
    ids[5, 3] = 500  # beyond the vocabulary, and there
    teacher[6] = 0.9 * low
    teacher[6, 1] = high
    e = Exact(x, w, ids, teacher, s)
    o = G.distill_rows(x, w, ids, teacher, temperature=s)
    assert o["loss"][5].isnan() and not o["loss"][:5].isnan().any()
    e.check_rows(o)
    g = torch.ones(T, device="cuda")
    e.check_grad(G.distill_grad(x, w, ids, teacher, o["lse"], g, temperature=s), g)


# ------------------------------------------------------------------------------ no rows
def test_no_rows_and_dx_alone(G):
    """An empty batch asked for dx alone gets an empty dx."""
    x, w, ids, teacher = loss_case(4, 50, 64, 1, K=3)
    none = torch.zeros(0, device="cuda")
    d = G.cross_entropy_grad(x[:0], w, ids[:0, 0].contiguous(), none, none, dw=False)
    assert set(d) == {"dx"} and d["dx"].shape == (0, 64)
    d = G.distill_grad(x[:0], w, ids[:0], teacher[:0], none, none, dw=False)
    assert set(d) == {"dx"} and d["dx"].shape == (0, 64)
    d = G.layer_norm_grad(x[:0], x[:0], w[0], none, none, dweight=False, bias=False)
    assert set(d) == {"dx"} and d["dx"].shape == (0, 64)


# ------------------------------------------------------------------------------ what a kept output keeps
def test_a_kept_output_does_not_keep_the_workspace(G):
    """Small outputs share an allocation with one another, and with nothing else."""
    x, w, ids, teacher = loss_case(4, 400, 64, 1, K=6, skip=0.0)
    one, g = ids[:, 0].contiguous(), torch.ones(4, device="cuda")
    n = G.layer_norm_rows(x, w[0])
    lse = torch.zeros(4, device="cuda")
    for o in (G.cross_entropy_rows(x, w, one), G.distill_rows(x, w, ids, teacher), n, G.layer_norm_grad(x, x, w[0], n["mean"], n["rstd"]),
              G.cross_entropy_grad(x, w, one, lse, g, dw=False), G.distill_grad(x, w, ids, teacher, lse, g, dw=False)):
        own = sum((t.numel() * t.element_size() + 255) // 256 * 256 for t in o.values())
        for t in o.values():
            assert t.untyped_storage().nbytes() <= own


# ------------------------------------------------------------------------------ automatic differentiation
def test_gradients_that_nothing_records_are_told(G):
    """Automatic differentiation passes these calls by: one that it would have to record says so."""
    import warnings
    x, w, ids, teacher = loss_case(4, 400, 64, 1, K=6, skip=0.0)
    one = ids[:, 0].contiguous()
    leaf, head = x.clone().requires_grad_(), w.clone().requires_grad_()
    for call in (lambda x, w: G.cross_entropy_rows(x, w, one), lambda x, w: G.distill_rows(x, w, ids, teacher), lambda x, w: G.layer_norm_rows(x, w[0].detach())):
        with pytest.warns(UserWarning, match="not recorded"):
            o = call(leaf, w)
        assert not any(t.requires_grad for t in o.values())
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(x, w)
            with torch.no_grad():
                call(leaf, head)
            call(leaf.detach(), head.detach())
    with pytest.warns(UserWarning, match="not recorded"):
        G.cross_entropy_rows(x, head, one)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):
            G.cross_entropy_rows(leaf, w, one)
    assert G.tail_errors() == 0


# ------------------------------------------------------------------------------ accumulators that go from tile to tile
# rows, ids, width: blocks with several tiles one after another, of two SMs and of one, whose logits are one sum, two, or runs of an even or
# an odd number (tests/loss_kinds_check.cu holds which they are)
KINDS = [(400, 90000, 1088), (500, 50000, 2056), (600, 40000, 1032), (100, 60000, 2056), (64, 90000, 576), (100, 90000, 1536), (90, 120000, 264),
         (2000, 40000, 520)]


@pytest.mark.parametrize("T,V,H", KINDS)
def test_sums_handed_from_tile_to_tile(G, T, V, H):
    x, w, ids, _ = loss_case(T, V, H, T + H)
    x[ids < 0] = math.nan
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    e.check_rows(o)
    g = _normal(_gen(1), T)
    e.check_grad(G.cross_entropy_grad(x, w, ids, o["lse"], g), g)
    again = G.cross_entropy_rows(x, w, ids)
    assert all(torch.equal(o[k], again[k]) for k in o) and G.tail_errors() == 0


@pytest.mark.parametrize("T,V,H", [(400, 90000, 1088), (500, 50000, 2056), (100, 60000, 2056), (64, 90000, 576)])
def test_the_gradients_of_sure_rows_over_many_tiles(G, T, V, H):
    x, w, ids = sure_case(T, V, H, T + H)
    x = (x.float() + 2 * w[ids.long()].float()).to(BF)  # sure among more ids, too
    e = Exact(x, w, ids)
    o = G.cross_entropy_rows(x, w, ids)
    check_sure(e, G.cross_entropy_grad(x, w, ids, o["lse"], torch.ones(T, device="cuda")), 3)
