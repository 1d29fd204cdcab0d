"""Calls of the operators around the sampler at the edges of what they take, and next to the sampler's own calls."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    import request_token_sampling_gb300 as G
    return G


# ------------------------------------------------------------------------------ draw_rows
@pytest.mark.parametrize("dtype", [F32, BF])
def test_draw_refuses_ids_beyond_the_rows(G, dtype):
    """V is at most the rows' width: columns beyond it belong to somebody else, or to nobody."""
    u = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    one = torch.zeros(1, 1001, dtype=dtype, device="cuda")
    many = torch.zeros(3, 1024, dtype=dtype, device="cuda")
    for x, V in ((one, 1002), (one, 1008), (many[:, :1000], 1001), (many[:, :1000], 1024), (many, 1025), (many, 0), (many, -1),
                 (many, -2 ** 31), (many, 5 - 2 ** 32), (many, 5 + 2 ** 32), (one[:0], 1002)):
        with pytest.raises(ValueError):
            G.draw_rows(x, u(x.shape[0]), V=V)
    assert G.draw_rows(one, u(1), V=1001)["ids"].tolist() == [0]
    assert G.draw_rows(many[:, :1000], u(3), V=1000)["ids"].tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [304, 5000, 40000])
def test_draw_infinity_above_the_largest_finite_logits(G, dtype, V):
    """An infinite logit weighs all; the greatest finite ones beside it are next in order, whatever the cut."""
    from test_gpu_tail import check_draw
    big = torch.finfo(dtype).max
    B = 8
    x = torch.full((B, V), big, dtype=dtype, device="cuda")
    x[:, V // 3] = math.inf
    x[2, 5 * V // 6] = math.inf
    x[3, ::2] = big / 2
    x[4, 1::3] = -big
    x[5, ::2] = torch.randn((V + 1) // 2, generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").to(dtype)
    x[6, ::3] = math.nan
    x[6, V // 3] = math.inf
    x[7] = big
    u = [(b + 0.5) / B for b in range(B)]
    check_draw(G, x, u)
    for k in (1, 2, 60, V // 2, V - 1):
        check_draw(G, x, u, k=[k] * B)
        check_draw(G, x, u, k=[k] * B, p=[0.9] * B, m=[0.0, 0.1] * (B // 2))
        out = dict(ids=torch.full((B,), -7, dtype=torch.int32, device="cuda"), lps=torch.full((B,), -7.0, device="cuda"))
        o = G.draw_rows(x, torch.tensor(u, device="cuda"), top_k=torch.full((B,), k, dtype=torch.int32, device="cuda"), out=out)
        assert (o["ids"] >= 0).all() and (o["lps"] <= 0).all() and (o["lps"] > -20).all()
    check_draw(G, x, u, p=[0.5, 0.99] * (B // 2))
    check_draw(G, x, u, m=[0.5] * B, t=[0.3] * B)


# ------------------------------------------------------------------------------ norm_rows
def test_norm_of_as_many_rows_as_an_int_counts(G):
    T = 2 ** 31 - 2
    x = torch.ones(T, 1, dtype=BF, device="cuda")
    x[::3] = -2
    y = G.norm_rows(x, torch.full((1,), 3.0, dtype=BF, device="cuda"), eps=0.0)["y"]
    x.sign_().mul_(3)
    assert y.shape == (T, 1)
    for at in range(0, T, 1 << 28):
        assert torch.equal(y[at:at + (1 << 28)], x[at:at + (1 << 28)])


# ------------------------------------------------------------------------------ project_rows
def _time(f):
    """Median of five calls, in ms."""
    f()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[2]


@pytest.mark.parametrize("T,N,K,S,R,spread", [(2049, 4096, 4096, 8, 64, True), (4099, 4096, 4096, 8, 64, False), (1500, 3001, 1096, 40, 16, True),
                                              (1031, 4100, 520, 3, 48, False), (2500, 2304, 264, 2, 256, True), (700, 20000, 136, 300, 32, True)])
def test_project_broken_requests_stay_alone_and_cost_little(G, T, N, K, S, R, spread):
    """Prompts with infinities and NaN in one request's adapter or rows: the other rows are what they were, the call takes
    no more than a few times as long, and no wait runs out."""
    from test_gpu_tail import check_project, project_case
    of = None if spread else [(i // 300) % (S + 1) - 1 for i in range(T)]
    s = project_case(T, N, K, S, R, "bf16", T + K, of=of)
    c = int(s["row_adapter"][T // 2].clamp(min=0))
    s["row_adapter"][7] = -1
    mine = s["row_adapter"] == c
    assert mine.any() and (~mine).any()
    y = G.project_rows(**s)
    check_project(s, y)
    sound = _time(lambda: G.project_rows(**s))
    inf, nan = math.inf, math.nan

    def run(**over):
        t = dict(s, **over)
        got = G.project_rows(**t)
        assert _time(lambda: G.project_rows(**t)) < 10 * sound + 0.05
        assert G.tail_errors() == 0
        return got

    def same_but(got, rows, columns):
        """The rows' outputs in these columns are not finite, all others in these columns right, the rest the same bits."""
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[rows.nonzero(), columns] = True
        assert not got[hit].isfinite().any()
        rest = torch.ones(N, dtype=torch.bool, device="cuda")
        rest[columns] = False
        assert torch.equal(got[:, rest], y[:, rest])
        check_project(s, torch.where(hit, y, got))

    b = s["b"].clone()
    b[c, 100, 3] = inf
    same_but(run(b=b), mine, torch.tensor([100], device="cuda"))
    b[c, 101, 0], b[c, N - 1, R - 1], b[c, 0, 5] = nan, -inf, nan
    same_but(run(b=b), mine, torch.tensor([0, 100, 101, N - 1], device="cuda"))
    b[c] = nan
    same_but(run(b=b), mine, torch.arange(N, device="cuda"))
    a = s["a"].clone()
    a[c, 2, K // 2] = nan
    got = run(a=a)
    assert got[mine].isnan().all() and torch.equal(got[~mine], y[~mine])
    x = s["x"].clone()
    x[mine] = nan
    got = run(x=x)
    assert got[mine].isnan().all() and torch.equal(got[~mine], y[~mine])
    # broken rows of one request and a broken adapter of another
    other = (s["row_adapter"] >= 0) & ~mine
    d = int(s["row_adapter"][other][0])
    b = s["b"].clone()
    b[d, 50] = inf
    got = run(x=x, b=b)
    assert got[mine].isnan().all() and not got[s["row_adapter"] == d, 50].isfinite().any()
    keep = ~mine & (s["row_adapter"] != d)
    assert torch.equal(got[keep][:, 51:], y[keep][:, 51:]) and got[keep].isfinite().all()


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("T,N", [(1, 1000), (20, 4000), (64, 300), (100, 30000), (300, 700), (2049, 4096)])
def test_project_inner_rows_keep_their_bits(G, kind, T, N):
    """Adapters whose two halves nearly cancel: what is left of the output shows the rounding of the inner rows, which is
    2^-16 at most (two bfloat16 of 2^-8 each), next to 32-bit sums of K and of R products."""
    from test_gpu_tail import HALF, U, project_case
    K, S, R = 64, 3, 32
    s = project_case(T, N, K, S, R, kind, T + N)
    s["w"].zero_()
    a, b = s["a"], s["b"]
    a[:, R // 2:] = a[:, :R // 2]
    a[:, R // 2:, ::16] *= 1.0625
    b[:, :, R // 2:] = -b[:, :, :R // 2]
    y = G.project_rows(**s).double()
    x = s["x"].double() * (1 if s["x_scale"] is None else s["x_scale"].double()[:, None])
    want, off = torch.zeros_like(y), torch.zeros_like(y)
    for c in range(S):
        rows = (s["row_adapter"] == c).nonzero().flatten()
        ad, bd, g = a[c].double(), b[c].double(), s["adapter_scale"][c].double()
        h, hb = g * (x[rows] @ ad.T), g * (x[rows].abs() @ ad.abs().T)
        want[rows] = h @ bd.T
        off[rows] = (2.0 ** -16 * h.abs() + (K + 4) * U * hb) @ bd.abs().T + (R + 4) * U * (h.abs() @ bd.abs().T)
    assert ((y - want).abs() <= off + (want.abs() + off) * HALF).all()
    assert (want.abs() > 4 * off).double().mean() > 0.5 or T < 5


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("T,S,R", [(4099, 256, 64), (4500, 300, 128), (9001, 128, 64)])
def test_project_rows_in_slabs(G, kind, T, S, R):
    """More rows times adapters than the workspace takes at once: each slab is the call of its own rows."""
    from test_gpu_tail import check_project, project_case
    s = project_case(T, 500, 128, S, R, kind, T)
    wide = torch.full((T, 504 + 8), -7.0, dtype=BF, device="cuda")
    y = G.project_rows(**s, out=wide[:, 4:504])
    check_project(s, y)
    assert (wide[:, :4] == -7).all() and (wide[:, 504:] == -7).all()
    rows = slice(T - 700, T)
    part = dict(s, x=s["x"][rows], row_adapter=s["row_adapter"][rows].contiguous())
    if kind == "f8":
        part["x_scale"] = s["x_scale"][rows].contiguous()
    check_project(part, y[rows])
    assert G.tail_errors() == 0


def test_project_rows_do_not_see_other_rows(G):
    """What a row gives does not depend on what the other rows of the call hold: the same bits with others in their place."""
    from test_gpu_tail import project_case
    for T, kind in ((5, "bf16"), (40, "f8"), (100, "bf16"), (300, "bf16"), (2049, "bf16")):
        s = project_case(T, 1000, 520 if kind == "bf16" else 528, 4, 32, kind, T)
        y = G.project_rows(**s)
        x = s["x"].clone()
        rest = torch.arange(T, device="cuda") % 3 != 1
        x[rest] = s["x"][rest.nonzero().flatten().flip(0)]
        assert torch.equal(G.project_rows(**dict(s, x=x))[~rest], y[~rest])


# ------------------------------------------------------------------------------ beside the sampler
def _projection(V, H=2048, T=8):
    g = torch.Generator(device="cuda").manual_seed(V)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=r(T, H).to(BF), w=r(V, H).mul_(H ** -0.5).to(BF), a=r(2, 16, H).mul_(H ** -0.5).to(BF),
                b=r(2, V, 16).mul_(0.25).to(BF), adapter_scale=torch.ones(2, device="cuda"),
                row_adapter=(torch.arange(T, device="cuda") % 2).int())


@pytest.mark.parametrize("between", ["own outputs", "early load", "own outputs twice"])
def test_sampling_calls_behind_a_projection_see_all_of_it(G, between):
    """A projection lets the next call start at once.  A sampling call of other logits that waits for nothing, or late,
    comes between it and the calls that read its rows."""
    V, T = 131072, 8
    s = _projection(V)
    want = G.project_rows(**s)
    other = torch.randn(T, 4096, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    slot, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    flags = G.STRATA_FLAG_PDL | G.STRATA_FLAG_EARLY_LOAD
    between_flags = flags if between == "early load" else flags | G.STRATA_FLAG_OWN_OUTPUTS
    reading = flags if between == "early load" else G.STRATA_FLAG_PDL
    ones = torch.ones(T, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), G.Sampler(device=0, max_slots=1, max_vocab=V, max_rows=T) as sampler:
        sampler.set_slot(0, dict(temperature=0.0, seed=1))
        stream.synchronize()
        ref = sampler.sample(want, slot, pos, chosen_lp=True, flags=reading)  # the flags choose the split, and so the last bits
        ref_draw = G.draw_rows(want, ones * 0.5)
        y = torch.empty_like(want)
        for i in range(10):
            y.zero_()
            own = [torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2)]
            assert sampler.errors() == 0   # drains the stream: the flag counts again
            G.project_rows(**s, out=y)
            for ids in own[:2 if between == "own outputs twice" else 1]:
                sampler.sample(other, slot, pos, flags=between_flags, out=dict(ids=ids))
            o = sampler.sample(y, slot, pos, chosen_lp=True, flags=reading)
            d = G.draw_rows(y, ones * 0.5)
            assert torch.equal(o["ids"], ref["ids"]) and torch.equal(o["chosen_lp"], ref["chosen_lp"]), i
            assert torch.equal(d["ids"], ref_draw["ids"]) and torch.equal(d["lps"], ref_draw["lps"]), i
        assert sampler.errors() == 0 and G.tail_errors() == 0


def test_operators_in_a_row_after_own_outputs_on_two_streams(G):
    """norm -> project -> draw on two streams, each behind sampling calls that wait for nothing, eager and captured."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, V = 8, 2048, 32000
    s = _projection(V, H)
    h = torch.randn(T, H, generator=g, device="cuda").to(BF)
    weight, u = torch.ones(H, dtype=BF, device="cuda"), torch.rand(T, generator=g, device="cuda")
    other = torch.randn(T, V, generator=g, device="cuda")
    slot, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    flags = G.STRATA_FLAG_PDL | G.STRATA_FLAG_EARLY_LOAD | G.STRATA_FLAG_OWN_OUTPUTS

    def step(x):
        y = G.project_rows(**dict(s, x=G.norm_rows(x, weight)["y"]))
        return y, G.draw_rows(y, u)

    want = step(h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    contexts = [G.Sampler(device=0, max_slots=1, max_vocab=V, max_rows=T) for _ in streams]
    try:
        for c in contexts:
            c.set_slot(0, dict(temperature=0.7, seed=3))
        torch.cuda.synchronize()
        got, own = [], []
        for _ in range(10):
            for stream, c in zip(streams, contexts):
                with torch.cuda.stream(stream):
                    late = torch.zeros_like(h)
                    late.copy_(h)
                    own.append(c.sample(other, slot, pos, flags=flags))
                    got += [step(late), step(late)]
        graph = torch.cuda.CUDAGraph()
        x = torch.zeros_like(h)
        outs = [torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2)]
        with torch.cuda.graph(graph):
            x.copy_(h)
            contexts[0].sample(other, slot, pos, flags=flags, out=dict(ids=outs[0]))
            captured = step(x)
            contexts[0].sample(other, slot, pos, flags=flags, out=dict(ids=outs[1]))
            captured2 = step(x)
        for _ in range(3):
            x.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for y, d in [*got, captured, captured2]:
            assert torch.equal(y, want[0]) and torch.equal(d["ids"], want[1]["ids"]) and torch.equal(d["lps"], want[1]["lps"])
        assert all(c.errors() == 0 for c in contexts) and G.tail_errors() == 0
    finally:
        for c in contexts:
            c.close()


# ------------------------------------------------------------------------------ error bits
@pytest.mark.parametrize("name", ["errors_check", "draw_wait_check"])
def test_errors_are_told(G, tmp_path, name):
    """Programs with the library's source: bits raised on one stream and asked for on another, none is lost; draws whose waits
    run out."""
    import os
    import shutil
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(root, "include"),
                        "-o", exe, os.path.join(root, "tests", name + ".cu")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout[-500:]


# ------------------------------------------------------------------------------ from one to the next
@pytest.mark.parametrize("N", [50257, 32001, 1003, 7, 1])
@pytest.mark.parametrize("T", [1, 2, 40, 300])
def test_projected_rows_go_to_the_draw_and_to_the_sampler(G, N, T):
    """Logits of any vocabulary, as project_rows allocates them, are taken by draw_rows and by the sampler."""
    from test_gpu_tail import check_project, project_case
    s = project_case(T, N, 128, 3, 16, "bf16", N + T)
    y = G.project_rows(**s)
    check_project(s, y)
    wide = torch.full((T, (N + 7) // 8 * 8 + 8), math.nan, dtype=BF, device="cuda")
    wide[:, :N] = y
    wide = wide[:, :N]
    u = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(N), device="cuda")
    keys = dict(temperature=torch.full((T,), 0.8, device="cuda"), top_k=torch.full((T,), 100, dtype=torch.int32, device="cuda"))
    got, want = G.draw_rows(y, u, **keys), G.draw_rows(wide, u, **keys)
    assert torch.equal(got["ids"], want["ids"]) and torch.equal(got["lps"], want["lps"])
    slot, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int64, device="cuda")
    with G.Sampler(device=0, max_slots=1, max_vocab=max(N, 64), max_rows=T) as sampler:
        for rows in (y, wide):
            sampler.set_slot(0, dict(temperature=0.7, top_k=20, top_p=0.95, seed=5), reset_counter=True)
            got = sampler.sample(rows, slot, pos, chosen_lp=True)
            if rows is y:
                first = got
        assert torch.equal(first["ids"], got["ids"]) and torch.equal(first["chosen_lp"], got["chosen_lp"])
        assert ((got["ids"] >= 0) & (got["ids"] < N)).all() and sampler.errors() == 0


def test_the_example_takes_any_vocabulary(G):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_tail.py")
    spec = importlib.util.spec_from_file_location("decode_tail", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    ids, lps = mod.decode(5, 4099, 256, 4)
    again, _ = mod.decode(5, 4099, 256, 4, graph=False)
    assert torch.equal(ids, again) and ((ids >= 0) & (ids < 4099)).all() and (lps <= 0).all()
