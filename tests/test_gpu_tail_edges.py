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
