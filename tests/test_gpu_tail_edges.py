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
