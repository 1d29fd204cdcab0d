"""The ABI of the operators around the sampler (include/strata_tail.h): exports, constants, and every refusal,
which comes before any CUDA call and so needs no GPU.  The addresses below are never read."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "strata_tail.h")


@pytest.fixture(scope="module")
def S():
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "_strata_build", os.path.join(ROOT, "request_token_sampling_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build_library()
    import request_token_sampling_gb300 as S
    return S


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_every_declared_symbol_is_exported(S):
    names = set(re.findall(r"\b(strata_[a-z_]+)\s*\(", _header()))
    assert names == set(S.tail.EXPORTED) and len(names) == 5
    for n in names:
        assert hasattr(S.lib, n) and callable(getattr(S, n))


def test_constants_match(S):
    found = dict(re.findall(r"^#define (STRATA_[A-Z0-9_]+)[ \t]+(\d+)", _header(), flags=re.M))
    assert len(found) == 4
    for name, value in found.items():
        assert getattr(S, name) == int(value)


P = 1 << 20  # an aligned address that nothing reads

NORM = dict(x=P, ldx=64, residual=P, ldr=64, weight=P, dtype=1, T=4, H=64, eps=1e-6, residual_out=P, ldro=64, y=P, ldy=64,
            q=P, ldq=64, scale=P, stream=None)
PROJECT = dict(x=P, ldx=64, x_scale=None, w=P, ldw=64, w_scale=None, dtype=1, T=4, N=8, K=64, a=P, b=P, S=2, R=16,
               row_adapter=P, adapter_scale=P, y=P, ldy=8, workspace=P, workspace_bytes=1 << 30, stream=None)
DRAW = dict(logits=P, dtype=0, B=2, V=8, ld=8, u=P, temperature=P, top_k=P, top_p=P, min_p=P, out_ids=P, out_lps=P,
            stream=None)


def _refused(S, name, base, over, code):
    args = dict(base, **over)
    assert getattr(S.lib, name)(*args.values()) == getattr(S, code), (name, over, S.strata_last_error())
    assert S.strata_last_error()


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), "STRATA_EINVAL"), (dict(T=-1), "STRATA_EINVAL"), (dict(H=0), "STRATA_ERANGE"),
    (dict(H=131073, ldx=1 << 20), "STRATA_ERANGE"), (dict(eps=-1.0), "STRATA_EINVAL"), (dict(eps=float("nan")), "STRATA_EINVAL"),
    (dict(residual_out=None, y=None, q=None, scale=None), "STRATA_EINVAL"), (dict(scale=None), "STRATA_EINVAL"),
    (dict(q=None), "STRATA_EINVAL"), (dict(ldx=63), "STRATA_EINVAL"), (dict(ldr=63), "STRATA_EINVAL"),
    (dict(ldro=63), "STRATA_EINVAL"), (dict(ldy=63), "STRATA_EINVAL"), (dict(ldq=63), "STRATA_EINVAL"),
    (dict(x=None), "STRATA_EINVAL"), (dict(weight=None), "STRATA_EINVAL"), (dict(x=P + 1), "STRATA_EALIGN"),
    (dict(dtype=0, y=P + 2), "STRATA_EALIGN"), (dict(scale=P + 2), "STRATA_EALIGN"),
])
def test_norm_refuses(S, over, code):
    _refused(S, "strata_norm_rows", NORM, over, code)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=0), "STRATA_EINVAL"), (dict(T=-1), "STRATA_EINVAL"), (dict(N=0), "STRATA_EINVAL"), (dict(K=0), "STRATA_ERANGE"),
    (dict(K=131080, ldx=1 << 20, ldw=1 << 20), "STRATA_ERANGE"), (dict(S=-1), "STRATA_ERANGE"), (dict(S=1025), "STRATA_ERANGE"),
    (dict(R=8), "STRATA_ERANGE"), (dict(R=24), "STRATA_ERANGE"), (dict(R=272), "STRATA_ERANGE"), (dict(ldx=56), "STRATA_EINVAL"),
    (dict(ldw=56), "STRATA_EINVAL"), (dict(ldy=7), "STRATA_EINVAL"), (dict(x_scale=P), "STRATA_EINVAL"),
    (dict(dtype=2), "STRATA_EINVAL"), (dict(dtype=2, x_scale=P), "STRATA_EINVAL"), (dict(x=None), "STRATA_EINVAL"),
    (dict(w=None), "STRATA_EINVAL"), (dict(y=None), "STRATA_EINVAL"), (dict(a=None), "STRATA_EINVAL"), (dict(b=None), "STRATA_EINVAL"),
    (dict(row_adapter=None), "STRATA_EINVAL"), (dict(adapter_scale=None), "STRATA_EINVAL"), (dict(x=P + 8), "STRATA_EALIGN"),
    (dict(w=P + 8), "STRATA_EALIGN"), (dict(a=P + 8), "STRATA_EALIGN"), (dict(b=P + 2), "STRATA_EALIGN"),
    (dict(K=60), "STRATA_EALIGN"), (dict(ldx=68), "STRATA_EALIGN"), (dict(ldw=68), "STRATA_EALIGN"), (dict(y=P + 1), "STRATA_EALIGN"),
    (dict(dtype=2, x_scale=P, w_scale=P, K=56), "STRATA_EALIGN"), (dict(workspace=None), "STRATA_EINVAL"),
    (dict(workspace_bytes=1), "STRATA_EINVAL"), (dict(workspace=P + 16), "STRATA_EINVAL"), (dict(row_adapter=P + 2), "STRATA_EALIGN"),
])
def test_project_refuses(S, over, code):
    _refused(S, "strata_project_rows", PROJECT, over, code)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), "STRATA_EINVAL"), (dict(B=-1), "STRATA_EINVAL"), (dict(V=0), "STRATA_ERANGE"),
    (dict(V=524289, ld=1 << 20), "STRATA_ERANGE"), (dict(ld=7), "STRATA_EINVAL"), (dict(logits=None), "STRATA_EINVAL"),
    (dict(u=None), "STRATA_EINVAL"), (dict(out_ids=None), "STRATA_EINVAL"), (dict(logits=P + 4), "STRATA_EALIGN"),
    (dict(ld=9), "STRATA_EALIGN"), (dict(u=P + 2), "STRATA_EALIGN"), (dict(out_lps=P + 1), "STRATA_EALIGN"),
])
def test_draw_refuses(S, over, code):
    _refused(S, "strata_draw_rows", DRAW, over, code)


def test_no_rows_is_no_work(S):
    assert S.lib.strata_norm_rows(*dict(NORM, T=0, x=None).values()) == S.STRATA_OK
    assert S.lib.strata_project_rows(*dict(PROJECT, T=0, x=None, workspace=None).values()) == S.STRATA_OK
    assert S.lib.strata_draw_rows(*dict(DRAW, B=0, logits=None).values()) == S.STRATA_OK
    assert S.lib.strata_tail_errors(None, None) == S.STRATA_EINVAL


def test_workspace_sizes(S):
    assert S.strata_project_workspace(0, 4, 16) == 0 and S.strata_project_workspace(4, 0, 0) == 0
    sizes = [S.strata_project_workspace(t, 8, 32) for t in (1, 2, 64, 129, 4096)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_binding_refuses_host_tensors_and_wrong_types(S):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        S.norm_rows(x, x[0])
    with pytest.raises(TypeError):
        S.norm_rows(x.half(), x[0])
    with pytest.raises(TypeError):
        S.project_rows(x.float(), x)
    with pytest.raises(ValueError):
        S.draw_rows(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(TypeError):
        S.draw_rows(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(2))
