"""The ABI of the operators that score and train the end of a model (include/strata_train.h): exports, constants, and every
refusal, which comes before any CUDA call and so needs no GPU.  The addresses below are never read."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "strata_train.h")


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
    assert names == set(S.train.EXPORTED) and len(names) == 8
    for n in names:
        assert hasattr(S.lib, n) and callable(getattr(S, n))
    for n in ("layer_norm_rows", "layer_norm_grad", "cross_entropy_rows", "cross_entropy_grad", "distill_rows", "distill_grad"):
        assert callable(getattr(S, n)) and n in S.train.__all__


def test_constants_match(S):
    found = dict(re.findall(r"^#define (STRATA_[A-Z0-9_]+)[ \t]+(\d+)", _header(), flags=re.M))
    assert len(found) == 3
    for name, value in found.items():
        assert getattr(S, name) == int(value)


P = 1 << 20  # an aligned address that nothing reads
BIG = 1 << 50

NORM = dict(x=P, ldx=64, residual=P, ldr=64, weight=P, bias=P, dtype=1, T=4, H=64, eps=1e-6, residual_out=P, ldro=64, y=P, ldy=64,
            mean=P, rstd=P, stream=None)
NORM_GRAD = dict(dy=P, lddy=64, x=P, ldx=64, weight=P, mean=P, rstd=P, dresidual=P, lddr=64, dtype=1, T=4, H=64, dx=P, lddx=64, dweight=P,
                 dbias=P, workspace=P, workspace_bytes=BIG, stream=None)
ROWS = dict(x=P, ldx=64, w=P, ldw=64, T=4, V=100, H=64)
CE = dict(ROWS, ids=P, loss=P, lse=P, workspace=P, workspace_bytes=BIG, stream=None)
CE_GRAD = dict(ROWS, ids=P, lse=P, g=P, dx=P, lddx=64, dw=P, lddw=64, workspace=P, workspace_bytes=BIG, stream=None)
DISTILL = dict(ROWS, K=20, ids=P, teacher=P, temperature=1.0, loss=P, lse=P, workspace=P, workspace_bytes=BIG, stream=None)
DISTILL_GRAD = dict(ROWS, K=20, ids=P, teacher=P, temperature=1.0, lse=P, g=P, dx=P, lddx=64, dw=P, lddw=64, workspace=P, workspace_bytes=BIG,
                    stream=None)


def _refused(S, name, base, over, code):
    args = dict(base, **over)
    assert set(args) == set(base)
    assert getattr(S.lib, name)(*args.values()) == getattr(S, code), (name, over, S.strata_last_error())
    assert S.strata_last_error()


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), "STRATA_EINVAL"), (dict(T=-1), "STRATA_EINVAL"), (dict(H=0), "STRATA_ERANGE"),
    (dict(H=131073, ldx=1 << 20), "STRATA_ERANGE"), (dict(eps=-1.0), "STRATA_EINVAL"), (dict(eps=float("nan")), "STRATA_EINVAL"),
    (dict(residual_out=None, y=None, mean=None, rstd=None), "STRATA_EINVAL"), (dict(ldx=63), "STRATA_EINVAL"), (dict(ldr=63), "STRATA_EINVAL"),
    (dict(ldro=63), "STRATA_EINVAL"), (dict(ldy=63), "STRATA_EINVAL"), (dict(x=None), "STRATA_EINVAL"), (dict(weight=None), "STRATA_EINVAL"),
    (dict(x=P + 1), "STRATA_EALIGN"), (dict(bias=P + 1), "STRATA_EALIGN"), (dict(dtype=0, y=P + 2), "STRATA_EALIGN"),
    (dict(mean=P + 2), "STRATA_EALIGN"), (dict(rstd=P + 1), "STRATA_EALIGN"),
])
def test_layer_norm_refuses(S, over, code):
    _refused(S, "strata_layer_norm_rows", NORM, over, code)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), "STRATA_EINVAL"), (dict(T=-1), "STRATA_EINVAL"), (dict(H=0), "STRATA_ERANGE"),
    (dict(H=131073, ldx=1 << 20), "STRATA_ERANGE"), (dict(dx=None, dweight=None, dbias=None), "STRATA_EINVAL"), (dict(lddy=63), "STRATA_EINVAL"),
    (dict(ldx=63), "STRATA_EINVAL"), (dict(lddr=63), "STRATA_EINVAL"), (dict(lddx=63), "STRATA_EINVAL"), (dict(dy=None), "STRATA_EINVAL"),
    (dict(x=None), "STRATA_EINVAL"), (dict(weight=None), "STRATA_EINVAL"), (dict(mean=None), "STRATA_EINVAL"), (dict(rstd=None), "STRATA_EINVAL"),
    (dict(dy=P + 1), "STRATA_EALIGN"), (dict(dx=P + 1), "STRATA_EALIGN"), (dict(dweight=P + 1), "STRATA_EALIGN"), (dict(dbias=P + 1), "STRATA_EALIGN"),
    (dict(mean=P + 2), "STRATA_EALIGN"), (dict(workspace=None), "STRATA_EINVAL"), (dict(workspace=P + 16), "STRATA_EINVAL"),
    (dict(workspace_bytes=1), "STRATA_EINVAL"), (dict(dx=None, dbias=None, workspace=None), "STRATA_EINVAL"),
])
def test_layer_norm_grad_refuses(S, over, code):
    _refused(S, "strata_layer_norm_grad", NORM_GRAD, over, code)


BOTH = [
    (dict(T=-1), "STRATA_EINVAL"), (dict(V=0), "STRATA_EINVAL"), (dict(T=131073), "STRATA_ERANGE"), (dict(V=524289), "STRATA_ERANGE"),
    (dict(H=0), "STRATA_ERANGE"), (dict(H=32776, ldx=1 << 20, ldw=1 << 20), "STRATA_ERANGE"), (dict(H=60), "STRATA_EALIGN"),
    (dict(ldx=56), "STRATA_EINVAL"), (dict(ldw=56), "STRATA_EINVAL"), (dict(ldx=68), "STRATA_EALIGN"), (dict(ldw=68), "STRATA_EALIGN"),
    (dict(x=None), "STRATA_EINVAL"), (dict(w=None), "STRATA_EINVAL"), (dict(ids=None), "STRATA_EINVAL"), (dict(lse=None), "STRATA_EINVAL"),
    (dict(x=P + 8), "STRATA_EALIGN"), (dict(w=P + 8), "STRATA_EALIGN"), (dict(ids=P + 2), "STRATA_EALIGN"), (dict(lse=P + 2), "STRATA_EALIGN"),
    (dict(workspace=None), "STRATA_EINVAL"), (dict(workspace=P + 128), "STRATA_EINVAL"), (dict(workspace_bytes=1), "STRATA_EINVAL"),
]
FORWARD = [(dict(loss=None), "STRATA_EINVAL"), (dict(loss=P + 2), "STRATA_EALIGN")]
BACKWARD = [
    (dict(dx=None, dw=None), "STRATA_EINVAL"), (dict(g=None), "STRATA_EINVAL"), (dict(g=P + 1), "STRATA_EALIGN"), (dict(dx=P + 8), "STRATA_EALIGN"),
    (dict(dw=P + 8), "STRATA_EALIGN"), (dict(lddx=56), "STRATA_EINVAL"), (dict(lddw=56), "STRATA_EINVAL"), (dict(lddx=68), "STRATA_EALIGN"),
    (dict(lddw=68), "STRATA_EALIGN"),
]
TEACHER = [
    (dict(K=0), "STRATA_ERANGE"), (dict(K=-1), "STRATA_ERANGE"), (dict(K=129), "STRATA_ERANGE"), (dict(teacher=None), "STRATA_EINVAL"),
    (dict(teacher=P + 2), "STRATA_EALIGN"), (dict(temperature=0.0), "STRATA_EINVAL"), (dict(temperature=-1.0), "STRATA_EINVAL"),
    (dict(temperature=float("nan")), "STRATA_EINVAL"), (dict(temperature=float("inf")), "STRATA_EINVAL"), (dict(temperature=1e-35), "STRATA_EINVAL"),
    (dict(temperature=0.0009), "STRATA_EINVAL"), (dict(temperature=1001.0), "STRATA_EINVAL"),
]


@pytest.mark.parametrize("over,code", BOTH + FORWARD)
def test_cross_entropy_refuses(S, over, code):
    _refused(S, "strata_cross_entropy_rows", CE, over, code)


@pytest.mark.parametrize("over,code", BOTH + BACKWARD)
def test_cross_entropy_grad_refuses(S, over, code):
    _refused(S, "strata_cross_entropy_grad", CE_GRAD, over, code)


@pytest.mark.parametrize("over,code", BOTH + FORWARD + TEACHER)
def test_distill_refuses(S, over, code):
    _refused(S, "strata_distill_rows", DISTILL, over, code)


@pytest.mark.parametrize("over,code", BOTH + BACKWARD + TEACHER)
def test_distill_grad_refuses(S, over, code):
    _refused(S, "strata_distill_grad", DISTILL_GRAD, over, code)


def test_no_rows_is_no_work(S):
    none = dict(T=0, x=None)
    assert S.lib.strata_layer_norm_rows(*dict(NORM, **none).values()) == S.STRATA_OK
    assert S.lib.strata_layer_norm_grad(*dict(NORM_GRAD, dy=None, dweight=None, dbias=None, workspace=None, **none).values()) == S.STRATA_OK
    assert S.lib.strata_cross_entropy_rows(*dict(CE, workspace=None, **none).values()) == S.STRATA_OK
    assert S.lib.strata_cross_entropy_grad(*dict(CE_GRAD, dw=None, workspace=None, **none).values()) == S.STRATA_OK
    assert S.lib.strata_distill_rows(*dict(DISTILL, workspace=None, **none).values()) == S.STRATA_OK
    assert S.lib.strata_distill_grad(*dict(DISTILL_GRAD, dw=None, workspace=None, **none).values()) == S.STRATA_OK


def test_workspace_sizes(S):
    assert S.strata_loss_workspace(0, 100, 64) == 0 and S.strata_layer_norm_workspace(0, 64) == 0
    for K in (0, 20):
        for grad in (False, True):
            sizes = [S.strata_loss_workspace(t, 32000, 64, K, grad) for t in (1, 64, 128, 129, 4096, 131072)]
            assert all(0 < a for a in sizes)
            # copies of the rows, at most 512 MB of a piece (or 512 ids) and 256 MB of parts (or one), and the rows' own words
            for t, n in zip((1, 64, 128, 129, 4096, 131072), sizes):
                pad = (t + 255) // 256 * 256
                assert n <= pad * 64 * 2 * 2 + max(600 << 20, pad * 1024) + max(256 << 20, pad * 64 * 4) + 16 * t * (K + 2) + (8192 * 2048 * 8) + 65536
    for over in ((2 ** 31 - 1, 100, 64, 0), (131073, 100, 64, 0), (4, 524289, 64, 0), (4, 100, 32776, 0), (4, 100, 64, 129), (4, 100, 64, -1)):
        assert S.strata_loss_workspace(*over, False) == 0 and S.strata_loss_workspace(*over, True) == 0
    big = S.strata_loss_workspace(131072, 524288, 32768, 128, True)
    assert 0 < big < 64 << 30
    assert 0 < S.strata_layer_norm_workspace(2 ** 31 - 1, 131072) <= 16 * 2 * 131072 * 4


def test_the_workspace_that_is_asked_for_is_enough(S):
    """One byte less than the size is refused, whatever the sizes."""
    for T, V, H, K in ((1, 7, 8, 0), (128, 300, 64, 5), (129, 300, 64, 0), (5000, 70001, 520, 20)):
        for grad, base, name in ((False, CE, "cross_entropy_rows"), (True, CE_GRAD, "cross_entropy_grad")):
            if K:
                base, name = (DISTILL_GRAD, "distill_grad") if grad else (DISTILL, "distill_rows")
            need = S.strata_loss_workspace(T, V, H, K, grad)
            over = dict(T=T, V=V, H=H, ldx=H, ldw=H, workspace_bytes=need - 1, **(dict(K=K) if K else {}))
            if grad:
                over.update(lddx=H, lddw=H)
            _refused(S, "strata_" + name, base, over, "STRATA_EINVAL")


def test_binding_refuses_host_tensors_and_wrong_types(S):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    s = torch.zeros(2)
    with pytest.raises(ValueError):
        S.layer_norm_rows(x, x[0])
    with pytest.raises(TypeError):
        S.layer_norm_rows(x.half(), x[0])
    with pytest.raises(ValueError):
        S.layer_norm_grad(x, x, x[0], s, s)
    with pytest.raises(ValueError):
        S.cross_entropy_rows(x, x, ids)
    with pytest.raises(TypeError):
        S.cross_entropy_rows(x.float(), x, ids)
    with pytest.raises(TypeError):
        S.cross_entropy_grad(x.float(), x, ids, s, s)
    with pytest.raises(TypeError):
        S.distill_rows(x, x, ids, None)
    with pytest.raises(ValueError):
        S.distill_rows(x, x, ids, s)


def test_the_calls_need_the_built_binding():
    code = """
import request_token_sampling_gb300 as S
S.tail.MODULE_PATH = "/nowhere/_strata_tail.so"
for call in (lambda: S.layer_norm_rows(1, 2), lambda: S.cross_entropy_rows(1, 2, 3), lambda: S.distill_grad(1, 2, 3, 4, 5, 6)):
    try:
        call()
    except ImportError as e:
        assert "not built" in str(e)
    else:
        raise SystemExit("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
