"""Host rules of the operators around the sampler, checked on the CPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _program(tmp_path, name):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", "-I", os.path.join(ROOT, "include"),
                        "-o", exe, os.path.join(ROOT, "tests", name + ".cu")], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def test_overlapped_launches_keep_the_order_of_a_stream(tmp_path):
    r = subprocess.run([_program(tmp_path, "chain_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:]
    assert r.stdout.startswith("0 bad")


def _build_module():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_strata_build", os.path.join(ROOT, "request_token_sampling_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_sampler_needs_neither_pytorch_nor_the_operators_binding():
    """The package imports without PyTorch; only a call of an operator asks for it, or for a binding that loads."""
    _build_module().build_library()
    code = """
import sys
sys.modules["torch"] = None
import request_token_sampling_gb300 as S
assert S.lib.strata_sample_rows and S.lib.strata_norm_rows and S.strata_project_workspace(4, 2, 16) > 0
assert "_strata_tail" not in sys.modules
for call in (S.norm_rows, S.project_rows, S.draw_rows):
    try:
        call(1, 2)
    except ImportError:
        continue
    raise SystemExit("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    code = """
import request_token_sampling_gb300 as S
S.tail.MODULE_PATH = "/nowhere/_strata_tail.so"
try:
    S.draw_rows(1, 2)
except ImportError as e:
    assert "not built" in str(e)
else:
    raise SystemExit("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_library_builds_without_pytorch(monkeypatch, tmp_path):
    """Its commands are nvcc's alone; with PyTorch the binding's come beside them."""
    import importlib.util
    for installed in (False, True):
        mod = _build_module()
        monkeypatch.setattr(mod, "LIB_DIR", str(tmp_path))
        for name in ("LIB_PATH", "MODULE_PATH"):
            monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
        ran = []

        class Ran:
            returncode, stdout, stderr = 0, "", ""

            def __init__(self, args, **kw):
                self.args = args
                ran.append(args)
                out = args[args.index("-o") + 1]
                assert os.path.dirname(out) == str(tmp_path)
                open(out, "w").close()

            def communicate(self):
                return "", ""

        monkeypatch.setattr(mod.subprocess, "Popen", Ran)
        monkeypatch.setattr(mod.subprocess, "run", Ran)
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" and not installed else find(n, *a))
        if installed:
            pytest.importorskip("torch")
        assert mod.build_library(force=True) == mod.LIB_PATH and mod.up_to_date()
        assert os.path.exists(mod.MODULE_PATH) == installed
        assert any("g++" in a[0] for a in ran) == installed
        monkeypatch.undo()


def test_a_failed_device_setup_is_tried_again(tmp_path):
    r = subprocess.run([_program(tmp_path, "setup_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.endswith("0 bad\n"), r.stdout[-2000:]


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 256])
def test_project_refuses_more_outputs_than_it_counts(N):
    """Before any CUDA call: the outputs of the last tile count in 31 bits."""
    _build_module().build_library()
    import request_token_sampling_gb300 as S
    P = 1 << 20
    args = [P, 64, None, P, 64, None, S.STRATA_DTYPE_BF16, 4, N, 64, None, None, 0, 0, None, None, P, N, None, 0, None]
    assert S.lib.strata_project_rows(*args) == S.STRATA_ERANGE
    assert S.strata_project_workspace(2 ** 31 - 1, 1, 16) > 0


def test_the_workspace_has_a_limit():
    """Rows times adapters of the largest calls go through it in slabs: 256 MB and the lists, or 2,048 rows' if that is more.  A
    single row takes no more than its own adapter's."""
    _build_module().build_library()
    import request_token_sampling_gb300 as S
    for T in (129, 4099, 16384, 524288):
        for n in (1, 64, 256, 1024):
            for R in (16, 64, 256):
                row = min(n, 256) * R * 4
                lists = 20 * T + 4096
                assert S.strata_project_workspace(T, n, R) <= min(T * row, max(256 << 20, 2048 * row)) + 256 * row + lists
    for n in (1, 64, 1024):
        assert S.strata_project_workspace(1, n, 64) <= 16 * 64 * 4 + 1024
