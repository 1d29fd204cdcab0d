"""Host rules of the operators that score and train the end of a model, checked on the CPU."""
import os
import shutil
import subprocess

import pytest

from test_train_abi import CE_GRAD, DISTILL_GRAD, NORM_GRAD, S, _refused  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _program(tmp_path, name, *flags):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", *flags, "-I", os.path.join(ROOT, "include"),
                        "-o", exe, os.path.join(ROOT, "tests", name + ".cu")], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


@pytest.mark.parametrize("base,name", [(CE_GRAD, "cross_entropy_grad"), (DISTILL_GRAD, "distill_grad"), (NORM_GRAD, "layer_norm_grad")])
def test_an_empty_dx_alone_may_have_no_address(S, base, name):  # noqa: F811
    """PyTorch gives an empty tensor none.  With rows, and no output, the call is refused as before."""
    none = dict.fromkeys(("dx", "dw", "dweight", "dbias", "workspace", "x", "dy"))
    args = dict(base, T=0, **{k: v for k, v in none.items() if k in base})
    assert getattr(S.lib, "strata_" + name)(*args.values()) == S.STRATA_OK
    _refused(S, "strata_" + name, base, {k: None for k in ("dx", "dw", "dweight", "dbias") if k in base}, "STRATA_EINVAL")
    _refused(S, "strata_" + name, base, dict(T=0, H=0), "STRATA_ERANGE")


def test_no_size_of_a_norm_overflows(tmp_path):
    exe = _program(tmp_path, "norm_sizes_check", "-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler", "-fsanitize-undefined-trap-on-error")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout == "0 bad\n", (r.returncode, r.stdout[-2000:])


def test_the_sizes_of_every_loss(tmp_path):
    r = subprocess.run([_program(tmp_path, "loss_sizes_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.endswith(" 0 bad\n"), r.stdout[-2000:]


def test_no_loss_launches_more_blocks_than_sms(tmp_path):
    r = subprocess.run([_program(tmp_path, "loss_units_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.endswith(" 0 bad\n"), r.stdout[-2000:]


def test_the_sizes_of_the_gpu_tests_are_of_all_kinds(tmp_path):
    r = subprocess.run([_program(tmp_path, "loss_kinds_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout == "0 bad\n", r.stdout[-2000:]


def test_no_norm_launches_more_turning_blocks_than_run_at_a_time(tmp_path):
    r = subprocess.run([_program(tmp_path, "norm_blocks_check")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.endswith(" 0 bad\n"), r.stdout[-2000:]
