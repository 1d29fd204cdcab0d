"""Host rules of the operators that score and train the end of a model, checked on the CPU."""
import pytest

from test_train_abi import CE_GRAD, DISTILL_GRAD, NORM_GRAD, S, _refused  # noqa: F401


@pytest.mark.parametrize("base,name", [(CE_GRAD, "cross_entropy_grad"), (DISTILL_GRAD, "distill_grad"), (NORM_GRAD, "layer_norm_grad")])
def test_an_empty_dx_alone_may_have_no_address(S, base, name):  # noqa: F811
    """PyTorch gives an empty tensor none.  With rows, and no output, the call is refused as before."""
    none = dict.fromkeys(("dx", "dw", "dweight", "dbias", "workspace", "x", "dy"))
    args = dict(base, T=0, **{k: v for k, v in none.items() if k in base})
    assert getattr(S.lib, "strata_" + name)(*args.values()) == S.STRATA_OK
    _refused(S, "strata_" + name, base, {k: None for k in ("dx", "dw", "dweight", "dbias") if k in base}, "STRATA_EINVAL")
    _refused(S, "strata_" + name, base, dict(T=0, H=0), "STRATA_ERANGE")
