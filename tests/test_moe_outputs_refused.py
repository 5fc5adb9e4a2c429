"""CPU: an output that a call would not write is refused, not ignored."""
import pytest
import torch

import w4a8_gemm_amd as w4


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,text", [
    (dict(values=False, fp8=True, out=_t(2, 8)), "out needs values=True"),
    (dict(values=False, residual=_t(2, 8), out=_t(2, 8)), "out needs values=True"),
    (dict(x_fp8=_t(2, 8, dtype=torch.uint8)), "x_fp8 and x_scale need fp8=True"),
    (dict(x_scale=_t(2, dtype=torch.float32)), "x_fp8 and x_scale need fp8=True"),
    (dict(residual=_t(2, 8), values=False, x_fp8=_t(2, 8, dtype=torch.uint8), x_scale=_t(2, dtype=torch.float32)), "need fp8=True")])
def test_residual_norm(kw, text):
    with pytest.raises(ValueError, match=text):
        w4.residual_norm(_t(2, 8), **kw)


def test_one_of_the_fp8_outputs_may_be_given():
    # past the checks of what is asked for, to the one of the device
    for kw in (dict(x_fp8=_t(2, 8, dtype=torch.uint8)), dict(x_scale=_t(2, dtype=torch.float32)), dict(out=_t(2, 8))):
        with pytest.raises(ValueError, match="on a GPU"):
            w4.residual_norm(_t(2, 8), fp8=True, **kw)
