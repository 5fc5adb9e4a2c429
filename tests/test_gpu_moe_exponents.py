"""GPU: experts' products on weights at both ends of the exponent bytes, for few and for staged slots."""
import pytest
import torch

import moe_tight as tight
import w4a8_gemm_amd as w4
from gpu_util import say
from test_gpu_moe import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


@pytest.mark.parametrize("which", ["up", "down"])
@pytest.mark.parametrize("byte", [0, 1, 2, 8, 252])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [(2, 8, 2, 256, 256), (20, 16, 4, 640, 256), (100, 64, 2, 640, 1408)])
def test_exponent_bytes(which, byte, tokens, experts, top_k, hidden, inter):
    """2^(byte - 127) beside token scales, or shares of the slots, that bring the result back to about 1."""
    say("moe_mxfp4 exponent byte", which, byte, tokens)
    c = Case(tokens, experts, top_k, hidden, inter, seed=byte + tokens)
    usual = 121                                     # of Case's weights, about
    if which == "up":
        c.up[1][:] = torch.where(c.up[1] >= usual, byte, min(byte + 1, 252)).to(torch.uint8)
        c.xs *= 2.0 ** min(max(usual - byte, -100), 120)
        c.x8 &= 0x8F if byte == 252 else 0xFF       # values below 2^-5: sums stay below 2^128
    else:
        c.down[1][:] = torch.where(c.down[1] >= usual, byte, min(byte + 1, 252)).to(torch.uint8)
        c.w *= 2.0 ** min(max(usual - byte, -100), 120)
        if byte == 252:
            c.xs *= 2.0 ** -8
    c.e = w4.ExpertsMXFP4.prepare(*(t.cuda() for t in (*c.up, *c.down)), experts=experts)
    want = tight.experts(c.x8, c.xs, c.ids, c.w, c.up, c.down, c.n, "silu")
    assert bool(want[0].isfinite().all()) and float(want[0].abs().amax()) > 2.0 ** -20
    tight.check(c.run(), want)
