"""GPU: experts' products within close bounds (moe_tight.py) for each token, whatever the number of tokens
beside it: the first product's sums are exact to fp32, so that values of v change codes no more often
than fp32 work makes them."""
import pytest
import torch

import moe_ref as ref
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


def _want(c, act="silu"):
    return tight.experts(c.x8, c.xs, c.ids, c.w, c.up, c.down, c.n, act)


# tokens, experts, top_k, hidden, inter: few slots; lists in LDS with the columns from the cache; columns in
# LDS, hidden of 1 to 17 steps of 128 (whole and partial chunks of four), units of one column tile to
# four; few large units and many small ones
SHAPES = [(1, 8, 8, 1152, 640), (7, 9, 7, 128, 3968), (8, 64, 8, 512, 384), (64, 1, 1, 128, 1152), (33, 8, 2, 2048, 1408),
          (100, 64, 2, 640, 768), (100, 64, 2, 768, 896), (90, 48, 2, 896, 1152), (60, 60, 4, 1152, 640), (120, 64, 3, 384, 1408),
          (70, 32, 4, 640, 1408), (100, 16, 4, 1152, 1408), (77, 32, 3, 640, 384), (30, 64, 4, 640, 640), (200, 4, 2, 640, 2176),
          (260, 8, 2, 640, 2176), (140, 2, 1, 896, 3968), (500, 4, 2, 768, 1152), (2100, 4, 1, 128, 2688), (150, 2, 2, 2176, 2944)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_close(shape):
    say("moe_mxfp4 close", shape)
    c = Case(*shape, seed=7 + sum(shape))
    act = "gelu_tanh" if shape[0] % 20 == 0 else "silu"
    tight.check(c.run(act=act), _want(c, act), shape)


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [
    (1, 8, 2, 640, 256), (20, 16, 4, 640, 256), (100, 64, 2, 640, 768), (100, 64, 2, 640, 1408), (300, 4, 2, 640, 1408)])
def test_small_products_beside_large_ones_that_cancel(tokens, experts, top_k, hidden, inter):
    """6 x 448 and -6 x 448 in the same 128 of every sum, the rest products of up to 2^-4: all partial sums are
    exact in 32 bits, and 126 products of the sum's 638 count as the others do."""
    say("moe_mxfp4 cancelling", tokens, experts, top_k, hidden, inter)
    c = Case(tokens, experts, top_k, hidden, inter, seed=5)
    g = torch.Generator().manual_seed(6)

    def positive(w):    # codes 1 to 5: 0.5, 1, 1.5, 2, 3
        low, high = (torch.randint(1, 6, w[0].shape, generator=g, dtype=torch.uint8) for _ in range(2))
        return low | high << 4, torch.full_like(w[1], 127)

    c.up, c.down = positive(c.up), positive(c.down)
    c.up[0][:, 2] = c.up[0][:, 2] & 0x0F | 0x70      # element 5: 6
    c.up[0][:, 35] = c.up[0][:, 35] & 0xF0 | 0x0F    # element 70: -6
    c.e = w4.ExpertsMXFP4.prepare(*(t.cuda() for t in (*c.up, *c.down)), experts=experts)
    c.x8.fill_(0x08)                                 # 2^-6
    c.x8[:, 5] = c.x8[:, 70] = 0x7E                  # 448
    c.xs.copy_(2.0 ** (torch.arange(tokens) % 3 - 1.0))
    tight.check(c.run(), _want(c))
