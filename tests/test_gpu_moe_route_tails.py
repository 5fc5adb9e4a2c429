"""GPU: sigmoid scores of logits far below zero, where 1 + exp(-logit) leaves 32 bits, against plain
loops in 64 bits (moe_ref.py); weights within 2^-18 as in test_gpu_moe_route.py."""
import pytest
import torch

import moe_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def _logits(tokens, experts, seed):
    """Rows near one level each, from 0 to -735; below -709 the score is 0 in 64 bits too."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, experts), generator=g)
    level = torch.linspace(0, -735, tokens)
    x = x + level[:, None]
    x[1] = -90.0 - torch.arange(experts) % 7
    x[2, 1:] = float("-inf")
    x[3, ::2] += 60.0          # some of a row within 32 bits, others not
    return x


# a wave to a token, and 16 lanes
@pytest.mark.parametrize("tokens,experts,top_k", [(40, 8, 3), (40, 128, 8), (17, 1000, 32), (1040, 16, 16), (1040, 128, 8),
                                                  (1030, 256, 1), (1030, 300, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
def test_sigmoid_of_low_logits(tokens, experts, top_k, dtype):
    say("moe_route low logits", tokens, experts, top_k, dtype)
    x = _logits(tokens, experts, experts).to(dtype).cuda()
    for kw in (dict(renormalize=True), dict(renormalize=True, scale=2.5), dict(renormalize=False)):
        want = ref.route(x, top_k, score="sigmoid", **kw)
        for bias in (None, torch.zeros(experts, device="cuda")):
            w, ids = (t.cpu() for t in w4.moe_route(x, top_k, score="sigmoid", bias=bias, **kw))
            if bias is None:    # a bias of zero goes by the scores, whose ties are others
                assert torch.equal(ids, want[1])
            assert bool(((w.double() - want[0]).abs() <= 2.0 ** -18 * want[0].abs() + 1e-37).all()), (kw, bias is None)


def test_three_logits_by_hand():
    say("moe_route by hand")
    e = torch.exp(-torch.arange(3.0, dtype=torch.float64))
    want = e / e.sum()                               # 0.665, 0.245, 0.090
    for tokens in (1, 1024):
        x = torch.tensor([-92.0, -90.0, -91.0, -200.0]).repeat(tokens, 1).cuda()
        w, ids = w4.moe_route(x, 3, score="sigmoid")
        assert ids.cpu().tolist() == [[1, 2, 0]] * tokens
        assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -18 * want).all())
