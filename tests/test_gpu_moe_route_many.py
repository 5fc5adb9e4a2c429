"""GPU: routing of many tokens, on both sides of the sizes from which 16 lanes take a token, against sorted
scores in 64 bits; the tolerance of the weights is that of test_gpu_moe_route.py."""
import pytest
import torch

import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def _want(x, top_k, score, renormalize):
    x = x.cpu().double()
    by, ids = torch.sort(x, dim=1, descending=True, stable=True)      # ties to the lower index
    by, ids = by[:, :top_k], ids[:, :top_k].to(torch.int32)
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.where(by == top, 1.0, torch.exp(by - top)) / torch.where(x == top, 1.0, torch.exp(x - top)).sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-by))
    off = by == float("-inf")
    p, ids = p.masked_fill(off, 0.0), ids.masked_fill(off, -1)
    if renormalize:
        p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    return p, ids


@pytest.mark.parametrize("tokens,experts,top_k", [
    (1, 32, 16), (500, 32, 8), (2047, 60, 6), (2049, 60, 6), (2100, 64, 16), (4095, 128, 8), (4097, 128, 8), (4100, 70, 3),
    (8191, 256, 8), (8195, 256, 8), (8200, 129, 16), (8200, 257, 8), (8200, 256, 17)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
def test_many_tokens(tokens, experts, top_k, dtype):
    say("moe_route many", tokens, experts, top_k, dtype)
    g = torch.Generator().manual_seed(tokens + experts)
    x = (2 * torch.randn((tokens, experts), generator=g)).to(dtype)
    if tokens > 8:
        x[3] = float("-inf")
        x[4, 2:] = float("-inf")
        x[5] = 0.0
        x[6] -= 90.0
        x[7] = x[7] * 0 - 300.0
    x = x.cuda()
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            w, ids = (t.cpu() for t in w4.moe_route(x, top_k, score=score, renormalize=renormalize))
            p, want = _want(x, top_k, score, renormalize)
            p = p.nan_to_num(0.0)          # a row without experts
            assert torch.equal(ids, want), (score, (ids != want).any(1).nonzero()[:4])
            assert bool(((w.double() - p).abs() <= 2.0 ** -18 * p + 1e-37).all()), (score, renormalize)
