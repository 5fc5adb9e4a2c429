"""GPU: the experts of each token, against plain loops in 64 bits (moe_ref.py): the same ids, and
weights within 2^-18: exponents of differences to 2^5 are off by 2^5 U, their sums by some 30 U."""
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


def _check(logits, top_k, **kw):
    got = w4.moe_route(logits, top_k, **kw)
    want = ref.route(logits, top_k, **kw)
    assert got[0].dtype == torch.float32 and got[1].dtype == torch.int32
    w, ids = (x.cpu() for x in got)
    assert torch.equal(ids, want[1]), (ids[(ids != want[1]).any(1)][:3], want[1][(ids != want[1]).any(1)][:3])
    assert bool(((w.double() - want[0]).abs() <= 2.0 ** -18 * want[0].abs() + 1e-37).all())


SHAPES = [(1, 1, 1), (1, 128, 8), (3, 2, 2), (5, 7, 3), (61, 60, 4), (17, 64, 32), (9, 65, 1), (33, 128, 8), (7, 200, 5),
          (4, 256, 16), (11, 257, 8), (3, 512, 10), (2, 1000, 32), (5, 1024, 8), (1030, 8, 2), (130, 16, 16),
          (1024, 1, 1), (2050, 60, 4), (1500, 16, 16), (1111, 256, 16), (1027, 200, 3), (1026, 32, 17), (1025, 128, 8)]


@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
def test_shapes(tokens, experts, top_k, score, dtype):
    say("moe_route", tokens, experts, top_k, score, dtype)
    g = torch.Generator().manual_seed(tokens + 7 * experts)
    x = (2 * torch.randn((tokens, experts), generator=g)).to(dtype).cuda()   # many ties in 16 bits
    for renormalize in (True, False):
        _check(x, top_k, score=score, renormalize=renormalize, scale=1.0 if renormalize else 2.5)
    _check(x, top_k, score=score, bias=0.3 * torch.randn(experts, generator=g).cuda())


@pytest.mark.parametrize("experts,groups,kept,top,top_k", [
    (64, 8, 4, 2, 8), (64, 8, 1, 1, 8), (256, 8, 4, 2, 8), (128, 64, 10, 2, 8), (60, 4, 2, 1, 6), (64, 64, 5, 2, 8),
    (1024, 16, 3, 2, 32), (16, 2, 2, 2, 16), (24, 8, 3, 2, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(experts, groups, kept, top, top_k, score):
    say("moe_route groups", experts, groups, kept, top, top_k, score)
    g = torch.Generator().manual_seed(experts + kept)
    x = torch.randn((21, experts), generator=g).cuda()
    x[3] = 0                                    # everything ties
    x[5, :experts // 2] = float("-inf")
    x[6, 1:] = float("-inf")
    x[7] = float("-inf")
    kw = dict(score=score, groups=groups, groups_kept=kept, group_top=top)
    _check(x, top_k, **kw)
    _check(x, top_k, bias=0.2 * torch.randn(experts, generator=g).cuda(), **kw)


@pytest.mark.parametrize("tokens,experts", [(16, 8), (16, 100), (16, 300), (1040, 8), (1040, 100)])
def test_masks_ties_and_what_is_no_number(tokens, experts):
    say("moe_route masks", tokens, experts)
    g = torch.Generator().manual_seed(experts)
    x = torch.randn((tokens, experts), generator=g)
    x[0] = float("-inf")
    x[1, 3:] = float("-inf")
    x[2] = float("nan")
    x[3, ::2] = float("nan")
    x[4] = 0.0
    x[5, ::3] = -0.0                            # -0 and 0 are one value
    x[5, 1::3] = 0.0
    x[5, 2::3] = -1.0
    x[6] = 3e38
    x[7] = -3e38
    x[8, 5] = float("inf")
    x[9, 2:4] = float("inf")
    x[10] = torch.finfo(torch.float32).min
    x = x.cuda()
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            _check(x, 6, score=score, renormalize=renormalize)
            bias = 0.1 * torch.randn(experts, generator=g)
            bias[1], bias[4] = float("-inf"), float("nan")
            _check(x, 6, score=score, renormalize=renormalize, bias=bias.cuda())


def test_near_scores_are_told_apart():
    # sigmoids that are equal in 32 bits but not in 64, and sums with a bias that differ in the last bits
    say("moe_route near scores")
    x = torch.tensor([[20.0, 20.5, 19.0, 21.0], [1.0, 1.0 + 2.0 ** -23, 1.0, 1.0 - 2.0 ** -24]]).cuda()
    _check(x, 4, score="sigmoid", bias=torch.tensor([0.25, 0.25, 0.25, 0.25]).cuda())
    _check(x, 4, score="softmax", bias=torch.tensor([0.0, 0.0, 2.0 ** -24, 0.0]).cuda())


def test_strides_outputs_and_rows_behind():
    say("moe_route strides")
    g = torch.Generator().manual_seed(3)
    wide = torch.randn((19, 300), generator=g).to(torch.bfloat16).cuda()
    _check(wide[:, 1:130], 5)
    _check(wide[:1].expand(9, 300), 5)
    w, ids = torch.full((6, 3), 9.0, device="cuda"), torch.full((6, 3), 77, dtype=torch.int32, device="cuda")
    got = w4.moe_route(wide[:5], 3, weights=w[:5], ids=ids[:5])
    assert got[0].data_ptr() == w.data_ptr() and got[1].data_ptr() == ids.data_ptr()
    assert bool((w[5] == 9).all()) and bool((ids[5] == 77).all())
    assert torch.equal(ids[:5].cpu(), ref.route(wide[:5], 3)[1])
    a, b = w4.moe_route(wide[:0], 3)
    assert a.shape == b.shape == (0, 3)
