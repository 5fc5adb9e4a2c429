"""GPU: experts' products where the columns are staged in LDS, captured and on a workspace that other
calls used; and the activation, told apart from its like."""
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


# many small experts (32 or 16 of inter to a wave) and few large ones, hidden of five steps
STAGED = [(100, 64, 2, 640, 768), (100, 64, 2, 640, 1408), (300, 4, 2, 640, 1408), (1100, 4, 2, 640, 1408)]


@pytest.mark.parametrize("shape", STAGED, ids=lambda s: "x".join(map(str, s)))
def test_captured(shape):
    say("moe_mxfp4 staged, in a graph", shape)
    tokens, experts, top_k, hidden, inter = shape
    c = Case(*shape)
    ws, out = w4.MoEWorkspace(tokens, top_k, experts, hidden, inter), torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    c.run(workspace=ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(workspace=ws, out=out)
    for i in range(4):
        if i == 2:
            c.ids[: tokens // 2] = -1
        else:
            c.ids.copy_(torch.roll(c.ids, 1 + i, 0))
        ws.buf.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run()), i
        torch.cuda.synchronize()
    tight.check(out, tight.experts(c.x8, c.xs, c.ids, c.w, c.up, c.down, c.n, "silu"))


def test_one_workspace_for_all_forms():
    say("moe_mxfp4 staged, one workspace")
    cases = [Case(*s) for s in ((300, 64, 2, 640, 1408), (5, 64, 2, 640, 1408), (100, 64, 2, 640, 1408), (33, 64, 2, 640, 1408),
                                (299, 64, 2, 640, 1408))]
    ws = w4.MoEWorkspace(300, 2, 64, 640, 1408)
    want = [c.run() for c in cases]
    for fill in (0xFF, 0x00):
        ws.buf.fill_(fill)
        for i in (0, 1, 2, 3, 4, 2, 1, 0, 3):
            assert torch.equal(cases[i].run(workspace=ws), want[i]), (fill, i)


@pytest.mark.parametrize("tokens,experts,top_k,inter", [(2, 4, 2, 256), (60, 4, 2, 384), (100, 64, 2, 1408)])
def test_gelu_is_the_tanh_form(tokens, experts, top_k, inter):
    """Gates near -2.6, where the tanh form is 4 % from the error function's."""
    say("moe_mxfp4 gelu", tokens, experts, top_k, inter)
    hidden = 256
    c = Case(tokens, experts, top_k, hidden, inter, seed=3)
    g = torch.Generator().manual_seed(8)
    x = 0.2 * torch.randn((tokens, hidden), generator=g)
    x[:, 0] = 3.5
    c.xs.fill_(3.5 / 448)
    c.x8.copy_((x * 128).to(torch.float8_e4m3fn).view(torch.uint8))
    gates = (torch.arange(experts * 2 * inter) // inter) % 2 == 0
    c.up[0][gates, :16] = 0
    c.up[0][gates, 0] = 0x0D                         # element 0: -3
    c.up[1][gates, 0] = 125                          # 2^-2
    c.e = w4.ExpertsMXFP4.prepare(*(t.cuda() for t in (*c.up, *c.down)), experts=experts)
    args = (c.x8, c.xs, c.ids, c.w, c.up, c.down, c.n)
    want, other = tight.experts(*args, "gelu_tanh"), tight.experts(*args, "gelu_erf")[0]
    _, bound = tight.check(c.run(act="gelu_tanh"), want)
    assert float((other - want[0]).norm() / want[0].norm()) > 2 * bound      # the other form would have failed
