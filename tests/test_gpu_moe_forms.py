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


# many small experts and few large ones, hidden of five steps
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


@pytest.mark.parametrize("shape", STAGED, ids=lambda s: "x".join(map(str, s)))
def test_tokens_that_are_no_numbers_and_slots_without_experts(shape):
    say("moe_mxfp4 staged, no numbers, no experts", shape)
    tokens, experts, top_k, hidden, inter = shape
    c = Case(*shape, seed=2)
    usual = c.run()
    bad = [0, 7, tokens - 1]
    c.xs[0], c.xs[7] = float("nan"), float("inf")
    c.x8[tokens - 1, hidden - 1] = 0x7F                  # a code that is no number, in the last of five steps
    got = c.run()
    others = [t for t in range(tokens) if t not in bad]
    assert bool(got[bad].isnan().all())
    assert torch.equal(got[others], usual[others])
    # slots without an expert, the bad tokens' among them: their weights are not looked at
    c.ids[::3] = torch.tensor([-1, experts], dtype=torch.int32, device="cuda")
    c.ids[bad] = -1
    c.w[(c.ids < 0) | (c.ids >= experts)] = float("nan")
    got = c.run()
    assert not got[::3].any() and not got[bad].any()
    c.xs[bad], c.x8[bad] = 1.0, 0
    tight.check(got, tight.experts(c.x8, c.xs, c.ids, c.w.nan_to_num(0.0), c.up, c.down, c.n, "silu"))
    c.ids.fill_(-1)
    out = torch.full((tokens + 1, hidden), 5.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out[:tokens])
    assert not out[:tokens].any() and bool((out[tokens] == 5).all())


@pytest.mark.parametrize("shape", STAGED, ids=lambda s: "x".join(map(str, s)))
def test_one_expert_takes_every_slot(shape):
    say("moe_mxfp4 staged, one expert", shape)
    c = Case(*shape, seed=4)
    c.ids.fill_(shape[1] - 1)                            # for every token, top_k times
    tight.check(c.run(), tight.experts(c.x8, c.xs, c.ids, c.w, c.up, c.down, c.n, "silu"))


def test_staged_calls_on_two_streams():
    say("moe_mxfp4 staged, two streams")
    cases = [Case(*STAGED[1], seed=5), Case(*STAGED[2], seed=6)]
    want = [c.run() for c in cases]
    spaces = [w4.MoEWorkspace(s[0], s[2], s[1], s[3], s[4]) for s in STAGED[1:3]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(8):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run(workspace=spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert torch.equal(x, want[i]), i
