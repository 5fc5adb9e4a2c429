"""GPU: the calls of the expert half of a layer as they follow each other, on other streams, in
captured graphs, the example, and the measured cases at their own sizes."""
import importlib.util
import os

import pytest
import torch

import moe_ref as ref
import perf.more_operators as ops
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()
    before, ops.own = ops.own, True
    yield
    ops.own = before


HIDDEN, INTER, EXPERTS, TOP_K = 512, 384, 16, 4


class Layer:
    """Norm after attention, router, experts, norm before the next attention."""

    def __init__(self):
        g = torch.Generator().manual_seed(11)
        self.up, self.down = ref.mxfp4_random(EXPERTS * 2 * INTER, HIDDEN, g), ref.mxfp4_random(EXPERTS * HIDDEN, INTER, g)
        self.e = w4.ExpertsMXFP4.prepare(*(t.cuda() for t in (*self.up, *self.down)), experts=EXPERTS)
        self.router = (torch.randn((HIDDEN, EXPERTS), generator=g) / 16).to(torch.bfloat16).cuda()
        self.w = [(1 + torch.randn(HIDDEN, generator=g) / 5).cuda() for _ in range(3)]
        self.ws = w4.MoEWorkspace(64, TOP_K, EXPERTS, HIDDEN, INTER)

    def __call__(self, attn, residual):
        r, h, x8, xs = w4.residual_norm(attn, residual, weight=self.w[0], fp8=True)
        weights, ids = w4.moe_route(h @ self.router, TOP_K)
        y = w4.moe_mxfp4(x8, xs, ids, weights, self.e, workspace=self.ws)
        r2, _, n8, ns = w4.residual_norm(y, r, weight=self.w[1], post_weight=self.w[2], values=False, fp8=True)
        return r, h, x8, xs, weights, ids, y, r2, n8, ns


@pytest.fixture(scope="module")
def layer():
    return Layer()


def _inputs(tokens, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((tokens, HIDDEN), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]


@pytest.mark.parametrize("tokens", [1, 5, 64])
def test_run_together(layer, tokens):
    say("expert layer", tokens)
    attn, residual = _inputs(tokens, tokens)
    r, h, x8, xs, weights, ids, y, r2, n8, ns = layer(attn, residual)
    # each stage from the stage before it, as the GPU left it
    er, eh, off_r, off_h = ref.residual_norm(attn, residual, layer.w[0])
    half = 2.0 ** -8
    assert bool(((r.double().cpu() - er).abs() <= half * (er.abs() + off_r) + off_r).all())
    assert bool(((h.double().cpu() - eh).abs() <= half * (eh.abs() + off_h) + off_h).all())
    want = ref.route(h @ layer.router, TOP_K)
    assert torch.equal(ids.cpu(), want[1])
    out, err = ref.experts(x8, xs, ids, weights, layer.up, layer.down, EXPERTS, "silu")
    assert bool(((y.double().cpu() - out).abs() <= half * (out.abs() + err) + err).all())
    er, eh, off_r, off_h = ref.residual_norm(y, r, layer.w[1], layer.w[2])
    assert bool(((r2.double().cpu() - er).abs() <= half * (er.abs() + off_r) + off_r).all())
    back = ref.e4m3(n8) * ns.double().cpu()[:, None]
    assert bool(((back - eh).abs() <= 2.0 ** -4 * (eh.abs() + off_h) + 2.0 ** -9 * ns.double().cpu()[:, None] + off_h).all())


def test_captured_and_replayed(layer):
    say("expert layer in a graph")
    tokens = 24
    attn, residual = _inputs(tokens, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(attn, residual)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(attn, residual)
    other = w4.MoEWorkspace(64, TOP_K, EXPERTS, HIDDEN, INTER)
    for i in range(4):
        a, b = _inputs(tokens, 20 + i)
        attn.copy_(a)
        residual.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        seen = [x.clone() for x in got]
        kept, layer.ws = layer.ws, other
        want = layer(a, b)
        layer.ws = kept
        torch.cuda.synchronize()
        for n, (x, y) in enumerate(zip(seen, want)):
            assert torch.equal(x, y), (i, n)


def test_two_graphs_share_a_workspace(layer):
    say("two graphs, one workspace")
    sets = [_inputs(t, 40 + t) for t in (3, 40)]
    graphs, outs = [], []
    for a, b in sets:
        layer(a, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(a, b))
        graphs.append(graph)
    want = [[x.clone() for x in layer(a, b)] for a, b in sets]
    for i in (0, 1, 1, 0, 1, 0):
        for x in outs[i]:
            x.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        for n, (x, y) in enumerate(zip(outs[i], want[i])):
            assert torch.equal(x, y), (i, n)


def test_calls_on_two_streams(layer):
    say("two streams")
    sets = [_inputs(t, 60 + t) for t in (40, 7)]
    want = [[x.clone() for x in layer(a, b)] for a, b in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = [Layer() for _ in sets]      # a workspace each: calls that share one must not overlap
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, (a, b) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i] = both[i](a, b)
    torch.cuda.synchronize()
    for i in range(2):
        for x, y in zip(got[i], want[i]):
            assert torch.equal(x, y), i


HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def test_the_layer_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("expert block example")
    # v is rounded to e4m3, at most 2^-4 of each value, errors of either sign over all of inter
    assert example.main() < 2 ** -4
    assert example.main(hidden=384, inter=640, experts=8, top_k=2, prompt=300, batch=40) < 2 ** -4


@pytest.mark.parametrize("case", ops.listed(), ids=lambda c: c["name"])
def test_listed_case(case):
    """Relative (Frobenius) error: half a step of the output's type for its one rounding, fp32 work and, for
    codes against codes, the rare ones on a border's other side below 2^-10 of the whole."""
    say("more operator case", case["name"])
    got, want = ops.run(ops.prepare(case, 3)), ops.exact(case, 3)
    got, want = (x if isinstance(x, (tuple, list)) else (x,) for x in (got, want))
    assert len(got) == len(want)
    for i, (g, e) in enumerate(zip(got, want)):
        if e is None:
            continue
        bound = 2.0 ** -10 if g.dtype == torch.float8_e4m3fn else HALF[g.dtype] + 2.0 ** -16
        assert float((g.double() - e).norm() / e.norm()) <= bound, i
    if case["op"] == "route":
        ops.own = False
        plain = ops.run(ops.prepare(case, 3))
        ops.own = True
        assert torch.equal(got[1], plain[1])
