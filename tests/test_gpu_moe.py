"""GPU: experts' products on MXFP4 weights against the definition in 64 bits (moe_ref.py, where the
tolerance is derived): bf16's half step, fp32 sums, and for a value next to the border of two
codes the other code."""
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


class Case:
    def __init__(self, tokens, experts, top_k, hidden, inter, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.n = experts
        self.up = ref.mxfp4_random(experts * 2 * inter, hidden, g)
        self.down = ref.mxfp4_random(experts * hidden, inter, g)
        x = torch.randn((tokens, hidden), generator=g) * (0.2 + torch.rand((tokens, 1), generator=g) * 2)
        self.xs = (x.abs().amax(1) / 448).cuda()
        self.x8 = (x / self.xs.cpu()[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        order = torch.rand((tokens, experts), generator=g).argsort(1)
        self.ids = order[:, :top_k].to(torch.int32).contiguous().cuda()
        self.w = torch.softmax(torch.randn((tokens, top_k), generator=g), 1).cuda()
        self.e = w4.ExpertsMXFP4.prepare(*(t.cuda() for t in (*self.up, *self.down)), experts=experts)

    def run(self, **kw):
        return w4.moe_mxfp4(self.x8, self.xs, self.ids, self.w, self.e, **kw)

    def want(self, act="silu"):
        return ref.experts(self.x8, self.xs, self.ids, self.w, self.up, self.down, self.n, act)


def _check(got, want, rows=None, name=""):
    out, err = want
    got = got.double().cpu()
    if rows is not None:
        got, out, err = got[rows], out[rows], err[rows]
    bad = ~((got - out).abs() <= 2.0 ** -8 * (out.abs() + err) + err)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4], out[bad][:4], err[bad][:4])


SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (1, 8, 8, 1152, 640), (3, 5, 3, 384, 128), (17, 4, 4, 128, 640),
          (64, 2, 2, 256, 256), (130, 2, 1, 128, 256), (200, 16, 8, 256, 128), (1030, 4, 2, 128, 128), (7, 300, 5, 128, 128),
          (2, 1024, 32, 128, 128), (5, 64, 6, 512, 896), (33, 8, 2, 2048, 1408), (64, 1, 1, 128, 1152), (300, 3, 3, 256, 128),
          (40, 1, 1, 640, 256), (2049, 3, 1, 128, 128), (15, 16, 1, 256, 256), (16, 60, 4, 256, 2048), (4, 40, 2, 4096, 128),
          (70, 1, 1, 128, 8192), (300, 1, 1, 256, 4096), (513, 2, 2, 128, 2048), (140, 3, 1, 1152, 1152), (260, 8, 2, 640, 2176),
          (90, 30, 4, 384, 1152), (150, 1, 1, 5120, 128),
          # many experts with few slots each; few slots and a long inter; the widest
          (40, 1024, 8, 128, 128), (200, 1024, 8, 128, 128), (1, 8, 8, 128, 2816), (7, 9, 7, 128, 3968), (64, 8, 1, 128, 2944),
          (8, 4, 2, 128, 8192), (3, 2, 2, 65536, 128), (3, 2, 1, 128, 65536), (70, 2, 1, 65536, 128), (70, 2, 1, 128, 65536)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape):
    say("moe_mxfp4", shape)
    c = Case(*shape, seed=sum(shape))
    act = "gelu_tanh" if shape[0] % 2 == 0 else "silu"
    _check(c.run(act=act), c.want(act))


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 8, 4), (6, 8, 4), (90, 6, 3), (700, 6, 3)])
def test_ids_outside_the_same_expert_twice_and_no_expert(tokens, experts, top_k):
    say("moe_mxfp4 ids", tokens)
    c = Case(tokens, experts, top_k, 256, 256, seed=tokens)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
    for v in (-1, experts, 2 ** 31 - 1, -2 ** 31):
        ids[torch.rand((tokens, top_k), generator=g) < 0.1] = v
    ids[tokens // 2] = 3
    if tokens > 2:
        ids[2] = -1
    c.ids = ids.cuda()
    c.w[(c.ids < 0) | (c.ids >= experts)] = float("nan")      # a left-out slot's weight is not looked at
    want = ref.experts(c.x8, c.xs, c.ids, c.w.nan_to_num(0.0), c.up, c.down, experts, "silu")
    got = c.run()
    _check(got, want)
    if tokens > 2:
        assert not got[2].any()
    c.ids.fill_(-1)
    assert not c.run().any()


def test_one_expert_takes_everything():
    # the grid is laid out for evenly spread slots
    for tokens, experts, top_k in ((100, 64, 4), (512, 32, 4)):
        say("moe_mxfp4 one expert", tokens)
        c = Case(tokens, experts, top_k, 128, 128, seed=9)
        c.ids.fill_(experts - 1)
        _check(c.run(), c.want())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_no_number_stays_alone(bad):
    say("moe_mxfp4 non-finite token", bad)
    c = Case(9, 4, 2, 256, 256)
    c.xs[4] = bad
    got = c.run()
    assert bool(got[4].isnan().all())
    c.xs[4] = 1.0
    want = c.want()
    _check(got, want, rows=[i for i in range(9) if i != 4])


def test_zero_and_tiny_activations():
    say("moe_mxfp4 zero and tiny")
    c = Case(6, 4, 2, 256, 256)
    c.x8[1] = 0
    c.xs[2] *= 2.0 ** -60
    c.xs[3] *= 2.0 ** 20
    got = c.run()
    assert not got[1].any()
    _check(got, c.want(), rows=[0, 1, 3, 4, 5])
    # v near 2^-120: fp32 and the blocks' powers reach it, bf16 holds it
    out, err = c.want()
    assert bool(((got[2].double().cpu() - out[2]).abs() <= 2.0 ** -7 * out[2].abs().max()).all())


def test_outputs_workspaces_and_rows_behind():
    say("moe_mxfp4 workspaces")
    ws = w4.MoEWorkspace(tokens=300, top_k=4, experts=8, hidden=256, inter=384)
    for tokens, top_k in ((300, 4), (1, 2), (37, 4), (300, 1)):
        c = Case(tokens, 8, top_k, 256, 384, seed=tokens)
        ws.buf.fill_(0xFF)
        out = torch.full((tokens + 1, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        got = c.run(workspace=ws, out=out[:tokens])
        assert got.data_ptr() == out.data_ptr() and bool((out[tokens] == 5).all())
        _check(got, c.want())
        assert torch.equal(got, c.run())       # the same bits with a workspace of its own
    small = w4.MoEWorkspace(tokens=2, top_k=1, experts=8, hidden=256, inter=384)
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=small)
    assert w4.moe_mxfp4(c.x8[:0], c.xs[:0], c.ids[:0], c.w[:0], c.e).shape == (0, 256)


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [
    (70, 1, 1, 128, 8192), (65, 2, 1, 256, 16384), (300, 2, 1, 128, 8192), (64, 4, 1, 128, 128), (2, 33, 32, 128, 128),
    (1000, 4, 3, 128, 512), (9, 8, 8, 384, 1152), (3, 8, 8, 128, 2816), (8, 4, 2, 128, 8192)])
def test_nothing_is_written_past_the_workspace(tokens, experts, top_k, hidden, inter):
    say("moe_mxfp4 end of the workspace", tokens, experts, top_k, hidden, inter)
    c = Case(tokens, experts, top_k, hidden, inter)
    ws = w4.MoEWorkspace(tokens, top_k, experts, hidden, inter)
    guard = 4 << 20
    whole = torch.full((ws.nbytes + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    ws.buf = whole[:ws.nbytes]
    got = c.run(workspace=ws)
    assert bool((whole[ws.nbytes:] == 0xA5).all())
    _check(got, c.want())


def test_captured_with_many_slots_to_an_expert():
    say("moe_mxfp4 in a graph, many slots")
    c = Case(200, 4, 2, 256, 384)
    ws, out = w4.MoEWorkspace(200, 2, 4, 256, 384), torch.empty((200, 256), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(workspace=ws, out=out)
    for i in range(3):
        c.ids.copy_(torch.roll(c.ids, 1 + i, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run()), i
        torch.cuda.synchronize()
    _check(out, c.want())


def test_weights_past_4_gib():
    say("moe_mxfp4 weights past 4 GiB")
    experts, hidden, inter = 1024, 8192, 1024
    g = torch.Generator(device="cuda").manual_seed(2)

    def weight(rows, cols):
        return (torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.randint(118, 121, (rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8))

    up, down = weight(experts * 2 * inter, hidden), weight(experts * hidden, inter)
    e = w4.ExpertsMXFP4.prepare(*up, *down, experts=experts)
    c = Case(3, 2, 2, hidden, 128)
    met = torch.tensor([0, 511, 1023, 1022], dtype=torch.int32)
    ids = torch.tensor([[0, 3], [1, 2], [2, 3]])
    got = w4.moe_mxfp4(c.x8, c.xs, met[ids].cuda(), c.w, e)

    def rows(w, n):
        return tuple(torch.cat([t[int(i) * n:(int(i) + 1) * n].cpu() for i in met]) for t in w)

    want = ref.experts(c.x8, c.xs, ids.to(torch.int32), c.w, rows(up, 2 * inter), rows(down, hidden), 4, "silu")
    _check(got, want)
