"""GPU: softmax attention over the paged MXFP4 cache against a plain 64-bit form, at the
lengths, masks, pages and layouts where it can go wrong.  Each output is held to the
error that its roundings allow (probabilities to bf16, or two bf16 pieces for fp16
queries; the output once; fp32 sums)."""
import pytest
import torch

import attention_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu

P_HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


class Case:
    """A cache of random codes, a block table in random order and queries; lengths: (query tokens, context)."""

    def __init__(self, lengths, hq, hk, d, page, dtype, seed=0, spare=3, q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.hq, self.hk, self.d, self.page, self.dtype = lengths, hq, hk, d, page, dtype
        used = [-(-c // page) for _, c in lengths]
        pages = sum(used) + spare
        codes = torch.randint(0, 256, (2, pages, hk, page, d // 2), generator=g, dtype=torch.uint8)
        exps = torch.randint(124, 128, (2, pages, hk, d // 32, page), generator=g, dtype=torch.uint8)
        self.kc, self.vc, self.ke, self.ve = codes[0], codes[1], exps[0], exps[1]
        names = torch.randperm(pages, generator=g).int()
        self.width = max(1, max(used)) + 1
        self.table = torch.full((len(lengths), self.width), -7, dtype=torch.int32)   # never read past a context
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = names[at:at + u]
            at += u
        self.seqs, t = [], 0
        for n, c in lengths:
            self.seqs.append((t, n, c))
            t += n
        self.tokens = t
        self.q = (torch.randn(t, hq, d, generator=g) * q_scale).to(dtype)
        self.max_q = max(n for n, _ in lengths)
        self.ragged = any(n != 1 for n, _ in lengths)

    def cache(self):
        return w4.KVCacheMXFP4(self.kc.cuda(), self.ke.cuda(), self.vc.cuda(), self.ve.cuda())

    def rows(self, s, codes, exps):
        c = self.seqs[s][2]
        p = self.table[s, :-(-c // self.page)].long()
        x = ref.decode(ref.unpack(codes[p]), exps[p].transpose(2, 3))     # [pages, heads, page, d]
        return x.transpose(1, 2).flatten(0, 1)[:c]

    def run(self, cache=None, **kw):
        cu = torch.tensor([s[0] for s in self.seqs] + [self.tokens], dtype=torch.int32).cuda() if self.ragged else None
        ctx = torch.tensor([s[2] for s in self.seqs], dtype=torch.int32).cuda()
        kw.setdefault("q", self.q.cuda())
        q = kw.pop("q")
        return w4.attention_mxfp4(q, cache or self.cache(), self.table.cuda(), ctx, cu_q=cu, max_q=self.max_q, **kw)

    def want(self, scale=None, causal=True, window=0):
        return ref.attention(self.q, lambda s: self.rows(s, self.kc, self.ke), lambda s: self.rows(s, self.vc, self.ve),
                             self.seqs, self.d ** -0.5 if scale is None else scale, causal, window, self.hq // self.hk,
                             P_HALF[self.dtype])

    def check(self, **kw):
        got = self.run(**kw).cpu().double()
        want, tol = self.want(**kw)
        far = (got - want).abs()
        assert not got.isnan().any()
        assert (far <= tol).all(), (int((far > tol).sum()), float((far - tol).max()))
        return got


HEADS = [(24, 4, 256), (6, 1, 256), (32, 8, 128), (5, 5, 128), (20, 1, 128), (16, 2, 64), (3, 3, 64), (64, 4, 128)]
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_single_tokens(hq, hk, d, dtype):
    for page, lengths in ((16, [(1, 1), (1, 15), (1, 16), (1, 17), (1, 0), (1, 63)]), (64, [(1, 64), (1, 65), (1, 1021)]),
                          (32, [(1, 300)])):
        say("attention tokens", (hq, hk, d, dtype, page, lengths))
        Case(lengths, hq, hk, d, page, dtype, seed=page).check()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("window", [0, 1, 37])
def test_drafts(hq, hk, d, dtype, window):
    lengths = [(3, 3), (1, 100), (5, 131), (2, 1), (4, 0), (5, 257)]      # more queries than keys among them
    say("attention drafts", (hq, hk, d, dtype, window))
    got = Case(lengths, hq, hk, d, 16, dtype, seed=window).check(window=window)
    assert (got[9] == 0).all() and (got[11:15] == 0).all()              # the first of (2, 1); all of (4, 0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("kw", [dict(), dict(window=50), dict(causal=False)])
def test_prompts(hq, hk, d, dtype, kw):
    lengths = [(130, 130), (1, 77), (67, 200), (90, 60), (20, 0)]
    say("attention prompts", (hq, hk, d, dtype, kw))
    Case(lengths, hq, hk, d, 32, dtype, seed=d).check(**kw)


@pytest.mark.parametrize("q_len", [1, 2, 6, 11, 33, 65, 257])
def test_one_sequence_of_every_kernel(q_len):
    # row counts on both sides of the kernels' tiles, one sequence: its keys are split over workgroups
    for hq, hk, d, dtype in ((6, 1, 256, BF), (4, 2, 128, HF), (2, 2, 64, BF)):
        say("attention split", (q_len, hq, hk, d, dtype))
        Case([(q_len, 2000 + q_len)], hq, hk, d, 64, dtype, seed=q_len).check()


def test_many_sequences():
    # more sequences than a wave scans at once, empty entries between
    g = torch.Generator().manual_seed(4)
    for page in (16, 128):
        ctx = torch.randint(0, 400, (150,), generator=g).tolist()
        ctx[::7] = [0] * len(ctx[::7])
        say("attention many sequences", page)
        Case([(1, c) for c in ctx], 4, 2, 64, page, BF, seed=page).check()


def test_no_keys_at_all():
    say("attention no keys")
    got = Case([(1, 0), (1, 0), (1, 0)], 4, 2, 128, 16, BF).run()
    assert (got == 0).all()
    got = Case([(40, 0), (3, 0)], 4, 2, 128, 16, BF).run()
    assert (got == 0).all()


def test_scale_and_large_scores():
    # scores in the hundreds: the running maximum moves often, most probabilities vanish
    for scale in (1.0, -0.3, 0.0):
        say("attention scale", scale)
        Case([(1, 700), (1, 90)], 4, 2, 128, 16, BF, seed=1).check(scale=scale)
        Case([(80, 300)], 4, 2, 128, 16, BF, seed=1).check(scale=scale)


def test_query_magnitudes():
    # rows of mixed magnitude: tiny and huge queries, a zero row
    for dtype, big in ((BF, 2.0 ** 60), (HF, 2.0 ** 9)):
        c = Case([(1, 90), (1, 33)], 4, 2, 128, 16, dtype, seed=2)
        c.q[0, 0] *= 2.0 ** -20 if dtype is HF else 2.0 ** -70
        c.q[0, 1] *= big
        c.q[1, 2] = 0
        c.q[1, 3, ::2] *= 2.0 ** -12
        say("attention magnitudes", dtype)
        scale = 2.0 ** -60 if dtype is BF else None
        c.check(scale=scale)


def test_strides_and_given_output():
    c = Case([(1, 200), (1, 31)], 4, 2, 64, 16, BF, seed=3)
    plain = c.run()
    for off in (0, 1, 8):
        say("attention strides", off)
        wide = torch.zeros(c.tokens, c.hq + 3, c.d + 16, dtype=BF)
        wide[:, 2:2 + c.hq, off:off + c.d] = c.q
        out = torch.full_like(plain, 7.0)
        got = c.run(q=wide.cuda()[:, 2:2 + c.hq, off:off + c.d], out=out)
        assert got is out and torch.equal(got, plain)
    table = torch.full((2, c.width + 5), -1, dtype=torch.int32)
    table[:, 1:1 + c.width] = c.table
    ctx = torch.tensor([200, 31], dtype=torch.int32).cuda()
    got = w4.attention_mxfp4(c.q.cuda(), c.cache(), table.cuda()[:, 1:1 + c.width], ctx)
    assert torch.equal(got, plain)


def test_workspace_is_reused_and_results_repeat():
    c = Case([(1, 3000), (1, 10)], 8, 2, 128, 64, BF, seed=5)
    ws = w4.AttentionWorkspace(4, 1, 8, 2, 128)
    say("attention workspace")
    head = int(w4.lib().w4a8_attention_counter_bytes())
    assert (ws.buf[:head] == 0).all()
    ws.buf[head:].fill_(255)                         # NaN bytes: nothing of it is read before it is written
    cache, first = c.cache(), None
    for _ in range(3):
        got = c.run(cache=cache, workspace=ws)
        assert first is None or torch.equal(got, first)
        first = got
    assert (ws.buf[:head] == 0).all()                # every call leaves its counters at zero
    small = Case([(1, 40)], 8, 2, 128, 64, BF, seed=6)
    got = small.run(workspace=ws).cpu().double()
    want, tol = small.want()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("q_len", [1, 4, 120])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_keys_may_hold_anything(q_len, d):
    # NaN blocks and exponents at the end of the range in rows that no query, or only some, may see
    hq, hk, page = 4, 2, 16
    c = Case([(q_len, 150), (q_len, 37 + q_len)], hq, hk, d, page, BF, seed=q_len)
    clean = c.run(window=20)
    for s, (_, n, ctx) in enumerate(c.seqs):
        pages = c.table[s, :-(-ctx // page)].long()
        for codes, exps in ((c.kc, c.ke), (c.vc, c.ve)):
            # past the context in its last page
            if ctx % page:
                exps[pages[-1], :, :, ctx % page:] = 255
                codes[pages[-1], :, ctx % page:] = 0x77
            # before every query's window
            for i in range(0, max(0, ctx - n + 1 - 20)):
                exps[pages[i // page], :, :, i % page] = (255, 254, 253)[i % 3]
                codes[pages[i // page], :, i % page] = 0x77
    say("attention hidden keys", (q_len, d))
    assert torch.equal(c.run(window=20), clean)
    # pages that lie before every window may have been given away
    for s, (_, n, ctx) in enumerate(c.seqs):
        gone = max(0, ctx - n + 1 - 20) // page
        c.table[s, :gone] = -1
    assert torch.equal(c.run(window=20), clean)


@pytest.mark.parametrize("q_len", [3, 120])
def test_nan_reaches_only_the_queries_that_see_it(q_len):
    for codes_of in ("k", "v"):
        c = Case([(q_len, 200)], 4, 2, 128, 16, BF, seed=9)
        want, tol = c.want()
        at = 200 - q_len + 1                         # the second query's own position: the first does not see it
        exps = c.ke if codes_of == "k" else c.ve
        exps[c.table[0, at // 16].long(), 1, 2, at % 16] = 255
        say("attention nan", (q_len, codes_of))
        got = c.run().cpu().double()
        ok = (got - want).abs() <= tol
        assert ok[:, :2].all() and ok[0].all()       # the other key head's queries; the first query
        assert got[1:, 2:].isnan().all()


@pytest.mark.parametrize("q_len", [1, 70])
def test_non_finite_queries_and_bad_pages(q_len):
    c = Case([(q_len, 100), (q_len, 90)], 4, 2, 64, 16, BF, seed=10)
    clean = c.run()
    want, tol = c.want()
    c.q[0, 1, 5] = float("inf")
    c.q[0, 2, 6] = float("nan")
    say("attention non-finite queries", q_len)
    got = c.run().cpu().double()
    assert got[0, 1:3].isnan().all()
    ok = (got - want).abs() <= tol
    ok[0, 1:3] = True
    assert ok.all()
    c.q = Case([(q_len, 100), (q_len, 90)], 4, 2, 64, 16, BF, seed=10).q
    for bad in (-1, 10 ** 6):                        # an entry outside the cache: NaN, and no read there
        c.table[0, 1] = bad
        got = c.run()
        assert got[:q_len].isnan().all() and torch.equal(got[q_len:], clean[q_len:])


def test_lengths_are_bounded_by_the_tensors():
    # a context past the table, query counts past max_q and past the tokens: clamped, nothing out of bounds
    c = Case([(1, 64), (1, 64)], 4, 2, 64, 16, BF, seed=11)
    table = c.table[:, :4].contiguous().cuda()
    q, cache = c.q.cuda(), c.cache()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    plain = w4.attention_mxfp4(q, cache, table, i32(64, 64))
    say("attention bounds")
    assert torch.equal(w4.attention_mxfp4(q, cache, table, i32(10 ** 9, 64)), plain)
    got = w4.attention_mxfp4(q, cache, table, i32(-5, 64))
    assert (got[0] == 0).all() and torch.equal(got[1], plain[1])
    got = w4.attention_mxfp4(q, cache, table, i32(64, 64), cu_q=i32(0, 1, 50), max_q=1)
    assert torch.equal(got, plain)


def test_on_another_stream_and_in_a_graph():
    c = Case([(1, 500), (1, 77), (1, 0)], 8, 2, 128, 16, BF, seed=12)
    cache, q = c.cache(), c.q.cuda()
    table, ctx = c.table.cuda(), torch.tensor([500, 77, 0], dtype=torch.int32).cuda()
    ws = w4.AttentionWorkspace(3, 1, 8, 2, 128)
    out = torch.empty_like(q)
    say("attention graph")
    eager = w4.attention_mxfp4(q, cache, table, ctx, workspace=ws).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w4.attention_mxfp4(q, cache, table, ctx, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.attention_mxfp4(q, cache, table, ctx, workspace=ws, out=out)
    for step in range(4):                            # lengths and queries change between replays
        n = 500 - 100 * step
        ctx.copy_(torch.tensor([n, 77 - step, step], dtype=torch.int32))
        q.mul_(1.0 + 0.125 * step)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, plain = out.clone(), w4.attention_mxfp4(q, cache, table, ctx)
        # bits: the last sequence has no pages, so its keys read as NaN from the second replay on
        assert torch.equal(got.view(torch.int16), plain.view(torch.int16))
        assert not got[:2].isnan().any() and got[2].isnan().all() == (step > 0)
