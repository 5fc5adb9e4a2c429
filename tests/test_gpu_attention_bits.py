"""GPU: the bits that the attention keeps of its probabilities, and values over the whole range
of a block's exponent, against the plain 64-bit form.

p.v takes two bf16 pieces of a probability (relative 2^-16); with bf16 queries and a prompt's
rows it takes one, 2^-8.  Few keys and outputs that cancel show a probability of fewer bits:
the output's own rounding is relative to the output, a probability's to the values."""
import pytest
import torch

import attention_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import say
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def many_rows(c):
    """Whether the case's rows per key head are a prompt's."""
    return c.max_q * (c.hq // c.hk) > (32 if c.d == 256 else 64)


def held(c, **kw):
    want, tol = ref.attention(c.q, lambda s: c.rows(s, c.kc, c.ke), lambda s: c.rows(s, c.vc, c.ve), c.seqs, c.d ** -0.5,
                              kw.get("causal", True), kw.get("window", 0), c.hq // c.hk,
                              2.0 ** -8 if many_rows(c) and c.dtype is BF else 2.0 ** -16)
    got = c.run(**kw).cpu().double()
    far = (got - want).abs()
    assert not got.isnan().any()
    assert (far <= tol).all(), (int((far > tol).sum()), float((far / tol).max()))


SHAPES = [(6, 1, 256), (8, 2, 128), (3, 3, 64)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", SHAPES)
@pytest.mark.parametrize("lengths", [[(1, c) for c in (2, 3, 5, 9, 40, 700)], [(3, 3), (2, 9), (5, 6)],
                                     [(1, 9000)], [(90, 90), (70, 75), (5, 300)]])
def test_probabilities_keep_their_bits(lengths, hq, hk, d, dtype):
    say("attention bits", (lengths, hq, hk, d, dtype))
    held(Case(lengths, hq, hk, d, 16, dtype, seed=d + len(lengths)))


@pytest.mark.parametrize("kw", [dict(window=7), dict(causal=False)])
@pytest.mark.parametrize("hq,hk,d", SHAPES)
def test_probabilities_keep_their_bits_under_masks(hq, hk, d, kw):
    for lengths in ([(4, 30), (2, 5)], [(100, 120), (70, 20), (9, 9)]):
        say("attention bits, masks", (lengths, hq, hk, d, kw))
        held(Case(lengths, hq, hk, d, 32, BF, seed=d), **kw)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", SHAPES)
@pytest.mark.parametrize("lengths", [[(1, 90), (3, 40)], [(100, 100), (70, 300)], [(70, 4000)]])
def test_values_over_the_range_of_the_exponent(lengths, hq, hk, d, dtype):
    # fp16 queries' outputs are fp16: exponents that keep them inside its range
    low, high = (30, 240) if dtype is BF else (114, 138)
    for seed in range(3):
        c = Case(lengths, hq, hk, d, 16, dtype, seed=seed)
        g = torch.Generator().manual_seed(seed)
        if seed == 0:                               # a block of dims far below the others
            c.ve[:, :, 1] = low
        elif seed == 1:                             # any exponent in any block
            c.ve = torch.randint(low, high + 1, c.ve.shape, generator=g, dtype=torch.uint8)
        else:                                       # the last key's values alone, at the far end
            for t0, n, ctx in c.seqs:
                s = [x[0] for x in c.seqs].index(t0)
                c.ve[c.table[s, (ctx - 1) // 16].long(), :, 0, (ctx - 1) % 16] = high
        say("attention value exponents", (lengths, hq, hk, d, dtype, seed))
        held(c)


@pytest.mark.parametrize("at", [0, 15, 40, 88, 89])
@pytest.mark.parametrize("hq,hk,d", SHAPES)
def test_a_huge_value_reaches_only_the_queries_that_see_it(hq, hk, d, at):
    c = Case([(90, 90)], hq, hk, d, 16, BF, seed=at)
    c.ve[c.table[0, at // 16].long(), :, -1, at % 16] = 240
    say("attention huge value", (hq, hk, d, at))
    held(c)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_exponents_change_no_bit(d):
    # past the context in its last page, and before the window, any exponent may lie
    c = Case([(90, 150), (70, 77)], 4, 2, d, 32, BF, seed=d)
    clean = c.run(window=20)
    for s, (_, n, ctx) in enumerate(c.seqs):
        pages = c.table[s, :-(-ctx // 32)].long()
        for i in list(range(0, max(0, ctx - n + 1 - 20))) + list(range(ctx, len(pages) * 32)):
            c.ve[pages[i // 32], :, :, i % 32] = (1, 60, 200, 252, 255)[i % 5]
    say("attention hidden exponents", d)
    assert torch.equal(c.run(window=20), clean)
