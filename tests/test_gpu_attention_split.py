"""GPU: the attention's cuts of long contexts -- eight-wave runs, joins of one and of two
rounds, key parts of prompts, block tables longer than their LDS copy -- against the plain
64-bit form with the roundings' bounds; and the example that runs the block in a layer."""
import importlib.util
import os

import pytest
import torch

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


def widened(c, keys):
    """The case with a block table for `keys` keys: what chooses between four and eight waves."""
    pad = torch.full((len(c.lengths), max(0, keys // c.page - c.width)), -7, dtype=torch.int32)
    c.table = torch.cat([c.table, pad], 1)
    return c


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 64), (4, 2, 128), (20, 1, 128), (6, 1, 256)])
def test_eight_waves(hq, hk, d, dtype):
    # empty, one key, ends inside and at a tile, fewer tiles than waves, more
    lengths = [(1, c) for c in (0, 1, 63, 64, 65, 511, 513, 3000)]
    say("attention eight waves", (hq, hk, d, dtype))
    for page in (16, 128):
        widened(Case(lengths, hq, hk, d, page, dtype, seed=page), 1 << 18).check()


@pytest.mark.parametrize("wide", [0, 1 << 18])
@pytest.mark.parametrize("lengths", [[(1, 60000)], [(1, 20000), (1, 0), (1, 90)], [(3, 9000), (1, 9000)]])
def test_joins(lengths, wide):
    # 4 and 8 waves; hundreds of pieces (two rounds), tens (one), drafts; repeated calls give the same bits
    for hq, hk, d in ((2, 1, 64), (6, 1, 256)):
        say("attention joins", (lengths, wide, d))
        c = widened(Case(lengths, hq, hk, d, 64, BF, seed=d), wide)
        first = c.check()
        assert torch.equal(c.run().cpu().double(), first)


def test_eight_waves_with_a_window():
    say("attention eight waves, window")
    c = widened(Case([(1, 30000)] + [(1, 100 + i) for i in range(7)], 2, 1, 64, 128, BF, seed=7), 1 << 18)
    c.check(window=25000)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 64), (4, 2, 128), (6, 1, 256)])
@pytest.mark.parametrize("kw", [dict(), dict(window=900), dict(causal=False)])
def test_key_parts_of_prompts(hq, hk, d, dtype, kw):
    # parts of many keys beside sequences that have keys for one part, or none
    lengths = [(100, 5000), (67, 67), (90, 60), (1, 2500), (30, 0)]
    say("attention key parts", (hq, hk, d, dtype, kw))
    Case(lengths, hq, hk, d, 32, dtype, seed=d).check(**kw)


def test_block_table_past_its_copy():
    # row tiles enough that keys are not cut: one workgroup walks 20000 keys in pages of 16 rows
    say("attention long block table")
    Case([(70, 20000)] + [(70, 70)] * 64, 8, 8, 64, 16, BF, seed=3).check()


@pytest.mark.parametrize("hq,hk,d,dtype", [(2, 2, 64, BF), (4, 2, 128, HF), (6, 1, 256, BF), (6, 1, 256, HF)])
@pytest.mark.parametrize("q_len,ctx", [(90, 60), (5, 2), (4, 0)])
def test_queries_without_keys_may_hold_anything(hq, hk, d, dtype, q_len, ctx):
    say("attention queries without keys", (hq, hk, d, dtype, q_len, ctx))
    c = Case([(q_len, ctx), (2, 40)], hq, hk, d, 16, dtype, seed=11)
    clean = c.run()
    none = q_len - ctx
    c.q[:none:2], c.q[1:none:2, :, 3] = float("nan"), float("inf")
    got = c.run()
    assert (got[:none] == 0).all() and torch.equal(got, clean)


def test_the_layer_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    say("attention layer example")
    # probabilities and outputs round to bf16, at most 2^-8 each, errors of either sign over many values
    assert layer.main() < 2 ** -7
    assert layer.main(q_heads=8, kv_heads=2, head_dim=128, rot=128) < 2 ** -7
