"""GPU: sliding windows from a single key to the largest number that the argument holds, beside
sequences of more query tokens than keys."""
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


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d", [(6, 1, 256), (4, 2, 128), (2, 2, 64)])
@pytest.mark.parametrize("lengths", [[(5, 2), (3, 60)], [(63, 60), (5, 2)], [(90, 60), (300, 20), (7, 200)]])
def test_windows_past_the_context_are_none(lengths, hq, hk, d, dtype):
    c = Case(lengths, hq, hk, d, 16, dtype, seed=d)
    say("attention wide windows", (lengths, hq, hk, d, dtype))
    clean = c.check()
    room = c.width * 16
    for window in (2 ** 31 - 1, 2 ** 31 - 40, 2 ** 30, 2 ** 30 + 7, room + 1, room):
        assert torch.equal(c.run(window=window).cpu().double(), clean), window
    assert torch.equal(c.check(window=room - 1), clean)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65])
def test_windows_beside_queries_without_keys(window):
    for hq, hk, d in ((6, 1, 256), (2, 2, 64)):
        say("attention windows", (window, hq, hk, d))
        Case([(5, 2), (3, 130)], hq, hk, d, 16, BF, seed=window).check(window=window)
        Case([(90, 60), (70, 333), (9, 9)], hq, hk, d, 16, BF, seed=window).check(window=window)
