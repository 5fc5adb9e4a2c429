"""GPU: the measured cases of perf/operators.py at their own sizes, the calls a user makes against
the definition in 64 bits that stands beside them.

Relative (Frobenius) error of an output: half a step of its type for its one rounding, and in
prompts of bf16 queries as much again for the probabilities, which are rounded to bf16 there;
fp32 work stays below 2^-16 of the result.  Cached rows are equal to the last bit."""
import pytest
import torch

import perf.operators as ops
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()
    before, ops.own = ops.own, True
    yield
    ops.own = before


@pytest.mark.parametrize("case", ops.listed(), ids=lambda c: c["name"])
def test_listed_case(case):
    say("operator case", case["name"])
    got = ops.run(ops.prepare(case, 3))
    want = ops.exact(case, 3)
    got, want = (x if isinstance(x, tuple) else (x,) for x in (got, want))
    assert len(got) == len(want)
    for i, (g, e) in enumerate(zip(got, want)):
        g = g.double()
        if case["op"] == "append" and i > 0:
            assert torch.equal(g, e), i
            continue
        half = HALF[ops.DTYPES[case["dtype"]]]
        prompt = case["op"] == "attention" and case["q_len"] > 64 and case["dtype"] == "bf16"
        bound = half * (2 if prompt else 1) + 2.0 ** -16
        assert float((g - e).norm() / e.norm()) <= bound, i
