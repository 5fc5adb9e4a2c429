"""GPU: both ends of the cache's exponent bytes.  Rows read back are the decoded codes in bf16:
subnormals at byte 0, infinity where e2m1 times 2^126 passes the type; the attention reads the
same numbers at byte 0 and counts value bytes of 253 and more as NaN."""
import pytest
import torch

import attention_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import say
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def test_every_exponent_byte_reads_as_what_it_holds():
    # one exponent a row, all sixteen codes in it
    codes = (torch.arange(32) % 16).to(torch.uint8).expand(256, 2, 32).reshape(256, 64)
    exps = torch.arange(256).to(torch.uint8)
    cache = w4.KVCacheMXFP4.empty(16, 1, 64, 16)
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).view(16, 1, 16, 32).cuda()
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(packed)
    for t in (cache.k_e8m0, cache.v_e8m0):
        t.copy_(exps.view(16, 1, 1, 16).expand(16, 1, 2, 16))
    want = ref.decode(codes, exps[:, None].expand(256, 2)).to(BF)         # 2^128 and more: infinity
    say("read of every exponent")
    for got in w4.kv_read_mxfp4(cache, torch.arange(256).cuda()):
        got = got.cpu()[:, 0]
        assert torch.equal(got.isnan(), want.isnan()) and bool(want[255].isnan().all())
        assert torch.equal(got.nan_to_num(nan=0.0, posinf=None, neginf=None).double()[:253], want.double()[:253])
        assert torch.equal(got[253:255].double(), want[253:255].double()) and bool(want[254].isinf().any())


@pytest.mark.parametrize("mode,byte,back", [("ocp", 252, 1.5 * 2.0 ** 127), ("noclip", 253, float("inf"))])
def test_the_largest_inputs(mode, byte, back):
    x = torch.zeros(3, 1, 64, dtype=BF)
    x[0, 0, 0], x[1, 0, 5], x[2, 0, 33] = 3.3895e38, -3.3895e38, 1.5 * 2.0 ** 127
    cache = w4.KVCacheMXFP4.empty(1, 1, 64, 16)
    slots = torch.arange(3).cuda()
    say("append of the largest", mode)
    w4.kv_append_mxfp4(cache, x.cuda(), x.cuda(), slots, mode=mode)
    assert cache.k_e8m0[0, 0, 0, :2].tolist() == [byte, byte] and cache.v_e8m0[0, 0, 1, 2].item() == 252
    for got in w4.kv_read_mxfp4(cache, slots):
        got = got.cpu().double()
        assert got[0, 0, 0] == back and got[1, 0, 5] == -back and got[2, 0, 33] == 1.5 * 2.0 ** 127


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_over_byte_zero(n, d):
    # values of 2^-127 times e2m1 are subnormal in fp32 and in the bf16 that comes out
    for which in ("ve", "ke"):
        c = Case([(n, n), (n, n + 7)], 2, 1, d, 16, BF, seed=n)
        getattr(c, which)[:] = 0
        say("attention byte zero", (n, d, which))
        got = c.check()
        assert bool((got != 0).any())


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("byte", [252, 253, 254, 255])
def test_attention_at_the_last_bytes(n, byte):
    c = Case([(n, 120)], 2, 1, 128, 16, BF, seed=byte)
    clean = c.run()
    c.ve[c.table[0, 7].long(), :, 2, 7] = byte                              # key 119, the last query's own
    c.vc[c.table[0, 7].long(), :, 7] = 0x22                                 # codes 1
    say("attention last bytes", (n, byte))
    got = c.run()
    assert torch.equal(got[:n - 1], clean[:n - 1])
    assert got[n - 1].isnan().all() if byte > 252 else not got[n - 1].isnan().any()
