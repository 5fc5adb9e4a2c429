"""GPU: head norms with the position rotation, and the paged MXFP4 cache's append and read,
against plain 64-bit forms.  Norm and rotation outputs are within half a rounding step of
their type plus the fp32 sums' share; cached codes and exponents are equal to the last
bit (keys are normed and turned in 64 bits, values come as they are)."""
import pytest
import torch

import attention_ref as ref
import oracle
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def _rows(tokens, heads, d, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, d, generator=g) * 1.5
    if spread:
        x = x * 10.0 ** (2 * torch.rand(tokens, heads, 1, generator=g) - 1)
    return x.to(dtype)


def _weights(d, seed):
    g = torch.Generator().manual_seed(seed)
    return 1 + 0.2 * torch.randn(d, generator=g)


def _check(got, want, mag, dtype, d):
    """Half a step of the type, and the fp32 work: a d-term sum of squares, a root, two products and a sum."""
    tol = ref.HALF[dtype] * want.abs() + (d / 2 + 16) * 2.0 ** -24 * mag
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25                    # fp16's smallest step
    bad = (got.cpu().double() - want).abs() > tol
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,norm", [
    (1, 24, 4, 256, 64, False, True), (7, 6, 1, 256, 256, False, True), (13, 5, 3, 128, 128, True, True),
    (3, 16, 16, 64, 64, False, False), (65, 3, 2, 64, 16, True, True), (2, 2, 1, 128, 96, False, True),
    (5, 1, 1, 128, 48, True, False), (9, 4, 2, 256, 16, False, False)])
def test_norm_rope(dtype, tokens, hq, hk, d, rot, inter, norm):
    say("norm_rope", (dtype, tokens, hq, hk, d, rot, inter, norm))
    qkv = _rows(tokens, hq + 2 * hk, d, dtype, seed=tokens + d)
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hk]        # views: rows of a fused projection
    cs = ref.table(300, rot)
    pos = torch.randint(0, 300, (tokens,), generator=torch.Generator().manual_seed(rot))
    qw, kw = (_weights(d, 1), _weights(d, 2)) if norm else (None, None)
    qo, ko = w4.qk_norm_rope(q, k, cs.cuda(), pos.cuda(), q_weight=None if qw is None else qw.cuda(),
                             k_weight=None if kw is None else kw.cuda(), eps=1e-6, interleaved=inter)
    for got, x, w in ((qo, qkv[:, :hq], qw), (ko, qkv[:, hq:hq + hk], kw)):
        want, mag = ref.norm_rope(x, w, cs, pos, 1e-6, inter)
        _check(got, want, mag, dtype, d)


def test_norm_rope_unaligned_strides_one_side_and_in_place():
    d, tokens = 128, 11
    for off in (1, 3, 8):                         # 2-byte and 16-byte offsets of the heads
        say("norm_rope strides", off)
        buf = _rows(tokens, 5, d + 16, torch.bfloat16, seed=off)
        x = buf.cuda()[:, 1:4, off:off + d]
        w, cs, pos = _weights(d, 3), ref.table(64, 64), torch.arange(tokens) * 5
        qo, ko = w4.qk_norm_rope(x, None, cs.cuda(), pos.cuda(), q_weight=w.cuda())
        assert ko is None
        want, mag = ref.norm_rope(buf[:, 1:4, off:off + d], w, cs, pos, 1e-6, False)
        _check(qo, want, mag, torch.bfloat16, d)
        _, k2 = w4.qk_norm_rope(None, x, cs.cuda(), pos.cuda(), k_weight=w.cuda())
        assert torch.equal(k2, qo)
    y = qo.clone()
    w4.qk_norm_rope(y, None, None, None, q_weight=w.cuda(), q_out=y)
    again, _ = w4.qk_norm_rope(qo, None, q_weight=w.cuda())
    assert torch.equal(y, again)


def test_norm_rope_position_outside_the_table_and_zero_rows():
    say("norm_rope positions")
    x = _rows(4, 2, 64, torch.bfloat16, seed=5)
    x[3] = 0
    pos = torch.tensor([0, -1, 32, 31])
    qo, _ = w4.qk_norm_rope(x.cuda(), None, ref.table(32, 32).cuda(), pos.cuda(), q_weight=_weights(64, 1).cuda())
    out = qo.cpu().float()
    assert out[[1, 2], :, :32].isnan().all() and not out[[1, 2], :, 32:].isnan().any()
    assert not out[0].isnan().any() and (out[3] == 0).all()


def _cache_rows(cache, slots):
    """Codes and exponents of the slots as the kernels wrote them, on the CPU: [n, heads, d], [n, heads, d / 32]."""
    p, r = slots // cache.page, slots % cache.page
    out = []
    for c, e in ((cache.k_codes, cache.k_e8m0), (cache.v_codes, cache.v_e8m0)):
        out.append((ref.unpack(c.cpu()[p, :, r]), e.cpu()[p, :, :, r]))
    return out


@pytest.mark.parametrize("mode", ["ocp", "noclip"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hq,hk,d,page,rot,inter,norm", [
    (1, 24, 4, 256, 64, 64, False, True), (37, 4, 2, 128, 16, 128, True, True), (18, 3, 3, 64, 32, 32, False, False),
    (5, 0, 1, 256, 128, 256, False, True), (21, 2, 2, 64, 16, 0, False, True), (9, 1, 1, 128, 1024, 0, False, False)])
def test_append(mode, dtype, tokens, hq, hk, d, page, rot, inter, norm):
    say("append", (mode, dtype, tokens, hq, hk, d, page, rot, inter, norm))
    x = _rows(tokens, hq + 2 * hk, d, dtype, seed=tokens * d + rot)
    dev = x.cuda()
    pages = tokens // page + 3
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    skipped = torch.zeros(tokens, dtype=torch.bool)
    if tokens > 4:
        skipped[[1, 3]] = True
        slots[1], slots[3] = -1, pages * page      # padding, and one past the cache
    cache = w4.KVCacheMXFP4.empty(pages, hk, d, page)
    kw, qw = (_weights(d, 7), _weights(d, 8)) if norm else (None, None)
    cs, pos = (ref.table(100, rot), torch.randint(0, 100, (tokens,), generator=g)) if rot else (None, None)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo = w4.kv_append_mxfp4(cache, dev[:, hq:hq + hk], dev[:, hq + hk:], slots.cuda(), mode=mode, cos_sin=c(cs),
                            positions=c(pos), k_weight=c(kw), interleaved=inter, q=dev[:, :hq] if hq else None,
                            q_weight=c(qw) if hq else None)
    if hq:
        want, mag = ref.norm_rope(x[:, :hq], qw, cs, pos, 1e-6, inter)
        _check(qo, want, mag, dtype, d)
    else:
        assert qo is None
    key = ref.norm_rope(x[:, hq:hq + hk], kw, cs, pos, 1e-6, inter)[0].float()
    live = slots[~skipped]
    got = _cache_rows(cache, live)
    for (codes, exps), v in zip(got, (key, x[:, hq + hk:].float())):
        wc, we = ref.encode(v[~skipped], mode)
        assert torch.equal(exps, we)
        assert torch.equal(codes, wc)
    # nothing else was written
    total = sum(int((t != 0).sum()) for t in (cache.k_codes, cache.v_codes))
    assert total == sum(int((c.reshape(*c.shape[:-1], -1, 2).sum(-1) != 0).sum()) for c, _ in got)
    # read back: exact, zeros where nothing lies
    k, v = w4.kv_read_mxfp4(cache, slots.cuda())
    for out, (codes, exps) in zip((k, v), got):
        assert torch.equal(out.cpu()[~skipped].double(), ref.decode(codes, exps))
        assert (out.cpu()[skipped] == 0).all()


def test_values_are_encoded_as_weights_are():
    # the library's own weight encoder and the oracle's, on the same bf16 rows
    say("append against the weight encoder")
    x = _rows(40, 3, 128, torch.bfloat16, seed=3)
    for mode in ("ocp", "noclip"):
        cache = w4.KVCacheMXFP4.empty(5, 3, 128, 16)
        slots = torch.arange(40) + 16
        w4.kv_append_mxfp4(cache, x.cuda(), x.cuda(), slots.cuda(), mode=mode)
        (kc, ke), (vc, ve) = _cache_rows(cache, slots)
        rows = x.reshape(120, 128)
        p, e = w4.quant_bf16_to_mxfp4(rows.cuda(), mode=mode)
        op, oe = oracle.quant_bf16_to_mxfp4(rows.view(torch.int16).numpy().view("uint16"), mode=mode)[:2]
        assert (p.cpu().numpy() == op).all() and (e.cpu().numpy() == oe).all()
        for codes, exps in ((kc, ke), (vc, ve)):
            assert torch.equal(codes.reshape(120, 128), ref.unpack(p.cpu()))
            assert torch.equal(exps.reshape(120, 4), e.cpu())


def test_append_extremes_and_non_finite_blocks():
    say("append extremes")
    x = torch.zeros(6, 1, 64, dtype=torch.bfloat16)
    x[0, 0, :32] = 2.0 ** -133                     # below the smallest normal exponent
    x[0, 0, 40] = -(2.0 ** -126)
    x[1, 0, 3] = 3.3895e38                         # the largest bf16
    x[1, 0, 50] = float("inf")
    x[2, 0, 0], x[2, 0, 63] = float("nan"), -1.0
    x[3, 0, 1] = -0.0
    x[4] = torch.linspace(-6, 6, 64).to(torch.bfloat16)
    x[5, 0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])   # ties
    for mode in ("ocp", "noclip"):
        cache = w4.KVCacheMXFP4.empty(1, 1, 64, 16)
        slots = torch.arange(6)
        w4.kv_append_mxfp4(cache, x.cuda(), x.cuda(), slots.cuda(), mode=mode)
        wc, we = ref.encode(x.float(), mode)
        for codes, exps in _cache_rows(cache, slots):
            assert torch.equal(exps, we) and torch.equal(codes, wc)
        k, _ = w4.kv_read_mxfp4(cache, slots.cuda())
        k = k.cpu()
        assert k[1, 0, 32:].isnan().all() and k[2, 0, :32].isnan().all()
        assert not k[1, 0, :32].isnan().any() and not k[2, 0, 32:].isnan().any()


def test_empty_batches():
    say("append nothing")
    cache = w4.KVCacheMXFP4.empty(2, 2, 128, 16)
    z = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    assert w4.kv_append_mxfp4(cache, z, z, s, q=z).shape == z.shape
    k, v = w4.kv_read_mxfp4(cache, s)
    assert k.shape == v.shape == z.shape
    q, k = w4.qk_norm_rope(z, z)
    assert q.shape == k.shape == z.shape
