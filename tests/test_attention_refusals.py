"""CPU: what the attention block's calls refuse, at the C entry points (before any device
work: the fake pointers are never touched) and in the binding."""
import ctypes

import pytest
import torch

import w4a8_gemm_amd as w4
from w4a8_gemm_amd import attention as at

OK, INVALID, SHAPE, WORKSPACE, ASYM, HIP = range(6)
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    return at._lib()


def _cache(**kw):
    v = dict(k_codes=FAKE, k_e8m0=FAKE, v_codes=FAKE, v_e8m0=FAKE, pages=4, kv_heads=2, page=16, head_dim=128)
    v.update(kw)
    return ctypes.byref(at._Cache(*v.values()))


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(v_e8m0=None), INVALID), (dict(k_codes=FAKE + 8), INVALID),
              (dict(v_codes=FAKE + 4), INVALID), (dict(k_e8m0=FAKE + 1), INVALID), (dict(pages=0), INVALID),
              (dict(kv_heads=0), INVALID), (dict(kv_heads=1025), INVALID), (dict(page=24), SHAPE), (dict(page=8), SHAPE),
              (dict(page=2048), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=512), SHAPE),
              (dict(pages=1 << 37), SHAPE)]


def _norm(L, **kw):
    a = dict(type=0, q=FAKE, qst=256, qsh=128, hq=2, k=FAKE, kst=256, ksh=128, hk=2, tokens=3, d=128, qw=None, kw=None,
             eps=1e-6, cs=FAKE, rows=10, pos=FAKE, rot=64, inter=0, qo=FAKE, ko=FAKE)
    a.update(kw)
    return L.w4a8_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(q=None), INVALID), (dict(q=None, hq=0, k=None, hk=0), INVALID), (dict(hq=0), INVALID),
    (dict(hk=2000), INVALID), (dict(tokens=0), INVALID), (dict(q=FAKE + 1), INVALID), (dict(qst=-1), INVALID),
    (dict(qo=None), INVALID), (dict(ko=FAKE + 8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(cs=None), INVALID), (dict(pos=None), INVALID), (dict(pos=FAKE + 4), INVALID), (dict(rows=0), INVALID),
    (dict(rot=-16), INVALID), (dict(qw=FAKE + 2), INVALID), (dict(d=96), SHAPE), (dict(rot=24), SHAPE),
    (dict(rot=144), SHAPE), (dict(tokens=1 << 29), SHAPE)])
def test_norm_rope_refusals(L, kw, status):
    assert _norm(L, **kw) == status


def _append(L, cache=None, **kw):
    a = dict(type=0, k=FAKE, kst=256, ksh=128, v=FAKE, vst=256, vsh=128, tokens=3, slots=FAKE, mode=0, kw=None, eps=1e-6,
             cs=None, rows=0, pos=None, rot=0, inter=0, q=None, qst=0, qsh=0, hq=0, qw=None, qo=None)
    a.update(kw)
    return L.w4a8_kv_append_mxfp4(cache or _cache(), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(v=FAKE + 1), INVALID),
    (dict(tokens=0), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(mode=2), INVALID),
    (dict(mode=-1), INVALID), (dict(hq=3), INVALID), (dict(q=FAKE, hq=3), INVALID), (dict(q=FAKE, hq=0, qo=FAKE), INVALID),
    (dict(rot=64), INVALID), (dict(rot=8), SHAPE), (dict(tokens=1 << 28), SHAPE)])
def test_append_refusals(L, kw, status):
    assert _append(L, **kw) == status


def test_caches_refused_everywhere(L):
    for kw, status in BAD_CACHES:
        assert _append(L, cache=_cache(**kw)) == status, kw
        assert L.w4a8_kv_read_mxfp4(_cache(**kw), 1, FAKE, FAKE, FAKE, None) == status, kw
        assert _attention(L, cache=_cache(**kw)) == status, kw
    assert L.w4a8_kv_append_mxfp4(None, 0, *[0] * 22, None) == INVALID
    assert L.w4a8_kv_read_mxfp4(None, 1, FAKE, FAKE, FAKE, None) == INVALID


def test_read_refusals(L):
    f = L.w4a8_kv_read_mxfp4
    assert f(_cache(), 0, FAKE, FAKE, FAKE, None) == INVALID
    assert f(_cache(), 1, None, FAKE, FAKE, None) == INVALID
    assert f(_cache(), 1, FAKE, None, FAKE, None) == INVALID
    assert f(_cache(), 1, FAKE, FAKE, FAKE + 2, None) == INVALID
    assert f(_cache(), 1 << 28, FAKE, FAKE, FAKE, None) == SHAPE


def _attention(L, cache=None, **kw):
    a = dict(type=0, q=FAKE, qst=512, qsh=128, hq=4, tokens=3, seqs=3, cu=None, max_q=1, table=FAKE, tst=8, tw=8, ctx=FAKE,
             scale=0.1, causal=1, window=0, out=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.w4a8_attention_mxfp4(cache or _cache(), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=5), INVALID), (dict(q=None), INVALID), (dict(hq=3), INVALID), (dict(hq=0), INVALID), (dict(tokens=0), INVALID),
    (dict(seqs=0), INVALID), (dict(tokens=4), INVALID), (dict(max_q=2), INVALID), (dict(max_q=0, cu=FAKE), INVALID),
    (dict(cu=FAKE + 2), INVALID), (dict(table=None), INVALID), (dict(table=FAKE + 2), INVALID), (dict(tw=0), INVALID),
    (dict(tst=7), INVALID), (dict(ctx=None), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(window=-1), INVALID), (dict(window=5, causal=0), INVALID),
    (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 64), WORKSPACE),
    (dict(wsb=1024), WORKSPACE), (dict(tokens=1 << 28, seqs=1 << 28), SHAPE), (dict(tw=1 << 26, tst=1 << 26), SHAPE),
    (dict(cu=FAKE, max_q=1 << 28), SHAPE)])
def test_attention_refusals(L, kw, status):
    assert _attention(L, **kw) == status


def test_workspace_bytes(L):
    f = w4.attention_workspace_bytes
    assert f(0, 1, 4, 2, 128) == f(1, 1, 3, 2, 128) == f(1, 1, 4, 2, 96) == f(1, 0, 4, 2, 64) == 0
    # a workspace serves every smaller batch too
    for hq, hk, d in ((4, 2, 128), (24, 4, 256), (16, 2, 64)):
        need = [f(s, n, hq, hk, d) for n in (1, 2, 5, 9, 17, 40, 300, 5000) for s in (1, 3, 64, 300)]
        assert need[0] > 0 and need == sorted(need)


def test_binding_refusals():
    bf = torch.bfloat16
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    good = [u8(3, 2, 16, 64), u8(3, 2, 4, 16), u8(3, 2, 16, 64), u8(3, 2, 4, 16)]
    cache = w4.KVCacheMXFP4(*good)
    assert (cache.pages, cache.kv_heads, cache.page, cache.head_dim) == (3, 2, 16, 128)
    for i, t in ((0, u8(3, 2, 16, 48)), (0, u8(3, 2, 24, 64)), (1, u8(3, 2, 16, 4)), (2, u8(2, 2, 16, 64)),
                 (3, u8(3, 2, 4, 16, 1)), (0, u8(3, 2, 64, 16).transpose(2, 3))):
        bad = list(good)
        bad[i] = t
        with pytest.raises(ValueError):
            w4.KVCacheMXFP4(*bad)
    with pytest.raises(TypeError):
        w4.KVCacheMXFP4(good[0].float(), *good[1:])
    with pytest.raises(ValueError):
        w4.KVCacheMXFP4.empty(2, 2, 96, device="cpu")
    x = torch.zeros(2, 4, 128, dtype=bf)
    with pytest.raises(ValueError, match="GPU"):
        w4.qk_norm_rope(x, x)
    with pytest.raises(TypeError):
        w4.qk_norm_rope(x.float(), None)
    with pytest.raises(ValueError, match="GPU"):
        w4.kv_append_mxfp4(cache, x[:, :2], x[:, :2], torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        w4.kv_read_mxfp4(good, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        w4.attention_mxfp4(x, cache, torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        at._mode("mse")
    for args in ((0, 1, 4, 2, 128), (1, 1, 4, 3, 128), (1, 1, 4, 2, 80)):
        with pytest.raises(ValueError):
            w4.AttentionWorkspace(*args, device="cpu")
    cpu = torch.device("cpu")
    cs = torch.zeros(5, 24)
    with pytest.raises(ValueError, match="multiple of 16"):
        at._turn(cs, None, cpu, 2, 128)
    with pytest.raises(ValueError, match="positions"):
        at._turn(cs[:, :16].contiguous(), None, cpu, 2, 128)
    with pytest.raises(TypeError):
        at._turn(cs.double(), None, cpu, 2, 128)
    with pytest.raises(ValueError):
        at._heads(x[:, :, ::2], "q", bf, cpu, 64)
    with pytest.raises(ValueError):
        at._heads(x, "q", bf, cpu, 128, tokens=3)
    with pytest.raises(ValueError):
        at._weight(torch.zeros(64), "q_weight", cpu, 128)
