"""CPU: what the attention block's calls refuse, at the C entry points (before any device
work: the fake pointers are never touched) and in their Python interface."""
import ctypes

import pytest
import torch

import w4a8_gemm_amd as w4
from w4a8_gemm_amd import binding

OK, INVALID, SHAPE, WORKSPACE, ASYM, HIP = range(6)
FAKE = 0x100000


_vp, _i64, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_e8m0", _vp), ("v_codes", _vp), ("v_e8m0", _vp), ("pages", _i64),
                ("kv_heads", _int), ("page", _int), ("head_dim", _int)]


@pytest.fixture(scope="module")
def L():
    """The library with the calls' signatures set, on a handle of its own."""
    lib = ctypes.CDLL(binding.LIB_PATH)
    cache, heads, turn = ctypes.POINTER(_Cache), [_vp, _i64, _i64], [_vp, _i64, _vp, _int, _int]
    lib.w4a8_qk_norm_rope.argtypes = [_int, *heads, _int, *heads, _int, _i64, _int, _vp, _vp, _f32, *turn, _vp, _vp, _vp]
    lib.w4a8_kv_append_mxfp4.argtypes = [cache, _int, *heads, *heads, _i64, _vp, _int, _vp, _f32, *turn, *heads, _int, _vp,
                                         _vp, _vp]
    lib.w4a8_kv_read_mxfp4.argtypes = [cache, _i64, _vp, _vp, _vp, _vp]
    lib.w4a8_attention_mxfp4.argtypes = [cache, _int, *heads, _int, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _f32, _int,
                                         _int, _vp, _vp, ctypes.c_size_t, _vp]
    return lib


def _cache(**kw):
    v = dict(k_codes=FAKE, k_e8m0=FAKE, v_codes=FAKE, v_e8m0=FAKE, pages=4, kv_heads=2, page=16, head_dim=128)
    v.update(kw)
    return ctypes.byref(_Cache(*v.values()))


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


BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _tensors():
    return [_u8(3, 2, 16, 64), _u8(3, 2, 4, 16), _u8(3, 2, 16, 64), _u8(3, 2, 4, 16)]


def test_cache_and_workspace_refusals():
    good = _tensors()
    cache = w4.KVCacheMXFP4(*good)
    assert (cache.pages, cache.kv_heads, cache.page, cache.head_dim) == (3, 2, 16, 128)
    assert cache.k_codes is good[0] and cache.v_e8m0 is good[3]
    for i, t in ((0, _u8(3, 2, 16, 48)), (0, _u8(3, 2, 24, 64)), (1, _u8(3, 2, 16, 4)), (2, _u8(2, 2, 16, 64)),
                 (3, _u8(3, 2, 4, 16, 1)), (0, _u8(3, 2, 64, 16).transpose(2, 3))):
        bad = list(good)
        bad[i] = t
        with pytest.raises(ValueError):
            w4.KVCacheMXFP4(*bad)
    for bad in (good[0].float(), None, "codes"):
        with pytest.raises(TypeError):
            w4.KVCacheMXFP4(bad, *good[1:])
    with pytest.raises(ValueError):
        w4.KVCacheMXFP4.empty(2, 2, 96, device="cpu")
    for args in ((0, 1, 4, 2, 128), (1, 1, 4, 3, 128), (1, 1, 4, 2, 80), (1 << 29, 1, 4, 2, 128)):
        with pytest.raises(ValueError):
            w4.AttentionWorkspace(*args, device="cpu")


# Every other check comes before the one for a GPU, so that all of them show on CPU tensors.
X = torch.zeros(3, 4, 128, dtype=BF)
CS, POS, W = torch.zeros(5, 64), torch.zeros(3, dtype=I64), torch.ones(128)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU", {}), (ValueError, "GPU", dict(q=None)), (ValueError, "GPU", dict(cos_sin=None, positions=None)),
    (TypeError, "float", dict(q=X.float())), (TypeError, "k must", dict(k=X.half())), (TypeError, "tensor", dict(q=None, k=None)),
    (ValueError, "head_dim", dict(q=X[:, :, :96])), (ValueError, "head_dim", dict(q=X[0])),
    (ValueError, "k must", dict(k=X[:2])), (ValueError, "contiguous heads", dict(q=X.repeat(1, 1, 2)[:, :, ::2])),
    (ValueError, "multiple of 16", dict(cos_sin=torch.zeros(5, 24))), (ValueError, "multiple of 16", dict(cos_sin=torch.zeros(5, 144))),
    (ValueError, "cos_sin", dict(cos_sin=CS[:, ::2])), (ValueError, "cos_sin", dict(cos_sin=CS[:0])),
    (TypeError, "cos_sin", dict(cos_sin=CS.double())), (ValueError, "positions", dict(positions=None)),
    (TypeError, "positions", dict(positions=POS.int())), (ValueError, "positions", dict(positions=POS[:2])),
    (ValueError, "q_weight", dict(q_weight=W[:64])), (TypeError, "k_weight", dict(k_weight=W.to(BF))),
    (TypeError, "real number", dict(eps="small"))])
def test_norm_rope_arguments(error, match, kw):
    a = dict(q=X, k=X[:, :2], cos_sin=CS, positions=POS, q_weight=W, k_weight=W)
    a.update(kw)
    with pytest.raises(error, match=match):
        w4.qk_norm_rope(**a)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU", {}), (ValueError, "GPU", dict(q=X, cos_sin=CS, positions=POS)), (TypeError, "cache", dict(cache=None)),
    (TypeError, "cache", dict(cache=_tensors())), (ValueError, "k must", dict(k=X)), (ValueError, "v must", dict(v=X[:2, :2])),
    (TypeError, "v must", dict(v=X[:, :2].half())), (TypeError, "slots", dict(slots=POS.int())),
    (ValueError, "slots", dict(slots=POS[:2])), (ValueError, "mode", dict(mode="mse")), (ValueError, "mode", dict(mode=0)),
    (ValueError, "q must", dict(q=X[:2])), (TypeError, "q must", dict(q=X.float())), (ValueError, "positions", dict(cos_sin=CS))])
def test_append_arguments(error, match, kw):
    a = dict(cache=w4.KVCacheMXFP4(*_tensors()), k=X[:, :2], v=X[:, 2:], slots=POS)
    a.update(kw)
    with pytest.raises(error, match=match):
        w4.kv_append_mxfp4(**a)


def test_read_arguments():
    cache = w4.KVCacheMXFP4(*_tensors())
    for error, args in ((ValueError, (cache, POS)), (TypeError, (_tensors(), POS)), (TypeError, (cache, POS.int())),
                        (ValueError, (cache, POS[None])), (TypeError, (cache, [0, 1]))):
        with pytest.raises(error):
            w4.kv_read_mxfp4(*args)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU", {}), (TypeError, "cache", dict(cache=None)), (TypeError, "q must", dict(q=X.float())),
    (ValueError, "q must", dict(q=X[:, :, :64])), (ValueError, "multiple", dict(q=X[:, :3])),
    (ValueError, "one query token", dict(q=X[:2])), (ValueError, "one query token", dict(max_q=2)),
    (ValueError, "max_q", dict(max_q=0)), (TypeError, "context_lens", dict(context_lens=POS)),
    (ValueError, "context_lens", dict(context_lens=torch.ones(3, 1, dtype=I32))),
    (ValueError, "block_table", dict(block_table=torch.zeros(2, 4, dtype=I32))),
    (ValueError, "block_table", dict(block_table=torch.zeros(4, 3, dtype=I32).T)),
    (ValueError, "block_table", dict(block_table=torch.zeros(3, 0, dtype=I32))),
    (TypeError, "block_table", dict(block_table=torch.zeros(3, 4))), (ValueError, "cu_q", dict(cu_q=torch.zeros(3, dtype=I32))),
    (TypeError, "cu_q", dict(cu_q=torch.zeros(4, dtype=I64))), (ValueError, "window", dict(window=-1)),
    (ValueError, "window", dict(window=4, causal=False)), (TypeError, "real number", dict(scale="1"))])
def test_attention_arguments(error, match, kw):
    a = dict(q=X, cache=w4.KVCacheMXFP4(*_tensors()), block_table=torch.zeros(3, 4, dtype=I32),
             context_lens=torch.ones(3, dtype=I32))
    a.update(kw)
    with pytest.raises(error, match=match):
        w4.attention_mxfp4(**a)
