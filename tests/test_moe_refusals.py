"""CPU: what the calls of the expert half of a layer refuse, at the C entry points (before any
device work: the fake pointers are never touched) and in their Python interface."""
import ctypes

import pytest
import torch

import w4a8_gemm_amd as w4
from w4a8_gemm_amd import binding

OK, INVALID, SHAPE, WORKSPACE, ASYM, HIP = range(6)
FAKE = 0x100000

_vp, _i64, _int, _f32, _size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _Experts(ctypes.Structure):
    _fields_ = [("up_w", _vp), ("up_s", _vp), ("down_w", _vp), ("down_s", _vp), ("experts", _int), ("hidden", _i64),
                ("inter", _i64)]


@pytest.fixture(scope="module")
def L():
    """The library with the calls' signatures set, on a handle of its own."""
    lib = ctypes.CDLL(binding.LIB_PATH)
    lib.w4a8_residual_norm.argtypes = [_int, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _f32, _vp, _int, _i64, _vp, _i64,
                                       _vp, _f32, _vp, _vp, _vp, _vp]
    lib.w4a8_moe_route.argtypes = [_int, _vp, _i64, _i64, _int, _int, _int, _vp, _int, _int, _int, _int, _f32, _vp, _vp, _vp]
    lib.w4a8_moe_mxfp4.argtypes = [ctypes.POINTER(_Experts), _vp, _vp, _i64, _vp, _vp, _int, _int, _vp, _vp, _size, _vp]
    lib.w4a8_moe_workspace_bytes.argtypes = [_i64, _int, _i64, _i64]
    lib.w4a8_moe_workspace_bytes.restype = _size
    return lib


def _norm(L, **kw):
    a = dict(type=0, y=FAKE, ldy=64, tokens=3, hidden=64, pw=None, gate=None, gst=0, gsc=0, scale=1.0, res=FAKE, f32=0,
             ldr=64, ro=FAKE, ldro=64, w=None, eps=1e-6, out=FAKE, x8=None, xs=None)
    a.update(kw)
    return L.w4a8_residual_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=-1), INVALID), (dict(y=None), INVALID), (dict(tokens=0), INVALID),
    (dict(hidden=0), INVALID), (dict(ro=None, out=None), INVALID), (dict(x8=FAKE), INVALID), (dict(xs=FAKE), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(gate=FAKE + 1), INVALID), (dict(out=FAKE + 1), INVALID), (dict(res=FAKE + 1), INVALID),
    (dict(res=FAKE + 2, f32=1), INVALID), (dict(ro=FAKE + 2, f32=1), INVALID), (dict(pw=FAKE + 2), INVALID),
    (dict(w=FAKE + 2), INVALID), (dict(x8=FAKE, xs=FAKE + 2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(ldy=-1), INVALID), (dict(ldr=-1), INVALID), (dict(ldro=63), INVALID), (dict(gate=FAKE, gst=-1), INVALID),
    (dict(gate=FAKE, gsc=2), INVALID), (dict(gate=FAKE, gsc=-1), INVALID), (dict(hidden=32769, ldro=40000), SHAPE),
    (dict(tokens=1 << 30), SHAPE), (dict(tokens=1 << 26, hidden=32768, ldro=32768), SHAPE),
    (dict(tokens=1 << 24, hidden=32768, ldro=32768), SHAPE)])
def test_residual_norm_refusals(L, kw, status):
    assert _norm(L, **kw) == status


def _route(L, **kw):
    a = dict(type=2, x=FAKE, ld=64, tokens=3, experts=64, top_k=8, score=0, bias=None, groups=1, kept=1, top=1, renorm=1,
             scale=1.0, ids=FAKE, w=FAKE)
    a.update(kw)
    return L.w4a8_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(score=2), INVALID), (dict(x=None), INVALID),
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(tokens=0), INVALID), (dict(experts=0), INVALID),
    (dict(top_k=0), INVALID), (dict(groups=0), INVALID), (dict(kept=0), INVALID), (dict(ld=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(top=0), INVALID), (dict(top=3), INVALID), (dict(x=FAKE + 2), INVALID),
    (dict(type=0, x=FAKE + 1), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(ids=FAKE + 2), INVALID),
    (dict(w=FAKE + 1), INVALID), (dict(experts=1025), SHAPE), (dict(top_k=33), SHAPE), (dict(experts=4, top_k=5), SHAPE),
    (dict(groups=65, experts=130), SHAPE), (dict(groups=7), SHAPE), (dict(groups=4, kept=5), SHAPE),
    (dict(tokens=1 << 30), SHAPE), (dict(tokens=1 << 26), SHAPE)])
def test_route_refusals(L, kw, status):
    assert _route(L, **kw) == status


def _moe(L, **kw):
    a = dict(up_w=FAKE, up_s=FAKE, down_w=FAKE, down_s=FAKE, experts=8, hidden=256, inter=128, x=FAKE, xs=FAKE, tokens=3,
             ids=FAKE, w=FAKE, top_k=2, act=0, out=FAKE, ws=FAKE, wsn=1 << 40)
    a.update(kw)
    e = _Experts(*list(a.values())[:7])
    return L.w4a8_moe_mxfp4(ctypes.byref(e), *list(a.values())[7:], None)


@pytest.mark.parametrize("kw,status", [
    (dict(up_w=None), INVALID), (dict(up_s=None), INVALID), (dict(down_w=None), INVALID), (dict(down_s=None), INVALID),
    (dict(up_w=FAKE + 8), INVALID), (dict(down_s=FAKE + 4), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(xs=None), INVALID), (dict(xs=FAKE + 2), INVALID), (dict(ids=None), INVALID), (dict(ids=FAKE + 2), INVALID),
    (dict(w=None), INVALID), (dict(w=FAKE + 1), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 4), INVALID),
    (dict(tokens=0), INVALID), (dict(top_k=0), INVALID), (dict(experts=0), INVALID), (dict(hidden=0), INVALID),
    (dict(inter=-128), INVALID), (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(experts=1025), SHAPE),
    (dict(top_k=9), SHAPE), (dict(top_k=33, experts=64), SHAPE), (dict(hidden=192), SHAPE), (dict(inter=64), SHAPE),
    (dict(inter=200), SHAPE), (dict(hidden=65664), SHAPE), (dict(inter=65664), SHAPE), (dict(tokens=1 << 29), SHAPE),
    (dict(tokens=(1 << 25) + 1), SHAPE), (dict(tokens=1 << 25, hidden=65536), SHAPE), (dict(ws=None), WORKSPACE),
    (dict(ws=FAKE + 128), WORKSPACE), (dict(wsn=100), WORKSPACE)])
def test_moe_refusals(L, kw, status):
    assert _moe(L, **kw) == status
    if "ws" not in kw and "wsn" not in kw:
        assert L.w4a8_moe_mxfp4(None, *([FAKE] * 2), 3, FAKE, FAKE, 2, 0, FAKE, FAKE, 1 << 40, None) == INVALID


def test_workspace_bytes(L):
    b = L.w4a8_moe_workspace_bytes
    # one byte a value and an exponent byte for each of 32, in dwords of four steps; fp32 sums of the slots,
    # up to four parts of each while there are no more than 2048 rows; the slots by expert, for each 2017 slots
    plan = 2048 * 6 + 16
    assert b(1, 8, 2048, 768) == 8 * (768 + 32) + 32 * 2048 * 4 + plan
    assert b(5, 2, 256, 512) == 10 * (512 + 16) + 40 * 256 * 4 + plan
    assert b(500, 2, 256, 512) == 1000 * (512 + 16) + 2048 * 256 * 4 + plan
    assert b(3000, 2, 256, 512) == 6000 * (512 + 16) + 6000 * 256 * 4 + 3 * plan
    assert b(0, 2, 256, 512) == b(5, 0, 256, 512) == b(5, 33, 256, 512) == b(5, 2, 256, 64) == b(5, 2, 256, 130) == 0
    assert b(5, 2, 100, 512) == b(5, 2, 0, 512) == b(5, 2, 1 << 17, 512) == b(1 << 29, 2, 256, 128) == 0
    for t in (1, 7, 255, 300, 1023, 1024, 2000):
        assert b(t + 1, 2, 256, 384) > b(t, 2, 256, 384)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,kind,text", [
    (lambda: w4.residual_norm([1.0]), TypeError, "torch tensor"),
    (lambda: w4.residual_norm(_t(2, 8, dtype=torch.float32)), TypeError, "bfloat16 or float16"),
    (lambda: w4.residual_norm(_t(8)), ValueError, r"\[tokens, hidden\]"),
    (lambda: w4.residual_norm(_t(8, 2).T), ValueError, "contiguous rows"),
    (lambda: w4.residual_norm(_t(2, 8), _t(2, 9)), ValueError, "residual must be"),
    (lambda: w4.residual_norm(_t(2, 8), _t(2, 8, dtype=torch.float16)), TypeError, "residual must be of y's type"),
    (lambda: w4.residual_norm(_t(2, 8), weight=_t(8)), TypeError, "weight must be a float32"),
    (lambda: w4.residual_norm(_t(2, 8), weight=_t(7, dtype=torch.float32)), ValueError, "contiguous vector of 8"),
    (lambda: w4.residual_norm(_t(2, 8), post_weight=_t(2, 8, dtype=torch.float32)), ValueError, "post_weight"),
    (lambda: w4.residual_norm(_t(2, 8), gate=_t(3, 8)), ValueError, "gate must be"),
    (lambda: w4.residual_norm(_t(2, 8), gate=_t(8)), ValueError, "gate must be"),
    (lambda: w4.residual_norm(_t(2, 8), gate=_t(8, 2).T), ValueError, "gate must have"),
    (lambda: w4.residual_norm(_t(2, 8), gate=_t(2, 8, dtype=torch.float16)), TypeError, "gate must be"),
    (lambda: w4.residual_norm(_t(2, 8), values=False), ValueError, "nothing to compute"),
    (lambda: w4.residual_norm(_t(2, 8), scale="x"), TypeError, "real number"),
    (lambda: w4.residual_norm(_t(2, 8)), ValueError, "on a GPU"),
    (lambda: w4.moe_route(_t(2, 8, dtype=torch.float64), 2), TypeError, "logits must be"),
    (lambda: w4.moe_route(_t(8, dtype=torch.float32), 2), ValueError, "logits must be"),
    (lambda: w4.moe_route(_t(2, 1025), 2), ValueError, "logits must be"),
    (lambda: w4.moe_route(_t(8, 2).T, 2), ValueError, "contiguous rows"),
    (lambda: w4.moe_route(_t(2, 8), 9), ValueError, "top_k must be from 1 to 8"),
    (lambda: w4.moe_route(_t(2, 64), 33), ValueError, "top_k must be from 1 to 32"),
    (lambda: w4.moe_route(_t(2, 64), 0), ValueError, "top_k"),
    (lambda: w4.moe_route(_t(2, 64), 2.5), TypeError, "integer"),
    (lambda: w4.moe_route(_t(2, 64), 2, score="relu"), ValueError, "score must be one of"),
    (lambda: w4.moe_route(_t(2, 64), 2, bias=_t(64)), TypeError, "bias must be a float32"),
    (lambda: w4.moe_route(_t(2, 64), 2, groups=3), ValueError, "must divide"),
    (lambda: w4.moe_route(_t(2, 64), 2, groups=4, groups_kept=5), ValueError, "groups_kept"),
    (lambda: w4.moe_route(_t(2, 64), 2, group_top=3), ValueError, "group_top"),
    (lambda: w4.moe_route(_t(2, 64), 2), ValueError, "on a GPU")])
def test_python_refusals(call, kind, text):
    with pytest.raises(kind, match=text):
        call()


def _prepared(N, K):
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert binding.lib().w4a8_mxfp4_prepared_bytes(N, K, ctypes.byref(w), ctypes.byref(s)) == OK
    return w4.PreparedMXFP4(_t(w.value, dtype=torch.uint8), _t(s.value, dtype=torch.uint8), N, K)


def test_experts_refusals():
    up, down = _prepared(4 * 2 * 128, 256), _prepared(4 * 256, 128)
    e = w4.ExpertsMXFP4(up, down, 4)
    assert (e.experts, e.hidden, e.inter) == (4, 256, 128)
    with pytest.raises(TypeError, match="PreparedMXFP4"):
        w4.ExpertsMXFP4(up.w, down, 4)
    for n in (0, 3, 8, -4):
        with pytest.raises(ValueError):
            w4.ExpertsMXFP4(up, down, n)
    with pytest.raises(ValueError, match="need up weights"):
        w4.ExpertsMXFP4(down, up, 4)
    short = w4.PreparedMXFP4(up.w[:-1], up.s, up.N, up.K)
    with pytest.raises(ValueError, match="fewer than"):
        w4.ExpertsMXFP4(short, down, 4)
    wrong = w4.PreparedMXFP4(up.w.view(torch.int8), up.s, up.N, up.K)
    with pytest.raises(TypeError, match="uint8"):
        w4.ExpertsMXFP4(wrong, down, 4)


def test_moe_python_refusals():
    e = w4.ExpertsMXFP4(_prepared(4 * 2 * 128, 256), _prepared(4 * 256, 128), 4)
    x, xs = _t(3, 256, dtype=torch.uint8), _t(3, dtype=torch.float32)
    ids, w = _t(3, 2, dtype=torch.int32), _t(3, 2, dtype=torch.float32)
    for args, kind, text in [
            ((x, xs, ids, w, None), TypeError, "ExpertsMXFP4"), ((x[:, :128], xs, ids, w, e), ValueError, "x_fp8"),
            ((x.T.contiguous().T, xs, ids, w, e), ValueError, "x_fp8"), ((x.view(torch.int8), xs, ids, w, e), TypeError, "x_fp8"),
            ((x, xs[:2], ids, w, e), ValueError, "x_scale"), ((x, xs, ids.long(), w, e), TypeError, "ids"),
            ((x, xs, ids[:2], w, e), ValueError, "ids"), ((x, xs, ids, w[:, :1], e), ValueError, "weights"),
            ((x, xs, _t(3, 5, dtype=torch.int32), w, e), ValueError, "ids"), ((x, xs, ids[:, :0], w, e), ValueError, "ids"),
            ((x, xs, ids.T.contiguous().T, w, e), ValueError, "contiguous"), ((x, xs, ids, w.bfloat16(), e), TypeError, "weights"),
            ((x[0], xs, ids, w, e), ValueError, "x_fp8"), ((x, xs, ids, w, e), ValueError, "on a GPU")]:
        with pytest.raises(kind, match=text):
            w4.moe_mxfp4(*args)
    with pytest.raises(ValueError, match="act must be one of"):
        w4.moe_mxfp4(x, xs, ids, w, e, act="relu")
    with pytest.raises(TypeError, match="MoEWorkspace"):
        w4.moe_mxfp4(x, xs, ids, w, e, workspace=x)
    for kw in (dict(tokens=0), dict(top_k=5), dict(hidden=100), dict(inter=100), dict(top_k=33, experts=64),
               dict(tokens=1 << 40)):
        with pytest.raises(ValueError):
            w4.MoEWorkspace(**{**dict(tokens=3, top_k=2, experts=4, hidden=256, inter=128, device="cpu"), **kw})
    assert w4.MoEWorkspace(3, 2, 4, 256, 128, device="cpu").nbytes == w4.moe_workspace_bytes(3, 2, 256, 128)
