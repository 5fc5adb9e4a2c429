"""GPU: norms around a block with gate, scale and residual sum, and the per-token fp8 codes of the
result, against the formulas in 64 bits (moe_ref.py, where the tolerances are derived)."""
import pytest
import torch

import moe_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import say

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need an MI355X")
    w4.lib()


def _normal(gen, *shape, dtype=FP32):
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def _near(got, want, off, name):
    """got was rounded once to its type from a value within `off` of `want`."""
    got, half = got.double().cpu(), ref.HALF[got.dtype]
    tiny = 2.0 ** -25 if half == 2.0 ** -11 else 0.0   # half the step under fp16's smallest normal
    bad = (got - want).abs() > half * (want.abs() + off) + off + tiny
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4], want[bad][:4])


def _check(got, want, name=""):
    r, h, x8, xs = got
    er, eh, off_r, off_h = want
    if r is not None:
        _near(r, er, off_r, name + " residual")
    if h is not None:
        _near(h, eh, off_h, name + " values")
    if x8 is not None:
        most = eh.abs().amax(1)
        s = xs.double().cpu()
        want_s = torch.where(most > 0, most, 448.0) / 448
        slack = off_h.amax(1) / 448 + 4 * ref.U * want_s
        assert bool(((s - want_s).abs() <= slack).all()), name + " scale"
        code = ref.e4m3(x8)
        assert bool(code.isfinite().all())
        # half a step of e4m3: 2^-4 of the value, 2^-10 under its normal values; h / s within off / s and 4 U
        y = eh / s[:, None]
        off = off_h / s[:, None] + 4 * ref.U * y.abs()
        assert bool(((code - y).abs() <= 2.0 ** -4 * (y.abs() + off) + 2.0 ** -10 + off).all()), name + " codes"
        q, step = ref.nearest_e4m3(y.clamp(-448, 448))
        mid = ((y / step - 0.5).round() + 0.5) * step
        clear = (y - mid).abs() > off + 1e-300   # no border of two codes within the error: the code itself
        assert torch.equal(code[clear], q[clear]), name + " codes"
        assert float(clear.double().mean()) > 0.99


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 1000), (64, 513), (600, 256), (1, 32768), (70, 5120), (513, 2051), (4, 12345),
          (65, 64), (130, 520), (1, 5120), (700, 4096), (515, 8200)]


@pytest.mark.parametrize("tokens,hidden", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_all_at_once(tokens, hidden, dtype):
    say("residual_norm", tokens, hidden, dtype)
    g = torch.Generator().manual_seed(tokens * 40000 + hidden)
    y, res = _normal(g, tokens, hidden, dtype=dtype), _normal(g, tokens, hidden, dtype=dtype) * 2
    w, pw, gate = 1 + _normal(g, hidden) / 5, 1 + _normal(g, hidden) / 5, _normal(g, tokens, hidden, dtype=dtype)
    kw = dict(weight=w, post_weight=pw, gate=gate, scale=0.3)
    _check(w4.residual_norm(y, res, fp8=True, **kw), ref.residual_norm(y, res, **kw))


@pytest.mark.parametrize("residual", [None, "same", "fp32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "full", "token", "channel", "one", "expanded"])
@pytest.mark.parametrize("hidden", [384, 1027])
def test_options(residual, post, gate, hidden):
    say("residual_norm options", residual, post, gate, hidden)
    tokens = 37
    g = torch.Generator().manual_seed(hidden)
    y = _normal(g, tokens, hidden, dtype=BF16)
    res = None if residual is None else _normal(g, tokens, hidden, dtype=BF16 if residual == "same" else FP32)
    shape = {"full": (tokens, hidden), "token": (tokens, 1), "channel": (1, hidden), "one": (1, 1), "expanded": (tokens, 1)}
    gt = None if gate is None else _normal(g, *shape[gate], dtype=BF16)
    if gate == "expanded":
        gt = gt.expand(tokens, hidden)
    kw = dict(post_weight=1 + _normal(g, hidden) / 4 if post else None, gate=gt)
    want = ref.residual_norm(y, res, **kw)
    for values, fp8 in ((True, False), (False, True), (True, True)):
        got = w4.residual_norm(y, res, values=values, fp8=fp8, **kw)
        assert [x is not None for x in got] == [residual is not None, values, fp8, fp8]
        _check(got, want, f"values={values} fp8={fp8}")
    if residual:
        got = w4.residual_norm(y, res, values=False, **kw)
        assert got[1:] == (None, None, None)
        _check(got, want, "residual alone")
    store = torch.empty((tokens, hidden), dtype=BF16 if res is None else res.dtype, device="cuda")
    got = w4.residual_norm(y, res, residual_out=store, **kw)
    assert got[0].data_ptr() == store.data_ptr()
    _check(got, want, "given residual_out")


@pytest.mark.parametrize("res_type", [BF16, FP32], ids=["bf16", "fp32"])
def test_strides_places_and_rows_behind(res_type):
    say("residual_norm strides")
    g = torch.Generator().manual_seed(5)
    tokens, hidden = 33, 333
    wide = _normal(g, tokens, 3 * hidden, dtype=BF16)
    y, gate = wide[:, hidden:2 * hidden], wide[:, 1:hidden + 1]
    res = _normal(g, tokens + 2, hidden + 5, dtype=res_type)
    want = ref.residual_norm(y, res[:tokens, :hidden], gate=gate)
    keep = res.clone()
    out, x8 = torch.full((tokens + 1, hidden), 7.0, dtype=BF16, device="cuda"), torch.full((tokens + 1, hidden), 9, dtype=torch.uint8, device="cuda")
    xs = torch.full((tokens + 1,), 5.0, device="cuda")
    view = res[:tokens, :hidden]
    got = w4.residual_norm(y, view, gate=gate, fp8=True, residual_out=view, out=out[:tokens], x_fp8=x8[:tokens], x_scale=xs[:tokens])
    _check(got, want, "in place")
    assert torch.equal(res[tokens:], keep[tokens:]) and torch.equal(res[:, hidden:], keep[:, hidden:])
    assert bool((out[tokens] == 7).all()) and bool((x8[tokens] == 9).all()) and float(xs[tokens]) == 5
    # a row that all tokens share
    one = _normal(g, 1, hidden, dtype=BF16)
    _check(w4.residual_norm(one.expand(tokens, hidden), keep[:tokens, :hidden]),
           ref.residual_norm(one.expand(tokens, hidden), keep[:tokens, :hidden]), "shared row")
    y2 = y.contiguous()
    want = ref.residual_norm(y2)
    got = w4.residual_norm(y2, out=y2)
    assert got[1].data_ptr() == y2.data_ptr()
    _check(got, want, "out is y")


def test_extremes():
    say("residual_norm extremes")
    hidden = 640
    g = torch.Generator().manual_seed(6)
    y = _normal(g, 8, hidden, dtype=BF16)
    y[1] = 0
    y[2] = float("nan")
    y[3, 17] = float("inf")
    y[4] *= 1e-18
    y[5] *= 2.0 ** 50
    y[6, 3:] = 0
    w = torch.ones(hidden, device="cuda")
    w[5] = 0
    r, h, x8, xs = w4.residual_norm(y, weight=w, fp8=True)
    good = [0, 1, 4, 5, 6, 7]
    want = [x[good] for x in ref.residual_norm(y, weight=w)]
    _check((None, h[good], x8[good], xs[good]), want)
    assert float(xs[1]) == 1.0 and not h[1].any() and not (x8[1] & 0x7F).any()
    assert bool(h[2].isnan().all()) and bool(xs[2:4].isnan().all()) and bool(h[3, 17].isnan())
    # rows that are scaled as if their largest were 2^-110
    _, h, x8, xs = w4.residual_norm(torch.ones((1, hidden), dtype=BF16, device="cuda"),
                                    weight=torch.full((hidden,), 2.0 ** -125, device="cuda"), eps=0.0, fp8=True)
    # 2^-110 / 448 = 2^-116 / 7 is no fp32 value: the nearest one, half a step away at most
    assert abs(float(xs[0]) - 2.0 ** -110 / 448) <= ref.U * 2.0 ** -110 / 448
    assert bool(((ref.e4m3(x8) * xs.double().cpu()[:, None] - 2.0 ** -125).abs() <= 2.0 ** -10 * 2.0 ** -110 / 448).all())


def test_no_tokens():
    y = torch.empty((0, 640), dtype=BF16, device="cuda")
    r, h, x8, xs = w4.residual_norm(y, y, fp8=True)
    assert r.shape == h.shape == x8.shape == (0, 640) and xs.shape == (0,)


def test_codes_serve_the_linear():
    say("residual_norm into the linear")
    g = torch.Generator().manual_seed(7)
    codes, exps = ref.mxfp4_random(256, 512, g)
    pw = w4.mxfp4_prepare(codes.cuda(), exps.cuda())
    y = _normal(g, 5, 512, dtype=BF16)
    _, h, x8, xs = w4.residual_norm(y, fp8=True)
    out = w4.mxfp4_gemm_prepared(x8, xs, pw)
    w = ref.mxfp4(codes, exps)
    x = ref.e4m3(x8) * xs.double().cpu()[:, None]
    want, off = x @ w.T, ref.product_error(x, w)
    assert bool(((out.double().cpu() - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all())
