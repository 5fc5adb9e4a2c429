"""CPU: calls whose launch would pass HIP's 2^32 threads of a grid are refused as unsupported
shapes at the C entry points, before any device work (the fake pointers are never touched)."""
import pytest

from test_attention_refusals import FAKE, SHAPE, L, _append, _attention, _cache, _norm  # noqa: F401


def test_read(L):  # noqa: F811
    for d, tokens in ((256, 1 << 26), (256, (1 << 26) + 5), (128, 1 << 27), (256, (1 << 29) - 1)):
        c = _cache(kv_heads=1, head_dim=d)
        assert L.w4a8_kv_read_mxfp4(c, tokens, FAKE, FAKE, FAKE, None) == SHAPE, (d, tokens)


@pytest.mark.parametrize("d,tokens,hq", [(256, 1 << 27, 1), (128, 1 << 28, 1), (64, 1 << 29, 1), (256, 1 << 27, 6)])
def test_norms(L, d, tokens, hq):  # noqa: F811
    assert _norm(L, q=FAKE, hq=hq, k=None, hk=0, ko=None, tokens=tokens, d=d, rot=0) == SHAPE


@pytest.mark.parametrize("d,tokens,hk", [(256, 1 << 26, 1), (256, 1 << 24, 8), (128, 1 << 27, 1), (64, 1 << 28, 1)])
def test_append(L, d, tokens, hk):  # noqa: F811
    assert _append(L, cache=_cache(kv_heads=hk, head_dim=d), tokens=tokens) == SHAPE


@pytest.mark.parametrize("type", [0, 1])
@pytest.mark.parametrize("d,max_q,seqs", [(64, 65, 1 << 23), (128, 100, 1 << 23), (256, 33, 1 << 24)])
def test_prompts(L, type, d, max_q, seqs):  # noqa: F811
    c = _cache(kv_heads=1, head_dim=d)
    assert _attention(L, cache=c, type=type, hq=1, cu=FAKE, seqs=seqs, max_q=max_q, tw=1, tst=1) == SHAPE
