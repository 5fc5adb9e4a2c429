"""Close bounds for the experts' products (plain torch in 64 bits, CPU), beside moe_ref.py's worst cases.

What a token's output may differ by, as a norm over its values:

  its rounding to bf16   half steps of 2^-8 of each value's power of two, as uniform errors at most
                         2^-7 / sqrt(12) = 2^-8.79 of the norm; over n values the mean square of uniform
                         errors, weighted by squares of a normal value's kind, spreads by some
                         sqrt(0.8 * 3 / n), of which four are allowed
  values of v on the     v is off by fp32 work alone: the first product's sum of exact products passes
  other side of a        K / 32 + 16 additions, each within 2^-24 of a partial sum; as errors of random sign of
  border of two codes    sums of about the root of the products' squares, sqrt(K / 32 + 16) 2^-24 of it, of
                         which four are taken; exp and 1 / x are within 2^-17 of f for |g| to 2^6, and some 16
                         roundings beside.  Where a border is that near, the step between the codes counts
  the second product     cuts of 2^-14 of the largest of 128 products, of uniform size and random sign: sqrt(128 / 12)
                         2^-14 of the largest for each step, which is taken from the factors' largest in
                         each output, and sqrt of the number of steps for their sum
"""
import math

import torch

import moe_ref as ref

ROUND = 2.0 ** -7 / math.sqrt(12)


def act_of(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu_erf":     # no activation of the library: what gelu_tanh must not be taken for
        return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))
    return 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


def experts(x8, xs, ids, weights, up, down, n_experts, act):
    """(out, border, cut): the exact output, and per token the norms that borders of v and the second
    product's cuts may add."""
    x = ref.e4m3(x8) * xs.cpu().double()[:, None]
    ids, weights = ids.cpu().long(), weights.cpu().double()
    tokens, hidden = x.shape
    inter = down[0].shape[1] * 2
    out = torch.zeros((tokens, hidden), dtype=torch.float64)
    border, cut = torch.zeros_like(out), torch.zeros_like(out)
    rows = lambda w, e, n: ref.mxfp4(w[0][e * n:(e + 1) * n], w[1][e * n:(e + 1) * n])
    step = lambda a: a.abs().unflatten(1, (-1, 128)).amax(2)
    for e in range(n_experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        w = rows(up, e, 2 * inter)
        a = x[t] @ w.T
        off = 4 * math.sqrt(hidden / 32 + 16) * ref.U * (x[t].square() @ w.square().T).sqrt()
        g, u, dg, du = a[:, :inter], a[:, inter:], off[:, :inter], off[:, inter:]
        f = act_of(g, act)
        v = f * u
        q, slack = ref.held(v, 1.13 * dg * u.abs() + f.abs() * du + v.abs() * (2.0 ** -17 + 16 * ref.U))
        w = rows(down, e, hidden)
        s = weights[t, j, None]
        out.index_add_(0, t, s * (q @ w.T))
        border.index_add_(0, t, s.abs() * (slack @ w.abs().T))
        # squares, as errors of independent sign
        cut.index_add_(0, t, (s * math.sqrt(128 / 12) * 2.0 ** -14).square() * (step(q).square() @ step(w).square().T))
    return out, border.norm(dim=1), cut.sum(1).sqrt()


def check(got, want, name=""):
    out, border, cut = want
    off = (got.double().cpu() - out).norm(dim=1)
    n = out.norm(dim=1)
    wide = ROUND * (1 + 4 * math.sqrt(2.4 / out.shape[1]))
    bad = ~(off <= wide * n + border + 2 * cut)
    assert not bad.any(), (name, int(bad.sum()), (off / n)[bad][:4], ((wide * n + border + 2 * cut) / n)[bad][:4])
    # all of them: borders of many tokens are independent
    whole = float(ROUND * (1 + 4 * math.sqrt(2.4 / out.numel())) * n.norm() + border.norm() + 2 * cut.norm())
    assert float(off.norm()) <= whole, (name, float(off.norm() / n.norm()), whole / float(n.norm()))
    return float(off.norm() / n.norm()), whole / float(n.norm())
