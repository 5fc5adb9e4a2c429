"""Plain 64-bit forms of the attention block's operators, on the CPU, for the tests:
norms with rotation, the MXFP4 encoding of a 32-block by nearest-value search, and
softmax attention over a paged cache, sequence by sequence and head by head."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# half a rounding step, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half of the smallest step (subnormals)
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def table(rows, rot, base=10000.0):
    """fp32 [rows, rot]: cosines, then sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """(values, bound) in 64 bits for x [tokens, heads, d]: bound is the sum of magnitudes that
    each result is made of, which its fp32 error is relative to."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    y, mag = x.clone(), x.abs()
    if cos_sin is not None:
        r = cos_sin.shape[1]
        i = torch.arange(r // 2)
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        t = cos_sin.double()[positions][:, None]
        c, s = t[..., :r // 2], t[..., r // 2:]
        a, b = x[..., p], x[..., q]
        y[..., p], y[..., q] = a * c - b * s, b * c + a * s
        mag[..., p] = mag[..., q] = a.abs() + b.abs()
    return y, mag


def encode(x, mode):
    """fp32 [..., n] -> codes uint8 [..., n] (0..15) and exponent bytes [..., n / 32]."""
    b = x.double().unflatten(-1, (-1, 32))
    codes = torch.zeros(b.shape, dtype=torch.uint8)
    exps = torch.zeros(b.shape[:-1], dtype=torch.uint8)
    for at in range(exps.numel()):
        v = b.reshape(-1, 32)[at]
        most = float(v.abs().max())
        if not math.isfinite(most):
            exps.view(-1)[at] = 255
            continue
        e = 0
        if most > 0:
            m, p = math.frexp(max(most, 2.0 ** -126))    # most = m 2^p, m in [0.5, 1)
            e = p - 3 if mode == "ocp" or m <= 0.75 else p - 2
            e = max(-127, min(127, e))
        a = (v.abs() * 2.0 ** -e).float().double()
        far = (a[:, None] - GRID).abs()
        near = far.amin(1, keepdim=True)
        tied = far == near                                # at most two neighbours
        odd = torch.arange(8) % 2 == 1
        pick = torch.where(tied & odd, 1, torch.where(tied, 0, 2)).argmin(1)
        c = torch.where((v < 0) & (pick > 0), pick + 8, pick)
        codes.view(-1, 32)[at] = c.to(torch.uint8)
        exps.view(-1)[at] = e + 127
    return codes.flatten(-2), exps


def decode(codes, exps):
    """codes (0..15) [..., n], bytes [..., n / 32] -> fp64 [..., n]; byte 255 -> NaN."""
    v = GRID[(codes & 7).long()] * torch.where(codes > 7, -1.0, 1.0)
    s = torch.where(exps == 255, torch.nan, torch.exp2(exps.double() - 127))
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def attention(q, k_of, v_of, seqs, scale, causal, window, group, p_half):
    """q [tokens, heads, d] (its own type); k_of / v_of(sequence) -> fp64 [keys, kv_heads, d]; seqs: (first
    token, tokens, context).  Returns fp64 outputs and how far a kernel's may be off: probabilities rounded
    by p_half, scores by fp32 sums and by the smallest query values, outputs rounded once."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    d = q.shape[2]
    for s, (t0, n, ctx) in enumerate(seqs):
        if ctx == 0 or n == 0:
            continue
        k, v = k_of(s), v_of(s)
        for h in range(q.shape[1]):
            kh, vh = k[:, h // group], v[:, h // group]
            x = q[t0:t0 + n, h].double()
            sc = x @ kh.T * scale
            pos = ctx - n + torch.arange(n)[:, None]
            j = torch.arange(ctx)
            seen = torch.ones((n, ctx), dtype=torch.bool)
            if causal:
                seen = j <= pos
                if window:
                    seen &= j > pos - window
            some = seen.any(1)
            sc = sc.masked_fill(~seen, -math.inf)
            p = torch.where(seen, torch.exp(sc - sc.amax(1, keepdim=True)), 0.0)
            p = torch.where(some[:, None], p / p.sum(1, keepdim=True).clamp_min(1e-300), 0.0)
            o = torch.where(some[:, None], torch.where(p[..., None] > 0, p[..., None] * vh, 0.0).sum(1), 0.0)
            mag = torch.where(p[..., None] > 0, p[..., None] * vh.abs(), 0.0).sum(1)
            dot = (x.abs() @ torch.where(seen.any(0)[:, None], kh, 0.0).abs().T) * abs(scale)
            kabs = torch.where(seen.any(0)[:, None], kh, 0.0).abs().sum(1).max() * abs(scale)
            err = (d + 8) * 2.0 ** -23 * dot.amax(1) + 2.0 ** -21 * x.abs().amax(1) * kabs
            rel = p_half + 2 * err + 4 * ctx * 2.0 ** -24 + 2.0 ** -20
            out[t0:t0 + n, h] = o
            tol[t0:t0 + n, h] = rel[:, None] * mag + HALF[q.dtype] * o.abs() + LEAST[q.dtype]
    return out, tol
