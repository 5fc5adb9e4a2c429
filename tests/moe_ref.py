"""Plain references in 64 bits (torch, CPU) of the expert half of a layer, with how far a
kernel that works in fp32 and rounds once may be off.  No code of the library.

U = 2^-24, half a step of fp32.  A sum of squares over a row passes at most 64 additions in a
thread, 6 in a wave and 16 over the waves, all of one sign, so its relative error is under
90 U; the root halves it, and division, root and products add some 10 U: a norm's factor is
within 2^-18 (64 U)."""
import torch

U = 2.0 ** -24
NORM = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}


def residual_norm(y, residual=None, weight=None, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """(r, h, error of r, error of h): exact values, and the error of fp32 work before any rounding."""
    d = lambda x: None if x is None else x.detach().cpu().double()
    u, residual, weight, post_weight, gate = d(y), d(residual), d(weight), d(post_weight), d(gate)
    if post_weight is not None:
        u = u / (u.square().mean(1, keepdim=True) + eps).sqrt() * post_weight
    if gate is not None:
        u = u * gate
    u = scale * u
    r = u if residual is None else residual + u
    off = 2 * NORM * u.abs() + 2 * U * r.abs()
    k = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
    w = torch.ones(r.shape[1], dtype=torch.float64) if weight is None else weight
    h = r * k * w
    norm = r.norm(dim=1, keepdim=True)
    carried = torch.where(norm > 0, off.norm(dim=1, keepdim=True) / norm.clamp_min(1e-300), 0.0)
    return r, h, off, off * k * w.abs() + h.abs() * (carried + 2 * NORM)


def route(logits, top_k, score="softmax", bias=None, groups=1, groups_kept=1, group_top=1, renormalize=True, scale=1.0):
    """(weights, ids) by plain loops."""
    x = logits.detach().cpu().double()
    x = torch.where(x.isnan(), float("-inf"), x)
    tokens, experts = x.shape
    weights, ids = torch.zeros((tokens, top_k), dtype=torch.float64), torch.full((tokens, top_k), -1, dtype=torch.int32)
    for t in range(tokens):
        row = x[t]
        top = row.max()
        if score == "softmax":
            p = torch.where(row == top, 1.0, torch.exp(row - top))
            p = torch.where(row == float("-inf"), 0.0, p)
            p = p / p.sum() if float(p.sum()) > 0 else p
        else:
            p = 1 / (1 + torch.exp(-row))
        by = row.clone()
        if bias is not None or groups > 1:
            by = p + (0 if bias is None else bias.detach().cpu().double())
            by = torch.where((row == float("-inf")) | by.isnan(), float("-inf"), by)
        by = by.tolist()
        size = experts // groups
        if groups > 1:
            count = [sum(sorted(by[g * size:(g + 1) * size], reverse=True)[:group_top]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-count[g], g))[:groups_kept]
            by = [v if e // size in kept else float("-inf") for e, v in enumerate(by)]
        order = [e for e in sorted(range(experts), key=lambda e: (-by[e], e)) if by[e] > float("-inf")][:top_k]
        w = p[order]
        if renormalize:
            w = w / w.sum() if len(order) and float(w.sum()) > 0 else torch.zeros_like(w)
        weights[t, :len(order)] = w * scale
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
    return weights, ids


GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def mxfp4(codes, exps):
    """codes uint8 [rows, n / 2], exponents uint8 [rows, n / 32] -> fp64 [rows, n]."""
    codes, exps = codes.cpu(), exps.cpu()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    return GRID[c % 8] * (1 - 2 * (c // 8)) * torch.exp2(exps.double() - 127).repeat_interleave(32, 1)


def e4m3(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def nearest_e4m3(a):
    """(nearest values of |a| <= 448, ties to even; the grid's step at each a)."""
    _, e = torch.frexp(a)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (a / step).round() * step, step


def held(v, off):
    """The values that v [n, inter] is held as between the products (e4m3 with a power of two per 32), and
    how far those of v + o with |o| <= off may be from them: a step of the grid where v is that near a
    border of two codes, twice that where the block's power may change as well."""
    b, o = v.unflatten(1, (-1, 32)), off.unflatten(1, (-1, 32))
    most, near = b.abs().amax(2, keepdim=True), (b.abs() + o).amax(2, keepdim=True)

    def power(m):
        m = m.clamp_min(2.0 ** -126)
        _, e = torch.frexp(m)              # m in [2^(e - 1), 2^e): 448 2^k is in [2^(k + 8), 2^(k + 9))
        k = e - 9
        return torch.where(m > 448 * torch.exp2(k.double()), k + 1, k).clamp_min(-127)

    k = power(most)
    p = torch.exp2(k.double())
    q, step = nearest_e4m3(b / p)
    mid = ((b / p / step - 0.5).round() + 0.5) * step    # the nearest border of two codes
    slack = torch.where((b / p - mid).abs() <= o / p, step * p, 0.0)
    other = power(near) != k
    low = power((b.abs() - o).clamp_min(0).amax(2, keepdim=True)) != k
    slack = torch.where(other | low, 2 * step * p, slack)
    return (q * p).flatten(1), slack.flatten(1)


def product_error(x, w):
    """How far the matrix instructions' x [n, K] @ w [rows, K].T may be off.  fp32 sums of K / 128 steps, joined
    from at most 16 parts, are within 2^-18 of the sum of magnitudes.  Inside a step the 128 products are
    aligned to the largest and cut 2^-14 below it (448 - 448 + 2^-6 gives 0, with 2^-5 it is exact): cuts
    of uniform size and random sign add up to sqrt(128 / 12) 2^-14 = 2^-12.3 of the largest at one standard
    deviation, of which 2^-11 is two and a half; it is taken for every step, and the largest product as that
    of the step's largest factors, which they hardly ever are at one place."""
    step = lambda a: a.abs().unflatten(1, (-1, 128)).amax(2)
    return NORM * (x.abs() @ w.abs().T) + 2.0 ** -11 * (step(x) @ step(w).T)


def experts(x8, xs, ids, weights, up, down, n_experts, act):
    """(out, error): up and down are row-major (codes, exponents)."""
    x = e4m3(x8) * xs.cpu().double()[:, None]
    ids, weights = ids.cpu().long(), weights.cpu().double()
    tokens, hidden = x.shape
    inter = down[0].shape[1] * 2
    out, err = torch.zeros((tokens, hidden), dtype=torch.float64), torch.zeros((tokens, hidden), dtype=torch.float64)
    for e in range(n_experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        w = mxfp4(up[0][e * 2 * inter:(e + 1) * 2 * inter], up[1][e * 2 * inter:(e + 1) * 2 * inter])
        a, off = x[t] @ w.T, product_error(x[t], w)
        g, u, dg, du = a[:, :inter], a[:, inter:], off[:, :inter], off[:, inter:]
        if act == "silu":
            f = g / (1 + torch.exp(-g))
        else:
            f = 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
        v = f * u
        # |act'| < 1.13; exponentials of |g| up to 2^7 are within 2^7 U, some 16 roundings beside
        dv = 1.13 * dg * u.abs() + f.abs() * du + 1.13 * dg * du + v.abs() * 160 * U
        q, slack = held(v, dv)
        w = mxfp4(down[0][e * hidden:(e + 1) * hidden], down[1][e * hidden:(e + 1) * hidden])
        s = weights[t, j, None]
        out.index_add_(0, t, s * (q @ w.T))
        err.index_add_(0, t, s.abs() * (slack @ w.abs().T + product_error(q, w)))
    return out, err


def mxfp4_random(rows, cols, gen, device="cpu"):
    """Codes and exponents of about unit-variance rows: [rows, cols / 2], [rows, cols / 32]."""
    codes = torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=torch.uint8)
    mid = 127 - round(0.5 * float(torch.log2(torch.tensor(float(cols)))) + 1.5)
    exps = torch.randint(mid - 1, mid + 2, (rows, cols // 32), generator=gen, dtype=torch.uint8)
    return codes.to(device), exps.to(device)
