"""Measured cases of the mixture-of-experts half of a decoder layer on MXFP4 weights.

Three operators, each with its plain form in elementary torch operations:

  norm     norm after a block, its gate and scale, the residual sum, and the norm before the next
           block, whose result leaves as 16-bit values, as per-token fp8 codes with scales, or both
  route    top experts of each token from the router's logits, with their weights
  experts  gated products of each token with its experts' MXFP4 weights, summed by the router's weights

Weights are e2m1 codes, two per byte with the even element in the low nibble, with one power-of-two
exponent byte (exponent + 127) per 32 elements of a row.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(tokens, hidden, post=True, gate="none", scale=1.0, residual="same", out="both", dtype="bf16", **name):
    return dict(name, op="norm", tokens=tokens, hidden=hidden, post=post, gate=gate, scale=scale, residual=residual,
                out=out, dtype=dtype)


def _route(tokens, experts, top_k, score="softmax", bias=False, groups=1, kept=1, group_top=1, renormalize=True,
           scale=1.0, masked=0.0, dtype="fp32", **name):
    return dict(name, op="route", tokens=tokens, experts=experts, top_k=top_k, score=score, bias=bias, groups=groups,
                kept=kept, group_top=group_top, renormalize=renormalize, scale=scale, masked=masked, dtype=dtype)


def _experts(tokens, experts, top_k, hidden, inter, act="silu", padded=0, **name):
    return dict(name, op="experts", tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter, act=act,
                padded=padded)


def listed():
    return [
        # one user's decode step: norm after attention, residual, norm for the router and codes for the experts
        _norm(1, 5120, name="norm one token"),
        # a decode batch of an odd size in fp16, one gate per channel, a residual scale
        _norm(61, 4096, gate="channel", scale=0.22, dtype="fp16", name="norm decode batch fp16"),
        # rows that no vector load fits, a 32-bit residual stream, one gate per token, 16-bit output alone
        _norm(777, 2051, post=False, gate="token", residual="fp32", out="16", name="norm odd rows fp32 residual"),
        # the prompts of a full prefill batch, codes alone for the next linear
        _norm(16384, 5120, post=False, out="fp8", name="norm prompts"),
        # one token's eight of 128 experts
        _route(1, 128, 8, name="route one token"),
        # a decode batch whose experts are limited to groups, with a balancing bias, bf16 logits
        _route(61, 256, 8, score="sigmoid", bias=True, groups=8, kept=4, group_top=2, scale=2.5, dtype="bf16",
               name="route decode batch groups"),
        # few experts of which some are off, weights as the softmax gives them
        _route(1021, 8, 2, renormalize=False, masked=0.1, name="route few experts masked"),
        # the prompts of a full prefill batch
        _route(16384, 128, 8, name="route prompts"),
        # one user's decode step through 128 experts
        _experts(1, 128, 8, 2048, 768, name="experts one token"),
        # drafted tokens of a padded batch, wider experts
        _experts(13, 64, 6, 2048, 1408, act="gelu_tanh", padded=2, name="experts drafts padded"),
        # a decode batch that meets nearly every expert
        _experts(64, 128, 8, 2048, 768, name="experts decode batch"),
        # a large decode batch on few large experts
        _experts(251, 8, 2, 4096, 8192, name="experts few large"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {c: max(_cost(x) for x in listed() if x["op"] == c) for c in ("norm", "route", "experts")}
    op = rng.choice(["norm", "route", "experts", "experts"])
    while True:
        if op == "norm":
            hidden = _log(rng, 32, 1024) * 8 if rng.random() < 0.75 else _log(rng, 65, 8191)
            case = _norm(_log(rng, 1, 16384), hidden, rng.random() < 0.6, rng.choice(["none", "none", "channel", "token", "full"]),
                         rng.choice([1.0, 1.0, 0.22, 0.5]), rng.choice(["same", "same", "fp32", "none"]),
                         rng.choice(["16", "fp8", "both"]), rng.choice(["bf16", "bf16", "fp16"]))
        elif op == "route":
            experts = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512])
            groups = rng.choice([1, 1, 4, 8]) if experts >= 64 and experts % 8 == 0 else 1
            kept = max(1, groups // 2)
            top_k = _log(rng, 1, min(10, experts // 2))
            case = _route(_log(rng, 1, 16384), experts, top_k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.4, groups,
                          kept, rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                          rng.choice([0.0, 0.0, 0.1]), rng.choice(["fp32", "bf16", "fp16"]))
        else:
            experts = rng.choice([8, 16, 32, 60, 64, 128, 256])
            top_k = _log(rng, 1, min(8, experts // 4))
            tokens = _log(rng, 1, 256)
            case = _experts(tokens, experts, top_k, 128 * _log(rng, 4, 40), 128 * _log(rng, 2, 64),
                            rng.choice(["silu", "silu", "gelu_tanh"]), rng.choice([0, 0, rng.randint(0, tokens // 4)]))
            # the plain form holds all experts' weights and products in 32 bits
            if experts * case["hidden"] * case["inter"] > 2 ** 28 or experts * tokens * (case["hidden"] + 2 * case["inter"]) > 2 ** 29:
                continue
        if _cost(case) <= most[op]:
            return case


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        values = t * case["hidden"]
        r = {"same": 2, "fp32": 4, "none": 0}[case["residual"]]
        gates = {"none": 0, "channel": case["hidden"], "token": t, "full": values}[case["gate"]]
        out = {"16": 2, "fp8": 1, "both": 3}[case["out"]]
        return {"bytes": values * (2 + 2 * r + out) + 2 * gates + (4 * t if case["out"] != "16" else 0) +
                4 * case["hidden"] * (2 if case["post"] else 1), "flops": values * (12 if case["post"] else 8)}
    if case["op"] == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": t * case["experts"] * size + 8 * t * case["top_k"] + (4 * case["experts"] if case["bias"] else 0),
                "flops": 6 * t * case["experts"]}
    live = t - case["padded"]
    e, k, h, i = case["experts"], case["top_k"], case["hidden"], case["inter"]
    met = e * (1 - (1 - k / e) ** live)  # experts that some token goes to, were all as likely
    return {"bytes": met * 3 * h * i * (1 / 2 + 1 / 32) + t * (h + 4 + 8 * k + 2 * h), "flops": 6 * live * k * h * i}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weights(rows, cols, gen):
    """An MXFP4 weight of about normal values of variance 1 / cols: codes [rows, cols / 2], exponents [rows, cols / 32]."""
    def codes():
        x = torch.randn((rows, cols // 2), generator=gen, device="cuda", dtype=torch.float32).mul_(3.0)
        mag = x.abs().clamp_max_(7.0).to(torch.uint8)
        return mag.add_((x < 0).to(torch.uint8).mul_(8))
    low = codes()
    low.add_(codes().mul_(16))
    mid = 127 + round(math.log2(cols ** -0.5 / 2.2))
    exps = torch.randint(mid - 1, mid + 2, (rows, cols // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return low, exps


def _masked(x, share, gen):
    return x.masked_fill_(torch.rand(x.shape, generator=gen, device="cuda") < share, float("-inf")) if share else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = case["tokens"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=case)
    if case["op"] == "norm":
        dtype, hidden = DTYPES[case["dtype"]], case["hidden"]
        s["y"] = (normal(t, hidden) * (0.5 + normal(t, 1).abs())).to(dtype)
        kind = {"same": dtype, "fp32": torch.float32, "none": None}[case["residual"]]
        s["residual"] = None if kind is None else (normal(t, hidden) * 3 * torch.exp(0.5 * normal(hidden))).to(kind)
        s["post_weight"] = 1 + 0.2 * normal(hidden) if case["post"] else None
        s["weight"] = 1 + 0.2 * normal(hidden)
        shape = {"none": None, "channel": (1, hidden), "token": (t, 1), "full": (t, hidden)}[case["gate"]]
        s["gate"] = None if shape is None else (1 + 0.5 * normal(*shape)).to(dtype).expand(t, hidden)
    elif case["op"] == "route":
        e = case["experts"]
        s["logits"] = _masked((normal(t, e) + 0.5 * normal(e)).to(DTYPES[case["dtype"]]), case["masked"], gen)
        s["bias"] = 0.1 * normal(e) if case["bias"] else None
    else:
        e, k, h, i = case["experts"], case["top_k"], case["hidden"], case["inter"]
        x = normal(t, h) * (0.5 + normal(t, 1).abs())
        s["x_scale"] = x.abs().amax(1) / 448
        s["x_fp8"] = (x / s["x_scale"][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        top = torch.sort(normal(t, e) + 0.5 * normal(e), dim=1, descending=True)
        s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top.values[:, :k], 1).contiguous()
        if case["padded"]:
            s["ids"][t - case["padded"]:] = -1
        s["up"] = _weights(e * 2 * i, h, gen)
        s["down"] = _weights(e * h, i, gen)
        if own:
            import w4a8_gemm_amd as w4
            s["experts"] = w4.ExpertsMXFP4.prepare(*s["up"], *s["down"], experts=e)
            s["workspace"] = w4.MoEWorkspace(tokens=t, top_k=k, experts=e, hidden=h, inter=i)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import w4a8_gemm_amd as w4
    case = s["case"]
    if case["op"] == "norm":
        r, h, x8, xs = w4.residual_norm(s["y"], s["residual"], weight=s["weight"], post_weight=s["post_weight"], gate=s["gate"],
                                        scale=case["scale"], eps=EPS, values=case["out"] != "fp8", fp8=case["out"] != "16")
        return [r, h, None if x8 is None else x8.view(torch.float8_e4m3fn), xs]
    if case["op"] == "route":
        return w4.moe_route(s["logits"], case["top_k"], score=case["score"], bias=s["bias"], groups=case["groups"],
                            groups_kept=case["kept"], group_top=case["group_top"], renormalize=case["renormalize"],
                            scale=case["scale"])
    return w4.moe_mxfp4(s["x_fp8"], s["x_scale"], s["ids"], s["weights"], s["experts"], act=case["act"],
                        workspace=s["workspace"])


def _run_plain(s):
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}[s["case"]["op"]](s, s["case"])


def _plain_norm(s, case):
    u = s["y"].float()
    if case["post"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * s["post_weight"]
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = u * case["scale"]
    if s["residual"] is not None:
        r = r + s["residual"].float()
    h = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    stored = None if s["residual"] is None else r.to(s["residual"].dtype)
    h16 = None if case["out"] == "fp8" else h.to(s["y"].dtype)
    if case["out"] == "16":
        return [stored, h16, None, None]
    most = h.abs().amax(-1, keepdim=True)
    most = torch.where(most > 0, most, 448.0)
    return [stored, h16, (h * (448 / most)).to(torch.float8_e4m3fn), (most / 448).squeeze(-1)]


def _plain_route(s, case):
    """The choice is by the logits themselves where it goes by nothing else, else by scores in 64 bits: which expert is
    met must not depend on a rounding."""
    logits, k = s["logits"].double(), case["top_k"]
    off = logits == float("-inf")
    if case["score"] == "softmax":
        scores = torch.exp(logits - logits.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float64).min))
        total = scores.sum(1, keepdim=True)
        scores = scores / total.where(total > 0, 1.0)
    else:
        scores = 1 / (1 + torch.exp(-logits))
    by = logits
    if case["bias"] or case["groups"] > 1:
        by = scores if s["bias"] is None else scores + s["bias"].double()
        by = by.masked_fill(off, float("-inf"))
    if case["groups"] > 1:
        parts = by.unflatten(1, (case["groups"], -1))
        top = torch.sort(parts, dim=2, descending=True).values[..., :case["group_top"]].sum(2)
        keep = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        kept = torch.zeros_like(top, dtype=torch.bool).scatter_(1, keep, True)
        by = parts.masked_fill(~kept[..., None], float("-inf")).flatten(1)
    best = torch.sort(by, dim=1, descending=True, stable=True)
    ids, none = best.indices[:, :k], best.values[:, :k] == float("-inf")
    weights = scores.gather(1, ids).masked_fill(none, 0.0)
    if case["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = weights / total.where(total > 0, 1.0)
    return (weights * case["scale"]).float(), ids.to(torch.int32).masked_fill(none, -1)


def _values(codes, exps):
    """codes [.., n / 2] and exponent bytes [.., n / 32] -> fp32 [.., n]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    return (grid[pair].unflatten(-1, (-1, 32)) * torch.exp2(exps.float() - 127)[..., None]).flatten(-2)


def _held_in_8_bits(x):
    """fp32 [.., n, t] -> the values that its blocks of 32 along n are held as: e4m3 times the least power of two that
    keeps the block's largest magnitude within 448."""
    b = x.unflatten(-2, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-2, keepdim=True).clamp_min(2.0 ** -126))  # m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875)).clamp_min(-127).float()
    return ((b * torch.exp2(-e)).to(torch.float8_e4m3fn).float() * torch.exp2(e)).flatten(-3, -2)


def _plain_experts(s, case):
    e, i, t = case["experts"], case["inter"], case["tokens"]
    live = s["ids"] >= 0
    at = s["ids"].clamp_min(0).long()
    share = torch.zeros((t, e), device="cuda").scatter_add_(1, at, s["weights"] * live)
    met = torch.zeros((t, e), device="cuda").scatter_add_(1, at, live.float()).amax(0).nonzero().squeeze(1)
    n = met.shape[0]  # the experts that some token goes to
    up, down = ((codes.unflatten(0, (e, -1))[met].flatten(0, 1), exps.unflatten(0, (e, -1))[met].flatten(0, 1))
                for codes, exps in (s["up"], s["down"]))
    x = s["x_fp8"].view(torch.float8_e4m3fn).float() * s["x_scale"][:, None]
    a = torch.matmul(_values(*up), x.T.contiguous()).unflatten(0, (n, 2 * i))
    g, u = a[:, :i], a[:, i:]
    if case["act"] == "silu":
        g = g / (1 + torch.exp(-g))
    else:
        g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    h = _held_in_8_bits(g * u)
    y = torch.matmul(_values(*down).unflatten(0, (n, -1)), h)  # [experts met, hidden, tokens]
    return (y * share[:, met].T[:, None]).sum(0).T.contiguous().to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "experts": _exact_experts}[case["op"]](s, case)


def _unit(x):
    """Rows over their root mean square."""
    return x / ((x.pow(2).sum(1) / x.shape[1] + EPS) ** 0.5)[:, None]


def _nearest_e4m3(a):
    """The nearest e4m3 value of each a, |a| <= 448, ties to even."""
    _, e = torch.frexp(a)  # |a| = m 2^e, m in [0.5, 1): four bits from 2^(e - 1) down, and none under 2^-9
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (a / step).round() * step


def _exact_norm(s, case):
    r = s["y"].double()
    if s["post_weight"] is not None:
        r = _unit(r) * s["post_weight"].double()
    r = r * case["scale"] * (1 if s["gate"] is None else s["gate"].double())
    stored = None
    if s["residual"] is not None:
        stored = r = r + s["residual"].double()
    h = _unit(r) * s["weight"].double()
    step = h.abs().max(1).values / 448
    step[step == 0] = 1.0
    return [stored, None if case["out"] == "fp8" else h,
            *((None, None) if case["out"] == "16" else (_nearest_e4m3(h / step[:, None]), step))]


def _exact_route(s, case):
    x = s["logits"].double()
    w = torch.softmax(x, 1).nan_to_num(0.0) if case["score"] == "softmax" else torch.sigmoid(x)
    by = x
    if case["bias"] or case["groups"] > 1:
        by = torch.where(x == -math.inf, -math.inf, w + (0.0 if s["bias"] is None else s["bias"].double()))

    def lowest_of_largest(v):
        index = torch.arange(v.shape[1], device="cuda")
        return torch.where(v == v.amax(1, keepdim=True), index, v.shape[1]).amin(1, keepdim=True)

    if case["groups"] > 1:
        size = case["experts"] // case["groups"]
        group = torch.topk(by.reshape(-1, case["groups"], size), min(case["group_top"], size), 2).values.sum(2)
        out = torch.ones_like(group, dtype=torch.bool)
        rank = torch.where(group == -math.inf, -1e300, group)  # a group with nothing to choose is the last, and counts once
        for _ in range(case["kept"]):
            at = lowest_of_largest(rank)
            out.scatter_(1, at, False)
            rank = rank.scatter(1, at, -math.inf)
        by = torch.where(out.repeat_interleave(size, 1), -math.inf, by)
    chosen, values = [], []
    for _ in range(case["top_k"]):
        at = lowest_of_largest(by)
        values.append(torch.where(by.gather(1, at) == -math.inf, 0.0, w.gather(1, at)))
        chosen.append(at)
        by = by.scatter(1, at, -math.inf)
    w = torch.cat(values, 1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return w * case["scale"], None


def _exact_experts(s, case):
    e, h, i = case["experts"], case["hidden"], case["inter"]
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")

    def rows(w, lo, n):
        codes, exps = w[0][lo:lo + n], w[1][lo:lo + n].double()
        c = torch.stack([codes & 15, codes >> 4], -1).reshape(n, -1).long()
        return grid[c % 8] * (1 - 2 * (c // 8)) * torch.exp2(exps - 127).repeat_interleave(32, 1)

    x = s["x_fp8"].view(torch.float8_e4m3fn).double() * s["x_scale"].double()[:, None]
    out = torch.zeros((case["tokens"], h), dtype=torch.float64, device="cuda")
    for n in range(e):
        t, j = (s["ids"] == n).nonzero(as_tuple=True)
        if not t.numel():
            continue
        a = x[t] @ rows(s["up"], 2 * i * n, 2 * i).T.contiguous()
        g, u = a[:, :i], a[:, i:]
        g = g * torch.sigmoid(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        b = (g * u).reshape(-1, i // 32, 32)
        most = b.abs().amax(2, keepdim=True).clamp_min(2.0 ** -126)
        p = torch.ceil(torch.log2(most / 448))
        p = torch.where(most > 448 * torch.exp2(p), p + 1, p)
        p = torch.exp2(torch.where(most <= 448 * torch.exp2(p - 1), p - 1, p).clamp_min(-127))
        v = (_nearest_e4m3(b / p) * p).reshape(-1, i)
        out.index_add_(0, t, s["weights"].double()[t, j, None] * (v @ rows(s["down"], h * n, h).T.contiguous()))
    return out
