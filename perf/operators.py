"""Measured cases of the attention block on the 4-bit paged cache.

Three operators, each with its plain form in elementary torch operations:

  norm_rope   norms of queries and keys for each head, position rotation in the same pass
  append      keys (normed and rotated on the way) and values into the paged MXFP4 cache,
              the queries of the same tokens in the same call; the rows written are read back
              as the values that their 4-bit codes stand for
  attention   softmax attention of new tokens over the paged MXFP4 cache

The cache holds e2m1 codes, two per byte with the even element in the low nibble, as
[pages, kv_heads, page, head_dim / 2], and one power-of-two exponent byte (exponent + 127) per 32
elements as [pages, kv_heads, head_dim / 32, page].  Token i of a sequence lies in row i % page of
the page that entry i // page of the sequence's block table names.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm_rope(tokens, q_heads, kv_heads, head_dim, rot, interleaved=False, norm=True, dtype="bf16", **name):
    return dict(name, op="norm_rope", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, rot=rot,
                interleaved=interleaved, norm=norm, dtype=dtype)


def _append(tokens, seqs, q_heads, kv_heads, head_dim, rot, page, mode="ocp", interleaved=False, norm=True,
            dtype="bf16", padded=0, **name):
    return dict(name, op="append", tokens=tokens, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                rot=rot, page=page, mode=mode, interleaved=interleaved, norm=norm, dtype=dtype, padded=padded)


def _attention(seqs, q_len, context, q_heads, kv_heads, head_dim, page, ragged=True, window=0, causal=True,
               dtype="bf16", **name):
    return dict(name, op="attention", seqs=seqs, q_len=q_len, context=context, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, ragged=ragged, window=window, causal=causal, dtype=dtype)


def listed():
    return [
        # one user's decode step: a single token, where the call's latency is all
        _norm_rope(1, 24, 4, 256, 64, name="norm_rope one token"),
        # a decode batch of an odd size, whole heads rotated
        _norm_rope(61, 32, 8, 128, 128, name="norm_rope decode batch"),
        # a long prompt in fp16 with pairs side by side, without norms
        _norm_rope(4099, 16, 16, 64, 64, interleaved=True, norm=False, dtype="fp16", name="norm_rope fp16 pairs"),
        # the prompts of a full prefill batch
        _norm_rope(16384, 24, 4, 256, 64, name="norm_rope prompts"),
        # one token of one sequence appended, its query in the same call
        _append(1, 1, 24, 4, 256, 64, 64, name="append one token"),
        # a decode batch captured at a larger size than it has sequences: the last slots are padding
        _append(128, 128, 32, 8, 128, 128, 16, padded=9, name="append decode batch"),
        # prompts of five sequences written to the cache
        _append(16381, 5, 24, 4, 256, 64, 64, mode="noclip", name="append prompts"),
        # one user's decode step at a short context
        _attention(1, 1, 1021, 24, 4, 256, 64, name="attention one token"),
        # a decode batch of ragged contexts
        _attention(64, 1, 8192, 32, 8, 128, 32, name="attention decode batch"),
        # few sequences of long contexts: the context is what is read
        _attention(3, 1, 131072, 24, 4, 256, 64, name="attention long context"),
        # verification of drafted tokens, a sliding window, fp16
        _attention(23, 5, 4096, 16, 2, 64, 16, window=1024, dtype="fp16", name="attention drafts fp16"),
        # whole prompts of two sequences
        _attention(2, 8191, 8191, 24, 4, 256, 64, name="attention prompts"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = [(24, 4, 256), (12, 2, 256), (6, 1, 256), (32, 8, 128), (16, 16, 64), (8, 8, 128), (16, 2, 64),
             (28, 4, 128), (20, 1, 128), (64, 4, 128)]
    most = {c: max(_cost(x) for x in listed() if x["op"] == c) for c in ("norm_rope", "append", "attention")}
    op = rng.choice(["norm_rope", "append", "attention", "attention"])
    while True:
        hq, hk, d = rng.choice(heads)
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        page = rng.choice([16, 32, 64, 128])
        rot = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= d])
        tokens = _log(rng, 1, 16384)
        if op == "norm_rope":
            case = _norm_rope(tokens, hq, hk, d, rot, rng.random() < 0.4, rng.random() < 0.7, dtype)
        elif op == "append":
            seqs = tokens if rng.random() < 0.5 and tokens <= 512 else rng.randint(1, min(tokens, 16))
            case = _append(tokens, seqs, hq, hk, d, rot, page, rng.choice(["ocp", "noclip"]), rng.random() < 0.4,
                           rng.random() < 0.7, dtype, rng.randint(0, min(8, tokens - 1)) if seqs == tokens else 0)
        else:
            kind = rng.choice(["decode", "decode", "drafts", "prompts", "chunk"])
            if kind == "decode":
                seqs, q_len, context = _log(rng, 1, 256), 1, _log(rng, 1, 131072)
            elif kind == "drafts":
                seqs, q_len, context = _log(rng, 1, 64), rng.randint(2, 8), _log(rng, 16, 32768)
            elif kind == "prompts":
                seqs, q_len = rng.randint(1, 6), _log(rng, 17, 8192)
                context = q_len
            else:
                seqs, q_len = rng.randint(1, 4), _log(rng, 17, 1024)
                context = q_len + _log(rng, 1, 32768)
            window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
            case = _attention(seqs, q_len, context, hq, hk, d, page, rng.random() < 0.8, window,
                              rng.random() < 0.85 or window > 0, dtype)
        # the plain form holds padded scores, and the batch's keys and values, in 32 bits
        if _cost(case) <= most[op] and _padded_scores(case) <= 2 ** 32 and _padded_keys(case) <= 2 ** 30:
            return case


# ---------------------------------------------------------------------------
# what a case is made of
# ---------------------------------------------------------------------------

def _lengths(case):
    """(query tokens, context) of each sequence of an attention case: with "ragged", spread from about a twelfth of
    the largest to the largest by a fixed rule; of eight or more sequences the last is an unused entry of the batch
    (one token, an empty context)."""
    n, ql, ctx = case["seqs"], case["q_len"], case["context"]
    out = []
    for i in range(n):
        f = 1.0 if i == 0 or not case["ragged"] else 1.0 - 0.92 * ((i * 0.6180339887498949) % 1.0)
        c = max(1, int(ctx * f))
        q = min(c, max(1, int(ql * f)) if ql == ctx else max(1, ql - (i % ql if case["ragged"] else 0)))
        out.append((q, c))
    if case["ragged"] and n >= 8:
        out[-1] = (1, 0)
    return out


def _pairs(case):
    """(query token, key) pairs that the mask of an attention case leaves."""
    total = 0
    for q, c in _lengths(case):
        if case["causal"]:
            w = case["window"] or c
            p0 = c - q
            # sum over i < q of min(w, p0 + i + 1)
            full = max(0, min(q, q - (w - 1 - p0))) if p0 + q > w else 0
            part = q - full
            first = p0 + 1
            total += full * w + part * first + part * (part - 1) // 2 if c else 0
        else:
            total += q * c
    return total


def _keys(case):
    """Keys of the cache that an attention case reads, over its sequences."""
    total = 0
    for q, c in _lengths(case):
        w = case["window"]
        total += min(c, w + q - 1) if w else c
    return total


def _padded_scores(case):
    if case["op"] != "attention":
        return 0
    per = _lengths(case)
    return len(per) * case["q_heads"] * max(q for q, _ in per) * max(c for _, c in per)


def _padded_keys(case):
    if case["op"] != "attention":
        return 0
    per = _lengths(case)
    return len(per) * max(c for _, c in per) * case["kv_heads"] * case["head_dim"]


def work(case):
    d, hq, hk = case["head_dim"], case["q_heads"], case["kv_heads"]
    cached = d / 2 + d / 32  # bytes of one head's row in the cache
    if case["op"] == "norm_rope":
        t = case["tokens"]
        values = t * (hq + hk) * d
        return {"bytes": 4 * values + 4 * t * case["rot"] + 8 * t + (8 * d if case["norm"] else 0),
                "flops": values * (5 if case["norm"] else 1) + 3 * t * (hq + hk) * case["rot"]}
    if case["op"] == "append":
        t = case["tokens"]
        live = t - case["padded"]
        # q, k and v in, q out, the cache's rows written, read again and handed back as 16-bit values
        b = 2 * t * (hq + 2 * hk) * d + 2 * t * hq * d + 4 * t * case["rot"] + 16 * t
        b += 2 * live * hk * cached * 2 + 2 * t * hk * d * 2
        return {"bytes": b, "flops": 6 * t * (hq + 2 * hk) * d}
    t = sum(q for q, _ in _lengths(case))
    return {"bytes": 2 * 2 * t * hq * d + 2 * _keys(case) * hk * cached, "flops": 4 * d * hq * _pairs(case)}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _angles(positions, rot):
    """fp32 [positions, rot]: cosines of the rot / 2 angles, then their sines; the angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _encode_random(shape, head_dim, gen, scale, shift):
    """A cache's worth of normal values of unequal channels, as codes [.., page, head_dim / 2] and exponent bytes
    [.., head_dim / 32, page]."""
    x = torch.randn((*shape, head_dim), generator=gen, device="cuda", dtype=torch.float32)
    channel = torch.exp(0.5 * torch.randn(head_dim, generator=gen, device="cuda")) * scale
    x = x * channel + shift * torch.randn(head_dim, generator=gen, device="cuda")
    codes, e = _encode(x, "ocp")
    return _pack(codes), e.transpose(-1, -2).contiguous()


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=case)
    if case["op"] in ("norm_rope", "append"):
        t = case["tokens"]
        # the rows that a fused projection writes: queries, keys and values of a token side by side
        qkv = (normal(t, (hq + 2 * hk) * d) * 1.5).to(dtype)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["q_weight"] = 1 + 0.2 * normal(d) if case["norm"] else None
        s["k_weight"] = 1 + 0.2 * normal(d) if case["norm"] else None
        seqs = case.get("seqs", 1)
        per = -(-t // seqs)
        first = torch.randint(0, 100_000, (seqs,), generator=gen, device="cuda")
        token = torch.arange(t, device="cuda")
        s["positions"] = (first[token // per] + token % per).contiguous()
        s["cos_sin"] = _angles(100_000 + per, case["rot"])
    if case["op"] == "append":
        page = case["page"]
        pages_of = -(-per // page) + 1
        names = torch.randperm(seqs * pages_of + 3, generator=gen, device="cuda")
        row = first[token // per] % page + token % per
        at = names[(token // per) * pages_of + row // page]
        s["slots"] = (at * page + row % page).contiguous()
        if case["padded"]:
            s["slots"][-case["padded"]:] = -1
        n = names.numel()
        s["cache"] = tuple(torch.zeros(shape, dtype=torch.uint8, device="cuda")
                           for shape in ((n, hk, page, d // 2), (n, hk, d // 32, page)) * 2)
    if case["op"] == "attention":
        page = case["page"]
        per = _lengths(case)
        t = sum(q for q, _ in per)
        s["q"] = (normal(t, hq, d) * 1.5).to(dtype)
        cu = [0]
        for q, _ in per:
            cu.append(cu[-1] + q)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if case["q_len"] > 1 else None
        s["context_lens"] = torch.tensor([c for _, c in per], dtype=torch.int32, device="cuda")
        width = max(1, max(-(-c // page) for _, c in per))
        used = [-(-c // page) for _, c in per]
        names = torch.randperm(sum(used) + 3, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((len(per), width), dtype=torch.int32, device="cuda")
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = names[at:at + u]
            at += u
        s["block_table"] = table
        n = names.numel()
        s["cache"] = (*_encode_random((n, hk, page), d, gen, 1.0, 0.5), *_encode_random((n, hk, page), d, gen, 1.0, 0.3))
        s["max_q"] = max(q for q, _ in per)
        s["scale"] = d ** -0.5
    if own and "cache" in s:
        import w4a8_gemm_amd as w4
        s["cache"] = w4.KVCacheMXFP4(*s["cache"])
        if case["op"] == "attention":
            s["workspace"] = w4.AttentionWorkspace(len(per), s["max_q"], hq, hk, d)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import w4a8_gemm_amd as w4
    case = s["case"]
    if case["op"] == "norm_rope":
        return w4.qk_norm_rope(s["q"], s["k"], s["cos_sin"], s["positions"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"])
    if case["op"] == "append":
        q = w4.kv_append_mxfp4(s["cache"], s["k"], s["v"], s["slots"], mode=case["mode"], cos_sin=s["cos_sin"],
                               positions=s["positions"], k_weight=s["k_weight"], eps=EPS,
                               interleaved=case["interleaved"], q=s["q"], q_weight=s["q_weight"])
        return (q, *w4.kv_read_mxfp4(s["cache"], s["slots"]))
    return w4.attention_mxfp4(s["q"], s["cache"], s["block_table"], s["context_lens"], cu_q=s["cu_q"],
                              max_q=s["max_q"], scale=s["scale"], causal=case["causal"], window=case["window"],
                              workspace=s["workspace"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm_rope":
        return tuple(_norm_rotate(s[n].float(), s[n + "_weight"], s, case).to(s[n].dtype) for n in ("q", "k"))
    if case["op"] == "append":
        q = _norm_rotate(s["q"].float(), s["q_weight"], s, case).to(s["q"].dtype)
        # keys in 64 bits, rounded to 32 before they are encoded: a value next to the border of two codes
        k = _norm_rotate(s["k"].double(), s["k_weight"], s, case).float()
        k_codes, k_exp, v_codes, v_exp = s["cache"]
        slots, page = s["slots"], case["page"]
        live = slots >= 0
        at, row = slots[live] // page, slots[live] % page
        for values, codes, exps in ((k, k_codes, k_exp), (s["v"].float(), v_codes, v_exp)):
            c, e = _encode(values[live], case["mode"])
            codes[at, :, row] = _pack(c)
            exps[at, :, :, row] = e
        return (q, *(_rows(codes, exps, slots, page) for codes, exps in ((k_codes, k_exp), (v_codes, v_exp))))
    return _attend(s, case)


def _norm_rotate(x, weight, s, case):
    """x [tokens, heads, head_dim] in the precision of the work."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    half = case["rot"] // 2
    cs = s["cos_sin"][s["positions"]].to(x.dtype)[:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., :half], r[..., half:])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if case["interleaved"] else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _encode(x, mode):
    """fp32 [.., n] -> codes uint8 [.., n] and exponent bytes uint8 [.., n / 32]: the exponent that puts a block's
    largest magnitude in [4, 8) (ocp) or in (3, 6] (noclip), codes to the nearest of the grid, ties to the even one."""
    b = x.unflatten(-1, (-1, 32))
    most = b.abs().amax(-1)
    m, e = torch.frexp(most.clamp_min(2.0 ** -126))  # most = m 2^e, m in [0.5, 1)
    e = e - 3
    if mode == "noclip":
        e = e + (m > 0.75)
    e = torch.where(most > 0, e, 0).clamp(-127, 127)
    a = (b * torch.exp2(-e.float())[..., None]).abs()
    up = torch.zeros(a.shape, dtype=torch.uint8, device=a.device)
    for i, mid in enumerate(MIDPOINTS):  # a tie goes to the even one of codes i and i + 1
        up += (a > mid) if i % 2 == 0 else (a >= mid)
    codes = torch.where((b < 0) & (up > 0), up | 8, up)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _values(codes, exps):
    """codes [.., n / 2] and exponent bytes [.., n / 32] -> fp32 [.., n]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    x = grid[pair].unflatten(-1, (-1, 32))
    return torch.ldexp(x, exps.int()[..., None] - 127).flatten(-2)


def _rows(codes, exps, slots, page):
    """The cache's rows at `slots` as bf16 [tokens, heads, head_dim] (every value is exact in it); zeros where < 0."""
    at = slots.clamp_min(0)
    x = _values(codes[at // page, :, at % page], exps[at // page, :, :, at % page])
    return torch.where((slots >= 0)[:, None, None], x, 0.0).to(torch.bfloat16)


def _attend(s, case):
    k_codes, k_exp, v_codes, v_exp = s["cache"]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    table = s["block_table"].long()
    n, ctx = table.shape[0], s["context_lens"].long()
    keys, values = (
        _values(c[table].transpose(1, 2).flatten(2, 3), e[table].permute(0, 2, 1, 4, 3).flatten(2, 3))
        for c, e in ((k_codes, k_exp), (v_codes, v_exp)))                     # [n, hk, tokens, d]
    t, most = s["q"].shape[0], s["max_q"]
    cu = torch.arange(n + 1, device=table.device) if s["cu_q"] is None else s["cu_q"].long()
    token = torch.arange(t, device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    q = torch.zeros((n, most, hq, d), device=table.device)
    q[seq, token - cu[seq]] = s["q"].float()
    q = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, hk, group x most, d]
    scores = torch.matmul(q * s["scale"], keys.transpose(-1, -2).contiguous())
    at = torch.arange(keys.shape[2], device=table.device)
    pos = (ctx - (cu[1:] - cu[:-1]))[:, None] + torch.arange(most, device=table.device)
    seen = (at < ctx[:, None])[:, None]
    if case["causal"]:
        seen = seen & (at <= pos[..., None])
        if case["window"]:
            seen = seen & (at > pos[..., None] - case["window"])
    hidden = ~seen.expand(n, most, -1)[:, None, None]
    scores = scores.unflatten(2, (hq // hk, most)).masked_fill_(hidden, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), values).unflatten(2, (hq // hk, most)) / total.where(total > 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                                # [n, most, hq, d]
    return o[seq, token - cu[seq]].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_turned(s[n], s[n + "_weight"], s, case) for n in ("q", "k"))
    if case["op"] == "append":
        k = _exact_turned(s["k"], s["k_weight"], s, case).float().double()  # the cache encodes 32-bit values
        live = (s["slots"] >= 0).double()[:, None, None]
        return (_exact_turned(s["q"], s["q_weight"], s, case),
                *(_exact_cached(x, case["mode"]) * live for x in (k, s["v"].double())))
    return _exact_attention(s, case)


def _exact_turned(x, weight, s, case):
    """Each pair as a complex number times exp(i angle), the norm before it."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    r = case["rot"]
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    turn = s["cos_sin"].double()[s["positions"]]
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(turn[:, :r // 2], turn[:, r // 2:])[:, None]
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_cached(x, mode):
    """The value that each element of a 32-block is held as: the nearest grid point times 2^e, ties to the even code."""
    b = x.unflatten(-1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    safe = most.clamp_min(2.0 ** -126)
    e = torch.floor(torch.log2(safe))
    e = torch.where(torch.exp2(e) > safe, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= safe, e + 1, e) - 2
    if mode == "noclip":
        e = torch.where(safe > 6 * torch.exp2(e), e + 1, e)
    step = torch.exp2(torch.where(most > 0, e, 0.0).clamp(-127, 127))
    a = (b.abs() / step).clamp_max(6.0)
    near = torch.where(a < 2, (2 * a).round() / 2, torch.where(a < 4, a.round(), 2 * (a / 2).round()))
    return (near * step * b.sign()).flatten(-2)


def _exact_attention(s, case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    g, page = hq // hk, case["page"]
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    cache = s["cache"]
    if not isinstance(cache, tuple):
        cache = (cache.k_codes, cache.k_e8m0, cache.v_codes, cache.v_e8m0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(_lengths(case)):
        rows = s["q"][at:at + n].double()
        pages = s["block_table"][b, :-(-c // page)].long()
        pos = torch.arange(c - n, c, device="cuda")
        key = torch.arange(c, device="cuda")
        hidden = torch.zeros((n, c), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = key > pos[:, None]
            if case["window"]:
                hidden |= key <= pos[:, None] - case["window"]
        for h in range(hk if c else 0):
            kv = []
            for codes, exps in (cache[:2], cache[2:]):
                low, high = codes[pages, h] & 15, codes[pages, h] >> 4
                code = torch.stack([low, high], -1).reshape(-1, d)[:c].long()
                e = exps[pages, h].transpose(1, 2).reshape(-1, d // 32)[:c].double() - 127
                kv.append(grid[code % 8] * (1 - 2 * (code // 8)) * torch.exp2(e).repeat_interleave(32, 1))
            step = max(1, (1 << 28) // (g * c))  # rows at a time, so that the scores stay near 2 GB
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                q = rows[lo:hi, h * g:(h + 1) * g].reshape(-1, d)
                x = (q @ kv[0].T.contiguous() * s["scale"]).reshape(-1, g, c)
                x = x.masked_fill_(hidden[lo:hi, None], -math.inf)
                x = torch.exp(x - x.amax(-1, keepdim=True))
                o = (x.reshape(-1, c) @ kv[1]).reshape(-1, g, d) / x.sum(-1, keepdim=True)
                out[at + lo:at + hi, h * g:(h + 1) * g] = o
        at += n
    return out
