"""One attention layer served from MXFP4: W4A8 projections around the attention block on
the 4-bit paged cache.

    python examples/attention_layer.py

takes two prompts, then decodes a token at a time with the step captured in a HIP graph,
and compares the attention's outputs with a plain computation on the cache's contents.
A layer's four calls: the merged q/k/v projection, the append (norms, rotation and MXFP4
encoding on the way; the queries normed and turned in the same launch), the attention, the
output projection."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a8_gemm_amd as w4  # noqa: E402


class AttentionLayer:
    def __init__(self, hidden, q_heads, kv_heads, head_dim, rot, max_positions, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=gen, device=device)

        self.hq, self.hk, self.d = q_heads, kv_heads, head_dim
        self.qkv = self._weight(normal((q_heads + 2 * kv_heads) * head_dim, hidden) * hidden ** -0.5)
        self.out = self._weight(normal(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5)
        self.q_norm, self.k_norm = 1 + 0.1 * normal(head_dim), 1 + 0.1 * normal(head_dim)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
        angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    @staticmethod
    def _weight(w):
        return w4.quant_bf16_to_mxfp4_prepared(w.to(torch.bfloat16).contiguous())

    def project(self, x):
        """Rows of q, k and v side by side -> views [tokens, heads, head_dim] of them."""
        rows = w4.mxfp4_linear_prepared(x, self.qkv)[0].unflatten(1, (-1, self.d))
        return rows[:, :self.hq], rows[:, self.hq:self.hq + self.hk], rows[:, self.hq + self.hk:]

    def attend(self, x, cache, batch, workspace=None):
        """(turned queries, attention outputs) [tokens, q_heads, head_dim]; the tokens' keys
        and values are in the cache afterwards."""
        q, k, v = self.project(x)
        q = w4.kv_append_mxfp4(cache, k, v, batch["slots"], cos_sin=self.cos_sin, positions=batch["positions"],
                               k_weight=self.k_norm, q=q, q_weight=self.q_norm)
        return q, w4.attention_mxfp4(q, cache, batch["block_table"], batch["context_lens"], cu_q=batch.get("cu_q"),
                                     max_q=batch["max_q"], workspace=workspace)

    def forward(self, x, cache, batch, workspace=None):
        return w4.mxfp4_linear_prepared(self.attend(x, cache, batch, workspace)[1].flatten(1), self.out)[0]


def batch_of(lengths, table, page):
    """What a call needs for sequences of (new tokens, context with them), on the GPU."""
    positions = torch.cat([torch.arange(c - n, c) for n, c in lengths])
    seq = torch.cat([torch.full((n,), i) for i, (n, _) in enumerate(lengths)])
    slots = table.cpu()[seq, positions // page].long() * page + positions % page
    new = torch.tensor([n for n, _ in lengths])
    batch = dict(positions=positions.cuda(), slots=slots.cuda(), block_table=table, max_q=int(new.max()),
                 context_lens=torch.tensor([c for _, c in lengths], dtype=torch.int32).cuda())
    if batch["max_q"] > 1:
        batch["cu_q"] = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]).int().cuda()
    return batch


def plain(q, cache, table, lengths):
    """Attention of the same queries over the cache's contents, in 64 bits."""
    out, at = torch.empty(q.shape, dtype=torch.float64, device=q.device), 0
    for s, (n, c) in enumerate(lengths):
        i = torch.arange(c, device=q.device)
        slots = table[s].long()[i // cache.page] * cache.page + i % cache.page
        k, v = (x.double().repeat_interleave(q.shape[1] // cache.kv_heads, 1) for x in w4.kv_read_mxfp4(cache, slots))
        x = (q[at:at + n].double()[:, :, None] * k.transpose(0, 1)).sum(-1) * cache.head_dim ** -0.5    # [n, heads, c]
        x = x.masked_fill(i > torch.arange(c - n, c, device=q.device)[:, None, None], float("-inf")).softmax(-1)
        out[at:at + n] = (x[..., None] * v.transpose(0, 1)).sum(2)
        at += n
    return out


def main(hidden=512, q_heads=6, kv_heads=1, head_dim=256, rot=64, page=16, prompts=(37, 21), steps=4):
    """The largest relative (Frobenius) difference of the attention from the plain computation."""
    most = max(prompts) + steps
    layer = AttentionLayer(hidden, q_heads, kv_heads, head_dim, rot, most)
    width = -(-most // page)
    cache = w4.KVCacheMXFP4.empty(len(prompts) * width, kv_heads, head_dim, page)
    table = torch.randperm(len(prompts) * width).view(len(prompts), width).int().cuda()
    workspace = w4.AttentionWorkspace(len(prompts), max(prompts), q_heads, kv_heads, head_dim)
    worst = 0.0

    def compare(q, got, lengths):
        nonlocal worst
        want = plain(q, cache, table, lengths)
        worst = max(worst, float((got.double() - want).norm() / want.norm()))

    lengths = [(n, n) for n in prompts]
    x = torch.randn(sum(prompts), hidden, device="cuda").to(torch.bfloat16)
    compare(*layer.attend(x, cache, batch_of(lengths, table, page), workspace), lengths)

    # one token of each sequence: a step's inputs change in place, its launches are one graph
    x = x[:len(prompts)].clone()
    lengths = [(1, n + 1) for n in prompts]
    step = batch_of(lengths, table, page)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, cache, step, workspace)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o = layer.attend(x, cache, step, workspace)
        y = w4.mxfp4_linear_prepared(o.flatten(1), layer.out)[0]
    for i in range(steps):
        lengths = [(1, n + 1 + i) for n in prompts]
        for name, value in batch_of(lengths, table, page).items():
            if torch.is_tensor(value):
                step[name].copy_(value)
        graph.replay()
        compare(q, o, lengths)
        x.copy_(y)
    return worst


if __name__ == "__main__":
    print(f"attention against the plain computation: relative difference {main():.2e}")
