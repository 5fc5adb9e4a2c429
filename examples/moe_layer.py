"""The expert half of a decoder layer served from MXFP4: norms, the choice of experts and their
gated products.

    python examples/moe_layer.py

takes a prompt's tokens, then decodes a few steps for a batch of sequences with the step
captured in a HIP graph, and compares the block's outputs with a plain computation on the
same weights and activations.  A block's four calls beside the router's own product: the
residual sum with its norm (values for the router, fp8 codes for the experts in the same
pass), the choice of each token's experts, the experts, the residual sum with the norms
behind the block and before the next."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a8_gemm_amd as w4  # noqa: E402


class ExpertBlock:
    def __init__(self, hidden, inter, experts, top_k, max_tokens, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=gen, device=device)

        self.top_k = top_k
        up = w4.quant_bf16_to_mxfp4((normal(experts * 2 * inter, hidden) * hidden ** -0.5).to(torch.bfloat16))
        down = w4.quant_bf16_to_mxfp4((normal(experts * hidden, inter) * inter ** -0.5).to(torch.bfloat16))
        self.experts = w4.ExpertsMXFP4.prepare(*up, *down, experts=experts)
        self.rows = [values(*w).unflatten(0, (experts, -1)) for w in (up, down)]   # for the plain computation
        self.router = normal(hidden, experts) * hidden ** -0.5
        self.norms = [1 + 0.1 * normal(hidden) for _ in range(3)]
        self.workspace = w4.MoEWorkspace(max_tokens, top_k, experts, hidden, inter)

    def forward(self, y, residual):
        """An attention's output and the residual before it -> the new residual, the next linear's fp8 activations
        with their scales, and what the plain computation compares."""
        r, h, x, s = w4.residual_norm(y, residual, weight=self.norms[0], fp8=True)
        logits = h.float() @ self.router
        weights, ids = w4.moe_route(logits, self.top_k)
        o = w4.moe_mxfp4(x, s, ids, weights, self.experts, workspace=self.workspace)
        r, _, x2, s2 = w4.residual_norm(o, r, weight=self.norms[2], post_weight=self.norms[1], values=False, fp8=True)
        return r, x2, s2, (logits, x, s, o)

    def plain(self, logits, x, s):
        """The experts' outputs of the same logits and activations, in 64 bits."""
        x = x.view(torch.float8_e4m3fn).double() * s.double()[:, None]
        weights, ids = logits.double().softmax(1).topk(self.top_k)
        weights = weights / weights.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        for e in range(self.experts.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            gate, up = (x[t] @ self.rows[0][e].T).chunk(2, 1)
            out.index_add_(0, t, weights[t, j, None] * (gate * gate.sigmoid() * up @ self.rows[1][e].T))
        return out


def values(packed, exponents):
    """Row-major MXFP4 codes and exponents in 64 bits."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=packed.device)
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(1).long()
    size = torch.exp2(exponents.double() - 127).repeat_interleave(32, 1)
    return grid[codes % 8] * (1 - 2 * (codes // 8)) * size


def main(hidden=512, inter=256, experts=16, top_k=4, prompt=75, batch=3, steps=4):
    """The largest relative (Frobenius) difference of the experts' outputs from the plain computation."""
    block = ExpertBlock(hidden, inter, experts, top_k, max(prompt, batch))
    worst = 0.0

    def compare(logits, x, s, o):
        nonlocal worst
        want = block.plain(logits, x, s)
        worst = max(worst, float((o.double() - want).norm() / want.norm()))

    def tokens(n):
        return [torch.randn(n, hidden, device="cuda").to(torch.bfloat16) for _ in range(2)]

    compare(*block.forward(*tokens(prompt))[3])

    # one token of each sequence: a step's inputs change in place, its launches are one graph
    y, residual = tokens(batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(y, residual)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, _, _, seen = block.forward(y, residual)
    for _ in range(steps):
        graph.replay()
        compare(*seen)
        y.copy_(torch.randn_like(y))   # the next layer's attention would stand here
        residual.copy_(r)
    return worst


if __name__ == "__main__":
    print(f"experts against the plain computation: relative difference {main():.2e}")
