"""A model's expert block with block-scaled 8-bit weights, from fp32 weights to a prompt and a decoded token.

    python examples/blk_layer.py

The steps of a program that uses it: the weights are quantised once on the GPU; then, for each layer, moe_rmsnorm adds the
last result to the residual stream and writes its norm twice, in bf16 for the router and in 8 bits for the experts;
moe_router_logits and moe_blk_layer (routing, experts, sum) follow.  The same calls serve the prompt and the token after
it.  Prints how far the block is from fp32 weights and activations, and the times.  Needs a GPU and the built library.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_moe_expert_gb300 as bm  # noqa: E402

D, I, E, K, SHARED = 1024, 256, 64, 6, 256  # widths, experts, experts per token, the shared expert's width
GROUPS, KEPT, EPS = 8, 4, 1e-6


def experts(g, n, width):
    def draw(rows, cols):
        return torch.randn(n, rows, cols, generator=g, device="cuda") / math.sqrt(cols)

    def quantise(w):
        m = bm.BlkMat.empty(*w.shape)
        bm.moe_blk_quantize_weights(w, m)
        return m

    w = {"gate": draw(width, D), "up": draw(width, D), "down": draw(D, width)}
    return w, bm.BlkExperts(**{name: quantise(m) for name, m in w.items()})


class Block:
    """The block's weights and, for one number of tokens, the buffers of a call."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.routed_fp32, self.routed = experts(g, E, I)
        self.shared_fp32, self.shared = experts(g, 1, SHARED)
        self.gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        self.router = (torch.randn(E, D, generator=g, device="cuda") / math.sqrt(D)).to(torch.bfloat16)
        bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.scoring = bm.Scoring("sigmoid", bias, n_group=GROUPS, topk_group=KEPT, scale=1.5)

    def buffers(self, T):
        rows = 16 if T * K < 16 * E else 64  # tile height: about the rows of an expert
        return {"rows": rows, "normed": torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), "act": bm.BlkAct.empty(T, D),
                "logits": torch.empty(T, E, device="cuda"), "routing": bm.Routing.empty(T, E, K, rows),
                "y": torch.empty(T, D, dtype=torch.bfloat16, device="cuda"),
                "ws": bm.workspace(bm.moe_blk_layer_workspace_bytes(T, D, I, E, K, SHARED, rows))}

    def __call__(self, x, stream, b):
        """x is added to the residual stream, in place; the experts' sum comes back."""
        bm.moe_rmsnorm(x, self.gamma, EPS, residual=stream, Y=b["normed"], out=b["act"])
        bm.moe_router_logits(b["normed"], self.router, b["logits"])
        bm.moe_blk_layer(b["logits"], self.scoring, b["act"], self.routed, self.shared, K, b["rows"], b["routing"], b["y"],
                         b["ws"])
        return b["y"]

    def fp32(self, stream, routing):
        """The same experts without any quantisation, from the stream after the addition."""
        def ffn(w, e, rows):
            h = torch.nn.functional.silu(rows @ w["gate"][e].t()) * (rows @ w["up"][e].t())
            return h @ w["down"][e].t()

        x = stream.float()
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * self.gamma.float()
        y = ffn(self.shared_fp32, 0, x)
        for e in range(E):
            t, j = torch.nonzero(routing.ids == e, as_tuple=True)
            if len(t):
                y.index_add_(0, t, routing.w[t, j][:, None] * ffn(self.routed_fp32, e, x[t]))
        return y


def timed(f, n=50):
    f()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    stop.record()
    stop.synchronize()
    return start.elapsed_time(stop) / n * 1e3


def main():
    block = Block()
    result = {}
    for T in (512, 1):
        x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
        stream = (3 * torch.randn(T, D, device="cuda")).to(torch.bfloat16)
        b = block.buffers(T)
        y = block(x, stream, b).float()
        ref = block.fp32(stream, b["routing"])
        status = bm.moe_check_status(b["ws"])
        if status:
            raise RuntimeError(bm.moe_status_string(status))
        result[T] = float((y - ref).norm() / ref.norm())
        zeros = torch.zeros_like(x)
        print(f"{T} tokens: {timed(lambda: block(zeros, stream, b)):.1f} us a block; relative distance from fp32 {result[T]:.3f}")
    return result


if __name__ == "__main__":
    main()
