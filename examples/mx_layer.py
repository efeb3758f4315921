"""An expert layer with MXFP4 weights, from fp32 weights to a prompt and a decoded token.

    python examples/mx_layer.py

The steps of a program that uses the layer: the weights are quantised once on the GPU; a router with a balance bias and
expert groups scores the tokens (moe_router_logits, then moe_mx_layer: routing, quantised activations, experts, sum); the
same call serves the prompt and the token after it.  Prints how far the layer is from fp32 weights and activations, and the
times.  Needs a GPU and the built library.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_moe_expert_gb300 as bm  # noqa: E402

D, I, E, K, SHARED = 1024, 256, 64, 6, 256  # widths, experts, experts per token, the shared expert's width
GROUPS, KEPT = 8, 4


def quantise(w):
    """fp32 [E][N][K] -> MxMat.  N is a multiple of 128 here, so the stack is one matrix of E * N rows."""
    n, rows, cols = w.shape
    m = bm.MxMat.empty(1, n * rows, cols)
    bm.moe_mx_quantize(w.reshape(n * rows, cols), m)
    return bm.MxMat(m.q.view(n, rows, cols // 2), m.sp.view(n, rows // 128, cols // 128, 512))


def experts(g, n, width):
    def draw(rows, cols):
        return torch.randn(n, rows, cols, generator=g, device="cuda") / math.sqrt(cols)

    w = {"gate": draw(width, D), "up": draw(width, D), "down": draw(D, width)}
    return w, bm.MxExperts(**{name: quantise(m) for name, m in w.items()})


class Layer:
    """The layer's weights and, for one number of tokens, the buffers of a call."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.routed_fp32, self.routed = experts(g, E, I)
        self.shared_fp32, self.shared = experts(g, 1, SHARED)
        self.router = (torch.randn(E, D, generator=g, device="cuda") / math.sqrt(D)).to(torch.bfloat16)
        bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.scoring = bm.Scoring("sigmoid", bias, n_group=GROUPS, topk_group=KEPT, scale=1.5)

    def buffers(self, T):
        rows = 16 if T * K < 16 * E else 64  # tile height: about the rows of an expert
        return {"rows": rows, "logits": torch.empty(T, E, device="cuda"), "routing": bm.Routing.empty(T, E, K, rows),
                "y": torch.empty(T, D, dtype=torch.bfloat16, device="cuda"),
                "ws": bm.workspace(bm.moe_mx_layer_workspace_bytes(T, D, I, E, K, SHARED, rows))}

    def __call__(self, x, b):
        bm.moe_router_logits(x, self.router, b["logits"])
        bm.moe_mx_layer(b["logits"], self.scoring, x, self.routed, self.shared, K, b["rows"], b["routing"], b["y"], b["ws"])
        return b["y"]

    def fp32(self, x, routing):
        """The same experts without any quantisation."""
        def ffn(w, e, rows):
            h = torch.nn.functional.silu(rows @ w["gate"][e].t()) * (rows @ w["up"][e].t())
            return h @ w["down"][e].t()

        x = x.float()
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
    layer = Layer()
    result = {}
    for T in (512, 1):
        x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
        b = layer.buffers(T)
        y = layer(x, b).float()
        ref = layer.fp32(x, b["routing"])
        status = bm.moe_check_status(b["ws"])
        if status:
            raise RuntimeError(bm.moe_status_string(status))
        result[T] = float((y - ref).norm() / ref.norm())
        print(f"{T} tokens: {timed(lambda: layer(x, b)):.1f} us a layer; relative distance from fp32 {result[T]:.3f}")
    return result


if __name__ == "__main__":
    main()
