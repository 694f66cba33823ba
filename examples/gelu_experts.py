"""Training steps of a mixture of biased GELU experts, put together from the library's operators.

    router logits   Linear (fp32 out)            -> mok_route_topk, mok_build_schedule
    sort            TokenSort.build, dispatch
    experts         Linear per expert (bias, GELU), Linear per expert (bias)
    back            TokenSort.combine with the routing weights, plus the residual
    gradients       the same operators in reverse
    update          AdamW over every weight and bias

Run it on a GPU: python examples/gelu_experts.py [--steps N] [--eight-bit] [--graph]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_deterministic_gb300 import binding as B  # noqa: E402
from mixture_experts_layer_deterministic_gb300.buffers import (  # noqa: E402
    AdamW, Linear, MoELayer, TokenSort)


class GeluExperts:
    """y = x + sum_k w[t,k] (W2[e] gelu(W1[e] x + b1[e]) + b2[e]), e the k-th expert of token t."""

    def __init__(self, T, H, I, E, K, capacity=0, seed=0, lr=1e-3, eight_bit=False,
                 capturable=False):
        gen = torch.Generator("cuda").manual_seed(seed)
        bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
        self.T, self.H, self.I, self.E, self.K = T, H, I, E, K
        self.route = MoELayer(T, H, I, E, K)
        self.sort = TokenSort(T, K, E, H, capacity=capacity)
        n = self.sort.n_rows
        self.gate = Linear(T, H, E, out_dtype=torch.float32)
        self.up = Linear(n, H, I, groups=E, act=B.MOK_ACT_GELU_TANH)
        self.down = Linear(n, I, H, groups=E)
        shapes = dict(gate=(1, E, H), w1=(E, I, H), w2=(E, H, I), b1=(E, I), b2=(E, H))
        self.p, self.w, self.g = {}, {}, {}
        for k, s in shapes.items():
            std = 0.0 if k[0] == "b" else s[-1] ** -0.5
            self.p[k] = torch.randn(*s, generator=gen, **f32) * std      # fp32 masters
            # biases are used in fp32; matrices through their bf16 copies
            self.w[k] = self.p[k] if k[0] == "b" else self.p[k].to(torch.bfloat16)
            self.g[k] = torch.zeros_like(self.w[k])
        self.opt = AdamW([dict(p=self.p[k], g=self.g[k],
                               copy=None if k[0] == "b" else self.w[k],
                               weight_decay=0.0 if k[0] == "b" else 0.01) for k in shapes],
                         lr=lr, eight_bit=eight_bit, capturable=capturable)
        self.logits = torch.zeros(T, E, **f32)
        self.y, self.dx = torch.zeros(T, H, **bf), torch.zeros(T, H, **bf)
        self.dx_gate = torch.zeros(T, H, **bf)
        self.d_topk_w, self.d_logits = torch.zeros(T, K, **f32), torch.zeros(T, E, **f32)
        r = self.sort.rows
        self.xs, self.out, self.dout, self.dxs = r(), r(), r(), r()
        self.z, self.h, self.dh = r(I), r(I), r(I)

    def forward(self, x):
        self.gate.forward(x, self.w["gate"], self.logits)
        idx, self.topk_w = self.route.route(self.logits)
        self.sort.build(idx, self.route.schedule())
        self.sort.dispatch(x, self.xs)
        self.up.forward(self.xs, self.w["w1"], self.h, bias=self.w["b1"], z=self.z,
                        sort=self.sort)
        self.down.forward(self.h, self.w["w2"], self.out, bias=self.w["b2"], sort=self.sort)
        return self.sort.combine(self.out, self.topk_w, self.y, residual=x)

    def backward(self, x, dy):
        """Gradients of every weight into self.g, of x (the residual's among them) returned."""
        self.sort.combine_backward(dy, self.out, self.topk_w, self.dout, self.d_topk_w)
        self.down.backward(self.h, self.w["w2"], self.dout, dx=self.dh, dw=self.g["w2"],
                           db=self.g["b2"], sort=self.sort)
        self.up.backward(self.xs, self.w["w1"], self.dh, z=self.z, dx=self.dxs,
                         dw=self.g["w1"], db=self.g["b1"], sort=self.sort)
        self.sort.dispatch_backward(self.dxs, self.dx)
        # the softmax over the chosen logits: dl_k = w_k (dw_k - sum_j w_j dw_j)
        w = self.topk_w.view(self.T, self.K)
        dl = w * (self.d_topk_w - (w * self.d_topk_w).sum(1, keepdim=True))
        self.d_logits.zero_().scatter_(1, self.route.idx.view(self.T, self.K).long(), dl)
        self.gate.backward(x, self.w["gate"], self.d_logits, dx=self.dx_gate, dw=self.g["gate"])
        return self.dx + self.dx_gate + dy

    def step(self, x, target):
        """One training step on the mean squared error; returns the loss (a device scalar)."""
        diff = self.forward(x).float() - target
        loss = diff.square().mean()
        self.backward(x, (diff * (2.0 / diff.numel())).to(torch.bfloat16))
        self.opt.step()
        return loss

    def capture(self, x, target):
        """A training step as a graph to replay (of a `capturable` model, after a first step): the
        graph, and the loss that each replay writes."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss = self.step(x, target)
        return graph, loss


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--eight-bit", action="store_true", help="MXFP8 optimizer states")
    ap.add_argument("--graph", action="store_true", help="replay the steps from a CUDA graph")
    a = ap.parse_args()
    torch.manual_seed(0)
    m = GeluExperts(T=1024, H=512, I=1024, E=8, K=2, eight_bit=a.eight_bit, capturable=a.graph)
    x = torch.randn(1024, 512, device="cuda").to(torch.bfloat16)
    target = x.float() + 0.5 * torch.tanh(x.float().roll(1, 1))
    graph = None
    for k in range(a.steps):
        if graph is not None:
            graph.replay()
        else:
            loss = m.step(x, target)
        if k % 10 == 0 or k == a.steps - 1:
            print("step %3d  loss %.5f" % (k, loss.item()))
        if a.graph and graph is None:
            graph, loss = m.capture(x, target)
    print("device status:", B.status_string(B.mok_read_device_status()[1]))


if __name__ == "__main__":
    main()
