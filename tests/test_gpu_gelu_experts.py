"""The example that runs the operators together: its output and gradients against the same model in
64 bits by automatic differentiation, and training steps that learn."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def model(**kw):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from gelu_experts import GeluExperts
    finally:
        sys.path.pop(0)
    return GeluExperts(**kw)


def reference(m, x):
    """(y, parameters and x as 64-bit leaves) with the routing the library chose."""
    import torch
    p = {k: m.w[k].double().requires_grad_() for k in m.w}
    xd = x.double().requires_grad_()
    idx = m.route.idx.view(m.T, m.K).long()
    w = torch.softmax(torch.gather(xd @ p["gate"][0].T, 1, idx), 1)
    kept = (m.sort.map.view(m.T, m.K) >= 0).double()
    y = xd
    for k in range(m.K):
        e = idx[:, k]
        h = torch.einsum("th,tih->ti", xd, p["w1"][e]) + p["b1"][e]
        h = torch.nn.functional.gelu(h, approximate="tanh")
        o = torch.einsum("ti,thi->th", h, p["w2"][e]) + p["b2"][e]
        y = y + (w[:, k] * kept[:, k])[:, None] * o
    return y, p, xd


@pytest.mark.parametrize("capacity", [0, 20])
def test_output_and_gradients(capacity):
    import torch
    m = model(T=96, H=128, I=256, E=8, K=2, capacity=capacity, seed=3)
    gen = torch.Generator("cuda").manual_seed(1)
    for k in ("b1", "b2"):
        m.p[k].normal_(0, 0.3, generator=gen)
    x = torch.randn(96, 128, device="cuda", generator=gen).to(torch.bfloat16)
    dy = torch.randn(96, 128, device="cuda", generator=gen).to(torch.bfloat16)
    y = m.forward(x).double()
    dx = m.backward(x, dy).double()
    ref, p, xd = reference(m, x)
    ref.backward(dy.double())
    # h, out, y and every gradient pass through bf16 a few times on their way: each time 2^-8 of
    # a value, independent from element to element, so a few times 2^-8 of the whole in norm
    rel = lambda a, b: float((a - b).norm() / b.norm())  # noqa: E731
    assert rel(y, ref.detach()) <= 4 * 2.0 ** -8
    assert rel(dx, xd.grad) <= 6 * 2.0 ** -8
    for k in m.g:
        assert rel(m.g[k].double(), p[k].grad) <= 6 * 2.0 ** -8, k
    if capacity:
        assert int((m.sort.map < 0).sum()) > 0


@pytest.mark.parametrize("eight_bit", [False, True])
def test_steps_learn_and_repeat_bit_for_bit(eight_bit):
    import torch
    runs = []
    for _ in range(2):
        m = model(T=256, H=128, I=256, E=8, K=2, eight_bit=eight_bit, lr=2e-3)
        gen = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(256, 128, device="cuda", generator=gen).to(torch.bfloat16)
        target = x.float() + 0.5 * torch.tanh(x.float().roll(1, 1))
        losses = [m.step(x, target) for _ in range(30)]
        losses = torch.stack(losses).cpu().numpy()
        assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
        runs.append((losses, m.p["w1"].clone()))
    assert np.array_equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
