"""The operators together, as a training step of a language model's last block runs them: norm, router
logits, router, experts, norm of the residual sum, loss over the vocabulary, and all of it backwards,
then the balance bias and AdamW. Against the same model in 64 bits by automatic differentiation, and
replayed from a graph.

Tolerances: values pass through bf16 on their way (y, the experts' h and slots, m, h2, y2, and every
gradient likewise), each time 2^-8 of a value, independent from element to element: a few times 2^-8 of
the whole in norm, as many as there are roundings between. The loss sums over the vocabulary what its
rows pick up, so its own error is that of y2, 5 roundings, times its gradient's norm."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B
from mixture_experts_layer_deterministic_gb300.buffers import (AdamW, Linear, MoELayer, Norm, Router,
                                                               VocabLoss)

pytestmark = pytest.mark.gpu
RATE, Z, SCALE = 1e-2, 1e-3, 2.0


def _t():
    import torch
    return torch


class Block:
    """h2 = r + experts(norm(r)); loss of norm(h2) over the vocabulary."""

    def __init__(self, T=96, H=256, I=128, E=16, K=4, V=1000, kind=B.MOK_NORM_RMS, seed=0,
                 capturable=False):
        torch = _t()
        gen = torch.Generator("cuda").manual_seed(seed)
        self.T, self.H, self.E, self.K, self.V, self.layer = T, H, E, K, V, kind == B.MOK_NORM_LAYER
        bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
        self.moe = MoELayer(T, H, I, E, K, backward=True)
        self.gate = Linear(T, H, E, out_dtype=torch.float32)
        self.route = Router(T, E, K, score=B.MOK_SCORE_SIGMOID, groups=4, topk_groups=2, group_top=2,
                            scale=SCALE)
        self.norm = [Norm(T, H, kind) for _ in range(2)]
        self.head = VocabLoss(T, H, V, z_loss=Z)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=gen, **f32) * std  # noqa: E731
        self.master = dict(gate=rand(1, E, H, std=H ** -0.5), w13=rand(E, 2 * I, H, std=H ** -0.5),
                           w2=rand(E, H, I, std=I ** -0.5), head=rand(V, H, std=2 * H ** -0.5),
                           n0=1 + rand(H, std=0.1), n1=1 + rand(H, std=0.1))
        self.w = {k: v if k[0] == "n" else v.to(torch.bfloat16) for k, v in self.master.items()}
        self.g = {k: torch.zeros_like(v) for k, v in self.w.items()}
        self.opt = AdamW([dict(p=self.master[k], g=self.g[k], copy=None if k[0] == "n" else self.w[k])
                          for k in self.w], lr=1e-3, capturable=capturable)
        self.bias = rand(E, std=0.05)
        self.counts = torch.zeros(E, dtype=torch.int32, device="cuda")
        row = lambda *s: torch.zeros(*s, **bf)  # noqa: E731
        vec = lambda: torch.zeros(T, **f32)  # noqa: E731
        for k in ("y", "m", "h2", "y2", "dy2", "dh2", "dy", "dy_gate", "dr"):
            setattr(self, k, row(T, H))
        self.pre = row(T * K, 2 * I)
        self.logits, self.dlogits = torch.zeros(T, E, **f32), torch.zeros(T, E, **f32)
        self.dw = torch.zeros(T, K, **f32)
        self.mean, self.rstd = [vec(), vec()], [vec(), vec()]
        self.loss, self.lse = vec(), vec()

    def forward(self, r, targets):
        stat = lambda i: dict(mean=self.mean[i] if self.layer else None, rstd=self.rstd[i])  # noqa: E731
        self.norm[0].forward(r, self.w["n0"], self.y, **stat(0))
        self.gate.forward(self.y, self.w["gate"], self.logits)
        self.route.forward(self.logits, self.moe.idx, self.moe.w, bias=self.bias, counts=self.counts)
        self.moe.schedule()
        self.moe.forward(self.y, self.w["w13"], self.w["w2"], self.m, saved_preact=self.pre)
        self.norm[1].forward(self.m, self.w["n1"], self.y2, residual=r, h=self.h2, **stat(1))
        return self.head.forward(self.y2, self.w["head"], targets, self.loss, self.lse)

    def backward(self, r, targets, d_loss):
        g, stat = self.g, lambda i: dict(mean=self.mean[i] if self.layer else None)
        self.head.backward(self.y2, self.w["head"], targets, self.lse, d_loss, dx=self.dy2, dw=g["head"])
        self.norm[1].backward(self.h2, self.w["n1"], self.dy2, self.rstd[1], dx=self.dh2, dw=g["n1"],
                              **stat(1))
        self.moe.backward(self.y, self.pre, self.w["w13"], self.w["w2"], self.dh2, self.dy, g["w13"],
                          g["w2"], self.dw)
        self.route.backward(self.logits, self.moe.idx, self.dw, self.dlogits)
        self.gate.backward(self.y, self.w["gate"], self.dlogits, dx=self.dy_gate, dw=g["gate"])
        self.dy.add_(self.dy_gate)
        self.norm[0].backward(r, self.w["n0"], self.dy, self.rstd[0], dh=self.dh2, dx=self.dr,
                              dw=g["n0"], **stat(0))
        return self.dr

    def step(self, r, targets, d_loss):
        self.forward(r, targets)
        self.backward(r, targets, d_loss)
        self.route.update_bias(self.counts, RATE, self.bias)
        self.opt.step()

    def reference(self, r, targets, d_loss):
        """Loss per row, and 64-bit leaves with their gradients, with the experts that were chosen."""
        torch = _t()
        p = {k: v.double().requires_grad_() for k, v in self.w.items()}
        x = r.double().requires_grad_()

        def norm(h, w):
            if self.layer:
                h = h - h.mean(1, keepdim=True)
            return h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w

        y = norm(x, p["n0"])
        idx = self.moe.idx.view(self.T, self.K).long()
        s = torch.sigmoid(y @ p["gate"][0].T).gather(1, idx)
        w = SCALE * s / s.sum(1, keepdim=True)
        h2 = x
        I = p["w2"].shape[2]
        for k in range(self.K):
            a = torch.einsum("th,tih->ti", y, p["w13"][idx[:, k]])
            o = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
            h2 = h2 + w[:, k:k + 1] * torch.einsum("ti,thi->th", o, p["w2"][idx[:, k]])
        l = norm(h2, p["n1"]) @ p["head"].T
        lse = torch.logsumexp(l, 1)
        hit = l.gather(1, targets.long().clamp(min=0)[:, None])[:, 0]
        loss = torch.where(targets >= 0, lse - hit + Z * lse * lse, 0.0)
        (loss * d_loss.double()).sum().backward()
        return loss.detach(), p, x

    def choice(self):
        """The choice of the router's definition in 64 bits, from the logits that it got."""
        torch = _t()
        s = torch.sigmoid(self.logits.double()) + self.bias.double()
        best = s.view(self.T, 4, -1).sort(dim=2, descending=True)[0][:, :, :2].sum(2)
        kept = torch.zeros(self.T, 4, device="cuda").scatter_(
            1, best.sort(dim=1, descending=True, stable=True)[1][:, :2], 1.0)
        s = torch.where(kept.repeat_interleave(self.E // 4, 1) > 0, s, -9.0)
        return s.sort(dim=1, descending=True, stable=True)[1][:, :self.K]


def inputs(m, seed):
    torch = _t()
    gen = torch.Generator("cuda").manual_seed(seed)
    r = (torch.randn(m.T, m.H, device="cuda", generator=gen) * 0.7).to(torch.bfloat16)
    targets = torch.randint(0, m.V, (m.T,), device="cuda", generator=gen, dtype=torch.int32)
    targets[::9] = -1
    d = (targets >= 0).float() / (targets >= 0).sum()
    return r, targets, d


@pytest.mark.parametrize("kind", [B.MOK_NORM_RMS, B.MOK_NORM_LAYER])
def test_loss_and_gradients(kind):
    torch = _t()
    m = Block(kind=kind, seed=3)
    r, targets, d = inputs(m, 1)
    loss = m.forward(r, targets).double()
    assert torch.equal(m.moe.idx.view(m.T, m.K).long(), m.choice())
    assert torch.equal(m.counts.long(), torch.bincount(m.moe.idx.long(), minlength=m.E))
    dr = m.backward(r, targets, d).double()
    assert B.mok_read_device_status()[1] == B.MOK_OK
    ref, p, x = m.reference(r, targets, d)
    u = 2.0 ** -8
    # |dl/dy2| <= 2 max |W_v|, so a row's loss moves by at most that times the error of y2
    slope = 2 * m.w["head"].double().norm(dim=1).max() * m.y2.double().norm(dim=1)
    assert bool(((loss - ref).abs() <= 5 * u * slope).all())
    rel = lambda a, b: float((a - b).norm() / b.norm())  # noqa: E731
    assert rel(dr, x.grad) <= 10 * u
    for k in m.g:
        assert rel(m.g[k].double(), p[k].grad) <= 10 * u, k


def test_step_replayed_from_a_graph_on_other_inputs():
    """Three steps by calls, and the same by one graph after a first call: the same bits."""
    torch = _t()
    ends = []
    for graphed in (False, True):
        m = Block(seed=5, capturable=True)
        held = [t.clone() for t in inputs(m, 0)]
        m.step(*held)
        if graphed:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                m.step(*held)
        losses = []
        for k in range(3):
            for t, new in zip(held, inputs(m, 10 + k)):
                t.copy_(new)
            if graphed:
                graph.replay()
            else:
                m.step(*held)
            losses.append(m.loss.clone())
        assert B.mok_read_device_status()[1] == B.MOK_OK
        ends.append((losses, m.bias.clone(), {k: v.clone() for k, v in m.master.items()}))
    for a, b in zip(ends[0][0], ends[1][0]):
        assert torch.equal(a, b)
    assert torch.equal(ends[0][1], ends[1][1])
    for k in ends[0][2]:
        assert torch.equal(ends[0][2][k], ends[1][2][k]), k


def test_two_host_threads():
    """Two threads with models, streams and workspaces of their own give what each gives alone."""
    import threading
    torch = _t()
    models = [Block(seed=s) for s in (1, 2)]
    data = [inputs(m, s) for s, m in enumerate(models)]
    want = []
    for m, (r, t, d) in zip(models, data):
        m.forward(r, t)
        m.backward(r, t, d)
        want.append((m.loss.clone(), m.dr.clone(), {k: v.clone() for k, v in m.g.items()}))
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                r, t, d = data[i]
                for _ in range(20):
                    models[i].forward(r, t)
                    models[i].backward(r, t, d)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed
    for m, (loss, dr, g) in zip(models, want):
        assert torch.equal(m.loss, loss) and torch.equal(m.dr, dr)
        for k in g:
            assert torch.equal(m.g[k], g[k]), k
    assert B.mok_read_device_status()[1] == B.MOK_OK


@pytest.mark.parametrize("op", ["router", "norm", "loss"])
def test_operators_replayed_on_other_inputs(op):
    """Each operator alone, captured once and replayed on other inputs, against calls."""
    torch = _t()
    import test_gpu_norm
    import test_gpu_router
    import test_gpu_vocab_loss
    if op == "router":
        make = lambda s: test_gpu_router.Case(T=600, E=64, K=6, score="sigmoid", G=4, keep=2, top=2,  # noqa: E731
                                              bias=True, seed=s)
        swap = ("buf", "bias")

        def run(c):
            out = c.forward()
            d = torch.ones(600, 6, device="cuda")
            g = torch.zeros_like(c.buf)
            B.check(B.mok_router_backward(c.cfg, c.buf, out[0], d, None, g))
            return (*out, g)
    elif op == "norm":
        make = lambda s: test_gpu_norm.Case(R=300, H=9000, seed=s)  # noqa: E731
        swap = ("x", "res", "w", "b")

        def run(c):
            h, y, mean, rstd = c.forward()
            return (h, y, mean, rstd, *c.backward(h, mean, rstd, y, c.x))
    else:
        make = lambda s: test_gpu_vocab_loss.Case(R=200, H=96, V=900, piece=512, seed=s)  # noqa: E731
        swap = ("x", "w", "t", "d")

        def run(c):
            loss, lse = c.forward()
            return (loss, lse, *c.backward(lse))
    c, other = make(0), make(1)
    want = [t.clone() for t in run(other)]
    run(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(c)
    for k in swap:
        getattr(c, k).copy_(getattr(other, k))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert B.mok_read_device_status()[1] == B.MOK_OK
