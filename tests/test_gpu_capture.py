"""The operators inside CUDA graphs: a replay gives what the calls give, and an optimizer step that
reads its number, lr and seed from the device moves with each replay.

Tolerances: test_gpu_adamw.py's, the scalars of a step being the same formulas in 64 bits."""
import numpy as np
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B
from test_gpu_adamw import LR, MODES, Tensors, check, config
from test_gpu_gelu_experts import model
from test_gpu_linear import Lin, device_ok
from test_gpu_rows import Case

pytestmark = pytest.mark.gpu
SEED, STRIDE = 0x123456789ABCDEF0, 3


def _t():
    import torch
    return torch


def clock(lr=LR, step=0):
    torch = _t()
    c = torch.zeros(B.ADAMW_CLOCK_WORDS, dtype=torch.int64, device="cuda")
    c[0], c[1] = step, STRIDE
    c.view(torch.float64)[2] = lr
    return c


@pytest.mark.parametrize("sr", [0, 1])
@pytest.mark.parametrize("p,g,state", MODES)
def test_step_at(p, g, state, sr):
    """Steps 1, 2 and 3 by the clock, each against the definition; 100 tensors are two launches."""
    sizes = [1, 7, 8, 31, 32, 33, 0, 100, 2047, 2048, 2049, 5000, 4096] + [50] * 87
    t = Tensors(sizes, p, g, state, copy=p == "fp32", seed=sr)
    lst, c, flags = t.list(), clock(), sr * B.MOK_ADAMW_STOCHASTIC
    cfg = config(t, 1, flags, SEED, lr=0.5)  # the clock's lr counts
    for step in (1, 2, 3):
        before = t.host()
        B.check(B.mok_adamw_advance(cfg, c))
        B.check(B.mok_adamw_step_at(cfg, lst, c, t.gs))
        check(before, t.host(), t, step, sr, SEED + STRIDE * step)
        t.guards_intact()
    assert c[:2].tolist() == [3, STRIDE] and device_ok()


def test_a_bad_clock_is_reported_and_moves_no_parameter():
    torch = _t()
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(step=-1)):
        t = Tensors([500])
        p0, c = t.t[0]["p"].clone(), clock(**kw)
        B.mok_clear_device_status()
        B.check(B.mok_adamw_advance(config(t), c))
        B.check(B.mok_adamw_step_at(config(t), t.list(), c, t.gs))
        assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()
        assert torch.equal(t.t[0]["p"], p0)


def test_clock_refusals():
    t, c = Tensors([64], "fp32", "bf16", "8bit"), clock()
    cfg, lst, bad = config(t), t.list(), B.MOK_ERR_INVALID_ARG
    assert B.mok_adamw_advance(cfg, None) == bad
    assert B.mok_adamw_advance(cfg, c.data_ptr() + 8) == bad
    assert B.mok_adamw_advance(config(t, beta1=1.0), c) == bad
    assert B.mok_adamw_advance(config(t, abi_version=1), c) == B.MOK_ERR_ABI
    assert B.mok_adamw_step_at(cfg, lst, None) == bad
    assert B.mok_adamw_step_at(cfg, lst, c.data_ptr() + 8) == bad
    assert B.mok_adamw_step_at(config(t, eps=-1.0), lst, c) == bad
    d = {k: v for k, v in t.t[0].items() if k != "first"}
    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        assert B.mok_adamw_step_at(cfg, B.make_adamw_list([dict(d, **{k: None})]), c) == bad
    assert B.mok_adamw_step_at(cfg, B.make_adamw_list([]), c) == B.MOK_OK
    assert c[0].item() == 0 and device_ok()


@pytest.mark.parametrize("eight_bit", [False, True])
def test_whole_training_step_replayed(eight_bit):
    """Steps of the example by calls, and the same ones with all but the first as replays of one
    graph: the same losses and weights bit for bit. A change of lr takes effect between replays."""
    torch = _t()
    runs = []
    for graphed in (False, True):
        m = model(T=256, H=128, I=256, E=8, K=2, eight_bit=eight_bit, lr=2e-3, capturable=True)
        gen = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(256, 128, device="cuda", generator=gen).to(torch.bfloat16)
        target = x.float() + 0.5 * torch.tanh(x.float().roll(1, 1))
        losses = [float(m.step(x, target))]
        if graphed:
            graph, loss = m.capture(x, target)
        for k in range(12):
            if k == 8:
                m.opt.set_lr(5e-4)
            if graphed:
                graph.replay()
            else:
                loss = m.step(x, target)
            losses.append(float(loss))
        assert m.opt.clock[0].item() == 13 and device_ok()
        runs.append((losses, {k: v.clone() for k, v in m.p.items()}))
    assert runs[0][0] == runs[1][0] and runs[0][0][-1] < 0.7 * runs[0][0][0]
    for k in runs[0][1]:
        assert torch.equal(runs[0][1][k], runs[1][1][k]), k


def test_steps_by_clock_are_the_steps_by_call():
    """The same numbers, seeds and rates, whoever counts: scalars may differ in their last bit."""
    torch = _t()
    ends = []
    for capturable in (False, True):
        m = model(T=256, H=128, I=256, E=8, K=2, lr=2e-3, capturable=capturable)
        gen = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(256, 128, device="cuda", generator=gen).to(torch.bfloat16)
        target = x.float() + 0.5 * torch.tanh(x.float().roll(1, 1))
        first = m.step(x, target)
        ends.append((float(first), {k: v.clone() for k, v in m.p.items()}))
    assert ends[0][0] == ends[1][0]
    for k in ends[0][1]:
        a, b = ends[0][1][k].double(), ends[1][1][k].double()
        # one step moves a weight by about lr; an ulp of the rate, and one of the weight
        assert bool(((a - b).abs() <= 2.0 ** -22 * 2e-3 + 2.0 ** -23 * a.abs()).all()), k


@pytest.mark.parametrize("kw", [dict(R=3, Kin=500, N=300, act="silu"),
                                dict(R=700, Kin=520, N=300, act="gelu_tanh", grad="fp32"),
                                dict(R=300, Kin=4096, N=60),
                                dict(G=5, counts=[1, 0, 300, 16, 257], Kin=200, N=136, act="silu")])
def test_linear_replayed_on_other_inputs(kw):
    torch = _t()
    c, other = Lin(z=True, **kw), Lin(z=True, seed=1, **kw)
    want, wz = other.forward()
    grads = other.backward()
    ws = [c.ws(k) for k in (B.MOK_LINEAR_FORWARD, B.MOK_LINEAR_BACKWARD)]
    y, z = (c.empty(c.rows, c.ld_out, t) for t in (c.out_dt, torch.bfloat16))
    o = [c.empty(c.rows, c.ld_in, c.grad_dt), c.empty(c.G * c.N, c.ld_in, c.grad_dt),
         torch.full((c.G * c.N + 3,), 7.0, device="cuda")]

    def both():
        B.check(B.mok_linear_forward(c.cfg, c.x, c.w, c.b, c.res, c.d_starts, c.d_counts, y, z,
                                     *ws[0]))
        B.check(B.mok_linear_backward(c.cfg, c.x, c.w, c.z, c.dy, c.d_starts, c.d_counts, *o,
                                      *ws[1]))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for name in ("x", "w", "b", "res", "z", "dy"):
        getattr(c, name).copy_(getattr(other, name))
    for _ in range(3):
        graph.replay()
    assert device_ok()
    for got, ref in zip((y, z, *o), (want, wz, *grads)):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_sort_replayed_on_other_inputs():
    torch = _t()
    c = Case(T=500, K=4, E=16, H=264, seed=2, capacity=100)
    sched, idx, w = c.sched(), c.dev(c.idx), c.dev(c.w)
    m, starts, kept = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2000, 17, 16))
    x, xs, y = c.array(500), c.array(c.n_rows, fill=0.0), c.array(500, fill=0.0)
    drows, dw = c.array(c.n_rows, fill=0.0), torch.zeros(2000, device="cuda")

    def all_passes():
        B.check(B.mok_build_row_map(c.cfg, idx, sched, m, starts, kept))
        B.check(B.mok_dispatch(c.cfg, x, m, starts, kept, xs))
        B.check(B.mok_combine(c.cfg, xs, m, w, x, y))
        B.check(B.mok_combine_backward(c.cfg, y, xs, m, starts, kept, w, drows, dw))

    all_passes()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_passes()
    x.copy_(c.array(500))
    w.mul_(0.5)
    all_passes()
    want = [t.clone() for t in (xs, y, drows, dw)]
    for t in (xs, y, drows, dw):
        t.zero_()
    graph.replay()
    assert device_ok() and np.array_equal(m.cpu().numpy(), c.map)
    for got, ref in zip((xs, y, drows, dw), want):
        got, ref = (t[:, :264] if t.dim() == 2 else t for t in (got, ref))
        assert torch.equal(got, ref)
