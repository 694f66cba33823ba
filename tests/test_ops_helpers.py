"""The helpers that hold the operators' buffers (no GPU): what they pass on and what they refuse.
The entry points are replaced by recorders, so nothing is launched; the arrays live on the host."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

torch = pytest.importorskip("torch")
from mixture_experts_layer_deterministic_gb300.buffers import AdamW, Linear, TokenSort  # noqa: E402

F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture
def calls(monkeypatch):
    """Names of the entry points that were reached, which do nothing."""
    seen = []
    for name in ("mok_linear_forward", "mok_linear_backward", "mok_build_row_map", "mok_dispatch",
                 "mok_dispatch_backward", "mok_combine", "mok_combine_backward",
                 "mok_adamw_step"):
        monkeypatch.setattr(B, name, lambda *a, _n=name: seen.append(_n) or B.MOK_OK)
    return seen


def refused(calls, f, *a, **kw):
    n = len(calls)
    with pytest.raises(ValueError):
        f(*a, **kw)
    assert len(calls) == n


class Arrays:
    """A Linear of 20 rows, 1001 -> 24 (rows of x are 1008 apart) and arrays that fit it."""

    def __init__(self, groups=1, K=1001, N=24, **kw):
        self.lin = Linear(20, K, N, groups=groups, device="cpu", **kw)
        out, grad = kw.get("out_dtype", BF), kw.get("grad_dtype", BF)
        row = lambda n, dt: torch.zeros(20, (n + 7) // 8 * 8, dtype=dt)[:, :n]  # noqa: E731
        self.fwd = dict(x=row(K, BF), w=self.lin.weights(), y=row(N, out),
                        bias=torch.zeros(groups * N), residual=row(N, BF), z=row(N, BF))
        self.bwd = dict(x=row(K, BF), w=self.lin.weights(), dy=row(N, out), z=row(N, BF),
                        dx=row(K, grad), dw=self.lin.weights(grad), db=torch.zeros(groups, N))


@pytest.mark.parametrize("kw", [dict(), dict(out_dtype=F32, grad_dtype=F32), dict(K=64, N=1)])
def test_linear_takes_what_fits(calls, kw):
    a = Arrays(**kw)
    assert a.lin.forward(**a.fwd) is a.fwd["y"]
    assert a.lin.backward(**a.bwd) is a.bwd["dx"]
    a.lin.forward(a.fwd["x"], a.fwd["w"], a.fwd["y"])
    a.lin.backward(a.bwd["x"], a.bwd["w"], a.bwd["dy"], dx=a.bwd["dx"])
    # more rows than the layer's, weights as [out][in], a padded buffer as a whole
    a.lin.forward(torch.zeros(30, a.lin.cfg.ld_in, dtype=BF), a.fwd["w"][0], a.fwd["y"])
    assert len(calls) == 5


def test_linear_weights_have_the_padded_stride():
    lin = Linear(20, 1001, 24, groups=3, device="cpu")
    w = lin.weights()
    assert w.shape == (3, 24, 1001) and w.stride() == (24 * 1008, 1008, 1) and w.dtype == BF
    assert lin.weights(F32).dtype == F32 and not bool(w.any())


def test_linear_refuses_weights_that_are_not_its_own(calls):
    a = Arrays()
    good = a.fwd["w"]
    for w in (torch.zeros(1, 24, 1001, dtype=BF),              # packed: rows 1001 apart
              torch.zeros(24, 1001, dtype=BF),
              torch.zeros(1, 24, 1008, dtype=F32)[..., :1001],
              torch.zeros(1, 24, 1008, dtype=F16)[..., :1001],
              torch.zeros(1, 23, 1008, dtype=BF)[..., :1001],  # too few features
              torch.zeros(1, 24, 1008, dtype=BF)[..., :1000],  # too few inputs
              torch.zeros(1, 24, 1008 * 2, dtype=BF)[..., :2002:2],
              good[0, 0]):
        refused(calls, a.lin.forward, **dict(a.fwd, w=w))
        refused(calls, a.lin.backward, **dict(a.bwd, w=w))
        refused(calls, a.lin.backward, **dict(a.bwd, dw=w))
    # groups further apart than their matrices
    g = Linear(20, 1001, 24, groups=2, device="cpu")
    wide = torch.zeros(2, 30, 1008, dtype=BF)[:, :24, :1001]
    sort = type("Sort", (), dict(E=2, starts=None, kept=None))()
    refused(calls, g.forward, a.fwd["x"], wide, a.fwd["y"], sort=sort)
    g.forward(a.fwd["x"], g.weights(), a.fwd["y"], sort=sort)


@pytest.mark.parametrize("kw", [dict(), dict(out_dtype=F32, grad_dtype=F32)])
def test_linear_refuses_arrays_that_do_not_fit(calls, kw):
    a = Arrays(**kw)
    for call, args in ((a.lin.forward, a.fwd), (a.lin.backward, a.bwd)):
        for k, t in args.items():
            if k in ("w", "dw"):
                continue
            other = F32 if t.dtype == BF else BF
            wrong = [t.to(other), t.to(F16)]
            if k in ("bias", "db"):
                wrong += [t.reshape(-1)[:-1], torch.zeros(2 * t.numel())[::2]]
            else:
                ld = t.stride(0)
                wrong += [t[:-1], torch.zeros(20, ld, dtype=t.dtype)[:, :t.shape[1] - 1],
                          torch.zeros(20, ld + 8, dtype=t.dtype)[:, :t.shape[1]],
                          torch.zeros(20, 2 * t.shape[1], dtype=t.dtype)[:, ::2], t[0]]
            for w in wrong:
                refused(calls, call, **dict(args, **{k: w}))
            refused(calls, call, **dict(args, **{k: t.to("meta")}))  # another device's
    assert not calls


def test_linear_refuses_other_types_and_a_sort_of_other_groups(calls):
    for dt in (F16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            Linear(20, 64, 24, out_dtype=dt, device="cpu")
        with pytest.raises(ValueError):
            Linear(20, 64, 24, grad_dtype=dt, device="cpu")
    a = Arrays(groups=3)
    sort = type("Sort", (), dict(E=4, starts=None, kept=None))()
    refused(calls, a.lin.forward, **a.fwd, sort=sort)
    refused(calls, a.lin.backward, **a.bwd, sort=sort)
    refused(calls, a.lin.forward, **a.fwd)  # groups without their rows
    refused(calls, a.lin.backward, **a.bwd)
    sort.E = 3
    a.lin.forward(**a.fwd, sort=sort)
    a.lin.backward(**a.bwd, sort=sort)


class Sorted:
    """A TokenSort of 20 tokens with 3 of 7 experts, 101 columns, and arrays that fit it."""

    def __init__(self, dtype, T=20):
        self.sort = TokenSort(T, 3, 7, 101, dtype=dtype, device="cpu")
        ld = 104
        tok = lambda: torch.zeros(T, ld, dtype=dtype)[:, :101]  # noqa: E731
        r, w = self.sort.rows, lambda: torch.zeros(T, 3)  # noqa: E731
        self.sched = type("Sched", (), dict(R=3 * T, counts=torch.zeros(7), struct=None))()
        self.args = dict(dispatch=dict(x=tok(), xs=r()), dispatch_backward=dict(dxs=r(), dx=tok()),
                         combine=dict(rows=r(), topk_w=w(), y=tok(), residual=tok()),
                         combine_backward=dict(dy=tok(), rows=r(), topk_w=w(), drows=r(),
                                               d_topk_w=w()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [20, 1])
def test_sort_takes_what_fits(calls, dtype, T):
    s = Sorted(dtype, T)
    s.sort.build(torch.zeros(3 * T, dtype=torch.int32), s.sched)
    for name, args in s.args.items():
        getattr(s.sort, name)(**args)
    s.sort.combine(s.sort.rows(), None, s.args["combine"]["y"])  # weights of one, no residual
    s.sort.combine_backward(s.args["combine"]["y"], None, None, s.sort.rows(), None)
    if T == 1:  # one row has no stride
        s.sort.dispatch(torch.zeros(1, 101, dtype=dtype), s.sort.rows())
    assert len(calls) == (8 if T == 1 else 7)
    empty = TokenSort(0, 3, 7, 101, dtype=dtype, device="cpu")
    empty.combine(empty.rows(), torch.zeros(1), torch.zeros(0, 104, dtype=dtype)[:, :101])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sort_refuses_arrays_that_do_not_fit(calls, dtype):
    s = Sorted(dtype)
    for name, args in s.args.items():
        call = getattr(s.sort, name)
        for k, t in args.items():
            other = F32 if t.dtype == BF else BF
            wrong = [t.to(other), t.to(F16), t.to(torch.float64), t[:-1], t.to("meta"),
                     torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]]
            if "topk_w" not in k:
                wrong += [torch.zeros(t.shape[0], 112, dtype=dtype)[:, :101],
                          torch.zeros(t.shape[0], 104, dtype=dtype)[:, :100],
                          torch.zeros(t.shape[0], 101, dtype=dtype), t[0]]
            for w in wrong:
                refused(calls, call, **dict(args, **{k: w}))
    ids = torch.zeros(60, dtype=torch.int32)
    for idx in (ids.long(), ids[:-1], ids.float(), ids.to("meta"),
                torch.zeros(120, dtype=torch.int32)[::2]):
        refused(calls, s.sort.build, idx, s.sched)
    for kw in (dict(R=59), dict(counts=torch.zeros(8))):
        sched = type("Sched", (), dict(vars(type(s.sched)), **kw))()
        refused(calls, s.sort.build, ids, sched)


def test_sort_refuses_other_types():
    for dt in (F16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            TokenSort(20, 3, 7, 101, dtype=dt, device="cpu")


@pytest.mark.parametrize("eight_bit", [False, True])
def test_adamw_takes_what_fits(calls, eight_bit):
    mk = lambda *s, dt=F32: torch.zeros(*s, dtype=dt)  # noqa: E731
    opt = AdamW([dict(p=mk(3, 40), g=mk(3, 40, dt=BF), copy=mk(3, 40, dt=BF)),
                 dict(p=mk(7), g=mk(7), weight_decay=0.1), dict(p=mk(5, dt=BF), g=mk(5, dt=BF)),
                 dict(p=mk(9, dt=BF), g=mk(9)), dict(p=mk(2), g=mk(2))], lr=1e-3,
                eight_bit=eight_bit, device="cpu")
    opt.step()
    opt.step(grad_scale=torch.ones(1))
    assert [k for k, _ in opt.lists] == [(B.MOK_DTYPE_F32, B.MOK_DTYPE_BF16),
                                         (B.MOK_DTYPE_F32, B.MOK_DTYPE_F32),
                                         (B.MOK_DTYPE_BF16, B.MOK_DTYPE_BF16),
                                         (B.MOK_DTYPE_BF16, B.MOK_DTYPE_F32)]
    assert len(calls) == 8 and opt.t == 2


def test_adamw_refuses_arrays_that_do_not_fit(calls):
    mk = lambda n, dt=F32: torch.zeros(n, dtype=dt)  # noqa: E731
    good = dict(p=mk(40), g=mk(40, BF), copy=mk(40, BF))
    for kw in [dict(p=mk(40, dt)) for dt in (F16, torch.float64, torch.int8)] + \
              [dict(g=mk(40, dt)) for dt in (F16, torch.float64, torch.uint8)] + \
              [dict(copy=mk(40, dt)) for dt in (F32, F16, torch.uint8)] + \
              [dict(g=mk(39)), dict(copy=mk(39, BF)), dict(p=mk(41)), dict(p=mk(80)[::2]),
               dict(g=mk(80)[::2]), dict(copy=mk(80, BF)[::2]), dict(p=mk(40, BF)),
               dict(g=mk(40).to("meta")), dict(copy=mk(40, BF).to("meta"))]:
        refused(calls, AdamW, [dict(good, **kw)], lr=1e-3, device="cpu")
    opt = AdamW([good], lr=1e-3, device="cpu")
    for gs in (mk(1, BF), mk(2), mk(1).to("meta")):
        refused(calls, opt.step, gs)
    assert opt.t == 0
