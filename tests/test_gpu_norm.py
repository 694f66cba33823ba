"""Layer and RMS norm and their gradients against the definitions in 64 bits.

Tolerances (derived): a sum over a row adds at most 32 terms a thread, 5 steps of a warp and 32
warps in turn: it is within 2^-17 of the sum of its terms' magnitudes (for 2^20 elements 128 terms a
thread: 2^-16). The mean is corrected by that of the differences from it, so the normalised value n
is off by 2^-16 (1 + |n|) and by the mean's last digit, 2^-23 |mean| rstd. dw and db add rows one
after another (20 a block for 6000 rows, 304 blocks in 16 slices): 2^-16 of their terms' magnitudes.
bf16 outputs add 2^-8 of a value, fp32 ones 2^-23."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu
E = 2.0 ** -16


def _t():
    import torch
    return torch


def device_ok():
    st, dev = B.mok_read_device_status()
    B.mok_clear_device_status()
    return (st, dev) == (B.MOK_OK, B.MOK_OK)


def dt(name):
    torch = _t()
    return torch.float32 if name == "fp32" else torch.bfloat16


class Case:
    """Inputs with guard columns (NaN) that must not be read; outputs are filled with 7."""

    def __init__(self, R=5, H=64, kind="layer", x="bf16", y="bf16", w=True, b=True, res=True,
                 extra=0, mean=0.3, std=1.0, seed=0, eps=1e-5):
        torch = _t()
        self.R, self.H, self.layer, self.eps = R, H, kind == "layer", eps
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.xd, self.yd = dt(x), dt(y)
        up8 = (H + 7) // 8 * 8
        self.ld_x, self.ld_y = up8 + extra, up8 + 2 * extra
        self.x = self.rand(self.ld_x, self.xd, mean, std)
        self.res = self.rand(self.ld_x, self.xd, 0, std) if res else None
        vec = lambda m: m + torch.randn(H, device="cuda", generator=self.gen) * 0.3  # noqa: E731
        self.w, self.b = vec(1.0) if w else None, vec(0.0) if b else None
        kinds = {"fp32": B.MOK_DTYPE_F32, "bf16": B.MOK_DTYPE_BF16}
        self.cfg = B.make_norm(R, H, B.MOK_NORM_LAYER if self.layer else B.MOK_NORM_RMS, eps,
                               kinds[x], kinds[y], self.ld_x, self.ld_y)
        assert B.mok_check_norm_config(self.cfg) == B.MOK_OK
        self.u = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8}

    def rand(self, ld, dtype, mean=0.0, std=1.0):
        torch = _t()
        buf = torch.full((max(self.R, 1), ld), float("nan"), device="cuda", dtype=dtype)
        size = torch.rand(self.R, 1, device="cuda", generator=self.gen) * 3 + 0.1
        live = torch.randn(self.R, self.H, device="cuda", generator=self.gen) * std * size + mean
        buf[:self.R, :self.H] = live.to(dtype)
        return buf

    def out(self, ld, dtype):
        return _t().full((max(self.R, 1), ld), 7.0, device="cuda", dtype=dtype)

    def stat(self):
        return _t().full((self.R + 3,), 7.0, device="cuda")

    def forward(self, stats=True, stream=None):
        h = self.out(self.ld_x, self.xd) if self.res is not None else None
        y = self.out(self.ld_y, self.yd)
        mean = self.stat() if stats and self.layer else None
        rstd = self.stat() if stats else None
        B.check(B.mok_norm_forward(self.cfg, self.x, self.res, self.w, self.b, h, y, mean, rstd,
                                   stream))
        return h, y, mean, rstd

    def live(self, t):
        return t[:self.R, :self.H].double()

    def moments(self, h):
        torch = _t()
        mean = h.mean(1) if self.layer else torch.zeros(self.R, device="cuda", dtype=torch.float64)
        return mean, ((h - mean[:, None]).square().mean(1) + self.eps).rsqrt()

    def backward(self, h, mean, rstd, dy, dh, parts=(True, True, True), stream=None):
        torch = _t()
        dx = self.out(self.ld_x, self.xd) if parts[0] else None
        dw, db = (torch.full((self.H + 3,), 7.0, device="cuda") if p else None for p in parts[1:])
        n = B.mok_norm_workspace_size(self.cfg)
        assert n > 0
        ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        B.check(B.mok_norm_backward(self.cfg, h, mean, rstd, self.w, dy, dh, dx, dw, db, ws, n,
                                    stream))
        self._keep = ws
        return dx, dw, db


CASES = [
    dict(R=1, H=1), dict(R=3, H=1, kind="rms", x="fp32", y="fp32"),
    dict(R=1, H=4096, kind="rms", b=False),
    dict(R=2, H=7, extra=8), dict(R=1000, H=16), dict(R=999, H=24, kind="rms", x="fp32"),
    dict(R=77, H=100, x="fp32", y="fp32", extra=8), dict(R=33, H=256, w=False, b=False, res=False),
    dict(R=31, H=264, kind="rms", res=False, extra=16), dict(R=13, H=1111, x="fp32", y="fp32"),
    dict(R=700, H=1000, y="fp32"), dict(R=9, H=4100, kind="rms", x="fp32", y="bf16"),
    dict(R=6000, H=512), dict(R=5, H=8193), dict(R=4, H=16384, x="fp32", y="fp32"),
    dict(R=3, H=30001, kind="rms"), dict(R=3, H=32768, x="fp32", y="fp32"),
    dict(R=40, H=32776, extra=8), dict(R=700, H=9000), dict(R=500, H=20000, x="fp32"),
    dict(R=11, H=65536), dict(R=11, H=65544, extra=8), dict(R=2, H=100003, x="fp32", y="fp32"),
    dict(R=2, H=1 << 20, kind="rms", res=False),
]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_forward(kw):
    torch = _t()
    c = Case(**kw)
    h, y, mean, rstd = c.forward()
    assert device_ok()
    x = c.live(c.x)
    if h is not None:
        s = x + c.live(c.res)
        got = c.live(h)
        assert bool(((got - s).abs() <= (c.u[c.xd] + 2.0 ** -23) * s.abs()).all())
        assert bool((h[:c.R, c.H:] == 7).all())
        x = got
    m, r = c.moments(x)
    n = (x - m[:, None]) * r[:, None]
    en = E * (1 + n.abs()) + 2.0 ** -23 * (m.abs() * r)[:, None]
    w = 1.0 if c.w is None else c.w.double()
    ref = n * w + (0.0 if c.b is None else c.b.double())
    tol = en * (1.0 if c.w is None else w.abs()) + 2.0 ** -22 * (n * w).abs() + 2.0 ** -23 * ref.abs()
    tol = tol + c.u[c.yd] * (ref.abs() + tol)
    assert bool(((c.live(y) - ref).abs() <= tol).all())
    assert bool((y[:c.R, c.H:] == 7).all()) and bool((rstd[c.R:] == 7).all())
    assert bool(((rstd[:c.R].double() - r).abs() <= E * r).all())
    if mean is not None:
        # relative to the row's spread, and the mean's own last digit
        assert bool(((mean[:c.R].double() - m).abs() <= E / r + 2.0 ** -23 * m.abs()).all())
        assert bool((mean[c.R:] == 7).all())


def check_backward(c, dh=True, parts=(True, True, True)):
    torch = _t()
    h = c.x
    m, r = c.moments(c.live(h))
    mean, rstd = (m.float() if c.layer else None), r.float()
    dy = c.rand(c.ld_y, c.yd)
    dh = c.rand(c.ld_x, c.xd) if dh else None
    dx, dw, db = c.backward(h, mean, rstd, dy, dh, parts)
    assert device_ok()
    r64 = rstd.double()[:, None]
    m64 = mean.double()[:, None] if c.layer else 0.0
    n = (c.live(h) - m64) * r64
    d = c.live(dy)
    en = 2.0 ** -22 * (n.abs() + (abs(m64) * r64 if c.layer else 0.0))
    g = d * (1.0 if c.w is None else c.w.double())
    if dx is not None:
        gn, mg = (g * n).mean(1, keepdim=True), g.mean(1, keepdim=True)
        ref = g - n * gn - (mg if c.layer else 0.0)
        agn, ag = (g * n).abs().mean(1, keepdim=True), g.abs().mean(1, keepdim=True)
        tol = E * (g.abs() + (n.abs() + 1) * agn + ag) + en * agn + \
            n.abs() * (g.abs() * en).mean(1, keepdim=True)
        ref, tol = ref * r64, tol * r64
        if dh is not None:
            ref = ref + c.live(dh)
            tol = tol + 2.0 ** -23 * ref.abs()
        tol = tol + c.u[c.xd] * (ref.abs() + tol)
        assert bool(((c.live(dx) - ref).abs() <= tol).all())
        assert bool((dx[:c.R, c.H:] == 7).all())
    if dw is not None:
        tol = E * (d * n).abs().sum(0) + (d.abs() * en).sum(0)
        assert bool(((dw[:c.H].double() - (d * n).sum(0)).abs() <= tol).all())
        assert bool((dw[c.H:] == 7).all())
    if db is not None:
        assert bool(((db[:c.H].double() - d.sum(0)).abs() <= E * d.abs().sum(0)).all())
        assert bool((db[c.H:] == 7).all())
    return h, mean, rstd, dy, dh, dx, dw, db


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_backward(kw):
    check_backward(Case(**kw), dh=kw.get("res", True))


@pytest.mark.parametrize("parts", [(True, False, False), (False, True, False), (False, False, True),
                                   (True, False, True), (False, True, True)], ids=str)
def test_backward_parts_have_the_same_bits(parts):
    torch = _t()
    for H in (520, 40000, 70000):  # a block's rows, a cluster's, rows that are read again
        c = Case(R=300 if H < 1000 else 40, H=H)
        *ins, dx, dw, db = check_backward(c)
        out = c.backward(*ins, parts)
        for got, want, asked in zip(out, (dx, dw, db), parts):
            assert (got is None) == (not asked)
            assert got is None or torch.equal(got, want)


def test_backward_of_the_forwards_own_statistics_against_differences():
    """d(sum(dy y)) along a random direction of x, from 64-bit values at h +- step, against the
    kernels' dx in fp32 from the forward's h, mean and rstd."""
    torch = _t()
    for kind in ("layer", "rms"):
        c = Case(R=6, H=130, kind=kind, x="fp32", y="fp32", res=True)
        h, _, mean, rstd = c.forward()
        dy = c.rand(c.ld_y, c.yd)
        dx, dw, db = c.backward(h, mean, rstd, dy, None)
        along = torch.randn(6, 130, device="cuda", dtype=torch.float64, generator=c.gen)

        def value(x, w, b):
            m, r = c.moments(x)
            return (c.live(dy) * ((x - m[:, None]) * r[:, None] * w + b)).sum()

        x, w, b, e = c.live(h), c.w.double(), c.b.double(), 1e-5
        for got, f, size in (
                ((c.live(dx) * along).sum(), lambda t: value(x + t * along, w, b),
                 (c.live(dx).abs() * along.abs()).sum()),
                ((dw[:130].double() * along[0]).sum(), lambda t: value(x, w + t * along[0], b),
                 (c.live(dy).abs() * 4).sum()),
                ((db[:130].double() * along[1]).sum(), lambda t: value(x, w, b + t * along[1]),
                 (c.live(dy).abs() * 4).sum())):
            slope = (f(e) - f(-e)) / (2 * e)
            assert abs(float(got - slope)) <= 1e-4 * float(size)


def test_rows_far_from_zero_keep_their_digits():
    """A mean of 1000 spreads: n is within what the mean's last digit allows."""
    c = Case(R=20, H=999, x="fp32", y="fp32", res=False, mean=1000.0)
    _, y, mean, rstd = c.forward()
    x = c.live(c.x)
    m, r = c.moments(x)
    ref = (x - m[:, None]) * r[:, None] * c.w.double() + c.b.double()
    tol = (E * (2 + ref.abs()) + 2.0 ** -23 * (m.abs() * r)[:, None]) * (1 + c.w.abs().double())
    assert bool(((c.live(y) - ref).abs() <= tol).all())
    assert bool(((rstd[:20].double() - r).abs() <= E * r).all())


def test_constant_rows():
    """No spread: y is the bias, rstd 1 / sqrt(eps) (the mean of equal values is exact)."""
    torch = _t()
    c = Case(R=3, H=300, x="fp32", y="fp32", res=False)
    c.x[:, :300] = torch.tensor([[0.0], [2.5], [-7.0]], device="cuda")
    _, y, mean, rstd = c.forward()
    assert bool(((rstd[:3] - 1e-5 ** -0.5).abs() <= 1e-3).all())
    assert bool(((c.live(y) - c.b.double()).abs() <= 1e-3 * c.w.abs().double()).all())
    assert bool(((mean[:3].cpu() - torch.tensor([0.0, 2.5, -7.0])).abs() <= 1e-6).all())


def test_a_row_that_is_not_finite_spoils_itself_alone():
    torch = _t()
    for H in (70, 4096, 40000):
        c = Case(R=12, H=H, x="fp32", y="fp32", res=False)
        _, y, _, _ = c.forward()
        c.x[5, 3], c.x[8, 1] = float("nan"), float("inf")
        _, y2, _, _ = c.forward()
        keep = [r for r in range(12) if r not in (5, 8)]
        assert torch.equal(y[keep, :H], y2[keep, :H]) and bool(y2[5, :H].isnan().all())
        assert device_ok()


@pytest.mark.parametrize("kw", [dict(R=40, H=520, x="fp32", y="fp32"), dict(R=20, H=40000),
                                dict(R=20, H=70000)], ids=str)
def test_in_place(kw):
    torch = _t()
    c = Case(**dict(kw, extra=0))
    h, y, mean, rstd = c.forward()
    n = B.mok_norm_workspace_size(c.cfg)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    live = lambda t: t[:, :c.H]  # noqa: E731
    x2, y2 = c.x.clone(), torch.empty_like(y)
    B.check(B.mok_norm_forward(c.cfg, x2, c.res, c.w, c.b, x2, y2))      # h over x
    assert torch.equal(live(x2), live(h)) and torch.equal(live(y2), live(y))
    r2 = c.res.clone()
    B.check(B.mok_norm_forward(c.cfg, c.x, r2, c.w, c.b, r2, y2))        # h over the residual
    assert torch.equal(live(r2), live(h)) and torch.equal(live(y2), live(y))
    x3 = c.x.clone()
    B.check(B.mok_norm_forward(c.cfg, x3, c.res, c.w, c.b, None, x3))    # y over x
    assert torch.equal(live(x3), live(y))
    dy, dh = c.rand(c.ld_y, c.yd), c.rand(c.ld_x, c.xd)
    dx, dw, db = c.backward(h, mean, rstd, dy, dh)
    for over in ("dh", "dy"):
        t = dict(dh=dh.clone(), dy=dy.clone())
        w2, b2 = torch.zeros(c.H, device="cuda"), torch.zeros(c.H, device="cuda")
        B.check(B.mok_norm_backward(c.cfg, h, mean, rstd, c.w, t["dy"], t["dh"], t[over], w2, b2, ws, n))
        assert torch.equal(live(t[over]), live(dx))
        assert torch.equal(w2, dw[:c.H]) and torch.equal(b2, db[:c.H])
    assert device_ok()


def test_repeated_and_on_a_stream():
    torch = _t()
    c = Case(R=900, H=1030)
    h, y, mean, rstd = c.forward()
    dy, dh = c.rand(c.ld_y, c.yd), c.rand(c.ld_x, c.xd)
    first = c.backward(h, mean, rstd, dy, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, None, s):
        for a, b in zip((h, y, mean, rstd), c.forward(stream=stream)):
            torch.cuda.synchronize()
            assert torch.equal(a, b)
        for a, b in zip(first, c.backward(h, mean, rstd, dy, dh, stream=stream)):
            torch.cuda.synchronize()
            assert torch.equal(a, b)


def test_no_rows():
    torch = _t()
    c = Case(R=0, H=24)
    c.forward()
    dx, dw, db = c.backward(c.x, c.stat(), c.stat(), c.x, None)
    assert dw[:24].tolist() == [0.0] * 24 and db[:24].tolist() == [0.0] * 24 and device_ok()


def test_refusals():
    torch = _t()
    c = Case(R=8, H=64, extra=0)
    h, y, mean, rstd = c.forward()
    bad, nows = B.MOK_ERR_INVALID_ARG, B.MOK_ERR_WORKSPACE
    f = lambda cfg=c.cfg, x=c.x, r=c.res, w=c.w, b=c.b, h=h, y=y, m=mean, s=rstd: \
        B.mok_norm_forward(cfg, x, r, w, b, h, y, m, s)  # noqa: E731
    assert f() == B.MOK_OK and f(h=None, m=None, s=None, w=None, b=None) == B.MOK_OK
    assert f(x=None) == bad and f(y=None) == bad and f(r=None) == bad  # h without a residual
    assert f(y=h) == bad
    for k in ("x", "r", "w", "b", "h", "y", "m", "s"):
        assert f(**{k: y.data_ptr() + 8}) == bad
    rms = B.make_norm(8, 64, B.MOK_NORM_RMS)
    assert f(cfg=rms) == bad and f(cfg=rms, m=None) == B.MOK_OK
    wide = B.make_norm(8, 64, ld_y=72)
    big = torch.zeros(8, 72, device="cuda", dtype=torch.bfloat16)
    assert f(cfg=wide, y=big) == B.MOK_OK and f(cfg=wide, y=c.x, x=c.x, h=None) == bad
    assert f(cfg=wide, y=c.res, h=None) == bad and f(y=c.res, h=None) == B.MOK_OK
    assert f(cfg=B.make_norm(8, 64, eps=0.0)) == bad
    n = B.mok_norm_workspace_size(c.cfg)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.zeros_like(h), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    dy = torch.zeros_like(y)
    g = lambda h=h, m=mean, s=rstd, w=c.w, dy=dy, dh=None, dx=dx, dw=dw, db=db, ws=ws, n=n: \
        B.mok_norm_backward(c.cfg, h, m, s, w, dy, dh, dx, dw, db, ws, n)  # noqa: E731
    assert g() == B.MOK_OK and g(dw=None, db=None, ws=None, n=0) == B.MOK_OK
    assert g(dx=None, dw=None, db=None) == bad
    for k in ("h", "m", "s", "dy"):
        assert g(**{k: None}) == bad
    assert g(dx=h) == bad
    assert g(ws=None) == nows and g(n=n - 1) == nows and g(ws=ws[8:]) == nows
    for k in ("h", "m", "s", "w", "dy", "dh", "dx", "dw", "db"):
        assert g(**{k: y.data_ptr() + 8}) == bad
    assert device_ok()
