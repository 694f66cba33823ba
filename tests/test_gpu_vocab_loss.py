"""The loss over a vocabulary and its gradients against the definitions in 64 bits.

Tolerances (derived): an fp32 tensor-core sum of n terms is within 2^-19 max(1, sqrt(n / 2048)) of
the sum of its terms' magnitudes (measured on this hardware, tests/test_gpu_backward.py): el for a
logit. lse moves by at most the largest el; 2^x is within 2^-22 and its argument's rounding within
2^-24 |l - lse| log2(e), both relative (results below 2^-126 become 0: that much on top for a
probability's factor of at most 1), and a sum of V terms over 16-column runs and joins adds
2^-17: 2^-16 in all; rounding lse and the loss 2^-22 of their size. dl is off by what its logit and lse
are off, relative to the probability; it enters the products rounded to bf16 (2^-8), as two values (2^-16)
up to 512 rows, or as three (2^-17) for fp32 gradients; outputs are rounded to their type."""
import math

import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def device_ok():
    st, dev = B.mok_read_device_status()
    B.mok_clear_device_status()
    return (st, dev) == (B.MOK_OK, B.MOK_OK)


def dot_rel(n):
    return 2.0 ** -19 * max(1.0, math.sqrt(n / 2048))


class Case:
    """Inputs with guard columns (NaN) that must not be read; outputs are filled with 7."""

    def __init__(self, R=20, H=64, V=300, z=0.0, grad="bf16", piece=0, extra=0, ignore=0.2, std=2.0,
                 seed=0):
        torch = _t()
        self.R, self.H, self.V, self.z = R, H, V, z
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.gd = torch.float32 if grad == "fp32" else torch.bfloat16
        up8 = (H + 7) // 8 * 8
        self.ld_x, self.ld_w = up8 + extra, up8 + 2 * extra
        self.x = self.rand(R, self.ld_x, 1.0)
        self.w = self.rand(V, self.ld_w, std / math.sqrt(H))
        self.t = torch.randint(0, V, (R,), device="cuda", generator=self.gen, dtype=torch.int32)
        off = torch.rand(R, device="cuda", generator=self.gen) < ignore
        self.t[off] = -1 - torch.arange(R, device="cuda", dtype=torch.int32)[off] * 1000
        self.d = torch.rand(R, device="cuda", generator=self.gen) - 0.3
        self.d[off] = float("nan")  # of rows that take no part: not looked at
        self.cfg = B.make_vocab_loss(R, H, V, z, B.MOK_DTYPE_F32 if grad == "fp32"
                                     else B.MOK_DTYPE_BF16, piece, self.ld_x, self.ld_w)
        assert B.mok_check_vocab_loss_config(self.cfg) == B.MOK_OK

    def rand(self, rows, ld, std):
        torch = _t()
        buf = torch.full((max(rows, 1), ld), float("nan"), device="cuda", dtype=torch.bfloat16)
        buf[:rows, :self.H] = (torch.randn(rows, self.H, device="cuda", generator=self.gen) *
                               std).to(torch.bfloat16)
        return buf

    def ws(self, which):
        n = B.mok_vocab_loss_workspace_size(self.cfg, which)
        assert n > 0
        self._keep = _t().full((n,), 0xFF, dtype=_t().uint8, device="cuda")
        return self._keep, n

    def forward(self, stream=None):
        torch = _t()
        loss, lse = (torch.full((self.R + 3,), 7.0, device="cuda") for _ in range(2))
        ws, n = self.ws(B.MOK_VOCAB_LOSS_FORWARD)
        B.check(B.mok_vocab_loss_forward(self.cfg, self.x, self.w, self.t, loss, lse, ws, n, stream))
        return loss, lse

    def backward(self, lse, dx=True, dw=True, stream=None):
        torch = _t()
        o = lambda rows, ld: torch.full((max(rows, 1), ld), 7.0, device="cuda", dtype=self.gd)  # noqa: E731
        dx = o(self.R, self.ld_x) if dx else None
        dw = o(self.V, self.ld_w) if dw else None
        ws, n = self.ws(B.MOK_VOCAB_LOSS_BACKWARD)
        B.check(B.mok_vocab_loss_backward(self.cfg, self.x, self.w, self.t, lse, self.d, dx, dw, ws, n,
                                          stream))
        return dx, dw

    def exact(self):
        """x, w, logits and the bound of their errors, lse, in 64 bits."""
        torch = _t()
        x, w = self.x[:self.R, :self.H].double(), self.w[:self.V, :self.H].double()
        l = x @ w.T
        el = dot_rel(self.H) * (x.abs() @ w.abs().T)
        return x, w, l, el, torch.logsumexp(l, 1)


def check_forward(c):
    torch = _t()
    loss, lse = c.forward()
    assert device_ok()
    _, _, l, el, ref = c.exact()
    e = el.amax(1) + 2.0 ** -16 + 2.0 ** -22 * (ref.abs() + l.abs().amax(1))
    assert bool(((lse[:c.R].double() - ref).abs() <= e).all())
    live = c.t >= 0
    hit = l.gather(1, c.t.long().clamp(min=0)[:, None])[:, 0]
    want = torch.where(live, ref - hit + c.z * ref * ref, 0.0)
    tol = 2 * e + c.z * (2 * ref.abs() * e + 2.0 ** -22 * ref * ref) + 2.0 ** -22 * hit.abs()
    assert bool(((loss[:c.R].double() - want).abs() <= tol * live).all())
    assert bool((loss[c.R:] == 7).all()) and bool((lse[c.R:] == 7).all())
    return loss, lse


def check_backward(c, **parts):
    torch = _t()
    x, w, l, el, ref = c.exact()
    lse = ref.float()
    dx, dw = c.backward(lse, **parts)
    assert device_ok()
    live = c.t >= 0
    d = torch.where(live, c.d.double(), 0.0)[:, None]
    a = lse.double()[:, None]
    p = torch.exp(l - a) * d * (1 + 2 * c.z * a)
    dl = p.clone()
    dl.scatter_add_(1, c.t.long().clamp(min=0)[:, None], -d)
    arg = (l - a).abs()
    edl = p.abs() * (el + 2.0 ** -23 * arg + 2.0 ** -20) + 2.0 ** -23 * dl.abs() + 2.0 ** -126
    step = 2.0 ** -17 if c.gd != torch.bfloat16 else 2.0 ** -16 if c.R <= 512 else 2.0 ** -8
    edl = edl + step * (dl.abs() + edl)
    u = 2.0 ** -8 if c.gd == torch.bfloat16 else 2.0 ** -23
    pieces = 1 + (c.cfg.piece > 0) * c.V // max(c.cfg.piece, 1)
    for got, want, mag, err, n, rows in (
            (dx, dl @ w, dl.abs() @ w.abs(), edl @ w.abs(), c.V, c.R),
            (dw, dl.T @ x, dl.T.abs() @ x.abs(), edl.T @ x.abs(), c.R, c.V)):
        if got is None:
            continue
        tol = err + (dot_rel(n) + (pieces + 1) * 2.0 ** -23) * (mag + err)
        tol = tol + u * (want.abs() + tol) + 1e-38
        assert bool(((got[:rows, :c.H].double() - want).abs() <= tol).all())
        assert bool((got[:rows, c.H:] == 7).all())
    return lse, dx, dw


CASES = [
    dict(R=1, H=1, V=1, ignore=0.0), dict(R=1, H=64, V=2, ignore=0.0), dict(R=2, H=15, V=17),
    dict(R=4, H=4096, V=1000, std=3.0), dict(R=33, H=100, V=257, z=1e-2, extra=8),
    dict(R=256, H=256, V=256), dict(R=257, H=264, V=513, grad="fp32"),
    dict(R=1000, H=72, V=5003, z=1e-3), dict(R=300, H=1030, V=1500, grad="fp32", z=1e-3, extra=16),
    dict(R=70, H=2100, V=900, piece=256), dict(R=70, H=2100, V=900, piece=512, grad="fp32"),
    dict(R=513, H=129, V=3000, piece=1024, extra=8), dict(R=40, H=64, V=32001, piece=8192, z=1e-3),
    dict(R=5000, H=40, V=70, grad="fp32"), dict(R=129, H=520, V=300, ignore=1.0),
    dict(R=4200, H=128, V=700),                        # more than one band of row blocks
    dict(R=50, H=512, V=4000, std=40.0),               # one entry takes all, logits of +-100
    # few rows' bf16 gradients, whole, in pieces and cut along the vocabulary; and one row more
    dict(R=3, H=45, V=11962),
    dict(R=5, H=72, V=1000, piece=256),
    dict(R=130, H=1030, V=20000),
    dict(R=256, H=200, V=3000, z=1e-3),
    dict(R=512, H=200, V=3000, z=1e-3),
    dict(R=513, H=200, V=3000, z=1e-3),
]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_forward(kw):
    check_forward(Case(**kw))


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_backward(kw):
    check_backward(Case(**kw))


@pytest.mark.parametrize("kw", [dict(grad="bf16"), dict(grad="fp32"), dict(grad="bf16", piece=256),
                                dict(grad="fp32", piece=256)], ids=str)
def test_one_gradient_alone_and_repetition(kw):
    torch = _t()
    c = Case(R=300, H=200, V=1111, z=1e-3, **kw)
    lse, dx, dw = check_backward(c)
    for parts in (dict(dx=False), dict(dw=False), dict()):
        a, b = c.backward(lse, **parts)
        assert a is None or torch.equal(a, dx)
        assert b is None or torch.equal(b, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = c.backward(lse, stream=s)
    loss = c.forward(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dw)
    for u, v in zip(loss, c.forward()):
        assert torch.equal(u, v)


def test_without_a_loss():
    """lse alone, for a program that wants probabilities."""
    torch = _t()
    c = Case(R=40, H=100, V=500)
    loss, lse = c.forward()
    out = torch.full_like(lse, 7.0)
    ws, n = c.ws(B.MOK_VOCAB_LOSS_FORWARD)
    B.check(B.mok_vocab_loss_forward(c.cfg, c.x, c.w, c.t, None, out, ws, n))
    assert torch.equal(out, lse)


def test_targets_past_the_vocabulary():
    torch = _t()
    for piece in (0, 256):
        c = Case(R=30, H=64, V=300, piece=piece, ignore=0.0)
        c.t[3], c.t[7], c.t[11] = 300, 2 ** 31 - 1, 511
        loss, lse = c.forward()
        assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()
        dx, dw = c.backward(lse[:30])
        assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()
        c.t[[3, 7, 11]] = -1
        loss2, lse2 = c.forward()
        dx2, dw2 = c.backward(lse[:30])
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and device_ok()
        assert bool((dx[3, :64] == 0).all())


def test_a_row_that_is_not_finite_spoils_its_own_loss_alone():
    torch = _t()
    c = Case(R=40, H=96, V=700, ignore=0.0)
    loss, lse = c.forward()
    c.x[9, 5] = float("nan")
    loss2, lse2 = c.forward()
    keep = [r for r in range(40) if r != 9]
    assert torch.equal(loss[keep], loss2[keep]) and bool(loss2[9].isnan())
    dx, _ = c.backward(lse2[:40], dw=False)
    c.x[9, 5] = 0.0
    dx2, _ = c.backward(lse[:40], dw=False)
    assert torch.equal(dx[keep], dx2[keep])
    # such a row without a target: no gradient of its own, and nothing of it in any other
    c.t[9] = -1
    _, dw2 = c.backward(lse[:40])
    for bad in (float("nan"), float("inf")):
        c.x[9, 5] = bad
        dx, dw = c.backward(lse2[:40])
        assert torch.equal(dx[keep], dx2[keep]) and bool((dx[9, :96] == 0).all())
        assert torch.equal(dw, dw2)
    assert device_ok()


def test_gradients_against_differences():
    """The slope of sum(d loss) along a random direction of x and of W, in 64 bits."""
    torch = _t()
    c = Case(R=12, H=48, V=90, z=1e-2, grad="fp32", ignore=0.3)
    loss, lse = c.forward()
    dx, dw = c.backward(lse[:12])
    live = c.t >= 0
    d = torch.where(live, c.d.double(), 0.0)
    x, w = c.x[:12, :48].double(), c.w[:90, :48].double()

    def value(x, w):
        l = x @ w.T
        a = torch.logsumexp(l, 1)
        return (d * (a - l.gather(1, c.t.long().clamp(min=0)[:, None])[:, 0] + c.z * a * a)).sum()

    for got, like, f in ((dx[:12, :48], x, lambda s: value(x + s, w)),
                         (dw[:90, :48], w, lambda s: value(x, w + s))):
        along = torch.randn(*like.shape, device="cuda", dtype=torch.float64, generator=c.gen)
        slope = (f(1e-5 * along) - f(-1e-5 * along)) / 2e-5
        size = float((got.double().abs() * along.abs()).sum())
        assert abs(float((got.double() * along).sum() - slope)) <= 2e-5 * size


def test_no_rows():
    torch = _t()
    for grad in ("bf16", "fp32"):
        c = Case(R=0, H=20, V=30, grad=grad, extra=8)
        c.forward()
        _, dw = c.backward(None)
        assert bool((dw[:, :20] == 0).all()) and bool((dw[:, 20:] == 7).all()) and device_ok()


def test_refusals():
    torch = _t()
    c = Case(R=16, H=32, V=40)
    loss, lse = c.forward()
    bad, nows = B.MOK_ERR_INVALID_ARG, B.MOK_ERR_WORKSPACE
    ws, n = c.ws(B.MOK_VOCAB_LOSS_FORWARD)
    f = lambda x=c.x, w=c.w, t=c.t, o=loss, s=lse, ws=ws, n=n: \
        B.mok_vocab_loss_forward(c.cfg, x, w, t, o, s, ws, n)  # noqa: E731
    assert f() == B.MOK_OK
    for k in ("x", "w", "t", "s"):
        assert f(**{k: None}) == bad
    for k in ("x", "w", "t", "o", "s"):
        assert f(**{k: loss.data_ptr() + 8}) == bad
    assert f(ws=None) == nows and f(n=n - 1) == nows and f(ws=ws[8:]) == nows
    ws, n = c.ws(B.MOK_VOCAB_LOSS_BACKWARD)
    dx, dw = torch.zeros_like(c.x), torch.zeros_like(c.w)
    g = lambda x=c.x, w=c.w, t=c.t, s=lse, d=c.d, dx=dx, dw=dw, ws=ws, n=n: \
        B.mok_vocab_loss_backward(c.cfg, x, w, t, s, d, dx, dw, ws, n)  # noqa: E731
    assert g() == B.MOK_OK and g(dx=None) == B.MOK_OK and g(dw=None) == B.MOK_OK
    assert g(dx=None, dw=None) == bad
    assert g(dx=c.x) == bad and g(dw=c.w) == bad and g(dx=c.w) == bad and g(dw=c.x) == bad
    for k in ("x", "w", "t", "s", "d"):
        assert g(**{k: None}) == bad
    for k in ("x", "w", "t", "s", "d", "dx", "dw"):
        assert g(**{k: loss.data_ptr() + 8}) == bad
    assert g(ws=None) == nows and g(n=n - 1) == nows and g(ws=ws[8:]) == nows
    assert device_ok()
