"""The router, the norm and the vocabulary loss at corners that the other files do not reach. References
and tolerances: those of test_gpu_router.py, test_gpu_norm.py and test_gpu_vocab_loss.py unless said."""
import math

import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B
import test_gpu_norm
import test_gpu_router
import test_gpu_vocab_loss

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def device_ok():
    st, dev = B.mok_read_device_status()
    B.mok_clear_device_status()
    return (st, dev) == (B.MOK_OK, B.MOK_OK)


# ------------------------------------------------------------------------------- router

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [dict(E=64), dict(E=200), dict(E=128, G=2, keep=1)], ids=str)
def test_ties_that_are_better_than_a_run_of_close_scores(score, kw):
    """More than 32 close scores, the last of them in order ties that are better than the first."""
    torch = _t()
    E = kw["E"]
    for low, high, b in ((20.0, 21.0, 0.0), (1.0, 1.0 + 2.0 ** -23, 0.25)):
        if low == 20.0 and score == "softmax":
            continue  # far apart there
        for first in (31, 5, 32):
            logits = torch.full((3, E), low, device="cuda")
            logits[:, first:] = high
            logits[1, -1] = low
            logits[2, :2] = high
            bias = torch.full((E,), b, device="cuda")
            for K in (1, 8, 31, 32):
                test_gpu_router.check_forward(test_gpu_router.Case(
                    T=3, K=K, score=score, top=2, bias=bias, logits=logits, **kw))


@pytest.mark.parametrize("kw", [dict(E=16, G=4, keep=2, K=5), dict(E=64, G=8, keep=3, K=20)], ids=str)
def test_groups_whose_sum_of_two_passes_32_bits(kw):
    """Biases near the lowest value: two of them are no fp32 number, and still before a masked group."""
    torch = _t()
    E, per = kw["E"], kw["E"] // kw["G"]
    gen = torch.Generator("cuda").manual_seed(3)
    logits = torch.randn(4, E, device="cuda", generator=gen)
    logits[0, :per], logits[1, per:2 * per], logits[2, :2 * per] = -math.inf, -math.inf, -math.inf
    bias = torch.full((E,), -3.0e38, device="cuda")
    bias[-per:] = 0.0
    for score in ("softmax", "sigmoid"):
        test_gpu_router.check_forward(test_gpu_router.Case(T=4, score=score, top=2, bias=bias,
                                                           logits=logits, **kw))


@pytest.mark.parametrize("E", [8, 64])
def test_no_tokens_leave_the_gradient_alone(E):
    torch = _t()
    cfg = B.make_router(0, E, 2)
    d = torch.full((4, E), 7.0, device="cuda")
    i, w = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")
    l = torch.zeros(4, E, device="cuda")
    for dsum in (None, torch.ones(E, device="cuda")):
        assert B.mok_router_backward(cfg, l, i, w, dsum, d) == B.MOK_OK
    assert bool((d == 7).all()) and device_ok()


# --------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [64, 4096])
def test_gradient_of_rows_of_one_value_with_a_small_eps(kind, H):
    """rstd is 1e20 and its square no fp32 number; n is 0, so dx = rstd (g - mean(g))."""
    torch = _t()
    c = test_gpu_norm.Case(R=3, H=H, kind=kind, x="fp32", y="fp32", res=False, eps=1e-40)
    c.x[:, :H] = 0.0
    _, y, mean, rstd = c.forward()
    dy = c.rand(c.ld_y, c.yd)
    dx, dw, db = c.backward(c.x, mean, rstd, dy, None)
    g = c.live(dy) * c.w.double()
    want = g - (g.mean(1, keepdim=True) if kind == "layer" else 0.0)
    want = want * rstd[:3].double()[:, None]
    size = rstd[:3].double()[:, None] * (g.abs() + g.abs().mean(1, keepdim=True))
    assert bool(((c.live(dx) - want).abs() <= 2.0 ** -16 * size).all())
    assert bool((dw[:H] == 0).all()) and device_ok()


# --------------------------------------------------------------------- vocabulary loss

def test_targets_past_the_vocabulary_without_a_loss():
    torch = _t()
    for R in (40, 300):
        c = test_gpu_vocab_loss.Case(R=R, H=100, V=500, ignore=0.0)
        loss, lse = c.forward()
        assert device_ok()
        c.t[5] = 500
        out = torch.full_like(lse, 7.0)
        ws, n = c.ws(B.MOK_VOCAB_LOSS_FORWARD)
        B.check(B.mok_vocab_loss_forward(c.cfg, c.x, c.w, c.t, None, out, ws, n))
        assert torch.equal(out, lse)
        assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()


@pytest.mark.parametrize("R", [40, 520])
@pytest.mark.parametrize("H", [4104, 1 << 18])
def test_logits_of_long_rows(R, H):
    """Logits of some 300 out of H terms of one sign. A tensor-core sum loses at most 2^-23 of what it has
    with every 16 terms, so up to 4096 terms, which are what is summed at a time, 4096 / 32 of that: 2^-16;
    adding the H / 4096 parts loses 2^-24 each of what they have so far. dl is off by its logit's error (and as
    test_gpu_vocab_loss.py says)."""
    torch = _t()
    V = 60
    c = test_gpu_vocab_loss.Case(R=R, H=H, V=V, ignore=0.1)
    c.x[:R, :H] = 0.5 + torch.rand(R, H, device="cuda", generator=c.gen)
    c.w[:V, :H] = (0.5 + torch.rand(V, H, device="cuda", generator=c.gen)) * (300.0 / H)
    x, w = c.x[:R, :H].double(), c.w[:V, :H].double()
    l = x @ w.T
    lse = torch.logsumexp(l, 1)
    d = torch.where(c.t >= 0, c.d.double(), 0.0)[:, None]
    dl = torch.exp(l - lse.float().double()[:, None]) * d
    err = dl.abs() * (l.abs() * (2.0 ** -16 + H / 4096 / 2 * 2.0 ** -24) + 2.0 ** -16)
    dl.scatter_add_(1, c.t.long().clamp(min=0)[:, None], -d)
    err = err + (2.0 ** -8 if R > 512 else 2.0 ** -16) * dl.abs()
    dx, dw = c.backward(lse.float())
    assert device_ok()
    for got, want, tol in ((dx[:R, :H], dl @ w, err @ w.abs()), (dw[:V, :H], dl.T @ x, err.T @ x.abs())):
        tol = tol + 2.0 ** -18 * (dl.abs() @ w.abs() if want.shape[0] == R else dl.T.abs() @ x.abs())
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
        assert bool(((got.double() - want).abs() <= tol).all())


def test_many_rows_of_one_target_and_of_none():
    torch = _t()
    for kw in (dict(R=3000, H=264, V=2300), dict(R=9000, H=40, V=2), dict(R=600, H=64, V=700, piece=256)):
        c = test_gpu_vocab_loss.Case(ignore=0.0, std=1.0, **kw)
        for at in (0, c.V - 1):
            c.t.fill_(at)
            test_gpu_vocab_loss.check_backward(c)
        c.t.fill_(-1)
        _, dx, dw = test_gpu_vocab_loss.check_backward(c)
        assert not bool(dx[:c.R, :c.H].any()) and not bool(dw[:c.V, :c.H].any())


def test_many_rows_in_place_of_stale_gradients():
    """dW and dx hold anything, NaN among it, before the call; the same bits each time."""
    torch = _t()
    for kw in (dict(V=3000), dict(V=3000, piece=512), dict(V=60)):
        c = test_gpu_vocab_loss.Case(R=700, H=100, ignore=0.2, **kw)
        lse, dx, dw = test_gpu_vocab_loss.check_backward(c)
        for fill in (float("nan"), float("inf"), 0.0):
            a, b = torch.full_like(dx, fill), torch.full_like(dw, fill)
            ws, n = c.ws(B.MOK_VOCAB_LOSS_BACKWARD)
            B.check(B.mok_vocab_loss_backward(c.cfg, c.x, c.w, c.t, lse, c.d, a, b, ws, n))
            assert torch.equal(a[:700, :100], dx[:700, :100])
            assert torch.equal(b[:c.V, :100], dw[:c.V, :100])


def gradients64(c, lse):
    """x, W, dl and the gradients in 64 bits."""
    torch = _t()
    x, w = c.x[:c.R, :c.H].double(), c.w[:c.V, :c.H].double()
    d = torch.where(c.t >= 0, c.d.double(), 0.0)[:, None]
    a = lse.double()[:, None]
    dl = torch.exp(x @ w.T - a) * d * (1 + 2 * c.z * a)
    dl.scatter_add_(1, c.t.long().clamp(min=0)[:, None], -d)
    return x, w, dl, dl @ w, dl.T @ x


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("grad, R, H, V, piece, most", [
    # three planes leave 2^-24 of a value, two 2^-16: 2.7e-6 of the norm at these sizes. What remains are
    # sums of 1000 to 5003 terms in runs of 512 and the exponent's rounding
    ("fp32", 1001, 1000, 5003, 0, 1.5e-6), ("fp32", 300, 2100, 1500, 0, 2e-6), ("fp32", 700, 200, 3000, 0, 2e-6),
    ("fp32", 700, 200, 3000, 256, 2e-6),  # in pieces of 256 entries
    # logits of few entries, which share their errors among few: 32 steps of 16 terms lose 2^-24 each in the mean, of
    # 1.5, a third of which is left of dl's norm: 5e-7, beside 7e-7 of the sums. (One run of 1024: 1.4e-6)
    ("fp32", 6251, 1044, 90, 0, 1.1e-6), ("fp32", 2000, 1000, 64, 0, 1.1e-6),
    # rounding to bf16 is off by half a step at most and evenly so: 2^-8 / sqrt(3) of a value just above a power of
    # two, half that just below, 1.66e-3 in the mean of squares over evenly spread logarithms. One plane adds as much
    # again, which is 2.35e-3 in all
    ("bf16", 3, 1000, 5003, 0, 1.8e-3), ("bf16", 300, 1000, 5003, 0, 1.8e-3), ("bf16", 512, 1000, 5003, 0, 1.8e-3),
    ("bf16", 513, 1000, 5003, 0, 2.6e-3), ("bf16", 4096, 512, 8000, 0, 2.6e-3),
])
def test_gradients_in_norm(grad, R, H, V, piece, most):
    torch = _t()
    c = test_gpu_vocab_loss.Case(R=R, H=H, V=V, z=1e-4, grad=grad, std=1.5, ignore=0.1 if R > 3 else 0.0,
                                 piece=piece)
    lse = torch.logsumexp(c.x[:R, :H].double() @ c.w[:V, :H].double().T, 1).float()
    dx, dw = c.backward(lse)
    _, _, _, wx, ww = gradients64(c, lse)
    got = relative(dx[:R, :H], wx), relative(dw[:V, :H], ww)
    print("relative errors of dx and dW", got)
    assert max(got) <= most and device_ok()


@pytest.mark.parametrize("kw", [dict(V=3000), dict(V=3000, piece=512), dict(V=20000, z=1e-3)], ids=str)
def test_many_rows_of_which_few_take_part(kw):
    """More than 512 rows are rounded to one bf16 value each, live or not: a row of dx is off by at most 2^-8 of
    its dl's terms and half a step of itself. The live rows alone, as a call of few rows, have two values."""
    torch = _t()
    c = test_gpu_vocab_loss.Case(R=4096, H=136, ignore=0.0, std=1.0, **kw)
    live = torch.tensor([0, 1, 255, 256, 1000, 2047, 2048, 4000, 4094, 4095], device="cuda")
    dead = torch.ones(4096, dtype=torch.bool, device="cuda")
    dead[live] = False
    c.t[dead], c.d[dead] = -1, float("nan")
    _, dx, dw = test_gpu_vocab_loss.check_backward(c)
    assert not bool(dx[dead][:, :136].any())
    few = test_gpu_vocab_loss.Case(R=10, H=136, ignore=0.0, std=1.0, **kw)
    few.x, few.w, few.t, few.d = c.x[live].contiguous(), c.w, c.t[live].contiguous(), c.d[live].contiguous()
    _, fx, fw = test_gpu_vocab_loss.check_backward(few)
    assert relative(dx[live][:, :136].double(), fx[:10, :136].double()) <= 2.0 ** -7
    assert relative(dw[:c.V, :136].double(), fw[:c.V, :136].double()) <= 2.0 ** -7
