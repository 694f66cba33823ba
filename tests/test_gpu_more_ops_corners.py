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
