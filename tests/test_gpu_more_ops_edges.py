"""The router, the norm and the vocabulary loss at the edges of what they take: masks of the types'
lowest values, arrays past 2^31 elements, rows of one element, strides of wider arrays, runs of close
scores longer than a warp. References and tolerances: those of test_gpu_router.py, test_gpu_norm.py and
test_gpu_vocab_loss.py, at the rows that are looked at."""
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


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kw", [dict(), dict(renorm=False), dict(score="sigmoid"),
                                dict(score="sigmoid", bias=True, G=4, keep=2, top=2)], ids=str)
def test_masks_of_the_lowest_value(dtype, kw):
    """Finite, so not masked: scores of 0, chosen after all others and before logits of -inf; rows of
    nothing else share their weights evenly."""
    torch = _t()
    low = torch.finfo(torch.float32 if dtype == "fp32" else torch.bfloat16).min
    gen = torch.Generator("cuda").manual_seed(2)
    logits = torch.randn(60, 40, device="cuda", generator=gen)
    logits[torch.rand(60, 40, device="cuda", generator=gen) < 0.85] = low
    logits[torch.rand(60, 40, device="cuda", generator=gen) < 0.1] = -math.inf
    logits[7], logits[8, :], logits[8, 3:] = low, -math.inf, low
    if "bias" in kw:
        kw = dict(kw, bias=torch.randn(40, device="cuda", generator=gen))
    c = test_gpu_router.Case(T=60, E=40, K=6, dtype=dtype, logits=logits, **kw)
    idx, w = test_gpu_router.check_forward(c)
    if kw.get("renorm", True) and "G" not in kw:
        assert bool(((w[42:48] - 1 / 6).abs() < 1e-6).all())
    dw = torch.randn(60, 6, device="cuda", generator=gen)
    got = test_gpu_router.backward(c, idx[:360].view(60, 6).contiguous(), dw, None)
    ref, mag = test_gpu_router.gradient64(c, idx[:360].view(60, 6).long(), dw.double(), None)
    tol = 2.0 ** -14 * mag + 1e-36
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((got[:, :40].double() - ref).abs() <= tol).all()) and device_ok()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [40, 200])
def test_long_runs_of_close_scores(score, E):
    """More experts than a warp has lanes whose scores 32 bits cannot tell apart, some of them ties."""
    torch = _t()
    gen = torch.Generator("cuda").manual_seed(E)
    step = torch.argsort(torch.rand(40, E, device="cuda", generator=gen), 1) // 2  # pairs of ties
    logits = 1.0 + step * 2.0 ** -23
    same = torch.full((E,), 0.25, device="cuda")
    for bias in (same, same + (torch.arange(E, device="cuda") % 3) * 2.0 ** -25):
        for K in (1, 7, 31, 32):
            test_gpu_router.check_forward(test_gpu_router.Case(T=40, E=E, K=K, score=score, bias=bias,
                                                               logits=logits))
    # all alike but one that is a hair better, at the end
    logits = torch.zeros(5, E, device="cuda")
    logits[:, -1] = 2.0 ** -24
    c = test_gpu_router.Case(T=5, E=E, K=3, score=score, bias=same, logits=logits)
    idx, _ = test_gpu_router.check_forward(c)
    assert idx[:3].tolist() == [E - 1, 0, 1]


def test_router_past_2_31_elements():
    torch = _t()
    T, E, K = 2_100_000, 1024, 4
    logits = torch.zeros(T, E, device="cuda")
    live = torch.randn(64, E, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    logits[-64:] = live
    cfg = B.make_router(T, E, K, renormalize=False)
    idx = torch.empty(T * K, dtype=torch.int32, device="cuda")
    w, counts, sums = torch.empty(T * K, device="cuda"), idx.new_empty(E), torch.empty(E, device="cuda")
    n = B.mok_router_workspace_size(cfg)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.mok_router_forward(cfg, logits, None, idx, w, counts, sums, ws, n))
    small = test_gpu_router.Case(T=64, E=E, K=K, renorm=False, logits=live)
    ref, rw, _, _ = small.forward()
    assert torch.equal(idx[-64 * K:], ref[:64 * K]) and torch.equal(w[-64 * K:], rw[:64 * K])
    assert idx[:4].tolist() == [0, 1, 2, 3] and int(counts.sum()) == T * K
    # T - 64 rows of 1 / 1024: a partial sum of 900 exact terms, 456 of them
    assert bool(((sums - (T - 64) / E).abs() <= 64.0 + 1e-5 * T / E).all())
    d = torch.ones(T, K, device="cuda")
    B.check(B.mok_router_backward(cfg, logits, idx, d, None, logits))
    g = test_gpu_router.backward(small, ref[:64 * K].contiguous(), d[-64:], None)
    assert torch.equal(logits[-64:], g[:64]) and device_ok()


def test_norm_past_2_31_elements():
    torch = _t()
    R, H = 132_000, 16_384
    c = test_gpu_norm.Case(R=64, H=H, res=False)
    x = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    x[-64:] = c.x
    cfg = B.make_norm(R, H)
    y, mean, rstd = torch.empty_like(x), torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    B.check(B.mok_norm_forward(cfg, x, None, c.w, c.b, None, y, mean, rstd))
    _, want, m, r = c.forward()
    assert torch.equal(y[-64:], want) and torch.equal(mean[-64:], m[:64]) and torch.equal(rstd[-64:], r[:64])
    assert torch.equal(y[:1], y[R // 2:R // 2 + 1])
    dy = torch.zeros_like(x)
    dy[-64:] = c.rand(H, c.yd)
    n = B.mok_norm_workspace_size(cfg)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    small = c.backward(c.x, m, r, dy[-64:].contiguous(), None)
    B.check(B.mok_norm_backward(cfg, x, mean, rstd, c.w, dy, None, y, dw, db, ws, n))
    assert torch.equal(y[-64:], small[0]) and not bool(y[:-64].any())
    # the other rows add zeros, but the 64 rows meet in another order: 64 additions of 2^-24 each, twice
    d = dy[-64:].double()
    norm = (c.x[:64].double() - m[:64].double()[:, None]) * r[:64].double()[:, None]
    for a, b, mag in ((dw, small[1][:H], (d * norm).abs().sum(0)), (db, small[2][:H], d.abs().sum(0))):
        assert bool(((a - b).abs().double() <= 2.0 ** -17 * mag + 1e-30).all())
    assert device_ok()


def test_vocab_loss_past_2_31_elements():
    """dl of the whole vocabulary in one piece of 2.3e9 values."""
    torch = _t()
    R, H, V = 33_024, 64, 70_144
    c = test_gpu_vocab_loss.Case(R=R, H=H, V=V, piece=V, ignore=0.0)
    loss, lse = c.forward()
    pick = torch.tensor([0, 1, R // 2, R - 2, R - 1], device="cuda")
    x, w = c.x.double(), c.w.double()
    l = x[pick] @ w.T
    ref = torch.logsumexp(l, 1)
    el = test_gpu_vocab_loss.dot_rel(H) * (x[pick].abs() @ w.abs().T).amax(1)
    assert bool(((lse[pick].double() - ref).abs() <= el + 2.0 ** -15).all())
    c.d.fill_(1.0)
    dx, dw = c.backward(lse[:R].contiguous())
    p = torch.exp(l - lse[pick].double()[:, None])
    p.scatter_add_(1, c.t[pick].long()[:, None], -torch.ones(5, 1, device="cuda", dtype=torch.float64))
    tol = 2.0 ** -6 * (p.abs() @ w.abs())
    assert bool(((dx[pick].double() - p @ w).abs() <= tol).all())
    cols = torch.tensor([0, 255, 256, V - 257, V - 1], device="cuda")
    dl = torch.exp(x @ w[cols].T - lse[:R].double()[:, None])
    dl -= (c.t.long()[:, None] == cols[None, :]).double()
    tol = 2.0 ** -6 * (dl.T.abs() @ x.abs())
    assert bool(((dw[cols].double() - dl.T @ x).abs() <= tol).all())
    assert device_ok()


def test_columns_of_wider_arrays():
    """Rows that lie in other arrays, whose other columns are left alone: by the helpers, whose rows are
    up8(H) apart, only where that is the array's stride; by the entry points for any stride of theirs."""
    torch = _t()
    wide = torch.full((50, 200), 7.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 64:164] = torch.randn(50, 100, device="cuda").to(torch.bfloat16)
    x = wide[:, 64:164]
    cfg = B.make_norm(50, 100, ld_x=200, ld_y=104)
    y = torch.zeros(50, 104, device="cuda", dtype=torch.bfloat16)
    B.check(B.mok_norm_forward(cfg, x, None, None, None, None, y))
    ref = torch.nn.functional.layer_norm(x.double(), (100,))
    assert float((y[:, :100].double() - ref).abs().max()) <= 2.0 ** -7 * 4
    B.check(B.mok_norm_forward(B.make_norm(50, 100, ld_x=200, ld_y=200), x, None, None, None, None, x))
    assert torch.equal(x, y[:, :100]) and bool((wide[:, :64] == 7).all()) and bool((wide[:, 164:] == 7).all())
    assert device_ok()


@pytest.mark.parametrize("K", [1, 32])
def test_one_token_and_one_expert_each_way(K):
    for E in (K, 1024):
        for score in ("softmax", "sigmoid"):
            test_gpu_router.check_forward(test_gpu_router.Case(T=1, E=E, K=K, score=score, bias=True))
            test_gpu_router.check_forward(test_gpu_router.Case(T=1, E=E, K=K, score=score, renorm=False))
