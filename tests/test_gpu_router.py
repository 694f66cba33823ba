"""The router against its definition in 64 bits: ids, loads and the bias's step to the bit, weights,
score sums and gradients within tolerances.

Tolerances (derived): an fp32 score is within 96 x 2^-24 of itself plus its exponent's rounding,
2^-24 |x|, |x| < 160 here: 2^-16 in all, of its own value; a weight (one quotient and a sum of at
most 32 more) 2^-15; a gradient 2^-14 of the sum of its terms' magnitudes; score sums 2^-16 and one
rounding a partial sum (at most 8 tokens a warp and 8 + 38 + 16 partial sums below 6000 tokens):
2^-15 of themselves. bf16 gradients add 2^-8 of a value."""
import math

import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu
INF = math.inf


def _t():
    import torch
    return torch


def device_ok():
    st, dev = B.mok_read_device_status()
    B.mok_clear_device_status()
    return (st, dev) == (B.MOK_OK, B.MOK_OK)


def scores64(l, score):
    """(s, 1 - s as the sigmoid's slope needs it), masked experts 0."""
    torch = _t()
    if score == "sigmoid":
        return torch.sigmoid(l), torch.sigmoid(-l)
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -INF, 0.0, top))
    s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    return s, 1 - s


def choice64(l, bias, K, score, G, keep, top):
    torch = _t()
    T, E = l.shape
    off = torch.isneginf(l)
    c = scores64(l, score)[0]
    if bias is not None:
        c = c + bias.double()
    by = torch.where(off, -INF, c).reshape(T, G, E // G).sort(dim=2, descending=True)[0]
    total = by[:, :, 0]
    if top == 2 and E // G > 1:
        total = total + torch.where(torch.isneginf(by[:, :, 1]), 0.0, by[:, :, 1])
    rank = total.sort(dim=1, descending=True, stable=True)[1][:, :keep]
    kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, rank, True)
    key = torch.where(off, -1e300, c if bias is not None else l)
    key = torch.where(kept.repeat_interleave(E // G, 1), key, -INF)
    return key.sort(dim=1, descending=True, stable=True)[1][:, :K]


class Case:
    """Inputs of one configuration; logits have guard columns (NaN) that must not be read, outputs
    guards that must not be written."""

    def __init__(self, T=50, E=64, K=4, score="softmax", G=1, keep=1, top=1, renorm=True, scale=1.0,
                 dtype="fp32", bias=False, masked=0.0, extra=0, std=1.0, seed=0, logits=None):
        torch = _t()
        self.__dict__.update(T=T, E=E, K=K, score=score, G=G, keep=keep, top=top, renorm=renorm,
                             scale=scale)
        self.dt = torch.float32 if dtype == "fp32" else torch.bfloat16
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen = gen
        self.ld = E + extra
        self.buf = torch.full((max(T, 1), self.ld), float("nan"), device="cuda", dtype=self.dt)
        live = torch.randn(T, E, device="cuda", generator=gen) * std if logits is None else logits
        if masked:
            live = live.masked_fill(torch.rand(T, E, device="cuda", generator=gen) < masked, -INF)
            live[::7] = -INF
        self.buf[:T, :E] = live.to(self.dt)
        self.l = self.buf[:T, :E].double()
        self.bias = None
        if bias is True:
            self.bias = torch.randn(E, device="cuda", generator=gen) * 0.1
        elif bias is not False:
            self.bias = bias
        self.cfg = B.make_router(T, E, K, B.MOK_SCORE_SIGMOID if score == "sigmoid"
                                 else B.MOK_SCORE_SOFTMAX, G, keep, top, renorm, scale,
                                 B.MOK_DTYPE_F32 if dtype == "fp32" else B.MOK_DTYPE_BF16, self.ld)
        assert B.mok_check_router_config(self.cfg) == B.MOK_OK

    def forward(self, load=True, stream=None):
        torch = _t()
        n = self.T * self.K
        idx = torch.full((n + 3,), -7, dtype=torch.int32, device="cuda")
        w = torch.full((n + 3,), 7.0, device="cuda")
        counts = torch.full((self.E + 3,), -7, dtype=torch.int32, device="cuda") if load else None
        sums = torch.full((self.E + 3,), 7.0, device="cuda") if load else None
        size = B.mok_router_workspace_size(self.cfg)
        assert size > 0
        ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
        B.check(B.mok_router_forward(self.cfg, self.buf, self.bias, idx, w, counts, sums, ws, size,
                                     stream))
        self._keep = ws
        return idx, w, counts, sums

    def weights64(self, idx):
        """Weights of the chosen ids, as shares of logarithms where they are renormalised."""
        torch = _t()

        def shares(v):  # less the largest first: a sum's logarithm is lost beside 1e38
            top = v.amax(1, keepdim=True)
            v = v - torch.where(top == -INF, 0.0, top)
            return torch.where(top == -INF, -INF, v - torch.logsumexp(v, 1, keepdim=True))

        ls = -torch.logaddexp(torch.zeros_like(self.l), -self.l) if self.score == "sigmoid" \
            else shares(self.l)
        ls = ls.gather(1, idx)
        return torch.exp(shares(ls) if self.renorm else ls)


def check_forward(c):
    torch = _t()
    idx, w, counts, sums = c.forward()
    assert device_ok()
    n = c.T * c.K
    assert bool((idx[n:] == -7).all()) and bool((w[n:] == 7).all())
    assert bool((counts[c.E:] == -7).all()) and bool((sums[c.E:] == 7).all())
    ref = choice64(c.l, c.bias, c.K, c.score, c.G, c.keep, c.top)
    got = idx[:n].view(c.T, c.K).long()
    assert torch.equal(got, ref)
    want = c.scale * c.weights64(ref)
    assert bool(((w[:n].view(c.T, c.K).double() - want).abs() <= 2.0 ** -15 * want + 1e-37).all())
    assert torch.equal(counts[:c.E].long(), torch.bincount(ref.reshape(-1), minlength=c.E))
    total = scores64(c.l, c.score)[0].sum(0)
    assert bool(((sums[:c.E].double() - total).abs() <= 2.0 ** -15 * total + 1e-37 * c.T).all())
    return idx, w


CASES = [
    dict(T=1, E=1, K=1),
    dict(T=1, E=512, K=10),
    dict(T=33, E=32, K=32),
    dict(T=100, E=60, K=6, renorm=False, dtype="bf16", masked=0.2, extra=4),
    dict(T=100, E=33, K=7, score="sigmoid", extra=3, scale=2.5),
    dict(T=5000, E=512, K=10, extra=8),
    dict(T=700, E=1024, K=16, renorm=False),
    dict(T=3000, E=256, K=8, score="sigmoid", G=8, keep=4, top=2, scale=2.5, bias=True),
    dict(T=300, E=256, K=8, score="sigmoid", G=8, keep=4, top=2, dtype="bf16", bias=True),
    dict(T=300, E=256, K=8, score="softmax", G=8, keep=3, top=1, bias=True, masked=0.3),
    dict(T=300, E=160, K=6, score="softmax", G=8, keep=3, top=1, renorm=False),
    dict(T=200, E=160, K=6, score="softmax", G=8, keep=3, top=2, masked=0.6),
    dict(T=100, E=1020, K=20, score="sigmoid", G=17, keep=5, top=2, bias=True),
    dict(T=100, E=1023, K=11, G=3, keep=2, top=2, score="sigmoid"),
    dict(T=100, E=32, K=5, G=32, keep=6, top=2, bias=True),
    dict(T=100, E=64, K=2, G=32, keep=1, top=1, bias=True, score="sigmoid"),
    dict(T=100, E=96, K=12, score="sigmoid", masked=0.95, bias=True),
    dict(T=64, E=96, K=12, score="sigmoid", std=40.0),
    dict(T=64, E=96, K=12, score="softmax", std=40.0, renorm=False),
    dict(T=3000, E=128, K=4, bias=True),
    dict(T=2000, E=60, K=6, bias=True, dtype="bf16", renorm=False),
    dict(T=700, E=5, K=2, score="sigmoid", bias=True),
    # few experts: rows that a thread holds, in all its sizes, and one past them
    dict(T=1, E=2, K=1, score="sigmoid", renorm=False),
    dict(T=700, E=8, K=2),
    dict(T=700, E=8, K=4, dtype="bf16", renorm=False, scale=2.5),
    dict(T=70, E=4, K=4, masked=0.5),
    dict(T=129, E=7, K=3, extra=2, masked=0.5),
    dict(T=300, E=16, K=4, extra=4, dtype="bf16", masked=0.3),
    dict(T=300, E=13, K=3, score="sigmoid", dtype="bf16", std=30.0),
    dict(T=1000, E=16, K=4, score="sigmoid", masked=0.8),
    dict(T=1000, E=16, K=4, renorm=False, std=20.0),
    dict(T=300, E=15, K=4, extra=1),
    dict(T=300, E=16, K=5),
    dict(T=300, E=17, K=4),
    dict(T=250001, E=8, K=2),
]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_forward(kw):
    check_forward(Case(**kw))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
def test_close_scores_are_told_apart(score, G):
    """Logits one unit in the last place apart, whose fp32 scores are the same number, in random
    order, with biases that differ by as little: every choice is a close call."""
    torch = _t()
    gen = torch.Generator("cuda").manual_seed(5)
    T, E = 64, 64
    step = torch.argsort(torch.rand(T, E, device="cuda", generator=gen), 1)
    logits = 2.0 + step * 2.0 ** -22
    for bias in (torch.zeros(E, device="cuda"),
                 0.5 + torch.randint(0, 3, (E,), device="cuda", generator=gen) * 2.0 ** -24):
        c = Case(T=T, E=E, K=8, score=score, G=G, keep=max(1, G // 2), top=2, bias=bias,
                 logits=logits)
        check_forward(c)
    check_forward(Case(T=T, E=E, K=8, score=score, G=G, keep=max(1, G // 2), top=2, logits=logits))


def test_equal_logits_go_to_the_lower_id():
    torch = _t()
    for kw in (dict(), dict(bias=torch.zeros(48, device="cuda")), dict(G=4, keep=2, top=2),
               dict(G=4, keep=2, top=1, score="sigmoid")):
        logits = torch.zeros(9, 48, device="cuda")
        logits[3, 20:] = 1.0
        logits[4] = -0.0
        check_forward(Case(T=9, E=48, K=10, logits=logits, **kw))


def test_shares_of_scores_that_round_to_nothing():
    """Sigmoid scores of logits around -200 are below any fp32 number; their shares are not."""
    torch = _t()
    logits = -200.0 + torch.randn(20, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for score in ("sigmoid", "softmax"):
        c = Case(T=20, E=40, K=4, score=score, logits=logits)
        idx, w, _, _ = c.forward()
        want = c.weights64(idx[:80].view(20, 4).long())
        assert bool(((w[:80].view(20, 4).double() - want).abs() <= 2.0 ** -15 * want).all())
        assert float(want.min()) > 1e-3


def test_without_loads_and_repeated():
    torch = _t()
    c = Case(T=1500, E=256, K=8, score="sigmoid", G=8, keep=4, top=2, bias=True)
    idx, w, counts, sums = c.forward()
    for _ in range(3):
        again = c.forward()
        for a, b in zip((idx, w, counts, sums), again):
            assert torch.equal(a, b)
    i2, w2, _, _ = c.forward(load=False)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i3, w3, c3, s3 = c.forward(stream=s)
    s.synchronize()
    assert torch.equal(idx, i3) and torch.equal(sums, s3) and device_ok()


@pytest.mark.parametrize("E, K", [(16, 4), (64, 8)])
def test_nan_logits_give_ids_in_range_each_once(E, K):
    torch = _t()
    for kw in (dict(), dict(bias=True), dict(score="sigmoid", G=2, keep=1, top=2, bias=True)):
        logits = torch.randn(40, E, device="cuda")
        logits[::2, 5] = float("nan")
        logits[::3] = float("nan")
        logits[1::3, 9:12] = INF
        logits[4, :] = -float("nan")
        c = Case(T=40, E=E, K=K, logits=logits, **kw)
        idx = c.forward()[0][:40 * K].view(40, K)
        assert bool(((idx >= 0) & (idx < E)).all()) and device_ok()
        for row in idx.tolist():
            assert len(set(row)) == K


def test_no_tokens():
    torch = _t()
    c = Case(T=0, E=16, K=2)
    idx, w, counts, sums = c.forward()
    assert counts[:16].tolist() == [0] * 16 and sums[:16].tolist() == [0.0] * 16
    d = torch.full((16,), 7.0, device="cuda")
    assert B.mok_router_backward(c.cfg, None, None, None, None, None) == B.MOK_OK
    assert bool((d == 7).all()) and device_ok()


# ------------------------------------------------------------------------------- gradient

def gradient64(c, idx, dw, dsum):
    """(gradient, sum of its terms' magnitudes)."""
    torch = _t()
    s, rest = scores64(c.l, c.score)
    w = c.weights64(idx)
    live = ~torch.isneginf(c.l)
    dw = torch.where(live.gather(1, idx), dw, 0.0)
    d = dw - (dw * w).sum(1, keepdim=True) if c.renorm else dw
    m = dw.abs() + (dw.abs() * w).sum(1, keepdim=True) if c.renorm else dw.abs()
    g, mag = torch.zeros_like(c.l), torch.zeros_like(c.l)
    if c.score == "sigmoid" or c.renorm:
        f = c.scale * w * (rest.gather(1, idx) if c.score == "sigmoid" else 1.0)
        g.scatter_add_(1, idx, f * d)
        mag.scatter_add_(1, idx, f * m)
    else:
        ds = torch.zeros_like(c.l).scatter_add_(1, idx, c.scale * dw)
        g += s * (ds - (s * ds).sum(1, keepdim=True))
        mag += s * (ds.abs() + (s * ds.abs()).sum(1, keepdim=True))
    if dsum is not None:
        e = dsum.double()[None, :]
        if c.score == "sigmoid":
            g += e * s * rest
            mag += e.abs() * s * rest
        else:
            g += s * (e - (s * e).sum(1, keepdim=True))
            mag += s * (e.abs() + (s * e.abs()).sum(1, keepdim=True))
    return torch.where(live, g, 0.0), mag


def backward(c, idx, dw, dsum, in_place=False):
    torch = _t()
    out = c.buf.clone() if in_place else torch.full_like(c.buf, 7.0)
    B.check(B.mok_router_backward(c.cfg, out if in_place else c.buf, idx, dw, dsum, out))
    return out


@pytest.mark.parametrize("sums", [False, True])
@pytest.mark.parametrize("kw", CASES, ids=str)
def test_backward(kw, sums):
    torch = _t()
    c = Case(**kw)
    idx = choice64(c.l, c.bias, c.K, c.score, c.G, c.keep, c.top)
    dw = torch.randn(c.T, c.K, device="cuda", generator=c.gen)
    dsum = torch.randn(c.E, device="cuda", generator=c.gen) * 0.3 if sums else None
    ids = idx.to(torch.int32)
    got = backward(c, ids, dw, dsum)
    assert device_ok()
    ref, mag = gradient64(c, idx, dw.double(), dsum)
    tol = 2.0 ** -14 * mag + 1e-36
    if c.dt == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((got[:c.T, :c.E].double() - ref).abs() <= tol).all())
    assert bool((got[:, c.E:] == 7).all())
    again = backward(c, ids, dw, dsum, in_place=True)
    assert torch.equal(again[:c.T, :c.E], got[:c.T, :c.E])


@pytest.mark.parametrize("kw", [dict(), dict(renorm=False), dict(score="sigmoid"),
                                dict(score="sigmoid", renorm=False, scale=2.5)], ids=str)
def test_gradient_against_differences(kw):
    """The slope along a random direction, from weights and score sums in 64 bits at l +- h: the
    difference quotient is off by h^2 |f'''| / 6 < 1e-9 of the sum of magnitudes at h = 1e-5."""
    torch = _t()
    c = Case(T=11, E=24, K=5, **kw)
    idx = choice64(c.l, None, 5, c.score, 1, 1, 1)
    dw = torch.randn(11, 5, device="cuda", generator=c.gen)
    dsum = torch.randn(24, device="cuda", generator=c.gen)
    got = backward(c, idx.to(torch.int32), dw, dsum)[:11].double()
    step = torch.randn(11, 24, device="cuda", dtype=torch.float64, generator=c.gen)

    def value(l):
        keep, c.l = c.l, l
        v = c.scale * (c.weights64(idx) * dw).sum() + (scores64(l, c.score)[0].sum(0) * dsum).sum()
        c.l = keep
        return v

    h = 1e-5
    slope = (value(c.l + h * step) - value(c.l - h * step)) / (2 * h)
    mag = gradient64(c, idx, dw.double(), dsum)[1]
    assert abs(float((got * step).sum() - slope)) <= 2.0 ** -13 * float((mag * step.abs()).sum())


@pytest.mark.parametrize("E", [16, 20])
def test_bad_and_repeated_ids(E):
    torch = _t()
    c = Case(T=6, E=E, K=3, score="softmax", renorm=False)
    dw = torch.randn(6, 3, device="cuda", generator=c.gen)
    idx = torch.tensor([[0, 1, 2], [3, 3, 3], [5, 15, 5], [-1, 4, E], [7, 8, 9], [2 ** 30, 1, 0]],
                       dtype=torch.int32, device="cuda")
    got = backward(c, idx, dw, None)
    assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
    B.mok_clear_device_status()
    ok = (idx >= 0) & (idx < E)
    ref, mag = gradient64(c, torch.where(ok, idx, 0).long(), torch.where(ok, dw, 0.0).double(), None)
    assert bool(((got.double() - ref).abs() <= 2.0 ** -14 * mag + 1e-36).all())


def test_weights_gradient_of_a_masked_choice_does_not_matter():
    torch = _t()
    for kw in (dict(), dict(renorm=False), dict(score="sigmoid")):
        logits = torch.full((4, 8), -INF, device="cuda")
        logits[0, 3], logits[1, 2], logits[1, 6] = 0.5, 1.0, 2.0
        c = Case(T=4, E=8, K=4, logits=logits, **kw)
        idx = choice64(c.l, None, 4, c.score, 1, 1, 1)
        dw = torch.randn(4, 4, device="cuda")
        bad = torch.where(torch.isneginf(c.l.gather(1, idx)), float("nan"), dw)
        i32 = idx.to(torch.int32)
        assert torch.equal(backward(c, i32, dw, None), backward(c, i32, bad, None))


# ------------------------------------------------------------------------------- the bias

def test_bias_update():
    torch = _t()
    for T, E, K in ((100, 7, 3), (64, 16, 4), (1, 1, 1), (2 ** 30, 1024, 1)):
        cfg = B.make_router(T, E, K)
        g = torch.Generator("cuda").manual_seed(T % 1000)
        mean = T * K / E
        counts = (mean + torch.randint(-2, 3, (E,), device="cuda", generator=g)).floor().to(torch.int32)
        bias = torch.randn(E, device="cuda", generator=g)
        out = torch.full((E + 3,), 7.0, device="cuda")
        B.check(B.mok_router_update_bias(cfg, counts, 0.25, bias, out))
        sign = torch.sign(T * K - counts.long() * E).float()
        assert torch.equal(out[:E], bias + 0.25 * sign) and bool((out[E:] == 7).all())
        B.check(B.mok_router_update_bias(cfg, counts, 0.25, bias, bias))
        assert torch.equal(out[:E], bias) and device_ok()


# ------------------------------------------------------------------------------- refusals

def test_refusals():
    torch = _t()
    c = Case(T=10, E=16, K=2)
    idx, w, counts, sums = c.forward()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    n = B.mok_router_workspace_size(c.cfg)
    f = lambda cfg=c.cfg, l=c.buf, b=None, i=idx, o=w, k=counts, s=sums, a=ws, m=n: \
        B.mok_router_forward(cfg, l, b, i, o, k, s, a, m)  # noqa: E731
    bad, nows = B.MOK_ERR_INVALID_ARG, B.MOK_ERR_WORKSPACE
    assert f() == B.MOK_OK
    assert f(k=None, s=None, a=None, m=0) == B.MOK_OK
    assert f(l=None) == bad and f(i=None) == bad and f(o=None) == bad
    assert f(a=None) == nows and f(m=n - 1) == nows and f(a=ws[1:]) == nows
    assert f(l=c.buf.data_ptr() + 4) == bad and f(b=w.data_ptr() + 4) == bad
    assert f(cfg=B.make_router(10, 16, 17)) == bad
    d = torch.zeros(10, 16, device="cuda")
    g = lambda l=c.buf, i=idx, dw=w, ds=None, o=d: \
        B.mok_router_backward(c.cfg, l, i, dw, ds, o)  # noqa: E731
    assert g() == B.MOK_OK
    for k in ("l", "i", "dw", "o"):
        assert g(**{k: None}) == bad
        assert g(**{k: w.data_ptr() + 4}) == bad
    u = lambda k=counts, r=0.1, b=sums, o=sums: \
        B.mok_router_update_bias(c.cfg, k, r, b, o)  # noqa: E731
    assert u() == B.MOK_OK
    assert u(k=None) == bad and u(b=None) == bad and u(o=None) == bad
    assert u(r=float("nan")) == bad and u(r=INF) == bad
    assert device_ok()
