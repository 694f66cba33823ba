"""The helpers of the router, the norm and the vocabulary loss (no GPU): what they pass on and what
they refuse. The entry points are replaced by recorders; the arrays live on the host."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

torch = pytest.importorskip("torch")
from mixture_experts_layer_deterministic_gb300.buffers import Norm, Router, VocabLoss  # noqa: E402

F32, BF, F16, I32, I64 = (torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.int64)


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments) of the entry points that were reached, which do nothing."""
    seen = []
    for name in ("mok_router_forward", "mok_router_backward", "mok_router_update_bias",
                 "mok_norm_forward", "mok_norm_backward", "mok_vocab_loss_forward",
                 "mok_vocab_loss_backward"):
        monkeypatch.setattr(B, name, lambda *a, _n=name: seen.append((_n, a)) or B.MOK_OK)
    return seen


def refused(calls, f, **kw):
    n = len(calls)
    with pytest.raises(ValueError):
        f(**kw)
    assert len(calls) == n


def variants(good, **wrong):
    for k, values in wrong.items():
        for v in values:
            yield dict(good, **{k: v})


def rows(n, cols, dtype, per=8, cut=True):
    return torch.zeros(n, (cols + per - 1) // per * per, dtype=dtype)[:, :cols] if cut else \
        torch.zeros(n, cols, dtype=dtype)


@pytest.mark.parametrize("dtype,per", [(F32, 4), (BF, 8)])
def test_router(calls, dtype, per):
    r = Router(20, 30, 4, dtype=dtype, device="cpu")
    good = dict(logits=rows(20, 30, dtype, per), idx=torch.zeros(20, 4, dtype=I32),
                topk_w=torch.zeros(20, 4))
    assert r.forward(**good) == (good["idx"], good["topk_w"])
    more = dict(good, bias=torch.zeros(30), counts=torch.zeros(30, dtype=I32),
                score_sum=torch.zeros(30))
    r.forward(**more)
    assert calls[0][1][7] is None and calls[1][1][7].numel() == calls[1][1][8] > 0  # workspace
    for bad in variants(more, logits=(rows(20, 30, F16, per), rows(19, 30, dtype, per),
                                      torch.zeros(20, 30, dtype=dtype), rows(20, 29, dtype, per)),
                        idx=(torch.zeros(20, 4, dtype=I64), torch.zeros(20, 3, dtype=I32)),
                        topk_w=(torch.zeros(20, 4, dtype=BF), torch.zeros(4, 20)[:, ::2]),
                        bias=(torch.zeros(31), torch.zeros(30, dtype=BF)),
                        counts=(torch.zeros(30), torch.zeros(29, dtype=I32)),
                        score_sum=(torch.zeros(60)[::2], torch.zeros(30, dtype=I32))):
        refused(calls, r.forward, **bad)
    back = dict(logits=good["logits"], idx=good["idx"], d_topk_w=torch.zeros(20, 4),
                d_logits=rows(20, 30, dtype, per), d_score_sum=torch.zeros(30))
    assert r.backward(**back) is back["d_logits"]
    for bad in variants(back, d_topk_w=(torch.zeros(20, 4, dtype=BF),),
                        d_logits=(rows(20, 30, F16, per), torch.zeros(20, 30, dtype=dtype)),
                        d_score_sum=(torch.zeros(20),)):
        refused(calls, r.backward, **bad)
    bias = torch.zeros(30)
    assert r.update_bias(more["counts"], 0.1, bias) is bias
    assert calls[-1][1][3] is bias and calls[-1][1][4] is bias
    refused(calls, r.update_bias, counts=torch.zeros(30), rate=0.1, bias=bias)
    refused(calls, r.update_bias, counts=more["counts"], rate=0.1, bias=bias, new_bias=torch.zeros(3))
    with pytest.raises(ValueError):
        Router(20, 30, 4, dtype=F16, device="cpu")
    with pytest.raises(B.MokError):
        Router(20, 30, 31, device="cpu")


@pytest.mark.parametrize("x,y", [(BF, BF), (F32, BF), (F32, F32)])
def test_norm(calls, x, y):
    n = Norm(20, 100, x_dtype=x, y_dtype=y, device="cpu")
    good = dict(x=rows(20, 100, x), weight=torch.zeros(100), y=rows(20, 100, y), bias=torch.zeros(100),
                residual=rows(20, 100, x), h=rows(20, 100, x), mean=torch.zeros(20),
                rstd=torch.zeros(20))
    assert n.forward(**good) is good["y"]
    n.forward(good["x"], None, good["y"])
    packed = lambda dt: torch.zeros(20, 100, dtype=dt)  # noqa: E731 (rows 100 apart, not 104)
    for bad in variants(good, x=(packed(x), rows(19, 100, x), rows(20, 100, F16)),
                        y=(packed(y), rows(20, 99, y), rows(20, 100, F16)),
                        residual=(packed(x),), h=(packed(x), rows(20, 100, F16)),
                        weight=(torch.zeros(99), torch.zeros(100, dtype=BF)),
                        bias=(torch.zeros(200)[::2],), mean=(torch.zeros(19),),
                        rstd=(torch.zeros(20, dtype=torch.float64),)):
        refused(calls, n.forward, **bad)
    back = dict(h=good["h"], weight=good["weight"], dy=good["y"], rstd=good["rstd"], mean=good["mean"],
                dh=rows(20, 100, x), dx=rows(20, 100, x), dw=torch.zeros(100), db=torch.zeros(100))
    assert n.backward(**back) is back["dx"]
    assert calls[-1][1][-3].numel() == calls[-1][1][-2] > 0
    n.backward(**dict(back, dw=None, db=None))
    assert calls[-1][1][-3] is None
    for bad in variants(back, h=(packed(x),), dy=(packed(y),), dh=(packed(x),),
                        dx=(packed(x), rows(20, 100, F16)), dw=(torch.zeros(99),),
                        db=(torch.zeros(100, dtype=BF),), rstd=(torch.zeros(21),)):
        refused(calls, n.backward, **bad)
    with pytest.raises(B.MokError):
        Norm(20, 100, eps=0.0, device="cpu")


@pytest.mark.parametrize("grad", [BF, F32])
def test_vocab_loss(calls, grad):
    v = VocabLoss(20, 100, 50, grad_dtype=grad, device="cpu")
    w = v.weights()
    assert w.shape == (50, 100) and w.stride() == (104, 1) and w.dtype == BF and not bool(w.any())
    good = dict(x=rows(20, 100, BF), w=w, targets=torch.zeros(20, dtype=I32), loss=torch.zeros(20),
                lse=torch.zeros(20))
    assert v.forward(**good) is good["loss"]
    v.forward(**dict(good, loss=None))
    for bad in variants(good, x=(torch.zeros(20, 100, dtype=BF), rows(20, 100, F32), rows(19, 100, BF)),
                        w=(torch.zeros(50, 100, dtype=BF), rows(49, 100, BF), rows(50, 100, F16)),
                        targets=(torch.zeros(20, dtype=I64), torch.zeros(19, dtype=I32)),
                        loss=(torch.zeros(20, dtype=BF),), lse=(torch.zeros(40)[::2],)):
        refused(calls, v.forward, **bad)
    back = dict(x=good["x"], w=w, targets=good["targets"], lse=good["lse"], d_loss=torch.zeros(20),
                dx=rows(20, 100, grad), dw=v.weights(grad))
    assert v.backward(**back) is back["dx"]
    v.backward(**dict(back, dx=None))
    other = F32 if grad == BF else BF
    for bad in variants(back, d_loss=(torch.zeros(19), torch.zeros(20, dtype=BF)),
                        dx=(rows(20, 100, other), torch.zeros(20, 100, dtype=grad)),
                        dw=(v.weights(other), torch.zeros(50, 100, dtype=grad))):
        refused(calls, v.backward, **bad)
    with pytest.raises(B.MokError):
        VocabLoss(20, 100, 50, piece=100, device="cpu")


def test_nothing_to_do(calls):
    """No tokens or rows: arrays of any length for them."""
    Router(0, 8, 2, device="cpu").forward(torch.zeros(0, 8), torch.zeros(1, dtype=I32), torch.zeros(0))
    Norm(0, 16, device="cpu").forward(torch.zeros(0, 16, dtype=BF), None, torch.zeros(0, 16, dtype=BF),
                                      rstd=torch.zeros(1))
    v = VocabLoss(0, 16, 8, device="cpu")
    v.forward(torch.zeros(0, 16, dtype=BF), v.weights(), torch.zeros(1, dtype=I32), None,
              torch.zeros(0))
    assert len(calls) == 3


def test_arrays_of_another_device_than_the_current(monkeypatch):
    from mixture_experts_layer_deterministic_gb300 import buffers
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    buffers._check_current(torch.device("cuda", 0))
    buffers._check_current(torch.device("cpu"))
    with pytest.raises(ValueError):
        buffers._check_current(torch.device("cuda", 1))


def test_no_tokens_without_arrays(calls):
    """The entry points take null arrays where there is nothing in them."""
    r = Router(0, 8, 2, device="cpu")
    r.forward(torch.zeros(0, 8), None, None, counts=torch.zeros(8, dtype=I32))
    r.backward(None, None, None, None)
    assert len(calls) == 2 and calls[0][1][3] is None and calls[1][1][5] is None
