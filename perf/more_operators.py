"""More operators around the expert layer, as cases that can be timed and compared.

Three operators, each in its plain form (elementary torch operations, rounded once at the end)
and, where `own` is set, through the library's entry points:

  router  scores of router logits (softmax or sigmoid), choice of experts with a balance bias and
          within groups, routing weights, loads; the bias's update; the gradient of the logits
  norm    layer norm or RMS norm of a residual sum, and its gradients
  loss    softmax cross entropy over a vocabulary's projection with a penalty on the
          normaliser, and its gradients

`prepare` makes the inputs and the buffers a program keeps; `run` is one pass.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
RATE = 1e-3   # of the balance bias
Z_LOSS = 1e-4


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the layer of 512 experts: launch latency is all there is
        dict(name="router_fwd_t1", op="router_fwd", T=1, E=512, K=10, score="softmax", G=1, kept=1,
             top=1, renorm=True, scale=1.0, dtype="fp32", bias=False, load=False, masked=False),
        # a training step's routing without auxiliary loss: sigmoid scores, a balance bias, experts
        # from half of the groups, the loads and the bias's update
        dict(name="router_fwd_t16384_groups", op="router_fwd", T=16384, E=256, K=8, score="sigmoid",
             G=8, kept=4, top=2, renorm=True, scale=2.5, dtype="fp32", bias=True, load=True,
             masked=False),
        # the layer's training step: a softmax over all of 512 experts, its sums for a balance
        # loss, and their gradient
        dict(name="router_bwd_t16384", op="router_bwd", T=16384, E=512, K=10, score="softmax", G=1,
             kept=1, top=1, renorm=True, scale=1.0, dtype="fp32", bias=False, load=True,
             masked=False),
        # odd sizes, bf16 logits, experts that are masked out and tokens without any
        dict(name="router_bwd_t1023_odd", op="router_bwd", T=1023, E=60, K=6, score="softmax", G=1,
             kept=1, top=1, renorm=False, scale=1.0, dtype="bf16", bias=False, load=False,
             masked=True),
        # one decoded token: a residual sum and its RMS norm in front of the layer
        dict(name="norm_fwd_t1", op="norm_fwd", T=1, H=4096, kind="rms", x="bf16", y="bf16",
             bias=False, residual=True),
        # the same in a training step
        dict(name="norm_fwd_t16384", op="norm_fwd", T=16384, H=4096, kind="rms", x="bf16", y="bf16",
             bias=False, residual=True),
        # odd sizes in fp32, layer norm with a bias
        dict(name="norm_bwd_t1023_odd", op="norm_bwd", T=1023, H=1111, kind="layer", x="fp32",
             y="fp32", bias=True, residual=False),
        # the layer's backward configuration: layer norm of a bf16 residual stream
        dict(name="norm_bwd_t8192", op="norm_bwd", T=8192, H=4096, kind="layer", x="bf16", y="bf16",
             bias=True, residual=True),
        # log-probabilities of a few decoded tokens: the projection's bytes
        dict(name="loss_fwd_t4", op="loss_fwd", T=4, H=4096, V=131072, z=0.0, grad="bf16"),
        # a training step's loss
        dict(name="loss_fwd_t8192", op="loss_fwd", T=8192, H=4096, V=131072, z=Z_LOSS, grad="bf16"),
        # its gradients with sizes that fill no tile, kept in fp32
        dict(name="loss_bwd_t1001_odd", op="loss_bwd", T=1001, H=1000, V=5003, z=Z_LOSS,
             grad="fp32"),
        # the gradients of a training step
        dict(name="loss_bwd_t4096", op="loss_bwd", T=4096, H=4096, V=65536, z=Z_LOSS, grad="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["router_fwd", "router_bwd", "norm_fwd", "norm_bwd", "loss_fwd", "loss_bwd"])
    if op.startswith("router"):
        G = rng.choice([1, 1, 1, 2, 4, 8])
        E = G * _log(rng, 2, 1024 // G)
        kept = rng.randint(1, G)
        K = rng.randint(1, min(16, kept * (E // G)))
        # one expert's renormalised weight is constant: no gradient to speak of
        return dict(op=op, T=_log(rng, 1, 8_000_000 // E), E=E, K=K,
                    score=rng.choice(["softmax", "sigmoid"]), G=G, kept=kept,
                    top=rng.randint(1, 2), renorm=K > 1 and rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    bias=op == "router_fwd" and rng.random() < 0.5, load=rng.random() < 0.5,
                    masked=E >= 16 and rng.random() < 0.3)
    if op.startswith("norm"):
        H = _log(rng, 16, 16384)
        x = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, T=_log(rng, 1, 30_000_000 // H), H=H, kind=rng.choice(["layer", "rms"]),
                    x=x, y=rng.choice(["bf16", x]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.6)
    H, V = _log(rng, 16, 4096), _log(rng, 64, 131072)
    most = 4e12 if op == "loss_fwd" else 1e12
    return dict(op=op, T=_log(rng, 1, min(8192, int(most / (H * V)))), H=H, V=V,
                z=rng.choice([0.0, Z_LOSS]), grad=rng.choice(["bf16", "bf16", "fp32"]))


def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------------- preparation

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = {"r": _prepare_router, "n": _prepare_norm, "l": _prepare_loss}[case["op"][0]]
    st = make(case, gen)
    st["case"] = dict(case)
    return st


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    """Normal values in rows whose stride is a multiple of 8 elements."""
    full = torch.empty(*shape[:-1], _up(shape[-1], 8), device=DEV, dtype=dtype)
    full.normal_(0.0, std, generator=gen)
    return full[..., :shape[-1]]


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape[:-1], _up(shape[-1], 8), device=DEV, dtype=dtype)[..., :shape[-1]]


def _prepare_router(case, gen):
    T, E, K = case["T"], case["E"], case["K"]
    logits = _randn(gen, T, E, dtype=_dt(case["dtype"]))
    if case["masked"]:
        off = torch.rand(T, E, device=DEV, generator=gen) < 0.1
        off |= torch.rand(T, 1, device=DEV, generator=gen) < 0.02
        logits.masked_fill_(off, -math.inf)
    i32 = dict(device=DEV, dtype=torch.int32)
    st = dict(logits=logits, idx=torch.zeros(T, K, **i32), w=torch.zeros(T, K, device=DEV),
              bias=torch.empty(E, device=DEV).normal_(0, 0.05, generator=gen)
              if case["bias"] else None,
              counts=torch.zeros(E, **i32) if case["load"] else None,
              sums=torch.zeros(E, device=DEV) if case["load"] else None,
              new_bias=torch.zeros(E, device=DEV) if case["bias"] else None)
    if case["op"] == "router_bwd":
        st["idx"] = _choose(case, logits, None)[0].to(torch.int32)
        st["dw"] = torch.empty(T, K, device=DEV).normal_(0, 1, generator=gen)
        # of a balance loss: the same for every token
        st["dsum"] = torch.empty(E, device=DEV).normal_(0, 0.1, generator=gen) \
            if case["load"] else None
        st["dlogits"] = _zeros(T, E, dtype=logits.dtype)
    return st


def _prepare_norm(case, gen):
    T, H, x, y = case["T"], case["H"], _dt(case["x"]), _dt(case["y"])
    st = dict(x=_randn(gen, T, H, dtype=x),
              w=torch.empty(H, device=DEV).normal_(1, 0.2, generator=gen),
              b=torch.empty(H, device=DEV).normal_(0, 0.2, generator=gen)
              if case["bias"] else None)
    # rows of other means and sizes, as along a residual stream
    shift = torch.empty(T, 1, device=DEV).normal_(0, 0.5, generator=gen)
    size = torch.empty(T, 1, device=DEV).uniform_(0.2, 4.0, generator=gen)
    st["x"].copy_(st["x"].float() * size + shift)
    stat = lambda: torch.zeros(T, device=DEV)  # noqa: E731
    st.update(mean=stat() if case["kind"] == "layer" else None, rstd=stat())
    if case["op"] == "norm_fwd":
        st["res"] = _randn(gen, T, H, dtype=x) if case["residual"] else None
        st["h"] = _zeros(T, H, dtype=x) if case["residual"] else None
        st["y"] = _zeros(T, H, dtype=y)
        return st
    h = st["x"].double()
    if st["mean"] is not None:
        st["mean"].copy_(h.mean(1))
        h -= h.mean(1, keepdim=True)
    st["rstd"].copy_((h.square().mean(1) + EPS).rsqrt())
    st["dy"] = _randn(gen, T, H, dtype=y)
    st["dh"] = _randn(gen, T, H, dtype=x) if case["residual"] else None
    st["dx"] = _zeros(T, H, dtype=x)
    st["dweight"] = torch.zeros(H, device=DEV)
    st["dbias"] = torch.zeros(H, device=DEV) if case["bias"] else None
    return st


def _prepare_loss(case, gen):
    T, H, V = case["T"], case["H"], case["V"]
    bf = torch.bfloat16
    st = dict(x=_randn(gen, T, H, dtype=bf), w=_randn(gen, V, H, dtype=bf, std=1.5 / math.sqrt(H)),
              loss=torch.zeros(T, device=DEV), lse=torch.zeros(T, device=DEV))
    t = torch.randint(0, V, (T,), device=DEV, generator=gen, dtype=torch.int32)
    # prompts and padding take no part
    st["targets"] = t.masked_fill(torch.rand(T, device=DEV, generator=gen) < 0.1, -1)
    if case["op"] == "loss_bwd":
        st["lse"] = torch.logsumexp(st["x"].float() @ st["w"].float().T, 1)
        n = (st["targets"] >= 0).sum().clamp(min=1)
        st["d"] = torch.empty(T, device=DEV).uniform_(0.5, 1.5, generator=gen) / n
        st["dx"] = _zeros(T, H, dtype=_dt(case["grad"]))
        st["dw"] = _zeros(V, H, dtype=_dt(case["grad"]))
    return st


# -------------------------------------------------------------------- the plain forms

def run(st):
    return _RUN_OWN[st["case"]["op"]](st) if own else _RUN_PLAIN[st["case"]["op"]](st)


def _scores(kind, logits):
    """Scores in the logits' type; 0 for logits of -inf, rows of nothing else among them."""
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _choose(case, logits, bias):
    """(ids [T][K], scores [T][E]) in 64 bits: two scores may differ by less than 32 hold. Masked
    experts come after all others of the kept groups, experts of other groups never."""
    T, E, G, K = logits.shape[0], case["E"], case["G"], case["K"]
    l64 = logits.double()
    s = _scores(case["score"], l64)
    c = s if bias is None else s + bias.double()
    if bias is None and G == 1:
        c = l64  # the same order, and scores of far logits all round to 0 or 1
    off = torch.isneginf(l64)
    c = torch.where(off, -1e300, c)
    if G > 1:
        by = torch.where(off, -math.inf, c).reshape(T, G, E // G)
        best = torch.sort(by, dim=2, descending=True)[0][:, :, :case["top"]]
        none = best[:, :, :1].isneginf()
        total = torch.where(none, -math.inf, torch.where(best.isneginf(), 0.0, best).sum(2, True))
        rank = torch.sort(total[:, :, 0], dim=1, descending=True, stable=True)[1]
        keep = torch.zeros(T, G, device=DEV, dtype=torch.bool)
        keep.scatter_(1, rank[:, :case["kept"]], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -math.inf)
    idx = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :K]
    return idx, s


def _weights(case, chosen):
    """Routing weights of the chosen scores."""
    if case["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    return case["scale"] * chosen


def _router_fwd(st):
    case = st["case"]
    idx, s = _choose(case, st["logits"], st["bias"])
    out = dict(idx=idx.to(torch.int32), w=_weights(case, s.gather(1, idx)).float())
    if case["load"] or case["bias"]:
        e = torch.arange(case["E"], device=DEV)
        order = torch.sort(idx.reshape(-1))[0]
        counts = torch.searchsorted(order, e, right=True) - torch.searchsorted(order, e)
    if case["load"]:
        out.update(counts=counts.to(torch.int32), sums=s.sum(0).float())
    if case["bias"]:
        less = torch.sign(case["T"] * case["K"] - counts * case["E"])
        out["bias"] = st["bias"] + RATE * less
    return out


def _router_bwd(st):
    case = st["case"]
    l64, idx = st["logits"].double(), st["idx"].long()
    s = _scores(case["score"], l64)
    chosen, dw = s.gather(1, idx), case["scale"] * st["dw"].double()
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-300)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s) if st["dsum"] is None else st["dsum"].double().expand_as(s).clone()
    ds.scatter_add_(1, idx, dw)
    if case["score"] == "sigmoid":
        dl = ds * s * (1 - s)
    else:
        dl = s * (ds - (s * ds).sum(1, keepdim=True))
    return dict(dlogits=dl.to(st["logits"].dtype))


def _norm_fwd(st):
    case = st["case"]
    h = st["x"].float()
    out = {}
    if case["residual"]:
        out["h"] = (h + st["res"].float()).to(st["x"].dtype)
        h = out["h"].float()
    if case["kind"] == "layer":
        out["mean"] = h.mean(1)
        h = h - out["mean"][:, None]
    out["rstd"] = 1 / torch.sqrt(h.square().mean(1) + EPS)
    y = h * out["rstd"][:, None] * st["w"]
    if case["bias"]:
        y = y + st["b"]
    out["y"] = y.to(st["y"].dtype)
    return out


def _norm_bwd(st):
    case = st["case"]
    h, dy = st["x"].float(), st["dy"].float()
    if case["kind"] == "layer":
        h = h - st["mean"][:, None]
    n = h * st["rstd"][:, None]
    g = dy * st["w"]
    dx = g - n * (g * n).mean(1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * st["rstd"][:, None]
    if case["residual"]:
        dx = dx + st["dh"].float()
    out = dict(dx=dx.to(st["dx"].dtype), dw=(dy * n).sum(0))
    if case["bias"]:
        out["db"] = dy.sum(0)
    return out


def _loss_fwd(st):
    logits = st["x"].float() @ st["w"].float().T
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    at = st["targets"].long()
    hit = logits.gather(1, at.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(at >= 0, lse - hit + st["case"]["z"] * lse * lse, 0.0)
    return dict(loss=loss, lse=lse)


def _loss_bwd(st):
    x, w, lse, at = st["x"].float(), st["w"].float(), st["lse"], st["targets"].long()
    d = torch.where(at >= 0, st["d"], 0.0)
    dl = torch.exp(x @ w.T - lse[:, None]) * (d * (1 + 2 * st["case"]["z"] * lse))[:, None]
    dl.scatter_add_(1, at.clamp(min=0)[:, None], -d[:, None])
    return dict(dx=(dl @ w).to(st["dx"].dtype), dw=(dl.T @ x).to(st["dw"].dtype))


_RUN_PLAIN = dict(router_fwd=_router_fwd, router_bwd=_router_bwd, norm_fwd=_norm_fwd,
                  norm_bwd=_norm_bwd, loss_fwd=_loss_fwd, loss_bwd=_loss_bwd)


# ------------------------------------------------------------- the library's entry points

def _kind(B, t):
    return B.MOK_DTYPE_F32 if t.dtype == torch.float32 else B.MOK_DTYPE_BF16


def _workspace(st, n):
    st["ws_n"] = n
    st["ws"] = torch.empty(max(n, 256), device=DEV, dtype=torch.uint8)


def _router_config(B, st):
    """Configuration and workspace that a program makes once for its shapes."""
    if "cfg" not in st:
        c = st["case"]
        st["cfg"] = B.make_router(
            c["T"], c["E"], c["K"], groups=c["G"], topk_groups=c["kept"], group_top=c["top"],
            score=B.MOK_SCORE_SIGMOID if c["score"] == "sigmoid" else B.MOK_SCORE_SOFTMAX,
            renormalize=c["renorm"], scale=c["scale"], dtype=_kind(B, st["logits"]),
            ld=st["logits"].stride(0))
        _workspace(st, B.mok_router_workspace_size(st["cfg"]))
    return st["cfg"]


def _router_fwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg, case = _router_config(B, st), st["case"]
    if case["bias"] and st["counts"] is None:
        st["counts"] = torch.zeros(case["E"], device=DEV, dtype=torch.int32)
    B.check(B.mok_router_forward(cfg, st["logits"], st["bias"], st["idx"], st["w"], st["counts"],
                                 st["sums"], st["ws"], st["ws_n"]))
    out = dict(idx=st["idx"], w=st["w"])
    if case["load"]:
        out.update(counts=st["counts"], sums=st["sums"])
    if case["bias"]:
        B.check(B.mok_router_update_bias(cfg, st["counts"], RATE, st["bias"], st["new_bias"]))
        out["bias"] = st["new_bias"]
    return out


def _router_bwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    B.check(B.mok_router_backward(_router_config(B, st), st["logits"], st["idx"], st["dw"],
                                  st["dsum"], st["dlogits"]))
    return dict(dlogits=st["dlogits"])


def _norm_config(B, st):
    if "cfg" not in st:
        c, y = st["case"], st["y" if st["case"]["op"] == "norm_fwd" else "dy"]
        st["cfg"] = B.make_norm(c["T"], c["H"],
                                kind=B.MOK_NORM_LAYER if c["kind"] == "layer" else B.MOK_NORM_RMS,
                                eps=EPS, x_dtype=_kind(B, st["x"]), y_dtype=_kind(B, y),
                                ld_x=st["x"].stride(0), ld_y=y.stride(0))
        _workspace(st, B.mok_norm_workspace_size(st["cfg"]))
    return st["cfg"]


def _norm_fwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    B.check(B.mok_norm_forward(_norm_config(B, st), st["x"], st["res"], st["w"], st["b"], st["h"],
                               st["y"], st["mean"], st["rstd"]))
    return {k: st[k] for k in ("h", "mean", "rstd", "y") if st[k] is not None}


def _norm_bwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    B.check(B.mok_norm_backward(_norm_config(B, st), st["x"], st["mean"], st["rstd"], st["w"],
                                st["dy"], st["dh"], st["dx"], st["dweight"], st["dbias"], st["ws"],
                                st["ws_n"]))
    out = dict(dx=st["dx"], dw=st["dweight"])
    if st["dbias"] is not None:
        out["db"] = st["dbias"]
    return out


def _loss_config(B, st, which):
    if "cfg" not in st:
        c = st["case"]
        st["cfg"] = B.make_vocab_loss(c["T"], c["H"], c["V"], z_loss=c["z"],
                                      grad_dtype=B.MOK_DTYPE_F32 if c["grad"] == "fp32"
                                      else B.MOK_DTYPE_BF16,
                                      ld_x=st["x"].stride(0), ld_w=st["w"].stride(0))
        _workspace(st, B.mok_vocab_loss_workspace_size(st["cfg"], which))
    return st["cfg"]


def _loss_fwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg = _loss_config(B, st, B.MOK_VOCAB_LOSS_FORWARD)
    B.check(B.mok_vocab_loss_forward(cfg, st["x"], st["w"], st["targets"], st["loss"], st["lse"],
                                     st["ws"], st["ws_n"]))
    return dict(loss=st["loss"], lse=st["lse"])


def _loss_bwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg = _loss_config(B, st, B.MOK_VOCAB_LOSS_BACKWARD)
    B.check(B.mok_vocab_loss_backward(cfg, st["x"], st["w"], st["targets"], st["lse"], st["d"],
                                      st["dx"], st["dw"], st["ws"], st["ws_n"]))
    return dict(dx=st["dx"], dw=st["dw"])


_RUN_OWN = dict(router_fwd=_router_fwd_own, router_bwd=_router_bwd_own, norm_fwd=_norm_fwd_own,
                norm_bwd=_norm_bwd_own, loss_fwd=_loss_fwd_own, loss_bwd=_loss_bwd_own)


# ---------------------------------------------------------------------------- the floors

def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("router"):
        E, K, e = case["E"], case["K"], 4 if case["dtype"] == "fp32" else 2
        if op == "router_fwd":  # logits; ids and weights; per-expert vectors
            return dict(bytes=T * E * e + T * K * 8 + 8 * E * (case["bias"] + case["load"]),
                        flops=5 * T * E)
        # logits, their gradient; ids and the weights' gradient; the sums' gradient. The gradient of
        # renormalised or sigmoid scores needs the chosen logits alone.
        dense = case["load"] or (case["score"] == "softmax" and not case["renorm"])
        read = T * E if dense else T * K
        return dict(bytes=(read + T * E) * e + T * K * 8 + 4 * E * case["load"], flops=8 * read)
    if op.startswith("norm"):
        H = case["H"]
        x, y = (4 if case[k] == "fp32" else 2 for k in ("x", "y"))
        stats = 4 * T * (2 if case["kind"] == "layer" else 1)
        if op == "norm_fwd":  # x (and the residual, h); y
            return dict(bytes=T * H * (x + y + 2 * x * case["residual"]) + stats +
                        4 * H * (1 + case["bias"]), flops=8 * T * H)
        # h, dx (and dh); dy
        return dict(bytes=T * H * (2 * x + y + x * case["residual"]) + stats +
                    4 * H * (2 + case["bias"]), flops=14 * T * H)
    H, V = case["H"], case["V"]
    product = 2.0 * T * H * V
    if op == "loss_fwd":
        return dict(bytes=2 * (T + V) * H + 12 * T, flops=product)
    g = 4 if case["grad"] == "fp32" else 2  # logits again, dx, dW
    return dict(bytes=(2 + g) * (T + V) * H + 12 * T, flops=3 * product)


# ------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"r": _exact_router, "n": _exact_norm, "l": _exact_loss}[case["op"][0]](case, st)


def _log_scores(case, l):
    """Logarithms of the scores."""
    if case["score"] == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(l), -l)
    lse = torch.logsumexp(l, 1, keepdim=True)
    return torch.where(torch.isneginf(lse), -math.inf, l - lse)


def _exact_router(case, st):
    ls = _log_scores(case, st["logits"].double())
    T, E, K = case["T"], case["E"], case["K"]
    if case["op"] == "router_fwd":
        idx = _choose(case, st["logits"], st["bias"])[0]
        log_w = ls.gather(1, idx)
        if case["renorm"]:
            total = torch.logsumexp(log_w, 1, keepdim=True)
            log_w = torch.where(torch.isneginf(total), -math.inf, log_w - total)
        out = dict(idx=None, w=case["scale"] * torch.exp(log_w))
        if case["load"]:
            out.update(counts=None, sums=torch.exp(ls).sum(0))
        if case["bias"]:
            n = torch.zeros(E, device=DEV, dtype=torch.float64)
            n.index_add_(0, idx.reshape(-1), torch.ones(T * K, device=DEV, dtype=torch.float64))
            out["bias"] = st["bias"].double() + RATE * torch.sign(T * K / E - n)
        return out
    # by automatic differentiation of the definition; masked logits take no part
    l64 = st["logits"].double().masked_fill(torch.isneginf(st["logits"]), -1e4).requires_grad_()
    s = torch.sigmoid(l64) if case["score"] == "sigmoid" else torch.softmax(l64, 1)
    live = ~torch.isneginf(st["logits"])
    s = s * live
    chosen = s.gather(1, st["idx"].long())
    if case["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    value = case["scale"] * (chosen * st["dw"].double()).sum()
    if st["dsum"] is not None:
        value = value + (s.sum(0) * st["dsum"].double()).sum()
    value.backward()
    return dict(dlogits=torch.where(live, l64.grad, 0.0))


def _exact_norm(case, st):
    layer = case["kind"] == "layer"
    if case["op"] == "norm_fwd":
        h = st["x"].double()
        out = {}
        if case["residual"]:
            out["h"] = h + st["res"].double()
            h = out["h"].to(st["x"].dtype).double()  # the norm is of the stored sum
        var, mean = torch.var_mean(h, 1, correction=0)
        if layer:
            out["mean"] = mean
        else:
            var, mean = var + mean.square(), torch.zeros_like(mean)
        out["rstd"] = (var + EPS) ** -0.5
        y = torch.addcmul(torch.zeros_like(h), (h - mean[:, None]) / (var + EPS).sqrt()[:, None],
                          st["w"].double())
        out["y"] = y + st["b"].double() if case["bias"] else y
        return out
    r = st["rstd"].double()[:, None]
    n = (st["x"].double() - (st["mean"].double()[:, None] if layer else 0.0)) * r
    dy = st["dy"].double()
    g = torch.einsum("th,h->th", dy, st["w"].double())
    along = torch.einsum("th,th->t", g, n)[:, None] / case["H"]
    dx = r * (g - along * n - (g.mean(1, keepdim=True) if layer else 0.0))
    if case["residual"]:
        dx += st["dh"].double()
    out = dict(dx=dx, dw=torch.einsum("th,th->h", dy, n))
    if case["bias"]:
        out["db"] = torch.einsum("th->h", dy)
    return out


def _exact_loss(case, st):
    T, H, V = case["T"], case["H"], case["V"]
    x, w, at = st["x"].double(), st["w"].double(), st["targets"].long()
    step = max(1, min(T, (1 << 28) // V))
    if case["op"] == "loss_fwd":
        lse = torch.cat([torch.logsumexp(x[i:i + step] @ w.T, 1) for i in range(0, T, step)])
        hit = (x * w[at.clamp(min=0)]).sum(1)
        return dict(loss=(lse - hit + case["z"] * lse.square()) * (at >= 0), lse=lse)
    d, lse = st["d"].double() * (at >= 0), st["lse"].double()
    factor = d * (1 + 2 * case["z"] * lse)
    dx, dw = torch.empty_like(x), torch.zeros_like(w)
    for i in range(0, T, step):
        part = slice(i, min(i + step, T))
        p = torch.exp(x[part] @ w.T - lse[part, None]).mul_(factor[part, None])
        dx[part] = p @ w
        dw.addmm_(p.T, x[part])
    live = at >= 0
    dx -= d[:, None] * w[at.clamp(min=0)]
    dw.index_add_(0, at[live], -d[live, None] * x[live])
    return dict(dx=dx, dw=dw)
