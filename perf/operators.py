"""The operators around the expert layer, as cases that can be timed and compared.

Four operators, each in its plain form (elementary torch operations in fp32, rounded once at
the end) and, where `own` is set, through the library's entry points:

  sort    tokens sorted by expert (dispatch) and brought back with their routing weights
          (combine): row map, both directions, and both gradients
  linear  act(x W^T + b) + residual, for one matrix or one per expert, and its gradients
  adamw   an AdamW step over a list of tensors, states in fp32 or in MXFP8

`prepare` makes the inputs and the buffers a program keeps; `run` is one pass.
"""
import math

import torch

own = False

DEV = "cuda"
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1
GELU_C = 0.7978845608028654  # sqrt(2 / pi)
GELU_A = 0.044715


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the layer of 512 experts: launch latency is all there is
        dict(name="sort_fwd_t1", op="sort_fwd", T=1, H=4096, E=512, K=10, dtype="bf16",
             capacity=0, residual=True),
        # the layer's training forward: HBM traffic of 163840 routed rows
        dict(name="sort_fwd_t16384", op="sort_fwd", T=16384, H=4096, E=512, K=10,
             dtype="bf16", capacity=0, residual=False),
        # odd token count and width, fp32 rows, a per-expert capacity that drops rows
        dict(name="sort_bwd_t1023_odd", op="sort_bwd", T=1023, H=1111, E=60, K=6,
             dtype="fp32", capacity=110, residual=False),
        # the layer's backward configuration
        dict(name="sort_bwd_t8192", op="sort_bwd", T=8192, H=4096, E=512, K=10, dtype="bf16",
             capacity=0, residual=False),
        # a dense layer next to the experts while decoding one token: weight bandwidth
        dict(name="linear_fwd_m1", op="linear_fwd", G=1, R=1, Kin=4096, N=4096, act="silu",
             out="bf16", bias=True, residual=True, save_z=False),
        # router logits of a training step, kept in fp32 for the top-k
        dict(name="linear_fwd_router", op="linear_fwd", G=1, R=16384, Kin=4096, N=512,
             act="none", out="fp32", bias=True, residual=False, save_z=False),
        # biased GELU experts over sorted rows (uneven experts, some empty)
        dict(name="linear_fwd_experts", op="linear_fwd", G=64, R=20480, Kin=4096, N=1024,
             act="gelu_tanh", out="bf16", bias=True, residual=False, save_z=True),
        # a dense block's gradient with sizes that fill no tile
        dict(name="linear_bwd_odd", op="linear_bwd", G=1, R=2050, Kin=1000, N=1500, act="silu",
             out="bf16", bias=True, residual=False, save_z=True),
        # the gradient of the biased GELU experts
        dict(name="linear_bwd_experts", op="linear_bwd", G=64, R=20480, Kin=4096, N=1024,
             act="gelu_tanh", out="bf16", bias=True, residual=False, save_z=True),
        # biases, norms and small matrices: many short tensors, bf16 parameters without a
        # master copy, 8-bit states, stochastic rounding
        dict(name="adamw_8bit_short", op="adamw", tensors=60, largest=20000, experts=0, p="bf16",
             g="fp32", state="8bit", copy=False),
        # the weights of a 32-expert layer, fp32 master and states, bf16 working copy
        dict(name="adamw_fp32_layer", op="adamw", tensors=5, largest=0, experts=32, p="fp32",
             g="bf16", state="fp32", copy=True),
        # the same weights with 8-bit states
        dict(name="adamw_8bit_layer", op="adamw", tensors=5, largest=0, experts=32, p="fp32",
             g="bf16", state="8bit", copy=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["sort_fwd", "sort_bwd", "linear_fwd", "linear_fwd", "linear_bwd", "adamw"])
    if op.startswith("sort"):
        E = _log(rng, 2, 512)
        K = rng.randint(1, min(E, 16))
        H = _log(rng, 16, 8192)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 600_000_000 // (2 if dtype == "fp32" else 1)
        T = _log(rng, 1, max(1, min(65536, most // (K * H))))
        if op == "sort_bwd":
            T = max(1, T // 2)
        cap = 0 if rng.random() < 0.6 else max(1, int(1.2 * T * K / E))
        return dict(op=op, T=T, H=H, E=E, K=K, dtype=dtype, capacity=cap,
                    residual=op == "sort_fwd" and rng.random() < 0.5)
    if op.startswith("linear"):
        G = 1 if rng.random() < 0.5 else _log(rng, 2, 64)
        Kin, N = _log(rng, 16, 4096), _log(rng, 8, 4096)
        if G > 1:
            N = min(N, 1024)
        R = _log(rng, 1, 16384 if N * Kin <= (1 << 22) else 4096)
        act = rng.choice(["none", "relu", "silu", "gelu_tanh"])
        fwd = op == "linear_fwd"
        out = rng.choice(["bf16", "bf16", "fp32"]) if fwd else "bf16"
        return dict(op=op, G=G, R=R, Kin=Kin, N=N, act=act, out=out, bias=rng.random() < 0.7,
                    residual=fwd and rng.random() < 0.5, save_z=act != "none" or not fwd)
    state = rng.choice(["fp32", "8bit"])
    p = rng.choice(["fp32", "fp32", "bf16"])
    if rng.random() < 0.4:
        return dict(op=op, tensors=5, largest=0, experts=rng.randint(1, 16), p=p,
                    g=rng.choice(["bf16", "fp32"]), state=state, copy=p == "fp32")
    return dict(op=op, tensors=rng.randint(1, 200), largest=_log(rng, 100, 2_000_000), experts=0,
                p=p, g=rng.choice(["bf16", "fp32"]), state=state,
                copy=p == "fp32" and rng.random() < 0.5)


def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------------- preparation

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = {"s": _prepare_sort, "l": _prepare_linear, "a": _prepare_adamw}[case["op"][0]]
    st = make(case, gen)
    st["case"] = dict(case)
    return st


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    """Normal values in rows whose stride is a multiple of 8 elements."""
    ld = _up(shape[-1], 8)
    full = torch.empty(*shape[:-1], ld, device=DEV, dtype=dtype)
    full.normal_(0.0, std, generator=gen)
    return full[..., :shape[-1]]


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape[:-1], _up(shape[-1], 8), device=DEV, dtype=dtype)[..., :shape[-1]]


def _prepare_sort(case, gen):
    T, H, E, K = (case[k] for k in ("T", "H", "E", "K"))
    dt = _dt(case["dtype"])
    R = T * K
    logits = torch.empty(T, E, device=DEV).normal_(0.0, 1.0, generator=gen)
    top, idx = torch.topk(logits, K, dim=1)
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(R, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    n_rows = R + 15 * min(E, R)
    st = dict(idx=i32(idx), w=torch.softmax(top, 1).contiguous(), counts=i32(counts),
              offsets=i32(offsets), perm=i32(perm), inv=i32(inv), n_rows=n_rows,
              map=torch.zeros(R, device=DEV, dtype=torch.int32),
              starts=torch.zeros(E + 1, device=DEV, dtype=torch.int32),
              kept=torch.zeros(E, device=DEV, dtype=torch.int32))
    m, starts, kept = _row_map(st, case)
    valid = _valid_rows(starts, kept, n_rows)
    if case["op"] == "sort_fwd":
        st["x"] = _randn(gen, T, H, dtype=dt)
        st["rows"] = _randn(gen, n_rows, H, dtype=dt)
        st["rows"].mul_(valid[:, None].to(dt))
        st["res"] = _randn(gen, T, H, dtype=dt) if case["residual"] else None
        st["xs"], st["y"] = _zeros(n_rows, H, dtype=dt), _zeros(T, H, dtype=dt)
        return st
    st["map"], st["starts"], st["kept"] = i32(m), i32(starts), i32(kept)
    st["rows"] = _randn(gen, n_rows, H, dtype=dt)
    st["rows"].mul_(valid[:, None].to(dt))
    st["dxs"] = _randn(gen, n_rows, H, dtype=dt)
    st["dy"] = _randn(gen, T, H, dtype=dt)
    st["drows"], st["dx"] = _zeros(n_rows, H, dtype=dt), _zeros(T, H, dtype=dt)
    st["dw"] = torch.zeros(T, K, device=DEV)
    return st


def _prepare_linear(case, gen):
    G, R, Kin, N = (case[k] for k in ("G", "R", "Kin", "N"))
    bf = torch.bfloat16
    st = dict(counts=None, starts=None, rows=R, most=R)
    if G > 1:
        share = torch.empty(G, device=DEV).uniform_(0, 1, generator=gen)
        share = torch.where(share < 0.1, torch.zeros_like(share), share) + 1e-9
        counts = (share / share.sum() * R).floor().to(torch.int64)
        padded = (counts + 15) // 16 * 16
        starts = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
        st["rows"] = R + 15 * G
        st["most"] = max(1, int(counts.max()))
        st["counts"], st["starts"] = counts.to(torch.int32), starts.to(torch.int32)
        valid = _valid_rows(starts, counts, st["rows"])[:, None].to(bf)
    rows = st["rows"]
    st["x"] = _randn(gen, rows, Kin, dtype=bf)
    st["w"] = _randn(gen, G, N, Kin, dtype=bf, std=1 / math.sqrt(Kin))
    st["b"] = (torch.empty(G, N, device=DEV).normal_(0, 0.5, generator=gen)
               if case["bias"] else None)
    if G > 1:
        st["x"].mul_(valid)
    if case["op"] == "linear_fwd":
        st["res"] = _randn(gen, rows, N, dtype=bf) if case["residual"] else None
        st["y"] = _zeros(rows, N, dtype=_dt(case["out"]))
        st["z"] = _zeros(rows, N, dtype=bf) if case["save_z"] else None
    else:
        st["z"] = _randn(gen, rows, N, dtype=bf)
        st["dy"] = _randn(gen, rows, N, dtype=bf)
        if G > 1:
            st["z"].mul_(valid)
            st["dy"].mul_(valid)
        st["dx"], st["dw"] = _zeros(rows, Kin, dtype=bf), _zeros(G, N, Kin, dtype=bf)
        st["db"] = torch.zeros(G, N, device=DEV) if case["bias"] else None
    return st


def _sizes(case):
    """Element counts of the tensors; the first of them decay, the others do not."""
    if case["experts"]:
        E = case["experts"]
        return [E * 2048 * 4096, E * 4096 * 1024, E * 4096], [E * 2048, E * 4096]
    n, most = case["tensors"], case["largest"]
    sizes = [max(1, int(most ** ((7 * i % n + 1) / n))) for i in range(n)]
    return sizes[: (n + 1) // 2], sizes[(n + 1) // 2:]


def _prepare_adamw(case, gen):
    first, rest = _sizes(case)
    starts, at = [], 0
    for n in first + rest:  # every tensor begins at a multiple of 32 elements
        starts.append(at)
        at += _up(n, 32)
    total, edge = at, sum(_up(n, 32) for n in first)
    live = torch.zeros(total, device=DEV, dtype=torch.bool)
    for s, n in zip(starts, first + rest):
        live[s:s + n] = True
    norm = lambda std: torch.empty(total, device=DEV).normal_(0, std, generator=gen).mul_(live)  # noqa: E731
    p = norm(0.02)
    st = dict(total=total, edge=edge, sizes=first + rest, starts=starts, step=100,
              seed=0x9E3779B97F4A7C15, p=p.to(_dt(case["p"])),
              copy=p.to(torch.bfloat16) if case["copy"] else None,
              g=norm(1e-3).to(_dt(case["g"])),
              gscale=torch.empty(1, device=DEV).uniform_(0.3, 1.0, generator=gen))
    m, s = norm(4e-4), norm(1e-3).abs_().add_(2e-4).mul_(live)
    if case["state"] == "fp32":
        st["m"], st["v"] = m, s.square_()
    else:
        half = torch.full((1,), 1 << 19, device=DEV, dtype=torch.int64)
        st["m"], st["ms"] = _encode(m, half, False)
        st["s"], st["ss"] = _encode(s, half, True)
    return st


# -------------------------------------------------------------------- the plain forms

def run(st):
    return _RUN_OWN[st["case"]["op"]](st) if own else _RUN_PLAIN[st["case"]["op"]](st)


def _row_map(st, case):
    """Row of each routed id: its expert's first row (a multiple of 16) plus its rank among the
    expert's rows; -1 where the rank is at or past the capacity."""
    e = st["idx"].reshape(-1).long()
    rank = st["inv"].long() - st["offsets"].long()[e]
    kept = st["counts"].long()
    if case["capacity"]:
        kept = kept.clamp(max=case["capacity"])
    starts = torch.cat([kept.new_zeros(1), ((kept + 15) // 16 * 16).cumsum(0)])
    return torch.where(rank < kept[e], starts[e] + rank, -1), starts, kept


def _valid_rows(starts, counts, rows):
    r = torch.arange(rows, device=DEV)
    e = (torch.searchsorted(starts[1:].long(), r, right=True)).clamp(max=counts.numel() - 1)
    return (r - starts.long()[e]) < counts.long()[e]


def _sort_fwd(st):
    case = st["case"]
    T, H, K = case["T"], case["H"], case["K"]
    m, starts, kept = _row_map(st, case)
    has = m >= 0
    dest = torch.where(has, m, st["n_rows"])  # dropped ids go to a row that is cut off
    xs = torch.zeros(st["n_rows"] + 1, H, device=DEV, dtype=st["x"].dtype)
    xs[dest] = st["x"][torch.arange(T * K, device=DEV) // K]
    w = (st["w"].reshape(-1) * has).reshape(T, K, 1)
    rows = st["rows"][m.clamp(min=0)].float().reshape(T, K, H)
    y = torch.where(has.reshape(T, K, 1), rows * w, 0.0).sum(1)
    if st["res"] is not None:
        y = y + st["res"].float()
    return dict(map=m.to(torch.int32), starts=starts.to(torch.int32), kept=kept.to(torch.int32),
                xs=xs[:-1], y=y.to(st["x"].dtype))


def _sort_bwd(st):
    case = st["case"]
    T, H, K = case["T"], case["H"], case["K"]
    m = st["map"].long()
    has = (m >= 0).reshape(T, K, 1)
    at = m.clamp(min=0)
    dy = st["dy"].float().reshape(T, 1, H)
    dw = torch.where(has, st["rows"][at].float().reshape(T, K, H) * dy, 0.0).sum(2)
    drows = torch.zeros(st["n_rows"] + 1, H, device=DEV, dtype=st["dy"].dtype)
    drows[torch.where(m >= 0, m, st["n_rows"])] = (
        (dy * st["w"].reshape(T, K, 1)).reshape(T * K, H).to(st["dy"].dtype))
    dx = torch.where(has, st["dxs"][at].float().reshape(T, K, H), 0.0).sum(1)
    return dict(drows=drows[:-1], dw=dw, dx=dx.to(st["dy"].dtype))


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * z * z)
    return torch.ones_like(z)


def _by_group(st, t):
    """Rows [rows][C] -> [G][most][C] in fp32, absent rows zero."""
    if st["counts"] is None:
        return t.float()[None]
    pos = torch.arange(st["most"], device=DEV)
    at = st["starts"][:-1, None].long() + pos
    here = pos < st["counts"][:, None]
    return torch.where(here[:, :, None], t[at.clamp(max=st["rows"] - 1)].float(), 0.0)


def _by_row(st, t):
    """[G][most][C] -> rows [rows][C], rows of no group zero."""
    if st["counts"] is None:
        return t[0]
    r = torch.arange(st["rows"], device=DEV)
    starts = st["starts"].long()
    e = torch.searchsorted(starts[1:], r, right=True).clamp(max=t.shape[0] - 1)
    pos = r - starts[e]
    here = pos < st["counts"][e]
    return torch.where(here[:, None], t[e, pos.clamp(max=st["most"] - 1)], 0.0)


def _linear_fwd(st):
    case = st["case"]
    z = torch.bmm(_by_group(st, st["x"]), st["w"].float().transpose(1, 2))
    if st["b"] is not None:
        z = z + st["b"][:, None, :]
    y = _act(z, case["act"])
    if st["res"] is not None:
        y = y + _by_group(st, st["res"])
    out = dict(y=_by_row(st, y).to(_dt(case["out"])))
    if case["save_z"]:
        out["z"] = _by_row(st, z).to(torch.bfloat16)
    return out


def _linear_bwd(st):
    case = st["case"]
    dz = _by_group(st, st["dy"])
    if case["act"] != "none":
        dz = dz * _act_grad(_by_group(st, st["z"]), case["act"])
    dx = torch.bmm(dz, st["w"].float())
    dw = torch.bmm(dz.transpose(1, 2), _by_group(st, st["x"]))
    out = dict(dx=_by_row(st, dx).to(torch.bfloat16), dw=dw.to(torch.bfloat16))
    if case["bias"]:
        out["db"] = dz.sum(1)
    return out


def _mix32(h):
    """A 32-bit finaliser (xor-shift, multiply, twice) on int64 tensors holding 32-bit values."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random(st):
    """32 random bits for every element number i of the step, from i and the step's seed."""
    i = torch.arange(st["total"], device=DEV)
    seed = (st["seed"] + st["step"]) & 0xFFFFFFFFFFFFFFFF
    key = _mix32(_mix32((i >> 32) ^ (seed & 0xFFFFFFFF)) ^ (seed >> 32))
    return _mix32((i & 0xFFFFFFFF) ^ key)


def _encode(x, rnd, positive):
    """fp32 values in blocks of 32 -> E4M3 codes and E8M0 scales. The scale is the least power
    of two that brings the block's largest magnitude to 448 or less; a magnitude is rounded by
    adding `rnd` (20 bits) below its last kept bit and cutting off."""
    a = x.abs()
    top = a.reshape(-1, 32).amax(1).view(torch.int32).long()
    sb = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000)).clamp(min=0)
    inv = ((254 - sb) << 23).to(torch.int32).view(torch.float32)
    y = (a.reshape(-1, 32) * inv[:, None]).reshape(-1)
    low = y < 2.0 ** -6  # E4M3 subnormals: the octave above has their step
    z = torch.where(low, y + 2.0 ** -6, y)
    code = ((z.view(torch.int32).long() + rnd) >> 20) - torch.where(low, 121 << 3, 120 << 3)
    if positive:  # what is above zero stays above zero
        code = torch.maximum(code, (a > 0).long())
    code = code | ((x < 0).long() << 7)
    return code.to(torch.uint8), sb.to(torch.uint8)


def _decode(q, sb):
    v = q.view(torch.float8_e4m3fn).float().reshape(-1, 32)
    return (v * torch.exp2(sb.float() - 127)[:, None]).reshape(-1)


def _adamw(st):
    case = st["case"]
    st["step"] += 1
    t = st["step"]
    wide = case["state"] == "fp32"
    rnd = None if wide and case["p"] == "fp32" else _random(st)
    g = st["g"].float() * st["gscale"]
    p = st["p"].float()
    m = st["m"] if wide else _decode(st["m"], st["ms"])
    v = st["v"] if wide else _decode(st["s"], st["ss"]).square()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    s = torch.sqrt(v)
    p[: st["edge"]] *= 1 - LR * DECAY
    p -= (LR / (1 - BETA1 ** t)) * m / (s * (1 / math.sqrt(1 - BETA2 ** t)) + EPS)
    if case["p"] == "bf16":  # stochastic: 16 random bits under the last kept one
        r16 = _mix32((rnd + 0x9E3779B9) & 0xFFFFFFFF) >> 16
        bits = p.view(torch.int32).long() + r16
        st["p"].copy_((bits >> 16 << 16).to(torch.int32).view(torch.float32))
    else:
        st["p"].copy_(p)
    out = dict(p=st["p"])
    if case["copy"]:
        st["copy"].copy_(p)
        out["copy"] = st["copy"]
    if wide:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        for name, scale, x, bits in (("m", "ms", m, rnd & 0xFFFF), ("s", "ss", s, rnd >> 16)):
            q, sb = _encode(x, (bits << 4) + 8, name == "s")
            st[name].copy_(q)
            st[scale].copy_(sb)
    out.update(_states(st))
    return out


def _states(st):
    if "v" in st:
        return dict(m=st["m"], v=st["v"])
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return dict(m=st["m"].view(e4), ms=st["ms"].view(e8), s=st["s"].view(e4),
                ss=st["ss"].view(e8))


_RUN_PLAIN = dict(sort_fwd=_sort_fwd, sort_bwd=_sort_bwd, linear_fwd=_linear_fwd,
                  linear_bwd=_linear_bwd, adamw=_adamw)


# ------------------------------------------------------------- the library's entry points

def _rows_config(B, st):
    """The configuration a program makes once for its shapes."""
    if "cfg" not in st:
        c = st["case"]
        tok, row = (st["x"], st["rows"]) if c["op"] == "sort_fwd" else (st["dy"], st["rows"])
        st["cfg"] = B.make_rows(T=c["T"], K=c["K"], E=c["E"], H=c["H"], n_rows=st["n_rows"],
                                dtype=B.MOK_DTYPE_F32 if c["dtype"] == "fp32"
                                else B.MOK_DTYPE_BF16,
                                ld_tok=tok.stride(0), ld_row=row.stride(0),
                                capacity=c["capacity"])
        st["sched"] = B.make_schedule(st["counts"], st["offsets"], st["perm"], st["inv"],
                                      None, None)
    return st["cfg"], st["sched"]


def _sort_fwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg, sched = _rows_config(B, st)
    B.check(B.mok_build_row_map(cfg, st["idx"], sched, st["map"], st["starts"], st["kept"]))
    B.check(B.mok_dispatch(cfg, st["x"], st["map"], st["starts"], st["kept"], st["xs"]))
    B.check(B.mok_combine(cfg, st["rows"], st["map"], st["w"], st["res"], st["y"]))
    return dict(map=st["map"], starts=st["starts"], kept=st["kept"], xs=st["xs"], y=st["y"])


def _sort_bwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg, _ = _rows_config(B, st)
    B.check(B.mok_combine_backward(cfg, st["dy"], st["rows"], st["map"], st["starts"],
                                   st["kept"], st["w"], st["drows"], st["dw"]))
    B.check(B.mok_dispatch_backward(cfg, st["dxs"], st["map"], st["dx"]))
    return dict(drows=st["drows"], dw=st["dw"], dx=st["dx"])


def _linear_config(B, st):
    """Configuration and workspace, made once."""
    if "cfg" not in st:
        c = st["case"]
        act = dict(none=B.MOK_ACT_NONE, relu=B.MOK_ACT_RELU, silu=B.MOK_ACT_SILU,
                   gelu_tanh=B.MOK_ACT_GELU_TANH)[c["act"]]
        fwd = c["op"] == "linear_fwd"
        st["cfg"] = B.make_linear(rows=st["rows"], in_features=c["Kin"], out_features=c["N"],
                                  groups=c["G"], act=act,
                                  out_dtype=B.MOK_DTYPE_F32 if c["out"] == "fp32"
                                  else B.MOK_DTYPE_BF16,
                                  ld_in=st["x"].stride(0), ld_w=st["w"].stride(1),
                                  ld_out=(st["y"] if fwd else st["dy"]).stride(0))
        st["ws_n"] = B.mok_linear_workspace_size(
            st["cfg"], B.MOK_LINEAR_FORWARD if fwd else B.MOK_LINEAR_BACKWARD)
        st["ws"] = torch.empty(max(st["ws_n"], 256), device=DEV, dtype=torch.uint8)
    return st["cfg"]


def _linear_fwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg = _linear_config(B, st)
    B.check(B.mok_linear_forward(cfg, st["x"], st["w"], st["b"], st["res"], st["starts"],
                                 st["counts"], st["y"], st["z"], st["ws"], st["ws_n"]))
    return dict(y=st["y"]) if st["z"] is None else dict(y=st["y"], z=st["z"])


def _linear_bwd_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    cfg = _linear_config(B, st)
    B.check(B.mok_linear_backward(cfg, st["x"], st["w"], st["z"], st["dy"], st["starts"],
                                  st["counts"], st["dx"], st["dw"], st["db"], st["ws"],
                                  st["ws_n"]))
    out = dict(dx=st["dx"], dw=st["dw"])
    if st["db"] is not None:
        out["db"] = st["db"]
    return out


def _adamw_own(st):
    from mixture_experts_layer_deterministic_gb300 import binding as B
    c = st["case"]
    if "list" not in st:  # the tensor list of the program's parameters, made once
        def at(name, s, n, per=1):
            return st[name][s // per:(s + n + per - 1) // per] if st.get(name) is not None else None
        wide = c["state"] == "fp32"
        st["list"] = B.make_adamw_list([
            dict(p=at("p", s, n), copy=at("copy", s, n), g=at("g", s, n), m=at("m", s, n),
                 v=at("v" if wide else "s", s, n), n=n,
                 m_scale=None if wide else at("ms", s, n, 32),
                 v_scale=None if wide else at("ss", s, n, 32),
                 weight_decay=DECAY if s < st["edge"] else 0.0)
            for s, n in zip(st["starts"], st["sizes"])])
    st["step"] += 1
    dt = lambda k: B.MOK_DTYPE_F32 if c[k] == "fp32" else B.MOK_DTYPE_BF16  # noqa: E731
    cfg = B.make_adamw(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, step=st["step"],
                       seed=(st["seed"] + st["step"]) & 0xFFFFFFFFFFFFFFFF,
                       p_dtype=dt("p"), g_dtype=dt("g"),
                       state=B.MOK_STATE_F32 if c["state"] == "fp32" else B.MOK_STATE_MXFP8,
                       flags=B.MOK_ADAMW_STOCHASTIC)
    B.check(B.mok_adamw_step(cfg, st["list"], st["gscale"]))
    out = dict(p=st["p"])
    if c["copy"]:
        out["copy"] = st["copy"]
    out.update(_states(st))
    return out


_RUN_OWN = dict(sort_fwd=_sort_fwd_own, sort_bwd=_sort_bwd_own, linear_fwd=_linear_fwd_own,
                linear_bwd=_linear_bwd_own, adamw=_adamw_own)


# ---------------------------------------------------------------------------- the floors

def work(case):
    op = case["op"]
    if op.startswith("sort"):
        T, H, K = case["T"], case["H"], case["K"]
        e = 4 if case["dtype"] == "fp32" else 2
        R = T * K
        if case["capacity"]:
            R = min(R, case["capacity"] * case["E"])
        if op == "sort_fwd":  # x, xs, rows, y (and the residual); ids, places, map and weights
            return dict(bytes=2 * R * H * e + (2 + case["residual"]) * T * H * e + T * K * 16,
                        flops=2 * R * H)
        # dy, rows, drows, dxs, dx; map, weights and their gradient
        return dict(bytes=3 * R * H * e + 2 * T * H * e + T * K * 12, flops=4 * R * H)
    if op.startswith("linear"):
        G, R, Kin, N = (case[k] for k in ("G", "R", "Kin", "N"))
        flops = 2.0 * R * Kin * N
        if op == "linear_fwd":
            out = 4 if case["out"] == "fp32" else 2
            return dict(bytes=2 * (R * Kin + G * N * Kin) + R * N *
                        (out + 2 * case["residual"] + 2 * case["save_z"]) +
                        4 * G * N * case["bias"], flops=flops)
        z = 0 if case["act"] == "none" else 2
        return dict(bytes=2 * (2 * R * Kin + 2 * G * N * Kin) + R * N * (2 + z) +
                    4 * G * N * case["bias"], flops=2 * flops)
    first, rest = _sizes(case)
    n = sum(first) + sum(rest)
    each = 2 * (4 if case["p"] == "fp32" else 2) + (4 if case["g"] == "fp32" else 2)
    each += 2 * case["copy"] + (16 if case["state"] == "fp32" else 4 * 33 / 32)
    return dict(bytes=int(n * each), flops=15 * n)


# ------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"s": _exact_sort, "l": _exact_linear, "a": _exact_adamw}[case["op"][0]](case, st)


def _exact_sort(case, st):
    T, H, K = case["T"], case["H"], case["K"]
    f = torch.arange(T * K, device=DEV)
    if case["op"] == "sort_fwd":
        # walk the experts' rows in sorted order: rank r of expert e is the r-th entry of perm
        # in its range
        perm, off = st["perm"].long(), st["offsets"].long()
        expert = torch.repeat_interleave(torch.arange(case["E"], device=DEV), off.diff())
        rank = torch.arange(T * K, device=DEV) - off[expert]
        limit = case["capacity"] or T * K
        keep = rank < limit
        sizes = off.diff().clamp(max=limit)
        first = torch.cumsum(-(-sizes // 16) * 16, 0) - (-(-sizes // 16) * 16)
        src, dst = perm[keep], (first[expert] + rank)[keep]
        xs = torch.zeros(st["n_rows"], H, device=DEV, dtype=torch.float64)
        xs[dst] = st["x"].double()[src // K]
        part = st["rows"].double()[dst] * st["w"].double().reshape(-1)[src][:, None]
        y = torch.zeros(T, H, device=DEV, dtype=torch.float64).index_add_(0, src // K, part)
        if st["res"] is not None:
            y += st["res"].double()
        return dict(map=None, starts=None, kept=None, xs=xs, y=y)
    at = st["map"].long()
    f = f[at >= 0]
    at = at[at >= 0]
    dy = st["dy"].double()[f // K]
    drows = torch.zeros(st["n_rows"], H, device=DEV, dtype=torch.float64)
    drows[at] = dy * st["w"].double().reshape(-1)[f][:, None]
    dw = torch.zeros(T * K, device=DEV, dtype=torch.float64)
    dw[f] = (st["rows"].double()[at] * dy).sum(1)
    dx = torch.zeros(T, H, device=DEV, dtype=torch.float64)
    dx.index_add_(0, f // K, st["dxs"].double()[at])
    return dict(drows=drows, dw=dw.reshape(T, K), dx=dx)


def _exact_linear(case, st):
    G, rows, Kin, N = case["G"], st["rows"], case["Kin"], case["N"]
    d64 = dict(device=DEV, dtype=torch.float64)
    spans = [(0, rows)]
    if G > 1:
        begin, count = st["starts"].tolist(), st["counts"].tolist()
        spans = [(begin[e], begin[e] + count[e]) for e in range(G)]

    def gate(z):  # (act(z), act'(z)) by the logistic function: tanh(u) = 2 sigma(2u) - 1
        if case["act"] == "none":
            return z, torch.ones_like(z)
        if case["act"] == "relu":
            return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0)
        a, da = z, torch.ones_like(z)
        if case["act"] == "gelu_tanh":
            c = 2 * math.sqrt(2 / math.pi)
            a, da = c * (z + GELU_A * z ** 3), c * (1 + 3 * GELU_A * z ** 2)
        sig = 1 / (1 + torch.exp(-a))
        return z * sig, sig + z * sig * (1 - sig) * da

    if case["op"] == "linear_fwd":
        y, zs = torch.zeros(rows, N, **d64), torch.zeros(rows, N, **d64)
        for e, (a, b) in enumerate(spans):
            z = st["x"][a:b].double() @ st["w"][e].double().T
            if st["b"] is not None:
                z += st["b"][e].double()
            zs[a:b] = z
            y[a:b] = gate(z)[0]
            if st["res"] is not None:
                y[a:b] += st["res"][a:b].double()
        return dict(y=y, z=zs) if case["save_z"] else dict(y=y)
    dx, dw, db = torch.zeros(rows, Kin, **d64), torch.zeros(G, N, Kin, **d64), torch.zeros(G, N, **d64)
    for e, (a, b) in enumerate(spans):
        dz = st["dy"][a:b].double() * gate(st["z"][a:b].double())[1]
        dx[a:b] = dz @ st["w"][e].double()
        dw[e] = dz.T @ st["x"][a:b].double()
        db[e] = dz.sum(0)
    return dict(dx=dx, dw=dw, db=db) if case["bias"] else dict(dx=dx, dw=dw)


def _exact_adamw(case, st):
    t = st["step"] + 1
    d = lambda x: x.double()  # noqa: E731
    f32 = case["state"] == "fp32"

    def value(q, sb):  # E4M3 from its fields: 2^(e-7) (1 + m/8), or m 2^-9 where e is 0
        c = q.long()
        e, man = (c >> 3) & 15, d(c & 7)
        mag = torch.where(e > 0, torch.exp2(d(e) - 7) * (1 + man / 8), man / 512)
        mag = torch.where(c > 127, -mag, mag).reshape(-1, 32)
        return (mag * torch.exp2(d(sb) - 127)[:, None]).reshape(-1)

    g = d(st["g"]) * d(st["gscale"])
    m = d(st["m"]) if f32 else value(st["m"], st["ms"])
    v = d(st["v"]) if f32 else value(st["s"], st["ss"]) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    root = torch.sqrt(v)
    wd = torch.zeros(st["total"], device=DEV, dtype=torch.float64)
    wd[: st["edge"]] = DECAY
    p = d(st["p"]) * (1 - LR * wd)
    p -= LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = dict(p=p)
    if case["copy"]:
        out["copy"] = p
    if f32:
        return dict(out, m=m, v=v)
    del p, wd, g, v
    st["step"] = t
    bits = _random(st)

    def stored(x, u, positive):  # stochastic rounding to the next lower or higher E4M3 value
        a = x.abs().reshape(-1, 32)
        top = a.amax(1)
        ex = torch.ceil(torch.log2(top / 448)).clamp(min=-127)
        ex = torch.where(top > 0, ex, -127.0)
        y = (a / torch.exp2(ex)[:, None]).reshape(-1)
        step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
        q = torch.floor(y / step + u) * step
        if positive:
            q = torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
        return torch.where(x < 0, -q, q), torch.exp2(ex)

    out["m"], out["ms"] = stored(m, (d(bits & 0xFFFF) + 0.5) / 65536, False)
    out["s"], out["ss"] = stored(root, (d(bits >> 16) + 0.5) / 65536, True)
    return out
