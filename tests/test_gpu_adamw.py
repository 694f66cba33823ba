"""The AdamW step against a plain 64-bit implementation.

Tolerances (derived): each fp32 operation adds at most 2^-24 of its result (square root and
division at most 2^-22 each); the products beta m and (1 - beta) g and their constants add a
few such terms of their own magnitudes. A stored code must be one that the definition gives for
some value within that error of the exact one."""
import numpy as np
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8


def _t():
    import torch
    return torch


def mix(h):
    h = h.astype(np.uint32)
    with np.errstate(over="ignore"):
        h ^= h >> np.uint32(16)
        h *= np.uint32(0x85EBCA6B)
        h ^= h >> np.uint32(13)
        h *= np.uint32(0xC2B2AE35)
        h ^= h >> np.uint32(16)
    return h


def random_bits(first, n, seed):
    i = np.arange(first, first + n, dtype=np.uint64)
    hi, lo = (i >> np.uint64(32)).astype(np.uint32), (i & np.uint64(0xFFFFFFFF)).astype(np.uint32)
    key = mix(mix(hi ^ np.uint32(seed & 0xFFFFFFFF)) ^ np.uint32(seed >> 32))
    h = mix(lo ^ key)
    with np.errstate(over="ignore"):
        hp = mix(h + np.uint32(0x9E3779B9))
    return h & np.uint32(0xFFFF), h >> np.uint32(16), hp >> np.uint32(16)


def e4m3(code):
    code = np.asarray(code).astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8), m * 2.0 ** -9)
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def decode(q, sb):
    s = np.where(sb == 255, np.nan, 2.0 ** (sb.astype(np.float64) - 127))
    return e4m3(q) * np.repeat(s, 32)[:q.size]


def scale_bytes(x):
    """E8M0 byte per block of 32: the least power of two with max / scale <= 448."""
    n = x.size
    pad = np.zeros(-(-n // 32) * 32)
    pad[:n] = np.abs(x)
    top = pad.reshape(-1, 32).max(1)
    with np.errstate(divide="ignore"):
        k = np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0))
    k = np.where(2.0 ** k * 448 < top, k + 1, k)
    return np.where(top > 0, np.maximum(k + 127, 0), 0).astype(np.uint8)


def codes(x, sb, u, positive):
    """E4M3 codes of x / scale rounded with offsets u in [0, 1) (u = None: to nearest even)."""
    y = np.abs(x) / np.repeat(2.0 ** (sb.astype(np.float64) - 127), 32)[:x.size]
    e = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    k = np.round(y / step) if u is None else np.floor(y / step + u)  # np.round: ties to even
    v = k * step
    ev = np.floor(np.log2(np.maximum(v, 2.0 ** -6)))
    c = np.where(v < 2.0 ** -6, v * 512, (ev + 7) * 8 + (v / 2.0 ** ev - 1) * 8).astype(np.int64)
    if positive:
        c = np.where((x > 0) & (c == 0), 1, c)
    return c


class Tensors:
    """Tensors of the given sizes with guard elements behind each, and their 64-bit values."""

    def __init__(self, sizes, p="fp32", g="bf16", state="fp32", copy=True, seed=0, gstd=1e-2):
        torch = _t()
        gen = torch.Generator("cuda").manual_seed(seed)
        f, b = torch.float32, torch.bfloat16
        self.p_dt, self.g_dt = (f if p == "fp32" else b), (f if g == "fp32" else b)
        self.s8 = state == "8bit"
        self.sizes, self.t, first = sizes, [], 0
        rnd = lambda n, std: torch.randn(n, device="cuda", generator=gen) * std  # noqa: E731
        for k, n in enumerate(sizes):
            nb = -(-n // 32)
            d = dict(n=n, first=first, weight_decay=0.1 if k % 2 == 0 else 0.0)
            first += nb * 32
            guard = lambda t, v=7.0: torch.cat([t, torch.full((40,), v, device="cuda", dtype=t.dtype)])  # noqa: E731
            d["p"] = guard(rnd(n, 0.02).to(self.p_dt))
            d["g"] = guard(rnd(n, gstd).to(self.g_dt))
            d["copy"] = guard(torch.zeros(n, device="cuda", dtype=b)) if copy else None
            if self.s8:
                u8 = dict(dtype=torch.uint8, device="cuda")
                m = torch.randint(0, 256, (n,), generator=gen, **u8)
                m[(m & 127) == 127] = 3
                d["m"] = guard(m, 77)
                d["v"] = guard(torch.randint(1, 127, (n,), generator=gen, **u8), 77)
                d["m_scale"] = guard(torch.randint(95, 112, (nb,), generator=gen, **u8), 77)
                d["v_scale"] = guard(torch.randint(95, 112, (nb,), generator=gen, **u8), 77)
            else:
                d["m"], d["v"] = guard(rnd(n, 1e-3)), guard(rnd(n, 1e-3).square())
            self.t.append(d)
        self.gs = torch.tensor([0.5], device="cuda")

    def list(self):
        return B.make_adamw_list([{k: v for k, v in d.items() if k != "first"} for d in self.t])

    def host(self):
        h = []
        for d in self.t:
            n, e = d["n"], dict(d)
            for k in ("p", "g", "copy"):
                e[k] = None if d[k] is None else d[k][:n].double().cpu().numpy()
            for k, s in (("m", "m_scale"), ("v", "v_scale")):
                if self.s8:
                    e[k + "q"] = d[k][:n].cpu().numpy()
                    e[s] = d[s][:-(-n // 32)].cpu().numpy()
                    e[k] = decode(e[k + "q"], e[s])
                    if k == "v":
                        e[k] = e[k] ** 2
                else:
                    e[k] = d[k][:n].double().cpu().numpy()
            h.append(e)
        return h

    def guards_intact(self):
        for d in self.t:
            for k in ("p", "g", "copy"):
                if d[k] is not None:
                    assert bool((d[k][d["n"]:] == 7).all()), k
            for k in ("m", "v", "m_scale", "v_scale"):
                if d.get(k) is not None:
                    assert bool((d[k][-40:] == (77 if self.s8 else 7)).all()), k


def config(t, step=3, flags=0, seed=0x123456789ABCDEF0, **kw):
    torch = _t()
    d = lambda x: B.MOK_DTYPE_F32 if x == torch.float32 else B.MOK_DTYPE_BF16  # noqa: E731
    a = dict(lr=LR, beta1=B1, beta2=B2, eps=EPS, step=step, seed=seed, p_dtype=d(t.p_dt),
             g_dtype=d(t.g_dt), state=B.MOK_STATE_MXFP8 if t.s8 else B.MOK_STATE_F32, flags=flags)
    a.update(kw)
    return B.make_adamw(**a)


def check(before, after, t, step, sr, seed):
    for b, a in zip(before, after):
        n = b["n"]
        if n == 0:
            continue
        g = b["g"] * 0.5
        m = B1 * b["m"] + (1 - B1) * g
        v = B2 * b["v"] + (1 - B2) * g * g
        em = 5 * U * (np.abs(B1 * b["m"]) + np.abs((1 - B1) * g))
        ev = 8 * U * v
        s = np.sqrt(v)
        es = s * (0.5 * 8 * U + 4 * U)
        den = s / np.sqrt(1 - B2 ** step) + EPS
        k = LR / (1 - B1 ** step)
        upd = k * m / den
        keep = b["p"] * (1 - LR * b["weight_decay"])
        p = keep - upd
        ep = 3 * U * np.abs(keep) + k * em / den + 24 * U * np.abs(upd) + U * np.abs(p)
        rm, rv, rp = (r.astype(np.float64) for r in random_bits(b["first"], n, seed))
        if t.p_dt == _t().float32:
            assert (np.abs(a["p"] - p) <= ep).all()
            if a["copy"] is not None:
                assert (np.abs(a["copy"] - a["p"]) <= 2.0 ** -8 * np.abs(a["p"])).all()
                cp = _t().from_numpy(a["p"]).float().bfloat16().double().numpy()
                assert np.array_equal(a["copy"], cp)
        elif sr:
            mag = np.abs(p)
            step_ = 2.0 ** (np.floor(np.log2(np.maximum(mag, 1e-300))) - 7)
            lo = np.floor((mag - ep) / step_ + rp / 65536) * step_
            hi = np.floor((mag + ep) / step_ + rp / 65536) * step_
            got = np.abs(a["p"])
            assert ((got >= lo) & (got <= hi) | (np.abs(p) <= ep)).all()
        else:
            assert (np.abs(a["p"] - p) <= ep + 2.0 ** -8 * (np.abs(p) + ep)).all()
        if not t.s8:
            assert (np.abs(a["m"] - m) <= em).all() and (np.abs(a["v"] - v) <= ev).all()
            continue
        for name, x, e, r, pos in (("m", m, em, rm, False), ("v", s, es, rv, True)):
            sb = a[name + "_scale"].astype(np.int64)
            lo_s, hi_s = scale_bytes(np.abs(x) - np.minimum(e, np.abs(x))), scale_bytes(np.abs(x) + e)
            assert ((sb >= lo_s) & (sb <= hi_s)).all()
            u = (r + 0.5) / 65536 if sr else None
            mag = np.abs(x)
            top = 448 * np.repeat(2.0 ** (sb - 127.0), 32)[:n]
            lo = codes(np.maximum(mag - e, 0), sb, u, pos)
            hi = codes(np.minimum(mag + e, top), sb, u, pos)
            q = a[name + "q"].astype(np.int64)
            c = q & 127
            assert ((c >= lo) & (c <= hi)).all()
            if pos:
                assert (q < 128).all()
            else:
                assert ((q >> 7 == 1) == (x < 0))[np.abs(x) > e].all()


MODES = [("fp32", "bf16", "fp32"), ("fp32", "fp32", "fp32"), ("bf16", "bf16", "fp32"),
         ("bf16", "fp32", "8bit"), ("fp32", "bf16", "8bit"), ("fp32", "fp32", "8bit"),
         ("bf16", "bf16", "8bit"), ("bf16", "fp32", "fp32")]


@pytest.mark.parametrize("sr", [0, 1])
@pytest.mark.parametrize("p,g,state", MODES)
def test_step(p, g, state, sr):
    sizes = [1, 7, 8, 31, 32, 33, 0, 100, 2047, 2048, 2049, 5000, 4096]
    t = Tensors(sizes, p, g, state, copy=p == "fp32", seed=sr)
    lst, seed = t.list(), 0x123456789ABCDEF0
    for step in (1, 2, 50):
        before = t.host()
        B.check(B.mok_adamw_step(config(t, step, sr * B.MOK_ADAMW_STOCHASTIC, seed + step), lst,
                                 t.gs))
        check(before, t.host(), t, step, sr, seed + step)
        t.guards_intact()


def test_many_tensors_equal_one_by_one():
    """450 tensors go in several launches; the element numbers, and so the random bits, run on."""
    torch = _t()
    sizes = [1 + (37 * i) % 90 for i in range(450)]
    a, b = (Tensors(sizes, "bf16", "bf16", "8bit", copy=False, seed=5) for _ in range(2))
    cfg = config(a, 2, B.MOK_ADAMW_STOCHASTIC)
    before = a.host()
    B.check(B.mok_adamw_step(cfg, a.list(), a.gs))
    check(before, a.host(), a, 2, True, 0x123456789ABCDEF0)
    # the same again: the same bits
    B.check(B.mok_adamw_step(cfg, b.list(), b.gs))
    for x, y in zip(a.t, b.t):
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            assert torch.equal(x[k], y[k])
    a.guards_intact()


def test_no_grad_scale_and_side_stream():
    torch = _t()
    a, b = Tensors([3000], seed=1), Tensors([3000], seed=1)
    s = torch.cuda.Stream()
    one = torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    B.check(B.mok_adamw_step(config(a), a.list(), None, s))
    s.synchronize()
    B.check(B.mok_adamw_step(config(b), b.list(), one))
    for k in ("p", "m", "v", "copy"):
        assert torch.equal(a.t[0][k], b.t[0][k])


@pytest.mark.parametrize("state", ["fp32", "8bit"])
def test_zero_and_non_finite_gradients(state):
    torch = _t()
    t = Tensors([128], "fp32", "fp32", state, seed=3)
    d = t.t[0]
    for k in ("m", "v", "m_scale", "v_scale"):
        if d.get(k) is not None:
            d[k].zero_()
    d["g"].zero_()
    d["g"][40] = float("inf")
    d["g"][100] = float("nan")
    p0 = d["p"].clone()
    B.check(B.mok_adamw_step(config(t), t.list(), t.gs))
    h = t.host()[0]
    # zero state and zero gradient: only the decay, and the state stays zero
    assert np.array_equal(h["m"][:32], np.zeros(32)) and np.array_equal(h["v"][:32], np.zeros(32))
    keep = p0[:32].double().cpu().numpy() * (1 - LR * 0.1)
    assert (np.abs(h["p"][:32] - keep) <= 2 * U * np.abs(keep)).all()
    if state == "8bit":
        # the whole block of 32 that holds a non-finite value reads back as NaN
        assert np.isnan(h["m"][32:64]).all() and np.isnan(h["v"][96:128]).all()
        assert np.isfinite(h["m"][64:96]).all()
    else:
        assert np.isinf(h["m"][40]) and np.isnan(h["m"][100]) and np.isfinite(h["m"][41])


def test_eight_bit_states_keep_small_changes():
    """With zero gradients m shrinks by 1/1000 a step, far below a code's step: stochastic rounding
    keeps the decay on average, rounding to nearest never moves."""
    torch = _t()
    n, steps = 1 << 16, 100
    for sr in (1, 0):
        t = Tensors([n], "fp32", "bf16", "8bit", seed=9)
        d = t.t[0]
        d["g"][:n] = 0
        d["m"][:n] = 0x30          # 1/2 of the block's scale, and one larger value per block
        d["m"][0:n:32] = 0x70
        lst = t.list()
        m0 = t.host()[0]["m"]
        for k in range(steps):
            B.check(B.mok_adamw_step(config(t, 1 + k, sr, seed=1000 + k, beta1=0.999), lst, t.gs))
        m1 = t.host()[0]["m"]
        small = np.arange(n) % 32 != 0
        got = (m1[small] / m0[small]).mean()
        want = 0.999 ** steps
        if sr:
            # one element's spread: at most half a step (1/8) a move, at most 100 moves; the
            # mean of 63488 of them within 6 standard deviations
            assert abs(got - want) <= 6 * (0.5 / 8) * np.sqrt(steps) / np.sqrt(small.sum())
        else:
            assert got == 1.0


def test_element_numbers_past_32_bits():
    torch = _t()
    n, tail = (1 << 32) + 100, 4096
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    z = lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    d = dict(n=n, first=0, weight_decay=0.1, copy=None, p=z(n, torch.bfloat16),
             g=z(n, torch.bfloat16), m=z(n, torch.uint8), v=z(n, torch.uint8),
             m_scale=z(-(-n // 32), torch.uint8), v_scale=z(-(-n // 32), torch.uint8))
    small = Tensors([tail + 4], "bf16", "bf16", "8bit", copy=False, seed=8)
    lo = n - n % 32 - tail + 32  # a block boundary
    k = n - lo
    for name in ("p", "g", "m", "v"):
        d[name][lo:] = small.t[0][name][:k]
    for name in ("m_scale", "v_scale"):
        d[name][lo // 32:] = small.t[0][name][:-(-k // 32)]
    t = Tensors([k], "bf16", "bf16", "8bit", copy=False, seed=8)
    view = lambda: dict(d, n=k, first=lo, **{a: d[a][lo:] for a in ("p", "g", "m", "v")},  # noqa: E731
                        **{a: d[a][lo // 32:] for a in ("m_scale", "v_scale")})
    t.t = [view()]
    before = t.host()
    B.check(B.mok_adamw_step(config(t, 4, 1), B.make_adamw_list([d]), t.gs))
    t.t = [view()]
    check(before, t.host(), t, 4, True, 0x123456789ABCDEF0)


def test_refusals():
    t = Tensors([64], "fp32", "bf16", "8bit")
    cfg, d = config(t), {k: v for k, v in t.t[0].items() if k != "first"}
    bad = B.MOK_ERR_INVALID_ARG

    def call(c=cfg, **kw):
        return B.mok_adamw_step(c, B.make_adamw_list([dict(d, **kw)]), t.gs)

    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        assert call(**{k: None}) == bad, k
    for k in ("p", "g", "m", "v", "copy"):
        assert call(**{k: d[k].data_ptr() + 4}) == bad, k
    assert call(n=-1) == bad
    assert call(weight_decay=float("nan")) == bad
    b16 = config(t, p_dtype=B.MOK_DTYPE_BF16)
    assert call(b16) == bad  # a copy of parameters that are bf16 already
    assert call(config(t, step=0)) == bad
    assert call(config(t, abi_version=1)) == B.MOK_ERR_ABI
    assert B.mok_adamw_step(cfg, B.make_adamw_list([]), t.gs) == B.MOK_OK
    assert call(n=0, p=None, g=None) == B.MOK_OK
