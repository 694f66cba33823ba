"""The linear layer and its gradients against plain products in 64 bits.

Tolerances (derived): an fp32 tensor-core sum of n terms is within 2^-19 max(1, sqrt(n / 2048))
of the sum of its terms' magnitudes (measured on this hardware, tests/test_gpu_backward.py);
storing or feeding bf16 adds 2^-8 of a value; the activations and their slopes are within
2^-20 (1 + |z|) and have slopes of at most 1.2."""
import math

import numpy as np
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu
ACTS = dict(none=B.MOK_ACT_NONE, relu=B.MOK_ACT_RELU, silu=B.MOK_ACT_SILU,
            gelu_tanh=B.MOK_ACT_GELU_TANH, gelu=B.MOK_ACT_GELU)
U16 = 2.0 ** -8


def _t():
    import torch
    return torch


def dot_rel(n):
    return 2.0 ** -19 * max(1.0, math.sqrt(n / 2048))


def act64(z, name):
    torch = _t()
    one = torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return z, one


class Lin:
    """Inputs of one configuration; every array has guard columns (NaN) and, when grouped, rows
    outside every group (NaN) that must not be touched."""

    def __init__(self, G=1, R=64, Kin=64, N=64, act="none", out="bf16", grad="bf16", bias=True,
                 res=True, z=True, extra=0, counts=None, seed=0, grouped=None, spare=0):
        torch = _t()
        self.act, self.G, self.Kin, self.N = act, G, Kin, N
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen = gen
        grouped = G > 1 if grouped is None else grouped
        up8 = lambda n: (n + 7) // 8 * 8 + extra  # noqa: E731
        self.ld_in, self.ld_out = up8(Kin), up8(N)
        if grouped:
            if counts is None:
                r = np.random.default_rng(seed)
                p = r.random(G) * (r.random(G) > 0.25) + 1e-9
                counts = np.floor(p / p.sum() * R).astype(np.int64)
            counts = np.asarray(counts)
            self.counts = counts
            self.starts = np.concatenate([[0], np.cumsum((counts + 15) // 16 * 16)])
            self.rows = int(self.starts[-1]) + spare
        else:
            self.counts, self.starts, self.rows = np.array([R]), np.array([0, R]), R
        self.grouped = grouped
        f32, bf = torch.float32, torch.bfloat16
        self.out_dt = f32 if out == "fp32" else bf
        self.grad_dt = f32 if grad == "fp32" else bf
        dt = lambda s: B.MOK_DTYPE_F32 if s == "fp32" else B.MOK_DTYPE_BF16  # noqa: E731
        self.cfg = B.make_linear(self.rows, Kin, N, G, ACTS[act], dt(out), dt(grad), self.ld_in,
                                 self.ld_in, self.ld_out)
        assert B.mok_check_linear_config(self.cfg) == B.MOK_OK
        self.x = self.rand(self.rows, Kin, self.ld_in, bf)
        self.w = self.rand(G * N, Kin, self.ld_in, bf, 1 / math.sqrt(Kin), rows_all=True)
        self.b = torch.randn(G * N, device="cuda", generator=gen) * 0.5 if bias else None
        self.res = self.rand(self.rows, N, self.ld_out, bf) if res else None
        self.z = self.rand(self.rows, N, self.ld_out, bf, 2.0) if z else None
        self.dy = self.rand(self.rows, N, self.ld_out, self.out_dt)
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
        self.d_starts, self.d_counts = (i32(self.starts), i32(self.counts)) if grouped else (None, None)

    def spans(self):
        return [(int(self.starts[g]), int(self.starts[g] + self.counts[g])) for g in range(self.G)]

    def pads(self):
        if not self.grouped:
            return []
        return [(b, (b + 15) // 16 * 16) for _, b in self.spans()]

    def rand(self, rows, cols, ld, dt, std=1.0, rows_all=False):
        torch = _t()
        buf = torch.full((max(rows, 1), ld), float("nan"), device="cuda", dtype=dt)
        live = (torch.randn(rows, cols, device="cuda", generator=self.gen) * std).to(dt)
        if rows_all:
            buf[:rows, :cols] = live
            return buf
        for a, b in self.spans():
            buf[a:b, :cols] = live[a:b]
        for a, b in self.pads():
            buf[a:b, :cols] = 0
        return buf

    def empty(self, rows, ld, dt, fill=7.0):
        return _t().full((max(rows, 1), ld), fill, device="cuda", dtype=dt)

    def ws(self, which):
        torch = _t()
        n = B.mok_linear_workspace_size(self.cfg, which)
        assert n > 0
        return torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda"), n

    def forward(self, stream=None, y=None):
        y = self.empty(self.rows, self.ld_out, self.out_dt) if y is None else y
        z = self.empty(self.rows, self.ld_out, _t().bfloat16) if self.z is not None else None
        ws, n = self.ws(B.MOK_LINEAR_FORWARD)
        st = B.mok_linear_forward(self.cfg, self.x, self.w, self.b, self.res, self.d_starts,
                                  self.d_counts, y, z, ws, n, stream)
        assert st == B.MOK_OK
        self._keep = ws
        return y, z

    def backward(self, dx=True, dw=True, db=True, stream=None):
        torch = _t()
        o = [self.empty(self.rows, self.ld_in, self.grad_dt) if dx else None,
             self.empty(self.G * self.N, self.ld_in, self.grad_dt) if dw else None,
             torch.full((self.G * self.N + 3,), 7.0, device="cuda") if db else None]
        ws, n = self.ws(B.MOK_LINEAR_BACKWARD)
        st = B.mok_linear_backward(self.cfg, self.x, self.w, self.z, self.dy, self.d_starts,
                                   self.d_counts, *o, ws, n, stream)
        assert st == B.MOK_OK
        self._keep = ws
        return o


def device_ok():
    st, dev = B.mok_read_device_status()
    B.mok_clear_device_status()
    return (st, dev) == (B.MOK_OK, B.MOK_OK)


def untouched(c, buf, rows, cols):
    """Guard columns, and rows that belong to no group and no padding, keep their fill."""
    torch = _t()
    mask = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    for (a, b), (_, p) in zip(c.spans(), c.pads() or [(0, b) for _, b in c.spans()]):
        mask[a:max(b, p), :cols] = False
    assert bool((buf[mask] == 7).all())


def check_forward(c):
    torch = _t()
    y, z = c.forward()
    assert device_ok()
    k = c.Kin
    for g, (a, b) in enumerate(c.spans()):
        x, w = c.x[a:b, :k].double(), c.w[g * c.N:(g + 1) * c.N, :k].double()
        zz = x @ w.T
        mag = x.abs() @ w.abs().T
        if c.b is not None:
            zz = zz + c.b[g * c.N:(g + 1) * c.N].double()
        e = dot_rel(k) * mag + 2.0 ** -23 * zz.abs()
        val, _ = act64(zz, c.act)
        if c.res is not None:
            val = val + c.res[a:b, :c.N].double()
        ey = 1.2 * e + 2.0 ** -20 * (1 + zz.abs()) * (c.act != "none") + 2.0 ** -23 * val.abs()
        if c.out_dt == torch.bfloat16:
            ey = ey + U16 * (val.abs() + ey)
        assert bool(((y[a:b, :c.N].double() - val).abs() <= ey).all())
        if z is not None:
            assert bool(((z[a:b, :c.N].double() - zz).abs() <= e + U16 * (zz.abs() + e)).all())
    for a, b in c.pads():
        assert bool((y[a:b, :c.N] == 0).all())
        assert z is None or bool((z[a:b, :c.N] == 0).all())
    untouched(c, y, c.rows, c.N)
    if z is not None:
        untouched(c, z, c.rows, c.N)
    return y, z


def check_backward(c, parts=(True, True, True)):
    torch = _t()
    dx, dw, db = c.backward(*parts)
    assert device_ok()
    k, N = c.Kin, c.N
    exact_dz = c.act == "none" and c.out_dt == torch.bfloat16
    store = U16 if c.grad_dt == torch.bfloat16 else 2.0 ** -24
    for g, (a, b) in enumerate(c.spans()):
        n = b - a
        x, w = c.x[a:b, :k].double(), c.w[g * N:(g + 1) * N, :k].double()
        dy = c.dy[a:b, :N].double()
        dz, edz = dy, torch.zeros_like(dy)
        if c.act != "none":
            zz = c.z[a:b, :N].double()
            dz = dy * act64(zz, c.act)[1]
            edz = dy.abs() * 2.0 ** -20 * (1 + zz.abs())
        round_dz = edz + (0.0 if exact_dz else U16 * (dz.abs() + edz))
        if dx is not None:
            ref = dz @ w
            tol = round_dz @ w.abs() + dot_rel(N) * ((dz.abs() + round_dz) @ w.abs())
            tol = tol + store * (ref.abs() + tol)
            assert bool(((dx[a:b, :k].double() - ref).abs() <= tol).all())
        if dw is not None:
            ref = dz.T @ x
            tol = round_dz.T @ x.abs() + dot_rel(max(n, 1)) * ((dz.abs() + round_dz).T @ x.abs())
            tol = tol + store * (ref.abs() + tol)
            got = dw[g * N:(g + 1) * N, :k].double()
            assert bool(((got - ref).abs() <= tol).all())
        if db is not None:
            ref = dz.sum(0)
            tol = edz.sum(0) + (n + 8) * 2.0 ** -24 * dz.abs().sum(0)
            assert bool(((db[g * N:(g + 1) * N].double() - ref).abs() <= tol).all())
    if dx is not None:
        for a, b in c.pads():
            assert bool((dx[a:b, :k] == 0).all())
        untouched(c, dx, c.rows, k)
    if dw is not None:
        assert bool((dw[:, k:] == 7).all())
    if db is not None:
        assert bool((db[-3:] == 7).all())
    return dx, dw, db


CASES = [
    dict(R=1, Kin=1, N=1),
    dict(R=1, Kin=4096, N=513, act="silu"),
    dict(R=3, Kin=72, N=8, act="relu", bias=False),
    dict(R=8, Kin=1000, N=40, out="fp32"),
    dict(R=2, Kin=515, N=130, act="gelu", out="fp32"),
    dict(R=5, Kin=2050, N=300, act="silu"),
    dict(R=2, Kin=72, N=8200),
    dict(R=2, Kin=1029, N=2051, act="gelu", extra=8),
    dict(R=4, Kin=2070, N=77, act="silu"),
    dict(R=3, Kin=40, N=1024, out="fp32"),
    dict(R=30, Kin=500, N=500, act="silu"),
    dict(R=12, Kin=8200, N=100, act="relu"),
    dict(R=7, Kin=1030, N=8200),
    dict(R=14, Kin=1301, N=77, act="gelu_tanh", extra=8),
    dict(R=27, Kin=640, N=600, act="relu", out="fp32"),
    dict(R=40, Kin=2100, N=300, out="fp32", res=False, z=False),
    dict(R=5000, Kin=300, N=2600, act="silu"),
    dict(R=17, Kin=15, N=300, act="gelu"),
    dict(R=33, Kin=264, N=1030, act="gelu_tanh", extra=8),
    dict(R=255, Kin=129, N=127, act="silu", res=False),
    dict(R=257, Kin=64, N=256, z=False),
    dict(R=300, Kin=2600, N=130, out="fp32", act="relu"),
    dict(R=513, Kin=520, N=384, grad="fp32", extra=16),
    dict(R=1200, Kin=1024, N=640, act="gelu_tanh", out="fp32", grad="fp32"),
    dict(G=4, R=100, Kin=96, N=72, act="silu"),
    dict(G=3, counts=[0, 0, 0], Kin=64, N=64, spare=16),
    dict(G=5, counts=[1, 0, 300, 16, 257], Kin=200, N=136, act="gelu_tanh", extra=8, spare=48),
    dict(G=8, R=1500, Kin=512, N=257, act="none", spare=32),
    dict(G=40, R=900, Kin=128, N=128, act="relu", out="fp32"),
    dict(G=1, grouped=True, counts=[50], Kin=64, N=64, act="silu", spare=16),
    dict(G=1024, R=2000, Kin=16, N=24, act="gelu"),
    dict(R=9001, Kin=70, N=61, act="silu"),
    dict(R=16384, Kin=64, N=64, act="gelu_tanh", grad="fp32"),
    dict(R=150, Kin=8200, N=140, act="relu", extra=8),
    dict(R=100, Kin=5000, N=90, out="fp32", res=False, z=False),
    dict(R=40, Kin=4097, N=515, out="fp32", act="silu"),
    dict(R=90, Kin=130, N=6001, act="gelu"),
    dict(R=3000, Kin=520, N=300, grad="fp32", bias=False),
    dict(G=2, counts=[700, 41], Kin=300, N=200, act="silu", out="fp32"),
    dict(G=3, counts=[0, 1, 600], Kin=2000, N=90, act="gelu_tanh", spare=64),
]
ID = lambda k: "-".join("%s%s" % i for i in k.items()).replace(" ", "")  # noqa: E731


@pytest.mark.parametrize("kw", CASES, ids=ID)
def test_forward(kw):
    check_forward(Lin(**kw))


@pytest.mark.parametrize("kw", CASES, ids=ID)
def test_backward(kw):
    kw = dict(kw)
    if kw.get("act", "none") != "none":
        kw["z"] = True
    check_backward(Lin(**kw))


def test_each_gradient_alone_gives_the_same_bits():
    torch = _t()
    c = Lin(G=4, R=500, Kin=200, N=150, act="silu")
    every = check_backward(c)
    for i in range(3):
        parts = [j == i for j in range(3)]
        got = check_backward(c, parts)
        assert torch.equal(got[i][..., :8], every[i][..., :8])


def test_no_rows():
    c = Lin(R=0, Kin=40, N=24)
    c.forward()
    dx, dw, db = c.backward()
    assert bool((dw[:, :40] == 0).all()) and bool((dw[:, 40:] == 7).all())
    assert bool((db[:24] == 0).all()) and device_ok()


def test_repeat_side_stream_and_in_place_residual():
    torch = _t()
    c = Lin(R=700, Kin=320, N=264, act="gelu_tanh")
    y, z = check_forward(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, z2 = c.forward(stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(z, z2)
    a = c.backward()
    torch.cuda.synchronize()
    b = c.backward(stream=s)
    s.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    r = c.res.clone()  # y = act(z) + y
    c.res = r
    c.forward(y=r)
    assert torch.equal(r[:, :264], y[:, :264])


def test_gradients_against_differences():
    """<y, dy> along a random direction of the inputs, by central differences of the forward
    (fp32 outputs; the step moves bf16 weights and inputs by exact amounts)."""
    torch = _t()
    c = Lin(R=96, Kin=128, N=80, act="gelu_tanh", out="fp32", grad="fp32", res=False)
    _, c.z = c.forward()
    dx, dw, db = c.backward()
    N, k, eps = c.N, c.Kin, 2.0 ** -5

    def loss():
        y, _ = c.forward()
        return float((y[:, :N].double() * c.dy[:, :N].double()).sum())

    for name, grad in (("w", dw), ("x", dx), ("b", db)):
        p = getattr(c, name)
        keep = p.clone()
        if name == "b":
            d = torch.randn(p.shape, device="cuda", generator=c.gen)
            ana = float((db[:N].double() * d.double()).sum())
            terms = float((db[:N].double() * d.double()).abs().sum())
            moved = lambda s: keep + s * eps * d  # noqa: E731
        else:
            # a direction of bf16 values; what a rounded move really moved is what counts
            d = torch.randn(p[:, :k].shape, device="cuda", generator=c.gen).to(p.dtype)
            d = d * (0.1 if name == "w" else 1.0)
            hi, lo = keep.clone(), keep.clone()
            hi[:, :k] = (keep[:, :k].float() + eps * d.float()).to(p.dtype)
            lo[:, :k] = (keep[:, :k].float() - eps * d.float()).to(p.dtype)
            step = (hi[:, :k].double() - lo[:, :k].double()) / (2 * eps)
            ana = float((grad[:, :k].double() * step).sum())
            terms = float((grad[:, :k].double() * step).abs().sum())
            moved = lambda s: hi if s > 0 else lo  # noqa: E731
        setattr(c, name, moved(1))
        up = loss()
        setattr(c, name, moved(-1))
        down = loss()
        setattr(c, name, keep)
        # rounding of z and dz (2^-8 each) and the third-order term of a step of 1/32
        assert abs((up - down) / (2 * eps) - ana) <= 3 * U16 * terms, name


def test_bad_layouts_are_reported():
    torch = _t()
    for starts, counts, rows in (([0, 20, 40], [5, 5], 64),      # not a multiple of 16
                                 ([0, 16, 32], [17, 5], 64),     # runs into the next group
                                 ([0, 16, 25], [5, 9], 64),      # no room for the padding
                                 ([0, 16, 96], [5, 70], 64),     # past the rows
                                 ([0, 16, 32], [-1, 3], 64)):
        c = Lin(G=2, counts=[5, 3], Kin=32, N=24, spare=32)
        c.rows = rows
        c.d_starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        c.d_counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
        assert c.cfg.rows == 64
        B.mok_clear_device_status()
        c.forward()
        st, dev = B.mok_read_device_status()
        assert dev == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()
        c.backward()
        st, dev = B.mok_read_device_status()
        assert dev == B.MOK_ERR_DEVICE_INVARIANT
        B.mok_clear_device_status()


def test_refusals():
    c = Lin(R=32, Kin=64, N=48, act="silu")
    g = Lin(G=2, counts=[5, 3], Kin=32, N=24)
    bad = B.MOK_ERR_INVALID_ARG
    y, z = c.empty(32, 48, c.out_dt), c.z
    ws, n = c.ws(B.MOK_LINEAR_BACKWARD)

    def fwd(c=c, x=c.x, w=c.w, y=y, starts=None, counts=None, ws=ws, n=n):
        return B.mok_linear_forward(c.cfg, x, w, None, None, starts, counts, y, None, ws, n)

    assert fwd() == B.MOK_OK
    assert fwd(x=None) == bad and fwd(w=None) == bad and fwd(y=None) == bad
    assert fwd(x=c.x.data_ptr() + 2) == bad and fwd(y=y.data_ptr() + 8) == bad
    assert fwd(starts=g.d_starts) == bad
    assert fwd(c=g, x=g.x, w=g.w) == bad            # groups without their rows
    assert fwd(ws=None) == B.MOK_ERR_WORKSPACE and fwd(n=0) == B.MOK_ERR_WORKSPACE
    assert fwd(ws=ws.data_ptr() + 16) == B.MOK_ERR_WORKSPACE

    def bwd(x=c.x, w=c.w, z=z, dy=c.dy, dx=y, dw=None, db=None):
        return B.mok_linear_backward(c.cfg, x, w, z, dy, None, None, dx, dw, db, ws, n)

    assert bwd(dx=None) == bad                      # nothing asked for
    assert bwd(z=None) == bad and bwd(dy=None) == bad and bwd(w=None) == bad
    assert bwd(x=None, dx=None, dw=y) == bad
    assert device_ok()


@pytest.mark.parametrize("kw", [dict(R=9001, Kin=70, N=61, act="silu"),
                                dict(R=3000, Kin=520, N=300),
                                dict(G=5, counts=[1, 0, 3000, 16, 257], Kin=300, N=136)])
def test_each_gradient_alone_has_the_same_bits(kw):
    torch = _t()
    c = Lin(**kw)
    whole = c.backward()
    for i in range(3):
        alone = c.backward(*[i == j for j in range(3)])
        assert [g is not None for g in alone] == [i == j for j in range(3)]
        assert torch.equal(alone[i].view(torch.uint8), whole[i].view(torch.uint8))
