"""The token sort as operators (row map, dispatch, combine and their gradients) against a plain
64-bit implementation.

Tolerances (derived, not fitted): copies are exact; a sum of n fp32 terms in any order is
within (n + 1) 2^-24 of its exact value relative to the sum of magnitudes; storing bf16 adds
2^-8 of the value."""
import numpy as np
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


class Case:
    """Random routing of T tokens and its schedule (numpy), and the buffers of a configuration."""

    def __init__(self, T, K, E, H, dtype="bf16", capacity=0, ld_extra=0, seed=0, hot=False,
                 spare=0):
        torch = _t()
        r = np.random.default_rng(seed)
        self.T, self.K, self.E, self.H, self.cap = T, K, E, H, capacity
        if hot:  # every token's first choice is expert E - 1
            idx = np.array([(E - 1 + np.arange(K)) % E for _ in range(T)]).reshape(T, K)
        else:
            idx = np.array([r.permutation(E)[:K] for _ in range(T)]).reshape(T, K)
        self.idx = idx.astype(np.int32)
        flat = self.idx.reshape(-1)
        self.perm = np.argsort(flat, kind="stable").astype(np.int32)
        self.inv = np.empty_like(self.perm)
        self.inv[self.perm] = np.arange(T * K, dtype=np.int32)
        self.counts = np.bincount(flat, minlength=E).astype(np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        self.kept = np.minimum(self.counts, capacity) if capacity else self.counts.copy()
        self.starts = np.concatenate([[0], np.cumsum((self.kept + 15) // 16 * 16)]).astype(np.int32)
        rank = self.inv - self.offsets[flat]
        self.map = np.where(rank < self.kept[flat], self.starts[flat] + rank, -1).astype(np.int32)
        self.n_rows = T * K + 15 * min(E, T * K) + spare
        self.dt = torch.float32 if dtype == "fp32" else torch.bfloat16
        self.u = 2.0 ** -24 if dtype == "fp32" else 2.0 ** -8
        per = 4 if dtype == "fp32" else 8
        self.ld = (H + per - 1) // per * per + ld_extra
        self.cfg = B.make_rows(T, K, E, H, n_rows=self.n_rows, ld_tok=self.ld, ld_row=self.ld,
                               dtype=B.MOK_DTYPE_F32 if dtype == "fp32" else B.MOK_DTYPE_BF16,
                               capacity=capacity)
        self.w = r.random((T, K)).astype(np.float32)
        self.r = r
        assert B.mok_check_rows_config(self.cfg) == B.MOK_OK

    def dev(self, a):
        torch = _t()
        # one spare element: an empty array still has an address
        t = torch.zeros(max(a.size, 1), dtype=torch.from_numpy(a).dtype, device="cuda")
        t[:a.size] = torch.from_numpy(np.ascontiguousarray(a)).reshape(-1)
        return t

    def array(self, rows, fill=None):
        """[rows][ld] on the device with H live columns: (the whole buffer, its live values)."""
        torch = _t()
        buf = torch.full((max(rows, 1), self.ld), float("nan"), dtype=self.dt, device="cuda")
        if fill is None:
            live = torch.from_numpy(self.r.standard_normal((rows, self.H)).astype(np.float32))
            buf[:rows, :self.H] = live.to("cuda").to(self.dt)
        else:
            buf[:rows, :self.H] = fill
        return buf

    def values(self, buf, rows):
        return buf[:rows, :self.H].double().cpu().numpy()

    def sched(self):
        self._keep = [self.dev(a) for a in (self.counts, self.offsets, self.perm, self.inv)]
        return B.make_schedule(*self._keep, None, None)

    def valid(self):
        v = np.zeros(self.n_rows, bool)
        v[self.map[self.map >= 0]] = True
        return v

    def pads(self):
        p = np.zeros(self.n_rows, bool)
        for e in range(self.E):
            p[self.starts[e] + self.kept[e]: self.starts[e + 1]] = True
        return p


def clean_status():
    st, dev = B.mok_read_device_status()
    assert st == B.MOK_OK
    B.mok_clear_device_status()
    return dev


CASES = [
    dict(T=0, K=2, E=4, H=16),
    dict(T=1, K=1, E=1, H=1),
    dict(T=1, K=10, E=512, H=4096),
    dict(T=33, K=3, E=7, H=8),
    dict(T=33, K=3, E=7, H=7),
    dict(T=100, K=32, E=40, H=257),
    dict(T=70, K=2, E=1024, H=1030),
    dict(T=257, K=6, E=60, H=1111, dtype="fp32", capacity=20),
    dict(T=64, K=2, E=9, H=100, dtype="fp32", ld_extra=3),
    dict(T=64, K=4, E=9, H=130, ld_extra=1),
    dict(T=90, K=4, E=8, H=264, hot=True),
    dict(T=700, K=5, E=30, H=44, capacity=90, spare=8),
    dict(T=130, K=3, E=5, H=31, ld_extra=1),
    dict(T=130, K=3, E=5, H=250, hot=True),
    dict(T=75, K=9, E=12, H=127, dtype="fp32"),
    dict(T=90, K=4, E=8, H=520, capacity=1),
    dict(T=300, K=8, E=64, H=2056, capacity=17, spare=40),
    dict(T=50, K=1, E=3, H=2060, capacity=20),
    dict(T=50, K=4, E=8, H=1100, dtype="fp32", hot=True),
    dict(T=50, K=5, E=8, H=1300),
    dict(T=50, K=2, E=8, H=515, dtype="fp32", ld_extra=2),
    dict(T=5000, K=2, E=8, H=1027, capacity=1100),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join("%s%s" % i for i in k.items()))
def test_forward(kw):
    torch = _t()
    c = Case(**kw)
    sched = c.sched()
    i32 = dict(dtype=torch.int32, device="cuda")
    m = torch.full((max(c.T * c.K, 1),), 77, **i32)
    starts, kept = torch.full((c.E + 1,), 77, **i32), torch.full((c.E,), 77, **i32)
    assert B.mok_build_row_map(c.cfg, c.dev(c.idx), sched, m, starts, kept) == B.MOK_OK
    assert np.array_equal(m.cpu().numpy()[:c.T * c.K], c.map)
    assert np.array_equal(starts.cpu().numpy(), c.starts)
    assert np.array_equal(kept.cpu().numpy(), c.kept)

    x = c.array(c.T)
    xs = c.array(c.n_rows, fill=9.0)
    assert B.mok_dispatch(c.cfg, x, m, starts, kept, xs) == B.MOK_OK
    want = np.full((c.n_rows, c.H), 9.0)
    live = c.map >= 0
    want[c.map[live]] = c.values(x, c.T)[np.arange(c.T * c.K)[live] // c.K]
    want[c.pads()] = 0
    assert np.array_equal(c.values(xs, c.n_rows), want)
    assert bool(xs[:, c.H:].isnan().all())  # columns past H are left alone

    # rows that nothing maps to hold NaN and must not reach y
    rows = c.array(c.n_rows)
    rows[:c.n_rows][torch.from_numpy(~c.valid()).cuda()] = float("nan")
    rv = np.nan_to_num(c.values(rows, c.n_rows))
    terms = np.where(live[:, None], rv[np.maximum(c.map, 0)], 0.0) if c.T else np.zeros((0, c.H))
    terms = terms.reshape(c.T, c.K, c.H) * c.w[:, :, None]
    for res in (None, c.array(c.T)):
        y = c.array(c.T, fill=3.0)
        assert B.mok_combine(c.cfg, rows, m, c.dev(c.w), res, y) == B.MOK_OK
        add = 0.0 if res is None else c.values(res, c.T)
        ref = terms.sum(1) + add
        mag = np.abs(terms).sum(1) + np.abs(add)
        tol = c.u * np.abs(ref) + (c.K + 2) * 2.0 ** -24 * mag * (1 + c.u)
        assert (np.abs(c.values(y, c.T) - ref) <= tol).all()
        assert bool(y[:, c.H:].isnan().all())
        if res is not None:  # in place: y is its own residual
            r2 = res.clone()
            assert B.mok_combine(c.cfg, rows, m, c.dev(c.w), r2, r2) == B.MOK_OK
            assert torch.equal(r2[:c.T, :c.H], y[:c.T, :c.H])
    assert clean_status() == B.MOK_OK


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join("%s%s" % i for i in k.items()))
def test_backward(kw):
    torch = _t()
    c = Case(**kw)
    m, starts, kept = c.dev(c.map), c.dev(c.starts), c.dev(c.kept)
    live = c.map >= 0
    f = np.arange(c.T * c.K)
    bad = torch.from_numpy(~c.valid()).cuda()
    dxs = c.array(c.n_rows)
    dxs[:c.n_rows][bad] = float("nan")
    dx = c.array(c.T, fill=5.0)
    assert B.mok_dispatch_backward(c.cfg, dxs, m, dx) == B.MOK_OK
    dv = np.nan_to_num(c.values(dxs, c.n_rows))
    terms = np.where(live[:, None], dv[np.maximum(c.map, 0)], 0.0) if c.T else np.zeros((0, c.H))
    terms = terms.reshape(c.T, c.K, c.H)
    ref = terms.sum(1)
    tol = c.u * np.abs(ref) + (c.K + 1) * 2.0 ** -24 * np.abs(terms).sum(1) * (1 + c.u)
    assert (np.abs(c.values(dx, c.T) - ref) <= tol).all()

    rows, dy = c.array(c.n_rows), c.array(c.T)
    rows[:c.n_rows][bad] = float("nan")
    drows = c.array(c.n_rows, fill=9.0)
    dw = torch.full((c.T * c.K + 1,), 9.0, device="cuda")
    assert B.mok_combine_backward(c.cfg, dy, rows, m, starts, kept, c.dev(c.w), drows,
                                  dw) == B.MOK_OK
    g = c.values(dy, c.T)
    want = np.full((c.n_rows, c.H), 9.0)
    want[c.pads()] = 0
    want[c.map[live]] = (g[f // c.K] * c.w.reshape(-1, 1).astype(np.float64))[live]
    got = c.values(drows, c.n_rows)
    assert (np.abs(got - want) <= (c.u + 2.0 ** -23) * np.abs(want)).all()
    rv = np.nan_to_num(c.values(rows, c.n_rows))
    prod = (rv[np.maximum(c.map, 0)] if c.T else np.zeros((0, c.H))) * g[f // c.K]
    prod[~live] = 0
    err = np.abs(dw.double().cpu().numpy()[:-1] - prod.sum(1))
    assert (err <= (c.H + 1) * 2.0 ** -24 * np.abs(prod).sum(1)).all()
    assert float(dw[-1]) == 9.0
    # each output alone gives the same bits
    d2, w2 = c.array(c.n_rows, fill=9.0), torch.full_like(dw, 9.0)
    assert B.mok_combine_backward(c.cfg, dy, None, m, starts, kept, c.dev(c.w), d2,
                                  None) == B.MOK_OK
    assert B.mok_combine_backward(c.cfg, dy, rows, m, None, None, c.dev(c.w), None,
                                  w2) == B.MOK_OK
    assert torch.equal(d2[:c.n_rows, :c.H], drows[:c.n_rows, :c.H]) and torch.equal(w2, dw)
    assert clean_status() == B.MOK_OK


def test_gradients_against_differences():
    """L = <y, dy> is linear in the rows and in the weights, so central differences of the
    forward are its gradients up to the forward's rounding."""
    torch = _t()
    c = Case(T=40, K=3, E=6, H=96, dtype="fp32", capacity=15, seed=4)
    m, starts, kept = c.dev(c.map), c.dev(c.starts), c.dev(c.kept)
    rows, dy = c.array(c.n_rows), c.array(c.T)
    drows, dw = c.array(c.n_rows, fill=0.0), torch.zeros(c.T * c.K, device="cuda")
    B.check(B.mok_combine_backward(c.cfg, dy, rows, m, starts, kept, c.dev(c.w), drows, dw))

    def loss(rows_, w_):
        y = c.array(c.T, fill=0.0)
        B.check(B.mok_combine(c.cfg, rows_, m, c.dev(w_), None, y))
        return float((c.values(y, c.T) * c.values(dy, c.T)).sum())

    dirw = c.r.standard_normal(c.w.shape).astype(np.float32)
    num = (loss(rows, c.w + dirw) - loss(rows, c.w - dirw)) / 2
    ana = float((dw.double().cpu().numpy() * dirw.reshape(-1).astype(np.float64)).sum())
    scale = 40 * 96 * 3 * 2.0 ** -20  # terms of order one, each within a few fp32 ulps
    assert abs(num - ana) <= scale
    dirr = c.array(c.n_rows)
    num = (loss(rows + dirr, c.w) - loss(rows - dirr, c.w)) / 2
    ana = float((c.values(drows, c.n_rows) * c.values(dirr, c.n_rows)).sum())
    assert abs(num - ana) <= scale


def test_side_stream_and_repeat():
    torch = _t()
    c = Case(T=500, K=4, E=16, H=1032, seed=2)
    m, starts, kept = c.dev(c.map), c.dev(c.starts), c.dev(c.kept)
    x, rows, w = c.array(c.T), c.array(c.n_rows), c.dev(c.w)
    outs = []
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        xs, y, drows = (c.array(c.n_rows, fill=1.0), c.array(c.T, fill=1.0),
                        c.array(c.n_rows, fill=1.0))
        dw = torch.zeros(c.T * c.K, device="cuda")
        torch.cuda.synchronize()
        B.check(B.mok_dispatch(c.cfg, x, m, starts, kept, xs, s))
        B.check(B.mok_combine(c.cfg, rows, m, w, x, y, s))
        B.check(B.mok_combine_backward(c.cfg, x, rows, m, starts, kept, w, drows, dw, s))
        s.synchronize()
        outs.append([t[..., :c.H] if t.dim() == 2 else t for t in (xs, y, drows, dw)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H,extra", [(64, 0), (61, 0), (61, 1), (520, 0), (523, 3)])
def test_dispatch_copies_every_bit_pattern(H, extra):
    """bf16 patterns of every kind, NaN payloads among them, arrive unchanged."""
    torch = _t()
    c = Case(T=64, K=2, E=5, H=H, ld_extra=extra)
    bits = torch.from_numpy(c.r.integers(-(1 << 15), 1 << 15, (64, c.ld)).astype(np.int16)).cuda()
    bits[:, 0] = 0x7F81  # a signalling NaN
    xs = torch.zeros(c.n_rows, c.ld, dtype=torch.int16, device="cuda")
    B.check(B.mok_dispatch(c.cfg, bits, c.dev(c.map), None, None, xs))
    f = torch.arange(c.T * c.K, device="cuda")
    got = xs[torch.from_numpy(c.map).cuda().long(), :H]
    assert torch.equal(got, bits[f // c.K, :H])


def test_map_entries_out_of_range_are_reported_and_skipped():
    torch = _t()
    c = Case(T=20, K=2, E=4, H=64)
    bad = c.map.copy()
    bad[5] = c.n_rows          # one past the end
    bad[7] = 0x7FFFFFFF
    x, xs = c.array(c.T), c.array(c.n_rows, fill=1.0)
    B.mok_clear_device_status()
    B.check(B.mok_dispatch(c.cfg, x, c.dev(bad), None, None, xs))
    assert clean_status() == B.MOK_ERR_DEVICE_INVARIANT
    want = np.full((c.n_rows, c.H), 1.0)
    ok = (bad >= 0) & (bad < c.n_rows)
    want[bad[ok]] = c.values(x, c.T)[np.arange(40)[ok] // 2]
    assert np.array_equal(c.values(xs, c.n_rows), want)
    # an expert id out of range, and too few rows
    idx = c.idx.copy()
    idx[3, 1] = 4
    i32 = dict(dtype=torch.int32, device="cuda")
    m, starts, kept = torch.zeros(40, **i32), torch.zeros(5, **i32), torch.zeros(4, **i32)
    B.check(B.mok_build_row_map(c.cfg, c.dev(idx), c.sched(), m, starts, kept))
    assert clean_status() == B.MOK_ERR_DEVICE_INVARIANT and int(m[7]) == -1
    few = B.make_rows(20, 2, 4, 64, n_rows=17)
    B.check(B.mok_build_row_map(few, c.dev(c.idx), c.sched(), m, starts, kept))
    assert clean_status() == B.MOK_ERR_DEVICE_INVARIANT
    assert int(m.max()) < 17


def test_refusals():
    c = Case(T=20, K=2, E=4, H=64)
    x, m = c.array(c.T), c.dev(c.map)
    st, kp = c.dev(c.starts), c.dev(c.kept)
    xs, w = c.array(c.n_rows), c.dev(c.w)
    bad = B.MOK_ERR_INVALID_ARG
    assert B.mok_dispatch(c.cfg, None, m, st, kp, xs) == bad
    assert B.mok_dispatch(c.cfg, x, m, st, None, xs) == bad
    assert B.mok_dispatch(c.cfg, x, m, st, kp, None) == bad
    assert B.mok_dispatch(c.cfg, x.data_ptr() + 2, m, st, kp, xs) == bad
    assert B.mok_combine(c.cfg, xs, None, w, None, x) == bad
    assert B.mok_combine(c.cfg, xs, m, w, x.data_ptr() + 8, x) == bad
    assert B.mok_combine_backward(c.cfg, x, xs, m, st, kp, w, None, None) == bad
    assert B.mok_combine_backward(c.cfg, x, None, m, st, kp, w, xs, w) == bad
    assert B.mok_build_row_map(c.cfg, c.dev(c.idx), B.make_schedule(None, st, m, m, None, None),
                               m, st, kp) == bad
    wrong = B.make_rows(20, 2, 4, 64, abi_version=1)
    assert B.mok_dispatch(wrong, x, m, st, kp, xs) == B.MOK_ERR_ABI
