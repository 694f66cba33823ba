"""The operators around the layer at the edges of their definitions: layouts that break the rules,
schedules that do not fit, non-finite values, long sums kept in fp32.

Tolerances are those of test_gpu_linear.py and test_gpu_rows.py, and for fp32 gradients: dz enters
a product as two bf16 values, each rounded to nearest, so within 2^-17 of itself; a sum in
segments of 1024 terms is within 2^-19 of its norm (twice the 8.9e-7 that 4096 terms of one sign
pattern after another gave in four segments; one run of 4096 terms gave 3.9e-6, and the error of
a run grows with its length)."""
import numpy as np
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B
from test_gpu_adamw import Tensors, config
from test_gpu_linear import Lin, act64, check_backward, check_forward, device_ok, dot_rel
from test_gpu_rows import Case, clean_status

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def i32(a):
    return _t().tensor(a, dtype=_t().int32, device="cuda")


def norm_rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def test_a_group_that_overlaps_an_earlier_one_counts_as_empty():
    """starts that fall: the third group's rows are the first one's. It is reported and takes no
    part, so no row has two writers."""
    torch = _t()
    c = Lin(G=3, counts=[20, 0, 20], Kin=64, N=40)
    clean = check_forward(c)[0]
    c.d_starts, c.d_counts = i32([0, 32, 0, 32]), i32([20, 5, 20])
    y, _ = c.forward()
    assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
    B.mok_clear_device_status()
    assert torch.equal(y[:32, :40], clean[:32, :40])
    assert bool((y[32:] == 7).all())
    _, dw, db = c.backward()
    assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
    B.mok_clear_device_status()
    assert bool((dw[:40, :64] != 0).any())
    assert bool((dw[40:, :64] == 0).all()) and bool((db[40:120] == 0).all())


def test_falling_starts_over_more_than_2_to_the_30_rows():
    """Every other group asks for all of 2^30 rows and more: the first has them, the others count
    as empty, and no tile is counted twice. Arrays of more than 2^31 elements."""
    torch = _t()
    rows, G = (1 << 30) + 4096, 1024
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    cfg = B.make_linear(rows, 8, 8, G)
    assert B.mok_check_linear_config(cfg) == B.MOK_OK
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(rows, 8, **bf), torch.full((rows, 8), 7.0, **bf)
    w = torch.randn(G, 8, 8, device="cuda").to(torch.bfloat16)
    live = [slice(0, 300), slice((1 << 30) - 150, (1 << 30) + 150), slice(rows - 300, rows)]
    for s in live:
        x[s] = torch.randn(300, 8, device="cuda").to(torch.bfloat16)
    starts, counts = i32([0, rows] * (G // 2) + [0]), i32([rows, 0] * (G // 2))
    n = B.mok_linear_workspace_size(cfg, B.MOK_LINEAR_FORWARD)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.mok_linear_forward(cfg, x, w, None, None, starts, counts, y, None, ws, n))
    assert B.mok_read_device_status()[1] == B.MOK_ERR_DEVICE_INVARIANT
    B.mok_clear_device_status()
    for s in live:
        ref = x[s].double() @ w[0].double().T
        mag = x[s].double().abs() @ w[0].double().abs().T
        assert bool(((y[s].double() - ref).abs() <= dot_rel(8) * mag + 2.0 ** -8 * ref.abs()).all())
        y[s] = 0
    assert int(torch.count_nonzero(y)) == 0


def test_a_group_whose_sum_takes_seconds():
    """dW of a group of 2^30 rows: one sum of some seconds, longer than a wait for anything else
    may take."""
    torch = _t()
    rows = 1 << 30
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    cfg = B.make_linear(rows, 8, 8, 1, grad_dtype=B.MOK_DTYPE_BF16)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, dy, dw = torch.zeros(rows, 8, **bf), torch.zeros(rows, 8, **bf), torch.zeros(8, 8, **bf)
    live = [slice(0, 300), slice(rows // 2, rows // 2 + 300), slice(rows - 300, rows)]
    for s in live:
        x[s], dy[s] = torch.randn(300, 8, device="cuda"), torch.randn(300, 8, device="cuda")
    n = B.mok_linear_workspace_size(cfg, B.MOK_LINEAR_BACKWARD)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.mok_linear_backward(cfg, x, None, None, dy, i32([0, rows]), i32([rows]), None, dw,
                                  None, ws, n))
    assert device_ok()
    xs, ds = (torch.cat([t[s] for s in live]).double() for t in (x, dy))
    e = dot_rel(900) * (ds.abs().T @ xs.abs())
    assert bool(((dw.double() - ds.T @ xs).abs() <= e + 2.0 ** -8 * ((ds.T @ xs).abs() + e)).all())


def test_linear_helper_with_an_odd_width():
    """1001 inputs: weights and their gradient in rows 1008 apart, as weights() makes them."""
    torch = _t()
    from mixture_experts_layer_deterministic_gb300.buffers import Linear
    lin = Linear(70, 1001, 77, grad_dtype=torch.float32)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.randn(70, 1008, **bf)[:, :1001], torch.zeros(70, 80, **bf)[:, :77]
    w, dw, dx = lin.weights(), lin.weights(torch.float32), torch.zeros(70, 1008, device="cuda")
    w.copy_(torch.randn(77, 1001, device="cuda") / 32)
    dy = torch.randn(70, 80, **bf)[:, :77]
    lin.forward(x, w, y)
    lin.backward(x, w, dy, dx=dx, dw=dw)
    assert device_ok()
    xd, wd, dyd = x.double(), w[0].double(), dy.double()
    for got, a, b, n, u in ((y, xd, wd.T, 1001, 2.0 ** -8), (dx[:, :1001], dyd, wd, 77, 0.0),
                            (dw[0], dyd.T, xd, 70, 0.0)):
        e = dot_rel(n) * (a.abs() @ b.abs())
        assert bool(((got.double() - a @ b).abs() <= e + u * ((a @ b).abs() + e)).all())
    with pytest.raises(ValueError):
        lin.forward(x, torch.zeros(1, 77, 1001, **bf), y)


def test_workspaces_belong_to_the_stream_that_uses_them():
    """A Linear's workspace comes from the memory of the stream of the pass (other memory may still
    be in use by the current stream's earlier work), and the passes run on either kind of handle."""
    torch = _t()
    from mixture_experts_layer_deterministic_gb300.buffers import Linear
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, dy = torch.randn(300, 64, **bf), torch.randn(300, 48, **bf)
    y, dx = torch.zeros(300, 48, **bf), torch.zeros(300, 64, **bf)
    s = torch.cuda.Stream()

    def owner(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]

    for handle in (s, s.cuda_stream, None):
        lin = Linear(300, 64, 48, act=B.MOK_ACT_SILU)
        w = lin.weights()
        w.normal_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s if handle is None else None):
            lin.forward(x, w, y, stream=handle)
            lin.backward(x, w, dy, z=dy, dx=dx, stream=handle)
        s.synchronize()
        assert [owner(ws[0]) for ws in lin.ws] == [s.cuda_stream] * 2
        a, b = y.clone(), dx.clone()
        torch.cuda.synchronize()
        lin.forward(x, w, y)  # and on another stream than its own
        lin.backward(x, w, dy, z=dy, dx=dx)
        torch.cuda.synchronize()
        assert torch.equal(a, y) and torch.equal(b, dx) and device_ok()


@pytest.mark.parametrize("capacity", [0, 3])
def test_a_schedule_of_other_ids_is_reported(capacity):
    """The schedule of 12 ids of expert 0 and 4 of expert 1, used with ids the other way round:
    expert 1 then holds ranks 4 to 15, of which it counted four."""
    c = Case(T=16, K=1, E=2, H=16, capacity=capacity)
    idx = np.array([0] * 12 + [1] * 4, np.int32)
    c.counts, c.offsets = np.array([12, 4], np.int32), np.array([0, 12, 16], np.int32)
    c.perm = c.inv = np.arange(16, dtype=np.int32)
    m, starts, kept = i32([7] * 16), i32([0] * 3), i32([0] * 2)

    def build(ids):
        B.check(B.mok_build_row_map(c.cfg, c.dev(ids), c.sched(), m, starts, kept))
        return clean_status(), m.cpu().numpy()

    status, got = build(idx)
    assert status == B.MOK_OK
    keep = capacity or 16
    first1 = 16
    want = [f if f < keep else -1 for f in range(12)] + [first1 + r if r < keep else -1
                                                         for r in range(4)]
    assert got.tolist() == want
    # ids that the schedule did not see: id 12 (rank 12 of expert 0, which counted 12) is past the
    # count, with and without a capacity below it
    other = idx.copy()
    other[12] = 0
    status, got = build(other)
    assert status == B.MOK_ERR_DEVICE_INVARIANT
    want[12] = -1
    assert got.tolist() == want


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,extra", [(64, 0), (61, 3), (264, 0), (1030, 0), (4100, 1)])
def test_dropped_copies_have_zero_gradients_whatever_dy_holds(H, extra, dtype):
    torch = _t()
    c = Case(T=40, K=3, E=6, H=H, capacity=15, dtype=dtype, ld_extra=extra)
    rows, dy = c.array(c.n_rows), c.array(c.T)
    dy[:, 0] = float("inf")
    dy[:, H - 1] = float("nan")
    drows, dw = c.array(c.n_rows, fill=9.0), torch.full((c.T * c.K,), 9.0, device="cuda")
    B.check(B.mok_combine_backward(c.cfg, dy, rows, c.dev(c.map), c.dev(c.starts), c.dev(c.kept),
                                   c.dev(c.w), drows, dw))
    dropped = torch.from_numpy(c.map < 0).cuda()
    assert int(dropped.sum()) > 0
    assert bool((dw[dropped] == 0).all())
    assert bool(dw[~dropped].isnan().all())
    assert clean_status() == B.MOK_OK


def test_activations_and_slopes_far_from_zero():
    """Finite z of any size: the slopes are 0 or 1 there, and act(z) is z or 0."""
    torch = _t()
    far = torch.tensor([3.0e38, 1e30, 1e20, 1e14, 1e8, 200.0, 30.0], device="cuda")
    zs = torch.cat([far, -far]).to(torch.bfloat16)
    for act in ("relu", "silu", "gelu_tanh", "gelu"):
        for R in (1, 300):
            c = Lin(R=R, Kin=16, N=14, act=act, grad="fp32")
            c.z[:R, :14] = zs
            dx, dw, db = c.backward()
            assert device_ok()
            want = torch.where(zs > 0, c.dy[:R, :14].float(), 0.0).sum(0)
            mag = c.dy[:R, :14].float().abs().sum(0)
            # exp(-30) z is below 2^-38; the sums are fp32
            assert bool(((db[:14] - want).abs() <= (R + 8) * 2.0 ** -24 * mag + 1e-10).all()), act
            assert bool(dx[:R, :16].isfinite().all()) and bool(dw[:14, :16].isfinite().all())
        c = Lin(R=3, Kin=1, N=14, act=act, out="fp32", res=False, bias=False)
        c.x[:3, :1], c.w[:14, 0] = 1.0, zs
        y, z = c.forward()
        assert device_ok() and torch.equal(z[:3, :14], zs.expand(3, 14))
        want = zs.float().clamp(min=0)
        assert bool(((y[:3, :14] - want).abs() <= 2.0 ** -20 * want + 1e-10).all()), act


@pytest.mark.parametrize("kw", [
    dict(R=10000, Kin=2100, N=1030, res=False, z=False),
    dict(R=10000, Kin=2100, N=1030, act="silu"),
    dict(R=10000, Kin=2100, N=1030, res=True, z=False),
    dict(G=4, counts=[900, 0, 17, 300], Kin=2500, N=300, res=False, z=False, spare=16),
    dict(G=4, counts=[900, 0, 17, 300], Kin=2500, N=300, act="gelu_tanh", spare=16),
], ids=lambda k: "-".join("%s%s" % i for i in k.items()).replace(" ", ""))
def test_fp32_outputs_over_several_segments(kw):
    c = Lin(out="fp32", **kw)
    y, _ = check_forward(c)
    k = c.Kin
    for g, (a, b) in enumerate(c.spans()):
        if b == a:
            continue
        ref = c.x[a:b, :k].double() @ c.w[g * c.N:(g + 1) * c.N, :k].double().T
        if c.b is not None:
            ref = ref + c.b[g * c.N:(g + 1) * c.N].double()
        ref, _ = act64(ref, c.act)
        if c.res is not None:
            ref = ref + c.res[a:b, :c.N].double()
        assert norm_rel(y[a:b, :c.N], ref) <= 2.0 ** -19


@pytest.mark.parametrize("kw", [
    dict(R=16384, Kin=2048, N=2048),                     # no cut along K, dz = dy
    dict(R=16384, Kin=64, N=64),                         # parts of K
    dict(R=16384, Kin=64, N=64, act="gelu_tanh"),
    dict(R=3000, Kin=1200, N=2600, act="silu"),
    dict(R=3000, Kin=1200, N=2600, out="fp32"),
    dict(R=700, Kin=520, N=300, act="gelu", out="fp32", extra=8),
    dict(R=1, Kin=40, N=24, act="relu"),
    dict(R=33, Kin=15, N=17, act="silu"),
    dict(G=4, counts=[5000, 0, 17, 3001], Kin=300, N=200, spare=16),
    dict(G=4, counts=[5000, 0, 17, 3001], Kin=300, N=2100, act="gelu_tanh", out="fp32", spare=16),
    dict(G=3, counts=[0, 0, 0], Kin=64, N=64, act="silu", spare=16),
], ids=lambda k: "-".join("%s%s" % i for i in k.items()).replace(" ", ""))
def test_fp32_gradients_are_fp32(kw):
    torch = _t()
    c = Lin(grad="fp32", z=True, res=False, **kw)
    dx, dw, db = check_backward(c)
    k, N, u = c.Kin, c.N, 2.0 ** -17
    exact_dz = c.act == "none" and c.out_dt == torch.bfloat16
    for g, (a, b) in enumerate(c.spans()):
        if b == a:
            continue
        x, w = c.x[a:b, :k].double(), c.w[g * N:(g + 1) * N, :k].double()
        dz = c.dy[a:b, :N].double()
        edz = torch.zeros_like(dz)
        if c.act != "none":
            zz = c.z[a:b, :N].double()
            edz = dz.abs() * 2.0 ** -20 * (1 + zz.abs())
            dz = dz * act64(zz, c.act)[1]
        e = edz + (0.0 if exact_dz else u * (dz.abs() + edz))
        for got, ref, err, mag, n in (
                (dx[a:b, :k], dz @ w, e @ w.abs(), dz.abs() @ w.abs(), N),
                (dw[g * N:(g + 1) * N, :k], dz.T @ x, e.T @ x.abs(), dz.abs().T @ x.abs(), b - a)):
            assert bool(((got.double() - ref).abs() <= err + dot_rel(n) * (mag + err)).all())
            assert norm_rel(got, ref) <= 2.0 ** -19 + (0.0 if exact_dz else u)
    # the bits of a gradient do not depend on what else is asked for, and repeat
    for i in range(3):
        alone = c.backward(*[i == j for j in range(3)])
        assert torch.equal(alone[i].view(torch.uint8), (dx, dw, db)[i].view(torch.uint8))


@pytest.mark.parametrize("kw", [dict(R=2, Kin=200, N=130), dict(R=12, Kin=520, N=40, act="silu"),
                                dict(R=300, Kin=200, N=130, act="gelu_tanh"),
                                dict(R=100, Kin=5000, N=90, out="fp32"),
                                dict(R=10000, Kin=1100, N=1030, out="fp32"),
                                dict(G=4, counts=[900, 0, 17, 300], Kin=200, N=72, act="gelu")],
                         ids=lambda k: "-".join("%s%s" % i for i in k.items()).replace(" ", ""))
def test_non_finite_values_stay_in_their_rows_and_features(kw):
    """A NaN in a row of x reaches that row of y and dx alone, an infinity in a feature of W that
    feature alone; a sum past the range is infinite, and its neighbours keep their bits."""
    torch = _t()
    c = Lin(z=True, **kw)
    a, b = c.spans()[0]
    clean, clean_z = c.forward()
    dx0, dw0, db0 = c.backward()
    r, f, N, k = b - 1, 3, c.N, c.Kin
    x, w, dy = c.x.clone(), c.w.clone(), c.dy.clone()
    c.x[r, 1] = float("nan")
    c.w[f, 0] = float("inf")
    y, z = c.forward()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[a:b, f] = keep[r, :N] = False
    assert torch.equal(y[keep].isnan(), clean[keep].isnan())
    assert torch.equal(y[keep].nan_to_num(), clean[keep].nan_to_num())
    assert bool(y[r, :N].isnan().all()) and bool(z[r, :N].isnan().all())
    assert not bool(z[a:b, f].isfinite().any())
    # gradients: dx of the row takes the NaN of its dy, dW of the feature, db too
    c.x.copy_(x)
    c.w.copy_(w)
    c.dy[r, f] = float("nan")
    dx, dw, db = c.backward()
    keep = torch.ones_like(dx, dtype=torch.bool)
    keep[r, :k] = False
    assert torch.equal(dx[keep], dx0[keep]) and bool(dx[r, :k].isnan().all())
    keep = torch.ones_like(dw, dtype=torch.bool)
    keep[f, :k] = False
    assert torch.equal(dw[keep], dw0[keep]) and bool(dw[f, :k].isnan().all())
    assert bool(db[f].isnan()) and torch.equal(db[f + 1:], db0[f + 1:]) and device_ok()
    # a sum past the largest value of its type
    c.dy.copy_(dy)
    c.x[r, :k], c.w[f, :k] = 2.0 ** 100, 2.0 ** 60
    y, z = c.forward()
    assert bool((y[r, f] == float("inf")).all()) and bool((z[r, f] == float("inf")).all())
    assert torch.equal(z[a:r, :f], clean_z[a:r, :f]) and device_ok()


def test_sort_of_more_than_2_to_the_31_elements():
    """Rows past 2^31 elements of their array, against the plain passes on the GPU."""
    torch = _t()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    T, K, E, H = 8192, 32, 64, 8250
    c = Case(T=T, K=K, E=E, H=H)
    assert c.n_rows * c.ld > 1 << 31
    gen = torch.Generator("cuda").manual_seed(1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, xs = torch.zeros(T, c.ld, **bf), torch.full((c.n_rows, c.ld), 9.0, **bf)
    x.normal_(generator=gen)
    m, st, kp, w = c.dev(c.map), c.dev(c.starts), c.dev(c.kept), c.dev(c.w)
    B.check(B.mok_dispatch(c.cfg, x, m, st, kp, xs))
    for k in range(K):
        assert torch.equal(xs[m.view(T, K)[:, k].long(), :H], x[:, :H])
    assert bool((xs[:, H:] == 9).all())
    y = torch.zeros(T, c.ld, **bf)
    B.check(B.mok_combine(c.cfg, xs, m, w, None, y))
    ws = w.view(T, K).double()
    ref = x[:, :H].double() * ws.sum(1, keepdim=True)
    assert bool(((y[:, :H].double() - ref).abs() <=
                 (2.0 ** -8 + (K + 2) * 2.0 ** -23) * ref.abs()).all())
    drows, dw = torch.full((c.n_rows, c.ld), 9.0, **bf), torch.zeros(T * K, device="cuda")
    B.check(B.mok_combine_backward(c.cfg, x, xs, m, st, kp, w, drows, dw))
    for k in range(K):
        ref = (x[:, :H].float() * w.view(T, K)[:, k:k + 1]).to(torch.bfloat16)
        assert torch.equal(drows[m.view(T, K)[:, k].long(), :H], ref)
    sq = x[:, :H].double().square().sum(1, keepdim=True)
    assert bool(((dw.view(T, K).double() - sq).abs() <= (H + 1) * 2.0 ** -24 * sq).all())
    assert clean_status() == B.MOK_OK


def test_weights_of_more_than_2_to_the_31_elements():
    """1024 groups of 1024 x 2056: the last groups' matrices lie past 2^31 elements."""
    torch = _t()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    G, K, N = 1024, 2056, 1024
    assert G * N * K > 1 << 31
    rows, bf = 16 * G, dict(dtype=torch.bfloat16, device="cuda")
    cfg = B.make_linear(rows, K, N, G)
    gen = torch.Generator("cuda").manual_seed(1)
    x, w = torch.zeros(rows, K, **bf), torch.zeros(G, N, K, **bf)
    x.normal_(generator=gen)
    w.normal_(generator=gen)
    dy, y = torch.zeros(rows, N, **bf), torch.full((rows, N), 7.0, **bf)
    dy.normal_(generator=gen)
    starts, counts = i32(list(range(0, rows + 1, 16))), i32([16] * G)
    ws = torch.empty(max(B.mok_linear_workspace_size(cfg, i) for i in (0, 1)), dtype=torch.uint8,
                     device="cuda")
    B.check(B.mok_linear_forward(cfg, x, w, None, None, starts, counts, y, None, ws, ws.numel()))
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    B.check(B.mok_linear_backward(cfg, x, w, None, dy, starts, counts, dx, dw, None, ws,
                                  ws.numel()))
    assert device_ok()
    for g in (0, 1, 511, 1019, 1020, 1022, 1023):
        s = slice(16 * g, 16 * g + 16)
        xd, wd, dd = x[s].double(), w[g].double(), dy[s].double()
        for got, p, q, n in ((y[s], xd, wd.T, K), (dx[s], dd, wd, N), (dw[g], dd.T, xd, 16)):
            e = dot_rel(n) * (p.abs() @ q.abs())
            assert bool(((got.double() - p @ q).abs() <= e + 2.0 ** -8 * ((p @ q).abs() + e)).all())


def test_two_host_threads_on_two_streams():
    """Passes issued by two threads at once, each on a stream of its own, give the bits that each
    gives alone."""
    import threading
    torch = _t()
    jobs = [Lin(G=5, counts=[1, 0, 300, 16, 257], Kin=200, N=136, act="silu"),
            Lin(R=700, Kin=520, N=300, act="gelu_tanh", grad="fp32")]
    sorts = [Case(T=300, K=4, E=16, H=264, seed=i) for i in range(2)]
    alone, kept, failed = [], [[], []], []

    def work(i, stream):
        c, s = jobs[i], sorts[i]
        y, z = c.forward(stream=stream)
        keep = c._keep
        grads = c.backward(stream=stream)
        out = s.out
        B.check(B.mok_dispatch(s.cfg, s.x, s.m, s.st, s.kp, out[0], stream))
        B.check(B.mok_combine(s.cfg, out[0], s.m, s.dw, s.x, out[1], stream))
        return (y, z, *grads), (keep, c._keep)

    for s in sorts:
        s.x, s.m, s.st, s.kp, s.dw = (s.array(s.T), s.dev(s.map), s.dev(s.starts), s.dev(s.kept),
                                      s.dev(s.w))
        s.out = [s.array(s.n_rows, fill=1.0), s.array(s.T, fill=1.0)]
    for i in range(2):
        got, _ = work(i, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in (*got, *sorts[i].out)])
    streams = [torch.cuda.Stream() for _ in range(2)]

    def loop(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    kept[i].append(work(i, streams[i]))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and device_ok()
    for i in range(2):
        for got, _ in kept[i]:
            for a, b in zip(got, alone[i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(sorts[i].out, alone[i][5:]):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("g", ["bf16", "fp32"])
def test_first_moment_is_the_formula_in_fp32(g):
    """beta1 m + (1 - beta1) g with each operation rounded to fp32, bit for bit."""
    t = Tensors([100000], "fp32", g, "fp32", seed=6)
    d, n = t.t[0], 100000
    f = np.float32
    m0, g0 = d["m"][:n].cpu().numpy(), d["g"][:n].float().cpu().numpy() * f(0.5)
    B.check(B.mok_adamw_step(config(t), t.list(), t.gs))
    want = m0 * f(0.9) + g0 * f(1 - 0.9)
    assert np.array_equal(d["m"][:n].cpu().numpy(), want)
