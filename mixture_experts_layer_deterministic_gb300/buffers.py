"""Device-memory plumbing for the C ABI: torch allocates, the library computes.

`TokenSort`, `Linear` and `AdamW` do the same for the operators around the layer.

`MoELayer` owns the caller-side buffers of one configuration (schedule arrays and the
three workspaces) and strings the entry points together in the order a user calls them:
mok_route_topk -> mok_build_schedule -> mok_forward (-> mok_backward). Every method only
passes pointers; all arithmetic happens in libmok.so.
"""
import torch

from . import binding as B


def _empty(n, dtype, device):
    return torch.empty(max(int(n), 1), dtype=dtype, device=device)


class Schedule:
    """Device arrays of one schedule table (mok_schedule)."""

    def __init__(self, cfg, device):
        R = cfg.T * cfg.K
        self.cap = B.mok_segment_capacity(cfg)
        i32 = torch.int32
        self.counts = _empty(cfg.E, i32, device)
        self.offsets = _empty(cfg.E + 1, i32, device)
        self.perm = _empty(R, i32, device)
        self.inv = _empty(R, i32, device)
        self.segs = _empty(3 * self.cap, i32, device)
        self.n_segs = _empty(1, i32, device)
        self.struct = B.make_schedule(self.counts, self.offsets, self.perm, self.inv, self.segs,
                                      self.n_segs)
        self.R = R


def workspace(cfg, which, device):
    n = B.mok_workspace_size(cfg, which)
    return _empty(n, torch.uint8, device), n


def workspace_item(ws, cfg, which, item):
    """The bytes of one intermediate inside workspace tensor `ws` (a uint8 view, see
    mok_workspace_item); callers view it with the item's dtype and shape."""
    st, off, n = B.mok_workspace_item(cfg, which, item)
    B.check(st, "workspace item")
    return ws[off: off + n]


def stored_dtype(cfg):
    """torch dtype of the values the layer only stores (outputs, slots, saved A)."""
    return torch.float32 if cfg.flags & B.MOK_FLAG_FP32_STORAGE else torch.bfloat16


class MoELayer:
    """One layer configuration with its buffers on `device` (a CUDA device)."""

    def __init__(self, T, H, I, E, K, minibatch=2368, ring_capacity=0, prec=B.MOK_BF16,
                 device="cuda", backward=False, flags=0):
        self.cfg = B.make_config(T, H, I, E, K, minibatch, ring_capacity, prec, flags=flags)
        self.dtype = stored_dtype(self.cfg)
        B.check(B.mok_check_config(self.cfg), "config")
        self.device = torch.device(device)
        self.T, self.H, self.I, self.E, self.K = T, H, I, E, K
        self.sched = Schedule(self.cfg, self.device)
        self.ws_s, self.ws_s_n = workspace(self.cfg, B.MOK_WS_SCHEDULE, self.device)
        self.ws_f, self.ws_f_n = workspace(self.cfg, B.MOK_WS_FORWARD, self.device)
        self.idx = _empty(T * K, torch.int32, self.device)
        self.w = _empty(T * K, torch.float32, self.device)
        self.ws_b = None
        if backward:
            self.ws_b, self.ws_b_n = workspace(self.cfg, B.MOK_WS_BACKWARD, self.device)

    def route(self, logits, stream=None):
        B.check(B.mok_route_topk(self.cfg, logits, self.idx, self.w, stream), "route")
        return self.idx, self.w

    def schedule(self, idx=None, stream=None):
        B.check(B.mok_build_schedule(self.cfg, self.idx if idx is None else idx,
                                     self.sched.struct, self.ws_s, self.ws_s_n, stream),
                "schedule")
        return self.sched

    def forward(self, x, w13, w2, y, w13_scale=None, w2_scale=None, saved_preact=None,
                topk_w=None, stream=None):
        B.check(B.mok_forward(self.cfg, x, self.sched.struct, self.w if topk_w is None else
                              topk_w, w13, w13_scale, w2, w2_scale, y, saved_preact, self.ws_f,
                              self.ws_f_n, stream), "forward")
        return y

    def backward(self, x, saved_preact, w13, w2, dy, dx, dw13, dw2, d_topk_w, d_logits=None,
                 topk_w=None, stream=None):
        if saved_preact is None:  # recompute the pre-activations: larger workspace
            if getattr(self, "ws_r", None) is None:
                self.ws_r, self.ws_r_n = workspace(self.cfg, B.MOK_WS_BACKWARD_RECOMPUTE,
                                                   self.device)
            ws, ws_n = self.ws_r, self.ws_r_n
        else:
            if self.ws_b is None:
                self.ws_b, self.ws_b_n = workspace(self.cfg, B.MOK_WS_BACKWARD, self.device)
            ws, ws_n = self.ws_b, self.ws_b_n
        B.check(B.mok_backward(self.cfg, x, self.sched.struct, self.w if topk_w is None else
                               topk_w, saved_preact, w13, w2, dy, dx, dw13, dw2, d_topk_w,
                               d_logits, ws, ws_n, stream), "backward")
        return dx


def backward_mxfp8(layer, x, saved_preact, w13t, w2t, dy, dx, dw13, dw2, d_topk_w,
                   d_logits=None, topk_w=None, stream=None):
    """MXFP8 backward of a layer built with prec=MOK_MXFP8 (backward=True); w13t, w2t are
    (q, scale) pairs from quantize_mxfp8_transposed of the bf16 W13 and W2."""
    if layer.ws_b is None:
        layer.ws_b, layer.ws_b_n = workspace(layer.cfg, B.MOK_WS_BACKWARD, layer.device)
    B.check(B.mok_backward_mxfp8(layer.cfg, x, layer.sched.struct,
                                 layer.w if topk_w is None else topk_w, saved_preact, w13t[0],
                                 w13t[1], w2t[0], w2t[1], dy, dx, dw13, dw2, d_topk_w, d_logits,
                                 layer.ws_b, layer.ws_b_n, stream), "backward mxfp8")
    return dx


class SharedExpert:
    """The shared expert of a layer configuration (same H, I as the routed experts)."""

    def __init__(self, layer):
        self.cfg = layer.cfg
        self.ws, self.ws_n = workspace(self.cfg, B.MOK_WS_SHARED, layer.device)

    def forward(self, x, w13_s, w2_s, y, saved_preact=None, stream=None):
        """y += the shared expert's output for every token (after the routed forward).
        MXFP8 layers take w13_s, w2_s as (q, scale) pairs from quantize_mxfp8."""
        if self.cfg.prec == B.MOK_MXFP8:
            B.check(B.mok_shared_expert_forward_mxfp8(self.cfg, x, w13_s[0], w13_s[1],
                                                      w2_s[0], w2_s[1], y, saved_preact,
                                                      self.ws, self.ws_n, stream),
                    "shared forward mxfp8")
            return y
        B.check(B.mok_shared_expert_forward(self.cfg, x, w13_s, w2_s, y, saved_preact,
                                            self.ws, self.ws_n, stream), "shared forward")
        return y

    def backward(self, x, w13_s, w2_s, saved_preact, dy, dx, dw13_s, dw2_s, stream=None):
        """dx += the shared expert's input gradient; dw13_s, dw2_s = its weight gradients.
        MXFP8 layers take w13_s, w2_s as (q, scale) pairs from quantize_mxfp8_transposed
        (of W13s[None] and W2s[None])."""
        if getattr(self, "ws_b", None) is None:
            self.ws_b, self.ws_b_n = workspace(self.cfg, B.MOK_WS_SHARED_BACKWARD,
                                               x.device)
        if self.cfg.prec == B.MOK_MXFP8:
            B.check(B.mok_shared_expert_backward_mxfp8(self.cfg, x, w13_s[0], w13_s[1],
                                                       w2_s[0], w2_s[1], saved_preact, dy, dx,
                                                       dw13_s, dw2_s, self.ws_b, self.ws_b_n,
                                                       stream), "shared backward mxfp8")
            return dx
        B.check(B.mok_shared_expert_backward(self.cfg, x, w13_s, w2_s, saved_preact, dy, dx,
                                             dw13_s, dw2_s, self.ws_b, self.ws_b_n, stream),
                "shared backward")
        return dx


def quantize_mxfp8_transposed(src, stream=None):
    """MXFP8 of a [batch][rows][cols] bf16 tensor along rows, stored as [batch][cols][rows]
    (q) and [batch][cols][rows/32] (scale): the MXFP8 backward's pre-quantized weights."""
    b, r, c = src.shape
    q = torch.empty((b, c, r), dtype=torch.uint8, device=src.device)
    s = torch.empty((b, c, r // 32), dtype=torch.uint8, device=src.device)
    B.check(B.mok_quantize_mxfp8_transposed(src, b, r, c, q, s, stream), "quantize_transposed")
    return q, s


def quantize_mxfp8(src, stream=None):
    """MXFP8 along the last axis of a bf16 tensor: (q uint8, scale uint8)."""
    cols = src.shape[-1]
    rows = src.numel() // cols
    q = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    s = torch.empty(src.shape[:-1] + (cols // 32,), dtype=torch.uint8, device=src.device)
    B.check(B.mok_quantize_mxfp8(src, rows, cols, q, s, stream), "quantize")
    return q, s


# ------------------------------------------------- operators around the layer (mok_ops.h)

def _mok_dtype(dtype):
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp32 or bf16, not %s" % dtype)
    return B.MOK_DTYPE_F32 if dtype == torch.float32 else B.MOK_DTYPE_BF16


def _here(device):
    """`device` with its index, as tensors on it name it."""
    return torch.empty(0, device=device).device


def _check_matrix(name, t, dtype, device, rows, cols, ld):
    """`rows` rows of `cols` elements, `ld` apart (more of either does not matter); None passes."""
    if t is None:
        return
    shape = t.shape
    if t.dtype is dtype and t.device == device and len(shape) == 2 and shape[0] >= rows and \
            shape[1] >= cols:
        step = t.stride()
        if (step[1] == 1 or cols == 1) and (step[0] == ld or rows <= 1):
            return
    raise ValueError("%s: %s [%d][%d] with %d elements between rows on %s, not %s %s with strides "
                     "%s on %s" % (name, dtype, rows, cols, ld, device, t.dtype, list(shape),
                                   list(t.stride()), t.device))


def _check_vector(name, t, dtype, device, n):
    """`n` packed elements of any shape; None passes."""
    if t is None or (t.dtype is dtype and t.device == device and t.numel() == n and
                     t.is_contiguous()):
        return
    raise ValueError("%s: %d packed elements of %s on %s, not %s %s with strides %s on %s" %
                     (name, n, dtype, device, t.dtype, list(t.shape), list(t.stride()), t.device))


def _torch_stream(stream):
    """The torch stream that an entry point's `stream` argument names."""
    if stream is None:
        return torch.cuda.current_stream()
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream)


class TokenSort:
    """Tokens sorted by expert and back: the row map of a schedule and the four passes over it.
    Sorted arrays come from `rows()`: expert e owns rows starts[e] .. starts[e] + kept[e],
    padded with zero rows to a multiple of 16. Tokens and rows are bf16 or fp32 (`dtype`) in rows
    that start on 16-byte boundaries, ids int32, weights fp32. Arrays that do not fit raise
    ValueError before anything is launched."""

    def __init__(self, T, K, E, H, dtype=torch.bfloat16, capacity=0, device="cuda"):
        kind = _mok_dtype(dtype)
        per = 4 if dtype == torch.float32 else 8
        self.T, self.K, self.E, self.H, self.dtype = T, K, E, H, dtype
        self.ld = (H + per - 1) // per * per
        self.device = torch.device(device)
        self.cfg = B.make_rows(T, K, E, H, capacity=capacity, ld_tok=self.ld, ld_row=self.ld,
                               dtype=kind)
        B.check(B.mok_check_rows_config(self.cfg), "rows config")
        self.n_rows = int(self.cfg.n_rows)
        self.map = _empty(T * K, torch.int32, self.device)
        self.starts = _empty(E + 1, torch.int32, self.device)
        self.kept = _empty(E, torch.int32, self.device)
        self.here = self.map.device

    def rows(self, width=None):
        """A zeroed sorted array [n_rows][width] whose rows start on 16-byte boundaries."""
        w = self.H if width is None else width
        per = 4 if self.dtype == torch.float32 else 8
        return torch.zeros(self.n_rows, (w + per - 1) // per * per, dtype=self.dtype,
                           device=self.device)[:, :w]

    def _check(self, name, t, n):
        _check_matrix(name, t, self.dtype, self.here, n, self.H, self.ld)

    def _check_ids(self, name, t, dtype):
        """One value per routed id (the helpers' own arrays have one where there are no ids)."""
        n = self.T * self.K
        _check_vector(name, t, dtype, self.here, n if n or t is None else t.numel())

    def build(self, idx, sched, stream=None):
        """The row map of `sched` (a Schedule built from idx [T][K])."""
        self._check_ids("idx", idx, torch.int32)
        if sched.R != self.T * self.K or sched.counts.numel() != self.E:
            raise ValueError("the schedule has %d ids of %d experts, the sort %d of %d" %
                             (sched.R, sched.counts.numel(), self.T * self.K, self.E))
        B.check(B.mok_build_row_map(self.cfg, idx, sched.struct, self.map, self.starts, self.kept,
                                    stream), "row map")

    def dispatch(self, x, xs, stream=None):
        self._check("x", x, self.T)
        self._check("xs", xs, self.n_rows)
        B.check(B.mok_dispatch(self.cfg, x, self.map, self.starts, self.kept, xs, stream),
                "dispatch")
        return xs

    def dispatch_backward(self, dxs, dx, stream=None):
        self._check("dx", dx, self.T)
        self._check("dxs", dxs, self.n_rows)
        B.check(B.mok_dispatch_backward(self.cfg, dxs, self.map, dx, stream), "dispatch backward")
        return dx

    def combine(self, rows, topk_w, y, residual=None, stream=None):
        self._check("y", y, self.T)
        self._check("residual", residual, self.T)
        self._check("rows", rows, self.n_rows)
        self._check_ids("topk_w", topk_w, torch.float32)
        B.check(B.mok_combine(self.cfg, rows, self.map, topk_w, residual, y, stream), "combine")
        return y

    def combine_backward(self, dy, rows, topk_w, drows, d_topk_w, stream=None):
        self._check("dy", dy, self.T)
        self._check("rows", rows, self.n_rows)
        self._check("drows", drows, self.n_rows)
        self._check_ids("topk_w", topk_w, torch.float32)
        self._check_ids("d_topk_w", d_topk_w, torch.float32)
        B.check(B.mok_combine_backward(self.cfg, dy, rows, self.map, self.starts, self.kept,
                                       topk_w, drows, d_topk_w, stream), "combine backward")
        return drows


class Linear:
    """A linear layer and its workspaces: one matrix, or with groups > 1 one per group of sorted
    rows (forward and backward then take the TokenSort that sorted them). Weights are
    [groups][out][in] bf16; rows of x, y, z, dy, dx and of the weights start on 16-byte
    boundaries, which packed rows do where their width is a multiple of 8 (`weights()` makes an
    array for any width). Calls of one Linear share its workspaces, so calls on several streams
    have to be ordered by the caller. y and dy have out_dtype, dx and dw grad_dtype, bias and db are fp32,
    everything else is bf16. Arrays that do not fit raise ValueError before anything is
    launched."""

    def __init__(self, rows, in_features, out_features, groups=1, act=B.MOK_ACT_NONE,
                 out_dtype=torch.bfloat16, grad_dtype=torch.bfloat16, device="cuda"):
        self.cfg = B.make_linear(rows, in_features, out_features, groups, act,
                                 _mok_dtype(out_dtype), _mok_dtype(grad_dtype))
        B.check(B.mok_check_linear_config(self.cfg), "linear config")
        self.out_dtype, self.grad_dtype = out_dtype, grad_dtype
        self.device = torch.device(device)
        self.here = _here(self.device)
        self.ws = [None, None]
        self.groups = groups
        self.wide = (rows, in_features, int(self.cfg.ld_in))    # x, dx
        self.out = (rows, out_features, int(self.cfg.ld_out))   # y, dy, z, residual
        self.of_w = (out_features, in_features, int(self.cfg.ld_w))

    def weights(self, dtype=torch.bfloat16):
        """Zeros [groups][out][in] whose rows lie as the layer reads them: a view of a packed
        [groups][out][ld_w] array."""
        c = self.cfg
        return torch.zeros(c.groups, c.out_features, c.ld_w, dtype=dtype,
                           device=self.device)[..., :c.in_features]

    def _ws(self, which, stream):
        """The workspace of a pass, its size and the stream's handle. It comes from the memory of the stream that first
        runs the pass, whose earlier work is then done with it; other streams are recorded, so it
        is not given away under their work."""
        handle = B._stream(stream) if self.here.type == "cuda" else 0
        if self.ws[which] is None:
            n = B.mok_linear_workspace_size(self.cfg, which)
            with torch.cuda.stream(None if stream is None else _torch_stream(stream)):
                self.ws[which] = (_empty(n, torch.uint8, self.here), n, handle)
        ws, n, first = self.ws[which]
        if handle != first:
            ws.record_stream(_torch_stream(stream))
        return ws, n, handle

    def _check_weights(self, name, t, dtype):
        """[groups][out][in], or [groups * out][in]."""
        if t is None:
            return
        n, k, ld = self.of_w
        shape = t.shape
        if len(shape) == 3 and shape[0] == self.groups and shape[1] == n and \
                (self.groups == 1 or t.stride(0) == n * ld) and (n == 1 or t.stride(1) == ld) and \
                (k == 1 or t.stride(2) == 1) and shape[2] >= k and t.dtype is dtype and \
                t.device == self.here:
            return
        if len(shape) == 3:
            raise ValueError("%s: %s [%d][%d][%d] with %d elements between rows on %s, not %s %s "
                             "with strides %s on %s" % (name, dtype, self.groups, n, k, ld,
                                                        self.here, t.dtype, list(shape),
                                                        list(t.stride()), t.device))
        _check_matrix(name, t, dtype, self.here, self.groups * n, k, ld)

    def _check_sort(self, sort):
        if sort is None and self.groups > 1:
            raise ValueError("%d groups of rows need the TokenSort that made them" % self.groups)
        if sort is not None and sort.E != self.groups:
            raise ValueError("the sort has %d groups, the layer %d" % (sort.E, self.groups))

    def forward(self, x, w, y, bias=None, residual=None, z=None, sort=None, stream=None):
        bf, here = torch.bfloat16, self.here
        _check_matrix("x", x, bf, here, *self.wide)
        _check_matrix("y", y, self.out_dtype, here, *self.out)
        _check_matrix("residual", residual, bf, here, *self.out)
        _check_matrix("z", z, bf, here, *self.out)
        self._check_weights("w", w, bf)
        _check_vector("bias", bias, torch.float32, here, self.groups * self.of_w[0])
        self._check_sort(sort)
        ws, n, handle = self._ws(B.MOK_LINEAR_FORWARD, stream)
        B.check(B.mok_linear_forward(self.cfg, x, w, bias, residual, sort and sort.starts,
                                     sort and sort.kept, y, z, ws, n, handle), "linear forward")
        return y

    def backward(self, x, w, dy, z=None, dx=None, dw=None, db=None, sort=None, stream=None):
        bf, here = torch.bfloat16, self.here
        _check_matrix("x", x, bf, here, *self.wide)
        _check_matrix("dy", dy, self.out_dtype, here, *self.out)
        _check_matrix("z", z, bf, here, *self.out)
        _check_matrix("dx", dx, self.grad_dtype, here, *self.wide)
        self._check_weights("w", w, bf)
        self._check_weights("dw", dw, self.grad_dtype)
        _check_vector("db", db, torch.float32, here, self.groups * self.of_w[0])
        self._check_sort(sort)
        ws, n, handle = self._ws(B.MOK_LINEAR_BACKWARD, stream)
        B.check(B.mok_linear_backward(self.cfg, x, w, z, dy, sort and sort.starts,
                                      sort and sort.kept, dx, dw, db, ws, n, handle),
                "linear backward")
        return dx


class AdamW:
    """AdamW over a list of parameters: dicts with p (fp32 or bf16), g (its gradient, fp32 or
    bf16) and, where they apply, copy (bf16 working weights of an fp32 p) and weight_decay. All
    are packed and stay where they are: a step reads the gradients at the addresses they had when
    the list was given. The states are fp32, or MXFP8 with eight_bit. Parameters that share their
    types go in one launch. Arrays that do not fit raise ValueError.

    A step takes its number t, lr and seed from this object, so a CUDA graph that captured one
    would replay that step. With `capturable` they are on the device and move with each replay
    (one more launch a step): set_lr changes lr, and t does not count replays."""

    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, eight_bit=False,
                 stochastic=True, seed=0, device="cuda", capturable=False):
        self.lr, self.betas, self.eps, self.seed, self.t = lr, betas, eps, seed, 0
        self.state = B.MOK_STATE_MXFP8 if eight_bit else B.MOK_STATE_F32
        self.flags = B.MOK_ADAMW_STOCHASTIC if stochastic else 0
        device, groups = _here(device), {}
        for q in params:
            e, p = dict(q), q["p"]
            n, kinds = p.numel(), (_mok_dtype(p.dtype), _mok_dtype(q["g"].dtype))
            for k in ("p", "g"):
                _check_vector(k, q[k], q[k].dtype, device, n)
            _check_vector("copy", q.get("copy"), torch.bfloat16, device, n)
            if q.get("copy") is not None and p.dtype != torch.float32:
                raise ValueError("copy: only fp32 parameters have one")
            u8 = dict(dtype=torch.uint8, device=p.device)
            for k in ("m", "v"):
                e[k] = torch.zeros(n, **(u8 if eight_bit else
                                         dict(dtype=torch.float32, device=p.device)))
                if eight_bit:
                    e[k + "_scale"] = torch.zeros((n + 31) // 32, **u8)
            groups.setdefault(kinds, []).append(dict(e, n=n))
        self.lists = [(kinds, B.make_adamw_list(g)) for kinds, g in groups.items()]
        self.device, self.clock = device, None
        if capturable:
            self.clock = torch.zeros(B.ADAMW_CLOCK_WORDS, dtype=torch.int64, device=device)
            self.clock[1] = len(self.lists)
            self.set_lr(lr)

    def set_lr(self, lr):
        """The learning rate from the next step on."""
        self.lr = lr
        if self.clock is not None:
            self.clock.view(torch.float64)[2] = lr

    def step(self, grad_scale=None, stream=None):
        if grad_scale is not None:
            _check_vector("grad_scale", grad_scale, torch.float32, self.device, 1)
        self.t += 1
        if self.clock is not None:
            return self._step_at(grad_scale, stream)
        for k, ((p, g), tensors) in enumerate(self.lists):
            cfg = B.make_adamw(self.lr, *self.betas, self.eps, self.t,
                               (self.seed + self.t * len(self.lists) + k) & (2 ** 64 - 1), p, g,
                               self.state, self.flags)
            B.check(B.mok_adamw_step(cfg, tensors, grad_scale, stream), "adamw")

    def _step_at(self, grad_scale, stream):
        for k, ((p, g), tensors) in enumerate(self.lists):
            cfg = B.make_adamw(self.lr, *self.betas, self.eps, 1,
                               (self.seed + k) & (2 ** 64 - 1), p, g, self.state, self.flags)
            if k == 0:
                B.check(B.mok_adamw_advance(cfg, self.clock, stream), "adamw clock")
            B.check(B.mok_adamw_step_at(cfg, tensors, self.clock, grad_scale, stream), "adamw")
