"""Host-side validation of the router, the norm and the vocabulary loss (no GPU)."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

BAD, OK, ABI = B.MOK_ERR_INVALID_ARG, B.MOK_OK, B.MOK_ERR_ABI
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(T=0), OK), (dict(E=1, K=1), OK), (dict(E=1024, K=32), OK),
    (dict(groups=8, topk_groups=4, group_top=2), OK), (dict(groups=32, topk_groups=32), OK),
    (dict(E=1020, groups=17, topk_groups=1, K=32), OK), (dict(ld=70), OK), (dict(ld=1 << 30), OK),
    (dict(score=B.MOK_SCORE_SIGMOID, dtype=B.MOK_DTYPE_BF16, renormalize=False, scale=2.5), OK),
    (dict(T=-1), BAD), (dict(E=0), BAD), (dict(E=1025), BAD), (dict(K=0), BAD), (dict(K=33), BAD),
    (dict(E=8, K=9), BAD), (dict(groups=8, topk_groups=1, K=9), BAD), (dict(groups=0), BAD),
    (dict(groups=3), BAD), (dict(E=66, groups=33, topk_groups=33), BAD),
    (dict(groups=8, topk_groups=9), BAD), (dict(groups=8, topk_groups=0), BAD),
    (dict(group_top=0), BAD), (dict(group_top=3), BAD), (dict(score=2), BAD), (dict(score=-1), BAD),
    (dict(dtype=2), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=INF), BAD),
    (dict(scale=NAN), BAD), (dict(renormalize=2), BAD), (dict(ld=63), BAD),
    (dict(ld=(1 << 30) + 1), BAD), (dict(T=1 << 30, K=4), BAD), (dict(abi_version=1), ABI),
])
def test_router_config(kw, want):
    c = B.make_router(**dict(dict(T=20, E=64, K=4), **kw))
    assert B.mok_check_router_config(c) == want
    assert (B.mok_router_workspace_size(c) > 0) == (want == OK)
    c.reserved = 1
    assert B.mok_check_router_config(c) != OK


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(H=1), OK), (dict(H=1 << 20), OK), (dict(eps=1e-30), OK),
    (dict(kind=B.MOK_NORM_RMS, x_dtype=B.MOK_DTYPE_F32, y_dtype=B.MOK_DTYPE_BF16), OK),
    (dict(ld_x=104, ld_y=112), OK), (dict(rows=(1 << 31) - 513, H=8), OK),
    (dict(rows=-1), BAD), (dict(rows=(1 << 31) - 512), BAD), (dict(H=0), BAD),
    (dict(H=(1 << 20) + 1), BAD), (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=INF), BAD),
    (dict(eps=NAN), BAD), (dict(kind=2), BAD), (dict(kind=-1), BAD), (dict(x_dtype=2), BAD),
    (dict(y_dtype=-1), BAD), (dict(ld_x=96), BAD), (dict(ld_x=101), BAD), (dict(ld_y=108), BAD),
    (dict(ld_y=(1 << 30) + 8), BAD), (dict(abi_version=9), ABI),
])
def test_norm_config(kw, want):
    c = B.make_norm(**dict(dict(rows=20, H=100), **kw))
    assert B.mok_check_norm_config(c) == want
    assert (B.mok_norm_workspace_size(c) > 0) == (want == OK)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(H=1, V=1), OK), (dict(V=1 << 24, H=8), OK),
    (dict(z_loss=0.1, grad_dtype=B.MOK_DTYPE_F32), OK), (dict(piece=256), OK),
    (dict(piece=1 << 20), OK), (dict(ld_x=72, ld_w=80), OK),
    (dict(rows=-1), BAD), (dict(rows=(1 << 31) - 512), BAD), (dict(H=0), BAD),
    (dict(H=(1 << 20) + 1), BAD), (dict(V=0), BAD), (dict(V=(1 << 24) + 1), BAD),
    (dict(grad_dtype=2), BAD), (dict(z_loss=-1e-9), BAD), (dict(z_loss=INF), BAD),
    (dict(z_loss=NAN), BAD), (dict(piece=-256), BAD), (dict(piece=100), BAD), (dict(ld_x=56), BAD),
    (dict(ld_x=65), BAD), (dict(ld_w=68), BAD), (dict(abi_version=3), ABI),
    (dict(rows=1 << 26, V=1 << 20), BAD),   # more tiles than 31 bits number
])
def test_vocab_loss_config(kw, want):
    c = B.make_vocab_loss(**dict(dict(rows=100, H=64, V=1000), **kw))
    assert B.mok_check_vocab_loss_config(c) == want
    for which in (B.MOK_VOCAB_LOSS_FORWARD, B.MOK_VOCAB_LOSS_BACKWARD):
        assert (B.mok_vocab_loss_workspace_size(c, which) > 0) == (want == OK)
    assert B.mok_vocab_loss_workspace_size(c, 2) == 0


def test_vocab_loss_pieces_bound_the_workspace():
    """The gradient of a piece's logits stays within 1 GiB, in as few equal pieces as that takes; a
    piece of the caller's own is taken as it is."""
    size = lambda **kw: B.mok_vocab_loss_workspace_size(  # noqa: E731
        B.make_vocab_loss(**dict(dict(rows=8192, H=256, V=131072), **kw)), B.MOK_VOCAB_LOSS_BACKWARD)
    # dx in fp32 and the rows of x that take part, beside the piece
    whole, sums = 8192 * 131072 * 2, 8192 * 256 * (4 + 2)
    assert whole // 3 < size() - sums < (1 << 30) + (1 << 20)
    assert size(piece=1024) < 8192 * 1024 * 2 + sums + (1 << 20)
    assert size(V=32768) < (1 << 30) and size(V=32768) >= 8192 * 32768 * 2


def test_null_configs():
    L = B.lib()
    for name in ("router", "norm", "vocab_loss"):
        assert getattr(L, "mok_check_%s_config" % name)(None) == BAD
