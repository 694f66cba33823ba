"""Host-side validation of the operators around the layer (no GPU)."""
import pytest

from mixture_experts_layer_deterministic_gb300 import binding as B

BAD, OK = B.MOK_ERR_INVALID_ARG, B.MOK_OK


def rows(**kw):
    base = dict(T=20, K=2, E=4, H=64)
    base.update(kw)
    return B.make_rows(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(T=0), OK), (dict(H=1), OK), (dict(H=1111), OK), (dict(K=32, E=64), OK),
    (dict(K=3, E=2), OK),                       # a map may name any rows
    (dict(ld_tok=65, ld_row=70), OK), (dict(capacity=5), OK), (dict(n_rows=0), OK),
    (dict(dtype=B.MOK_DTYPE_F32), OK),
    (dict(T=-1), BAD), (dict(K=0), BAD), (dict(K=33, E=64), BAD), (dict(E=0), BAD),
    (dict(E=1025), BAD), (dict(H=0), BAD), (dict(ld_tok=63), BAD), (dict(ld_row=63), BAD),
    (dict(capacity=-1), BAD), (dict(dtype=2), BAD), (dict(n_rows=-1), BAD),
    (dict(n_rows=1 << 31), BAD), (dict(T=1 << 30, K=2, n_rows=10), BAD),
    (dict(abi_version=1), B.MOK_ERR_ABI),
])
def test_rows_config(kw, want):
    assert B.mok_check_rows_config(rows(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(lr=0.0), OK), (dict(eps=0.0), OK), (dict(beta1=0.0, beta2=0.0), OK),
    (dict(state=B.MOK_STATE_MXFP8, flags=B.MOK_ADAMW_STOCHASTIC), OK),
    (dict(lr=-1.0), BAD), (dict(lr=float("nan")), BAD), (dict(lr=float("inf")), BAD),
    (dict(beta1=1.0), BAD), (dict(beta2=-0.1), BAD), (dict(beta2=float("nan")), BAD),
    (dict(eps=-1e-8), BAD), (dict(eps=float("inf")), BAD), (dict(step=0), BAD),
    (dict(p_dtype=2), BAD), (dict(g_dtype=-1), BAD), (dict(state=2), BAD), (dict(flags=2), BAD),
    (dict(abi_version=1), B.MOK_ERR_ABI),
])
def test_adamw_config(kw, want):
    base = dict(lr=1e-3)
    base.update(kw)
    assert B.mok_check_adamw_config(B.make_adamw(**base)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(in_features=1, out_features=1), OK),
    (dict(groups=1024), OK), (dict(act=B.MOK_ACT_GELU), OK),
    (dict(out_dtype=B.MOK_DTYPE_F32, grad_dtype=B.MOK_DTYPE_F32), OK),
    (dict(ld_in=72, ld_w=80, ld_out=104), OK),
    (dict(rows=-1), BAD), (dict(rows=(1 << 31) - 512), BAD), (dict(groups=0), BAD),
    (dict(groups=1025), BAD), (dict(in_features=0), BAD), (dict(out_features=0), BAD),
    (dict(in_features=(1 << 20) + 1), BAD), (dict(ld_in=56), BAD), (dict(ld_in=65), BAD),
    (dict(ld_w=68), BAD), (dict(ld_out=90), BAD), (dict(act=5), BAD), (dict(act=-1), BAD),
    (dict(out_dtype=2), BAD), (dict(grad_dtype=2), BAD), (dict(abi_version=3), B.MOK_ERR_ABI),
    (dict(rows=1 << 30, out_features=1 << 20), BAD),  # more tiles than 31 bits number
])
def test_linear_config(kw, want):
    base = dict(rows=100, in_features=64, out_features=96)
    base.update(kw)
    c = B.make_linear(**base)
    assert B.mok_check_linear_config(c) == want
    for which in (B.MOK_LINEAR_FORWARD, B.MOK_LINEAR_BACKWARD):
        assert (B.mok_linear_workspace_size(c, which) > 0) == (want == OK)
    assert B.mok_linear_workspace_size(c, 2) == 0
