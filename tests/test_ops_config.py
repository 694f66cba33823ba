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
