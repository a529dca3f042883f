"""Products and loss gradients whose output shares memory with the rows that they read are
refused, before any launch (no GPU needed)."""
import pytest

import quantized_moe_expert_02_amd as moe
from test_w4_distill_host import INVAL, L, WORKSPACE, dims  # noqa: F401

P, FAR = 1 << 30, 1 << 40  # addresses that a refused call never touches


def call(L, backward, x, ldx, y, ldy, T, add=None, ldadd=0, K=64, N=64, ws_bytes=1 << 40):
    d = dims(N=N, K=K, group=32)
    return (L.moe_w4_backward if backward else L.moe_w4_forward)(d, FAR, x, ldx, T, None, add, ldadd, y, ldy, FAR, ws_bytes, None)


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("T", [1, 5, 700, 5000])
def test_products(L, backward, T):  # noqa: F811
    for ldx, at, ldy in ((64, 0, 64), (64, 16, 64), (64, -16, 64), (64, 2 * 64 * T - 16, 64), (64, -2 * 64 * T + 16, 64),
                         (160, 112, 160), (160, -112, 160), (160, 0, 64), (64, 0, 160), (160, 2 * 160 * (T - 1), 160),
                         (160, 2 * 160 * (T - 1) + 112, 168), (160, -2 * 160 * (T - 1) - 112, 160)):
        assert call(L, backward, P, ldx, P + at, ldy, T) == INVAL, (ldx, at, ldy)
        if at or (ldx != ldy and T > 1):  # (add may be y)
            assert call(L, backward, FAR << 1, 64, P, ldx, T, P + at, ldy) == INVAL, ("add", ldx, at, ldy)


def test_other_strides_in_one_stretch(L):  # noqa: F811
    """Rows of two strides between each other's: refused, although these do not meet."""
    assert call(L, 0, P, 256, P + 128, 512, 3) == INVAL


def test_missing_workspace_is_named_first(L):  # noqa: F811
    assert call(L, 0, P, 8192, P, 8192, 64, K=8192, N=8192, ws_bytes=16) == WORKSPACE


@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 2), (2, 4)])
def test_loss_gradient(L, dtype, size):  # noqa: F811
    for T, ldz, at, lddz in ((4, 1000, size, 1000), (4, 1000, -size, 1000), (4, 1000, 1000 * size, 1000), (4, 1000, 3999 * size, 1000),
                             (4, 2100, 999 * size, 2100), (4, 2100, -999 * size, 2100), (1, 1000, 999 * size, 1000), (4, 1000, 0, 1008),
                             (4, 1000, 4, 1008)):
        assert L.moe_distill_backward(P, dtype, ldz, T, 1000, FAR, FAR, 4, 1.0, FAR, FAR, P + at, lddz, None) == INVAL, (T, ldz, at, lddz)
