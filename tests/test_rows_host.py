"""Most rows of the expert-sorted buffers that the gradients take, and the status of
shapes that the binding refuses: decided on the host before any launch (no GPU needed)."""
import os

import pytest

import quantized_moe_expert_02_amd as moe

UNSUPPORTED, WORKSPACE = -2, -3
P = 1 << 20  # an aligned address that a refused call never touches
MOST = (1 << 25) + (1 << 20)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from quantized_moe_expert_02_amd import build
        build.build()
    return moe.lib()


def test_every_sort_fits(L):
    assert MOST >= L.moe_sort_rows(1 << 20, 32, 1024, 1024) > 1 << 25


@pytest.mark.parametrize("rows", [MOST + 1, 1 << 27, 1 << 29, 2 ** 31 - 65, 2 ** 31 - 1])
def test_more_rows_are_refused(L, rows):
    """Their indices would pass 32 bits inside the kernels."""
    for T in (0, 4, 600):
        assert L.moe_combine_backward(P, P, 0, rows, 64, P, P, P, T, 2, P, P, None) == UNSUPPORTED
        assert L.moe_route_backward(P, 0, T, 64, 8, 2, P, None, P, P, P, P, rows, None, P, P, P, P, 1 << 40, None) == UNSUPPORTED
        assert L.moe_route_backward_workspace_bytes(T, 2, 8, 64, rows) == 0


def test_the_most_is_accepted(L):
    """(As far as the size of the workspace, which is asked for next.)"""
    for T in (0, 4, 600):
        need = L.moe_route_backward_workspace_bytes(T, 2, 8, 64, MOST)
        assert need > 0
        assert L.moe_route_backward(P, 0, T, 64, 8, 2, P, None, P, P, P, P, MOST, None, P, P, P, P, need - 1, None) == WORKSPACE


@pytest.mark.parametrize("shape,status", [((1, 1, 2000, 1), UNSUPPORTED), ((1, 33, 64, 1), UNSUPPORTED), ((1 << 21, 1, 8, 1), UNSUPPORTED),
                                          ((1, 9, 8, 1), -1), ((1, 1, 8, 0), -1), ((-1, 1, 8, 1), -1)])
def test_binding_gives_the_status_of_a_refused_shape(L, shape, status):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_sort_rows(*shape)
    assert e.value.code == status
