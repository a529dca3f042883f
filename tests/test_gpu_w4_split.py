"""4-bit products of several experts by the kernels for many rows, with and without split sums,
against 64 bits.  Tolerances as in test_gpu_w4.py."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_w4 import BF16, DEV, F16, SHAPES, check, make, pack, tolerance
from w4_reference import product, weights

pytestmark = pytest.mark.gpu


def run(n, N, K, group, zeros, T, offsets, dtype, backward, add, split):
    c = make(T, K, N, n, group, dtype, zeros, n + T + N, offsets, backward)
    for e0, e1 in ((0, offsets[0]), (offsets[-1], T)):  # not read
        c["x"][e0:e1] = float("nan")
    w = pack(c)
    what = f"experts n={n} N={N} K={K} T={T} {dtype} backward={backward}"
    print(what, flush=True)
    assert (moe.lib().moe_w4_workspace_bytes(w.dims, T, int(backward)) > 0) == split
    assert backward or not moe.moe_w4_few_rows(w, T)
    call = moe.moe_w4_backward if backward else moe.moe_w4_forward
    got = call(c["x"].to(DEV), w, offsets=c["offsets"].to(DEV), add=c["add"].to(DEV) if add else None)
    torch.cuda.synchronize()
    c["x"] = torch.nan_to_num(c["x"])
    m = weights(c["q"], c["scales"], c["zeros"])
    ref, norm = product(c["x"], m, c["offsets"], backward)
    check(got, ref + c["add"].double() if add else ref, tolerance(c, m, norm, False, backward), dtype, what)


# rows before and after the groups, empty groups, one row, tiles that are full and not
OFFSETS = [(3, [2, 20, 20, 61], 64), (4, [0, 1, 1, 97, 130], 133), (4, [3, 3, 3, 3, 19], 20), (2, [0, 0, 300], 300)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,offsets,T", OFFSETS)
@pytest.mark.parametrize("N,K,group,zeros", [(200, 1280, 128, True), (72, 2080, 32, True), (136, 4160, 64, False), (264, 6240, 0, True)])
def test_split_forward(N, K, group, zeros, n, offsets, T, dtype):
    run(n, N, K, group, zeros, T, offsets, dtype, False, T % 2 == 0, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,offsets,T", OFFSETS)
@pytest.mark.parametrize("N,K,group,zeros", [(6152, 96, 32, True), (6280, 320, 64, False), (8200, 160, 0, True)])
def test_split_gradient(N, K, group, zeros, n, offsets, T, dtype):
    run(n, N, K, group, zeros, T, offsets, dtype, True, T % 2 == 0, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,offsets,T", [(4, [5, 80, 80, 290, 300], 310), (3, [0, 400, 401, 690], 700)])
def test_split_gradient_of_many_columns(n, offsets, T, dtype):
    """Too many tiles for the gradient's kernel without workspace, tiles of 64 and 128 rows."""
    run(n, 1000, 2080, 32, True, T, offsets, dtype, True, True, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [17, 33, 65, 129, 400])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES[:8])
def test_many_rows_of_two(N, K, group, zeros, T, dtype):
    """The kernel for many rows at every shape of the few rows' tests."""
    run(2, N, K, group, zeros, T, [1, 1 + T // 3, T], dtype, False, T % 2 == 0, K > 640)
