"""Products of few rows with 4-bit weights: the codes are exact factors, so that a result's
error is that of an fp32 sum of its own terms, however large an element stands at a code that
equals its zero point.

Tolerance: the output's rounding, half a step of its type, and of fp32 sums of n terms w x
with errors of either sign 4 sqrt(n) 2^-24 sum |w x|, as in test_gpu_w4.py but with the terms'
own magnitudes."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_w4 import BF16, DEV, F16, UNIT, make, pack
from w4_reference import weights

pytestmark = pytest.mark.gpu


def check(c, what):
    got = moe.moe_w4_forward(c["x"].to(DEV), pack(c)).double().cpu()
    w, x = weights(c["q"], c["scales"], c["zeros"])[0], c["x"].double()
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    bound = UNIT[c["x"].dtype] * ref.abs() + 2.0 ** -25 * (c["x"].dtype == F16) + 4 * x.shape[1] ** 0.5 * 2.0 ** -24 * size
    worst = float(((got - ref).abs() / bound.clamp(min=1e-300)).max())
    print(what, "worst error / tolerance %.3f" % worst, flush=True)
    assert bool(torch.isfinite(got).all()) and worst <= 1.0, (what, worst)
    return got


def cleared(c, columns):
    """Codes of `columns` that equal their zero points (0 without them)."""
    z = torch.zeros(c["scales"].shape, dtype=torch.int8) if c["zeros"] is None else c["zeros"]
    group = c["q"].shape[2] * 2 // z.shape[2]
    for k in columns:
        code, shift = (z[:, :, k // group].int() & 15).to(torch.uint8), 4 * (k % 2)
        c["q"][:, :, k // 2] = (c["q"][:, :, k // 2] & (0xF0 >> shift)) | (code << shift)
    return c


@pytest.mark.parametrize("dtype,large", [(F16, 6e4), (BF16, 3e4), (BF16, 1e6), (BF16, 1e30), (BF16, 3e38)])
@pytest.mark.parametrize("T,N,K,group,zeros", [(3, 72, 2048, 128, False), (16, 40, 2048, 32, True), (1, 200, 6272, 64, True),
                                               (5, 264, 320, 0, False), (40, 136, 4096, 128, True)])
def test_large_elements_at_zero_weights(T, N, K, group, zeros, dtype, large):
    c = cleared(make(T, K, N, 1, group, dtype, zeros, T + K), (5, K // 2 + 2, K - 1))
    c["x"][:, 5], c["x"][0, K // 2 + 2], c["x"][T // 2, K - 1] = large, -large, large
    print("large", T, N, K, group, zeros, dtype, large, flush=True)
    check(c, "large elements")


@pytest.mark.parametrize("zeros", [False, True])
def test_zero_weights_give_zero(zeros):
    c = make(4, 1024, 48, 1, 64, BF16, zeros, 3)
    print("zero weights", zeros, flush=True)
    assert bool((check(cleared(c, range(1024)), "zero weights") == 0).all())


def test_wide_zero_points():
    """|q - z| up to 136."""
    for T in (2, 16):
        check(make(T, 4128, 88, 1, 32, BF16, "wide", T), f"wide zero points T={T}")


def test_sums_past_the_range():
    """Sums of q x past fp32's range, before the scale, although the results are not."""
    c = make(6, 1280, 24, 1, 128, BF16, False, 5)
    c["q"][:] = 0x77
    c["x"] = torch.full((6, 1280), 2.5e38).to(BF16)
    c["scales"] = torch.full(c["scales"].shape, 2.0 ** -14).to(BF16)
    print("range", flush=True)
    check(c, "past the range")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinities_in_wide_rows(dtype):
    """Infinities and NaNs of a wide row stay in that row and are the formula's; the others are as without them."""
    c = make(5, 65536, 40, 1, 128, dtype, True, 6)
    w = pack(c)
    print("wide infinities", dtype, flush=True)
    plain = moe.moe_w4_forward(c["x"].to(DEV), w).cpu()
    c["x"][0, 40000], c["x"][2, 7], c["x"][3, 3], c["x"][3, 4] = float("inf"), float("nan"), float("inf"), float("-inf")
    got = moe.moe_w4_forward(c["x"].to(DEV), w).cpu()
    m = weights(c["q"], c["scales"], c["zeros"])[0]
    for row, ks in ((0, (40000,)), (2, (7,)), (3, (3, 4))):
        want = sum(c["x"][row, k].double() * m[:, k] for k in ks)
        mine = got[row].double()
        assert torch.equal(mine.isnan(), want.isnan()) and torch.equal(mine.nan_to_num(1, 2, -2), want.nan_to_num(1, 2, -2)), row
    assert torch.equal(got[[1, 4]], plain[[1, 4]])
