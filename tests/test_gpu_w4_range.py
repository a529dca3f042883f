"""4-bit products at the ends of their scales' range: the largest that the header allows, and
rows and scales so small that products are subnormal.  Tolerances as in test_gpu_w4.py."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_w4 import BF16, DEV, F16, UNIT, make, pack, run_case
from w4_reference import product, weights

pytestmark = pytest.mark.gpu
WAYS = [(6, False, True), (700, False, False), (6, True, False), (700, True, False)]  # T, backward, few rows


@pytest.mark.parametrize("zeros", [False, "wide"])
@pytest.mark.parametrize("T,backward,few", WAYS)
def test_largest_bfloat16_scales(T, backward, few, zeros):
    """Scales up to 2^117: weights up to 2^124, with rows that bring the results into range."""
    c = make(T, 640, 264, 1, 64, BF16, zeros, 21, backward=backward)
    c["scales"] = (2.0 ** 117 * torch.rand(c["scales"].shape, generator=torch.Generator().manual_seed(1))).to(BF16)
    c["scales"][:, ::3] = 2.0 ** 117
    c["x"] = (c["x"].float() * 2.0 ** -108).to(BF16)
    assert run_case(c, backward, False, f"large scales T={T} backward={backward} zeros={zeros}") == few


@pytest.mark.parametrize("zeros", [False, "wide"])
@pytest.mark.parametrize("T,backward,few", WAYS)
def test_largest_binary16_weights(T, backward, few, zeros):
    """Weights up to 65504 where they are rounded, scales up to 65504 where they are not."""
    top = 65504.0 if few else 65504.0 / (136 if zeros else 8)
    c = make(T, 640, 264, 1, 64, F16, zeros, 22, backward=backward)
    c["scales"] = (top * torch.rand(c["scales"].shape, generator=torch.Generator().manual_seed(2))).to(F16)
    c["scales"][:, ::3] = torch.tensor(top).to(F16) if few else 2.0 ** (8 if zeros else 12)
    c["x"] = (c["x"].float() * 2.0 ** -18).to(F16)
    assert run_case(c, backward, False, f"large weights T={T} backward={backward} zeros={zeros}") == few


@pytest.mark.parametrize("T,backward,few", WAYS)
def test_small_rows(T, backward, few):
    """Rows near bfloat16's smallest normal number: subnormal products are kept."""
    c = make(T, 640, 264, 1, 64, BF16, True, 23, backward=backward)
    c["scales"] = (c["scales"].float() * 64).to(BF16)
    c["x"] = (c["x"].float() * 2.0 ** -120).to(BF16)
    print("small", T, backward, flush=True)
    w, call = pack(c), moe.moe_w4_backward if backward else moe.moe_w4_forward
    assert backward or moe.moe_w4_few_rows(w, T) == few
    got = call(c["x"].to(DEV), w).double().cpu()
    ref, norm = product(c["x"], weights(c["q"], c["scales"], c["zeros"]), None, backward)
    # half a step of the outputs (2^-134 where subnormal) and, at random, of the weights; half a
    # subnormal step of fp32, 2^-150, of 640 terms, times 2^15 where factors are 2^-15 of the codes
    # (scales are below 1)
    bound = UNIT[BF16] * (ref.abs() + 7 * norm) + 2.0 ** -134 + 640 * 2.0 ** -135
    assert bool(((got - ref).abs() <= bound).all())
