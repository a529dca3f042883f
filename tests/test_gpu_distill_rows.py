"""The distillation loss' statistics where a row holds NaNs or infinities: (m, l) are the
formulas', m = max z (NaN if any logit is) and l = log sum exp((z - m) / tau)."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_distill import BF16, DEV, F16, F32, INF, NAN, dev, make

pytestmark = pytest.mark.gpu


# a wavefront per row, 512 threads per row, chunks, whole rows past 64 Ki columns
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,V", [(8, 700), (8, 30000), (8, 70001), (260, 70001)])
def test_statistics_of_nan_and_infinity(T, V, dtype):
    c = make(T, V, 8, dtype, 12)
    z = c["z"]
    z[0, 0], z[1, V - 1], z[2, V // 2] = NAN, NAN, NAN
    z[3, :] = NAN
    z[4, V // 3], z[4, 5] = INF, NAN
    z[5, V // 3] = INF
    z[6, :] = -INF
    z[6, V - 2] = NAN
    d = dev(c)
    print("statistics", T, V, dtype, flush=True)
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"])
    m = z.double().max(1)[0]
    assert torch.equal(stats[:, 0].double().cpu().nan_to_num(-1e30), m.nan_to_num(-1e30))
    assert bool(stats[:7, 1].isnan().all()) and bool(loss[:7].isnan().all()) and bool(grad[:7].isnan().all())
    assert bool(torch.isfinite(stats[7:]).all()) and bool(torch.isfinite(loss[7:]).all()) and bool(torch.isfinite(grad[7:]).all())


@pytest.mark.parametrize("V", [700, 30000, 70001])
def test_smallest_probabilities(V):
    """A teacher's entry below 2^-126 counts as 0, also at a logit of -infinity; one above does not."""
    c = make(4, V, 3, F32, 13)
    c["teacher"][:] = torch.tensor([[0.0, -88.0, -1.0], [0.0, -86.0, -1.0], [0.0, -200.0, -1.0], [0.0, -INF, -1.0]])
    c["z"].scatter_(1, c["ids"][:, 1:2].long(), -INF)
    d = dev(c)
    print("smallest", V, flush=True)
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"])
    assert torch.isfinite(loss).tolist() == [True, False, True, True] and loss[1] == INF
    assert bool(torch.isfinite(grad).all())
