"""Outputs and inputs in one buffer: rows between each other's are taken, shared memory is refused."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_distill import dev
from test_gpu_distill import make as make_logits
from test_gpu_w4 import DEV, F16, make, pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T", [1, 7, 40, 1300])
def test_products(T, backward):
    c = make(T, 256, 256, 1, 64, F16, True, 3, backward=backward)
    w, call = pack(c), moe.moe_w4_backward if backward else moe.moe_w4_forward
    x, add = c["x"].to(DEV), c["add"].to(DEV)
    print("overlap", T, backward, flush=True)
    want, plain = call(x, w, add=add), call(x, w)
    both = torch.full((T, 3 * 256), 7.0, dtype=F16, device=DEV)  # x, y and add touch, row by row
    for places in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        xs, ys, adds = (both[:, 256 * i:256 * i + 256] for i in places)
        xs.copy_(x)
        adds.copy_(add)
        call(xs, w, add=adds, out=ys)
        assert torch.equal(ys, want) and torch.equal(xs, x) and torch.equal(adds, add)
    stacked = torch.empty((2 * T, 256), dtype=F16, device=DEV)  # x's last row touches y's first
    stacked[:T].copy_(x)
    assert torch.equal(call(stacked[:T], w, out=stacked[T:]), plain)
    assert torch.equal(call(x, w, add=x), call(x, w, add=x.clone()))  # (both are read)
    for xs, ys in ((x, x), (stacked[:T], stacked[T - 1:-1]), (both[:, :256], both[:, 8:264])):
        with pytest.raises(moe.MoeError):
            call(xs, w, out=ys)
        if ys.data_ptr() != xs.data_ptr():  # (add may be out)
            with pytest.raises(moe.MoeError):
                call(want, w, add=xs, out=ys)


def test_loss_gradient():
    d = dev(make_logits(6, 3000, 5, F16, 2))
    print("overlap of logits", flush=True)
    _, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
    args = (d["ids"], d["teacher"], stats, d["dloss"])
    want = moe.moe_distill_backward(d["z"], *args)
    both = torch.full((6, 6000), 7.0, dtype=F16, device=DEV)
    for a, b in ((0, 3000), (3000, 0)):
        z = both[:, a:a + 3000]
        z.copy_(d["z"])
        assert torch.equal(moe.moe_distill_backward(z, *args, out=both[:, b:b + 3000]), want) and torch.equal(z, d["z"])
    flat = torch.zeros(7 * 3000, dtype=F16, device=DEV)
    for z, out in ((both[:, :3000], both[:, 2999:5999]), (flat[:18000].view(6, 3000), flat[3000:].view(6, 3000)),
                   (flat[1:18001].view(6, 3000), flat[:18000].view(6, 3000))):
        with pytest.raises(moe.MoeError):
            moe.moe_distill_backward(z, *args, out=out)
