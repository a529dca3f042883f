"""The fine-tuning example: its gradients against float64 autograd of the same
formulas, its loss, and its serving step.

Tolerance.  Between the input and a gradient lie about ten tensors rounded to
binary16 (2^-11 of a value each) and sums of such; the router's gradient takes
a difference of two such values besides.  1/64 of the gradient's norm is more
than ten roundings amplified three times (0.015).
"""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

import quantized_moe_expert_02_amd as moe
from quantized_moe_expert_02_amd import synth

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "finetune.py")


def _example():
    spec = importlib.util.spec_from_file_location("finetune_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(layer, x, idx):
    """The layer's formula, token by token and slot by slot, for the given slots (-1: dropped)."""
    p = layer.trained()
    mats = [[w.double().cpu() for w in f] for f in layer.frozen]
    rw, rb, a, b = (v.detach().double().cpu().requires_grad_() for v in p)
    a16, b16 = (v + (v.detach().half().double() - v.detach()) for v in (a, b))  # rounded, with the gradient passed through
    x = x.double().cpu().requires_grad_()
    silu = lambda v, g, u: F.silu(v @ g.t()) * (v @ u.t())  # noqa: E731
    s = torch.sigmoid(x @ rw.t() + rb)
    out = []
    for t in range(x.shape[0]):
        slots = [e for e in idx[t].tolist() if e >= 0]
        y = silu(x[t], *mats[-1][:2]) @ mats[-1][2].t() if layer.dims.has_shared else torch.zeros(x.shape[1]).double()
        for e in slots:
            h = silu(x[t], *mats[e][:2])
            y = y + s[t, e] / s[t, slots].sum() * (h @ mats[e][2].t() + layer.scale[e].item() * (h @ a16[e].t()) @ b16[e].t())
        out.append(y)
    return torch.stack(out), [x, rw, rb, a, b]


@pytest.mark.parametrize("T,k,shared,top_p", [(37, 2, 1, 0.0), (5, 4, 0, 0.6)])
def test_gradients(T, k, shared, top_p):
    ex = _example()
    dims = synth.Dims(256, 128, 8, k, shared, top_p=top_p)
    print("finetune gradients", dims, T, flush=True)
    layer = ex.Layer(dims, rank=8)
    g = torch.Generator().manual_seed(5)
    with torch.no_grad():
        layer.b.copy_(torch.randn(layer.b.shape, generator=g) * 0.05)
    x = synth.make_tokens(dims, T, "grads").to("cuda").requires_grad_()
    dy = torch.randn((T, dims.hidden), generator=g).half()
    y = layer.forward(x)
    grads = torch.autograd.grad(y, [x] + layer.trained(), dy.to("cuda"))
    idx = moe.moe_route(layer.packed, x.detach())["topk_idx"].cpu()
    ref, leaves = _plain(layer, x.detach(), idx)
    want = torch.autograd.grad(ref, leaves, dy.double())
    for name, got, r in zip(("y", "x", "router_w", "router_b", "a", "b"), (y, *grads), (ref, *want)):
        got, r = got.detach().double().cpu(), r.detach()
        off = float((got - r).norm() / r.norm())
        print(name, "%.2e" % off, flush=True)
        assert off <= 1 / 64, name


def test_training_lowers_the_loss():
    ex = _example()
    dims = synth.Dims(256, 128, 8, 2)
    print("finetune training", flush=True)
    layer = ex.Layer(dims)
    x = synth.make_tokens(dims, 256, "train").to("cuda")
    with torch.no_grad():
        target = 1.3 * layer.forward(x).float()
    losses = ex.train(layer, x, target, 20)
    print(losses[0], losses[-1], flush=True)
    assert losses[-1] < 0.9 * losses[0]


def test_serving_step():
    ex = _example()
    dims = synth.Dims(256, 128, 8, 2)
    print("finetune serving", flush=True)
    layer = ex.Layer(dims)
    x = synth.make_tokens(dims, 6, "serve").to("cuda")
    g = torch.Generator().manual_seed(6)
    a, b = torch.randn((3, 16, 256), generator=g).half(), torch.randn((3, 256, 16), generator=g).half()
    scale, ids = torch.tensor([0.01, 0.02, 0.03]), torch.tensor([2, 0, -1, 1, 2, 3], dtype=torch.int32)
    y = ex.serve(layer.packed, x, a.to("cuda"), b.to("cuda"), ids.to("cuda"), scale.to("cuda")).double().cpu()
    base = moe.moe_w4a16_forward(layer.packed, x).double().cpu()
    for t, i in enumerate(ids.tolist()):
        ref = base[t]
        if 0 <= i < 3:
            ref = ref + scale[i].double() * (b[i].double() @ (a[i].double() @ x[t].double().cpu()))
        # one rounding to binary16, and fp32 sums of up to 256 terms of the adapter's size
        assert bool(((y[t] - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -14 * ref.abs().max() + 2.0 ** -25).all()), t
