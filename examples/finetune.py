"""Fine-tunes a MoE layer with frozen 4-bit experts, and serves it with an
adapter per request.

Trained: the router, and a low-rank adapter on every expert's down projection.
A step runs the router (moe_route), lays the tokens out by expert
(moe_dispatch), multiplies them by the frozen experts' 4-bit matrices
(moe_w4_forward), adds the adapters to the experts' outputs
(moe_adapter_forward), combines them (moe_combine), and goes back through the
gradients of all five; torch.autograd strings the pieces together.  The layer is
first tuned towards outputs of its own width, then, under a frozen 4-bit output
head, towards a teacher's top logits (moe_distill_forward).

  python examples/finetune.py [--steps 30] [--tokens 512]
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_moe_expert_02_amd as moe  # noqa: E402
from quantized_moe_expert_02_amd import synth  # noqa: E402


class RouteDispatch(torch.autograd.Function):
    """(x, router_w, router_b) -> (xs, topk_w, offsets, pairs, pos, topk_idx)."""

    @staticmethod
    def forward(ctx, x, router_w, router_b, layer):
        r = moe.moe_route(layer, x)  # (router_w and router_b are the layer's own)
        d = moe.moe_dispatch(x, r["topk_idx"], layer.dims.n_experts)
        ctx.save_for_backward(x, router_w, router_b, r["topk_idx"], d["offsets"], d["pairs"], d["pos"])
        rest = d["offsets"], d["pairs"], d["pos"], r["topk_idx"]
        ctx.mark_non_differentiable(*rest)
        return (d["xs"], r["topk_w"], *rest)

    @staticmethod
    def backward(ctx, dxs, dw, *_):
        x, router_w, router_b, idx, offsets, pairs, pos = ctx.saved_tensors
        dx = moe.moe_dispatch_backward(dxs.contiguous(), pos)
        dx, d_router_w, d_router_b = moe.moe_route_backward(x, router_w, router_b, idx, dw.contiguous(), offsets, pairs,
                                                            add=dx)
        return dx, d_router_w, d_router_b, None


class Adapters(torch.autograd.Function):
    """base + scale B A x, a row's adapter by ids.  a and b are the 32-bit values
    that the optimiser keeps; the products take them rounded to x's type."""

    @staticmethod
    def forward(ctx, x, a, b, base, ids, scale, offsets, rows):
        a16, b16, order = a.to(x.dtype), b.to(x.dtype), dict(offsets=offsets, pairs=rows)
        y, u = moe.moe_adapter_forward(x, a16, b16, ids, scale, add=base, order=order, save_u=True)
        ctx.save_for_backward(x, u, a16, b16, ids, scale, offsets, rows)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, u, a16, b16, ids, scale, offsets, rows = ctx.saved_tensors
        dx, da, db = moe.moe_adapter_backward(dy.contiguous(), x, u, a16, b16, ids, scale,
                                              order=dict(offsets=offsets, pairs=rows))
        return dx, da, db, dy, None, None, None, None


class Combine(torch.autograd.Function):
    """add + the slots' rows of o with their routing weights."""

    @staticmethod
    def forward(ctx, o, topk_w, add, pairs, pos):
        ctx.save_for_backward(o, topk_w, pairs, pos)
        return moe.moe_combine(o, topk_w, pos, add=add)

    @staticmethod
    def backward(ctx, dy):
        o, topk_w, pairs, pos = ctx.saved_tensors
        do, dw = moe.moe_combine_backward(dy.contiguous(), o, topk_w, pos, pairs)
        return do, dw, dy if ctx.needs_input_grad[2] else None, None, None


class Product(torch.autograd.Function):
    """Rows times the frozen 4-bit matrix of their group (one matrix: of all rows)."""

    @staticmethod
    def forward(ctx, x, w, offsets=None):
        ctx.w, ctx.offsets = w, offsets
        return moe.moe_w4_forward(x, w, offsets=offsets)

    @staticmethod
    def backward(ctx, dy):
        return moe.moe_w4_backward(dy.contiguous(), ctx.w, offsets=ctx.offsets), None, None


class Distillation(torch.autograd.Function):
    """Every row's divergence from a teacher's top logits."""

    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature):
        loss, stats = moe.moe_distill_forward(logits, ids, teacher, temperature)
        ctx.save_for_backward(logits, ids, teacher, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, dloss):
        logits, ids, teacher, stats = ctx.saved_tensors
        return moe.moe_distill_backward(logits, ids, teacher, stats, dloss.contiguous(), ctx.temperature), None, None, None


def dequantise(dims, packed, dtype=torch.float16):
    """The three matrices of one packed int4 expert."""
    qg, sg, qu, su, qd, sd, _ = moe.moe_unpack(dims, packed)

    def matrix(q, s):
        codes = torch.stack((q & 0xF, q >> 4), dim=2).reshape(q.shape[0], -1).to(torch.int8)
        codes = torch.where(codes > 7, codes - 16, codes)
        return (codes.to(dtype) * s.to(dtype)[:, None]).contiguous()

    return matrix(qg, sg), matrix(qu, su), matrix(qd, sd)


def products(dims, packed):
    """(gate and up, down) of packed int4 experts [n], as moe_w4_forward takes them: one scale per row."""
    parts = [moe.moe_unpack(dims, p) for p in packed]
    qg, sg, qu, su, qd, sd = (torch.stack([p[i] for p in parts]) for i in range(6))
    gate_up = moe.moe_w4_pack(torch.cat((qg, qu), 1), torch.cat((sg, su), 1)[:, :, None].contiguous())
    return gate_up, moe.moe_w4_pack(qd, sd[:, :, None].contiguous())


def swiglu(x, gate_up, offsets=None):
    gate, up = Product.apply(x, gate_up, offsets).chunk(2, dim=1)
    return F.silu(gate) * up


class Layer:
    """The packed layer, its frozen matrices, and what is trained."""

    def __init__(self, dims, rank=16, device="cuda", seed="finetune"):
        self.dims, self.packed = dims, moe.PackedLayer.from_layer(synth.make_layer(dims, seed), device=device)
        if self.packed.router_b is None:
            self.packed.router_b = torch.zeros(dims.n_experts, device=device)
        self.experts = products(dims, self.packed.packed[:dims.n_experts])
        self.shared = products(dims, self.packed.packed[dims.n_experts:]) if dims.has_shared else None
        g = torch.Generator().manual_seed(1)
        shape = (dims.n_experts, rank, dims.inter)
        self.a = (torch.randn(shape, generator=g) / dims.inter ** 0.5).to(device)
        self.b = torch.zeros((dims.n_experts, dims.hidden, rank), device=device)
        self.scale = torch.full((dims.n_experts,), 2.0, device=device)
        for p in self.trained():
            p.requires_grad_()

    @property
    def frozen(self):
        """The frozen matrices, expert by expert (the shared one last), dequantised."""
        return [dequantise(self.dims, p) for p in self.packed.packed]

    def trained(self):
        return [self.packed.router_w, self.packed.router_b, self.a, self.b]

    def forward(self, x):
        """y [T][hidden] of x [T][hidden], with gradients."""
        xs, topk_w, offsets, pairs, pos, idx = RouteDispatch.apply(x, self.packed.router_w, self.packed.router_b, self.packed)
        act = swiglu(xs, self.experts[0], offsets)
        base = Product.apply(act, self.experts[1], offsets)  # (rows past the groups, of slots that top-p dropped: zeros)
        ids = torch.where(pairs < 0, -1, idx.reshape(-1)[pairs.clamp(min=0).long()])
        rows = torch.arange(xs.shape[0], dtype=torch.int32, device=x.device)  # they are in the adapters' order already
        o = Adapters.apply(act, self.a, self.b, base, ids, self.scale, offsets, rows)
        shared = None
        if self.dims.has_shared:
            shared = Product.apply(swiglu(x, self.shared[0]), self.shared[1])
        return Combine.apply(o, topk_w, shared, pairs, pos)


def train(layer, x, target, steps, lr=(1e-4, 5e-4)):
    """Adam (lr: the router's and the adapters') on the squared error relative to
    the target's: the losses before each step."""
    groups = [dict(params=p, lr=r) for p, r in zip((layer.trained()[:2], layer.trained()[2:]), lr)]
    losses, optimiser = [], torch.optim.Adam(groups)
    for _ in range(steps):
        optimiser.zero_grad()
        loss = (layer.forward(x).float() - target).square().sum() / target.square().sum()
        (loss * 1024).backward()  # (scaled, which Adam does not see, to keep the 16-bit gradients in range)
        optimiser.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def distil(layer, head, x, ids, teacher, steps, temperature=2.0, lr=(1e-4, 5e-4)):
    """Adam on the mean divergence of the logits head(layer(x)) (x added as the residual)
    from a teacher's top logits `teacher` at `ids`: the losses before each step."""
    groups = [dict(params=p, lr=r) for p, r in zip((layer.trained()[:2], layer.trained()[2:]), lr)]
    losses, optimiser = [], torch.optim.Adam(groups)
    for _ in range(steps):
        optimiser.zero_grad()
        logits = Product.apply(x + layer.forward(x), head)
        loss = Distillation.apply(logits, ids, teacher, temperature).mean()
        (loss * 1024).backward()
        optimiser.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve(packed, x, a, b, ids, scale, ranks=None):
    """One step for requests that share the layer and have an adapter each (or
    none: an id outside the adapters), hidden -> hidden."""
    with torch.no_grad():
        y = moe.moe_w4a16_forward(packed, x)
        return moe.moe_adapter_forward(x, a, b, ids, scale, ranks=ranks, add=y, out=y)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    args = ap.parse_args()
    dims = synth.Dims(256, 128, 8, 2)
    layer = Layer(dims)
    x = synth.make_tokens(dims, args.tokens, "finetune").to("cuda")
    with torch.no_grad():  # to be learnt: the layer's own output, turned a little
        turn = torch.randn((dims.hidden, dims.hidden), generator=torch.Generator().manual_seed(2)).to("cuda")
        y = layer.forward(x).float()
        target = y + 0.3 * y @ turn / dims.hidden ** 0.5
    losses = train(layer, x, target, args.steps)
    print(f"loss {losses[0]:.3e} -> {losses[-1]:.3e} in {args.steps} steps of {args.tokens} tokens")

    vocab, k = 1024, 16  # a 4-bit head with a scale for every 64 columns, and a teacher whose layer is turned as above
    g = torch.Generator().manual_seed(4)
    q = torch.randint(0, 256, (vocab, dims.hidden // 2), generator=g, dtype=torch.uint8).to("cuda")
    scales = (torch.rand((vocab, dims.hidden // 64), generator=g) * 0.04 + 0.02).half().to("cuda")
    head = moe.moe_w4_pack(q, scales)
    with torch.no_grad():
        teacher, ids = torch.topk(moe.moe_w4_forward((x + target).half(), head).float(), k, dim=1)
    losses = distil(Layer(dims), head, x, ids.int(), teacher, args.steps)
    print(f"distilled {losses[0]:.3e} -> {losses[-1]:.3e} in {args.steps} steps, {k} of {vocab} logits")

    torch.manual_seed(3)
    n, rank = 4, 8  # four requests' adapters of ranks up to 8
    a, b = torch.randn((n, rank, dims.hidden)) / 16, torch.randn((n, dims.hidden, rank)) / 16
    ids = torch.tensor([0, 3, -1, 1, 0], dtype=torch.int32, device="cuda")
    ranks = torch.tensor([8, 4, 8, 2], dtype=torch.int32, device="cuda")
    y = serve(layer.packed, x[:5], a.to("cuda").half(), b.to("cuda").half(), ids, torch.ones(n, device="cuda"), ranks)
    print(f"served {y.shape[0]} requests, {int((ids >= 0).sum())} of them with an adapter; |y| = {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()
