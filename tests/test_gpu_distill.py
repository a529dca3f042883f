"""The distillation loss and its gradient on the GPU, against 64 bits.

Tolerances.  Everything is formed in fp32 from exact logits.  An exponent
(z - m) / tau - l is off by at most 4 roundings of its size (2^-24 each) and l by
its own sum's, which is of positive terms: 4 sqrt(V) 2^-24 relative, as are the
teacher's sums over k terms.  So q and p are off by e = 2^-24 (4 (|exponent| + |l|
+ sqrt(V) + sqrt(k)) + 8) of themselves (the constant: exp2 and log of one or two
units, products), a loss by the same e times its terms' magnitudes plus p's.  The
gradient is rounded once more to its type.
"""
import pytest
import torch

import quantized_moe_expert_02_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
STEP = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -149}  # half of the smallest
INF, NAN = float("inf"), float("nan")


def make(T, V, k, dtype, seed, repeat=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, V), generator=g) * 2.5
    top, ids = torch.topk(z + torch.randn((T, V), generator=g), min(k, V), dim=1)
    if repeat or k > V:
        at = torch.randint(0, min(k, V), (T, k), generator=g)
        top, ids = top.gather(1, at), ids.gather(1, at)
    return dict(z=z.to(dtype), ids=ids.int().contiguous(), teacher=top.float().contiguous(), dloss=torch.rand(T, generator=g) + 0.5)


def reference(c, tau):
    """loss, stats, gradient and what the tolerances take, in 64 bits."""
    z, ids, V = c["z"].double(), c["ids"].long(), c["z"].shape[1]
    T, k = ids.shape
    o = dict(loss=torch.zeros(T).double(), stats=torch.zeros((T, 2)).double(), grad=torch.zeros((T, V)).double(),
             size=torch.zeros(T).double(), terms=torch.zeros((T, V)).double())
    for t in range(T):
        ok = (ids[t] >= 0) & (ids[t] < V)
        a = c["teacher"][t].double()[ok]
        if not ok.any() or bool((a == -INF).all()):
            continue
        p = torch.softmax(a / tau, 0)
        m = z[t].max()
        l = torch.logsumexp((z[t] - m) / tau, 0)
        logq = (z[t] - m) / tau - l
        at = ids[t][ok]
        terms = torch.where(p > 0, p * (torch.log(p) - logq[at]), 0.0)
        o["loss"][t], o["stats"][t] = terms.sum(), torch.stack((m, l))
        o["size"][t] = torch.where(p > 0, p * (torch.log(p).abs() + logq[at].abs() + 1), 0.0).sum()
        taken = torch.zeros(V).double().scatter_add_(0, at, p)
        o["grad"][t] = (torch.exp(logq) - taken) * c["dloss"][t].double() / tau
        o["terms"][t] = (torch.exp(logq) * (1 + logq.abs().clamp(max=1e4)) + taken) * c["dloss"][t].double() / tau
    return o


def dev(c):
    return {n: t.to(DEV) for n, t in c.items()}


def within(got, ref, bound, what):
    g = got.detach().double().cpu()
    assert g.shape == ref.shape and bool(torch.isfinite(g).all()), what
    worst = float(((g - ref).abs() / bound).max())
    print(what, "worst error / tolerance %.3f" % worst, flush=True)
    assert worst <= 1.0, (what, worst)


def run_case(c, tau, what, **kw):
    print(what, flush=True)
    d, o = dev(c), reference(c, tau)
    V, k = c["z"].shape[1], c["ids"].shape[1]
    e = 2.0 ** -24 * (4 * (o["stats"][:, 1].abs() + V ** 0.5 + k ** 0.5 + 20) + 8)
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"], temperature=tau)
    within(loss, o["loss"], e * o["size"] + 1e-30, what + " loss")
    assert torch.equal(stats[:, 0].double().cpu(), o["stats"][:, 0])
    within(stats[:, 1], o["stats"][:, 1], e + 2.0 ** -24 * o["stats"][:, 1].abs(), what + " l")
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"], temperature=tau)
    dt = c["z"].dtype
    within(grad, o["grad"], UNIT[dt] * o["grad"].abs() + STEP[dt] + e[:, None] * o["terms"] + 1e-44, what + " gradient")
    return d, stats, grad


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,V,k,tau", [(1, 1, 1, 1.0), (3, 5, 5, 0.5), (2, 513, 1, 2.0), (5, 1000, 64, 1.0), (7, 8193, 33, 1.5),
                                       (1, 100003, 20, 1.0), (4, 40001, 1024, 2.0), (600, 257, 16, 1.0), (30, 20000, 100, 0.7),
                                       (2, 65536, 9, 1.0), (9, 65537, 1024, 0.6), (3, 131075, 50, 2.0)])
def test_loss_and_gradient(T, V, k, tau, dtype):
    run_case(make(T, V, k, dtype, T + V, repeat=k > V), tau, f"T={T} V={V} k={k} tau={tau} {dtype}")


@pytest.mark.parametrize("T,V", [(6, 300), (6, 30000), (520, 300), (6, 70001)])
def test_entries(T, V):
    """Repeated ids, dropped entries, rows that keep none (their logits are not read)."""
    c = make(T, V, 40, F16, 1, repeat=True)
    c["ids"][0, :] = c["ids"][0, 0]
    c["ids"][1, 1::2] = -1
    c["ids"][2, 3:] = torch.tensor([V, 2 ** 31 - 1, -2 ** 31] * 13)[:37].int()
    c["teacher"][2, 3:] = NAN  # of dropped entries
    c["ids"][3, :] = -1
    c["teacher"][4, :] = -INF
    c["teacher"][5, 4:] = -INF
    d, stats, grad = run_case(c, 1.5, f"entries {T} {V}")
    for row in (3, 4):
        c["z"][row] = NAN
    d = dev(c)
    loss2, stats2 = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"], temperature=1.5)
    grad2 = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats2, d["dloss"], temperature=1.5)
    assert torch.equal(stats, stats2) and torch.equal(grad, grad2)
    assert bool((loss2[3:5] == 0).all()) and bool((grad2[3:5] == 0).all()) and bool((stats2[3:5] == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("V", [700, 30000, 70001])
def test_masks(V, dtype):
    """Masked logits: -infinity and the type's lowest value, whole stretches of them."""
    low = torch.finfo(dtype).min
    c = make(5, V, 8, dtype, 2)
    print("masks", V, dtype, flush=True)
    for t, v in ((0, -INF), (1, low)):
        keep = c["z"][t, c["ids"][t].long()].clone()
        c["z"][t, V // 3:] = v
        c["z"][t, c["ids"][t].long()] = keep
    c["z"][2, :] = low  # all the same: uniform
    c["z"][3, :] = -INF
    c["z"][3, c["ids"][3].long()] = 1.0  # nothing but the teacher's entries
    d, stats, grad = run_case(c, 1.0, f"masks {V} {dtype}")
    assert bool((grad[0, V // 3:][d["z"][0, V // 3:] == -INF] == 0).all())


@pytest.mark.parametrize("V", [700, 30000, 70001])
def test_infinite_results(V):
    """A teacher's entry at a logit of -infinity: an infinite loss, a finite gradient.
    Rows without a finite logit, with NaN or +infinity: NaN, in that row only."""
    c = make(5, V, 8, F32, 3)
    print("infinite", V, flush=True)
    ids = c["ids"].long()
    c["z"][0, ids[0, 0]] = -INF
    c["z"][1, :] = -INF
    c["z"][2, 11] = NAN
    c["z"][3, 11] = INF
    d = dev(c)
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"])
    assert loss[0] == INF and bool(loss[1:4].isnan().all()) and bool(torch.isfinite(loss[4]))
    o = reference({n: t[[0, 4]] for n, t in c.items()}, 1.0)["grad"]
    within(grad[[0, 4]], o, 2.0 ** -18 * o.abs() + 2.0 ** -20 * o.abs().max(), "infinite")
    assert bool(grad[1:4].isnan().all())


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("T,V,pad,shift", [(4, 1001, 0, 1), (3, 30001, 7, 3), (515, 129, 2, 0), (3, 70003, 5, 1)])
def test_strides_and_in_place(T, V, pad, shift, dtype):
    c = make(T, V, 9, dtype, 4)
    print("strides", T, V, pad, shift, dtype, flush=True)
    d = dev(c)
    wide = torch.full((T + 2, V + pad), 3.0, dtype=dtype, device=DEV).flatten()
    rows = wide[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    rows.copy_(d["z"])
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
    loss2, stats2 = moe.moe_distill_forward(rows, d["ids"], d["teacher"])
    assert torch.allclose(loss, loss2, rtol=2.0 ** -18, atol=2.0 ** -18) and torch.equal(stats[:, 0], stats2[:, 0])
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"])
    out = torch.full_like(wide, 5.0)
    into = out[1 - shift % 2:][:T * (V + pad)].view(T, V + pad)[:, :V]
    moe.moe_distill_backward(rows, d["ids"], d["teacher"], stats, d["dloss"], out=into)
    assert torch.equal(into, grad)
    into.fill_(5.0)
    assert bool((out == 5.0).all())
    moe.moe_distill_backward(rows, d["ids"], d["teacher"], stats, d["dloss"], out=rows)
    assert torch.equal(rows, grad)
    rows.fill_(3.0)
    assert bool((wide == 3.0).all())


def test_gradient_is_the_derivative():
    """Against differences of the loss in 32 bits: step h, error h^2 and 2^-20 / h."""
    c = make(6, 400, 12, F32, 5)
    print("difference", flush=True)
    d = dev(c)
    v = torch.randn((6, 400), generator=torch.Generator().manual_seed(6)).to(DEV)
    h = 2.0 ** -6

    def loss(z):
        return moe.moe_distill_forward(z, d["ids"], d["teacher"], temperature=1.5)

    _, stats = loss(d["z"])
    grad = moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, torch.ones(6, device=DEV), temperature=1.5)
    slope = (grad.double() * v.double()).sum(1)
    diff = (loss(d["z"] + h * v)[0].double() - loss(d["z"] - h * v)[0].double()) / (2 * h)
    # |v| up to 4: the third derivative of log sum exp along v is below 4^3
    assert bool(((slope - diff).abs() <= 64 * h * h / 6 + 2.0 ** -20 * 8 / h).all()), (slope, diff)


def test_captured_and_on_another_stream():
    c = make(9, 30000, 12, BF16, 7)
    d = dev(c)
    print("graph", flush=True)

    def step():
        loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"])
        return loss, stats, moe.moe_distill_backward(d["z"], d["ids"], d["teacher"], stats, d["dloss"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    z = d["z"].clone()
    for i in range(3):
        d["z"].copy_(z * (1 + i))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), i
    s2 = torch.cuda.Stream()
    loss, stats = moe.moe_distill_forward(d["z"], d["ids"], d["teacher"], stream=s2)
    s2.synchronize()
    assert torch.equal(loss, outs[0]) and torch.equal(stats, outs[1])


def test_no_rows():
    z, ids, te = torch.empty((0, 50), device=DEV), torch.empty((0, 4), dtype=torch.int32, device=DEV), torch.empty((0, 4), device=DEV)
    loss, stats = moe.moe_distill_forward(z, ids, te)
    assert loss.shape == (0,) and stats.shape == (0, 2)
    assert moe.moe_distill_backward(z, ids, te, stats, loss).shape == (0, 50)


def test_refuses():
    c = dev(make(3, 50, 4, F16, 8))
    stats = torch.zeros((3, 2), device=DEV)
    for kw in (dict(ids=c["ids"].long()), dict(teacher=c["teacher"].half()), dict(ids=c["ids"][:2]), dict(logits=c["z"].t()),
               dict(logits=c["z"].double()), dict(logits=c["z"].cpu()), dict(teacher=c["teacher"][:, :2])):
        with pytest.raises(ValueError):
            moe.moe_distill_forward(**{**dict(logits=c["z"], ids=c["ids"], teacher=c["teacher"]), **kw})
    for tau in (0.0, -1.0, INF, NAN):
        with pytest.raises(moe.MoeError):
            moe.moe_distill_forward(c["z"], c["ids"], c["teacher"], temperature=tau)
    with pytest.raises(ValueError):
        moe.moe_distill_backward(c["z"], c["ids"], c["teacher"], stats, c["dloss"].half())
    with pytest.raises(ValueError):
        moe.moe_distill_backward(c["z"], c["ids"], c["teacher"], stats[:, :1], c["dloss"])
