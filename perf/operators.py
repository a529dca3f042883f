"""Cases that measure the layer's training and serving operators: the expert
dispatch and combine with their gradients, the router's gradient, and the
low-rank adapters with theirs.

Where `own` is false, run() computes an operator in its plain form
(elementary torch operations in 32 bits, rounded once at the end); where it is
true, run() calls the library's entry points on the same inputs.  exact()
computes the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases.  Sizes are those of the layers this repository names (6144 wide with
# 256 experts top-8, 2048 wide with 256 experts top-8) or generic ragged ones.
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step, its row laid out for eight experts: latency
        dict(name="dispatch_token", op="dispatch", way="fwd", T=1, H=6144, E=256, k=8, dtype="f16", align=1, zipf=0.0, drop=0.0),
        # a prompt chunk with a skewed router
        dict(name="dispatch_prompt", op="dispatch", way="fwd", T=2048, H=6144, E=256, k=8, dtype="f16", align=1, zipf=1.1, drop=0.0),
        # gradient of the dispatch: ragged sizes, slots dropped by top-p, groups padded to whole tiles
        dict(name="dispatch_grad_ragged", op="dispatch", way="bwd", T=1501, H=2056, E=100, k=6, dtype="bf16", align=16, zipf=0.0, drop=0.3),
        # eight concurrent decode tokens, with the shared expert's rows added
        dict(name="combine_tokens", op="combine", way="fwd", T=8, H=6144, E=256, k=8, dtype="f16", align=1, zipf=0.0, drop=0.0, add=True),
        # the same for a prompt chunk
        dict(name="combine_prompt", op="combine", way="fwd", T=2048, H=6144, E=256, k=8, dtype="f16", align=1, zipf=1.1, drop=0.0, add=True),
        # gradient of the combine in a training step on the smaller layer
        dict(name="combine_grad", op="combine", way="bwd", T=4096, H=2048, E=256, k=8, dtype="bf16", align=64, zipf=1.1, drop=0.0, add=False),
        # gradient of the router for a short ragged batch
        dict(name="route_grad_short", op="route", way="bwd", T=45, H=2048, E=256, k=8, dtype="bf16", align=1, zipf=0.0, drop=0.3),
        # gradient of the router in a training step on the large layer
        dict(name="route_grad", op="route", way="bwd", T=2048, H=6144, E=256, k=8, dtype="f16", align=1, zipf=1.1, drop=0.0),
        # one decode token of one request among 64 loaded adapters: latency
        dict(name="adapter_token", op="adapter", way="fwd", T=1, K=6144, N=6144, n=64, R=16, dtype="f16", mixed=False, none=0.0, add=True, save=False),
        # a decode batch: 48 requests over 32 adapters of mixed ranks, some requests without one
        dict(name="adapter_requests", op="adapter", way="fwd", T=48, K=6144, N=2048, n=32, R=64, dtype="f16", mixed=True, none=0.2, add=True, save=False),
        # ragged prompts of eight requests, or the forward pass of a training step
        dict(name="adapter_prompts", op="adapter", way="fwd", T=1801, K=6144, N=6144, n=8, R=64, dtype="bf16", mixed=True, none=0.0, add=True, save=True),
        # gradients of four adapters in one training step
        dict(name="adapter_grad", op="adapter", way="bwd", T=2048, K=6144, N=6144, n=4, R=16, dtype="f16", mixed=False, none=0.0),
    ]


_FORMS = (("dispatch", "fwd"), ("dispatch", "bwd"), ("combine", "fwd"), ("combine", "bwd"), ("route", "bwd"),
          ("adapter", "fwd"), ("adapter", "bwd"))


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo=64, hi=6144):
    w = max(lo, _log_int(rng, lo // 8, hi // 8) * 8)
    return w + 8 if w == 3072 else w


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    op, way = rng.choice(_FORMS)
    T = _log_int(rng, 1, 8192)
    if op == "adapter":
        c = dict(op=op, way=way, T=T, K=_width(rng), N=_width(rng), n=_log_int(rng, 1, 64), R=8 * rng.randint(1, 16),
                 dtype=rng.choice(("f16", "bf16")), mixed=rng.random() < 0.5, none=rng.choice((0.0, 0.2)) if T >= 32 else 0.0)
        if way == "fwd":
            c.update(add=rng.random() < 0.5, save=rng.random() < 0.5)
    else:
        E = _log_int(rng, 2, 512)
        c = dict(op=op, way=way, T=T, H=_width(rng), E=E, k=rng.randint(2 if op == "route" else 1, min(E, 16)),  # one slot's weight is 1: no gradient
                 dtype=rng.choice(("f16", "bf16") if op == "route" else ("f16", "bf16", "f32")),
                 align=1 if op == "route" else rng.choice((1, 1, 16, 64)), zipf=rng.choice((0.0, 1.1)), drop=rng.choice((0.0, 0.3)))
        if op == "combine":
            c["add"] = way == "fwd" and rng.random() < 0.5
    most = max(_cost(x) for x in listed() if (x["op"] == "adapter") == (op == "adapter"))
    while _cost(c) > most and c["T"] > 1:
        c["T"] = c["T"] * 3 // 4
    return c


def _rows(T, k, E, align):
    """Rows of the expert-sorted buffers: every slot, and the most that padding each group to `align` can add."""
    n = T * k
    if align > 1:
        n = -(-(n + min(E, n) * (align - 1)) // align) * align
    return n


def work(case):
    c, T = case, case["T"]
    b = SIZE[c["dtype"]]
    if c["op"] == "adapter":
        K, N, n, R = c["K"], c["N"], min(c["n"], c["T"]), c["R"]
        used = n * R * (0.55 if c["mixed"] else 1.0)  # ranks of a mixed set average just over half of the largest
        r = used / n
        if c["way"] == "fwd":
            return {"bytes": T * (K + N * (2 if c["add"] else 1)) * b + used * (K + N) * b + 4 * T * (1 + R * c["save"]),
                    "flops": 2 * T * r * (K + N)}
        return {"bytes": T * (2 * K + N) * b + used * (K + N) * b + 4 * c["n"] * R * (K + N) + 4 * T * R,
                "flops": 2 * T * r * 2 * (K + N)}
    H, k, E = c["H"], c["k"], c["E"]
    kept = T * (k - c["drop"] * (k - 1) / 2)
    rows = _rows(T, k, E, c["align"])
    if c["op"] == "dispatch" and c["way"] == "fwd":
        return {"bytes": T * H * b + rows * H * b + 4 * (2 * T * k + rows + E), "flops": 0}
    if c["op"] == "dispatch":
        return {"bytes": kept * H * b + T * H * b + 4 * T * k, "flops": kept * H}
    if c["op"] == "combine" and c["way"] == "fwd":
        return {"bytes": kept * H * b + T * H * b * (2 if c["add"] else 1) + 8 * T * k, "flops": 2 * kept * H}
    if c["op"] == "combine":
        return {"bytes": kept * H * b + T * H * b + rows * H * b + 12 * T * k, "flops": 3 * kept * H}
    return {"bytes": 2 * T * H * b + 2 * 4 * E * H + 8 * T * k, "flops": 6 * kept * H}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _order(idx, E, align):
    """(offsets, pairs, pos): the slots of idx [T][k] sorted by expert, stably; negative entries are dropped slots."""
    T, k = idx.shape
    rows = _rows(T, k, E, align)
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, E)
    skey, perm = torch.sort(key, stable=True)
    first = torch.searchsorted(skey, torch.arange(E + 1, device=idx.device))
    count = first[1:] - first[:-1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.cumsum(-(-count // align) * align, 0)
    kept = skey < E
    e = skey.clamp(max=E - 1)
    row = torch.where(kept, offsets[e] + torch.arange(T * k, device=idx.device) - first[e], rows)
    pairs = torch.full((rows + 1,), -1, dtype=torch.int32, device=idx.device)
    pairs[row] = torch.where(kept, perm, -1).int()
    pos = torch.empty(T * k, dtype=torch.int32, device=idx.device)
    pos[perm] = torch.where(kept, row, -1).int()
    return offsets.int(), pairs[:rows].clone(), pos.reshape(T, k)


def _drop(idx, share, g):
    """Slots past a random prefix dropped (-1), as top-p leaves them."""
    T, k = idx.shape
    keep = torch.where(torch.rand((T, 1), device=DEV, generator=g) < share, torch.randint(1, k + 1, (T, 1), device=DEV, generator=g), k)
    return torch.where(torch.arange(k, device=DEV) < keep, idx, -1).int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, device=DEV, generator=g) * std).to(dtype)

    T = c["T"]
    s = dict(c=dict(c))
    if c["op"] == "adapter":
        K, N, n, R = c["K"], c["N"], c["n"], c["R"]
        if T >= 16 * n or c["way"] == "bwd":  # whole prompts: every request's rows are consecutive
            cut = torch.sort(torch.randint(0, T + 1, (n - 1,), device=DEV, generator=g))[0] if n > 1 else torch.zeros(0, device=DEV, dtype=torch.int64)
            ids = torch.searchsorted(cut, torch.arange(T, device=DEV), right=True)
        else:  # a decode batch: requests in order of arrival
            ids = torch.randint(0, n, (T,), device=DEV, generator=g)
        ids = torch.where(torch.rand(T, device=DEV, generator=g) < c["none"], -1, ids).int()
        s.update(x=randn(T, K), a=randn(n, R, K, std=K ** -0.5), b=randn(n, N, R, std=0.05), ids=ids,
                 scale=torch.rand(n, device=DEV, generator=g) + 0.5, ranks=None)
        if c["mixed"]:
            s["ranks"] = (torch.randint(1, max(2, R // 8 + 1), (n,), device=DEV, generator=g) * 8).clamp(max=R).int()
        if c["way"] == "fwd":
            s["add"] = randn(T, N) if c["add"] else None
        else:
            s["dy"] = randn(T, N)  # loss-scaled, as 16-bit training keeps gradients
            s["u"] = _plain_u(s)
            s["order"] = dict(zip(("offsets", "pairs", "pos"), _order(ids[:, None], n, 1)))
        return s
    H, E, k = c["H"], c["E"], c["k"]
    bias = None
    if c["zipf"]:
        rank = torch.randperm(E, device=DEV, generator=g).float() + 1
        bias = -c["zipf"] * torch.log(rank)
    if c["op"] == "route":
        x, wr = randn(T, H), randn(E, H, std=0.02, dtype=torch.float32)
        z = x.double() @ wr.double().t() + (0 if bias is None else bias.double())
        idx = _drop(torch.topk(z, k, dim=1)[1].int(), c["drop"], g)
        offsets, pairs, pos = _order(idx, E, c["align"])
        s.update(x=x, wr=wr, bias=bias, idx=idx, dw=randn(T, k, dtype=torch.float32), offsets=offsets, pairs=pairs, pos=pos)
        return s
    z = torch.randn((T, E), device=DEV, generator=g) * 1.5 + (0 if bias is None else bias)
    zk, idx = torch.topk(z, k, dim=1)
    idx = _drop(idx.int(), c["drop"], g)
    w = torch.sigmoid(zk) * (idx >= 0)
    w = (w / w.sum(1, keepdim=True)).float()
    if c["op"] == "dispatch" and c["way"] == "fwd":
        s.update(x=randn(T, H), idx=idx)
        return s
    offsets, pairs, pos = _order(idx, E, c["align"])
    rows = pairs.numel()
    o = randn(rows, H)
    o[pairs < 0] = 0
    s.update(w=w, pairs=pairs, pos=pos, o=o)
    if c["op"] == "combine" and c["way"] == "fwd":
        s["add"] = randn(T, H) if c["add"] else None
    if c["op"] == "combine" and c["way"] == "bwd":
        s["dy"] = randn(T, H)
    return s


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _mask(s):
    """[T][n][R]: true where token t uses adapter a and r is below the adapter's rank."""
    n, R = s["a"].shape[:2]
    m = (s["ids"][:, None] == torch.arange(n, device=DEV))[:, :, None]
    if s["ranks"] is not None:
        m = m & (torch.arange(R, device=DEV) < s["ranks"][:, None])
    return m.expand(-1, n, R)


def _plain_u(s):
    n, R, K = s["a"].shape
    u = (s["x"].float() @ s["a"].float().reshape(n * R, K).t()).reshape(-1, n, R)
    return torch.where(_mask(s), u, 0.0).sum(1)


def _plain_adapter(s):
    a, b, x = s["a"], s["b"], s["x"].float()
    (n, R, K), T, N = a.shape, x.shape[0], b.shape[1]
    if T <= n:  # few tokens: only the adapters that they use
        i = s["ids"].long().clamp(min=0)
        ok = (s["ids"] >= 0)[:, None]
        if s["ranks"] is not None:
            ok = ok & (torch.arange(R, device=DEV) < s["ranks"][i][:, None])
        u = torch.where(ok, (a[i].float() @ x[:, :, None])[:, :, 0], 0.0)
        y = (b[i].float() @ (u * s["scale"][i][:, None])[:, :, None])[:, :, 0]
    else:  # all adapters at once, masked
        m = _mask(s)
        u3 = torch.where(m, (x @ a.float().reshape(n * R, K).t()).reshape(T, n, R), 0.0)
        u = u3.sum(1)
        y = (u3 * s["scale"][:, None]).reshape(T, n * R) @ b.float().permute(0, 2, 1).reshape(n * R, N)
    y = y if s["add"] is None else y + s["add"].float()
    y = y.to(s["x"].dtype)
    return {"y": y, "u": u} if s["c"]["save"] else y


def _plain_adapter_grad(s):
    a, b, x, dy = s["a"].float(), s["b"].float(), s["x"].float(), s["dy"].float()
    (n, R, K), T, N = a.shape, x.shape[0], b.shape[1]
    m = _mask(s)
    bt = b.permute(0, 2, 1).reshape(n * R, N)
    v = torch.where(m, (dy @ bt.t()).reshape(T, n, R) * s["scale"][:, None], 0.0).reshape(T, n * R)
    us = (torch.where(m, s["u"][:, None, :], 0.0) * s["scale"][:, None]).reshape(T, n * R)
    dx = (v @ a.reshape(n * R, K)).to(s["x"].dtype)
    da = (v.t() @ x).reshape(n, R, K)
    db = (us.t() @ dy).reshape(n, R, N).permute(0, 2, 1).contiguous()
    return {"dx": dx, "da": da, "db": db}


def _plain(s):
    c = s["c"]
    if c["op"] == "adapter":
        return _plain_adapter(s) if c["way"] == "fwd" else _plain_adapter_grad(s)
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    dt = DT[c["dtype"]]
    if c["op"] == "dispatch" and c["way"] == "fwd":
        offsets, pairs, pos = _order(s["idx"], E, c["align"])
        xs = torch.where((pairs >= 0)[:, None], s["x"][pairs.clamp(min=0).long() // k], torch.zeros((), dtype=dt, device=DEV))
        return {"xs": xs, "offsets": offsets, "pairs": pairs, "pos": pos}
    if c["op"] == "route":
        idx, ok = s["idx"].clamp(min=0).long(), s["idx"] >= 0
        z = s["x"].float() @ s["wr"].t()
        z = z if s["bias"] is None else z + s["bias"]
        z = torch.gather(z, 1, idx)
        sg = torch.where(ok, 1 / (1 + torch.exp(-z)), 0.0)
        w = sg / sg.sum(1, keepdim=True)
        dz = w / (1 + torch.exp(z)) * (s["dw"] - (s["dw"] * w).sum(1, keepdim=True))
        full = torch.zeros((T, E), device=DEV).scatter_add_(1, idx, torch.where(ok, dz, 0.0))
        return {"dx": (full @ s["wr"]).to(dt), "dwr": full.t() @ s["x"].float(), "dbias": full.sum(0)}
    ok, at = (s["pos"] >= 0), s["pos"].clamp(min=0).long()
    if c["way"] == "bwd" and c["op"] == "combine":
        t = s["pairs"].clamp(min=0).long()
        kept = (s["pairs"] >= 0)[:, None]
        dyr = s["dy"].float()[t // k]
        do = torch.where(kept, s["w"].reshape(-1)[t][:, None] * dyr, 0.0).to(dt)
        dots = (dyr * s["o"].float()).sum(1)
        return {"do": do, "dw": torch.where(ok, dots[at], 0.0)}
    o = torch.where(ok[:, :, None], s["o"].float()[at], 0.0)
    if c["op"] == "dispatch":
        return o.sum(1).to(dt)
    y = (s["w"][:, :, None] * o).sum(1)
    return (y if s["add"] is None else y + s["add"].float()).to(dt)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import quantized_moe_expert_02_amd as moe
    c = s["c"]
    if c["op"] == "dispatch":
        if c["way"] == "fwd":
            return moe.moe_dispatch(s["x"], s["idx"], c["E"], align=c["align"])
        return moe.moe_dispatch_backward(s["o"], s["pos"])
    if c["op"] == "combine":
        if c["way"] == "fwd":
            return moe.moe_combine(s["o"], s["w"], s["pos"], add=s["add"])
        do, dw = moe.moe_combine_backward(s["dy"], s["o"], s["w"], s["pos"], s["pairs"])
        return {"do": do, "dw": dw}
    if c["op"] == "route":
        dx, dwr, dbias = moe.moe_route_backward(s["x"], s["wr"], s["bias"], s["idx"], s["dw"], s["offsets"], s["pairs"])
        return {"dx": dx, "dwr": dwr, "dbias": dbias}
    if c["way"] == "fwd":
        if c["save"]:
            y, u = moe.moe_adapter_forward(s["x"], s["a"], s["b"], s["ids"], s["scale"], ranks=s["ranks"], add=s["add"], save_u=True)
            return {"y": y, "u": u}
        return moe.moe_adapter_forward(s["x"], s["a"], s["b"], s["ids"], s["scale"], ranks=s["ranks"], add=s["add"])
    dx, da, db = moe.moe_adapter_backward(s["dy"], s["x"], s["u"], s["a"], s["b"], s["ids"], s["scale"], ranks=s["ranks"], order=s["order"])
    return {"dx": dx, "da": da, "db": db}


# ---------------------------------------------------------------------------
# 64-bit values, group by group from the definitions.
# ---------------------------------------------------------------------------
def exact(case, seed):
    def adapter(s):
        c = s["c"]
        x, ids, R = s["x"].double(), s["ids"], c["R"]
        T, K, N = c["T"], c["K"], c["N"]
        f64 = dict(dtype=torch.float64, device=DEV)
        u = torch.zeros((T, R), **f64)
        if c["way"] == "fwd":
            y = torch.zeros((T, N), **f64) if s["add"] is None else s["add"].double()
        else:
            dx, da, db = torch.zeros((T, K), **f64), torch.zeros((c["n"], R, K), **f64), torch.zeros((c["n"], N, R), **f64)
            dy = s["dy"].double()
        for i in range(c["n"]):
            rows = torch.nonzero(ids == i)[:, 0]
            if not rows.numel():
                continue
            r = R if s["ranks"] is None else int(s["ranks"][i])
            a, b, sc = s["a"][i, :r].double(), s["b"][i, :, :r].double(), float(s["scale"][i])
            if c["way"] == "fwd":
                ui = x[rows] @ a.t()
                u[rows, :r] = ui
                y[rows] += sc * (ui @ b.t())
            else:
                v = sc * (dy[rows] @ b)
                dx[rows] = v @ a
                da[i, :r] = v.t() @ x[rows]
                db[i, :, :r] = sc * (dy[rows].t() @ s["u"][rows, :r].double())
        if c["way"] == "fwd":
            return {"y": y, "u": u} if c["save"] else y
        return {"dx": dx, "da": da, "db": db}

    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "adapter":
        return adapter(s)
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    f64 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "dispatch" and c["way"] == "fwd":
        rows = _rows(T, k, E, c["align"])
        xs, at = torch.zeros((rows, H), **f64), 0
        for e in range(E):
            t = torch.nonzero((s["idx"] == e).any(1))[:, 0]
            xs[at:at + t.numel()] = s["x"][t].double()
            at += -(-t.numel() // c["align"]) * c["align"]
        return {"xs": xs, "offsets": None, "pairs": None, "pos": None}
    if c["op"] == "route":
        x, wr = s["x"].double(), s["wr"].double()
        dx, dwr, db = torch.zeros((T, H), **f64), torch.zeros((E, H), **f64), torch.zeros(E, **f64)
        sg, dz = torch.zeros((T, k), **f64), torch.zeros((T, k), **f64)
        ok = s["idx"] >= 0
        for j in range(k):
            e = s["idx"][:, j].clamp(min=0).long()
            z = (x * wr[e]).sum(1) + (0 if s["bias"] is None else s["bias"].double()[e])
            sg[:, j] = torch.sigmoid(z) * ok[:, j]
        S = sg.sum(1, keepdim=True)
        # w_j = s_j / S, so dL/ds_j = (dw_j - sum_i dw_i w_i) / S and ds_j/dz_j = s_j (1 - s_j)
        mean = (s["dw"].double() * sg / S).sum(1, keepdim=True)
        dz = (s["dw"].double() - mean) / S * sg * (1 - sg)
        for j in range(k):
            e = s["idx"][:, j].clamp(min=0).long()
            dx += dz[:, j:j + 1] * wr[e]
            dwr.index_add_(0, e, dz[:, j:j + 1] * x)
            db.index_add_(0, e, dz[:, j])
        return {"dx": dx, "dwr": dwr, "dbias": db}
    if c["op"] == "combine" and c["way"] == "bwd":
        do, dw = torch.zeros(s["o"].shape, **f64), torch.zeros((T, k), **f64)
        for j in range(k):
            t = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
            at = s["pos"][t, j].long()
            do[at] = s["w"][t, j].double()[:, None] * s["dy"][t].double()
            dw[t, j] = (s["dy"][t].double() * s["o"][at].double()).sum(1)
        return {"do": do, "dw": dw}
    y = torch.zeros((T, H), **f64)
    if c["op"] == "combine" and s["add"] is not None:
        y += s["add"].double()
    for j in range(k):
        t = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
        row = s["o"][s["pos"][t, j].long()].double()
        y[t] += row if c["op"] == "dispatch" else s["w"][t, j].double()[:, None] * row
    return y
