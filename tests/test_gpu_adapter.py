"""Low-rank adapters on the GPU, forward and backward, against 64-bit loops.

Tolerances as in test_gpu_dispatch.py: one rounding of the output's type, and
4 sqrt(n) 2^-24 of the magnitudes summed for sums of n terms in fp32.  A factor
of a second product (u in the forward pass, v in the backward) may be carried
to 2^-16 of itself where the output has 16 bits, and to 2^-21 of the largest
factor in the sum where it is a weight gradient in fp32.
"""
import pytest
import torch

import quantized_moe_expert_02_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _log(*a):
    print(*a, flush=True)


def make(T, K, N, n, R, dtype, mixed, none, seed, runs=False):
    g = torch.Generator()
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    c = dict(x=r(T, K).to(dtype), a=(r(n, R, K) / K ** 0.5).to(dtype), b=(r(n, N, R) * 0.1).to(dtype),
             scale=torch.rand(n, generator=g) + 0.5, ranks=None, dy=r(T, N).to(dtype), add=r(T, N).to(dtype),
             add_x=r(T, K).to(dtype))
    ids = torch.randint(0, n, (T,), generator=g)
    if runs:
        ids = ids.sort()[0]
    ids[torch.rand(T, generator=g) < none] = -1
    c["ids"] = ids.int()
    if mixed:
        c["ranks"] = torch.randint(0, R + 1, (n,), generator=g).int()
    return c


def reference(c, u=None):
    """y, u, dx, da, db and the magnitudes of their sums, adapter by adapter in 64 bits."""
    x, dy = c["x"].double(), c["dy"].double()
    (T, K), (n, N, R) = x.shape, c["b"].shape
    z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    o = dict(y=z(T, N), u=z(T, R), dx=z(T, K), da=z(n, R, K), db=z(n, N, R))
    m = {k: v.clone() for k, v in o.items()}
    for i in range(n):
        rows = torch.nonzero(c["ids"] == i)[:, 0]
        r = R if c["ranks"] is None else int(c["ranks"][i])
        a, b, s = c["a"][i, :r].double(), c["b"][i, :, :r].double(), float(c["scale"][i])
        o["u"][rows, :r] = x[rows] @ a.t()
        m["u"][rows, :r] = x[rows].abs() @ a.t().abs()
        o["y"][rows] = s * o["u"][rows, :r] @ b.t()
        m["y"][rows] = s * m["u"][rows, :r] @ b.t().abs()
        v, mv = s * dy[rows] @ b, s * dy[rows].abs() @ b.abs()
        o["dx"][rows], m["dx"][rows] = v @ a, mv @ a.abs()
        o["da"][i, :r], m["da"][i, :r] = v.t() @ x[rows], mv.t() @ x[rows].abs()
        w = (o["u"] if u is None else u.double())[rows, :r]
        o["db"][i, :, :r], m["db"][i, :, :r] = s * dy[rows].t() @ w, s * dy[rows].t().abs() @ w.abs()
        if rows.numel() and r:
            m.setdefault("da_top", z(n, R, K))[i, :r] = v.abs().max() * x[rows].abs().sum(0)
            m.setdefault("db_top", z(n, N, R))[i, :, :r] = s * w.abs().max() * dy[rows].abs().sum(0)[:, None]
    return o, m


def check(got, ref, tol, what):
    g = got.detach().double().cpu()
    assert g.shape == ref.shape and bool(torch.isfinite(g).all()), what
    err = (g - ref).abs()
    bound = UNIT[got.dtype] * ref.abs() + 2.0 ** -25 + tol
    worst = float((err / bound).max()) if err.numel() else 0.0
    _log(what, "worst error / tolerance %.3f" % worst)
    assert worst <= 1.0, (what, worst)


def to_dev(c):
    return {k: None if v is None else v.to(DEV) for k, v in c.items()}


CASES = [  # T, K, N, n, R, mixed, none, runs
    (1, 6144, 6144, 64, 16, False, 0.0, False), (1, 64, 8, 1, 8, False, 1.0, False), (0, 64, 64, 3, 8, False, 0.0, False),
    (7, 520, 264, 5, 24, True, 0.2, False), (48, 2048, 520, 32, 64, True, 0.2, False), (64, 136, 1000, 2, 128, False, 0.0, False),
    (65, 72, 40, 3, 40, True, 0.1, False), (300, 264, 328, 4, 16, False, 0.0, True), (513, 1032, 200, 40, 56, True, 0.3, False),
    (1000, 2048, 1024, 6, 64, True, 0.0, True), (700, 512, 264, 1024, 8, False, 0.1, False), (33, 8, 8, 1, 120, False, 0.0, True)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,N,n,R,mixed,none,runs", CASES)
def test_adapter(dtype, T, K, N, n, R, mixed, none, runs):
    _log("adapter", dtype, T, K, N, n, R, mixed, none, runs)
    c = make(T, K, N, n, R, dtype, mixed, none, 100 + T, runs)
    if c["ranks"] is not None:  # what lies past an adapter's rank is never used
        for i, r in enumerate(c["ranks"].tolist()):
            c["a"][i, r:], c["b"][i, :, r:] = float("nan"), float("nan")
    d = to_dev(c)
    args = [d[k] for k in ("x", "a", "b", "ids", "scale")]
    y, u = moe.moe_adapter_forward(*args, ranks=d["ranks"], save_u=True)
    ref, mag = reference(c, u.cpu())
    f = lambda k: (4 * k ** 0.5 + 2) * 2.0 ** -24  # noqa: E731
    check(u, ref["u"], f(K) * mag["u"], "u")
    ty = (f(K) + f(R) + 2.0 ** -16) * mag["y"]
    check(y, ref["y"], ty, "y")
    want = ref["y"] + c["add"].double()
    ta = ty + 2.0 ** -23 * c["add"].double().abs()
    ya = moe.moe_adapter_forward(*args, ranks=d["ranks"], add=d["add"])
    check(ya, want, ta, "y with add")
    order = moe.moe_sort(d["ids"][:, None].contiguous(), n)
    assert torch.equal(ya, moe.moe_adapter_forward(*args, ranks=d["ranks"], add=d["add"], order=order))
    moe.moe_adapter_forward(*args, ranks=d["ranks"], add=d["add"], out=d["add"])
    assert torch.equal(ya, d["add"])
    td = (f(N) + f(R) + 2.0 ** -16) * mag["dx"]
    none_top = torch.zeros(1, dtype=torch.float64)
    tops = [mag.get(k, none_top) * 2.0 ** -21 for k in ("da_top", "db_top")]
    for o in (order, None):
        dx, da, db = moe.moe_adapter_backward(d["dy"], d["x"], u, *args[1:], ranks=d["ranks"], order=o)
        check(dx, ref["dx"], td, "dx")
        check(da, ref["da"], (f(N) + f(max(T, 1)) + 2.0 ** -22) * mag["da"] + tops[0], "da")
        check(db, ref["db"], (f(max(T, 1)) + 2.0 ** -22) * mag["db"] + tops[1], "db")
    dxa, da2, db2 = moe.moe_adapter_backward(d["dy"], d["x"], u, *args[1:], ranks=d["ranks"], order=order, add=d["add_x"])
    check(dxa, ref["dx"] + c["add_x"].double(), td + 2.0 ** -23 * c["add_x"].double().abs(), "dx with add")
    skip, da3, db3 = moe.moe_adapter_backward(d["dy"], d["x"], u, *args[1:], ranks=d["ranks"], order=order, need_dx=False)
    assert skip is None
    for p, q in ((da, da2), (da, da3), (db, db2), (db, db3)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,N,n,R,mixed,none,runs", [
    (4500, 264, 136, 5, 24, True, 0.1, False), (4200, 136, 264, 3, 64, True, 0.0, True), (4097, 72, 80, 2, 128, False, 0.2, False),
    (1500, 264, 136, 1, 16, False, 0.0, False), (1500, 264, 136, 1, 72, False, 0.0, False), (3000, 64, 64, 70, 32, True, 0.3, True),
    (5000, 40, 520, 1, 8, False, 0.0, True), (4096, 72, 64, 64, 8, False, 0.3, False), (4095, 8, 72, 63, 24, True, 0.0, True)])
def test_adapter_of_many_rows(dtype, T, K, N, n, R, mixed, none, runs):
    """Adapters whose gradients several workgroups sum, and row counts past the wide tiles' threshold."""
    test_adapter(dtype, T, K, N, n, R, mixed, none, runs)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,N,n,R,mixed,none,runs", [
    (3, 20488, 136, 2, 16, False, 0.0, False), (20, 8200, 72, 4, 32, True, 0.2, False), (5, 8200, 264, 3, 64, True, 0.2, False),
    (60, 136, 6144, 60, 8, False, 0.1, False), (64, 1032, 1416, 64, 40, True, 0.3, False), (17, 264, 2048, 1, 8, False, 0.0, False)])
def test_adapter_of_few_rows(dtype, T, K, N, n, R, mixed, none, runs):
    """Both sides of the rule for one launch or two, at each number of rank tiles."""
    test_adapter(dtype, T, K, N, n, R, mixed, none, runs)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [3, 200])
def test_rows_of_wider_buffers(dtype, T):
    K, N, n, R = 264, 136, 3, 16
    _log("adapter strides", dtype, T)
    c = to_dev(make(T, K, N, n, R, dtype, False, 0.1, 7))
    wide = {k: torch.full((T, w + 40), 9.0, dtype=dtype, device=DEV) for k, w in (("x", K), ("dy", N), ("add", N), ("y", N))}
    view = {k: wide[k][:, 16:16 + (K if k == "x" else N)] for k in wide}
    for k in ("x", "dy", "add"):
        view[k].copy_(c[k])
    args = [c[k] for k in ("a", "b", "ids", "scale")]
    y, u = moe.moe_adapter_forward(c["x"], *args, add=c["add"], save_u=True)
    out = moe.moe_adapter_forward(view["x"], *args, add=view["add"], out=view["y"])
    assert torch.equal(out, y)
    assert bool((wide["y"][:, :16] == 9).all()) and bool((wide["y"][:, 16 + N:] == 9).all())
    for p, q in zip(moe.moe_adapter_backward(view["dy"], view["x"], u, *args), moe.moe_adapter_backward(c["dy"], c["x"], u, *args)):
        assert torch.equal(p, q)


def test_ids_outside_the_set_have_no_adapter():
    T, K, N, n, R = 70, 64, 72, 4, 8
    _log("adapter ids")
    c = to_dev(make(T, K, N, n, R, F16, False, 0.0, 8))
    odd = torch.tensor([-1, -2 ** 31, 4, 5, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    for t in (5, 70):
        ids = c["ids"][:t].clone()
        ids[:5] = odd
        clean = torch.where((ids >= 0) & (ids < n), ids, -1)
        ranks = torch.tensor([-3, 100, 8, 3], dtype=torch.int32, device=DEV)
        a = [c["a"], c["b"]]
        y, u = moe.moe_adapter_forward(c["x"][:t], *a, ids, c["scale"], ranks=ranks, add=c["add"][:t], save_u=True)
        y2, u2 = moe.moe_adapter_forward(c["x"][:t], *a, clean, c["scale"], ranks=ranks.clamp(0, R), add=c["add"][:t], save_u=True)
        assert torch.equal(y, y2) and torch.equal(u, u2)
        assert torch.equal(y[:5], c["add"][:5]) and bool((u[:5] == 0).all())
        g = moe.moe_adapter_backward(c["dy"][:t], c["x"][:t], u, *a, ids, c["scale"], ranks=ranks)
        g2 = moe.moe_adapter_backward(c["dy"][:t], c["x"][:t], u, *a, clean, c["scale"], ranks=ranks.clamp(0, R))
        for p, q in zip(g, g2):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype,big,small", [(F16, 2.0 ** 14, 2.0 ** -14), (BF16, 2.0 ** 60, 2.0 ** -60)])
@pytest.mark.parametrize("T", [2, 130])
def test_wide_range_of_sizes(dtype, big, small, T):
    """u and v past the 16-bit type's range, and rows of very different sizes side by side."""
    K, N, n, R = 128, 64, 2, 16
    _log("adapter range", dtype, T)
    c = make(T, K, N, n, R, dtype, False, 0.0, 9, runs=True)
    c["x"][::2] = (c["x"][::2].float() * big / 4).to(dtype)
    c["b"] = (c["b"].float() * small).to(dtype)
    c["a"] = (c["a"].float() * 8).to(dtype)
    c["dy"][1::2] = (c["dy"][1::2].float() * small * 16).to(dtype)
    d = to_dev(c)
    args = [d[k] for k in ("a", "b", "ids", "scale")]
    y, u = moe.moe_adapter_forward(d["x"], *args, save_u=True)
    ref, mag = reference(c, u.cpu())
    f = lambda k: (4 * k ** 0.5 + 2) * 2.0 ** -24  # noqa: E731
    check(u, ref["u"], f(K) * mag["u"], "u")
    check(y, ref["y"], (f(K) + f(R) + 2.0 ** -16) * mag["y"], "y")
    dx, da, db = moe.moe_adapter_backward(d["dy"], d["x"], u, *args)
    check(dx, ref["dx"], (f(N) + f(R) + 2.0 ** -16) * mag["dx"], "dx")
    check(da, ref["da"], (f(N) + f(T) + 2.0 ** -22) * mag["da"] + 2.0 ** -21 * mag["da_top"], "da")
    check(db, ref["db"], (f(T) + 2.0 ** -22) * mag["db"] + 2.0 ** -21 * mag["db_top"], "db")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinities_and_nans_stay_in_their_rows(dtype):
    T, K, N, n, R = 80, 64, 64, 2, 8
    _log("adapter non-finite", dtype)
    c = make(T, K, N, n, R, dtype, False, 0.0, 10)
    clean = to_dev(c)
    args = [clean[k] for k in ("a", "b", "ids", "scale")]
    y0, u0 = moe.moe_adapter_forward(clean["x"], *args, save_u=True)
    x, dy = clean["x"].clone(), clean["dy"].clone()
    x[3, 5], x[9, 0] = float("nan"), float("inf")
    y, u = moe.moe_adapter_forward(x, *args, save_u=True)
    other = [t for t in range(T) if t not in (3, 9)]
    assert torch.equal(y[other], y0[other]) and torch.equal(u[other], u0[other])
    assert bool(y[3].isnan().all()) and not bool(y[9].isfinite().any()) and not bool(u[9].isfinite().any())
    dy[4, 2], dy[8, 1] = float("inf"), float("nan")
    g0 = moe.moe_adapter_backward(clean["dy"], clean["x"], u0, *args)
    g = moe.moe_adapter_backward(dy, clean["x"], u0, *args)
    other = [t for t in range(T) if t not in (4, 8)]
    assert torch.equal(g[0][other], g0[0][other])
    assert not bool(g[0][4].isfinite().any()) and bool(g[0][8].isnan().all())
    for i in range(n):  # an adapter that none of these rows uses keeps its gradients
        hit = bool((clean["ids"][[4, 8]] == i).any())
        assert bool(g[1][i].isfinite().all()) != hit
        if not hit:
            assert torch.equal(g[1][i], g0[1][i]) and torch.equal(g[2][i], g0[2][i])


def test_gradients_against_differences():
    """<dy, y> moved along a direction of x, A or B changes by the gradient's product with it (the
    forward pass in 64 bits; y is linear in x, in A and in B, so the difference is exact)."""
    T, K, N, n, R = 40, 72, 56, 3, 16
    _log("adapter differences")
    c = make(T, K, N, n, R, F16, True, 0.1, 11)
    d = to_dev(c)
    args = [d[k] for k in ("a", "b", "ids", "scale")]
    _, u = moe.moe_adapter_forward(d["x"], *args, ranks=d["ranks"], save_u=True)
    grads = moe.moe_adapter_backward(d["dy"], d["x"], u, *args, ranks=d["ranks"])
    g = torch.Generator()
    g.manual_seed(12)
    for key, grad in zip(("x", "a", "b"), grads):
        step = torch.randn(c[key].shape, generator=g, dtype=torch.float64)
        at = []
        for sign in (1.0, -1.0):
            m = dict(c, **{k: c[k].double() for k in ("x", "a", "b")})
            m[key] = m[key] + sign * step
            at.append((reference(m)[0]["y"] * c["dy"].double()).sum())
        diff, terms = float(at[0] - at[1]) / 2, grad.double().cpu() * step
        tol = float(terms.abs().sum()) * (UNIT[grad.dtype] + 2.0 ** -18) + 1e-9
        assert abs(diff - float(terms.sum())) <= tol, (key, diff, float(terms.sum()), tol)


def test_row_does_not_depend_on_its_batch():
    """A request's output bits are the same alone and in a batch of any requests (T <= 64)."""
    K, N, n, R = 2048, 264, 8, 32
    _log("adapter batch independence")
    c = to_dev(make(64, K, N, n, R, F16, False, 0.0, 13))
    args = [c[k] for k in ("a", "b")]
    y = moe.moe_adapter_forward(c["x"], *args, c["ids"], c["scale"])
    for t in (0, 17, 63):
        one = moe.moe_adapter_forward(c["x"][t:t + 1], *args, c["ids"][t:t + 1], c["scale"])
        assert torch.equal(one[0], y[t])


def test_past_32_bits():
    T, K, N, n, R = 360000, 6144, 8, 3, 8
    _log("adapter past 32 bits")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn((T, K), device=DEV, generator=g, dtype=F16)
    a = torch.randn((n, R, K), device=DEV, generator=g).to(F16) / 64
    b = torch.randn((n, N, R), device=DEV, generator=g).to(F16)
    ids = torch.randint(0, n, (T,), device=DEV, generator=g).int()
    scale = torch.ones(n, device=DEV)
    y, u = moe.moe_adapter_forward(x, a, b, ids, scale, save_u=True)
    at = torch.tensor([0, 1, 349525, 349526, T - 2, T - 1], device=DEV)  # 349525.3 * 6144 = 2^31
    i = ids[at].long()
    ref = (a[i].double() @ x[at].double()[:, :, None])[:, :, 0]
    assert bool(((u[at].double() - ref).abs() <= 1e-4).all())
    dy = torch.randn((T, N), device=DEV, generator=g).to(F16)
    dx, _, _ = moe.moe_adapter_backward(dy, x, u, a, b, ids, scale)
    v = (dy[at].double()[:, None, :] @ b[i].double())
    ref = (v @ a[i].double())[:, 0]
    assert bool(((dx[at].double() - ref).abs() <= 2.0 ** -10 * ref.abs() + 1e-4).all())


def test_other_stream_and_graph():
    _log("adapter stream and graph")
    for T in (5, 200):
        c = to_dev(make(T, 512, 264, 5, 16, BF16, True, 0.1, 14))
        args = [c[k] for k in ("a", "b", "ids", "scale")]

        def step(stream=None):
            y, u = moe.moe_adapter_forward(c["x"], *args, ranks=c["ranks"], add=c["add"], save_u=True, stream=stream)
            return [y, u, *moe.moe_adapter_backward(c["dy"], c["x"], u, *args, ranks=c["ranks"], stream=stream)]

        eager = step()
        side = torch.cuda.Stream()
        on_side = step(side)
        side.synchronize()
        for p, q in zip(eager, on_side):
            assert torch.equal(p, q)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            rec = step()
        for seed in range(3):
            c["x"].copy_(torch.randn(c["x"].shape, device=DEV).to(BF16))
            eager = step()
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(eager, rec):
                assert torch.equal(p, q)


def test_binding_refuses():
    c = to_dev(make(4, 64, 72, 3, 8, F16, False, 0.0, 15))
    ok = dict(x=c["x"], a=c["a"], b=c["b"], ids=c["ids"], scale=c["scale"])
    for bad in (dict(x=c["x"].float()), dict(x=c["x"].cpu()), dict(x=c["x"][:, :56]), dict(a=c["a"].to(BF16)), dict(b=c["b"][:2]),
                dict(ids=c["ids"].long()), dict(ids=c["ids"][:3]), dict(scale=c["scale"].half()), dict(ranks=c["ids"]),
                dict(add=c["x"]), dict(out=c["x"]), dict(x=c["x"].t().contiguous().t())):
        with pytest.raises(ValueError):
            moe.moe_adapter_forward(**dict(ok, **bad))
    with pytest.raises(moe.MoeError):  # rank past 128
        moe.moe_adapter_forward(c["x"], torch.zeros((3, 136, 64), device=DEV).half(), torch.zeros((3, 72, 136), device=DEV).half(),
                                c["ids"], c["scale"])
    with pytest.raises(moe.MoeError):  # rows that start inside a vector
        moe.moe_adapter_forward(torch.zeros((4, 72), device=DEV).half()[:, 4:68], c["a"], c["b"], c["ids"], c["scale"])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,R", [(3, 64, 64), (20, 8200, 64), (80, 64, 64), (80, 64, 128), (200, 64, 16)])
def test_infinities_beside_a_lower_rank(dtype, T, K, R):
    """What lies past an adapter's rank adds nothing, not even to a row that holds an infinity."""
    _log("adapter infinity and rank", dtype, T, K, R)
    N, rank = 40, 8
    x = torch.ones((T, K), dtype=dtype, device=DEV)
    a, b = torch.ones((1, R, K), dtype=dtype, device=DEV), torch.ones((1, N, R), dtype=dtype, device=DEV)
    ids, scale = torch.zeros(T, dtype=torch.int32, device=DEV), torch.ones(1, device=DEV)
    ranks = torch.tensor([rank], dtype=torch.int32, device=DEV)
    x[1, 7] = float("inf")
    y, u = moe.moe_adapter_forward(x, a / K, b, ids, scale, ranks=ranks, save_u=True)
    assert bool((y[1] == float("inf")).all()) and bool(torch.isfinite(y[2:]).all())
    assert bool((u[1, :rank] == float("inf")).all()) and bool((u[:, rank:] == 0).all())
    dy = torch.ones((T, N), dtype=dtype, device=DEV)
    dy[2, 3] = float("inf")
    dx, da, db = moe.moe_adapter_backward(dy, torch.ones_like(x), torch.where(torch.isfinite(u), u, 1.0), a, b, ids, scale,
                                          ranks=ranks)
    assert bool((dx[2] == float("inf")).all()) and bool(torch.isfinite(dx[:2]).all())
    assert bool((da[0, rank:] == 0).all()) and bool((db[0, :, rank:] == 0).all())
