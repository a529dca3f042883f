"""Infinities and NaNs in an adapter's operands: results are infinite, with the
formula's sign, and NaN exactly where the formula's are, in 64 bits term by
term; the others keep the tolerances of test_gpu_adapter.py (one rounding of the
output's type, 4 sqrt(n) 2^-24 of the magnitudes of a sum of n terms in fp32, a
factor of a second product carried to 2^-16 of itself for 16-bit outputs and to
2^-21 of the sum's largest for weight gradients)."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8, torch.float32: 2.0 ** -24}
INF, NAN = float("inf"), float("nan")


def _dot(p, q):
    """p [m][c] times q [c][n], every term formed (no zero is skipped), in 64 bits."""
    return torch.stack([(r[:, None] * q).sum(0) for r in p]) if p.shape[0] else p.new_zeros((0, q.shape[1]))


def formula(c, u):
    """u, y, dx, da, db (the last four with the forward pass's u given), and the magnitudes and largest factors of their sums."""
    x, dy, u = c["x"].double(), c["dy"].double(), u.double()
    (T, K), (n, N, R) = x.shape, c["b"].shape
    o = dict(u=x.new_zeros((T, R)), y=x.new_zeros((T, N)), dx=x.new_zeros((T, K)), da=x.new_zeros((n, R, K)), db=x.new_zeros((n, N, R)))
    m, top = ({k: torch.zeros_like(v) for k, v in o.items()} for _ in range(2))
    size = lambda v: torch.where(torch.isfinite(v), v, torch.zeros_like(v)).abs()  # noqa: E731
    for i in range(n):
        rows = torch.nonzero(c["ids"] == i)[:, 0]
        if not rows.numel():
            continue
        a, b, s = c["a"][i].double(), c["b"][i].double(), float(c["scale"][i])
        v = s * _dot(dy[rows], b)
        o["u"][rows] = _dot(x[rows], a.t())
        o["y"][rows], o["dx"][rows] = s * _dot(u[rows], b.t()), _dot(v, a)
        o["da"][i], o["db"][i] = _dot(v.t(), x[rows]), s * _dot(dy[rows].t(), u[rows])
        mv = abs(s) * size(dy[rows]) @ size(b)
        mu = size(x[rows]) @ size(a).t()
        m["u"][rows] = mu
        m["y"][rows], m["dx"][rows] = abs(s) * mu @ size(b).t(), mv @ size(a)
        m["da"][i], m["db"][i] = mv.t() @ size(x[rows]), abs(s) * size(dy[rows]).t() @ size(u[rows])
        top["da"][i] = size(v).max() * size(x[rows]).sum(0)
        top["db"][i] = (abs(s) * size(u[rows]).max() * size(dy[rows]).sum(0))[:, None]
    return o, m, top


def same(got, ref, tol, what):
    g = got.double().cpu()
    assert torch.equal(g.isnan(), ref.isnan()), (what, int(g.isnan().sum()), int(ref.isnan().sum()))
    assert torch.equal(g.isinf(), ref.isinf()) and torch.equal(g[g.isinf()], ref[ref.isinf()]), what
    f = torch.isfinite(ref)
    bound = UNIT[got.dtype] * ref[f].abs() + 2.0 ** -25 + tol[f]
    worst = float(((g[f] - ref[f]).abs() / bound).max()) if bool(f.any()) else 0.0
    print(what, "infinite %d, NaN %d, worst error / tolerance %.3f" % (int(ref.isinf().sum()), int(ref.isnan().sum()), worst), flush=True)
    assert worst <= 1.0, (what, worst)


def make(T, K, N, n, R, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=r(T, K).to(dtype), a=(r(n, R, K) / K ** 0.5).to(dtype), b=(r(n, N, R) * 0.1).to(dtype),
                scale=torch.tensor([1.5, -0.5, 0.75])[:n].clone(), dy=r(T, N).to(dtype),
                ids=torch.randint(0, n, (T,), generator=g).int())


def run(c):
    d = {k: v.to(DEV) for k, v in c.items()}
    args = [d[k] for k in ("a", "b", "ids", "scale")]
    y, u = moe.moe_adapter_forward(d["x"], *args, save_u=True)
    return y, u, moe.moe_adapter_backward(d["dy"], d["x"], u, *args)


def check(c, only=("u", "y", "dx", "da", "db")):
    (T, K), (n, N, R) = c["x"].shape, c["b"].shape
    y, u, (dx, da, db) = run(c)
    ref, mag, top = formula(c, u.cpu())
    f = lambda k: (4 * k ** 0.5 + 2) * 2.0 ** -24  # noqa: E731
    tol = dict(u=f(K) * mag["u"], y=(f(K) + f(R) + 2.0 ** -16) * mag["y"], dx=(f(N) + f(R) + 2.0 ** -16) * mag["dx"],
               da=(f(N) + f(T) + 2.0 ** -22) * mag["da"] + 2.0 ** -21 * top["da"],
               db=(f(T) + 2.0 ** -22) * mag["db"] + 2.0 ** -21 * top["db"])
    for k, got in (("u", u), ("y", y), ("dx", dx), ("da", da), ("db", db)):
        if k in only:
            same(got, ref[k], tol[k], k)
    return ref


# one launch; two for few rows; tiles grouped by each workgroup; ranks over several fragments; parts of an adapter's rows
SHAPES = [(3, 72, 40, 2, 8), (3, 64, 136, 1, 64), (20, 8200, 72, 3, 64), (9, 72, 24, 2, 128), (80, 72, 40, 3, 16), (80, 40, 136, 2, 32),
          (200, 136, 264, 2, 64), (130, 64, 40, 1, 128), (700, 40, 72, 1, 16), (700, 40, 72, 1, 72), (4200, 24, 40, 2, 40)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,N,n,R", SHAPES)
@pytest.mark.parametrize("where", ["a", "b", "x", "dy"])
def test_infinities_keep_their_sign(dtype, T, K, N, n, R, where):
    print("adapter infinity", dtype, T, K, N, n, R, where, flush=True)
    c = make(T, K, N, n, R, dtype, 80 + T)
    v = c[where].view(-1)
    g = torch.Generator()
    g.manual_seed(81)
    at = torch.randperm(v.numel(), generator=g)[:7]
    v[at] = torch.tensor([INF, -INF, INF, INF, -INF, NAN, INF]).to(dtype)
    check(c)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,K,N,n,R", [(3, 64, 40, 1, 16), (20, 8200, 24, 1, 64), (80, 64, 40, 1, 16), (300, 64, 40, 1, 64)])
def test_whole_factors(dtype, T, K, N, n, R):
    """Factors of one bit, whose second piece is zero: 1 times an infinity."""
    print("adapter infinity, whole factors", dtype, T, K, N, n, R, flush=True)
    c = dict(x=torch.ones((T, K)).to(dtype), a=torch.zeros((n, R, K)).to(dtype), b=torch.ones((n, N, R)).to(dtype),
             scale=torch.ones(n), dy=torch.zeros((T, N)).to(dtype), ids=torch.zeros(T).int())
    c["a"][:, :, 3], c["dy"][:, 2] = 1.0, 1.0  # u = v = 1
    b = dict(c, b=c["b"].clone())
    b["b"][0, 5, 1], b["b"][0, 7, 2], b["b"][0, 8, :2] = INF, -INF, torch.tensor([INF, -INF]).to(dtype)
    ref = check(b, ("y",))
    assert bool((ref["y"][:, 5] == INF).all()) and bool((ref["y"][:, 7] == -INF).all()) and bool(ref["y"][:, 8].isnan().all())
    x, dy = dict(c, x=c["x"].clone()), dict(c, dy=c["dy"].clone())
    x["x"][1, 9], dy["dy"][1, 9] = INF, -INF
    check(x, ("dx",))
    check(dy, ("y", "db"))
    # x and dy in the weights' gradients of factors that stay finite: a column of A that is 0 where x is not finite would be NaN in u
    d = {k: v.to(DEV) for k, v in x.items()}
    u = torch.ones((T, R), device=DEV)
    _, da, db = moe.moe_adapter_backward(d["dy"], d["x"], u, *[d[k] for k in ("a", "b", "ids", "scale")])
    assert bool((da[0, :, 9] == INF).all()) and bool((da[0, :, :9] == T).all())
    d["dy"] = dy["dy"].to(DEV)
    _, da, db = moe.moe_adapter_backward(d["dy"], c["x"].to(DEV), u, *[d[k] for k in ("a", "b", "ids", "scale")])
    assert bool((db[0, 9] == -INF).all()) and bool((db[0, 2] == T).all()) and bool((db[0, 3] == 0).all())


@pytest.mark.parametrize("T,R", [(2, 16), (40, 64), (80, 16), (80, 64), (80, 128)])
def test_small_factors_beside_large(T, R):
    """A factor too small for any piece beside its row's largest still has a sign."""
    K, N = 64, 40
    print("adapter infinity, small factors", T, R, flush=True)
    c = make(T, K, N, 1, R, F16, 90)
    c["x"] = c["x"].abs() + 0.5
    c["a"] = c["a"].abs() * 2.0 ** 8
    c["a"][0, 2], c["a"][0, 3] = 0.0, 0.0
    c["a"][0, 2, 0], c["a"][0, 3, 0] = 2.0 ** -24, -2.0 ** -24
    c["x"][:, 0] = 2.0 ** -14  # u[2] = 2^-38, u[3] = -2^-38; the others about 2^10
    c["b"][0, :, 2], c["b"][0, :, 3] = 0.0, 0.0
    c["b"][0, 5, 2], c["b"][0, 6, 3] = INF, INF
    y, u, _ = run(c)
    assert bool((u[:, 2] == 2.0 ** -38).all()) and bool((u[:, 3] == -2.0 ** -38).all())
    assert bool((y[:, 5] == 1.5 * INF).all()) and bool((y[:, 6] == -INF).all())
    # and where the sum runs over rows: one row's u is small, and its dy infinite
    t = T - 1
    dy, u = c["dy"].to(DEV), u.clone()
    u[t] = 2.0 ** -40
    dy[t, 9] = -INF
    d = {k: v.to(DEV) for k, v in c.items()}
    _, _, db = moe.moe_adapter_backward(dy, d["x"], u, *[d[k] for k in ("a", "b", "ids", "scale")], need_dx=False)
    assert bool((db[0, 9] == -INF).all())


def test_products_past_fp32():
    """bfloat16 holds fp32's range: a product past it is infinite, whatever its pieces' signs."""
    print("adapter products past fp32", flush=True)
    for T, R in ((3, 16), (80, 16), (80, 64)):
        c = make(T, 64, 40, 1, R, BF16, 91)
        c["x"] = (c["x"].float() * 2.0 ** 60).to(BF16)
        c["a"] = (c["a"].float() * 2.0 ** 20).to(BF16)
        c["b"][0, 5], c["b"][0, 5, 0] = 0.0, 2.0 ** 90
        y, u, _ = run(c)
        big = u[:, 0].double().abs() > 2.0 ** 40
        assert bool((y[big, 5].double() == u[big, 0].double().sign() * INF).all())
