"""Products with 4-bit weights and their input gradient, on the GPU, against 64 bits.

Tolerance of an output element that sums n terms w x, with u = half a step of the
rows' type and r the 2-norm of the terms:
- its own rounding: u |value| (and 2^-25, half of binary16's smallest step);
- where weights are rounded to the rows' type (all but the path for few rows): every
  term is off by up to u |w x| (binary16: or 2^-25 |x|), with signs that do not
  follow the inputs'; by Hoeffding's inequality the sum of such errors passes 7 u r
  with probability below 2 exp(-24.5) = 5e-11;
- fp32 sums: 4 sqrt(n) 2^-24 sum |w x|, where the few rows' bfloat16 factors are
  codes plus up to 143 instead of the code (up to 8 + |z|): magnitudes 152 s |x|
  and more, taken as (160 + 2 |z|) s |x|.
"""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from w4_reference import product, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


def make(T, K, N, n, group, dtype, zeros, seed, offsets=None, backward=False):
    g = torch.Generator().manual_seed(seed)
    G = group or K
    c = dict(q=torch.randint(0, 256, (n, N, K // 2), generator=g, dtype=torch.uint8),
             scales=(K ** -0.5 * (0.1 + 0.2 * torch.rand((n, N, K // G), generator=g))).to(dtype),
             zeros=torch.randint(-128, 128, (n, N, K // G), generator=g, dtype=torch.int8) if zeros == "wide" else
             torch.randint(-8, 8, (n, N, K // G), generator=g, dtype=torch.int8) if zeros else None,
             x=torch.randn((T, N if backward else K), generator=g).to(dtype),
             add=torch.randn((T, K if backward else N), generator=g).to(dtype),
             offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32))
    return c


def pack(c):
    return moe.moe_w4_pack(c["q"].to(DEV), c["scales"].to(DEV), None if c["zeros"] is None else c["zeros"].to(DEV))


def tolerance(c, w, norm, few, backward):
    dt = c["x"].dtype
    u = UNIT[dt]
    big = 8.0 if c["zeros"] is None else 8.0 + float(c["zeros"].double().abs().max())
    if few and dt == BF16:
        big = 160.0 + 2 * big
    terms = w.shape[1] if backward else w.shape[2]
    top = float(c["scales"].double().abs().max()) * big
    mags = top * c["x"].double().abs().sum(1, keepdim=True)
    tol = 4 * terms ** 0.5 * 2.0 ** -24 * mags
    if not few:
        tol = tol + 7 * u * norm
        if dt == F16:
            tol = tol + 2.0 ** -25 * c["x"].double().abs().sum(1, keepdim=True)
    return tol


def check(got, ref, tol, dtype, what):
    g = got.detach().double().cpu()
    assert g.shape == ref.shape and bool(torch.isfinite(g).all()), what
    err, bound = (g - ref).abs(), UNIT[dtype] * ref.abs() + 2.0 ** -25 + tol
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(what, "worst error / tolerance %.3f" % worst, flush=True)
    assert worst <= 1.0, (what, worst)


def run_case(c, backward, add, what):
    print(what, flush=True)
    w = pack(c)
    n, N, K = w.shape
    T = c["x"].shape[0]
    off = None if c["offsets"] is None else c["offsets"].to(DEV)
    few = not backward and moe.moe_w4_few_rows(w, T)
    call = moe.moe_w4_backward if backward else moe.moe_w4_forward
    got = call(c["x"].to(DEV), w, offsets=off, add=c["add"].to(DEV) if add else None)
    torch.cuda.synchronize()
    m = weights(c["q"], c["scales"], c["zeros"])
    ref, norm = product(c["x"], m, c["offsets"], backward)
    if add:
        ref = ref + c["add"].double()
    check(got, ref, tolerance(c, m, norm, few, backward), c["x"].dtype, what)
    return few


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,N,K,group,zeros", [(1, 24, 96, 32, True), (2, 40, 320, 64, True), (3, 8, 256, 128, False),
                                               (1, 200, 160, 0, True), (2, 16, 768, 384, False)])
def test_pack_and_back(n, N, K, group, zeros, dtype):
    c = make(1, K, N, n, group, dtype, zeros, 1)
    print("pack", n, N, K, group, zeros, dtype, flush=True)
    q, s, z = moe.moe_w4_unpack(pack(c))
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), c["q"]) and torch.equal(s.cpu(), c["scales"])
    assert (z is None) == (c["zeros"] is None) and (z is None or torch.equal(z.cpu(), c["zeros"]))


SHAPES = [(8, 32, 32, False), (24, 96, 0, True), (200, 160, 32, True), (136, 320, 64, False), (264, 2080, 32, "wide"),
          (520, 1024, 128, True), (72, 768, 384, False), (1000, 1280, 0, False), (16400, 256, 64, True)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES)
def test_few_rows(N, K, group, zeros, T, dtype):
    c = make(T, K, N, 1, group, dtype, zeros, T + N)
    assert run_case(c, False, T == 3, f"few T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [17, 33, 65, 129, 400])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES[:8])
def test_many_rows(N, K, group, zeros, T, dtype):
    c = make(T, K, N, 1, group, dtype, zeros, T + N)
    run_case(c, False, T % 2 == 0, f"rows T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [513, 578, 1000])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES[:8])
def test_more_rows(N, K, group, zeros, T, dtype):
    """Past the kernel for few rows, with split sums where the matrix is small."""
    c = make(T, K, N, 1, group, dtype, zeros, T + N)
    assert not run_case(c, False, T % 2 == 0, f"more rows T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [17, 33, 70])
@pytest.mark.parametrize("N,K,group,zeros", [(10248, 4128, 32, True), (10312, 4160, 64, False), (20520, 2080, 0, True)])
def test_rows_of_large_matrices(N, K, group, zeros, T, dtype):
    """Few rows of a matrix too large for the kernel for few rows: tiles of 32 and 64 rows."""
    c = make(T, K, N, 1, group, dtype, zeros, T + N)
    assert not run_case(c, False, T % 2 == 0, f"large matrix T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,N,K,group,zeros,offsets", [(100, 40, 16384, 128, False, None), (70, 24, 8160, 32, True, [18, 55]),
                                                       (512, 8, 12800, 64, True, [0, 511]), (33, 72, 6240, 0, True, None),
                                                       (16, 40, 16384, 128, False, [3, 13]), (14, 72, 12320, 32, True, [5, 14])])
def test_wide_matrices(T, N, K, group, zeros, offsets, dtype):
    """Several passes over the columns by the kernel for few rows, and split sums; rows outside one group."""
    c = make(T, K, N, 1, group, dtype, zeros, T, offsets)
    few = run_case(c, False, offsets is not None, f"wide T={T} N={N} K={K} {dtype}")
    assert few == (T <= 16)


def test_borders_of_few_rows():
    """moe_w4_few_rows on both sides of its rule, with rows outside one group."""
    for N, K, T, few in ((2048, 2048, 320, True), (2048, 2048, 321, False), (64, 256, 512, True), (64, 256, 513, False),
                         (72, 6144, 400, True), (72, 6272, 400, False)):
        c = make(T, K, N, 1, 128, BF16, True, T, [3, T - 5])
        assert run_case(c, False, True, f"border N={N} K={K} T={T}") == few


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 16, 33, 65, 129, 400])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES[:8])
def test_gradient(N, K, group, zeros, T, dtype):
    c = make(T, K, N, 1, group, dtype, zeros, T + N, backward=True)
    run_case(c, True, T % 2 == 0, f"grad T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,N,K,group,zeros", [(2, 6144, 128, 128, False), (45, 6144, 96, 32, "wide"), (64, 1000, 2080, 32, True),
                                               (100, 2056, 2048, 64, True), (16, 8, 16384, 128, True), (17, 72, 8160, 0, False),
                                               (40, 6152, 256, 64, False), (512, 24, 1024, 512, True), (4096, 40, 32, 32, True)])
def test_short_gradient(T, N, K, group, zeros, dtype):
    """Around the borders between the gradient's kernels: most are a workgroup per CU or fewer of the one without workspace."""
    c = make(T, K, N, 1, group, dtype, zeros, T + N, backward=True)
    run_case(c, True, T % 2 == 1, f"short grad T={T} N={N} K={K} group={group} zeros={zeros} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_short_gradient_in_place(group, dtype):
    """Rows outside one group unread, add the same as out, called on two streams at once and replayed: the same bits."""
    c = make(50, 1152, 328, 1, group, dtype, True, 11, [5, 43], backward=True)
    c["x"][:5] = c["x"][43:] = float("nan")
    print("short grad in place", group, dtype, flush=True)
    w, dy, add, off = pack(c), c["x"].to(DEV), c["add"].to(DEV), c["offsets"].to(DEV)
    plain = moe.moe_w4_backward(dy, w, offsets=off, add=add)
    ref, norm = product(torch.nan_to_num(c["x"]), weights(c["q"], c["scales"], c["zeros"]), c["offsets"], True)
    m = weights(c["q"], c["scales"], c["zeros"])
    c["x"] = torch.nan_to_num(c["x"])
    check(plain, ref + c["add"].double(), tolerance(c, m, norm, False, True), dtype, "short grad")
    assert torch.equal(plain[:5], add[:5]) and torch.equal(plain[43:], add[43:])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [moe.moe_w4_backward(dy, w, offsets=off, add=add, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, plain) for o in outs)
    out, graph = add.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w4_backward(dy, w, offsets=off, add=out, out=out)
    for _ in range(3):
        out.copy_(add)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("N,K,group,zeros,backward", [(10000, 160, 32, True, False), (9800, 256, 128, False, False),
                                                      (72, 16384, 64, True, True), (136, 15000 // 32 * 32, 0, False, True)])
def test_large_tiles(N, K, group, zeros, backward, dtype):
    """Enough workgroups for tiles of 128 rows, the last of them ragged."""
    c = make(1100, K, N, 1, group, dtype, zeros, N, backward=backward)
    run_case(c, backward, False, f"large N={N} K={K} backward={backward} {dtype}")


# rows before, between and after the groups, empty groups, one group, uneven groups
OFFSETS = [(5, [0, 3, 3, 9, 10, 40], 47), (4, [2, 2, 2, 2, 2], 5), (3, [0, 0, 60, 61], 61), (1, [7, 40], 64),
           (1, [0, 100], 100), (7, [0, 130, 131, 131, 200, 201, 330, 700], 700), (130, list(range(0, 262, 2)), 261), (2, [0, 0, 0], 40),
           (6, [2, 3, 3, 9, 9, 12, 13], 16), (3, [0, 0, 16, 16], 16), (1, [3, 9], 12), (90, [0] * 30 + [1] * 20 + [5] * 40 + [40], 44)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("n,offsets,T", OFFSETS)
def test_groups(n, offsets, T, backward, dtype):
    offsets = [min(v, T) for v in offsets]
    for N, K, group, zeros, add in ((72, 160, 32, True, True), (200, 384, 128, False, False)) + ((40, 4128, 32, True, True),) * backward:
        c = make(T, K, N, n, group, dtype, zeros, n + T, offsets, backward)
        for e0, e1 in ((0, offsets[0]), (offsets[-1], T)):  # not read
            c["x"][e0:e1] = float("nan")
        w = pack(c)
        print("groups", n, T, N, K, backward, dtype, flush=True)
        call = moe.moe_w4_backward if backward else moe.moe_w4_forward
        got = call(c["x"].to(DEV), w, offsets=c["offsets"].to(DEV), add=c["add"].to(DEV) if add else None)
        torch.cuda.synchronize()
        c["x"] = torch.nan_to_num(c["x"])
        m = weights(c["q"], c["scales"], c["zeros"])
        ref, norm = product(c["x"], m, c["offsets"], backward)
        few = not backward and moe.moe_w4_few_rows(w, T)
        check(got, ref + c["add"].double() if add else ref, tolerance(c, m, norm, few, backward), dtype, "groups")


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T", [5, 90, 1200])
def test_strides_and_in_place(T, backward):
    """Rows of wider buffers, add the same as out, and nothing written beside the rows."""
    c = make(T, 416, 104, 1, 32, F16, True, 3, backward=backward)
    print("strides", T, backward, flush=True)
    w = pack(c)
    call = moe.moe_w4_backward if backward else moe.moe_w4_forward
    wide = torch.full((T, c["x"].shape[1] + 24), float("nan"), dtype=F16, device=DEV)
    wide[:, 8:8 + c["x"].shape[1]] = c["x"].to(DEV)
    plain = call(c["x"].to(DEV), w, add=c["add"].to(DEV))
    width = c["add"].shape[1]
    out = torch.full((T + 2, width + 16), 7.0, dtype=F16, device=DEV)
    rows = out[1:T + 1, 8:8 + width]
    rows.copy_(c["add"].to(DEV))
    call(wide[:, 8:8 + c["x"].shape[1]], w, add=rows, out=rows)
    torch.cuda.synchronize()
    assert torch.equal(rows, plain)
    out[1:T + 1, 8:8 + width] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,backward", [(2, False), (40, False), (2, True), (5000, False), (5000, True)])
def test_infinities(T, backward, dtype):
    """Infinities and NaNs of a row stay in that row and are the formula's."""
    c = make(T, 256, 64, 1, 64, dtype, True, 9, backward=backward)
    print("infinities", T, backward, dtype, flush=True)
    c["x"][0, 5], c["x"][1, 7] = float("inf"), float("nan")
    w = pack(c)
    got = (moe.moe_w4_backward if backward else moe.moe_w4_forward)(c["x"].to(DEV), w).double().cpu()
    m = weights(c["q"], c["scales"], c["zeros"])[0]
    want = torch.where((m[5] if backward else m[:, 5]) == 0, float("nan"), float("inf") * (m[5] if backward else m[:, 5]).sign())
    assert bool(got[1].isnan().all()) and bool(torch.isfinite(got[2:]).all())
    assert torch.equal(got[0].isnan(), want.isnan()) and torch.equal(got[0].nan_to_num(1, 2, -2), want.nan_to_num(1, 2, -2))


def test_bf16_past_the_range_of_offset_codes():
    """Rows whose products with 128 + u pass fp32's range although the formula's do not."""
    c = make(2, 128, 16, 1, 128, BF16, False, 4)
    print("range", flush=True)
    c["x"][0] = (c["x"][0].float().sign() * 3e36).to(BF16)
    got = moe.moe_w4_forward(c["x"].to(DEV), pack(c)).double().cpu()
    ref, norm = product(c["x"], weights(c["q"], c["scales"], None), None, False)
    assert bool(torch.isfinite(got).all())
    assert float(((got - ref).abs() / (2.0 ** -8 * ref.abs() + 2.0 ** -16 * norm + 2.0 ** -25)).max()) <= 1


def test_weights_past_32_bits():
    """Packed weights of 8.6 GB, rows of 17 GB: offsets past 32 bits."""
    n, N, K = 64, 16384, 16384
    print("large weights", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randint(0, 256, (n, N, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    scales = torch.full((n, N, 1), 2.0 ** -7, dtype=F16, device=DEV)
    w = moe.moe_w4_pack(q, scales)
    assert w.packed.numel() > 2 ** 33
    offsets = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    offsets[63:] = torch.tensor([1, 3], dtype=torch.int32)  # row 0 for expert 62, rows 1 and 2 for expert 63
    x = torch.randn((3, K), device=DEV, generator=g).half()
    y = moe.moe_w4_forward(x, w, offsets=offsets)
    dx = moe.moe_w4_backward(x, w, offsets=offsets)
    for e, r0, r1 in ((62, 0, 1), (63, 1, 3)):
        m = weights(q[e:e + 1].cpu(), scales[e:e + 1].cpu(), None)
        for got, back in ((y, False), (dx, True)):
            ref, norm = product(x[r0:r1].cpu(), m, None, back)
            off = (got[r0:r1].double().cpu() - ref).abs() / (2.0 ** -11 * (ref.abs() + 7 * norm) + 2.0 ** -8)
            assert float(off.max()) <= 1, (e, back)


def test_rows_past_32_bits():
    T, K, N = 1 << 19, 8192, 8
    print("large rows", flush=True)
    c = make(1, K, N, 1, 128, F16, False, 5)
    w = pack(c)
    x = torch.zeros((T, K), dtype=F16, device=DEV)
    x[-3:] = torch.randn((3, K), generator=torch.Generator().manual_seed(2)).half().to(DEV)
    y = moe.moe_w4_forward(x, w)
    m = weights(c["q"], c["scales"], None)
    ref, norm = product(x[-3:].cpu(), m, None, False)
    assert bool((y[:-3] == 0).all())
    assert float(((y[-3:].double().cpu() - ref).abs() / (2.0 ** -11 * (ref.abs() + 7 * norm) + 2.0 ** -11)).max()) <= 1
    dx = moe.moe_w4_backward(y, w, out=x)
    ref, norm = product(y[-3:].cpu(), m, None, True)
    assert bool((dx[:-3] == 0).all())
    assert float(((dx[-3:].double().cpu() - ref).abs() / (2.0 ** -11 * (ref.abs() + 7 * norm) + 2.0 ** -14)).max()) <= 1


def test_gradient_is_the_derivative():
    """<dx, v> equals the change of <dy, y> along v (the product is linear: one difference is exact but for rounding)."""
    c = make(40, 384, 104, 1, 64, F16, True, 6)
    print("difference", flush=True)
    w = pack(c)
    g = torch.Generator().manual_seed(8)
    x, v = c["x"].to(DEV), torch.randn((40, 384), generator=g).half().to(DEV)
    dy = torch.randn((40, 104), generator=g).half().to(DEV)
    dx = moe.moe_w4_backward(dy, w)
    diff = moe.moe_w4_forward((x + v), w).double() - moe.moe_w4_forward(x, w).double()
    change, slope = float((dy.double() * diff).sum()), float((dx.double() * ((x + v).double() - x.double())).sum())
    # 4,160 and 15,360 products of values rounded by up to 2^-11 each, signs at random
    y = moe.moe_w4_forward(x, w).double().abs().max()
    bound = 7 * 2.0 ** -11 * (float((dy.double() ** 2).sum()) ** 0.5 * float(y) * 2 * 2 + float((dx.double() * v.double()).norm()))
    print(change, slope, bound, flush=True)
    assert abs(change - slope) <= bound


@pytest.mark.parametrize("T", [0])
def test_no_rows(T):
    c = make(1, 64, 16, 1, 64, F16, False, 2)
    w = pack(c)
    x = torch.empty((0, 64), dtype=F16, device=DEV)
    assert moe.moe_w4_forward(x, w).shape == (0, 16)
    assert moe.moe_w4_backward(torch.empty((0, 16), dtype=F16, device=DEV), w).shape == (0, 64)


def test_captured_and_on_another_stream():
    c = make(70, 1280, 200, 3, 64, BF16, True, 7, [0, 30, 30, 66])
    print("graph", flush=True)
    w, off, add = pack(c), c["offsets"].to(DEV), c["add"].to(DEV)
    x, few = c["x"].to(DEV), c["x"][:20].to(DEV)
    off_few = torch.tensor([0, 5, 5, 20], dtype=torch.int32, device=DEV)

    def step():
        y = moe.moe_w4_forward(x, w, offsets=off, add=add)
        return y, moe.moe_w4_backward(y, w, offsets=off), moe.moe_w4_forward(few, w, offsets=off_few)

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(c["x"].to(DEV) * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
    x.copy_(c["x"].to(DEV))
    s2 = torch.cuda.Stream()
    y = moe.moe_w4_forward(x, w, offsets=off, add=add, stream=s2)
    dx = moe.moe_w4_backward(y, w, offsets=off, stream=s2)
    s2.synchronize()
    assert torch.equal(y, eager[0]) and torch.equal(dx, eager[1])


def test_refuses():
    c = make(4, 64, 16, 2, 64, F16, True, 2, [0, 2, 4])
    w, x, off = pack(c), c["x"].to(DEV), c["offsets"].to(DEV)
    for bad in (dict(offsets=None), dict(offsets=off[:2]), dict(offsets=off.long()), dict(offsets=off, add=x),
                dict(offsets=off, out=torch.empty((4, 16), dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            moe.moe_w4_forward(x, w, **bad)
    for t in (x.float(), x.bfloat16(), x[:, :32], x.t(), x.cpu()):
        with pytest.raises(ValueError):
            moe.moe_w4_forward(t, w, offsets=off)
    with pytest.raises(moe.MoeError):  # rows that are not 16-byte aligned
        moe.moe_w4_forward(torch.empty((4, 68), dtype=F16, device=DEV)[:, :64], w, offsets=off)
    q, s, z = (t.to(DEV) for t in (c["q"], c["scales"], c["zeros"]))
    for args in ((q, s.float(), z), (q, s[:, :8], z), (q.long(), s, z), (q, s, z[:1]), (q[0, 0], s, z)):
        with pytest.raises(ValueError):
            moe.moe_w4_pack(*args)
    with pytest.raises(moe.MoeError):
        moe.moe_w4_pack(q[:, :12].contiguous(), s[:, :12].contiguous())  # 12 rows
