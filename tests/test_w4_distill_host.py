"""Refusals and sizes of the 4-bit products' and the distillation loss' entry
points: decided on the host before any launch (no GPU needed)."""
import struct

import pytest

import quantized_moe_expert_02_amd as moe

OK, INVAL, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = 1 << 20  # an aligned address that a refused call never touches


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from quantized_moe_expert_02_amd import build
        build.build()
    return moe.lib()


def dims(n=1, N=64, K=256, group=64, zeros=0, dtype=0):
    return struct.pack("@iiiiii", n, N, K, group, zeros, dtype)


def _expect(fn, good, changes):
    names = list(good)
    for name, value, status in changes:
        args = dict(good, **{name: value})
        assert fn(*[args[n] for n in names]) == status, (name, value)


BAD_DIMS = [(dims(n=0), INVAL), (dims(N=0), INVAL), (dims(K=-32), INVAL), (dims(group=0), INVAL), (dims(zeros=2), INVAL),
            (dims(dtype=2), INVAL), (dims(dtype=-1), INVAL), (dims(group=96), INVAL), (dims(N=60), UNSUPPORTED),
            (dims(K=240, group=48), UNSUPPORTED), (dims(K=48, group=48), UNSUPPORTED), (dims(K=65568, group=32), UNSUPPORTED),
            (dims(group=16), UNSUPPORTED), (dims(K=384, group=192), UNSUPPORTED), (dims(n=1025), UNSUPPORTED),
            (dims(N=(1 << 20) + 8), UNSUPPORTED), (dims(n=32, N=(1 << 19) + 8), UNSUPPORTED), (None, INVAL)]


def test_w4_sizes(L):
    for n, N, K, group, zeros in ((1, 64, 256, 64, 0), (3, 8, 32, 32, 1), (2, 72, 160, 160, 1), (5, 1000, 768, 384, 0)):
        size = L.moe_w4_packed_bytes(dims(n, N, K, group, zeros))
        assert size % (256 * n) == 0 and size >= n * (N * K // 2 + N * K // group * (3 if zeros else 2))
        # rows padded to 16, columns to 128, a scale for at least every 128 columns
        rows, blocks = -(-N // 16) * 16, -(-K // 128)
        groups = blocks * (4 if group == 32 else 2 if group == 64 else 1)
        assert size <= n * (rows * blocks * 64 + rows * groups * 3 + 512)
    for d, _ in BAD_DIMS:
        assert L.moe_w4_packed_bytes(d) == 0 and L.moe_w4_workspace_bytes(d, 4, 1) == 0 and L.moe_w4_few_rows(d, 4) == 0
    for back in (0, 1):
        assert L.moe_w4_workspace_bytes(dims(), 0, back) == 0 and L.moe_w4_workspace_bytes(dims(), -1, back) == 0
    assert L.moe_w4_few_rows(dims(), 1) == 1 and L.moe_w4_few_rows(dims(), 2000) == 0
    assert L.moe_w4_workspace_bytes(dims(N=8192, K=6144, group=128), 64, 0) > 0  # few tiles: the columns are split
    # short gradients need none: up to 6,144 matrix rows, and a workgroup of 64 columns and 32 rows per CU
    for n, N, K, T, need in ((8, 1024, 1024, 128, 0), (8, 1024, 2048, 256, 1), (64, 512, 256, 64, 0), (8, 6152, 1024, 16, 1)):
        assert (L.moe_w4_workspace_bytes(dims(n, N, K, 128), T, 1) > 0) == bool(need), (n, N, K, T)
    for N, K, T, need in ((6144, 6144, 64, 0), (6152, 6144, 64, 1), (6144, 6144, 96, 1), (1024, 8192, 64, 0), (1024, 8192, 65, 1)):
        assert (L.moe_w4_workspace_bytes(dims(N=N, K=K, group=128), T, 1) > 0) == bool(need), (N, K, T)


def test_w4_pack_refuses(L):
    for fn in (L.moe_w4_pack, L.moe_w4_unpack):
        a, b = ("q", "packed") if fn is L.moe_w4_pack else ("packed", "q")
        good = {"d": dims(zeros=1)}
        good.update({"q": P, "scales": P, "zeros": P, "packed": P} if a == "q" else {"packed": P, "q": P, "scales": P, "zeros": P})
        good["stream"] = None
        _expect(fn, good, [("d", d, st) for d, st in BAD_DIMS] + [
            ("q", None, INVAL), ("q", P + 8, INVAL), ("scales", None, INVAL), ("scales", P + 1, INVAL), ("zeros", None, INVAL),
            ("packed", None, INVAL), ("packed", P + 128, INVAL)])
        _expect(fn, dict(good, d=dims()), [("zeros", P, INVAL)])


def test_w4_products_refuse(L):
    for fn, into, out in ((L.moe_w4_forward, 256, 64), (L.moe_w4_backward, 64, 256)):
        good = dict(d=dims(n=3), packed=P, x=P, ldx=into, T=2000, offsets=P, add=None, ldadd=0, y=P, ldy=out, ws=P, ws_bytes=1 << 40,
                    stream=None)
        _expect(fn, good, [("d", d, st) for d, st in BAD_DIMS] + [
            ("packed", None, INVAL), ("packed", P + 16, INVAL), ("x", None, INVAL), ("x", P + 8, INVAL), ("ldx", into - 8, INVAL),
            ("ldx", into + 4, INVAL), ("ldx", (1 << 22) + 8, UNSUPPORTED), ("T", -1, INVAL), ("T", (1 << 20) + 1, UNSUPPORTED),
            ("offsets", None, INVAL), ("offsets", P + 2, INVAL), ("add", P + 8, INVAL), ("add", P, INVAL), ("y", None, INVAL),
            ("y", P + 4, INVAL), ("ldy", out - 8, INVAL), ("ldy", out + 1, INVAL), ("T", 0, OK)])
        # a call that splits its sums needs a workspace
        d = dims(N=8192, K=8192, group=128)
        into = out = 8192
        assert L.moe_w4_workspace_bytes(d, 64, int(fn is L.moe_w4_backward)) > 0
        split = dict(good, d=d, ldx=into, ldy=out, T=64, offsets=None)
        _expect(fn, split, [("ws", None, INVAL), ("ws", P + 8, INVAL), ("ws_bytes", 1024, WORKSPACE)])
    # rows times width
    good = dict(d=dims(N=1 << 20, K=32, group=32), packed=P, x=P, ldx=32, T=1 << 16, offsets=None, add=None, ldadd=0, y=P, ldy=1 << 20,
                ws=P, ws_bytes=1 << 40, stream=None)
    _expect(L.moe_w4_forward, good, [("T", 1 << 16, UNSUPPORTED)])


def test_distill_refuses(L):
    f = dict(z=P, dtype=0, ldz=1000, T=8, V=1000, ids=P, teacher=P, k=4, tau=1.0, loss=P, stats=P, ws=P, ws_bytes=1 << 30, stream=None)
    common = [("z", None, INVAL), ("z", P + 1, INVAL), ("dtype", 3, INVAL), ("dtype", -1, INVAL), ("ldz", 999, INVAL), ("T", -1, INVAL),
              ("T", (1 << 20) + 1, UNSUPPORTED), ("V", 0, INVAL), ("ids", None, INVAL), ("ids", P + 2, INVAL), ("teacher", None, INVAL),
              ("k", 0, INVAL), ("k", 1025, UNSUPPORTED), ("tau", 0.0, INVAL), ("tau", -1.0, INVAL), ("tau", float("nan"), INVAL),
              ("tau", float("inf"), INVAL), ("tau", 2.0 ** -65, UNSUPPORTED), ("tau", 2.0 ** 65, UNSUPPORTED), ("ldz", 1 << 41, UNSUPPORTED), ("ldz", 1 << 39, UNSUPPORTED), ("stats", None, INVAL),
              ("stats", P + 2, INVAL), ("T", 0, OK)]
    _expect(L.moe_distill_forward, f, common + [("loss", None, INVAL), ("loss", P + 1, INVAL)])
    _expect(L.moe_distill_forward, dict(f, V=(1 << 24) + 1, ldz=1 << 25), [("k", 4, UNSUPPORTED)])
    wide = dict(f, V=100000, ldz=100000)
    assert L.moe_distill_workspace_bytes(8, 100000, 0) > 0
    _expect(L.moe_distill_forward, wide, [("ws", None, INVAL), ("ws", P + 8, INVAL), ("ws_bytes", 8, WORKSPACE)])
    b = dict(z=P, dtype=1, ldz=1000, T=8, V=1000, ids=P, teacher=P, k=4, tau=1.0, stats=P, dloss=P, dz=P << 4, lddz=1000, stream=None)
    _expect(L.moe_distill_backward, b, common + [("dloss", None, INVAL), ("dloss", P + 2, INVAL), ("dz", None, INVAL), ("dz", P + 1, INVAL),
                                                 ("lddz", 999, INVAL), ("lddz", 1 << 41, UNSUPPORTED)])
    _expect(L.moe_distill_backward, dict(b, dz=P), [("lddz", 1008, INVAL)])
    for bad in ((-1, 5, 0), (4, 0, 0), (4, 5, 3), (1 << 21, 5, 0), (4, 1 << 25, 0), (0, 5, 0)):
        assert L.moe_distill_workspace_bytes(*bad) == 0
