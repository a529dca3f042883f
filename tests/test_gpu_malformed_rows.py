"""Index arrays whose contents are not what a sort leaves: entries outside
their range count as dropped, and every row of an output is written."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,k,rows,H", [(5, 2, 16, 64), (0, 2, 9, 8), (300, 4, 1500, 264)])
def test_combine_gradient_zeroes_rows_without_a_slot(T, k, rows, H):
    """A row of d_o is zero if its pair is any value outside [0, T k), or a slot whose pos is none of the rows."""
    print("combine gradient, odd pairs", T, k, rows, H, flush=True)
    g = torch.Generator()
    g.manual_seed(70)
    n = T * k
    place = torch.randperm(rows, generator=g)[:n].int()
    odd = torch.tensor([-1, n, n + 1, 2 ** 31 - 1, -2 ** 31, -7], dtype=torch.int32)
    pairs = odd[torch.randint(0, odd.numel(), (rows,), generator=g)]
    pairs[place.long()] = torch.arange(n, dtype=torch.int32)
    pos = place.clone()
    for i, v in enumerate((rows, 2 ** 31 - 1, -3)):  # dropped slots that their rows still name
        pos[i::15] = v
    kept = (pos >= 0) & (pos < rows)
    clean_pos, clean_pairs = torch.where(kept, pos, -1).reshape(T, k), torch.full((rows,), -1, dtype=torch.int32)
    clean_pairs[place[kept].long()] = torch.arange(n, dtype=torch.int32)[kept]
    o, w, dy = torch.randn((rows, H), generator=g), torch.rand((T, k), generator=g), torch.randn((T, H), generator=g)
    dev = [v.to(DEV) for v in (dy, o, w, pos.reshape(T, k), pairs)]
    spoilt = torch.full((rows, H), 9.0, device=DEV)  # what the allocator hands out next
    del spoilt
    d_o, dw = moe.moe_combine_backward(*dev)
    ref_o, ref_w = moe.moe_combine_backward(*dev[:3], clean_pos.to(DEV), clean_pairs.to(DEV))
    assert torch.equal(d_o, ref_o) and torch.equal(dw, ref_w)
    assert bool((d_o[(clean_pairs < 0).to(DEV)] == 0).all()) and bool((dw[(clean_pos < 0).to(DEV)] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,R", [(70, 16), (70, 64), (1500, 24), (1500, 128), (4500, 16)])
def test_adapters_pass_over_rows_outside_the_batch(dtype, T, R):
    """Offsets outside [0, T] end at its ends, and a pair outside [0, T) is no row: as with a clean order."""
    print("adapters, odd order", dtype, T, R, flush=True)
    K, N, n = 72, 136, 4
    g = torch.Generator()
    g.manual_seed(71)
    r = lambda *s: torch.randn(s, generator=g).to(dtype).to(DEV)  # noqa: E731
    offsets = torch.tensor([-9, 20, 2 ** 31 - 1, -2 ** 31, -1], dtype=torch.int32, device=DEV)
    sane = torch.tensor([0, 20, T, T, T], dtype=torch.int32, device=DEV)
    rows = torch.randperm(T, generator=g).int()
    ids = torch.empty(T, dtype=torch.int32)
    ids[rows.long()] = (torch.arange(T) >= 20).int()
    odd = torch.rand(T, generator=g) < 0.2
    pairs, clean = rows.clone(), rows.clone()
    pairs[odd] = torch.tensor([-3, T, 2 ** 31 - 1, -2 ** 31, T + 5], dtype=torch.int32)[torch.arange(int(odd.sum())) % 5]
    clean[odd] = -1
    kept = rows[~odd].long().to(DEV)
    x, dy, a, b, scale = r(T, K), r(T, N), r(n, R, K) / 8, r(n, N, R) / 8, torch.ones(n, device=DEV)
    u = torch.randn((T, R), generator=g).to(DEV)
    ids, got = ids.to(DEV), []
    for o, p in ((offsets, pairs), (sane, clean)):
        order = dict(offsets=o, pairs=p.to(DEV))
        y, su = moe.moe_adapter_forward(x, a, b, ids, scale, order=order, save_u=True)
        dx, da, db = moe.moe_adapter_backward(dy, x, u, a, b, ids, scale, order=order)
        got.append((y[kept], su[kept], dx[kept], da, db))
    for p, q in zip(*got):
        assert torch.equal(p, q) and bool(torch.isfinite(p).all())
    assert bool((got[0][3][2:] == 0).all()) and bool((got[0][4][2:] == 0).all())
