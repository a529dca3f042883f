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
