"""A row's values do not depend on the rows beside it: with the same T and n, the same bits
wherever the row lies among its expert's, whatever the others hold and whomever they belong to."""
import pytest
import torch

import quantized_moe_expert_02_amd as moe
from test_gpu_w4 import BF16, DEV, F16, make, pack

pytestmark = pytest.mark.gpu


# the kernels for few and many rows, with split sums and without; T, n, N, K
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,n,N,K", [(16, 3, 200, 1280), (150, 3, 200, 1280), (150, 3, 6152, 160), (150, 300, 72, 320), (700, 2, 1000, 2080),
                                     (400, 2, 136, 320)])
def test_rows_beside(T, n, N, K, backward, dtype):
    c = make(T, K, N, n, 32, dtype, True, T + N, [0] * (n + 1), backward)
    w, x, call = pack(c), c["x"].to(DEV), moe.moe_w4_backward if backward else moe.moe_w4_forward
    print("beside", T, n, N, K, backward, dtype, flush=True)

    def run(start, rows, fill):
        """The values of `rows` rows of expert 0 (x[0], x[1], ...) from row `start` on, the others `fill`."""
        given = torch.full_like(x, fill) if fill is not None else x.flip(0)
        given[start:start + rows] = x[:rows]
        ends = [start, start + rows] + [start + rows + (T - start - rows) * e // (n - 1) for e in range(1, n)]
        return call(given, w, offsets=torch.tensor(ends, dtype=torch.int32, device=DEV))[start:start + rows]

    want = run(0, T, None)
    for start, rows, fill in ((0, 1, None), (T - 1, 1, 0.0), (3, 5, float("nan")), (1, T // 2, float("inf")), (T // 3, T // 2, None),
                              (0, T - 1, float("nan"))):
        assert torch.equal(run(start, rows, fill), want[:rows]), (start, rows, fill)
