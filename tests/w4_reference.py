"""The 4-bit products in 64 bits, from the canonical weights, for the GPU tests."""
import torch


def weights(q, scales, zeros):
    """fp64 [n][N][K] of q uint8 [n][N][K / 2], scales and zeros [n][N][K / group]."""
    lo, hi = (q & 15).long(), (q >> 4).long()
    code = torch.stack((lo, hi), 3).reshape(q.shape[0], q.shape[1], -1)
    code = torch.where(code >= 8, code - 16, code).double()
    group = code.shape[2] // scales.shape[2]
    if zeros is not None:
        code = code - zeros.double().repeat_interleave(group, 2)
    return code * scales.double().repeat_interleave(group, 2)


def spans(offsets, n, T):
    return [(0, T)] if offsets is None else list(zip(offsets.tolist(), offsets.tolist()[1:]))


def product(x, w, offsets, backward):
    """(sums, norms): x times each row's matrix, and the 2-norm of every sum's terms."""
    x = x.double()
    out = torch.zeros((x.shape[0], w.shape[2 if backward else 1]), dtype=torch.float64)
    norm = out.clone()
    for e, (r0, r1) in enumerate(spans(offsets, w.shape[0], x.shape[0])):
        m = w[e] if backward else w[e].t()
        out[r0:r1] = x[r0:r1] @ m
        norm[r0:r1] = ((x[r0:r1] ** 2) @ (m ** 2)).sqrt()
    return out, norm
