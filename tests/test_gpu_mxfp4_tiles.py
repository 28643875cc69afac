"""Every tile of the MXFP4 products on the GPU, with several turns of its ring, ragged rows and columns, an odd number of 128 columns
of K, bias and all output types, against sums in 64 bits. Sampled rows are compared over all columns and sampled columns over
all rows. test_mxfp4_tiles.py holds that each size takes the tile it stands for."""
import pytest
import torch

import decode_tile_interleaved_rans_amd as ep
import mx_reference as mx

SIZES = [((256, 256, 1), 3900, 8100, 2432), ((256, 192, 1), 1500, 6005, 3968), ((256, 128, 1), 701, 8001, 4224), ((128, 128, 1), 500, 8190, 2176),
         ((128, 64, 1), 333, 5003, 3968), ((64, 64, 1), 250, 4090, 2432), ((32, 32, 2), 61, 4090, 4224), ((32, 32, 2), 150, 1001, 2176),
         ((16, 32, 2), 5, 11510, 3968), ((16, 32, 2), 17, 2050, 4992), ((16, 32, 4), 1, 4090, 16512), ((16, 32, 4), 23, 515, 20608)]

# rows per expert, rows behind, N, K: 16 x 64, 64 x 128 (twice), 128 x 128 (twice), 256 x 256, 256 x 192, each with the 128-row form for few rows
EXPERTS = [([2, 0, 1, 3, 2, 0, 2, 1], 1, 515, 4224), ([17, 3, 0, 20, 9], 2, 1001, 3200), ([64, 66, 41], 0, 515, 3200), ([30, 0, 41, 25], 5, 1001, 2176),
           ([129, 70, 1, 200], 0, 515, 2176), ([700, 300, 100, 257], 3, 8190, 2176), ([300, 515, 128, 640], 9, 380, 2176)]


def sampled(n, g):
    """Positions of 0 ... n - 1: the first and last few and 24 others."""
    return torch.unique(torch.cat([torch.arange(min(n, 3)), torch.randint(0, n, (24,), generator=g), torch.arange(max(0, n - 20), n)]))


def rows_of(q, s, rows):
    return mx.values(q[rows].contiguous(), s[:, rows].contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("tile,M,N,K", SIZES)
def test_every_tile(tile, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    (xq, xs), (wq, ws) = mx.random_matrix(g, M, K), mx.random_matrix(g, N, K)
    bias = torch.randn(N, generator=g).to(torch.bfloat16)
    ms, ns = sampled(M, g), sampled(N, g)
    x, w = mx.values(xq, xs), mx.values(wq, ws)
    dev = [t.cuda() for t in (xq, xs, wq, ws)]
    for dtype, b in ((torch.float32, bias), (torch.bfloat16, None), (torch.float16, bias)):
        y = ep.gemm_mxfp4(*dev, b.cuda() if b is not None else None, out_dtype=dtype)
        assert y.shape == (M, N) and torch.equal(y, ep.gemm_mxfp4(*dev, b.cuda() if b is not None else None, out_dtype=dtype))
        y = y.cpu()
        mx.check_product(y[ms], x[ms], w, b, f"rows, {dtype}")
        mx.check_product(y[:, ns], x, w[ns], b[ns] if b is not None else None, f"columns, {dtype}")


@pytest.mark.gpu
@pytest.mark.parametrize("counts,behind,N,K", EXPERTS)
def test_every_tile_of_experts(counts, behind, N, K):
    g = torch.Generator().manual_seed(sum(counts) + N)
    E, R = len(counts), sum(counts) + behind
    (xq, xs), (wq, ws) = mx.random_matrix(g, R, K), mx.random_matrix(g, E, N, K)
    bias = torch.randn((E, N), generator=g).to(torch.bfloat16)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    dev = [t.cuda() for t in (xq, xs, wq, ws, offsets)]
    for dtype, b in ((torch.float32, bias), (torch.bfloat16, None), (torch.float16, bias)):
        y = ep.gemm_mxfp4_experts(*dev, b.cuda() if b is not None else None, out_dtype=dtype).cpu()
        for e in range(E):
            lo, hi = offsets[e].item(), offsets[e + 1].item()
            if lo == hi:
                continue
            ms = lo + sampled(hi - lo, g)
            mx.check_product(y[ms], rows_of(xq, xs, ms), mx.values(wq[e], ws[e]), None if b is None else b[e], f"expert {e}, {dtype}")
        assert not y[offsets[-1]:].any()
