"""Adapters: fp32 accuracy where sums are long, against 64 bits."""
import numpy as np
import pytest
import torch

import decoder_only_b200 as lb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _error(dtype, M, d, n, rank, room, mean=0.0, seed=0):
    """Error of each row of y relative to its norm; room: tiles that the call has room for (few are there)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, d, device="cuda", generator=g) + mean).to(dtype)
    A = ((torch.randn(2, rank, d, device="cuda", generator=g) + mean) * d ** -0.5).to(dtype)
    B = (torch.randn(2, n, rank, device="cuda", generator=g) + mean).to(dtype)
    s = torch.tensor([0.75, 1.5], device="cuda")
    tiles, rows = [], torch.arange(M, dtype=torch.int32, device="cuda")
    half = M // 2
    for a, (lo, hi) in enumerate(((0, half), (half, M))):
        tiles += [(a, t, min(64, hi - t), 0) for t in range(lo, hi, 64)]
    n_tiles = torch.tensor([len(tiles)], dtype=torch.int32, device="cuda")
    tiles = torch.tensor(tiles + [(-1, 0, 0, 0)] * (room - len(tiles)), dtype=torch.int32, device="cuda")
    y = lb.lora(x, A, B, s, torch.zeros(M, n, device="cuda"), rows, tiles, n_tiles)
    X, A, B, s = x.double(), A.double(), B.double(), s.double()
    want = torch.cat([s[a] * (X[r] @ A[a].T) @ B[a].T for a, r in ((0, slice(0, half)), (1, slice(half, M)))])
    return ((y.double() - want).norm(dim=1) / want.norm(dim=1)).max().item()


@pytest.mark.parametrize("M,d,n,rank,room", [
    (100, 13824, 64, 8, 700),       # a CTA sums all of d
    (70, 13824, 256, 256, 160),
    (33, 4096, 512, 64, 40),
    (130, 512, 1024, 256, 4),       # long sums over the rank
    (20, 13824, 1024, 128, 2),
])
@pytest.mark.parametrize("mean", [0.0, 0.5])      # signs that cancel, and sums that grow
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lora_sums_are_those_of_fp32(M, d, n, rank, room, mean, dtype):
    """Relative to a row's norm.  The matrix instructions cut what lies below an fp32 accumulator's last place: at most
    2^-23 of it each, half of that on average.  16 in a row, the accumulator growing evenly from nothing: 8 x 2^-23 = 2^-20
    at the worst, 2^-21 on average, for x A^T and again for what it is multiplied with: 2^-20 where all has one sign,
    and with the additions of the pieces, to nearest (2^-24 each on partial sums that only grow), below 2^-19.  Where
    signs cancel the cuts do too, in all but the last pieces' share, as do the additions': a quarter of that and the
    rounding of y.  h kept to two terms instead of three would be off by 2^-19.6 alone, 1.2e-6."""
    e = _error(dtype, M, d, n, rank, room, mean)
    print("relative error", e)
    assert e <= (6e-7 if mean == 0 else 2.0 ** -19), e
