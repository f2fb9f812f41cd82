"""Attention over the 4-bit cache where numbers are not finite or scores vanish: what a row sees counts, what it does
not see does not, and a row that sees nothing is zeros."""
import numpy as np
import pytest
import torch

import decoder_only_b200 as lb
from test_gpu_serving import _attend, _attend_case, _scales

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_seen_nan_value_shows_whatever_its_weight_and_wherever_the_sequence_ends(hd, dtype):
    """Position 35 has a key whose weight underflows and NaN in its values' first 64 channels: 0 * NaN is NaN, in a
    sequence that ends with its block of 32 positions (64) and in one that ends inside it (60)."""
    c = _attend_case(hd, [64, 60], [1, 1], 4, 2, hd, dtype)
    c["q"].abs_()
    zs, put = _scales(c, hd)
    for b in range(2):
        at = zs[c["table"][b, 0], :, 1, :, 3]         # [heads, keys or values, groups, (z, s)]
        at[:, 0] = [0xc47a, 0x0000]                   # keys: -1000, no step
        at[:, 1, 0] = 0x7fc0
    put()
    o = _attend(c).view(2, 4, hd)
    want = torch.zeros_like(o, dtype=torch.bool)
    want[..., :64] = True
    assert torch.equal(o.isnan(), want) and lb.op_last_error() == 0


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [
    (6, 2, 64, [3, 200, 0, 10], [7, 100, 2, 0]),              # few columns
    (4, 4, 128, [20, 0], [25, 3]),
    (40, 8, 128, [80, 200, 20, 90], [90, 150, 60, 100]),      # many
    (16, 16, 64, [100, 0, 300], [300, 5, 290]),
])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_nothing_are_zeros_whatever_their_query(H, n_kv, hd, lens, new, bad, dtype):
    c = _attend_case(H + hd, lens, new, H, n_kv, hd, dtype, poison=True)
    good = _attend(c)
    blind = np.zeros(len(c["q"]), bool)
    for b, n in enumerate(new):
        blind[c["cu"][b]:c["cu"][b] + max(n - lens[b], 0)] = True
    c["q"][torch.from_numpy(blind).cuda()] = bad
    o = _attend(c)
    assert blind.any() and not o[torch.from_numpy(blind).cuda()].any()
    assert torch.equal(o, good) and lb.op_last_error() == 0
