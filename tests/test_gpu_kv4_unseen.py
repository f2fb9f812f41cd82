"""Attention over the 4-bit cache where numbers are not finite or scores vanish: what a row sees counts, what it does
not see does not, and a row that sees nothing is zeros."""
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
