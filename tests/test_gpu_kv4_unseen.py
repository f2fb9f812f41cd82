"""Attention over the 4-bit cache where numbers are not finite or scores vanish: what a row sees counts, what it does
not see does not, and a row that sees nothing is zeros."""
import numpy as np
import pytest
import torch

import decoder_only_b200 as lb
import _serving as ref
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
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 0.0])
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


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [
    (4, 2, 128, [40, 300, 0], [9, 6, 1]),                     # few columns
    (32, 4, 128, [100, 300, 0, 0], [100, 80, 1, 0]),          # many
    (32, 4, 64, [200, 129], [70, 129]),
])
@pytest.mark.parametrize("keys", [0.0, 2.0 ** -60])
@pytest.mark.parametrize("queries", [0.0, 2.0 ** -60])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_that_vanish_weigh_alike(H, n_kv, hd, lens, new, keys, queries, dtype):
    """Queries and keys that are zero, or as good as: a row is the mean of the values that it sees."""
    c = _attend_case(H + hd, lens, new, H, n_kv, hd, dtype)
    c["q"].mul_(queries)
    zs, put = _scales(c, hd)
    if keys == 0:
        zs[..., 0, :, :] = 0
    else:
        zs[..., 0, :, :] -= 60 << 7                           # 2^-60 of what they were
    put()
    o = _attend(c).double().cpu().numpy()
    _, V, _, _ = ref.unpack(c["pool"], hd)
    half = 2.0 ** -9 if dtype == BF16 else 2.0 ** -24
    for b, (length, n) in enumerate(zip(lens, new)):
        for i in range(n):
            seen, row = length - n + i + 1, o[c["cu"][b] + i].reshape(H, hd)
            if seen <= 0:
                assert not row.any()
                continue
            for h in range(H):
                v = np.concatenate([V[p, h * n_kv // H] for p in c["table"][b][: -(-length // 128)]])[:seen]
                mean, most = v.mean(0), np.abs(v).max(0)
                # weights are one in every precision; values (many columns: fp16, 2^-12 of them next to a largest of 16
                # times as much at most) and weights times steps (fp16 again, 31 steps) are off by half a place each
                off = half * np.abs(mean) + (2.0 ** -6 if dtype == BF16 else 2.0 ** -18) * most
                assert np.all(np.abs(row[h] - mean) <= off), (b, i, h)
    assert lb.op_last_error() == 0
