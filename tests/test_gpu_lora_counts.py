"""Adapters: a count of tiles outside the list is recorded; the tiles that are there are used."""
import pytest
import torch

import decoder_only_b200 as lb
from test_gpu_serving import BF16, F32, _ints, _lora_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lora_count_of_tiles_outside_the_list_is_recorded(dtype):
    plan, x, A, B, s, y, want, mag, _ = _lora_case(21, 100, 64, 32, 8, 3, 5, dtype)
    n = int(plan.n_tiles)
    tiles = plan.lora_tiles[:n].clone()
    good = lb.lora(x, A, B, s, y.clone(), plan.lora_rows, tiles, _ints([n]))
    lb.op_last_error()
    assert torch.equal(lb.lora(x, A, B, s, y.clone(), plan.lora_rows, tiles, _ints([n + 1])), good)
    assert lb.op_last_error() == -1
    assert torch.equal(lb.lora(x, A, B, s, y.clone(), plan.lora_rows, tiles, _ints([-1])), y)
    assert lb.op_last_error() == -1
    lb.lora(x, A, B, s, y.clone(), plan.lora_rows, tiles, _ints([n]))
    assert lb.op_last_error() == 0
