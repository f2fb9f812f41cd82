"""batch_plan with the buffers of a plan of other sizes is refused, before any tensor is looked at (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

import decoder_only_b200 as lb


@pytest.mark.parametrize("asked", [dict(max_rows=7), dict(max_rows=9), dict(n_adapters=3), dict(max_rows=8, n_adapters=1)])
def test_plan_buffers_of_other_sizes_are_refused(asked):
    i = torch.zeros(2, dtype=torch.int32)
    out = SimpleNamespace(batch=2, max_rows=8, n_adapters=2, cu=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(lb.LlamaError, match="another max_rows or n_adapters"):
        lb.batch_plan(i, i, i.view(2, 1), i, i[:1], n_pages=4, adapter=i, out=out, **asked)


@pytest.mark.parametrize("asked", [dict(), dict(max_rows=8), dict(n_adapters=2), dict(max_rows=8, n_adapters=2)])
def test_plan_buffers_of_the_sizes_asked_for_are_not(asked):
    i = torch.zeros(2, dtype=torch.int32)
    out = SimpleNamespace(batch=2, max_rows=8, n_adapters=2, cu=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(lb.LlamaError, match="current CUDA device"):      # what CPU tensors get as far as
        lb.batch_plan(i, i, i.view(2, 1), i, i[:1], n_pages=4, adapter=i, out=out, **asked)
