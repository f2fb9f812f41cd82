"""The batch plan records what it leaves out, as the other serving operators do."""
import numpy as np
import pytest
import torch

import decoder_only_b200 as lb
from test_gpu_serving import _ints, _run_plan

pytestmark = pytest.mark.gpu


def _plan(past=(100, 0, 256), new=(30, 5, 1), table=((4, -1, -1), (-1, -1, -1), (5, 6, -1)), free=(0, 1, 2, 3), n_free=4, max_rows=64):
    lb.op_last_error()
    _run_plan(np.array(past), np.array(new), np.array(table), np.array(free), n_free, 8, max_rows, np.array([0, -1, 7]), 2)
    return lb.op_last_error()


@pytest.mark.parametrize("max_rows", [64, 4096])      # rows in the plan's kernel, and in one of their own
@pytest.mark.parametrize("bad", [
    dict(past=(-1, 0, 256)), dict(new=(30, -5, 1)), dict(past=(100, 0, 384)),              # lengths that cannot be
    dict(n_free=5), dict(n_free=-1),                                                      # a count outside the list
    dict(free=(0, 1, 2, 8)), dict(free=(0, -1, 2, 3)),                                    # a free page outside the pool
    dict(table=((9, -1, -1), (-1, -1, -1), (5, 6, -1))), dict(table=((-1, -1, -1),) * 3),   # a row's page outside it
])
def test_plan_records_what_is_out_of_range(bad, max_rows):
    assert _plan(max_rows=max_rows, **bad) == -1


@pytest.mark.parametrize("max_rows", [64, 4096])
@pytest.mark.parametrize("good", [
    dict(), dict(n_free=0), dict(n_free=2), dict(new=(0, 0, 0)), dict(new=(30, 300, 1)),      # held back is nothing wrong
    dict(free=(9, 1, 2, 3)),                                                                # nobody takes that page
    dict(table=((4, 99, -1), (77, -1, -1), (99, 6, 55))),      # entries that no row of the step is in, or that are replaced
])
def test_plan_records_nothing_where_all_is_in_range(good, max_rows):
    assert _plan(max_rows=max_rows, **good) == 0
