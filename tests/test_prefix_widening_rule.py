"""When the partitioner widens: where the copy, its kernels and the join cost less than the conversion."""
import pytest

from test_prefix_partition import _case, runner  # noqa: F401


@pytest.mark.parametrize("kv", [1, 2])
def test_a_copy_that_costs_more_than_it_saves_is_not_made(runner, kv):  # noqa: F811
    # (measured longer when widened: 16 groups of 4 row groups and 70 tiles by a fifth over 4 bits)
    _case(runner, [16] * 16, [4480] * 16, lambda i: 128, [1], 32, False, True, kv, 76, uniform=True, wide=False)
    _case(runner, [16] * 4, [16384] * 4, lambda i: 128, [1], 32, False, True, kv, 76, uniform=True, wide=False)
    _case(runner, [4] * 12, [8192] * 12, lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=False)
    _case(runner, [24], [16384], lambda i: 128, [1], 32, False, True, kv, 76, uniform=True, wide=False)
    _case(runner, [16], [2048], lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=False)


@pytest.mark.parametrize("kv", [1, 2])
def test_long_rows_behind_many_row_groups_are_widened(runner, kv):  # noqa: F811
    _case(runner, [32], [8192], lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=True)
    _case(runner, [16], [20480], lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=True)
    _case(runner, [64], [16384], lambda i: 128, [1], 32, False, True, kv, 76, uniform=True, wide=True)
    _case(runner, [8] * 4, [20480] * 4, lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=True)
    _case(runner, [16] * 12, [8192] * 12, lambda i: 128, [1], 128, False, True, kv, 76, uniform=True, wide=True)
