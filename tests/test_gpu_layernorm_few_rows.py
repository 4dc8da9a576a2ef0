"""Layer norm with row counts around those where it goes from one row at a time to several."""

import pytest

from test_gpu_layernorm import BF16, F32, run_both

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,dtype,groups", [(64, F32, 8), (1024, BF16, 4), (1600, BF16, 2), (2048, F32, 1)])
@pytest.mark.parametrize("rows_a_group", [1, 4])
def test_row_counts_around_the_limits(dim, dtype, groups, rows_a_group):
    limit = torch.cuda.get_device_properties(0).multi_processor_count * groups * rows_a_group
    for rows in (limit - 1, limit, limit + 1):
        run_both(rows, dim, dtype, F32, rows)
