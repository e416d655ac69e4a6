"""Expert plans whose waves hand an expert's next row from one step of 64 pairs to
the next, in other lanes each time.  Whole numbers, all equal."""
import numpy as np
import pytest

from test_gpu_moe_route import check_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [512, 4096, 4160, 20000, 131072 + 77])
@pytest.mark.parametrize("experts", [1, 2, 3, 63, 64, 65, 1000])
def test_next_rows_pass_between_lanes(pairs, experts):
    """Expert e's first pair of step s is in lane (e + 5 s) % 64: up to 64 experts
    every step takes on the rows of the one before it in another lane.  Then every
    second pair at expert 0, and steps of one expert each."""
    p = np.arange(pairs)
    for ids in ((p % 64 - 5 * (p // 64)) % 64 % experts, np.where(p % 2, p % experts, 0), p // 64 % experts,
                np.where(p // 64 % 3 == 1, -1, p // 7 % experts)):
        check_plan(ids.reshape(-1, 1), experts)
