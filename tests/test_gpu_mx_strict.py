"""GPU: the products of test_gpu_mx.py and test_gpu_mx_use.py once more, under the
comparison of mx_strict.py, which a NaN does not pass."""
import pytest

pytest.importorskip("torch")

import mx_strict  # noqa: E402
import test_gpu_mx as products  # noqa: E402
import test_gpu_mx_use as use  # noqa: E402
from test_gpu_mx import (test_grouped, test_grouped_of_1024_groups,  # noqa: E402,F401
                         test_grouped_of_many_groups_and_each_tile, test_grouped_rows_out_of_range_give_zeros,
                         test_linear, test_linear_in_slices, test_linear_of_each_tile,
                         test_linear_of_float_rows_and_ceil, test_linear_streamed, test_most_inputs, w4)
from test_gpu_mx_use import (test_experts_past_2_to_32_bytes, test_more_rows_than_one_launch_quantises,  # noqa: E402,F401
                             test_offsets_that_do_not_ascend_stay_inside, test_outputs_past_2_to_32_bytes,
                             test_router_and_experts_together)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    for module in (products, use):
        monkeypatch.setattr(module, "check", mx_strict.check)
