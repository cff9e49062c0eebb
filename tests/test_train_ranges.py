"""The training entry points (include/dynconv_train.h) at the ends of their ranges,
without a GPU: sizes near the integer types' last values, arguments that do not
fit."""
import pytest

import dynamic_convolution_b200 as dc
from dynamic_convolution_b200 import build as dcbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    dcbuild.build()
    return dc.load()


@pytest.mark.parametrize("n", [1, 4, 16, 300, 1024])
def test_balance_split_of_rows_up_to_the_types_last(n):
    """The workspace holds the parts of the sums: as many at 2^31 - 1 rows as at 10^9."""
    def size(rows):
        return dc.dynconv_balance_workspace_size(dc.make_balance_desc(rows, n))
    for rows in (2**31 - 1024, 2**31 - 256, 2**31 - 1):
        assert size(rows) == size(10**9)


@pytest.mark.parametrize("count", [0, 1, 768, 769, 2**31 - 768, 2**31 - 1])
def test_norm_workspace_of_any_count(count):
    """1184 fp64 parts for every 768 tensors begun, and for none."""
    assert dc.dynconv_grad_norm_workspace_size(count) == 8 * 1184 * max(1, -(-count // 768))
