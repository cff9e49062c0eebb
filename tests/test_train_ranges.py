"""The training entry points (include/dynconv_train.h) at the ends of their ranges,
without a GPU: sizes near the integer types' last values, arguments that do not
fit."""
import pytest
import torch

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


@pytest.mark.parametrize("kw", [dict(rows=2**32 + 8), dict(rows=2**31), dict(rows=-2**31 - 1),
                                dict(n=2**32 + 4), dict(groups=2**32 + 1), dict(top_k=2**32 + 1),
                                dict(mode=2**32), dict(row_stride=2**64 + 4)])
def test_numbers_that_a_descriptor_cannot_hold_are_refused(kw):
    """(2^32 + 8 rows would be taken for 8.)"""
    good = dict(rows=8, n=4)
    assert dc.make_balance_desc(**good).rows == 8
    assert dc.make_balance_desc(2**31 - 1, 4).rows == 2**31 - 1
    with pytest.raises(ValueError):
        dc.make_balance_desc(**{**good, **kw})


def test_step_numbers_that_64_bits_cannot_hold_are_refused():
    assert dc.make_adamw(1e-3, step=2**63 - 1, seed=2**32 + 3).step == 2**63 - 1
    assert dc.make_adamw(1e-3, seed=2**32 + 3).seed == 3
    with pytest.raises(ValueError):
        dc.make_adamw(1e-3, step=2**64 + 1)


def test_host_tensors_in_place_of_device_scalars_are_refused():
    """A rate, a step number, a factor or a workspace left on the host would be read by
    the kernels through its host address."""
    P = 256   # an aligned address that is never read
    entry = dc.dynconv_train_tensor(P, None, P, P, P, None, None, 0, dc.F32, dc.F32, 32, 1.0, 0.0)
    tensors, hyper = dc.train_tensors([entry]), dc.make_adamw(1e-3)
    one, number = torch.ones(1), torch.ones(1, dtype=torch.int64)
    for kw in (dict(lr=one), dict(grad_scale=one), dict(step=number)):
        assert dc.dynconv_adamw(tensors, hyper, **kw) == dc.ERR_INVALID_ARG
    byte = torch.empty(1 << 20, dtype=torch.uint8)
    for stats, step, ws in ((torch.zeros(2), None, P), (P, number, P), (P, None, byte)):
        assert dc.dynconv_grad_norm(tensors, 1.0, stats, step, ws, 1 << 20) == dc.ERR_INVALID_ARG
