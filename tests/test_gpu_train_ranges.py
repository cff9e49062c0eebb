"""The training operators (include/dynconv_train.h) on the GPU over the ranges that
small cases do not reach: several turns of every kernel's main loop, the last sizes
of the types, lists whose units cross from tensor to tensor, roots next to a
rounding's border."""
import pytest
import torch

import dynamic_convolution_b200 as dc

from . import train_ref as ref
from .test_gpu_balance import COEF, Case

pytestmark = pytest.mark.gpu
E = ref.E


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dynamic_convolution_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# ------------------------------------------------------------------- balance


@pytest.mark.parametrize("sigmoid", [False, True])
def test_as_many_rows_as_the_type_holds(sigmoid):
    """2^31 - 1 rows of one expert: the counts, the mean and both gradients, whose grids
    are rounded up from the rows. The mean of equal values is exact; c = coef / M / M
    times the counts is coef / M (coef and c rounded: 2 E), and a sigmoid row of one
    expert leaves none."""
    rows = 2**31 - 1
    c = Case(3, 1, 1, sigmoid=sigmoid)
    c.rows, c.desc = rows, dc.make_balance_desc(rows, 1, mode=dc.SIGMOID if sigmoid else dc.SOFTMAX)
    c.size = dc.dynconv_balance_workspace_size(c.desc)
    c.ws = torch.empty(c.size, dtype=torch.uint8, device="cuda")
    c.alpha = torch.full((rows,), 0.5, device="cuda")
    c.forward()
    c.dalpha = torch.full((rows + 1,), 5.0, device="cuda")
    c.stride = 1
    c.backward(0, dloss=False)
    torch.cuda.synchronize()
    assert c.counts[:2].tolist() == [rows, -7] and c.kept.tolist() == [rows, -7]
    assert c.mean[:2].tolist() == [1.0 if sigmoid else 0.5, -7.0]
    low, high = (float(x) for x in torch.aminmax(c.dalpha[:rows]))
    want = 0.0 if sigmoid else COEF / rows
    assert low == high and abs(low - want) <= 2 * E * want and float(c.dalpha[rows]) == 5.0
