"""The README's example, run as it stands: the balance gradient reaches the router's
gradients and the input's, and every parameter is in the norm and the step."""
import os
import re

import pytest
import torch

import dynamic_convolution_b200 as dc
from dynamic_convolution_b200 import build as dcbuild

pytestmark = pytest.mark.gpu


def example():
    """The indented code under the README's example heading."""
    text = open(os.path.join(dcbuild.ROOT, "README.md")).read()
    section = re.split(r"^## ", text.split("## Example", 1)[1], flags=re.M)[0]
    return "\n".join(line[4:] for line in section.splitlines() if line.startswith("    "))


def test_readme_example_trains_what_it_describes(monkeypatch):
    dcbuild.build()
    torch.manual_seed(3)
    seen = {}

    def watch(name, position):
        """Keeps the argument at `position` as it was before and after the call."""
        call = getattr(dc, name)

        def watched(*args, **kw):
            before = args[position].clone()
            status = call(*args, **kw)
            seen[name] = (before, args[position].clone())
            return status
        monkeypatch.setattr(dc, name, watched)

    watch("dynconv_balance_backward", 7)
    watch("dynconv_route_backward", 4)
    e = {}
    exec(example(), e)
    torch.cuda.synchronize()
    assert dc.dynconv_device_status(None) == dc.OK
    # dalpha has the balance gradient (not zero) in it when the router's gradients are taken
    layer, joined = seen["dynconv_balance_backward"]
    assert torch.equal(joined, seen["dynconv_route_backward"][0])
    alone = torch.empty_like(layer)
    dc.check(dc.dynconv_balance_backward(e["bd"], e["alpha"], None, 0.01, e["counts"], e["kept"],
                                         None, alone, e["n"], 0))
    torch.cuda.synchronize()
    c = 0.01 * e["n"] * e["counts"].double() / e["B"] ** 2
    assert bool(c.any()) and torch.allclose(alone.double(), c.expand(e["B"], -1), rtol=1e-6)
    assert torch.equal(layer + alone, joined)
    # the norm is that of every parameter's gradient
    norm = sum(float((e[g].double() ** 2).sum()) for g in ("dE", "dbias", "dWr", "dbr")) ** 0.5
    assert abs(float(e["stats"][0]) - norm) <= 1.01 * 2.0 ** -24 * norm and int(e["step"]) == 1
    # the biases start at zero: the first step moves them by the rate, against the gradient
    # (quotient, rate, factor and moments each rounded: well below 32 half steps)
    for param, grad in (("bias", "dbias"), ("br", "dbr")):
        x = e[grad].double() * float(e["stats"][1])
        want = -1e-3 * x / (x.abs() + 1e-8)
        assert bool(((e[param].double() - want).abs() <= 32 * 2.0 ** -24 * want.abs()).all()), param
