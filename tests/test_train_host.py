"""The training entry points (include/dynconv_train.h) without a GPU: the symbols
are there, the header is C, every refusal happens on the host before any CUDA
call, what is valid fails loudly with no device, and the reference that the GPU
tests compare with is itself pinned (central differences, torch.optim.AdamW,
torch's e4m3, the dither's mean)."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import dynamic_convolution_b200 as dc
from dynamic_convolution_b200 import build as dcbuild

from . import train_ref as ref

HEADER = os.path.join(dcbuild.ROOT, "include", "dynconv_train.h")
P = 256   # an aligned address that is never read
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


@pytest.fixture(scope="module", autouse=True)
def lib():
    dcbuild.build()
    return dc.load()


def test_symbols(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dynconv_[a-z_]+)\s*\(", text)))
    assert names == sorted(dc.TRAIN_SYMBOLS)
    for name in names:
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


def test_header_is_c_and_layouts_agree(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "dynconv_train.h"\n'
                   'int main(void) { printf("%zu %zu %zu\\n", sizeof(dynconv_balance_desc),'
                   ' sizeof(dynconv_train_tensor), sizeof(dynconv_adamw_hyper)); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    f"-I{dcbuild.INCLUDE}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == [str(ctypes.sizeof(t)) for t in
                           (dc.dynconv_balance_desc, dc.dynconv_train_tensor,
                            dc.dynconv_adamw_hyper)]


# ------------------------------------------------------------------- balance


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), dc.ERR_INVALID_ARG), (dict(n=0), dc.ERR_INVALID_ARG),
    (dict(groups=0), dc.ERR_INVALID_ARG), (dict(top_k=0), dc.ERR_INVALID_ARG),
    (dict(top_k=5), dc.ERR_INVALID_ARG), (dict(mode=2), dc.ERR_INVALID_ARG),
    (dict(row_stride=3), dc.ERR_INVALID_ARG), (dict(n=1025), dc.ERR_UNSUPPORTED),
    (dict(n=1, groups=65536), dc.ERR_UNSUPPORTED), (dict(n=64, top_k=33), dc.ERR_UNSUPPORTED), (dict(n=1024, groups=65), dc.ERR_UNSUPPORTED),
    (dict(row_stride=1 << 40), dc.ERR_UNSUPPORTED)])
def test_balance_descriptors_refused(kw, code):
    d = dc.make_balance_desc(**{**dict(rows=8, n=4), **kw})
    assert dc.dynconv_balance_workspace_size(d) == 0
    assert dc.dynconv_balance_forward(d, P, None, 0.01, P, P, P, P, P, 1 << 30) == code
    assert dc.dynconv_balance_backward(d, P, None, 0.01, P, P, None, P, 1 << 20, 0) == code


def test_balance_arguments_refused():
    d = dc.make_balance_desc(8, 4)
    need = dc.dynconv_balance_workspace_size(d)
    assert need > 0
    f, b = dc.dynconv_balance_forward, dc.dynconv_balance_backward
    good = [P, None, 0.01, P, P, P, P, P, need]
    for at in (0, 3, 4, 5, 6):
        bad = list(good)
        bad[at] = None
        assert f(d, *bad) == dc.ERR_INVALID_ARG
        bad[at] = P + 2
        assert f(d, *bad) == dc.ERR_MISALIGNED
    assert f(d, P, None, math.inf, P, P, P, P, P, need) == dc.ERR_INVALID_ARG
    assert f(d, P, None, 0.01, P, P, P, P, None, need) == dc.ERR_WORKSPACE
    assert f(d, P, None, 0.01, P, P, P, P, P, need - 1) == dc.ERR_WORKSPACE
    assert f(d, P, None, 0.01, P, P, P, P, P + 8, need) == dc.ERR_MISALIGNED
    s = dc.make_balance_desc(8, 4, mode=dc.SIGMOID)
    assert b(s, None, None, 0.01, P, P, None, P, 4, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, None, P, None, P, 4, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, P, None, None, P, 4, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, P, P, None, None, 4, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, math.nan, P, P, None, P, 4, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, P, P, None, P, 3, 0) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, P, P, None, P, 4, 2) == dc.ERR_INVALID_ARG
    assert b(d, P, None, 0.01, P, P, None, P, 1 << 40, 0) == dc.ERR_UNSUPPORTED
    assert b(d, P, None, 0.01, P, P, P + 1, P, 4, 0) == dc.ERR_MISALIGNED
    assert b(d, P, None, 0.01, P, P, None, P + 2, 4, 0) == dc.ERR_MISALIGNED
    # no rows: nothing to write
    none = dc.make_balance_desc(0, 4)
    assert b(none, None, None, 0.01, P, P, None, None, 4, 0) == dc.OK


@no_device
def test_balance_without_a_device_fails_loudly():
    d = dc.make_balance_desc(8, 4)
    need = dc.dynconv_balance_workspace_size(d)
    assert dc.dynconv_balance_forward(d, P, None, 0.01, P, P, P, P, P, need) == dc.ERR_CUDA
    assert dc.dynconv_balance_backward(d, None, None, 0.01, P, P, None, P, 4, 0) == dc.ERR_CUDA
    assert dc.dynconv_last_error() != ""


# ------------------------------------------------------------ lists of tensors


def entry(**kw):
    base = dict(param=P, master=0, grad=P, m=P, v=P, m_scale=0, v_scale=0, numel=8, dtype=dc.F32,
                grad_dtype=dc.F32, state_bits=32, lr_scale=1.0, weight_decay=0.0)
    base.update(kw)
    return dc.dynconv_train_tensor(*[base[f] for f, _ in dc.dynconv_train_tensor._fields_])


def adamw(entries, **kw):
    return dc.dynconv_adamw(dc.train_tensors(entries), dc.make_adamw(**{**dict(lr=1e-3), **kw}))


@pytest.mark.parametrize("kw,code", [
    (dict(param=0), dc.ERR_INVALID_ARG), (dict(grad=0), dc.ERR_INVALID_ARG),
    (dict(m=0), dc.ERR_INVALID_ARG), (dict(v=0), dc.ERR_INVALID_ARG),
    (dict(numel=-1), dc.ERR_INVALID_ARG), (dict(dtype=2), dc.ERR_INVALID_ARG),
    (dict(grad_dtype=-1), dc.ERR_INVALID_ARG), (dict(master=P), dc.ERR_INVALID_ARG),
    (dict(state_bits=8), dc.ERR_INVALID_ARG),
    (dict(state_bits=8, m_scale=P), dc.ERR_INVALID_ARG),
    (dict(lr_scale=-1.0), dc.ERR_INVALID_ARG), (dict(lr_scale=math.nan), dc.ERR_INVALID_ARG),
    (dict(weight_decay=math.inf), dc.ERR_INVALID_ARG), (dict(weight_decay=-0.1), dc.ERR_INVALID_ARG),
    (dict(state_bits=16), dc.ERR_UNSUPPORTED), (dict(numel=1 << 40), dc.ERR_UNSUPPORTED),
    (dict(param=P + 2), dc.ERR_MISALIGNED), (dict(grad=P + 2), dc.ERR_MISALIGNED),
    (dict(m=P + 1), dc.ERR_MISALIGNED), (dict(dtype=dc.BF16, master=P + 2), dc.ERR_MISALIGNED),
    (dict(dtype=dc.BF16, param=P + 1), dc.ERR_MISALIGNED),
    (dict(state_bits=8, m_scale=P + 1, v_scale=P), dc.ERR_MISALIGNED)])
def test_adamw_tensors_refused(kw, code):
    assert adamw([entry(**kw)]) == code
    assert adamw([entry(), entry(**{**dict(param=4096), **kw})]) == code   # wherever it stands


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf),
                                dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                                dict(beta2=math.nan), dict(eps=0.0), dict(eps=math.inf),
                                dict(step=0)])
def test_adamw_hyper_refused(kw):
    assert adamw([entry()], **kw) == dc.ERR_INVALID_ARG


def test_adamw_refuses_a_param_given_twice():
    assert adamw([entry(), entry()]) == dc.ERR_INVALID_ARG
    assert "twice" in dc.dynconv_last_error()
    # in any order, also when one only overlaps another
    assert adamw([entry(param=4096), entry(param=256), entry(param=4096 + 28)]) == dc.ERR_INVALID_ARG
    # an empty tensor has no range
    code = dc.OK if torch.cuda.is_available() else dc.ERR_CUDA
    assert adamw([entry(numel=0), entry(numel=0, param=0, grad=0, m=0, v=0)]) == code


def test_adamw_list_refused():
    hyper = dc.make_adamw(1e-3)
    lib = dc.load()
    assert lib.dynconv_adamw(None, 1, ctypes.byref(hyper), None, None, None,
                             None) == dc.ERR_INVALID_ARG
    assert lib.dynconv_adamw(None, -1, ctypes.byref(hyper), None, None, None,
                             None) == dc.ERR_INVALID_ARG
    one = dc.train_tensors([entry()])
    assert lib.dynconv_adamw(one, 1, None, None, None, None, None) == dc.ERR_INVALID_ARG
    for kw in (dict(grad_scale=P + 2), dict(lr=P + 2), dict(step=P + 4)):
        assert dc.dynconv_adamw(one, hyper, **kw) == dc.ERR_MISALIGNED


def test_grad_norm_refused():
    one = dc.train_tensors([entry()])
    need = dc.dynconv_grad_norm_workspace_size(one)
    f = dc.dynconv_grad_norm
    assert f(one, 0.0, P, None, P, need) == dc.ERR_INVALID_ARG
    assert f(one, math.nan, P, None, P, need) == dc.ERR_INVALID_ARG
    assert f(one, 1.0, None, None, P, need) == dc.ERR_INVALID_ARG
    assert f(dc.train_tensors([entry(grad=0)]), 1.0, P, None, P, need) == dc.ERR_INVALID_ARG
    assert f(dc.train_tensors([entry(numel=1 << 40)]), 1.0, P, None, P, need) == dc.ERR_UNSUPPORTED
    assert f(one, 1.0, P, None, None, need) == dc.ERR_WORKSPACE
    assert f(one, 1.0, P, None, P, need - 1) == dc.ERR_WORKSPACE
    assert f(one, 1.0, P, None, P + 8, need) == dc.ERR_MISALIGNED
    assert f(one, 1.0, P, P + 4, P, need) == dc.ERR_MISALIGNED
    assert dc.dynconv_grad_norm_workspace_size(-1) == 0
    assert dc.dynconv_grad_norm_workspace_size(100_000) > need


@no_device
def test_optimizer_without_a_device_fails_loudly():
    one = dc.train_tensors([entry()])
    assert dc.dynconv_adamw(one, dc.make_adamw(1e-3)) == dc.ERR_CUDA
    assert dc.dynconv_grad_norm(one, math.inf, P, None, P, 1 << 20) == dc.ERR_CUDA
    assert dc.dynconv_last_error() != ""


def test_lists_of_tensors_on_the_host_are_refused():
    f = lambda: torch.zeros(8)  # noqa: E731
    tensors = dc.train_tensors([dc.train_tensor(grad=f(), param=f(), m=f(), v=f())])
    assert dc.dynconv_adamw(tensors, dc.make_adamw(1e-3)) == dc.ERR_INVALID_ARG
    assert dc.dynconv_grad_norm(tensors, 1.0, P, None, P, 1 << 20) == dc.ERR_INVALID_ARG


def test_train_tensor_checks_what_it_is_given():
    f = lambda n=8, t=torch.float32: torch.zeros(n, dtype=t)  # noqa: E731
    e = dc.train_tensor(grad=f(), param=f(), m=f(), v=f(), weight_decay=0.5)
    assert (e.numel, e.dtype, e.grad_dtype, e.state_bits, e.weight_decay) == (8, dc.F32, dc.F32, 32, 0.5)
    e = dc.train_tensor(grad=f(8, torch.bfloat16))
    assert (e.grad_dtype, e.param) == (dc.BF16, None)
    fp8 = torch.float8_e4m3fn
    e = dc.train_tensor(grad=f(300), param=f(300, torch.bfloat16), master=f(300), m=f(300, fp8),
                        v=f(300, fp8), m_scale=f(2), v_scale=f(2))
    assert (e.state_bits, e.dtype) == (8, dc.BF16)
    # a list keeps its tensors alive
    import gc
    import weakref
    grad = f(8)
    alive = weakref.ref(grad)
    tensors = dc.train_tensors([dc.train_tensor(grad=grad)])
    del grad
    gc.collect()
    assert alive() is not None and tensors[0].grad == alive().data_ptr()
    del tensors
    gc.collect()
    assert alive() is None
    bad = [dict(grad=f(8, torch.float16)), dict(grad=f().view(2, 4).t()),
           dict(grad=f(), param=f()), dict(grad=f(), param=f(9), m=f(), v=f()),
           dict(grad=f(), param=f(8, torch.float64), m=f(), v=f()),
           dict(grad=f(), param=f(), m=f(), v=f(8, fp8)),
           dict(grad=f(), param=f(), m=f(8, fp8), v=f(8, fp8)),
           dict(grad=f(), param=f(), m=f(8, fp8), v=f(8, fp8), m_scale=f(2), v_scale=f(1)),
           dict(grad=f(), param=f(), m=f(), v=f(), m_scale=f(1), v_scale=f(1)),
           dict(grad=f(), param=f(), m=f(), v=f(), master=f()),
           dict(grad=f(), param=f(8, torch.bfloat16), m=f(), v=f(), master=f(8, torch.bfloat16)),
           dict(grad=f(), param=torch.zeros(8, device="meta"), m=f(), v=f())]
    for kw in bad:
        with pytest.raises(ValueError):
            dc.train_tensor(**kw)


# ------------------------------------------------------- the reference's own pins


@pytest.mark.parametrize("sigmoid", [False, True])
def test_reference_balance_gradient_against_differences(sigmoid):
    rng = np.random.default_rng(3)
    a = rng.random((7, 2, 5)) + 0.1
    mask = np.array([1, 1, 0, 1, 1, 1, 0])
    r = ref.balance(a, mask, 2, sigmoid, 0.3)
    g, _ = ref.balance_grad(a, mask, r["counts"], 2, sigmoid, 0.3, 1.7)
    assert r["counts"].sum() == 2 * 2 * r["kept"] and r["kept"] == 5
    assert np.isclose(r["loss"], ref.balance_loss(a, mask, r["counts"], 2, sigmoid, 0.3))
    h = 1e-6
    for at in np.ndindex(a.shape):
        up, down = a.copy(), a.copy()
        up[at] += h
        down[at] -= h
        d = [ref.balance_loss(x, mask, r["counts"], 2, sigmoid, 0.3) for x in (up, down)]
        assert abs(1.7 * (d[0] - d[1]) / (2 * h) - g[at]) < 1e-8


def test_reference_balance_of_even_routing_is_the_coefficient():
    a = np.eye(4)[np.arange(8) % 4][:, None, :]
    assert np.isclose(ref.balance(a, None, 1, False, 0.25)["loss"], 0.25)


def test_reference_adamw_against_torch():
    rng = np.random.default_rng(4)
    p, g1, g2 = (rng.standard_normal(33) for _ in range(3))
    t = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([t], lr=0.01, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(33)
    for step, g in ((1, g1), (2, g2)):
        t.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v, *_ = ref.adamw(p, g, m, v, lr=0.01, beta1=0.9, beta2=0.99, eps=1e-8, step=step,
                                decay=0.1)
    assert np.allclose(t.detach().numpy(), p, rtol=1e-12, atol=1e-14)


def test_reference_e4m3_grid_and_dither():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.to_e4m3(codes, np.full(127, 0.999)), codes)   # the grid stays
    assert np.array_equal(ref.to_e4m3(codes, np.zeros(127)), codes)
    y = np.random.default_rng(5).random(2000) ** 4 * 448
    near = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.mean(ref.to_e4m3(y, np.full(2000, 0.5)) == near) > 0.99       # ties apart
    u = ref.dither(9, 3, 1, 1 << 16)
    assert abs(u.mean() - 0.5) < 4 / math.sqrt(12 * (1 << 16)) and 0 <= u.min() and u.max() < 1
    assert abs(np.corrcoef(u[:-1], u[1:])[0, 1]) < 4 / 256
    x = np.full(1 << 16, 100.3)
    assert abs(ref.to_e4m3(x, u).mean() - 100.3) < 4 * 4 / 256              # no bias
    b = torch.randn(1000).bfloat16().double().numpy()
    assert np.array_equal(ref.to_bf16_dithered(b, u[:1000]), b)
