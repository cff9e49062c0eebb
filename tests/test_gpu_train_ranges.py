"""The training operators (include/dynconv_train.h) on the GPU over the ranges that
small cases do not reach: several turns of every kernel's main loop, the last sizes
of the types, lists whose units cross from tensor to tensor, roots next to a
rounding's border."""
import numpy as np
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


# --------------------------------------------------------------------- roots


def next_to_a_border():
    """The fp32 numbers of [1, 4) whose root lies within 2^-19 of a unit in the last place
    of the border between two fp32 numbers. A border is M 2^-24 with M odd, its square
    M^2 2^-48; a number x = M^2 2^-48 +- d 2^-48 has its root d / (4 M) units away."""
    m = np.arange(2**24 + 1, 2**25, 2, dtype=np.uint64)
    square, found = m * m, []
    for bits, inside in ((25, square < 2**49), (26, square >= 2**49)):   # x's spacing 2^(bits - 48)
        over = square[inside] & np.uint64(2**bits - 1)
        for d, sign in ((over, -1), (np.uint64(2**bits) - over, 1)):
            near = d < 4 * m[inside].astype(np.float64) * 2.0**-19
            x = square[inside][near].astype(np.int64) + sign * d[near].astype(np.int64)
            found.append(np.ldexp(x.astype(np.float64), -48))
    x = np.concatenate(found)
    assert np.array_equal(x, x.astype(np.float32)) and 60 <= len(x) <= 80
    return x


def root_states(v):
    """(scale of a block of codes 256, gradient) that a step with beta2 = 1/2 turns into
    exactly v: the largest root r whose rounded square is not above 2 v, and the root of
    what is left."""
    twice = (2.0 * v).astype(np.float32)
    r = np.sqrt(twice.astype(np.float64)).astype(np.float32)
    while True:
        over = r * r > twice
        if not over.any():
            break
        r = np.where(over, np.nextafter(r, np.float32(0)), r)
    g = np.sqrt((twice - r * r).astype(np.float64)).astype(np.float32)
    half = np.float32(0.5)
    assert np.array_equal((r * r) * half + (g * g) * half, v.astype(np.float32))
    return r * np.float32(2.0**-8), g


def check_roots(v, scale, g, beta2):
    """A step over blocks of 256 equal second moments: the scales and the codes are those
    of the correctly rounded roots of v."""
    count, step, seed = len(v), 4, 17
    spread = lambda a: torch.from_numpy(a).cuda().repeat_interleave(256)  # noqa: E731
    numel = 256 * count
    f = lambda k: torch.zeros(k, device="cuda")  # noqa: E731
    grad, param, ms = spread(g), f(numel), f(count)
    m = torch.zeros(numel, dtype=torch.uint8, device="cuda")
    code = torch.full((numel,), 0x78, dtype=torch.uint8, device="cuda")   # 256
    vs = torch.from_numpy(scale).cuda()
    tensors = dc.train_tensors([dc.train_tensor(grad=grad, param=param, m=m, v=code, m_scale=ms,
                                                v_scale=vs)])
    dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(1e-3, beta2=beta2, step=step, seed=seed)))
    torch.cuda.synchronize()
    root = np.sqrt(v.astype(np.float64)).astype(np.float32)   # (a double's root rounds innocuously)
    got = vs.cpu().numpy()
    wrong = got != root * np.float32(1 / 448)
    assert not wrong.any(), (wrong.sum(), v[wrong][:4], got[wrong][:4])
    inv = (np.float32(1) / root) * np.float32(448)
    y = np.repeat(root * inv, 256).view(np.int32)
    u = np.rint(ref.dither(seed, step, 0, numel) * 65536).astype(np.int32)
    want = ((y + (u << 4)) & -(1 << 20)).view(np.float32)
    stored = code.view(torch.float8_e4m3fn).float().cpu().numpy()
    assert np.array_equal(stored, want)


@pytest.mark.parametrize("half", range(-50, 63, 8))
def test_8_bit_roots_next_to_a_rounding_border(half):
    """The root that scales and codes come from, where Newton's step (within 2^-20 of a
    unit of the root) could round to the wrong side, from 2^-100 on and up to 2^126; the
    other numbers are further from a border than that step's error."""
    v = np.concatenate([next_to_a_border() * 4.0**k for k in range(half, min(half + 8, 63))])
    check_roots(v, *root_states(v), 0.5)


@pytest.mark.parametrize("low", [-100, 0, 125])
def test_8_bit_roots_of_many_numbers(low):
    """Both parities of the exponent from 2^low on."""
    rng = np.random.default_rng(low + 200)
    v = np.ldexp((1 + rng.random(8192)).astype(np.float32), low + rng.integers(0, 2, 8192))
    check_roots(v.astype(np.float64), *root_states(v.astype(np.float64)), 0.5)


def test_8_bit_roots_below_the_newton_steps_range():
    """Squares from 2^-149 (fp32's least) up to 2^-100."""
    g = np.exp2(np.random.default_rng(5).uniform(-74.4, -50, 8192)).astype(np.float32)
    v = g * g
    assert (v > 0).all() and (v < 2.0**-126).any()
    check_roots(v.astype(np.float64), np.zeros(len(g), np.float32), g, 0.0)


def test_8_bit_roots_of_the_last_numbers():
    """Squares up to the largest finite one."""
    last = np.float32(np.sqrt(np.finfo(np.float32).max))
    g = np.concatenate([np.linspace(last / 2, last, 4000).astype(np.float32),
                        [np.nextafter(last, np.float32(0)), last]]).astype(np.float32)
    v = g * g
    assert np.isfinite(v).all()
    check_roots(v.astype(np.float64), np.zeros(len(g), np.float32), g, 0.0)
