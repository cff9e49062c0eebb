"""The training operators (include/dynconv_train.h) on the GPU over the ranges that
small cases do not reach: several turns of every kernel's main loop, the last sizes
of the types, lists whose units cross from tensor to tensor, roots next to a
rounding's border."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import dynamic_convolution_b200 as dc
from dynamic_convolution_b200.build import ROOT

from . import train_ref as ref
from .test_gpu_balance import COEF, Case
from .test_gpu_optim import HYPER, KINDS, Tensor, step_and_check

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


@pytest.fixture
def sorted_reference(monkeypatch):
    """train_ref.balance with its top k from one stable sort (NaN last), for many rows."""
    def balance(alpha, mask, k, sigmoid, coef):
        rows, groups, n = alpha.shape
        a = torch.from_numpy(alpha if mask is None else alpha[mask.astype(bool)]).cuda()
        M = a.shape[0]
        key = torch.where(a.isnan(), -float("inf"), a)
        chosen = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]
        counts = torch.zeros(groups, n, dtype=torch.int64, device="cuda")
        counts.scatter_add_(1, chosen.transpose(0, 1).reshape(groups, M * k),
                            torch.ones(groups, M * k, dtype=torch.int64, device="cuda"))
        p = a / a.sum(-1, keepdim=True) if sigmoid else a
        mean = p.sum(0) / max(M, 1)
        loss = coef * n / (k * groups) * float((counts / max(M, 1) * mean).sum())
        return dict(counts=counts.cpu().numpy(), mean=mean.cpu().numpy(), kept=M, loss=loss)

    a = np.round(np.random.default_rng(0).random((40, 2, 9)) * 6) / 6
    mask = np.arange(40) % 3
    x, y = balance(a, mask, 3, True, 0.5), ref.balance(a, mask, 3, True, 0.5)
    assert np.array_equal(x["counts"], y["counts"]) and x["kept"] == y["kept"]
    assert np.allclose(x["mean"], y["mean"], rtol=1e-13) and np.isclose(x["loss"], y["loss"])
    monkeypatch.setattr(ref, "balance", balance)


# rows: beyond one turn of 148 CTAs of 1024, 512 or 384 threads, whose warps hold 32 / L rows
# (L = 1, 1, 2, 4, 8, 16, 32, 32, then 32 with 16 or 32 values a lane)
LONG = [(3, 160_001, 0), (8, 160_001, 0), (15, 80_011, 1), (16, 80_011, 4), (32, 40_009, 0),
        (33, 20_011, 0), (64, 20_011, 8), (100, 10_007, 4), (200, 10_007, 0), (256, 15_001, 0)]
WIDE = [(300, 7103, 4), (511, 7103, 0), (512, 7103, 0), (999, 5329, 0), (1000, 5329, 24),
        (1024, 5329, 0)]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n,rows,pad", LONG + WIDE)
def test_several_turns_with_masked_rows(sorted_reference, n, rows, pad, sigmoid):
    Case(rows, n, min(n - 1, 5), sigmoid=sigmoid, mask=0.7, pad=pad, seed=n).run()


@pytest.mark.parametrize("kept", [0.04, 1.0])
@pytest.mark.parametrize("n,rows,pad", [(16, 80_011, 0), (512, 7103, 0), (1000, 5329, 0)])
def test_several_turns_with_few_rows_kept_and_with_all(sorted_reference, n, rows, pad, kept):
    Case(rows, n, 4, sigmoid=True, mask=kept, pad=pad, seed=n).run()


@pytest.mark.parametrize("n,rows", [(16, 80_011), (200, 10_007), (300, 7103), (1000, 5329)])
def test_several_turns_with_ties(sorted_reference, n, rows):
    Case(rows, n, 7, mask=0.8, ties=True, seed=n).run()


@pytest.mark.parametrize("n,rows,groups,pad", [(4, 40_003, 5, 0), (100, 2003, 40, 0),
                                               (24, 3001, 100, 3), (12, 1500, 200, 0),
                                               (1000, 601, 3, 0)])
def test_several_turns_of_several_groups(sorted_reference, n, rows, groups, pad):
    Case(rows, n, 3, groups=groups, sigmoid=True, mask=0.7, pad=pad, seed=n).run()


@pytest.mark.parametrize("n,rows", [(16, 80_011), (100, 10_007), (512, 7103), (1000, 5329)])
def test_nan_in_rows_of_every_turn(sorted_reference, n, rows):
    """Some NaN in kept rows, and rows with fewer than k numbers left, between masked ones."""
    k = 6
    c = Case(rows, n, k, mask=0.8, seed=n)
    rng = np.random.default_rng(n)
    for r in range(0, rows, 97):
        gone = 2 if r % 2 else n - k + 2
        c.a[r, 0, rng.permutation(n)[:gone]] = np.nan
    kept = torch.from_numpy(c.mask != 0).cuda()
    held = c.alpha[:rows * n].view(rows, n)
    held[kept] = torch.from_numpy(c.a[:, 0].astype(np.float32)).cuda()[kept]
    c.forward()
    torch.cuda.synchronize()
    want = ref.balance(c.a, c.mask, k, False, COEF)
    assert np.array_equal(c.counts[:n].cpu().numpy(), want["counts"][0])
    assert bool(torch.isnan(c.loss[0])) and int(c.kept[0]) == want["kept"]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n,rows,groups", [(1, 4096, 1), (2, 2047, 8), (3, 1365, 3), (4, 1024, 8),
                                           (4, 1024, 16), (4, 32, 256), (4, 2, 1024), (1, 1, 4096),
                                           (3, 7, 300), (1, 5, 65535), (16, 3, 4096)])
def test_one_launch_over_several_turns_and_many_groups(sorted_reference, n, rows, groups, sigmoid):
    """(The fifth is a size beyond the one launch, the last two the most groups and columns.)"""
    Case(rows, n, 1, groups=groups, sigmoid=sigmoid, mask=0.8 if rows > 2 else None,
         seed=rows).run()


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


# ------------------------------------------------------------------- the norm


PIECE, CTAS = 4096, 1184   # elements of a piece, CTAs of a launch at most


def way_through(sizes):
    """How the CTAs of one launch get from unit to unit: a count of the steps that stay in
    a tensor and of those to the next one, to the one after it and further on."""
    pieces = sum(-(-s // PIECE) for s in sizes)
    per = max(1, min(2, pieces // (2 * CTAS)))
    of = np.repeat(np.arange(len(sizes)), [-(-s // (per * PIECE)) for s in sizes])
    hop = np.minimum(of[CTAS:] - of[:-CTAS], 3)
    return per, np.bincount(hop, minlength=4)


def sizes_in(pieces, ragged):
    return [max(1, PIECE * k - (i * 577 % 4095 if ragged else 0)) for i, k in enumerate(pieces)]


NORM_LISTS = {
    # one piece a unit (fewer than 2368 x 2 pieces), two pieces, and two with single pieces last
    "short": ([1300, 700, 500, 300] + [40] * 12 + [3] * 50 + [1] * 150 + [600], 1),
    "long": ([5000, 2500, 1200, 900, 700] + [90] * 20 + [7] * 60 + [1] * 100 + [2400, 300], 2),
    "long with a small end": ([4800, 3] + [601, 602] * 4 + [1] * 600 + [5], 2),
}


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("name", NORM_LISTS)
def test_norm_of_lists_whose_units_cross_tensors(name, ragged):
    """Mixed types and starts on and off the 16-byte grid, values between 1/2 and 1. Each
    tensor in turn is raised by 2^30, so that the norm is that tensor's alone: the others
    have at most 2^26 elements, less than 2^-32 of its square."""
    sizes = sizes_in(NORM_LISTS[name][0], ragged)
    per, hops = way_through(sizes)
    assert per == NORM_LISTS[name][1] and (hops[:2] > 0).all() and len(sizes) <= 768
    gen = torch.Generator("cuda").manual_seed(len(sizes))
    grads = []
    for i, k in enumerate(sizes):
        g = torch.rand(k + 8, device="cuda", generator=gen) / 2 + 0.5
        g = g.bfloat16() if i % 3 == 1 else g
        grads.append(g[1:k + 1] if i % 4 == 3 else g[:k])
    tensors = dc.train_tensors(dc.train_tensor(grad=g) for g in grads)
    size = dc.dynconv_grad_norm_workspace_size(tensors)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    squares = torch.stack([g.double().square().sum() for g in grads])
    stats = torch.empty(len(grads) + 1, 2, device="cuda")
    for i in range(len(grads) + 1):
        if i < len(grads):
            grads[i].mul_(2.0**30)
        dc.check(dc.dynconv_grad_norm(tensors, 1.0, stats[i], None, ws, size))
        if i < len(grads):
            grads[i].mul_(2.0**-30)
    raised = squares.sum() + squares * (2.0**60 - 1)
    want = torch.cat([raised, squares.sum().view(1)]).sqrt()
    assert bool(((stats[:, 0].double() - want).abs() <= 1.01 * E * want).all())


def test_the_norms_lists_take_every_way():
    """Between them the lists above make each kind of step, with units of one piece and of two."""
    seen = {1: np.zeros(4, int), 2: np.zeros(4, int)}
    for pieces, _ in NORM_LISTS.values():
        for ragged in (False, True):
            per, hops = way_through(sizes_in(pieces, ragged))
            seen[per] += hops
    assert all((hops > 0).all() for hops in seen.values())


def test_lists_of_several_launches_captured_and_replayed():
    """800 tensors: two launches of the norm, three of AdamW, 32 KB of parameters each; the
    graph keeps its own lists."""
    sets = [[Tensor(1 + (i * 37) % 600, *KINDS[i % len(KINDS)], seed=i) for i in range(800)]
            for _ in range(2)]
    side = torch.cuda.Stream()
    stats = [torch.zeros(2, device="cuda") for _ in sets]
    steps = [torch.zeros(1, dtype=torch.int64, device="cuda") for _ in sets]
    lists = [dc.train_tensors(x.entry() for x in t) for t in sets]
    size = dc.dynconv_grad_norm_workspace_size(lists[0])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def step(i):
        dc.check(dc.dynconv_grad_norm(lists[i], 0.5, stats[i], steps[i], ws, size, side))
        dc.check(dc.dynconv_adamw(lists[i], dc.make_adamw(**HYPER, seed=4), stats[i][1:],
                                  step=steps[i], stream=side))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(0)
    for _ in range(2):
        with torch.cuda.stream(side):
            graph.replay()
        step(1)
    side.synchronize()
    assert torch.equal(*stats) and steps[0].tolist() == [2] == steps[1].tolist()
    for a, b in zip(*sets):
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    del graph


@pytest.mark.parametrize("order", [1, -1])
def test_steps_whose_chunks_cross_tensors_of_other_types(order):
    """444 CTAs (with 8-bit states) go from tensor to tensor of every kind, with one, two
    or no chunks of 2048 in each: the staged inputs of one type follow those of another."""
    sizes = (1_000_003, 300_001, 5000, 920_000, 70_001, 2_100_000)
    tensors = [Tensor(sizes[i % 6], *kind, shift=i % 5 == 4, seed=i)
               for i, kind in enumerate((KINDS[1::2] + KINDS[::2])[::order] + KINDS[1::2])]
    step_and_check(tensors)


COLD = """
import torch
import dynamic_convolution_b200 as dc
f = lambda *s: torch.rand(s, device="cuda")
alpha, dalpha, mean, loss = f(5000, 300), f(5000, 300), f(300), f(1)
counts, kept = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (300, 1))
desc = dc.make_balance_desc(5000, 300, top_k=4, mode=dc.SIGMOID)
ws = torch.empty(dc.dynconv_balance_workspace_size(desc), dtype=torch.uint8, device="cuda")
byte = lambda: torch.zeros(3000, dtype=torch.uint8, device="cuda")
tensors = dc.train_tensors([
    dc.train_tensor(grad=f(3000), param=f(3000), m=f(3000), v=f(3000)),
    dc.train_tensor(grad=f(3000), param=f(3000), m=byte(), v=byte(), m_scale=f(12), v_scale=f(12))])
nws = torch.empty(dc.dynconv_grad_norm_workspace_size(tensors), dtype=torch.uint8, device="cuda")
stats, step = f(2), torch.zeros(1, dtype=torch.int64, device="cuda")
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=side):
    dc.check(dc.dynconv_balance_forward(desc, alpha, None, 0.01, counts, mean, kept, loss, ws,
                                        ws.numel(), side))
    dc.check(dc.dynconv_balance_backward(desc, alpha, None, 0.01, counts, kept, None, dalpha, 300,
                                         0, side))
    dc.check(dc.dynconv_grad_norm(tensors, 1.0, stats, step, nws, nws.numel(), side))
    dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(1e-3), stats[1:], step=step, stream=side))
graph.replay()
torch.cuda.synchronize()
print(int(kept), int(counts.sum()), int(step))
del graph
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing has to run before a capture (kernels loaded, attributes set, state queried)."""
    run = subprocess.run([sys.executable, "-c", COLD], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    assert run.stdout.split() == ["5000", "20000", "1"]
