"""The gradient norm and the AdamW step over lists of tensors
(include/dynconv_train.h) on the GPU against the plain 64-bit implementation:
every combination of parameter, gradient and state types, sizes around a vector,
a block and a chunk, unaligned starts, empty tensors, long lists, guards around
every buffer, not-finite gradients, device-side schedules in captured graphs."""
import math

import numpy as np
import pytest
import torch

import dynamic_convolution_b200 as dc

from . import train_ref as ref

pytestmark = pytest.mark.gpu
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8)
FP8 = torch.float8_e4m3fn
E = ref.E


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dynamic_convolution_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Guarded:
    """A device tensor inside a buffer whose bytes around it must stay."""

    def __init__(self, host, shift=0):
        size = host.element_size()
        self.pad = 64 + shift * size
        raw = (host.contiguous().view(torch.uint8) if host.numel()
               else torch.empty(0, dtype=torch.uint8))
        self.held = torch.full((raw.numel() + self.pad + 64,), 0x77, dtype=torch.uint8,
                               device="cuda")
        self.bytes = raw.numel()
        self.held[self.pad:self.pad + self.bytes].copy_(raw)
        inside = self.held[self.pad:self.pad + self.bytes]
        self.t = inside.view(host.dtype) if raw.numel() else host.cuda()

    def check(self):
        assert bool((self.held[:self.pad] == 0x77).all())
        assert bool((self.held[self.pad + self.bytes:] == 0x77).all())


class Tensor:
    """One list entry with its host values in float64."""

    def __init__(self, numel, param="fp32", grad="fp32", bits=32, decay=0.1, lr_scale=1.0, shift=0,
                 seed=0, zeros=0.1):
        rng = np.random.default_rng(seed + numel)
        self.numel, self.kind, self.bits, self.decay, self.lr_scale = numel, param, bits, decay, lr_scale
        p = torch.from_numpy(rng.standard_normal(numel) * 0.05).float()
        g = rng.standard_normal(numel) * np.exp(rng.standard_normal(numel)) * 1e-2
        g[rng.random(numel) < zeros] = 0.0
        g = torch.from_numpy(g).float()
        m = torch.from_numpy(rng.standard_normal(numel) * 3e-3).float()
        v = torch.from_numpy((rng.standard_normal(numel) * 1e-2) ** 2).float()
        v[torch.from_numpy(rng.random(numel) < zeros)] = 0.0
        self.master = Guarded(p, shift) if param == "bf16+master" else None
        self.param = Guarded(p if param == "fp32" else p.bfloat16(), shift)
        self.grad = Guarded(g if grad == "fp32" else g.bfloat16(), shift)
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = Guarded(m, shift), Guarded(v, shift)
        else:
            for name, x in (("m", m), ("v", v.sqrt())):
                b = ref.blocks(x.double().numpy())
                scale = (np.abs(b).max(1) / 448).astype(np.float32)
                code = b / np.maximum(scale, 1e-30)[:, None]
                code = torch.from_numpy(code.reshape(-1)[:numel].copy()).float().to(FP8)
                setattr(self, name, Guarded(code, shift))
                setattr(self, name + "s", Guarded(torch.from_numpy(scale)))
        self.read()

    def read(self):
        d = lambda g: g.t.float().cpu().double().numpy()  # noqa: E731
        self.g64 = d(self.grad)
        self.p64 = d(self.master if self.master else self.param)
        self.m64, self.v64 = d(self.m), d(self.v)
        if self.bits == 8:
            self.m64 = ref.widen(self.m64, d(self.ms))
            self.v64 = ref.widen(self.v64, d(self.vs)) ** 2

    def entry(self):
        t = lambda g: None if g is None else g.t  # noqa: E731
        return dc.train_tensor(grad=self.grad.t, param=self.param.t, m=self.m.t, v=self.v.t,
                               master=t(self.master), m_scale=t(self.ms), v_scale=t(self.vs),
                               lr_scale=self.lr_scale, weight_decay=self.decay)

    def state(self):
        every = (self.param, self.grad, self.m, self.v, self.master, self.ms, self.vs)
        return [g.held.clone() for g in every if g is not None]

    def check(self, place, step, seed=0, scale=1.0, lr=HYPER["lr"]):
        """Against one step from the values of the last read()."""
        h = {**HYPER, "lr": lr * float(np.float32(self.lr_scale))}
        decay = float(np.float32(self.decay))
        p1, m1, v1, ep, em, ev = ref.adamw(self.p64, self.g64, self.m64, self.v64, step=step,
                                           decay=decay, scale=scale, **h)
        if self.bits == 8:   # widening: m one rounding; sqrt(v) one, its square one
            em = em + E * np.abs(HYPER["beta1"] * self.m64)
            ev = ev + 3 * E * HYPER["beta2"] * self.v64
            size = h["lr"] / (1 - HYPER["beta1"] ** step)
            den = np.sqrt(v1 / (1 - HYPER["beta2"] ** step)) + HYPER["eps"]
            ep = ep + size / den * E * np.abs(HYPER["beta1"] * self.m64) + \
                np.abs(size * m1 / den) * 2 * E
        u = ref.dither(seed, step, place, self.numel)
        d = lambda g: g.t.float().cpu().double().numpy()  # noqa: E731
        got = d(self.param)
        if self.kind == "fp32":
            assert np.all(np.abs(got - p1) <= ep)
        elif self.kind == "bf16+master":
            master = d(self.master)
            assert np.all(np.abs(master - p1) <= ep)
            near = self.master.t.bfloat16().float().cpu().double().numpy()
            assert np.array_equal(got, near)        # the copy is the master, rounded
        else:
            a, b = ref.to_bf16_dithered(p1 - ep, u), ref.to_bf16_dithered(p1 + ep, u)
            assert np.all((got >= np.minimum(a, b)) & (got <= np.maximum(a, b)))
        if self.bits == 32:
            assert np.all(np.abs(d(self.m) - m1) <= em)
            assert np.all(np.abs(d(self.v) - v1) <= ev)
        else:
            r1 = np.sqrt(v1)
            er = np.where(v1 > 0, ev / np.maximum(r1, 1e-300) / 2, 0) + 2 * E * r1
            for x, ex, code, top, positive in ((m1, em, self.m, self.ms, False),
                                               (r1, er, self.v, self.vs, True)):
                scale64 = np.abs(ref.blocks(x)).max(1) / 448
                esc = (ref.blocks(ex).max(1) / 448 + 2 * E * scale64)
                got_scale, got_code = d(top), d(code)
                fine = scale64 * 448 >= 2.0 ** -100
                assert np.all(np.abs(got_scale - scale64)[fine] <= esc[fine])
                assert np.all(got_scale[~fine] == 0)
                s = np.repeat(np.where(fine, scale64, np.inf), 256)[:self.numel]
                rel = np.repeat(np.where(fine, esc / np.maximum(scale64, 1e-300), 0),
                                256)[:self.numel]
                y = np.abs(x) / s
                dy = ex / s + y * (rel + 4 * E)
                lo, hi = ref.to_e4m3(y - dy, u), ref.to_e4m3(y + dy, u)
                if positive:
                    # never zero, unless v itself may be (v1 <= ev: below fp32's range,
                    # where 1e-44 of ev covers the square's and the product's underflow)
                    lo = np.maximum(lo, np.where((v1 > ev) & np.isfinite(s), 2.0 ** -9, 0))
                    hi = np.maximum(hi, np.where((x > 0) & np.isfinite(s), 2.0 ** -9, 0))
                assert np.all((np.abs(got_code) >= lo) & (np.abs(got_code) <= hi))
                assert np.all((np.sign(got_code) == np.sign(x)) | (got_code == 0) |
                              (np.abs(x) <= ex))
        for g in (self.param, self.grad, self.m, self.v, self.master, self.ms, self.vs):
            if g is not None:
                g.check()


def step_and_check(tensors, step=3, seed=11):
    hyper = dc.make_adamw(step=step, seed=seed, **HYPER)
    dc.check(dc.dynconv_adamw(dc.train_tensors(t.entry() for t in tensors), hyper), "adamw")
    torch.cuda.synchronize()
    for i, t in enumerate(tensors):
        t.check(i, step, seed)


KINDS = [(p, g, b) for p in ("fp32", "bf16", "bf16+master") for g in ("fp32", "bf16")
         for b in (32, 8)]
SIZES = (1, 2, 3, 4, 5, 127, 128, 129, 255, 256, 257, 511, 2047, 2048, 2049, 5000)


@pytest.mark.parametrize("param,grad,bits", KINDS)
def test_every_kind_and_size(param, grad, bits):
    step_and_check([Tensor(n, param, grad, bits, seed=i) for i, n in enumerate(SIZES)])


@pytest.mark.parametrize("param,grad,bits", KINDS)
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_starts(param, grad, bits, shift):
    step_and_check([Tensor(n, param, grad, bits, shift=shift) for n in (1, 255, 257, 2049)])


def test_mixed_list_longer_than_one_launch():
    """More tensors than a kernel's parameters hold, of every kind, with empty ones
    between, their own rates and decays."""
    tensors = []
    for i in range(800):
        p, g, b = KINDS[i % len(KINDS)]
        tensors.append(Tensor((i * 37) % 600, p, g, b, decay=0.01 * (i % 3),
                              lr_scale=(1.0, 0.5, 0.0)[i % 3], seed=i))
    step_and_check(tensors)


@pytest.mark.parametrize("count", [31, 32, 33, 359, 360, 361, 721])
def test_list_lengths(count):
    step_and_check([Tensor(70 + i % 5, *KINDS[i % len(KINDS)], seed=i) for i in range(count)])


@pytest.mark.parametrize("step", [1, 2, 1000, 10**7])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_numbers(step, bits):
    step_and_check([Tensor(700, "bf16+master", "fp32", bits), Tensor(700, "fp32", "fp32", bits)],
                   step=step)


def test_large_tensor_and_its_tail():
    step_and_check([Tensor(3_000_001, "bf16+master", "fp32", 32), Tensor(3_000_001, "bf16", "bf16", 8)])


def test_more_elements_than_31_bits_count():
    """One tensor of 2^31 + 1000 elements: its start, its middle and its end against
    the formula, and its norm."""
    n = (1 << 31) + 1000
    fp8 = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda").view(FP8)  # noqa: E731
    p = torch.full((n,), 0.125, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-5] = 3.0
    m, v = fp8(n), fp8(n)
    ms, vs = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    tensors = dc.train_tensors([dc.train_tensor(grad=g, param=p, m=m, v=v, m_scale=ms, v_scale=vs)])
    want = math.sqrt(0.25 * (n - 1) + 9)
    got, _ = grad_norm(tensors)
    assert abs(got - want) <= 1.01 * E * want
    dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(step=1, seed=5, **HYPER)))
    torch.cuda.synchronize()
    for at in (0, (1 << 31) - 2048, (1 << 31) - 128, n - 488):   # multiples of 8
        k = min(2048, n - at)
        here = lambda t: t[at:at + k].float().cpu().double().numpy()  # noqa: E731
        zero = np.zeros(k)
        p1, m1, v1, ep, em, ev = ref.adamw(zero + 0.125, here(g), zero, zero, step=1, decay=0.0,
                                           **HYPER)
        u = ref.dither(5, 1, 0, k, at)
        a, b = ref.to_bf16_dithered(p1 - ep, u), ref.to_bf16_dithered(p1 + ep, u)
        assert np.all((here(p) >= np.minimum(a, b)) & (here(p) <= np.maximum(a, b)))
        first, last = at // 256, (at + k - 1) // 256
        top = ms[first:last + 1].double().cpu().numpy() * 448
        assert np.all(np.isclose(top, 0.05) | np.isclose(top, 0.3))
        assert np.all(here(m)[:8] > 0) and np.all(here(v) > 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_state_and_zero_gradients(bits):
    t = [Tensor(1000, "fp32", "fp32", bits, seed=i) for i in range(2)]
    for x in t:
        for g in (x.m, x.v, x.ms, x.vs):
            if g is not None:
                g.t.view(torch.uint8).zero_()
    t[1].grad.t.zero_()
    for x in t:
        x.read()
    step_and_check(t, step=1)
    decayed = t[1].p64 * (1 - HYPER["lr"] * float(np.float32(0.1)))
    assert np.all(np.abs(t[1].param.t.double().cpu().numpy() - decayed) <= 3 * E * np.abs(decayed))


def test_extremes_of_an_8_bit_block():
    """Gradients from 1e-30 to 1e15 in one block, tiny blocks, a root of a second
    moment that stays above zero."""
    t = Tensor(1024, "fp32", "fp32", 8)
    g = np.zeros(1024, np.float32)
    g[:256] = np.logspace(-30, 15, 256)
    g[256:512] = 1e-36
    g[512] = 1.0
    t.grad.t.copy_(torch.from_numpy(g))
    for x in (t.m, t.v, t.ms, t.vs):
        x.t.view(torch.uint8).zero_()
    t.read()
    step_and_check([t], step=1)
    code = t.v.t.float().cpu().numpy()
    assert code[512] == 448 and np.all(code[513:] == 0) and np.all(code[:256][g[:256] > 1e-20] > 0)


def test_8_bit_states_follow_the_32_bit_ones():
    """Dithered rounding has no bias: after 400 steps on noise around a constant
    gradient the mean second moment over 4096 elements is the 32-bit one's. An
    element's stored value has a spread below a quarter of it (the rounding walk at
    beta2 = 0.99 and a spacing of at most 1/8), so the mean of 4096 is within
    4 * 0.25 / 64 < 2 percent, and E[r^2] exceeds E[r]^2 by the spread's square,
    below 6 percent."""
    n = 4096
    a, b = Tensor(n, "fp32", "fp32", 32, seed=1), Tensor(n, "fp32", "fp32", 8, seed=1)
    gen = torch.Generator("cuda").manual_seed(0)
    for x in (a, b):
        for g in (x.m, x.v, x.ms, x.vs):
            if g is not None:
                g.t.view(torch.uint8).zero_()
    lists = [dc.train_tensors([x.entry()]) for x in (a, b)]
    for step in range(1, 401):
        g = 1e-3 * (0.5 + torch.randn(n, device="cuda", generator=gen))
        for x, tensors in zip((a, b), lists):
            x.grad.t.copy_(g)
            dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(step=step, seed=5, **HYPER)))
    b.read()
    v32 = a.v.t.double().cpu().numpy()
    assert abs(b.v64.mean() / v32.mean() - 1) < 0.08
    m32 = a.m.t.double().cpu().numpy()
    assert abs(b.m64.mean() / m32.mean() - 1) < 0.08


@pytest.mark.parametrize("param,grad", [("bf16+master", "fp32"), ("bf16", "bf16")])
def test_8_bit_states_are_the_fp32_formulas_bit_for_bit(param, grad):
    """Five steps against separate fp32 operations of torch (IEEE products, sums,
    square roots): every code and every scale, which also pins the kernel's own root
    on a million values per step."""
    n = 1 << 20
    t = Tensor(n, param, grad, 8, seed=3)
    m, v = t.m.t.float(), t.v.t.float()
    ms, vs = t.ms.t.clone(), t.vs.t.clone()
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    gen = torch.Generator("cuda").manual_seed(1)

    def store(x, u, positive):
        x = x.view(-1, 256)
        top = x.abs().amax(1)
        inv = top.reciprocal() * 448.0
        y = x.abs() * inv[:, None]
        base = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)
        q = (((y + base).view(torch.int32) + (u << 4)) & -(1 << 20)).view(torch.float32) - base
        if positive:
            q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
        return torch.copysign(q, x).view(-1), top * (1.0 / 448.0)

    for step in range(1, 6):
        g = (torch.randn(n, device="cuda", generator=gen) *
             torch.exp(torch.randn(n, device="cuda", generator=gen)) * 1e-3)
        t.grad.t.copy_(g)
        g = t.grad.t.float()
        dc.check(dc.dynconv_adamw(dc.train_tensors([t.entry()]),
                                  dc.make_adamw(step=step, seed=9, **HYPER)))
        u = torch.from_numpy((ref.dither(9, step, 0, n) * 65536).astype(np.int32)).cuda().view(-1, 256)
        m32 = (m.view(-1, 256) * ms[:, None]).view(-1)
        r32 = (v.view(-1, 256) * vs[:, None]).view(-1)
        m32 = m32 * b1 + g * (1.0 - b1)
        v32 = (r32 * r32) * b2 + (g * g) * (1.0 - b2)
        m, ms = store(m32, u, False)
        v, vs = store(v32.sqrt(), u, True)
        assert torch.equal(t.m.t.float(), m) and torch.equal(t.v.t.float(), v)
        assert torch.equal(t.ms.t, ms) and torch.equal(t.vs.t, vs)


def test_the_same_inputs_give_the_same_bits():
    runs = []
    for _ in range(2):
        t = [Tensor(3000, p, g, b, seed=7) for p, g, b in KINDS]
        dc.check(dc.dynconv_adamw(dc.train_tensors(x.entry() for x in t),
                                  dc.make_adamw(step=2, seed=3, **HYPER)))
        torch.cuda.synchronize()
        runs.append([s for x in t for s in x.state()])
    assert all(torch.equal(x, y) for x, y in zip(*runs))


# ------------------------------------------------------------------- the norm


def grad_norm(tensors, max_norm=math.inf, step=None, stream=None):
    stats = torch.full((3,), -7.0, device="cuda")
    size = dc.dynconv_grad_norm_workspace_size(tensors)
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN patterns
    dc.check(dc.dynconv_grad_norm(tensors, max_norm, stats, step, ws, size, stream), "grad_norm")
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xFF).all()) and float(stats[2]) == -7.0
    return stats[:2].double().tolist()


@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_of_sizes(grad, shift):
    t = [Tensor(n, grad=grad, shift=shift, seed=i) for i, n in enumerate(SIZES)]
    for some in (t, t[:1], t[4:5], t[-1:], []):
        want = math.sqrt(sum(float((x.g64 ** 2).sum()) for x in some))
        got, factor = grad_norm(dc.train_tensors(x.entry() for x in some), max_norm=0.25)
        assert abs(got - want) <= 1.01 * E * want     # fp64 sums, rounded once
        assert abs(factor - min(1.0, 0.25 / (want + 1e-6))) <= 1.01 * E * factor


def test_norm_of_a_long_list_and_of_a_large_tensor():
    t = [Tensor((i * 13) % 50, grad=("fp32", "bf16")[i % 2], seed=i) for i in range(1600)]
    t.append(Tensor(4_000_003))
    want = math.sqrt(sum(float((x.g64 ** 2).sum()) for x in t))
    got, factor = grad_norm(dc.train_tensors(dc.train_tensor(grad=x.grad.t) for x in t))
    assert abs(got - want) <= 1.01 * E * want and factor == 1.0


@pytest.mark.parametrize("value", [3e38, 1e-38, 1e-45])
def test_norm_neither_overflows_nor_underflows(value):
    g = torch.zeros(5000, device="cuda")
    g[77] = value
    got, _ = grad_norm(dc.train_tensors([dc.train_tensor(grad=g)]))
    assert got == float(g[77])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_not_finite_skips_the_step(bad):
    t = [Tensor(900, p, g, b) for p, g, b in KINDS]
    t[5].grad.t[123] = bad
    before = [s for x in t for s in x.state()]
    tensors = dc.train_tensors(x.entry() for x in t)
    step = torch.tensor([41], device="cuda")
    stats = torch.zeros(2, device="cuda")
    size = dc.dynconv_grad_norm_workspace_size(tensors)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dc.check(dc.dynconv_grad_norm(tensors, 1.0, stats, step, ws, size))
    dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(**HYPER), grad_scale=stats[1:], step=step))
    torch.cuda.synchronize()
    assert not math.isfinite(float(stats[0])) and math.isnan(float(stats[1]))
    assert int(step) == 41
    assert all(torch.equal(a, b) for a, b in zip(before, [s for x in t for s in x.state()]))


def test_a_bad_gradient_without_the_norm_spoils_its_block_only():
    t = Tensor(1024, "fp32", "fp32", 8)
    t.grad.t[300] = math.nan
    dc.check(dc.dynconv_adamw(dc.train_tensors([t.entry()]), dc.make_adamw(**HYPER)))
    torch.cuda.synchronize()
    spoilt = torch.isnan(t.ms.t).cpu().tolist()
    assert spoilt == [False, True, False, False] == torch.isnan(t.vs.t).cpu().tolist()
    assert torch.isnan(t.param.t).nonzero().flatten().tolist() == [300]


# --------------------------------------------- together, captured and replayed


@pytest.mark.parametrize("param,grad,bits", [("bf16+master", "fp32", 32), ("bf16", "bf16", 8)])
def test_clip_and_step_captured(param, grad, bits):
    """Norm, factor, step number and rate all on the device: three replays are three
    steps, on a side stream, and two graphs share the norm's workspace."""
    sets = [[Tensor(n, param, grad, bits, seed=s + n) for n in (300, 5000)] for s in (0, 1)]
    side = torch.cuda.Stream()
    lists = [dc.train_tensors(x.entry() for x in t) for t in sets]
    size = dc.dynconv_grad_norm_workspace_size(lists[0])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    stats = [torch.zeros(2, device="cuda") for _ in sets]
    steps = [torch.tensor([s], device="cuda") for s in (0, 9)]
    lr = torch.tensor([1e-3], device="cuda")
    hyper = dc.make_adamw(**{**HYPER, "lr": 0.5}, step=99, seed=21)   # both replaced
    torch.cuda.synchronize()

    def both(i):
        dc.check(dc.dynconv_grad_norm(lists[i], 0.05, stats[i], steps[i], ws, size, side))
        dc.check(dc.dynconv_adamw(lists[i], hyper, stats[i][1:], lr, steps[i], side))

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(i)
        graphs.append(g)
    for replay in range(3):
        rate = 1e-3 * (replay + 1)
        lr.fill_(rate)
        for t in sets:
            for x in t:
                x.read()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        side.synchronize()
        for i, t in enumerate(sets):
            number = (0, 9)[i] + replay + 1
            assert int(steps[i]) == number
            norm = math.sqrt(sum(float((x.g64 ** 2).sum()) for x in t))
            got, factor = stats[i].double().tolist()
            assert abs(got - norm) <= 1.01 * E * norm and factor < 1
            for place, x in enumerate(t):
                x.check(place, number, 21, scale=factor, lr=float(np.float32(rate)))
    del graphs


def test_two_steps_at_once_on_two_streams():
    sets = [[Tensor(20_000 + s, p, g, b, seed=s) for p, g, b in KINDS] for s in (0, 1)]
    lists = [dc.train_tensors(x.entry() for x in t) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for tensors, s in zip(lists, streams):
        dc.check(dc.dynconv_adamw(tensors, dc.make_adamw(step=3, seed=11, **HYPER), stream=s))
    torch.cuda.synchronize()
    for t in sets:
        for i, x in enumerate(t):
            x.check(i, 3, 11)


def test_no_clipping_leaves_the_factor_at_one():
    t = Tensor(500)
    tensors = dc.train_tensors([t.entry()])
    assert grad_norm(tensors, 1e9)[1] == 1.0
    step = torch.tensor([4], device="cuda")
    grad_norm(tensors, 1e9, step)
    assert int(step) == 5
