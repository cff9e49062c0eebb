"""The load-balance loss and its gradient (include/dynconv_train.h) on the GPU
against the plain 64-bit implementation, at the sizes and masks where they can go
wrong: every register layout of a row and its borders, one row and none, masks
that drop rows full of NaN (or all rows), ties, rows inside wider buffers, odd
strides and unaligned starts; streams, captured graphs that share a workspace."""
import numpy as np
import pytest
import torch

import dynamic_convolution_b200 as dc

from . import train_ref as ref

pytestmark = pytest.mark.gpu
COEF = 0.37


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dynamic_convolution_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Case:
    """Attentions inside a buffer of NaN (before, between and after the rows),
    outputs inside guarded buffers."""

    def __init__(self, rows, n, k, groups=1, sigmoid=False, mask=None, pad=0, shift=0, seed=0,
                 ties=False):
        rng = np.random.default_rng(seed)
        self.rows, self.n, self.k, self.groups, self.sigmoid = rows, n, k, groups, sigmoid
        self.width, self.stride = groups * n, groups * n + pad
        z = rng.standard_normal((rows, groups, n))
        if ties:
            z = np.round(z)
        a = 1 / (1 + np.exp(-z)) if sigmoid else np.exp(z) / np.exp(z).sum(-1, keepdims=True)
        self.a = a.astype(np.float32).astype(np.float64)
        self.mask = None
        if mask is not None:
            self.mask = (rng.random(rows) < mask).astype(np.uint8) * rng.integers(1, 256, rows,
                                                                                 dtype=np.uint8)
        held = torch.full((rows * self.stride + shift + 8,), float("nan"))
        view = held[shift:shift + rows * self.stride].view(rows, self.stride)
        view[:, :self.width] = torch.from_numpy(self.a.reshape(rows, self.width).astype(np.float32))
        if self.mask is not None:
            gone = torch.from_numpy(self.mask == 0)
            view[gone] = torch.tensor([float("nan"), float("inf"), -float("inf")])[
                torch.arange(self.stride) % 3]
        self.held = held.cuda()
        self.alpha = self.held[shift:]
        self.dmask = None if self.mask is None else torch.from_numpy(self.mask).cuda()
        self.desc = dc.make_balance_desc(rows, n, groups, k, dc.SIGMOID if sigmoid else dc.SOFTMAX,
                                         self.stride)
        self.size = dc.dynconv_balance_workspace_size(self.desc)
        self.ws = torch.full((self.size,), 0xAB, dtype=torch.uint8, device="cuda")
        self.counts = torch.full((self.width + 2,), -7, dtype=torch.int32, device="cuda")
        self.mean = torch.full((self.width + 2,), -7.0, device="cuda")
        self.kept = torch.full((2,), -7, dtype=torch.int32, device="cuda")
        self.loss = torch.full((2,), -7.0, device="cuda")
        self.before = rng.standard_normal((rows, self.stride)).astype(np.float32) * 1e-3
        self.dheld = torch.full((rows * self.stride + shift + 8,), 5.0, device="cuda")
        self.dalpha = self.dheld[shift:]
        self.dloss = torch.tensor([1.25], device="cuda")

    def forward(self, stream=None):
        dc.check(dc.dynconv_balance_forward(self.desc, self.alpha, self.dmask, COEF, self.counts,
                                            self.mean, self.kept, self.loss, self.ws, self.size,
                                            stream), "balance_forward")

    def backward(self, accumulate, stream=None, dloss=True):
        dc.check(dc.dynconv_balance_backward(self.desc, self.alpha if self.sigmoid else None,
                                             self.dmask, COEF, self.counts, self.kept,
                                             self.dloss if dloss else None, self.dalpha,
                                             self.stride, accumulate, stream), "balance_backward")

    def check_forward(self):
        torch.cuda.synchronize()
        r = ref.balance(self.a, self.mask, self.k, self.sigmoid, COEF)
        w = self.width
        counts = self.counts.cpu().numpy()
        assert np.array_equal(counts[:w].reshape(self.groups, self.n), r["counts"])
        assert np.all(counts[w:] == -7)
        assert self.kept.tolist() == [r["kept"], -7]
        # softmax: fp64 sums of the inputs, rounded once. sigmoid: a row's sum of
        # n positive terms (at most 32 in a lane, then five steps across lanes)
        # and the quotient before that.
        rel = (1 + (min(self.n, 32) + 5 + 1 if self.sigmoid else 0)) * ref.E
        mean = self.mean.double().cpu().numpy()
        assert np.all(np.abs(mean[:w] - r["mean"].ravel()) <= rel * r["mean"].ravel())
        assert np.all(mean[w:] == -7)
        loss = self.loss.double().cpu().numpy()
        # the coefficient arrives as fp32: one more rounding
        assert abs(loss[0] - r["loss"]) <= (rel + 2 * ref.E) * r["loss"] and loss[1] == -7
        return r

    def check_backward(self, r, accumulate, dloss=1.25):
        torch.cuda.synchronize()
        g, size = ref.balance_grad(self.a, self.mask, r["counts"], self.k, self.sigmoid, COEF, dloss)
        got = self.dheld.double().cpu().numpy()
        shift = self.dheld.numel() - 8 - self.rows * self.stride
        assert np.all(got[:shift] == 5.0) and np.all(got[shift + self.rows * self.stride:] == 5.0)
        got = got[shift:shift + self.rows * self.stride].reshape(self.rows, self.stride)
        before = self.before.astype(np.float64)
        assert np.array_equal(got[:, self.width:], before[:, self.width:])   # between the rows
        want, size = (x.reshape(self.rows, self.width) for x in (g, size))
        # c: the coefficient and the rounding (2); sigmoid: S and p as above, the
        # sum of n products, the difference, the quotient
        tol = 2 * ref.E * size
        if self.sigmoid:
            tol = (3 + 3 * (min(self.n, 32) + 7)) * ref.E * size
        if accumulate:
            want = want + before[:, :self.width]
            tol = tol + ref.E * np.abs(want)
        assert np.all(np.abs(got[:, :self.width] - want) <= tol + 1e-44)
        if self.mask is not None:
            gone = self.mask == 0
            assert np.array_equal(got[gone][:, :self.width],
                                  before[gone][:, :self.width] if accumulate
                                  else np.zeros((gone.sum(), self.width)))

    def fill(self):
        torch.cuda.synchronize()
        self.dalpha[:self.rows * self.stride].copy_(torch.from_numpy(self.before.ravel()))

    def run(self):
        self.forward()
        r = self.check_forward()
        for accumulate in (0, 1):
            self.fill()
            self.backward(accumulate)
            self.check_backward(r, accumulate)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129,
                               256, 257, 511, 512, 513, 1000, 1023, 1024])
def test_every_row_layout(n, sigmoid):
    Case(67, n, min(n, 3), sigmoid=sigmoid, seed=n).run()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("rows", [0, 1, 2, 7, 8, 9, 255, 256, 257, 5000])
def test_row_counts(rows, sigmoid):
    Case(rows, 12, 2, sigmoid=sigmoid, seed=rows).run()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kept", [0.0, 0.05, 0.7, 1.0])
@pytest.mark.parametrize("n,pad,shift", [(4, 0, 0), (24, 4, 0), (24, 4, 1), (24, 3, 0), (37, 0, 0)])
def test_masks_strides_and_starts(n, pad, shift, kept, sigmoid):
    Case(301, n, 2, sigmoid=sigmoid, mask=kept, pad=pad, shift=shift, seed=n + pad).run()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,n,k", [(2, 4, 1), (16, 128, 4), (3, 5, 5), (64, 3, 2), (7, 40, 9)])
def test_groups(groups, n, k, sigmoid):
    Case(70, n, k, groups=groups, sigmoid=sigmoid, mask=0.8, pad=groups, seed=groups).run()


@pytest.mark.parametrize("n,k", [(1, 1), (6, 6), (40, 40), (40, 32), (1024, 1024), (1000, 32)])
def test_top_k_sizes(n, k):
    Case(33, n, k, seed=k).run()


@pytest.mark.parametrize("n,k", [(4, 2), (16, 3), (64, 8), (300, 5)])
def test_ties_go_to_the_lowest_index(n, k):
    Case(200, n, k, ties=True, seed=n).run()
    c = Case(50, n, k, seed=1)
    c.a[:] = np.float32(1.0 / n)
    c.alpha[:50 * c.stride].fill_(1.0 / n)
    c.run()
    assert c.counts[:n].tolist() == [50 if i < k else 0 for i in range(n)]


def test_order_of_zeros_negatives_infinities_and_nan():
    row = [float("nan"), -0.0, 0.0, -1.0, -float("inf"), 2.0, float("inf"), float("nan")]
    for k in range(1, 8):
        c = Case(1, 8, k)
        c.alpha[:8].copy_(torch.tensor(row))
        c.forward()
        torch.cuda.synchronize()
        want = ref.top_k(np.array(row), k)
        assert want[:3] == [6, 5, 1][:k]
        assert c.counts[:8].tolist() == [1 if i in want else 0 for i in range(8)]
        assert bool(torch.isnan(c.loss[0]))   # a kept NaN shows


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n,k", [(12, 3), (100, 7), (300, 5), (1000, 32)])
def test_nan_among_many_experts(n, k, sigmoid):
    """Rows with some NaN, and with so many that fewer than k numbers are left."""
    rows = 40
    c = Case(rows, n, k, sigmoid=sigmoid, seed=n)
    rng = np.random.default_rng(n)
    c.a[3, 0, rng.integers(0, n, 2)] = np.nan
    c.a[7, 0, rng.permutation(n)[:n - k + 2]] = np.nan
    c.a[8] = np.nan
    c.alpha[:rows * n].copy_(torch.from_numpy(c.a.reshape(-1).astype(np.float32)))
    c.forward()
    torch.cuda.synchronize()
    want = np.zeros(n, np.int64)
    for row in c.a[:, 0]:
        want[ref.top_k(row, k)] += 1
    assert np.array_equal(c.counts[:n].cpu().numpy(), want)
    assert bool(torch.isnan(c.loss[0])) and int(c.kept[0]) == rows


@pytest.mark.parametrize("n,k", [(300, 9), (1000, 8)])
def test_wide_rows_with_a_few_equal_values_at_the_border(n, k):
    c = Case(64, n, k, seed=k)
    for b in range(64):                      # b % 9 equal largest values in a row
        c.a[b, 0, np.random.default_rng(b).permutation(n)[:b % 9 + 2]] = 0.5
    c.alpha[:64 * n].copy_(torch.from_numpy(c.a.reshape(-1).astype(np.float32)))
    c.forward()
    c.check_forward()


def test_sigmoid_rows_of_tiny_and_huge_sums():
    """Sums below and above the reciprocal's range take the division."""
    c = Case(4, 6, 2, sigmoid=True)
    scale = np.array([1e-35, 1e-41, 1e33, 1.0])[:, None, None]
    c.a = (c.a * scale).astype(np.float32).astype(np.float64)
    c.alpha[:24].copy_(torch.from_numpy(c.a.reshape(-1).astype(np.float32)))
    c.forward()
    torch.cuda.synchronize()
    r = ref.balance(c.a, None, 2, True, COEF)
    mean = c.mean[:6].double().cpu().numpy()
    assert np.all(np.abs(mean - r["mean"][0]) <= 13 * ref.E * r["mean"][0])


def test_sigmoid_rows_that_sum_to_zero():
    c = Case(5, 6, 1, sigmoid=True)
    c.a[2] = 0.0
    c.alpha[2 * 6:3 * 6].zero_()
    c.run()
    assert torch.equal(c.dalpha[12:18].cpu(), torch.from_numpy(c.before[2]))


def test_one_expert_leaves_no_gradient():
    c = Case(5000, 1, 1, sigmoid=True, seed=4)
    c.forward()
    c.fill()
    c.backward(0)
    torch.cuda.synchronize()
    assert not c.dalpha[:5000].any() and c.mean[:1].tolist() == [1.0]


def test_default_dloss_and_repeatability():
    c = Case(1003, 48, 4, sigmoid=True, mask=0.6)
    c.forward()
    r = c.check_forward()
    c.fill()
    c.backward(0, dloss=False)
    c.check_backward(r, 0, dloss=1.0)
    first = [t.clone() for t in (c.counts, c.mean, c.loss, c.dheld)]
    c.ws.fill_(0x5A)
    c.forward()
    c.fill()
    c.backward(0, dloss=False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (c.counts, c.mean, c.loss, c.dheld)))


def test_long_offsets():
    """Rows whose offsets pass 2^31 elements (stride 2^22 floats, 520 rows); only
    the first columns hold attentions."""
    rows, n, stride = 520, 12, 1 << 22
    held = torch.empty(rows * stride, device="cuda").view(rows, stride)
    c = Case(rows, n, 2, sigmoid=True)
    held[:, :n] = c.alpha[:rows * n].view(rows, n)
    c.desc.row_stride = stride
    c.alpha = held
    c.forward()
    r = c.check_forward()
    dheld = held   # the gradient goes beside the attentions, into the same wide rows
    dheld[:, 16:16 + n] = 0.0
    dc.check(dc.dynconv_balance_backward(c.desc, held, None, COEF, c.counts, c.kept, c.dloss,
                                         dheld[:, 16:], stride, 0))
    torch.cuda.synchronize()
    g, size = ref.balance_grad(c.a, None, r["counts"], 2, True, COEF, 1.25)
    got = dheld[:, 16:16 + n].double().cpu().numpy()
    assert np.all(np.abs(got - g[:, 0]) <= 60 * ref.E * size[:, 0])


def test_long_offsets_softmax_backward():
    rows, n, stride = 520, 12, 1 << 22
    c = Case(rows, n, 2)
    c.forward()
    r = c.check_forward()
    for accumulate in (0, 1):
        wide = torch.full((rows, stride), 2.0, device="cuda")
        dc.check(dc.dynconv_balance_backward(c.desc, None, None, COEF, c.counts, c.kept, c.dloss,
                                             wide[:, 8:], stride, accumulate))
        torch.cuda.synchronize()
        g, size = ref.balance_grad(c.a, None, r["counts"], 2, False, COEF, 1.25)
        got = wide[:, 8:8 + n].double().cpu().numpy() - 2.0 * accumulate
        assert np.all(np.abs(got - g[:, 0]) <= 2 * ref.E * size[:, 0] + 2 * accumulate * 2 * ref.E)
        assert bool((wide[:, :8] == 2.0).all()) and bool((wide[:, 8 + n:1024] == 2.0).all())


def test_two_calls_at_once():
    """On two streams, each with its own workspace and outputs."""
    cases = [Case(3000, 32, 3, sigmoid=bool(i), mask=0.8, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.forward(s)
            c.backward(0, s)
    torch.cuda.synchronize()
    for c in cases:
        r = c.check_forward()
        c.fill()
        c.backward(0)
        c.check_backward(r, 0)


def test_many_rows():
    """Enough rows for every part of the sums; the reference is vectorised."""
    rows, n, k = 300_007, 10, 2
    a = torch.softmax(torch.randn(rows, n, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(2)), -1)
    c = Case(3, n, k)
    c.rows, c.desc = rows, dc.make_balance_desc(rows, n, top_k=k)
    c.size = dc.dynconv_balance_workspace_size(c.desc)
    c.ws = torch.empty(c.size, dtype=torch.uint8, device="cuda")
    c.alpha = a
    c.forward()
    torch.cuda.synchronize()
    chosen = torch.sort(a, dim=-1, descending=True, stable=True).indices[:, :k]
    counts = torch.bincount(chosen.reshape(-1), minlength=n)
    assert torch.equal(c.counts[:n].long(), counts)
    mean = a.double().mean(0)
    assert torch.all((c.mean[:n].double() - mean).abs() <= 1.01 * ref.E * mean)
    loss = COEF * n / k * float((counts / rows * mean).sum())
    assert abs(float(c.loss[0]) - loss) <= 4 * ref.E * loss


def test_side_stream_and_graphs_sharing_a_workspace():
    a, b = (Case(400, 20, 2, sigmoid=s, mask=0.9, seed=s) for s in (False, True))
    b.ws = a.ws = torch.empty(max(a.size, b.size), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in (a, b):                       # first calls, on a stream of their own
        c.forward(side)
        c.fill()
        c.backward(1, side)
        side.synchronize()
        c.check_backward(c.check_forward(), 1)
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.forward(side)
            c.backward(0, side)
        graphs.append(g)
    for _ in range(3):
        for c in (a, b):
            c.counts.fill_(-7)
            c.fill()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
            graphs[1].replay()
        side.synchronize()
        for c in (a, b):
            c.check_backward(c.check_forward(), 0)
    del graphs
