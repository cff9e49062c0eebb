"""One layer's whole training step through the public calls: routing, balance loss,
forward, the layer's backward with the balance gradient joined into the
attentions' gradient, the gradients' norm and the AdamW step; against the
oracle's gradients and the 64-bit formulas, and the same step captured into a
CUDA graph and replayed."""
import numpy as np
import pytest
import torch

import dynamic_convolution_b200 as dc
import oracle
from dynamic_convolution_b200 import synth

from . import train_ref as ref
from .gpu_util import to_device

pytestmark = pytest.mark.gpu
COEF, HYPER, MAX_NORM = 50.0, dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8), 5.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dynamic_convolution_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Step:
    def __init__(self, cfg, bits=32):
        self.cfg, self.bits = cfg, bits
        self.inp = inp = synth.make_inputs(cfg, seed=3, structured=1.0)
        dys, self.dy64 = synth.make_upstream_grad(cfg)
        B, n, C, Co = cfg.B, cfg.n, cfg.C_in, cfg.C_out
        f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
        self.x, self.E = to_device(inp.x_store, cfg.dtype), to_device(inp.experts_store, cfg.dtype)
        self.dy = to_device(dys, cfg.dtype)
        self.Wr, self.br, self.bias = (torch.from_numpy(a).cuda() for a in (inp.Wr, inp.br, inp.bias))
        self.alpha, self.dalpha = f(B, n), f(B, n)
        self.y = torch.empty((B, cfg.H_out, cfg.W_out, Co), dtype=self.E.dtype, device="cuda")
        self.dE, self.dbias, self.dWr, self.dbr = f(*self.E.shape), f(n, Co), f(n, C), f(n)
        self.dg, self.dx = f(B, C), torch.empty_like(self.x)
        self.d = dc.desc_from_config(cfg)
        byte = lambda k: torch.empty(max(k, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = byte(max(dc.dynconv_workspace_size(self.d),
                           dc.dynconv_backward_workspace_size(self.d)))
        self.bd = dc.make_balance_desc(B, n, mode=cfg.mode)
        self.bws = byte(dc.dynconv_balance_workspace_size(self.bd))
        self.counts = torch.zeros(1, n, dtype=torch.int32, device="cuda")
        self.mean, self.kept, self.loss = f(1, n), torch.zeros(1, dtype=torch.int32, device="cuda"), f(1)
        self.master = self.E.float() if cfg.dtype == synth.BF16 else None
        entries = []
        self.states = []
        for p, g, master, decay in ((self.E, self.dE, self.master, 0.01), (self.bias, self.dbias, None, 0.0),
                                    (self.Wr, self.dWr, None, 0.0), (self.br, self.dbr, None, 0.0)):
            if bits == 8 and p is self.E:
                k = p.numel()
                m, v = (torch.zeros(p.shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                        for _ in range(2))
                scales = dict(m_scale=f(-(-k // 256)), v_scale=f(-(-k // 256)))
            else:
                m, v, scales = f(*p.shape), f(*p.shape), {}
            self.states.append((p, g, master, m, v, decay))
            entries.append(dc.train_tensor(grad=g, param=p, m=m, v=v, master=master,
                                           weight_decay=decay, **scales))
        self.tensors = dc.train_tensors(entries)
        self.nws = byte(dc.dynconv_grad_norm_workspace_size(self.tensors))
        self.stats, self.number = f(2), torch.zeros(1, dtype=torch.int64, device="cuda")
        self.hyper = dc.make_adamw(seed=7, **HYPER)

    def run(self, stream=None):
        d, cfg, ws, wsb = self.d, self.cfg, self.ws, self.ws.numel()
        ok = dc.check
        ok(dc.dynconv_route(d, self.x, self.Wr, self.br, cfg.mode, cfg.tau, self.alpha, stream))
        ok(dc.dynconv_balance_forward(self.bd, self.alpha, None, COEF, self.counts, self.mean,
                                      self.kept, self.loss, self.bws, self.bws.numel(), stream))
        ok(dc.dynconv_forward(d, self.x, self.E, self.alpha, self.bias, self.y, ws, wsb, stream))
        ok(dc.dynconv_backward_weight(d, self.x, self.dy, self.E, self.alpha, self.bias, self.dE,
                                      self.dbias, self.dalpha, ws, wsb, stream))
        ok(dc.dynconv_balance_backward(self.bd, self.alpha, None, COEF, self.counts, self.kept,
                                       None, self.dalpha, cfg.n, 1, stream))
        ok(dc.dynconv_route_backward(d, self.x, self.Wr, self.alpha, self.dalpha, cfg.mode,
                                     cfg.tau, self.dWr, self.dbr, self.dg, ws, wsb, stream))
        ok(dc.dynconv_backward_data(d, self.dy, self.E, self.alpha, self.dg, self.dx, ws, wsb,
                                    stream))
        ok(dc.dynconv_grad_norm(self.tensors, MAX_NORM, self.stats, self.number, self.nws,
                                self.nws.numel(), stream))
        ok(dc.dynconv_adamw(self.tensors, self.hyper, grad_scale=self.stats[1:], step=self.number,
                            stream=stream))


def small(dtype, mode):
    return synth.LayerConfig("small", dtype, 6, 16, 24, 9, 7, 3, 3, 1, 1, 1, 5, mode, 1.0)


@pytest.mark.parametrize("mode", [synth.SOFTMAX, synth.SIGMOID])
@pytest.mark.parametrize("dtype", [synth.F32, synth.BF16])
def test_step_against_the_oracle(dtype, mode):
    cfg = small(dtype, mode)
    s = Step(cfg)
    inp = s.inp
    before = [(p.float() if master is None else master).double().cpu().numpy().ravel()
              for p, _, master, _, _, _ in s.states]
    s.run()
    torch.cuda.synchronize()
    assert dc.dynconv_device_status(None) == dc.OK
    # the balance loss of the attentions that the kernel took, and its gradient
    a = s.alpha.double().cpu().numpy()
    b = ref.balance(a[:, None], None, 1, mode == synth.SIGMOID, COEF)
    assert np.array_equal(s.counts.cpu().numpy(), b["counts"])
    assert abs(float(s.loss) - b["loss"]) <= 16 * ref.E * b["loss"]
    g, _ = ref.balance_grad(a[:, None], None, b["counts"], 1, mode == synth.SIGMOID, COEF, 1.0)
    # the layer's gradients, then the router's from the joined gradient
    want = oracle.backward(inp.x_f64, s.dy64, inp.experts_f64, a, inp.bias, inp.Wr, mode, cfg.tau,
                           stride=1, pad=1)
    joined = want["dalpha"] + g[:, 0]
    dWr, dbr, _ = oracle.route_backward(inp.x_f64, inp.Wr, a, joined, mode, cfg.tau)
    rel = lambda t, w: np.linalg.norm(t.double().cpu().numpy() - w) / np.linalg.norm(w)  # noqa: E731
    assert rel(s.dE, want["dexperts"]) <= 1e-4 and rel(s.dalpha, joined) <= 1e-4
    assert rel(s.dWr, dWr) <= 1e-3 and rel(s.dbr, dbr) <= 1e-3
    # (a missing balance gradient would show in dalpha)
    assert np.linalg.norm(g[:, 0]) > 1e-3 * np.linalg.norm(want["dalpha"])
    # the norm, the factor, and the update from the gradients as they stand
    norm = np.sqrt(sum(float((x.double() ** 2).sum()) for _, x, *_ in s.states))
    got, factor = s.stats.double().tolist()
    assert abs(got - norm) <= 1.01 * ref.E * norm and int(s.number) == 1
    assert abs(factor - min(1, MAX_NORM / (norm + 1e-6))) <= 1.01 * ref.E * factor
    for p0, (p, grad, master, m, v, decay) in zip(before, s.states):
        zero = np.zeros_like(p0)
        p1, m1, v1, ep, em, ev = ref.adamw(p0, grad.double().cpu().numpy().ravel(), zero, zero,
                                           step=1, decay=float(np.float32(decay)), scale=factor,
                                           **HYPER)
        new = (p if master is None else master).double().cpu().numpy().ravel()
        assert np.all(np.abs(new - p1) <= ep)
        assert np.all(np.abs(m.double().cpu().numpy().ravel() - m1) <= em)
        assert np.all(np.abs(v.double().cpu().numpy().ravel() - v1) <= ev)
        if master is not None:
            assert torch.equal(p, master.bfloat16())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_equals_the_eager_one(bits):
    """Three replays of a captured step (its step number and clipping on the device)
    leave the bits that three eager steps leave."""
    cfg = synth.LayerConfig("mid", synth.BF16, 8, 64, 72, 14, 14, 3, 3, 1, 1, 1, 4, synth.SOFTMAX, 1.0)
    eager, graphed = Step(cfg, bits), Step(cfg, bits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    eager.run(side)
    graphed.run(side)          # first calls, before any capture
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        graphed.run(side)
    for _ in range(3):
        eager.run(side)
    with torch.cuda.stream(side):
        for _ in range(3):
            g.replay()
    side.synchronize()
    assert int(eager.number) == int(graphed.number) == 4
    for name in ("E", "master", "Wr", "br", "bias", "loss", "stats", "dx"):
        assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
    for a, b in zip(eager.states, graphed.states):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[3:5], b[3:5]))
    assert dc.dynconv_device_status(side) == dc.OK
    del g


def test_cell_routers():
    """Balance over the routers of kernel cells: attentions of dynconv_route_cells."""
    cfg = synth.LayerConfig("cells", synth.BF16, 10, 32, 32, 6, 6, 3, 3, 1, 1, 1, 9, synth.SOFTMAX, 2.0)
    cells, n = 4, 9
    ci = synth.make_cell_inputs(cfg, cells, n, seed=2, structured=1.0)
    d = dc.make_desc(cfg.B, 32, 6, 6, 32, 3, 3, 1, 1, 1, n, cfg.dtype)
    alpha = torch.empty((cfg.B, cells, n), device="cuda")
    ws = torch.empty(dc.dynconv_cells_workspace_size(d, cells), dtype=torch.uint8, device="cuda")
    Wr, br = torch.from_numpy(ci.Wr).cuda(), torch.from_numpy(ci.br).cuda()
    dc.check(dc.dynconv_route_cells(d, cells, to_device(ci.x_store, cfg.dtype), Wr, br, cfg.mode,
                                    cfg.tau, alpha, ws, ws.numel()))
    bd = dc.make_balance_desc(cfg.B, n, groups=cells, top_k=2, mode=cfg.mode)
    bws = torch.empty(dc.dynconv_balance_workspace_size(bd), dtype=torch.uint8, device="cuda")
    counts = torch.empty((cells, n), dtype=torch.int32, device="cuda")
    mean, loss = torch.empty((cells, n), device="cuda"), torch.empty(1, device="cuda")
    kept = torch.empty(1, dtype=torch.int32, device="cuda")
    dc.check(dc.dynconv_balance_forward(bd, alpha, None, COEF, counts, mean, kept, loss, bws,
                                        bws.numel()))
    dalpha = torch.empty_like(alpha)
    dc.check(dc.dynconv_balance_backward(bd, alpha, None, COEF, counts, kept, None, dalpha,
                                         cells * n, 0))
    torch.cuda.synchronize()
    a = alpha.double().cpu().numpy()
    r = ref.balance(a, None, 2, False, COEF)
    assert np.array_equal(counts.cpu().numpy(), r["counts"])
    assert abs(float(loss) - r["loss"]) <= 4 * ref.E * r["loss"]
    g, size = ref.balance_grad(a, None, r["counts"], 2, False, COEF, 1.0)
    assert np.all(np.abs(dalpha.double().cpu().numpy() - g) <= 2 * ref.E * size)
