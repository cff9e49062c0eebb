"""What a training step of dynamic-convolution layers does around the layers' own
backward, as measurable cases.

Three operators:

* ``balance``: the load-balance loss of a router (per-expert counts of the top-k
  choices, mean probabilities, the loss) and its gradient with respect to the
  attentions, added to or written as ``dalpha``;
* ``norm``: the 2-norm of a list of gradients and the factor that clips it;
* ``adamw``: one AdamW step over a list of tensors, with the two states in 32 bits or
  in 8 bits (e4m3 codes with one fp32 scale per 256 elements); ``step`` is the two
  together, the norm's factor feeding the step, the step number on the device.

``own`` chooses between the plain torch form and the package's kernels.
"""
import math

import torch

own = False

BLOCK = 256                       # elements per scale of an 8-bit state
E4M3_MAX = 448.0
TINY = 2.0 ** -100                # a block whose largest magnitude is below is stored as zeros
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.01
COEF = 0.01                       # weight of the balance loss
STEP = 7                          # the step's number, where the host gives it
MAX_NORM = 1.0
MASK32 = 0xFFFFFFFF


# ---------------------------------------------------------------- the cases


def _balance(rows, n, k, mode="softmax", groups=1, mask=False, pad=0, accumulate=True):
    return {"op": "balance", "rows": rows, "groups": groups, "n": n, "k": k, "mode": mode,
            "mask": mask, "pad": pad, "accumulate": accumulate}


def _tensors(op, layers, n, c_out, c_in, kernel, params="bf16+master", grads="fp32", state=32):
    return {"op": op, "layers": layers, "n": n, "c_out": c_out, "c_in": c_in, "kernel": kernel,
            "params": params, "grads": grads, "state": state}


def listed():
    cases = {
        # the router of one 3x3 layer, 64 samples, 4 experts: a call's latency
        "balance one layer": _balance(64, 4, 1),
        # 16 kernel cells, each a mixture of a warehouse of 128: a router per cell
        "balance cells": _balance(64, 128, 4, groups=16, accumulate=False),
        # sigmoid attentions of a long stream of positions with padded ones masked out
        "balance long": _balance(1_000_003, 16, 2, mode="sigmoid", mask=True),
        # hundreds of experts, eight chosen, rows inside a wider buffer
        "balance wide": _balance(30_011, 1000, 8, mask=True, pad=24),
        # one 3x3 layer's four gradients: a call's latency
        "norm one layer": _tensors("norm", 1, 4, 128, 128, 3),
        # twelve layers whose other framework leaves bf16 gradients
        "norm stack bf16": _tensors("norm", 12, 16, 256, 256, 3, grads="bf16"),
        # the 64-expert layer: 151 M gradients
        "norm large": _tensors("norm", 1, 64, 512, 512, 3),
        # one 3x3 layer: bf16 experts with fp32 master copies
        "adamw one layer": _tensors("adamw", 1, 4, 128, 128, 3),
        # a stack of deep 3x3 layers
        "adamw stack": _tensors("adamw", 8, 16, 256, 256, 3),
        # many small 1x1 layers, no master copies, bf16 gradients, 8-bit states
        "adamw 8-bit small layers": _tensors("adamw", 40, 8, 243, 41, 1, params="bf16",
                                             grads="bf16", state=8),
        # the 64-expert layer with 8-bit states
        "adamw 8-bit large": _tensors("adamw", 1, 64, 512, 512, 3, state=8),
        # the whole update as a training loop runs it: clip, then step
        "step stack": _tensors("step", 8, 16, 256, 256, 3),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.4:
        n = _log_int(rng, 1, 1024)
        groups = 1 if rng.random() < 0.6 else _log_int(rng, 2, max(2, min(32, 4096 // n)))
        rows = _log_int(rng, 1, max(16, 30_000_000 // (n * groups)))
        return _balance(rows, n, rng.randint(1, min(n, 12)), rng.choice(("softmax", "sigmoid")),
                        groups, rng.random() < 0.5, rng.choice((0, 0, 4, 7)),
                        rng.random() < 0.5)
    op = rng.choice(("norm", "adamw", "adamw", "step"))
    kernel = rng.choice((1, 3, 3, 5))
    n, c_out, c_in = _log_int(rng, 1, 64), _log_int(rng, 8, 512), _log_int(rng, 8, 512)
    one = n * c_out * c_in * kernel * kernel
    layers = _log_int(rng, 1, max(1, min(24, 75_000_000 // one)))
    while layers * one > 75_000_000:
        n = max(1, n // 2)
        one = n * c_out * c_in * kernel * kernel
    return _tensors(op, layers, n, c_out, c_in, kernel,
                    rng.choice(("fp32", "bf16", "bf16+master")), rng.choice(("fp32", "bf16")),
                    rng.choice((32, 8)))


# ---------------------------------------------------------------- the inputs


def _sizes(case):
    """Element counts of the experts and of the small tensors (expert biases, router
    weight, router bias), layer by layer."""
    experts = [case["n"] * case["c_out"] * case["c_in"] * case["kernel"] ** 2] * case["layers"]
    small = [case["n"] * case["c_out"], case["n"] * case["c_in"], case["n"]] * case["layers"]
    return experts, small


class Flat:
    """Tensors of one kind in flat buffers, each starting at a multiple of BLOCK."""

    def __init__(self, sizes, first, params, grads, state, decay, gen):
        self.sizes, self.first, self.params, self.state, self.decay = sizes, first, params, state, decay
        blocks = [-(-s // BLOCK) for s in sizes]
        self.starts = [BLOCK * sum(blocks[:i]) for i in range(len(sizes))]
        total = BLOCK * sum(blocks)
        count = torch.tensor(blocks, device="cuda")
        self.ordinal = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), count)
        begin = torch.tensor(self.starts, device="cuda")[self.ordinal]
        # first element of each block, counted within its tensor
        self.begin = torch.arange(sum(blocks), device="cuda") * BLOCK - begin
        inside = torch.zeros(total, dtype=torch.bool, device="cuda")
        for o, s in zip(self.starts, sizes):
            inside[o:o + s] = True

        def normal():
            return torch.randn(total, device="cuda", generator=gen) * inside

        # gradients with heavy tails, some exactly zero (channels that saw no input)
        g = normal() * torch.exp(normal()) * 1e-3
        self.dead = torch.rand(total, device="cuda", generator=gen) < 0.03
        g = torch.where(self.dead, 0.0, g)
        m = normal() * 3e-4
        v = (normal() * torch.exp(0.5 * normal()) * 1e-3).square()
        p = normal() * 0.03
        self.g = g if grads == "fp32" else g.bfloat16()
        self.master = p if params == "bf16+master" else None
        self.p = p.clone() if params == "fp32" else p.bfloat16()
        self.m_scale = self.v_scale = None
        if state == 32:
            self.m, self.v = m, v
        else:
            self.m, self.m_scale = self._store(m)
            self.v, self.v_scale = self._store(v.sqrt())

    @staticmethod
    def _store(x):
        x = x.view(-1, BLOCK)
        scale = x.abs().amax(1) / E4M3_MAX
        return (x / scale.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1), scale

    def parts(self, t):
        return [None if t is None else t[o:o + s] for o, s in zip(self.starts, self.sizes)]

    def scale_parts(self, t):
        return [None if t is None else t[o // BLOCK:-(-(o + s) // BLOCK)]
                for o, s in zip(self.starts, self.sizes)]

    def outputs(self):
        out = {"p": self.p, "m": self.m, "v": self.v, "master": self.master,
               "m_scale": self.m_scale, "v_scale": self.v_scale}
        return {k: t for k, t in out.items() if t is not None}


def _prepare_balance(case, gen):
    rows, width = case["rows"], case["groups"] * case["n"]
    wide = width + case["pad"]
    z = torch.randn(rows, case["groups"], case["n"], device="cuda", generator=gen)
    z = z + 0.5 * torch.randn(1, case["groups"], case["n"], device="cuda", generator=gen)
    # one row in eight has logits on a coarse grid, so that its attentions tie
    tied = torch.rand(rows, 1, 1, device="cuda", generator=gen) < 0.125
    z = torch.where(tied, z.round(), z)
    a = torch.softmax(z, -1) if case["mode"] == "softmax" else torch.sigmoid(z)
    alpha = torch.full((rows, wide), float("nan"), device="cuda")
    alpha[:, :width] = a.view(rows, width)
    mask = None
    if case["mask"]:
        mask = torch.rand(rows, device="cuda", generator=gen) < 0.8
        alpha[~mask] = float("nan")    # a padded row holds whatever was there before
    dalpha = torch.zeros(rows, wide, device="cuda")
    if case["accumulate"]:
        dalpha[:, :width] = 1e-6 * torch.randn(rows, width, device="cuda", generator=gen)
    dloss = 0.5 + torch.rand(1, device="cuda", generator=gen)
    f32, i32 = torch.float32, torch.int32
    shape = (case["groups"], case["n"])
    return {"case": case, "alpha": alpha[:, :width], "mask": mask, "dalpha": dalpha[:, :width],
            "dloss": dloss, "counts": torch.empty(shape, dtype=i32, device="cuda"),
            "mean": torch.empty(shape, dtype=f32, device="cuda"),
            "kept": torch.empty(1, dtype=i32, device="cuda"),
            "loss": torch.empty(1, dtype=f32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "balance":
        return _prepare_balance(case, gen)
    experts, small = _sizes(case)
    return {"case": case, "seed": seed & MASK32,
            "flats": [Flat(experts, 0, case["params"], case["grads"], case["state"], DECAY, gen),
                      Flat(small, len(experts), "fp32", "fp32", 32, 0.0, gen)],
            "stats": torch.zeros(2, device="cuda"),
            "step": torch.full((1,), STEP, dtype=torch.int64, device="cuda")}


# ------------------------------------------------------------- the plain form


def _mix(x):
    """Multiply-xorshift hash of 32-bit values held in int64."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & MASK32
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & MASK32
    return x ^ (x >> 16)


def _dither(flat, seed, step):
    """16 bits for every element: half of the hash of its pair's number, keyed by the
    call's seed and step and by the tensor's place in the list. [blocks][BLOCK]."""
    seed = torch.full((), seed, dtype=torch.int64, device="cuda")
    key = _mix(_mix(_mix(seed) ^ (step & MASK32)) ^ (flat.ordinal + flat.first))
    pair = flat.begin[:, None] // 2 + torch.arange(BLOCK // 2, device="cuda")
    h = _mix(key[:, None] ^ pair)
    return torch.stack((h & 0xFFFF, h >> 16), -1).view(-1, BLOCK).int()


def _store_e4m3(x, u, positive):
    """Block scales and dithered e4m3 codes of x [blocks][BLOCK]; a positive value never
    becomes zero where `positive` is set (a root of a second moment)."""
    top = x.abs().amax(1)
    fine = top >= TINY
    scale = torch.where(fine, top * (1.0 / E4M3_MAX), 0.0)
    inv = torch.where(fine, top.reciprocal() * E4M3_MAX, 0.0)
    y = x.abs() * inv[:, None]
    base = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)   # below: the fixed spacing 2^-9
    bits = (y + base).view(torch.int32) + (u << 4)
    q = ((bits & -(1 << 20)).view(torch.float32) - base).clamp_max(E4M3_MAX)
    if positive:
        q = torch.where((x > 0) & fine[:, None], q.clamp_min(2.0 ** -9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(-1), scale


def _adamw_plain(flat, seed, step, scale):
    """One step in place, fp32 arithmetic; `step` is an int64 tensor."""
    bc1 = 1.0 - BETA1 ** step.double()
    bc2 = 1.0 - BETA2 ** step.double()
    size, root2 = (LR / bc1).float(), bc2.rsqrt().float()
    g = flat.g.float()
    if scale is not None:
        g = g * scale
    if flat.state == 32:
        m, v = flat.m, flat.v
    else:
        m = (flat.m.float().view(-1, BLOCK) * flat.m_scale[:, None]).view(-1)
        r = (flat.v.float().view(-1, BLOCK) * flat.v_scale[:, None]).view(-1)
        v = r * r
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    root = v.sqrt()
    p = flat.p.float() if flat.master is None else flat.master
    p = p * (1.0 - LR * flat.decay) - m / (root * root2 + EPS) * size
    u = None
    if flat.state == 8 or flat.params == "bf16":
        u = _dither(flat, seed, step)
    if flat.state == 32:
        flat.m.copy_(m)
        flat.v.copy_(v)
    else:
        for x, code, top, positive in ((m, flat.m, flat.m_scale, False),
                                       (root, flat.v, flat.v_scale, True)):
            q, s = _store_e4m3(x.view(-1, BLOCK), u, positive)
            code.copy_(q)
            top.copy_(s)
    if flat.params == "bf16":        # no master copy: rounded up or down by the dither
        bits = (p.view(torch.int32) + u.view(-1)) & -(1 << 16)
        flat.p.copy_(bits.view(torch.float32))
    else:
        flat.p.copy_(p)
        if flat.master is not None:
            flat.master.copy_(p)


def _norm_plain(flats):
    total = sum(f.g.double().square().sum() for f in flats).sqrt()
    return torch.stack((total, (MAX_NORM / (total + 1e-6)).clamp_max(1.0))).float()


def _balance_plain(s):
    c = s["case"]
    rows, groups, n, k = c["rows"], c["groups"], c["n"], c["k"]
    a = s["alpha"].reshape(rows, groups, n)
    keep = s["mask"]
    if keep is not None:
        a = torch.where(keep[:, None, None], a, 0.0)
    kept = torch.full((), rows, device="cuda") if keep is None else keep.sum()
    chosen = torch.sort(a, dim=-1, descending=True, stable=True).indices[..., :k]
    hit = torch.zeros(rows, groups, n, dtype=torch.int32, device="cuda").scatter_(2, chosen, 1)
    if keep is not None:
        hit = hit * keep[:, None, None]
    counts = hit.sum(0, dtype=torch.int32)
    p, total = a, None
    if c["mode"] == "sigmoid":
        total = a.sum(-1, keepdim=True)
        p = torch.where(total != 0, a / total, 0.0)
    over = 1.0 / kept.clamp_min(1).double()
    mean = p.sum(0, dtype=torch.float64) * over
    weight = (COEF * n / (k * groups)) * over * counts.double()
    loss = (weight * mean).sum()
    d = (weight * over * s["dloss"].double()).float()
    grad = d.expand(rows, groups, n)
    if total is not None:
        grad = torch.where(total != 0, (grad - (grad * p).sum(-1, keepdim=True)) / total, 0.0)
    if keep is not None:
        grad = torch.where(keep[:, None, None], grad, 0.0)
    grad = grad.reshape(rows, groups * n)
    if c["accumulate"]:
        s["dalpha"].add_(grad)
    else:
        s["dalpha"].copy_(grad)
    return {"loss": loss.float().view(1), "counts": counts, "mean": mean.float(),
            "kept": kept.int().view(1), "dalpha": s["dalpha"]}


# ------------------------------------------------------------ the package's form


def _own_tensors(s):
    """The list of tensors that a program keeps beside its parameters."""
    import dynamic_convolution_b200 as dc
    if "tensors" not in s:
        every = []
        for f in s["flats"]:
            for p, g, m, v, master, ms, vs in zip(
                    f.parts(f.p), f.parts(f.g), f.parts(f.m), f.parts(f.v), f.parts(f.master),
                    f.scale_parts(f.m_scale), f.scale_parts(f.v_scale)):
                every.append(dc.train_tensor(grad=g, param=p, m=m, v=v, master=master, m_scale=ms,
                                             v_scale=vs, weight_decay=f.decay))
        s["tensors"] = dc.train_tensors(every)
        size = dc.dynconv_grad_norm_workspace_size(s["tensors"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return dc, s["tensors"]


def _own_balance(s):
    import dynamic_convolution_b200 as dc
    c = s["case"]
    if "desc" not in s:
        s["desc"] = dc.make_balance_desc(
            c["rows"], c["n"], groups=c["groups"], top_k=c["k"],
            mode=dc.SOFTMAX if c["mode"] == "softmax" else dc.SIGMOID,
            row_stride=s["alpha"].stride(0))
        size = dc.dynconv_balance_workspace_size(s["desc"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    dc.check(dc.dynconv_balance_forward(s["desc"], s["alpha"], s["mask"], COEF, s["counts"],
                                        s["mean"], s["kept"], s["loss"], s["workspace"],
                                        s["workspace"].numel()))
    dc.check(dc.dynconv_balance_backward(s["desc"], s["alpha"], s["mask"], COEF, s["counts"],
                                         s["kept"], s["dloss"], s["dalpha"],
                                         s["dalpha"].stride(0), c["accumulate"]))
    return {k: s[k] for k in ("loss", "counts", "mean", "kept", "dalpha")}


def _outputs(s, norm):
    out = [f.outputs() for f in s["flats"]]
    return {"layers": out[0], "small": out[1], **({"norm": norm} if norm is not None else {})}


def run(state):
    s, op = state, state["case"]["op"]
    if op == "balance":
        return _own_balance(s) if own else _balance_plain(s)
    if op == "norm":
        if not own:
            return _norm_plain(s["flats"])
        dc, tensors = _own_tensors(s)
        dc.check(dc.dynconv_grad_norm(tensors, MAX_NORM, s["stats"], None, s["workspace"],
                                      s["workspace"].numel()))
        return s["stats"]
    if own:
        dc, tensors = _own_tensors(s)
        hyper = dc.make_adamw(LR, BETA1, BETA2, EPS, STEP, s["seed"])
        if op == "adamw":
            dc.check(dc.dynconv_adamw(tensors, hyper))
            return _outputs(s, None)
        dc.check(dc.dynconv_grad_norm(tensors, MAX_NORM, s["stats"], s["step"], s["workspace"],
                                      s["workspace"].numel()))
        dc.check(dc.dynconv_adamw(tensors, hyper, grad_scale=s["stats"][1:], step=s["step"]))
        return _outputs(s, s["stats"])
    norm, step = None, s["step"][0]
    if op == "step":
        norm = _norm_plain(s["flats"])
        s["step"].add_(1)
    for f in s["flats"]:
        _adamw_plain(f, s["seed"], step, None if norm is None else norm[1])
    return _outputs(s, norm)


# ------------------------------------------------------------------ accounting


def work(case):
    if case["op"] == "balance":
        width = case["rows"] * case["groups"] * case["n"]
        softmax = case["mode"] == "softmax"
        touched = width * (0.8 if case["mask"] else 1.0)
        dalpha = 8 * touched if case["accumulate"] else 4 * width
        return {"bytes": 4 * touched + dalpha + (case["rows"] if case["mask"] else 0),
                "flops": touched * (2 + case["k"] + (0 if softmax else 5))}
    experts, small = (sum(x) for x in _sizes(case))
    g = 4 if case["grads"] == "fp32" else 2
    if case["op"] == "norm":
        return {"bytes": g * experts + 4 * small, "flops": 2 * (experts + small)}
    p = {"fp32": 8, "bf16": 4, "bf16+master": 10}[case["params"]]
    state = 16 if case["state"] == 32 else 4 + 16 / BLOCK
    more = 2 if case["op"] == "step" else 0
    return {"bytes": experts * (g + p + state) + small * 28,
            "flops": (experts + small) * (14 + more + (0 if case["state"] == 32 else 30))}


# ------------------------------------------------------- the definition in 64 bits


def _exact_balance(s):
    c = s["case"]
    rows, groups, n, k = c["rows"], c["groups"], c["n"], c["k"]
    live = torch.ones(rows, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    a = s["alpha"][live].double().view(-1, groups, n)
    kept = a.shape[0]
    counts = torch.zeros(groups, n, dtype=torch.int64, device="cuda")
    mean = torch.zeros(groups, n, dtype=torch.float64, device="cuda")
    out = s["dalpha"].double().clone()
    if kept:
        left, at = a.clone(), torch.arange(n, device="cuda")
        for _ in range(k):   # the largest, the lowest place first
            best = left.amax(-1, keepdim=True)
            first = torch.where(left == best, at, n).amin(-1, keepdim=True)
            counts += (at == first).sum(0)
            left = torch.where(at == first, -math.inf, left)
        total = a.sum(-1, keepdim=True) if c["mode"] == "sigmoid" else torch.ones_like(a[..., :1])
        mean = (a / total).mean(0)
        slope = COEF * n / (k * groups) * counts / kept / kept * s["dloss"].double()
        if c["mode"] == "softmax":
            grad = slope.expand(kept, groups, n)
        else:
            grad = slope / total - (slope * a).sum(-1, keepdim=True) / total ** 2
        grad = grad.reshape(kept, groups * n)
        out[live] = out[live] + grad if c["accumulate"] else grad
    loss = COEF * n / (k * groups) * (counts / max(kept, 1) * mean).sum()
    return {"loss": loss.view(1), "counts": counts, "mean": mean,
            "kept": torch.tensor([kept]), "dalpha": out}


def _exact_e4m3(x, u, positive):
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top >= TINY, top / E4M3_MAX, 0.0)
    y = torch.where(scale > 0, x.abs() / scale.clamp_min(1e-300), 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    q = (torch.floor(y / step + u.double() / 65536) * step).clamp_max(E4M3_MAX)
    if positive:
        q = torch.where((x > 0) & (scale > 0), q.clamp_min(2.0 ** -9), q)
    return (q * torch.sign(x)).view(-1), scale.view(-1)


def _exact_adamw(flat, seed, step, scale):
    g = flat.g.double() * scale
    if flat.state == 32:
        m, v = flat.m.double(), flat.v.double()
    else:
        m = (flat.m.double().view(-1, BLOCK) * flat.m_scale.double()[:, None]).view(-1)
        v = (flat.v.double().view(-1, BLOCK) * flat.v_scale.double()[:, None]).view(-1) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = flat.p.double() if flat.master is None else flat.master.double()
    ratio = (m / (1 - BETA1 ** step)) / ((v / (1 - BETA2 ** step)).sqrt() + EPS)
    p = p * (1 - LR * flat.decay) - LR * ratio
    out = {"p": p, "m": m, "v": v}
    if flat.master is not None:
        out["master"] = p
    if flat.state == 8:
        u = _dither(flat, seed, torch.tensor(step, device="cuda"))
        out["m"], out["m_scale"] = _exact_e4m3(m.view(-1, BLOCK), u, False)
        out["v"], out["v_scale"] = _exact_e4m3(v.sqrt().view(-1, BLOCK), u, True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s)
    norm = None
    if case["op"] != "adamw":
        total = math.sqrt(sum(float((f.g.double() ** 2).sum()) for f in s["flats"]))
        norm = torch.tensor([total, min(1.0, MAX_NORM / (total + 1e-6))], dtype=torch.float64)
        if case["op"] == "norm":
            return norm
    step = STEP + (case["op"] == "step")
    out = [_exact_adamw(f, s["seed"], step, 1.0 if norm is None else float(norm[1]))
           for f in s["flats"]]
    return {"layers": out[0], "small": out[1], **({"norm": norm} if norm is not None else {})}
