"""Forward, loss and gradient operators around the fused weight-gradient step, measured.

Three operators of a language model's training and serving step, each next to the fused
weight-gradient + optimizer step that consumes what it produces:

* the linear layer's product with bias, activation and residual in its epilogue, and the
  backward pass of that epilogue (gradient through the activation, bias gradient);
* the gated feed-forward block: both projections, activation and product in one kernel,
  and its backward pass (the gradients of both projections from the output gradient of
  the layer behind it, and the input gradient summed over both projections);
* softmax cross entropy of a linear head over a large vocabulary, in pieces of the
  vocabulary, without keeping the logits, and its gradients.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU, `run()` one
pass (the framework's calls where `own` is true, elementary torch operations in float32
where it is false), `work()` what a pass cannot do without, `exact()` the same outputs in
float64 from the definitions.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100


def _case(name, op, **kw):
    c = {"op": op, "dtype": "bf16"}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token through a square attention projection: latency, the weight is read once
        _case("linear one token", "linear", t=1, n_in=4096, n_out=4096, bias=True, act="none", res=True),
        # a prompt of odd length through an expanding projection of a biased, ungated MLP
        _case("linear prompt", "linear", t=777, n_in=4096, n_out=14336, bias=True, act="gelu", res=False),
        # down projection of a training step, the block's residual added in the epilogue
        _case("linear residual", "linear", t=8192, n_in=14336, n_out=4096, bias=False, act="none", res=True),
        # the float32 layer size that the framework's own fp32 benchmark uses
        _case("linear float32", "linear", t=512, n_in=256, n_out=256, bias=True, act="silu", res=True, dtype="f32"),
        # backward of the epilogue of a biased MLP layer: an odd number of tokens, memory bound
        _case("linear epilogue backward", "linear_bwd", t=8191, n_out=14336, act="gelu"),
        # one decoded token through gate and up
        _case("gated one token", "gated", t=1, n_in=4096, n_hid=14336, act="silu", save=False),
        # gate and up of a training step, projections kept for backward
        _case("gated train", "gated", t=8192, n_in=4096, n_hid=14336, act="silu", save=True),
        # backward of the whole gated block in a training step
        _case("gated backward", "gated_bwd", t=8192, n_in=4096, n_hid=14336, act="silu"),
        # backward on a shard with a ragged micro-batch
        _case("gated backward shard", "gated_bwd", t=1001, n_in=5120, n_hid=2176, act="gelu"),
        # loss of a training step and both gradients
        _case("loss train", "loss_train", t=8192, n_in=4096, n_voc=32768, ignored=0.0),
        # an odd vocabulary, an odd number of tokens, a tenth of them padding
        _case("loss train ragged", "loss_train", t=1999, n_in=1024, n_voc=50257, ignored=0.1),
        # evaluation: the loss of every token over a large vocabulary, no gradient
        _case("loss evaluation", "loss", t=4096, n_in=4096, n_voc=131072, ignored=0.05),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of `step`."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(x / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd", "gated_bwd", "loss", "loss_train",
                     "loss_train"])
    f32 = op in ("linear", "gated") and rng.random() < 0.15
    dt = "f32" if f32 else "bf16"
    t = rng.choice([1, 2, 3, 4, 7, 8]) if op in ("linear", "gated") and rng.random() < 0.3 else _log(rng, 5, 8192)
    if f32:
        t = min(t, 700)
    big = 1024 if f32 else 16384
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "linear":
        return _case(None, op, t=t, n_in=_log(rng, 64, big, 8), n_out=_log(rng, 64, big, 8), bias=rng.random() < 0.6,
                     act=rng.choice([act, "none"]), res=rng.random() < 0.5, dtype=dt)
    if op == "linear_bwd":
        return _case(None, op, t=t, n_out=_log(rng, 64, 16384, 8), act=act)
    if op == "gated":
        return _case(None, op, t=t, n_in=_log(rng, 64, min(big, 8192), 8), n_hid=_log(rng, 64, big, 8), act=act,
                     save=rng.random() < 0.6, dtype=dt)
    if op == "gated_bwd":
        return _case(None, op, t=t, n_in=_log(rng, 64, 5120, 8), n_hid=_log(rng, 64, 14336, 8), act=act)
    # the head: any vocabulary, odd ones included
    return _case(None, op, t=t, n_in=_log(rng, 64, 4096, 8), n_voc=_log(rng, 500, 32768),
                 ignored=rng.choice([0.0, 0.1, 0.5]))


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    dt = F32 if case["dtype"] == "f32" else BF16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=F32) * std).to(dt)

    op, t = case["op"], case["t"]
    s = dict(case)
    if op == "linear":
        i, o = case["n_in"], case["n_out"]
        s["X"], s["W"] = normal(t, i), normal(o, i, std=i ** -0.5)
        s["b"] = normal(o, std=0.5) if case["bias"] else None
        s["R"] = normal(t, o) if case["res"] else None
    elif op == "linear_bwd":
        s["dY"], s["Z"] = normal(t, case["n_out"], std=1e-3), normal(t, case["n_out"], std=1.5)
    elif op == "gated":
        i, h = case["n_in"], case["n_hid"]
        s["X"], s["Wg"], s["Wu"] = normal(t, i), normal(h, i, std=i ** -0.5), normal(h, i, std=i ** -0.5)
    elif op == "gated_bwd":
        i, h = case["n_in"], case["n_hid"]
        s["dY"] = normal(t, i, std=1e-3)
        s["G"], s["U"] = normal(t, h), normal(t, h)
        s["Wg"], s["Wu"] = normal(h, i, std=i ** -0.5), normal(h, i, std=i ** -0.5)
        s["Wd"] = normal(i, h, std=h ** -0.5)
    else:
        i, v = case["n_in"], case["n_voc"]
        y = torch.randint(0, v, (t,), generator=g, device=dev)
        s["W"] = normal(v, i, std=2.0 * i ** -0.5)
        # hidden states that already lean towards their target, as those of a partly trained model
        x = torch.randn(t, i, generator=g, device=dev, dtype=F32)
        lean = torch.rand(t, 1, generator=g, device=dev, dtype=F32) * 3.0
        s["X"] = (x + lean * s["W"][y].float()).to(dt)
        drop = torch.rand(t, generator=g, device=dev) < case["ignored"]
        drop[0] = False  # a batch holds one token at least that counts
        s["y"] = torch.where(drop, torch.full_like(y, IGNORE), y)
        s["dloss"] = torch.ones((), device=dev, dtype=F32)
    return s


# --------------------------------------------------------------------------- plain form

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    return 0.5 * z * (1.0 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    u = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + u) + 0.5 * z * (1.0 - u * u) * 0.7978845608028654 * (1.0 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    z = s["X"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return [y.to(s["X"].dtype)]


def _plain_linear_bwd(s):
    dz = s["dY"].float() * _act_grad(s["Z"].float(), s["act"])
    return [dz.to(s["dY"].dtype), dz.sum(0)]


def _plain_gated(s):
    x = s["X"].float()
    gt, up = x @ s["Wg"].float().t(), x @ s["Wu"].float().t()
    dt = s["X"].dtype
    h = (_act(gt, s["act"]) * up).to(dt)
    return [h, gt.to(dt), up.to(dt)] if s["save"] else [h]


def _plain_gated_bwd(s):
    dh = s["dY"].float() @ s["Wd"].float()
    gt, up = s["G"].float(), s["U"].float()
    a = _act(gt, s["act"])
    du, dg = dh * a, dh * up * _act_grad(gt, s["act"])
    dx = dg @ s["Wg"].float() + du @ s["Wu"].float()
    dt = s["dY"].dtype
    return [dg.to(dt), du.to(dt), (a * up).to(dt), dx.to(dt)]


def _plain_loss(s):
    z = s["X"].float() @ s["W"].float().t()
    top = z.max(dim=1, keepdim=True).values
    lse = (z - top).exp().sum(1).log() + top[:, 0]
    keep = s["y"] != IGNORE
    yc = torch.where(keep, s["y"], torch.zeros_like(s["y"]))
    loss = torch.where(keep, lse - z.gather(1, yc[:, None])[:, 0], torch.zeros_like(lse))
    if s["op"] == "loss":
        return [loss, lse]
    n = keep.sum().float()
    p = (z - lse[:, None]).exp()
    p.scatter_add_(1, yc[:, None], torch.full_like(p[:, :1], -1.0))
    p = p * (keep.float() * (s["dloss"] / n))[:, None]
    dt = s["X"].dtype
    return [loss.sum() / n, (p @ s["W"].float()).to(dt), (p.t() @ s["X"].float()).to(dt)]


# --------------------------------------------------------------------------- the framework's calls

def _own_run(s):
    import optimizer_gemm_amd as forge
    op = s["op"]
    if op == "linear":
        return [forge.linear(s["X"], s["W"], bias=s["b"], act=s["act"], residual=s["R"])]
    if op == "linear_bwd":
        return list(forge.linear_act_backward(s["dY"], s["Z"], act=s["act"]))
    if op == "gated":
        if s["save"]:
            return list(forge.gated(s["X"], s["Wg"], s["Wu"], act=s["act"], save=True))
        return [forge.gated(s["X"], s["Wg"], s["Wu"], act=s["act"])]
    if op == "gated_bwd":
        dg, du, h = forge.gated_dgrad(s["dY"], s["Wd"], s["G"], s["U"], act=s["act"])
        return [dg, du, h, forge.dgrad_group([dg, du], [s["Wg"], s["Wu"]])]
    if op == "loss":
        loss, lse, _ = forge.linear_cross_entropy(s["X"], s["W"], s["y"], ignore_index=IGNORE, reduction="none")
        return [loss, lse]
    loss, lse, total = forge.linear_cross_entropy(s["X"], s["W"], s["y"], ignore_index=IGNORE, reduction="mean")
    dx, dw = forge.linear_cross_entropy_backward(s["X"], s["W"], s["y"], lse, s["dloss"], ignore_index=IGNORE,
                                                 reduction="mean", total=total)
    return [loss, dx, dw]


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "linear":
        return _plain_linear(state)
    if op == "linear_bwd":
        return _plain_linear_bwd(state)
    if op == "gated":
        return _plain_gated(state)
    if op == "gated_bwd":
        return _plain_gated_bwd(state)
    return _plain_loss(state)


# --------------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    t, op = case["t"], case["op"]
    if op == "linear":
        i, o = case["n_in"], case["n_out"]
        return {"bytes": e * (t * i + o * i + t * o * (2 if case["res"] else 1) + (o if case["bias"] else 0)),
                "flops": 2 * t * i * o}
    if op == "linear_bwd":
        return {"bytes": e * 3 * t * case["n_out"] + 4 * case["n_out"], "flops": 10 * t * case["n_out"]}
    if op == "gated":
        i, h = case["n_in"], case["n_hid"]
        return {"bytes": e * (t * i + 2 * h * i + t * h * (3 if case["save"] else 1)), "flops": 4 * t * i * h}
    if op == "gated_bwd":
        i, h = case["n_in"], case["n_hid"]
        return {"bytes": e * (2 * t * i + 3 * h * i + 5 * t * h), "flops": 6 * t * i * h}
    i, v = case["n_in"], case["n_voc"]
    if op == "loss":
        return {"bytes": e * (t * i + v * i) + 16 * t, "flops": 2 * t * i * v}
    return {"bytes": e * 2 * (t * i + v * i) + 8 * t, "flops": 6 * t * i * v}


# --------------------------------------------------------------------------- float64 from the definitions

def _phi64(z, act):
    """act(z) and its derivative in float64."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        pos = z > 0
        return torch.where(pos, z, torch.zeros_like(z)), pos.double()
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c, k = math.sqrt(2 / math.pi), 0.044715
    th = torch.tanh(c * (z + k * z ** 3))
    return z * (1 + th) / 2, (1 + th) / 2 + z * (1 - th ** 2) * c * (1 + 3 * k * z ** 2) / 2


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "linear":
        z = torch.mm(d["X"], d["W"].t().contiguous())
        y = _phi64(z + d["b"] if "b" in d else z, case["act"])[0]
        return [y + d["R"] if "R" in d else y]
    if op == "linear_bwd":
        dz = d["dY"] * _phi64(d["Z"], case["act"])[1]
        return [dz, torch.sum(dz, dim=0)]
    if op == "gated":
        gt, up = torch.mm(d["X"], d["Wg"].t().contiguous()), torch.mm(d["X"], d["Wu"].t().contiguous())
        h = _phi64(gt, case["act"])[0] * up
        return [h, gt, up] if case["save"] else [h]
    if op == "gated_bwd":
        dh = torch.mm(d["dY"], d["Wd"])
        a, a1 = _phi64(d["G"], case["act"])
        dg, du = dh * d["U"] * a1, dh * a
        return [dg, du, a * d["U"], torch.mm(dg, d["Wg"]) + torch.mm(du, d["Wu"])]
    z = torch.mm(d["X"], d["W"].t().contiguous())
    lse = torch.logsumexp(z, dim=1)
    rows = torch.nonzero(s["y"] != IGNORE)[:, 0]
    per = torch.zeros_like(lse)
    per[rows] = lse[rows] - z[rows, s["y"][rows]]
    if op == "loss":
        return [per, lse]
    gz = torch.zeros_like(z)
    gz[rows] = torch.softmax(z[rows], dim=1)
    gz[rows, s["y"][rows]] -= 1
    gz *= d["dloss"] / rows.numel()
    return [per.sum() / rows.numel(), torch.mm(gz, d["W"]), torch.mm(gz.t().contiguous(), d["X"])]
