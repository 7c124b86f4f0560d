"""Layers of experts and 8-bit products, measured.

Three operators of a language model's training and serving step beside the framework's linear layer and
gated block:

* the way of tokens to experts and back: rows grouped by expert (stable, by counting), their results
  weighted and summed per token, and the backward pass of that;
* matrix products grouped by expert with ragged sizes: the gated block and the linear layer behind it,
  their input gradients, their weight gradients, and the optimizer step of the stacked weights;
* products of 8-bit integers with a scale for each token and each output channel, plain, gated and
  grouped by expert, with the quantisation of the tokens.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU, `run()` one pass (the
framework's calls where `own` is true, elementary torch operations in float32 where it is false), `work()`
what a pass cannot do without, `exact()` the same outputs in float64 from the definitions.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
STEP, LR, B1, B2, EPS, WD = 7, 1e-3, 0.9, 0.999, 1e-8, 0.01
MU = 0.9  # SGD with momentum


def _case(name, op, **kw):
    c = {"op": op, "dtype": "bf16", "act": "silu", "dropped": 0.0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token, two of eight experts: the chosen experts' weights are read once
        _case("experts one token", "block", t=1, k=2, e=8, d=4096, h=14336),
        # a short batch over many narrow experts, a few rows each, some of them empty
        _case("experts short batch", "block", t=37, k=4, e=64, d=2048, h=1024),
        # a prompt of odd length over shards of experts, a tenth of its routes dropped (full experts, padding)
        _case("experts prompt", "block", t=1777, k=2, e=16, d=4096, h=1792, dropped=0.1),
        # backward of a training step through both layers of the block: gradients of the projections and of the input
        _case("experts backward", "block_bwd", t=8192, k=2, e=8, d=4096, h=14336),
        # the stacked weights' gradient, ragged and narrow, as the two-phase schedule stores it
        _case("experts gradient", "gradient", t=999, k=4, e=32, d=1024, h=512),
        # the optimizer step of a stacked projection of a training step, the gradient never stored
        _case("experts step", "step", t=8192, k=2, e=8, d=4096, h=1792, opt="adamw"),
        # the way in: a training batch's routes counted and ordered, its rows copied to their experts
        _case("dispatch train", "dispatch", t=8192, k=8, e=64, d=2048),
        # the way back's backward pass: the rows' gradients and the routing weights' gradients, then the input's
        _case("combine backward", "combine_bwd", t=8191, k=8, e=64, d=2048),
        # one decoded token through a square projection with 8-bit weights
        _case("8-bit one token", "q8_linear", t=1, d=4096, h=4096, act="none", bias=True, res=True),
        # a prompt through gate and up
        _case("8-bit prompt", "q8_gated", t=777, d=4096, h=14336),
        # a large batch through the down projection, the block's residual added
        _case("8-bit batch", "q8_linear", t=8192, d=14336, h=4096, act="none", bias=False, res=True),
        # a served batch through 8-bit experts: quantised once per token, then copied to its experts
        _case("8-bit experts", "q8_experts", t=515, k=2, e=8, d=4096, h=3584),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of `step`."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(x / step)) * step)


def draw(rng):
    op = rng.choice(["block", "block", "block", "block_bwd", "block_bwd", "gradient", "step", "dispatch", "combine_bwd",
                     "q8_linear", "q8_linear", "q8_gated", "q8_experts", "q8_experts"])
    q8 = op.startswith("q8")
    f32 = op in ("block", "block_bwd", "gradient", "step") and rng.random() < 0.15
    dt = "f32" if f32 else "bf16"
    few = op in ("block", "q8_linear", "q8_gated", "q8_experts") and rng.random() < 0.35
    t = rng.choice([1, 2, 3, 5, 8, 16]) if few else _log(rng, 5, 8192)
    if f32:
        t = min(t, 700)
    step = 16 if q8 else 8
    d, h = _log(rng, 64, 1024 if f32 else 4096, step), _log(rng, 64, 1024 if f32 else 14336, step)
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "q8_linear":
        return _case(None, op, t=t, d=d, h=h, act=rng.choice([act, "none"]), bias=rng.random() < 0.5, res=rng.random() < 0.5)
    if op == "q8_gated":
        return _case(None, op, t=t, d=d, h=h, act=act)
    e = _log(rng, 1, 64)
    k = min(e, rng.choice([1, 2, 2, 4, 8]))
    # no more rows than the largest listed cases, no more stacked weights
    if op in ("dispatch", "combine_bwd"):
        return _case(None, op, t=t, k=k, e=e, d=d, dtype=dt)
    t = max(1, min(t, 16384 // k))
    while 3 * e * d * h > 1 << 30:
        e = max(1, e // 2)
    k = min(k, e)
    c = _case(None, op, t=t, k=k, e=e, d=d, h=h, act=act, dtype=dt)
    if op == "block":
        c["dropped"] = rng.choice([0.0, 0.0, 0.1, 0.6])
    if op == "step":
        while e * d * c["h"] > 1 << 26:
            c["h"] = max(64, c["h"] // 16 * 8)
        c["opt"] = rng.choice(["adamw", "sgd_momentum"])
    if op == "gradient":
        while e * d * c["h"] > 1 << 27:
            c["h"] = max(64, c["h"] // 16 * 8)
    return c


# --------------------------------------------------------------------------- inputs

def _routes(c, g):
    """Experts and weights of a router: the k largest of logits whose experts differ in how often they are
    chosen; a dropped route has expert -1."""
    t, k, e = c["t"], c["k"], c["e"]
    z = torch.randn(t, e, generator=g, device="cuda", dtype=F32) + torch.randn(1, e, generator=g, device="cuda", dtype=F32)
    w, idx = torch.topk(z, k, dim=1)
    w = torch.softmax(w, dim=1)
    if c["dropped"]:
        drop = torch.rand(t, k, generator=g, device="cuda") < c["dropped"]
        drop[0, 0] = False
        idx = torch.where(drop, torch.full_like(idx, -1), idx)
    return idx.contiguous(), w.contiguous()


def _codes(w):
    """8-bit weights as a user keeps them: codes and one scale for each output channel."""
    w = w.float()
    s = w.abs().amax(dim=-1) / 127.0
    q = torch.round(w / s[..., None]).clamp(-127, 127).to(torch.int8)
    return q, s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    dt = F32 if case["dtype"] == "f32" else BF16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=F32) * std).to(dt)

    def stacked(e, n_out, n_in, make=lambda w: w):
        # one expert at a time: the float32 draws of a large stack would not fit beside it
        parts = [make(normal(n_out, n_in, std=n_in ** -0.5)) for _ in range(e)]
        if isinstance(parts[0], tuple):
            return tuple(torch.stack([p[i] for p in parts]) for i in range(len(parts[0])))
        return torch.stack(parts)

    op, t = case["op"], case["t"]
    s = dict(case)
    if op in ("q8_linear", "q8_gated"):
        d, h = case["d"], case["h"]
        # hidden states with the few large channels that real ones have
        wide = 1.0 + 9.0 * (torch.rand(1, d, generator=g, device=dev) < 0.01).to(F32)
        s["X"] = (torch.randn(t, d, generator=g, device=dev, dtype=F32) * wide).to(dt)
        if op == "q8_linear":
            s["W"], s["ws"] = _codes(normal(h, d, std=d ** -0.5))
            s["b"] = normal(h, std=0.5) if case["bias"] else None
            s["R"] = normal(t, h) if case["res"] else None
        else:
            s["Wg"], s["gs"] = _codes(normal(h, d, std=d ** -0.5))
            s["Wu"], s["us"] = _codes(normal(h, d, std=d ** -0.5))
        return s
    k, e, d = case["k"], case["e"], case["d"]
    s["idx"], s["w"] = _routes(case, g)
    if op == "dispatch":
        s["X"] = normal(t, d)
        return s
    # what an earlier call of the step made: places and groups of the routes
    offsets, pos = _plain_plan(s["idx"], e)
    n = t * k
    if op == "combine_bwd":
        s["pos"] = pos
        s["dY"], s["Yp"], s["dXp"] = normal(t, d, std=1e-3), normal(n, d), normal(n, d, std=1e-3)
        return s
    h = case["h"]
    if op == "block":
        s["X"] = normal(t, d)
        s["Wg"], s["Wu"], s["Wd"] = stacked(e, h, d), stacked(e, h, d), stacked(e, d, h)
        return s
    if op == "q8_experts":
        wide = 1.0 + 9.0 * (torch.rand(1, d, generator=g, device=dev) < 0.01).to(F32)
        s["X"] = (torch.randn(t, d, generator=g, device=dev, dtype=F32) * wide).to(dt)
        s["Wg"], s["gs"] = stacked(e, h, d, _codes)
        s["Wu"], s["us"] = stacked(e, h, d, _codes)
        return s
    s["offsets"] = offsets
    if op == "block_bwd":
        s["dYp"], s["G"], s["U"] = normal(n, d, std=1e-3), normal(n, h), normal(n, h)
        s["Wg"], s["Wu"], s["Wd"] = stacked(e, h, d), stacked(e, h, d), stacked(e, d, h)
        return s
    s["Xp"], s["dYp"] = normal(n, d), normal(n, h, std=1e-3)
    if op == "step":
        scale = 1e-3 * max(1.0, n / e) ** 0.5  # about what a gradient's elements are
        s["W"] = stacked(e, h, d)
        s["m"] = torch.randn(e, h, d, generator=g, device=dev, dtype=F32) * (0.3 * scale)
        if case["opt"] == "adamw":
            s["v"] = (torch.rand(e, h, d, generator=g, device=dev, dtype=F32) + 0.5) * scale ** 2
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
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    u = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + u) + 0.5 * z * (1.0 - u * u) * 0.7978845608028654 * (1.0 + 3 * 0.044715 * z * z)


def _plain_plan(idx, e):
    """Expert x owns rows offsets[x] .. offsets[x + 1] of the ordered routes; pos: each route's row, -1 where dropped."""
    key = idx.reshape(-1)
    key = torch.where((key < 0) | (key >= e), torch.full_like(key, e), key)
    order = torch.sort(key, stable=True).indices
    counts = (key[None, :] == torch.arange(e, device=key.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    pos = torch.empty_like(key)
    pos[order] = torch.arange(key.numel(), device=key.device)
    pos = torch.where(key < e, pos, torch.full_like(pos, -1))
    return offsets, pos.reshape(idx.shape).to(torch.int32)


def _plain_dispatch(x, pos):
    t, k = pos.shape
    flat = pos.reshape(-1).long()
    keep = torch.nonzero(flat >= 0)[:, 0]
    out = x.new_zeros((t * k,) + x.shape[1:])
    out[flat[keep]] = x[keep // k]
    return out


def _plain_combine(yp, pos, w):
    """sum over a token's routes, in float32"""
    p = pos.long()
    rows = yp.float()[torch.clamp(p, min=0)]
    f = (p >= 0).to(F32) if w is None else torch.where(p >= 0, w, torch.zeros_like(w))
    return (rows * f[:, :, None]).sum(1)


def _plain_grouped(x, w, o):
    """rows o[e] .. o[e + 1] of x times w[e] transposed; the other rows stay zero"""
    y = torch.zeros(x.shape[0], w.shape[1], device=x.device, dtype=F32)
    for e in range(w.shape[0]):
        if o[e + 1] > o[e]:
            y[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].float() @ w[e].float().t()
    return y


def _plain_quantize(x):
    x = x.float()
    s = x.abs().amax(dim=1) / 127.0
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), torch.zeros_like(x))
    return torch.clamp(q, -127.0, 127.0), s


_M64 = [(1 << 34) - 1, (1 << 37) - 1, (1 << 33) - 1]  # what a logical shift right by 30, 27, 31 leaves


def _signed(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def _plain_rounded(w, seed, step):
    """float32 weights rounded to bfloat16 with 16 random bits each: the top ones of SplitMix64's output number
    ((step << 32) | element) + 1 from state `seed`."""
    n = w.numel()
    z = torch.arange(1, n + 1, device=w.device, dtype=torch.int64) * _signed(0x9E3779B97F4A7C15)
    z = z + _signed(seed + 0x9E3779B97F4A7C15 * (step << 32))
    z = (z ^ ((z >> 30) & _M64[0])) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & _M64[1])) * _signed(0x94D049BB133111EB)
    z = z ^ ((z >> 31) & _M64[2])
    r = ((z >> 48) & 0xFFFF).to(torch.int32)
    bits = w.reshape(-1).view(torch.int32) + r
    return ((bits >> 16) << 16).view(F32).to(BF16).reshape(w.shape)


def _plain_step(s):
    o = s["offsets"].tolist()
    x, dy, w = s["Xp"], s["dYp"], s["W"]
    wn, mn = torch.empty_like(w), torch.empty_like(s["m"])
    vn = torch.empty_like(s["v"]) if "v" in s else None
    w32 = torch.empty(w.shape, device=w.device, dtype=F32)
    for e in range(w.shape[0]):
        gr = dy[o[e]:o[e + 1]].float().t() @ x[o[e]:o[e + 1]].float()
        if s["opt"] == "adamw":
            wd = w[e].float() * (1.0 - LR * WD)
            mn[e] = B1 * s["m"][e] + (1.0 - B1) * gr
            vn[e] = B2 * s["v"][e] + (1.0 - B2) * gr * gr
            den = vn[e].sqrt() / math.sqrt(1.0 - B2 ** STEP) + EPS
            w32[e] = wd - (LR / (1.0 - B1 ** STEP)) * (mn[e] / den)
        else:
            mn[e] = MU * s["m"][e] + gr
            w32[e] = w[e].float() - LR * mn[e]
    wn = w32 if w.dtype == F32 else _plain_rounded(w32, 1234, STEP)
    return [wn, mn] if vn is None else [wn, mn, vn]


def _plain(s):
    op, act, dt = s["op"], s["act"], BF16 if s["dtype"] == "bf16" else F32
    if op == "block":
        offsets, pos = _plain_plan(s["idx"], s["e"])
        o = offsets.tolist()
        xp = _plain_dispatch(s["X"], pos)
        hid = _act(_plain_grouped(xp, s["Wg"], o), act) * _plain_grouped(xp, s["Wu"], o)
        return [_plain_combine(_plain_grouped(hid, s["Wd"], o), pos, s["w"]).to(dt)]
    if op == "block_bwd":
        o = s["offsets"].tolist()
        gt, up = s["G"].float(), s["U"].float()
        dh = _plain_grouped(s["dYp"], s["Wd"].transpose(1, 2), o)
        a = _act(gt, act)
        du, dg = dh * a, dh * up * _act_grad(gt, act)
        dx = _plain_grouped(dg, s["Wg"].transpose(1, 2), o) + _plain_grouped(du, s["Wu"].transpose(1, 2), o)
        return [dg.to(dt), du.to(dt), (a * up).to(dt), dx.to(dt)]
    if op == "gradient":
        o = s["offsets"].tolist()
        return [torch.stack([s["dYp"][o[e]:o[e + 1]].float().t() @ s["Xp"][o[e]:o[e + 1]].float() for e in range(s["e"])])]
    if op == "step":
        return _plain_step(s)
    if op == "dispatch":
        offsets, pos = _plain_plan(s["idx"], s["e"])
        return [offsets, pos, _plain_dispatch(s["X"], pos)]
    if op == "combine_bwd":
        p, w, dy = s["pos"].long(), s["w"], s["dY"].float()
        rows = s["Yp"].float()[torch.clamp(p, min=0)]
        dw = torch.where(p >= 0, (rows * dy[:, None, :]).sum(2), torch.zeros_like(w))
        dyp = torch.zeros(s["Yp"].shape, device=dy.device, dtype=F32)
        for j in range(p.shape[1]):
            keep = torch.nonzero(p[:, j] >= 0)[:, 0]
            dyp[p[keep, j]] = dy[keep] * w[keep, j, None]
        return [dyp.to(dt), dw, _plain_combine(s["dXp"], s["pos"], None).to(dt)]
    q, sx = _plain_quantize(s["X"])
    if op == "q8_linear":
        z = (q @ s["W"].float().t()) * sx[:, None] * s["ws"][None, :]
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, act)
        return [(y if s["R"] is None else y + s["R"].float()).to(dt)]
    if op == "q8_gated":
        gt = (q @ s["Wg"].float().t()) * sx[:, None] * s["gs"][None, :]
        up = (q @ s["Wu"].float().t()) * sx[:, None] * s["us"][None, :]
        return [(_act(gt, act) * up).to(dt)]
    offsets, pos = _plain_plan(s["idx"], s["e"])
    o = offsets.tolist()
    qp, sp = _plain_dispatch(q, pos), _plain_dispatch(sx, pos)
    ex = torch.repeat_interleave(torch.arange(s["e"], device=q.device), offsets[1:] - offsets[:-1])
    gt = _plain_grouped(qp, s["Wg"], o) * sp[:, None] * s["gs"][ex]
    up = _plain_grouped(qp, s["Wu"], o) * sp[:, None] * s["us"][ex]
    return [(_act(gt, act) * up).to(dt)]


# --------------------------------------------------------------------------- the framework's calls

def _own_run(s):
    import optimizer_gemm_amd as forge
    op, act = s["op"], s["act"]
    if op == "block":
        offsets, pos = forge.expert_plan(s["idx"], s["e"])
        xp = forge.expert_dispatch(s["X"], pos)
        hid = forge.expert_gated(xp, s["Wg"], s["Wu"], offsets, act=act)
        yp = forge.expert_linear(hid, s["Wd"], offsets, out_dtype=F32)
        return [forge.expert_combine(yp, pos, s["w"], out_dtype=s["X"].dtype)]
    if op == "block_bwd":
        dg, du, hid = forge.expert_gated_dgrad(s["dYp"], s["Wd"], s["G"], s["U"], s["offsets"], act=act)
        return [dg, du, hid, forge.expert_dgrad_group([dg, du], [s["Wg"], s["Wu"]], s["offsets"])]
    if op == "gradient":
        return [forge.expert_wgrad(s["Xp"], s["dYp"], s["offsets"])]
    if op == "step":
        # the call steps in place; a pass starts from the same weights and moments again
        w, m, v = s["W"].clone(), s["m"].clone(), s["v"].clone() if "v" in s else None
        hyper = {"lr": LR, "beta1": B1, "beta2": B2, "eps": EPS, "weight_decay": WD} if s["opt"] == "adamw" else \
            {"lr": LR, "momentum": MU, "weight_decay": 0.0}
        forge.expert_wgrad_step(s["Xp"], s["dYp"], w, m, v, s["offsets"], s["opt"], hyper, STEP, 1234)
        return [w, m] if v is None else [w, m, v]
    if op == "dispatch":
        offsets, pos = forge.expert_plan(s["idx"], s["e"])
        return [offsets, pos, forge.expert_dispatch(s["X"], pos)]
    if op == "combine_bwd":
        dyp, dw = forge.expert_combine_backward(s["dY"], s["Yp"], s["pos"], s["w"])
        return [dyp, dw, forge.expert_combine(s["dXp"], s["pos"])]
    q, sx = forge.quantize_rows(s["X"])
    if op == "q8_linear":
        return [forge.linear_q8(q, sx, s["W"], s["ws"], bias=s["b"], act=act, residual=s["R"])]
    if op == "q8_gated":
        return [forge.gated_q8(q, sx, s["Wg"], s["gs"], s["Wu"], s["us"], act=act)]
    offsets, pos = forge.expert_plan(s["idx"], s["e"])
    qp, sp = forge.expert_dispatch(q, pos, scale=sx)
    return [forge.expert_gated_q8(qp, sp, s["Wg"], s["gs"], s["Wu"], s["us"], offsets, act=act)]


def run(state):
    return _own_run(state) if own else _plain(state)


# --------------------------------------------------------------------------- work

def work(case):
    el = 4 if case["dtype"] == "f32" else 2
    op, t, d = case["op"], case["t"], case["d"]
    if op == "q8_linear":
        h = case["h"]
        return {"bytes": el * t * d + h * d + 4 * h + el * t * h * (2 if case["res"] else 1) + (el * h if case["bias"] else 0),
                "flops": 2 * t * d * h}
    if op == "q8_gated":
        h = case["h"]
        return {"bytes": el * t * d + 2 * h * d + 8 * h + el * t * h, "flops": 4 * t * d * h}
    k, e = case["k"], case["e"]
    n = t * k * (1.0 - case["dropped"])
    routes = 12 * t * k
    if op == "dispatch":
        return {"bytes": el * (t + n) * d + routes, "flops": 0}
    if op == "combine_bwd":
        return {"bytes": el * (2 * t + 3 * n) * d + routes, "flops": 5 * n * d}
    h = case["h"]
    used = min(e, max(1, n))  # experts that hold a route, at most
    if op == "block":
        return {"bytes": el * (2 * t * d + 3 * used * d * h) + routes, "flops": 6 * n * d * h}
    if op == "block_bwd":
        return {"bytes": el * (2 * n * d + 5 * n * h + 3 * used * d * h), "flops": 6 * n * d * h}
    if op == "gradient":
        return {"bytes": el * n * (d + h) + 4 * e * d * h, "flops": 2 * n * d * h}
    if op == "step":
        moments = 2 if case["opt"] == "adamw" else 1
        return {"bytes": el * n * (d + h) + e * d * h * (2 * el + 8 * moments), "flops": 2 * n * d * h}
    return {"bytes": el * t * d + 2 * used * h * d + el * n * h + routes, "flops": 4 * n * d * h}


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


def _codes64(x):
    """codes and scales: the scale is held in float32, the code is the nearest whole number"""
    s = (x.abs().amax(dim=1).float() / 127.0).double()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    return torch.round(x / safe[:, None]).clamp(-127, 127), s


def _members(idx, e):
    """The routes of expert x in the order of tokens: (token, slot) numbers."""
    flat = idx.reshape(-1)
    return torch.nonzero(flat == e)[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case["act"]
    if op == "dispatch":  # whole numbers, and copies
        rows = torch.cat([_members(s["idx"], a) for a in range(case["e"])])
        return [None, None, s["X"].double()[rows // case["k"]]]
    if op in ("q8_linear", "q8_gated"):
        q, sx = _codes64(s["X"].double())

        def product(w, ws):
            return torch.mm(q, w.double().t().contiguous()) * (sx[:, None] * ws.double()[None, :])

        if op == "q8_gated":
            return [_phi64(product(s["Wg"], s["gs"]), act)[0] * product(s["Wu"], s["us"])]
        z = product(s["W"], s["ws"])
        y = _phi64(z if s["b"] is None else z + s["b"].double(), act)[0]
        return [y if s["R"] is None else y + s["R"].double()]
    k, e = case["k"], case["e"]
    if op == "combine_bwd":
        dyp = torch.zeros(s["Yp"].shape, device=s["Yp"].device, dtype=torch.float64)
        dw = torch.zeros(s["w"].shape, device=dyp.device, dtype=torch.float64)
        dx = torch.zeros(s["dY"].shape, device=dyp.device, dtype=torch.float64)
        for j in range(k):
            p = s["pos"][:, j].long()
            r = torch.nonzero(p >= 0)[:, 0]
            dyp[p[r]] = s["w"][r, j].double()[:, None] * s["dY"][r].double()
            dw[r, j] = (s["Yp"][p[r]].double() * s["dY"][r].double()).sum(1)
            dx[r] += s["dXp"][p[r]].double()
        return [dyp, dw, dx]
    if op == "block":
        x = s["X"].double()
        y = torch.zeros_like(x)
        for a in range(e):
            r = _members(s["idx"], a)
            if r.numel() == 0:
                continue
            xt = x[r // k]
            hid = _phi64(torch.mm(xt, s["Wg"][a].double().t().contiguous()), act)[0] * \
                torch.mm(xt, s["Wu"][a].double().t().contiguous())
            out = torch.mm(hid, s["Wd"][a].double().t().contiguous()) * s["w"].reshape(-1)[r].double()[:, None]
            y.index_add_(0, r // k, out)
        return [y]
    if op == "q8_experts":
        q, sx = _codes64(s["X"].double())
        rows = []
        for a in range(e):
            r = _members(s["idx"], a) // k

            def product(w, ws):
                return torch.mm(q[r], w[a].double().t().contiguous()) * (sx[r][:, None] * ws[a].double()[None, :])

            rows.append(_phi64(product(s["Wg"], s["gs"]), act)[0] * product(s["Wu"], s["us"]))
        return [torch.cat(rows)]
    o = s["offsets"].tolist()
    parts = []
    for a in range(e):
        lo, hi = o[a], o[a + 1]
        if op == "block_bwd":
            dh = torch.mm(s["dYp"][lo:hi].double(), s["Wd"][a].double())
            gt, up = s["G"][lo:hi].double(), s["U"][lo:hi].double()
            v, d1 = _phi64(gt, act)
            dg, du = dh * up * d1, dh * v
            parts.append((dg, du, v * up, torch.mm(dg, s["Wg"][a].double()) + torch.mm(du, s["Wu"][a].double())))
            continue
        gr = torch.mm(s["dYp"][lo:hi].double().t().contiguous(), s["Xp"][lo:hi].double())
        if op == "gradient":
            parts.append((gr,))
        elif case["opt"] == "adamw":
            m = B1 * s["m"][a].double() + (1 - B1) * gr
            v = B2 * s["v"][a].double() + (1 - B2) * gr * gr
            w = s["W"][a].double() * (1 - LR * WD) - LR / (1 - B1 ** STEP) * m / ((v / (1 - B2 ** STEP)).sqrt() + EPS)
            parts.append((w, m, v))
        else:
            m = MU * s["m"][a].double() + gr
            parts.append((s["W"][a].double() - LR * m, m))
    join = torch.cat if op == "block_bwd" else torch.stack
    outs = [join([p[i] for p in parts]) for i in range(len(parts[0]))]
    if op == "step" and s["W"].dtype == BF16:
        outs[0] = None  # rounded at random: no one value
    return outs
