"""The operators around the fused step as a training loop uses them: ForgeLinear with bias,
activation and residual, the joined SwiGLU block, the head with its cross entropy, all of
them together, on other streams, at once, and captured in HIP graphs."""
import pytest
import torch

import optimizer_gemm_amd as forge
from _ops64 import act64, close, linear64, mm64
from optimizer_gemm_amd.nn import ForgeHead, ForgeLinear, SwiGLUBlock, linear_cross_entropy, step_all

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("act", forge.ACTS)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_layer_with_epilogue(act, bias):
    """Forward against float64; dX, the residual's gradient and the updates equal the calls made
    one by one."""
    W = rnd(1, 264, 136, std=0.1)
    x, r, dy = rnd(2, 3, 35, 136).requires_grad_(), rnd(3, 3, 35, 264).requires_grad_(), rnd(4, 3, 35, 264, std=1e-2)
    layer = ForgeLinear(136, 264, weight=W.clone(), seed=5, bias=bias, act=act)
    if bias:
        with torch.no_grad():
            layer.bias.copy_(rnd(6, 264))
    b0 = layer.bias.detach().clone() if bias else None
    y = layer(x, r)
    close("y", y.reshape(-1, 264), *linear64(x.reshape(-1, 136), W, b0, act, r.reshape(-1, 264))[:2])
    y.backward(dy)
    assert torch.equal(r.grad, dy) and layer.weight.grad is None
    x2, dy2 = x.detach().reshape(-1, 136), dy.reshape(-1, 264)
    _, z = forge.linear(x2, W, bias=b0, act=act, residual=r.detach().reshape(-1, 264), save=True)
    dz, db = forge.linear_act_backward(dy2, z, act=act)
    assert torch.equal(x.grad.reshape(-1, 136), forge.dgrad(dz, W))
    m, v, _, _ = forge.new_states(W, "adamw")
    w1 = W.clone()
    forge.wgrad_step(x2, dz, w1, m, v, "adamw", None, 1, layer.seed)
    assert torch.equal(w1, layer.weight) and torch.equal(m, layer.m)
    if bias:
        assert torch.allclose(layer.bias_m[0], 0.1 * db, rtol=1e-5, atol=0)
        assert not torch.equal(layer.bias.detach(), b0)


def test_linear_layer_gradient_against_differences():
    """float32: dX of a biased, activated layer against central differences of sum(Y dY)."""
    F = torch.float32
    W, b = rnd(1, 24, 16, dtype=F, std=0.3), rnd(2, 24, dtype=F)
    x, dy = rnd(3, 5, 16, dtype=F), rnd(4, 5, 24, dtype=F)
    for act in ("silu", "gelu", "gelu_tanh"):
        y, z = forge.linear(x, W, bias=b, act=act, save=True)
        dz, db = forge.linear_act_backward(dy, z, act=act)
        dx = forge.dgrad(dz, W)
        h = 2.0 ** -6
        for t, k in ((x, 0), (x, 37), (x, 79), (b, 3), (b, 23)):
            flat = t.view(-1)
            keep = float(flat[k])
            val = []
            for s in (h, -h):
                flat[k] = keep + s
                val.append(float((forge.linear(x, W, bias=b, act=act).double() * dy.double()).sum()))
            flat[k] = keep
            got = float((dx if t is x else db).view(-1)[k])
            # third derivatives of the activations are below 1.6, of z by x |W| <= 1.2; 24 terms
            # of |dY| <= 4; each y carries 2^-22 |y| (y <= 6) twice over 2 h
            tol = 24 * 4 * (1.6 * 1.2 ** 3 * h * h / 6 + 6 * 2.0 ** -22 / h)
            assert abs((val[0] - val[1]) / (2 * h) - got) <= tol, (act, k)


def test_two_phase_bias_layer_equals_fused():
    x, dy = rnd(2, 70, 64), rnd(3, 70, 128, std=1e-2)
    out = []
    for fused in (True, False):
        layer = ForgeLinear(64, 128, weight=rnd(1, 128, 64, std=0.1), bias=True, act="gelu", fused=fused, seed=3)
        for _ in range(2):
            layer(x).backward(dy)
            step_all(layer)
        out.append((layer.weight.detach(), layer.bias.detach(), layer.bias_m))
    assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][2], out[1][2])
    # the weights' fused and stand-alone steps take the same gradient sums
    assert float((out[0][0].float() - out[1][0].float()).abs().max()) <= 2.0 ** -8


def block(joined, ckpt=False, grouped=False, d=256, hidden=640, **kw):
    torch.manual_seed(0)
    return SwiGLUBlock(d, hidden, checkpoint=ckpt, seed=1, joined=joined, grouped=grouped, device="cuda", **kw)


def test_joined_block_equals_its_calls():
    """Output, input gradient and updates of the joined block against the same operator calls made
    by hand, bit for bit, and its output against float64."""
    T, d = 130, 256
    blk = block(True)
    wg, wu, wd = (L.weight.detach().clone() for L in (blk.gate, blk.up, blk.down))
    x, dy = rnd(7, T, d).requires_grad_(), rnd(8, T, d, std=1e-2)
    y = blk(x)
    y.backward(dy)
    xf = x.detach().float()
    h = (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + 1e-5)).to(BF)
    H, G, U = forge.gated(h, wg, wu, save=True)
    assert torch.equal(y.detach(), forge.linear(H, wd, residual=x.detach()))
    g64, e_g = mm64(h, wg.t())
    u64, e_u = mm64(h, wu.t())
    h64 = act64(g64, "silu")[0] * u64
    # H is rounded once before the down projection, whose sum it enters linearly
    e_h = 2.0 ** -8 * h64.abs() + 1.2 * e_g * u64.abs() + g64.abs() * e_u + 1e-6
    want = h64 @ wd.double().t() + x.detach().double()
    bound = e_h @ wd.double().abs().t() + 640 * 2.0 ** -24 * (h64.abs() @ wd.double().abs().t()) + 2.0 ** -24 * want.abs()
    close("block", y.detach(), want, bound)
    dG, dU, H2 = forge.gated_dgrad(dy, wd, G, U)
    dh = forge.dgrad_group([dG, dU], [wg, wu])
    hx = x.detach().clone().requires_grad_()
    hf = hx.float()
    ((hf * torch.rsqrt(hf.pow(2).mean(-1, keepdim=True) + 1e-5)).to(BF)).backward(dh)
    assert torch.allclose(x.grad.float(), hx.grad.float() + dy.float(), rtol=2.0 ** -6, atol=1e-5)
    m, v, _, _ = forge.new_states(wd, "adamw")
    forge.wgrad_step(H2, dy, wd, m, v, "adamw", None, 1, blk.down.seed)
    assert torch.equal(wd, blk.down.weight.detach()) and blk.gate.step_count == blk.up.step_count == 1
    sg, su = forge.new_states(wg, "adamw"), forge.new_states(wu, "adamw")
    forge.wgrad_step_group(h, [dG, dU], [wg, wu], [sg[0], su[0]], [sg[1], su[1]], "adamw", None, 1,
                           [blk.gate.seed, blk.up.seed])
    assert torch.equal(wg, blk.gate.weight.detach()) and torch.equal(wu, blk.up.weight.detach())


def test_joined_block_near_separate_layers():
    """One step of the joined block and of the separate layers from the same weights: outputs and
    input gradients differ by roundings of bfloat16 intermediates only."""
    x0, dy = rnd(7, 300, 256), rnd(8, 300, 256, std=1e-2)
    res = []
    for joined in (False, True):
        blk = block(joined)
        x = x0.clone().requires_grad_()
        y = blk(x)
        y.backward(dy)
        res.append((y.detach().double(), x.grad.double()))
    for a, b in zip(*res):
        # a handful of half steps (2^-8 each) of independent elements, in the norm
        assert float((a - b).norm() / a.norm()) <= 4 * 2.0 ** -8


@pytest.mark.parametrize("states", ["f32", "q8"])
def test_joined_block_checkpointed_equals_plain(states):
    x0, dy = rnd(7, 192, 256), rnd(8, 192, 256, std=1e-2)
    res = []
    for ckpt in (False, True):
        blk = block(True, ckpt=ckpt, states=states)
        for _ in range(3):
            x = x0.clone().requires_grad_()
            y = blk(x)
            y.backward(dy)
        res.append([y.detach(), x.grad] + [L.weight.detach() for L in (blk.gate, blk.up, blk.down)])
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_linear_cross_entropy_autograd(reduction):
    """Gradients through autograd equal the direct calls; leading dimensions are kept."""
    W = rnd(1, 515, 64, std=0.2).requires_grad_()
    x = rnd(2, 4, 9, 64).requires_grad_()
    y = torch.randint(0, 515, (4, 9), device="cuda")
    y[0, 2:5] = -100
    loss = linear_cross_entropy(x, W, y, reduction=reduction)
    assert loss.shape == ((4, 9) if reduction == "none" else ())
    up = torch.full_like(loss, 0.5)
    loss.backward(up)
    l2, lse, total = forge.linear_cross_entropy(x.detach().reshape(-1, 64), W.detach(), y.reshape(-1), reduction=reduction)
    assert torch.equal(l2.reshape(loss.shape), loss.detach())
    dx, dw = forge.linear_cross_entropy_backward(x.detach().reshape(-1, 64), W.detach(), y.reshape(-1), lse,
                                                 up.reshape(-1), reduction=reduction, total=total)
    assert torch.equal(x.grad.reshape(-1, 64), dx) and torch.equal(W.grad, dw)


def test_head_steps_and_leaves_no_gradient():
    head = ForgeHead(128, 1003, seed=2, weight=rnd(1, 1003, 128, std=0.05), piece=256)
    w0 = head.weight.detach().clone()
    x, y = rnd(2, 77, 128).requires_grad_(), torch.randint(0, 1003, (77,), device="cuda")
    loss = head(x, y)
    assert torch.equal(head.weight.detach(), w0)
    loss.backward()
    assert head.step_count == 1 and head.weight.grad is None and not torch.equal(head.weight.detach(), w0)
    with torch.no_grad():
        ev = head(x, y)
    assert head.step_count == 1 and ev.shape == ()
    m, v, _, _ = forge.new_states(w0, "adamw")
    l2, lse, total = forge.linear_cross_entropy(x.detach(), w0, y)
    dx = forge.linear_cross_entropy_step(x.detach(), w0, m, v, y, lse, torch.ones((), device="cuda"), "adamw", None, 1,
                                         head.seed, total=total, piece=256)
    assert torch.equal(l2, loss.detach()) and torch.equal(dx, x.grad) and torch.equal(w0, head.weight.detach())


def test_block_and_head_train_together():
    """Two joined blocks, a biased layer and the head: every parameter is stepped once per backward
    pass, nothing keeps a gradient, and the same run gives the same bits."""
    def run():
        torch.manual_seed(3)
        blocks = [SwiGLUBlock(128, 384, seed=k, joined=True, device="cuda") for k in range(2)]
        mid = ForgeLinear(128, 128, weight=rnd(9, 128, 128, std=0.1), bias=True, act="gelu", seed=7)
        head = ForgeHead(128, 777, weight=rnd(10, 777, 128, std=0.05), seed=8)
        x, y = rnd(11, 2, 61, 128).requires_grad_(), torch.randint(0, 777, (2, 61), device="cuda",
                                                                   generator=torch.Generator(device="cuda").manual_seed(1))
        for _ in range(3):
            z = x
            for b in blocks:
                z = b(z)
            loss = head(mid(z, residual=z), y)
            x.grad = None
            loss.backward()
        params = [p for m_ in blocks + [mid, head] for p in m_.parameters()]
        assert all(p.grad is None for p in params) and mid.step_count == head.step_count == 3
        return [loss.detach(), x.grad] + [p.detach() for p in params]

    for a, b in zip(run(), run()):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def calls(x, wg, wu, wd, b, w, y, stream=None):
    """The operators one after another, as a block and a head use them."""
    one = torch.ones((), device="cuda")
    H, G, U = forge.gated(x, wg, wu, save=True, stream=stream)
    z, pre = forge.linear(H, wd, bias=b, act="gelu", residual=x, save=True, stream=stream)
    loss, lse, total = forge.linear_cross_entropy(z, w, y, stream=stream)
    dz, dw = forge.linear_cross_entropy_backward(z, w, y, lse, one, total=total, stream=stream)
    da, db = forge.linear_act_backward(dz, pre, act="gelu", stream=stream)
    dG, dU, H2 = forge.gated_dgrad(da, wd, G, U, stream=stream)
    dx = forge.dgrad_group([dG, dU], [wg, wu], stream=stream)
    return [H, z, loss, lse, total, dz, dw, da, db, dG, dU, H2, dx]


def operands(seed, t=150, d=256, hid=520, voc=2003):
    y = torch.randint(0, voc, (t,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    y[::7] = -100
    return (rnd(seed, t, d), rnd(seed + 1, hid, d, std=0.06), rnd(seed + 2, hid, d, std=0.06), rnd(seed + 3, d, hid, std=0.05),
            rnd(seed + 4, d), rnd(seed + 5, voc, d, std=0.1), y)


def test_other_streams_and_two_at_once():
    a, b = operands(20), operands(40, t=333)
    want_a, want_b = calls(*a), calls(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got_a, got_b = calls(*a, stream=s1), calls(*b, stream=s2)
        with torch.cuda.stream(s2):
            again = calls(*a)
        torch.cuda.synchronize()
        for w, g, h in zip(want_a, got_a, again):
            assert torch.equal(w, g) and torch.equal(w, h)
        for w, g in zip(want_b, got_b):
            assert torch.equal(w, g)


def test_captured_and_replayed():
    """All the operators and the head's fused step in one graph, replayed with eager work between
    the replays; a second graph holds workspaces of its own."""
    a, b = operands(60), operands(80, t=77)
    one = torch.ones((), device="cuda")
    W0 = a[5].clone()
    w_live = a[5].clone()
    m, v, _, _ = forge.new_states(w_live, "adamw")

    def step(ops, w, m_, v_):
        out = calls(*ops)
        forge.linear_cross_entropy_step(ops[0], w, m_, v_, ops[6], out[3], one, "adamw", {"stochastic_round": 0}, 1, 5,
                                        total=out[4])
        return out

    want_a, want_b = calls(*a), calls(*b)
    eager_w = W0.clone()
    em, ev, _, _ = forge.new_states(eager_w, "adamw")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(a, w_live, m, v)
        calls(*b)
    torch.cuda.synchronize()
    w_live.copy_(W0), m.zero_(), v.zero_()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        out_a = step(a, w_live, m, v)
    with torch.cuda.graph(gb):
        out_b = calls(*b)
    torch.cuda.synchronize()
    for _ in range(4):
        for t in out_a + out_b:
            t.zero_()
        ga.replay()
        gb.replay()
        step(a, eager_w, em, ev)
        torch.cuda.synchronize()
        for w, g in zip(want_a + want_b, out_a + out_b):
            assert torch.equal(w, g)
        assert torch.equal(eager_w, w_live) and torch.equal(em, m) and torch.equal(ev, v)


def test_same_operand_twice():
    """The same tensor as several inputs of one call."""
    x, w = rnd(1, 90, 72), rnd(2, 264, 72, std=0.1)
    H, G, U = forge.gated(x, w, w, save=True)
    assert torch.equal(G, U)
    dy = rnd(3, 90, 264, std=0.1)
    two = forge.dgrad_group([dy, dy], [w, w])
    d, e = mm64(dy, w)
    close("twice", two, 2 * d, 4 * e)
    sq = rnd(4, 64, 64)
    close("square", forge.linear(sq, sq, residual=sq), *linear64(sq, sq, residual=sq)[:2])


def test_loss_of_other_weights_is_refused():
    """Backward needs the weights that the loss was computed with."""
    head = ForgeHead(64, 500, device="cuda")
    x = torch.randn(2, 20, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    y = torch.randint(0, 500, (2, 20), device="cuda")
    first, second = head(x, y), head(x, y)
    first.backward()
    w = head.weight.detach().clone()
    with pytest.raises(RuntimeError, match="stepped after"):
        second.backward()
    assert head.step_count == 1 and torch.equal(head.weight, w)
    head(x, y).backward()
    assert head.step_count == 2
    weight = torch.randn(500, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    loss = linear_cross_entropy(x, weight, y)
    with torch.no_grad():
        weight.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def pool_stream(t):
    """The stream in whose pool a tensor's memory lies."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_memory_of_a_call_on_another_stream():
    """What a call on another stream allocates is that stream's memory, for every entry point: blocks
    freed on the current stream, with work on them still queued there, are not taken."""
    a = operands(20)
    x, wg, wu, wd, b, w, y = a
    s = torch.cuda.Stream()
    one = torch.ones((), device="cuda")
    w1 = wg.clone()
    m, v, _, _ = forge.new_states(w1, "adamw")
    torch.cuda.synchronize()
    out = [forge.linear(x, wg, act="silu", save=True, stream=s), forge.gated(x, wg, wu, save=True, stream=s)]
    H, G, U = out[-1]
    out.append(forge.linear_act_backward(G, U, act="gelu", stream=s))
    out.append(forge.gated_backward(H, G, U, stream=s))
    out.append(forge.gated_dgrad(x, wd, G, U, stream=s))
    out.append([forge.dgrad_group([G, U], [wg, wu], stream=s)])
    loss, lse, total = forge.linear_cross_entropy(x, w, y, reduction="none", stream=s)
    out.append((loss, lse, total))
    out.append(forge.linear_cross_entropy_backward(x, w, y, lse, one, reduction="mean", total=total, stream=s))
    out.append([forge.dgrad(G, wg, stream=s), forge.wgrad(x, G, stream=s)])
    out.append([forge.wgrad_unfused(x, G, w1, m, v, stream=s)])
    for group in out:
        for t in group:
            assert pool_stream(t) == s.cuda_stream
    torch.cuda.synchronize()


def test_calls_on_another_stream_beside_queued_work():
    """Operators on a second stream while the current one writes, reads and frees memory of the same
    sizes, the operands waited for: the results are the same bits."""
    x, wg, wu, wd, b, w, y = operands(20)
    one = torch.ones((), device="cuda")
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()

    def run(stream):
        H, G, U = forge.gated(x, wg, wu, save=True, stream=stream)
        z, pre = forge.linear(H, wd, bias=b, act="gelu", residual=x, save=True, stream=stream)
        loss, lse, total = forge.linear_cross_entropy(z, w, y, stream=stream)
        dz, dw = forge.linear_cross_entropy_backward(z, w, y, lse, one, total=total, stream=stream)
        da, db = forge.linear_act_backward(dz, pre, act="gelu", stream=stream)
        dG, dU, H2 = forge.gated_dgrad(da, wd, G, U, stream=stream)
        return [H, z, loss, lse, dz, dw, da, db, dG, dU, H2, forge.dgrad_group([dG, dU], [wg, wu], stream=stream),
                forge.dgrad(dG, wg, stream=stream), forge.wgrad(x, dG, stream=stream)]

    want = run(None)
    for _ in range(6):
        s.wait_stream(cur)
        busy = [torch.full_like(t, 3.0) for t in want for _ in range(2)]
        sums = [(t.numel(), t.float().sum()) for t in busy]
        del busy
        got = run(s)
        cur.wait_stream(s)
        for w_, g_ in zip(want, got):
            assert torch.equal(w_, g_)
        for n, v in sums:
            assert float(v) == 3.0 * n  # whole numbers below 2^24: exact in any order
        del got


def joined_by_hand(blk, x, dy, counts):
    """The joined block's weights after one backward pass, its operators called one by one with the
    layers' own step counts."""
    gate, up, down = blk.gate, blk.up, blk.down
    wg, wu, wd = (L.weight.detach().clone() for L in (gate, up, down))
    xf = x.detach().float()
    h = (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + 1e-5)).to(x.dtype)
    H, G, U = forge.gated(h, wg, wu, save=True)
    dG, dU, H2 = forge.gated_dgrad(dy, wd, G, U)
    for L, w, a, d, n in ((gate, wg, h, dG, counts[0]), (up, wu, h, dU, counts[1]), (down, wd, H2, dy, counts[2])):
        m, v = (None if t is None else t.clone() for t in (L.m, L.v))
        forge.wgrad_step(a, d, w, m, v, L.opt, L.hyper, n, L.seed)
    return [wg, wu, wd]


def test_joined_block_steps_float32_layers():
    """float32, which the grouped step does not take: every layer is stepped, by its own call."""
    F = torch.float32
    blk = block(True, dtype=F)
    x, dy = rnd(7, 130, 256, dtype=F).requires_grad_(), rnd(8, 130, 256, std=1e-2, dtype=F)
    for n in (1, 2):
        want = joined_by_hand(blk, x, dy, (n, n, n))
        blk(x).backward(dy)
        for L, w in zip((blk.gate, blk.up, blk.down), want):
            assert L.step_count == n and torch.equal(L.weight.detach(), w)


def test_joined_block_of_layers_that_disagree():
    """gate has taken a step alone: gate and up step with their own counts (the grouped step would
    give up gate's)."""
    blk = block(True)
    x, dy = rnd(7, 130, 256), rnd(8, 130, 256, std=1e-2)
    blk.gate(x).backward(rnd(9, 130, 640, std=1e-2))
    want = joined_by_hand(blk, x, dy, (2, 1, 1))
    blk(x.requires_grad_()).backward(dy)
    assert (blk.gate.step_count, blk.up.step_count, blk.down.step_count) == (2, 1, 1)
    for L, w in zip((blk.gate, blk.up, blk.down), want):
        assert torch.equal(L.weight.detach(), w)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_joined_block_in_two_phases(dtype):
    """fused=False: backward keeps the float32 gradients of all three layers (a second pass adds to
    them), step_all applies them."""
    blk = block(True, dtype=dtype, fused=False)
    x, dy = rnd(7, 130, 256, dtype=dtype).requires_grad_(), rnd(8, 130, 256, std=1e-2, dtype=dtype)
    layers = (blk.gate, blk.up, blk.down)
    old = [L.weight.detach().clone() for L in layers]
    blk(x).backward(dy)
    xf = x.detach().float()
    h = (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + 1e-5)).to(dtype)
    H, G, U = forge.gated(h, old[0], old[1], save=True)
    dG, dU, H2 = forge.gated_dgrad(dy, old[2], G, U)
    want = [forge.wgrad(h, dG), forge.wgrad(h, dU), forge.wgrad(H2, dy)]
    for L, w, g in zip(layers, old, want):
        assert L.step_count == 0 and torch.equal(L.weight.detach(), w) and torch.equal(L.grad32, g)
    blk(x).backward(dy)
    for L, g in zip(layers, want):
        assert torch.equal(L.grad32, g + g)
    step_all(blk)
    for L, w, g in zip(layers, old, want):
        m, v, _, _ = forge.new_states(w, "adamw")
        forge.optimizer_step(g + g, w, m, v, "adamw", None, 1, L.seed)
        assert L.step_count == 1 and L.grad32 is None and torch.equal(L.weight.detach(), w)


@pytest.mark.parametrize("ckpt", [False, True])
def test_output_of_other_weights_is_refused_by_the_joined_block(ckpt):
    """Two forward passes, two backward passes: the second one's projections belong to weights that
    the first has stepped."""
    blk = block(True, ckpt=ckpt)
    x, dy = rnd(7, 70, 256).requires_grad_(), rnd(8, 70, 256, std=1e-2)
    first, second = blk(x), blk(x)
    first.backward(dy)
    kept = [L.weight.detach().clone() for L in (blk.gate, blk.up, blk.down)]
    with pytest.raises(RuntimeError, match="stepped after"):
        second.backward(dy)
    for L, w in zip((blk.gate, blk.up, blk.down), kept):
        assert L.step_count == 1 and torch.equal(L.weight.detach(), w)
    blk(x).backward(dy)
    assert blk.gate.step_count == blk.up.step_count == blk.down.step_count == 2


@pytest.mark.parametrize("bias,act,residual", [(True, "none", False), (False, "gelu", False), (False, "none", True)])
def test_output_of_other_weights_is_refused_by_the_linear_layer(bias, act, residual):
    layer = ForgeLinear(64, 128, weight=rnd(1, 128, 64, std=0.1), bias=bias, act=act)
    x, dy = rnd(2, 70, 64).requires_grad_(), rnd(3, 70, 128, std=1e-2)
    r = rnd(4, 70, 128) if residual else None
    first, second = layer(x, r), layer(x, r)
    first.backward(dy)
    w = layer.weight.detach().clone()
    with pytest.raises(RuntimeError, match="stepped after"):
        second.backward(dy)
    assert layer.step_count == 1 and torch.equal(layer.weight.detach(), w)
    layer(x, r).backward(dy)
    assert layer.step_count == 2
    # another writer of the weights: autograd's own check
    third = layer(x, r)
    with torch.no_grad():
        layer.weight.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        third.backward(dy)


def test_two_phase_layers_take_several_backward_passes():
    """Two phases: the weights stay until step_all, so two micro-batches add their gradients; an
    output from before the step is refused after it."""
    layer = ForgeLinear(64, 128, weight=rnd(1, 128, 64, std=0.1), bias=True, act="gelu", fused=False)
    x, dy = rnd(2, 70, 64).requires_grad_(), rnd(3, 70, 128, std=1e-2)
    first, second, third = layer(x), layer(x), layer(x)
    first.backward(dy)
    one = layer.grad32.clone()
    second.backward(dy)
    assert torch.equal(layer.grad32, one + one)
    step_all(layer)
    with pytest.raises(RuntimeError, match="stepped after"):
        third.backward(dy)


def test_second_derivatives_are_refused():
    """A gradient penalty on the operators' gradients is refused, not left out of the sum."""
    x, y = rnd(2, 20, 64).requires_grad_(), torch.randint(0, 300, (20,), device="cuda")
    W = rnd(1, 300, 64, std=0.2).requires_grad_()
    layer = ForgeLinear(64, 128, weight=rnd(3, 128, 64, std=0.1), act="silu")
    blk = block(True, d=64, hidden=128)
    for out in (linear_cross_entropy(x, W, y), layer(x).float().sum(), blk(x).float().sum()):
        g, = torch.autograd.grad(out, x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiated once"):
            (x.float().sum() + g.float().pow(2).sum()).backward()
    # a first derivative with a graph around it stays possible
    x.grad = None
    linear_cross_entropy(x * 2, W, y).backward()
    assert torch.isfinite(x.grad.float()).all()


def test_evaluation_keeps_nothing_for_backward(monkeypatch):
    """Without gradients the modules write neither pre-activations nor projections; the output is
    the same bits."""
    from optimizer_gemm_amd import nn as fnn

    saves = []
    for name in ("linear", "gated"):
        real = getattr(forge, name)
        monkeypatch.setattr(fnn.forge, name,
                            lambda *a, _real=real, **kw: saves.append(bool(kw.get("save"))) or _real(*a, **kw))
    x, r = rnd(2, 70, 256), rnd(3, 70, 512)
    layer = ForgeLinear(256, 512, weight=rnd(1, 512, 256, std=0.1), bias=True, act="gelu")
    blk = block(True)
    for module, args, trained in ((layer, (x, r), [True]), (blk, (x,), [True, False])):
        saves.clear()
        want = module(*args)
        assert saves == trained and want.requires_grad
        for p in module.parameters():
            p.requires_grad_(False)
        saves.clear()
        frozen = module(*args)
        assert not any(saves) and torch.equal(frozen, want)
        for p in module.parameters():
            p.requires_grad_(True)
        saves.clear()
        with torch.no_grad():
            got = module(*args)
        assert not any(saves) and torch.equal(got, want)
        with torch.inference_mode():
            assert torch.equal(module(*args), want)
    assert layer.step_count == 0


def test_a_refused_head_step_counts_nothing():
    """float32 steps of a head whose piece is no multiple of 8 are refused: weights and count stay."""
    head = ForgeHead(64, 200, dtype=torch.float32, device="cuda", piece=12)
    x = rnd(1, 20, 64, dtype=torch.float32).requires_grad_()
    w = head.weight.detach().clone()
    with pytest.raises(forge.ForgeError):
        head(x, torch.randint(0, 200, (20,), device="cuda")).backward()
    assert head.step_count == 0 and torch.equal(head.weight.detach(), w)
