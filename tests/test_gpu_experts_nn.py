"""The layers of experts and the 8-bit layers as a program uses them: ForgeExperts through autograd, fused and in two
phases, its serving form, on other streams, from two threads, captured in HIP graphs."""
import threading

import pytest
import torch

import optimizer_gemm_amd as forge
from _experts64 import combine64, expert_gated64, linear_q8_64, plan64, routes, spans
from _ops64 import U, act64, close
from optimizer_gemm_amd.nn import ExpertsQ8, ForgeExperts, ForgeLinear, LinearQ8, step_all

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def routed(seed, t, k, e, dropped=0.1):
    w = torch.softmax(rnd(seed + 1, t, k, dtype=F), 1)
    return routes(seed, t, k, e, dropped).cuda(), w


def make(d=128, h=192, e=5, **kw):
    torch.manual_seed(0)
    blk = ForgeExperts(d, h, e, seed=1, device="cuda", **kw)
    with torch.no_grad():
        for s in (blk.gate, blk.up, blk.down):
            s.weight.copy_(torch.randn(s.weight.shape, device="cuda") * s.weight.shape[2] ** -0.5)
    return blk


def stacks(blk):
    return [s.weight.detach().clone() for s in (blk.gate, blk.up, blk.down)]


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("t", [1, 130, 1500])
def test_block_equals_its_calls(t, dt):
    """Output, gradients and updates against the same operator calls made by hand, bit for bit."""
    blk = make(dtype=dt, act="gelu")
    wg, wu, wd = stacks(blk)
    idx, w = routed(t, t, 2, 5)
    x, r, dy = rnd(7, t, 128, dtype=dt).requires_grad_(), rnd(9, t, 128, dtype=dt).requires_grad_(), rnd(8, t, 128, std=1e-2, dtype=dt)
    w.requires_grad_()
    y = blk(x, idx, w, residual=r)
    y.backward(dy)
    offsets, pos = forge.expert_plan(idx, 5)
    n = int(offsets[-1])
    Xp = forge.expert_dispatch(x.detach(), pos)
    H, G, V = forge.expert_gated(Xp, wg, wu, offsets, act="gelu", save=True)
    Yp = forge.expert_linear(H, wd, offsets, out_dtype=F)
    assert torch.equal(y.detach(), forge.expert_combine(Yp, pos, w.detach(), residual=r.detach()))
    dYp, dw = forge.expert_combine_backward(dy, Yp, pos, w.detach())
    dG, dU, H2 = forge.expert_gated_dgrad(dYp, wd, G, V, offsets, act="gelu")
    dX = forge.expert_combine(forge.expert_dgrad_group([dG, dU], [wg, wu], offsets), pos)
    assert torch.equal(x.grad, dX) and torch.equal(w.grad, dw) and torch.equal(r.grad, dy)
    for s, W, a, b in ((blk.down, wd, H2, dYp), (blk.gate, wg, Xp, dG), (blk.up, wu, Xp, dU)):
        m, v, _, _ = forge.new_states(W, "adamw")
        forge.expert_wgrad_step(a, b, W, m, v, offsets, "adamw", None, 1, s.seed)
        assert torch.equal(W, s.weight.detach()) and torch.equal(m, s.m) and torch.equal(v, s.v)
        assert s.weight.grad is None and s.step_count == 1


def test_block_against_float64():
    """float32: output and gradients of x and the weights against autograd of the definition in float64. The chained sums
    are of at most 192 terms, three of them; the terms' magnitudes exceed the results' by a factor of 8 at most in
    the 2-norm: 3 * 192 * 8 * 2^-24 = 2.7e-4."""
    t, k, e = 60, 3, 5
    blk = make(dtype=F, act="silu")
    wg, wu, wd = [W.double() for W in stacks(blk)]
    idx, w = routed(3, t, k, e, 0.2)
    x, dy = rnd(7, t, 128, dtype=F).requires_grad_(), rnd(8, t, 128, dtype=F)
    w.requires_grad_()
    y = blk(x, idx, w)
    y.backward(dy)
    x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    out = torch.zeros(t, 128, device="cuda", dtype=torch.float64)
    for a in range(e):
        for j in range(k):
            rows = torch.nonzero(idx[:, j] == a)[:, 0]
            h = torch.nn.functional.silu(x64[rows] @ wg[a].t()) * (x64[rows] @ wu[a].t())
            out = out.index_add(0, rows, (h @ wd[a].t()) * w64[rows, j, None])
    (out * dy.double()).sum().backward()
    for name, got, want in (("y", y.detach(), out.detach()), ("dx", x.grad, x64.grad), ("dw", w.grad, w64.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.7e-4, name


@pytest.mark.parametrize("states", ["f32", "bf16", "q8"])
def test_two_phases_equal_fused(states):
    out = []
    idx, w = routed(5, 70, 2, 5)
    x, dy = rnd(2, 70, 128), rnd(3, 70, 128, std=1e-2)
    for fused in (True, False):
        blk = make(fused=fused, states=states, hyper={"lr": 1e-3})
        for n in range(2):
            blk(x, idx, w).backward(dy)
            assert blk.gate.step_count == (n + 1 if fused else n)
            step_all(blk)
        assert [s.step_count for s in (blk.gate, blk.up, blk.down)] == [2, 2, 2]
        out.append(stacks(blk))
    for a, b in zip(*out):
        # the same sums in float32, in another order: the update may round to the neighbouring bfloat16 (weights below
        # 0.4: 2^-9 a step), or, where the first moment is near zero, turn: twice the step of 1e-3, two times
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -9 + 4e-3
        assert float((a != b).float().mean()) < 0.02


def test_two_phases_accumulate():
    """two backward passes, then one step on the sum of their gradients"""
    idx, w = routed(5, 70, 2, 5)
    blk = make(fused=False, dtype=F)
    x, dy = rnd(2, 70, 128, dtype=F), rnd(3, 70, 128, std=1e-2, dtype=F)
    blk(x, idx, w).backward(dy)
    one = blk.down.grad32.clone()
    blk(x, idx, w).backward(dy)
    assert torch.equal(blk.down.grad32, 2 * one)
    step_all(blk)
    assert blk.down.grad32 is None and blk.down.step_count == 1


def test_stepped_weights_second_derivatives_and_shapes_are_refused():
    blk = make()
    idx, w = routed(5, 6, 2, 5)
    x = rnd(2, 6, 128).requires_grad_()
    a, b = blk(x, idx, w), blk(x, idx, w)
    a.sum().backward()
    with pytest.raises(RuntimeError, match="stepped after"):
        b.sum().backward()
    blk = make(fused=False)
    g, = torch.autograd.grad(blk(x, idx, w).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated once"):
        g.float().sum().backward()
    for args in ((x, idx, w[:, :1]), (x, idx[:5], w[:5]), (x, idx, w, rnd(1, 5, 128)), (rnd(1, 6, 64), idx, w)):
        with pytest.raises(ValueError):
            blk(*args)
    with pytest.raises(ValueError):
        ForgeExperts(16, 16, 0)
    with pytest.raises(ValueError):
        ForgeExperts(16, 16, 4, act="tanh")
    # leading dimensions of the tokens
    y = blk(x.reshape(2, 3, 128), idx.reshape(2, 3, 2), w.reshape(2, 3, 2))
    assert torch.equal(y.reshape(6, 128), blk(x, idx, w))


def test_without_gradients_nothing_is_kept():
    blk = make()
    idx, w = routed(5, 300, 2, 5)
    x = rnd(2, 300, 128)
    with torch.no_grad():
        blk(x, idx, w)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = blk(x, idx, w)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() - before <= y.numel() * 2 + 512
    # a router without a gradient: the experts' results are not kept
    y = blk(x, idx, w)
    saved = [t for t in y.grad_fn.saved_tensors if t is not None]
    assert not any(t.dtype == F and t.shape == (600, 128) for t in saved)
    y.float().sum().backward()


def test_no_tokens_and_no_routes():
    blk = make(opt="sgd", hyper={"lr": 0.5, "weight_decay": 0.5, "stochastic_round": 0})
    W = stacks(blk)
    y = blk(torch.empty(0, 128, device="cuda", dtype=BF), torch.empty(0, 2, device="cuda", dtype=torch.int64),
            torch.empty(0, 2, device="cuda"))
    assert y.shape == (0, 128)
    y.sum().backward()  # a step on zero gradients
    want = [(w.float() - 0.5 * (0.5 * w.float())).to(BF) for w in W]
    for a, b in zip(stacks(blk), want):
        assert torch.equal(a, b)
    x = rnd(1, 4, 128).requires_grad_()
    y = blk(x, torch.full((4, 2), -1, device="cuda"), torch.ones(4, 2, device="cuda"), residual=x.detach())
    assert torch.equal(y.detach(), x.detach())
    y.float().sum().backward()
    assert torch.all(x.grad == 0)


# ---- serving ---------------------------------------------------------------------------------------------------
def test_linear_layer_in_8_bits():
    layer = ForgeLinear(128, 264, weight=rnd(1, 264, 128, std=0.1), bias=True, act="silu")
    with torch.no_grad():
        layer.bias.copy_(rnd(2, 264))
    served = LinearQ8(layer)
    for shape in ((1, 128), (2, 17, 128)):
        x, r = rnd(3, *shape), rnd(4, *shape[:-1], 264)
        y = served(x, r)
        Q, s = forge.quantize_rows(x.reshape(-1, 128))
        close("y", y.reshape(-1, 264), *linear_q8_64(Q, s, served.codes, served.scale, layer.bias.detach(), "silu", r.reshape(-1, 264)))
    assert not served(rnd(3, 4, 128).requires_grad_()).requires_grad


def test_experts_in_8_bits_equal_their_calls():
    blk = make()
    served = ExpertsQ8(blk)
    for t in (1, 40, 700):
        idx, w = routed(t, t, 2, 5)
        x, r = rnd(3, t, 128), rnd(4, t, 128)
        y = served(x, idx, w, residual=r)
        offsets, pos = forge.expert_plan(idx, 5)
        n = int(offsets[-1])
        Q, s = forge.quantize_rows(x)
        Qp, sp = forge.expert_dispatch(Q, pos, scale=s)
        H = forge.expert_gated_q8(Qp, sp, served.gate, served.gate_scale, served.up, served.up_scale, offsets)
        Hq, hs = forge.quantize_rows(H)
        Yp = forge.expert_linear_q8(Hq, hs, served.down, served.down_scale, offsets, out_dtype=F)
        assert torch.equal(y, forge.expert_combine(Yp, pos, w, residual=r))
        # near the block it came from: two quantisations of tokens and of weights, each element off by 1/254 of its row's
        # largest at most, a third of that on average, independently
        want = blk(x, idx, w, residual=r).detach().double()
        assert float((y.double() - want).norm() / want.norm()) < 0.02


# ---- streams, threads, graphs ---------------------------------------------------------------------------------------
def chain(x, idx, w, W, stream=None):
    """plan to combination and back on one stream; everything that comes out of it"""
    kw = {} if stream is None else {"stream": stream}
    wg, wu, wd = W
    offsets, pos = forge.expert_plan(idx, wg.shape[0], **kw)
    Xp = forge.expert_dispatch(x, pos, **kw)
    H, G, V = forge.expert_gated(Xp, wg, wu, offsets, save=True, **kw)
    Yp = forge.expert_linear(H, wd, offsets, out_dtype=F, **kw)
    Y = forge.expert_combine(Yp, pos, w, out_dtype=BF, **kw)
    dYp, dw = forge.expert_combine_backward(Y, Yp, pos, w, **kw)
    dG, dU, _ = forge.expert_gated_dgrad(dYp, wd, G, V, offsets, **kw)
    dX = forge.expert_combine(forge.expert_dgrad_group([dG, dU], [wg, wu], offsets, **kw), pos, **kw)
    dW = forge.expert_wgrad(Xp, dG, offsets, **kw)
    Q, s = forge.quantize_rows(x, **kw)
    Qp, sp = forge.expert_dispatch(Q, pos, scale=s, **kw)
    return [offsets, pos, Y, dw, dX, dW, Q, s]


def data(seed, t=200, k=2, e=6, d=128, h=192):
    idx, w = routed(seed, t, k, e)
    W = [rnd(seed + 5, e, h, d, std=d ** -0.5), rnd(seed + 6, e, h, d, std=d ** -0.5), rnd(seed + 7, e, d, h, std=h ** -0.5)]
    return rnd(seed + 4, t, d), idx, w, W


def test_other_streams_and_two_at_once():
    a, b = data(1), data(50, t=333, k=3)
    want = [chain(*a), chain(*b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = [chain(*a, stream=s1), chain(*b, stream=s2)]
        with torch.cuda.stream(s2):
            more = chain(*a)
        torch.cuda.synchronize()
        for g, w in zip(got + [more], want + [want[0]]):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_two_threads():
    a, b = data(1), data(50, t=333, k=3)
    want = [chain(*a), chain(*b)]
    torch.cuda.synchronize()
    bad = []

    def work(args, ref):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = chain(*args)
                s.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, ref)):
                    bad.append(1)

    ts = [threading.Thread(target=work, args=p) for p in ((a, want[0]), (b, want[1]))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_captured_and_replayed_with_other_routes():
    """Two graphs captured once, replayed with new tokens, routes and weights of the routing: the sizes live on the
    device, so a replay follows them; checked after each replay against eager calls between."""
    a, b = data(1), data(50, t=2500, k=3, e=70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*a)
        chain(*b)
    torch.cuda.current_stream().wait_stream(side)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        oa = chain(*a)
    with torch.cuda.graph(gb):
        ob = chain(*b)
    for n in range(4):
        for (x, idx, w, W), e in ((a, 6), (b, 70)):
            x.copy_(rnd(100 + n, *x.shape))
            t, k = idx.shape
            i2, w2 = routed(200 + n, t, k, e, dropped=(0.0, 0.5, 1.0, 0.1)[n])
            idx.copy_(i2)
            w.copy_(w2)
        ga.replay()
        gb.replay()
        if n % 2:
            ga.replay()
        torch.cuda.synchronize()
        for got, args in ((oa, a), (ob, b)):
            want = chain(*args)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), n


def test_shared_input_gradient_captured_and_on_streams():
    """the input gradient whose tiles are shared along k, with its workspace: two streams at once, and two graphs replayed with
    other offsets"""
    W = [rnd(60 + j, 4, 5000, 136, std=5000 ** -0.5) for j in range(2)]
    sets = []
    for j, t in ((0, 300), (1, 77)):
        assert forge.lib().forge_expert_dgrad_group_workspace(t, 136, 10000, 4, forge.forge.BF16) > 0
        sets.append(([rnd(70 + j, t, 5000), rnd(80 + j, t, 5000)], torch.tensor([0, t // 3, t // 3, t // 2, t - 2], device="cuda")))
    want = [forge.expert_dgrad_group(D, W, off)[:off[-1]] for D, off in sets]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = [forge.expert_dgrad_group(D, W, off, stream=s) for (D, off), s in zip(sets, (s1, s2))]
        junk = [torch.full((4000, 136), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(a[:len(b)], b) for a, b in zip(got, want))
        del junk
    graphs, outs = [], []
    for D, off in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forge.expert_dgrad_group(D, W, off))
        graphs.append(g)
    for n in range(4):
        for D, off in sets:
            D[0].copy_(rnd(90 + n, *D[0].shape))
            t = D[0].shape[0]
            off.copy_(torch.tensor([0, n, t // 2 + n, t - 4, t - n], device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (D, off), out in zip(sets, outs):
            m = int(off[-1])
            assert torch.equal(out[:m], forge.expert_dgrad_group(D, W, off)[:m])


def test_block_step_captured():
    """Forward, backward and the fused steps of a block in one graph: a replay does what the eager calls do"""
    idx, w = routed(5, 300, 2, 5)
    x, dy = rnd(2, 300, 128), rnd(3, 300, 128, std=1e-2)
    eager, graphed = make(), make()
    offsets, pos = forge.expert_plan(idx, 5)

    def steps(blk):
        wg, wu, wd = (s.weight.detach() for s in (blk.gate, blk.up, blk.down))
        Xp = forge.expert_dispatch(x, pos)
        H, G, V = forge.expert_gated(Xp, wg, wu, offsets, save=True)
        dYp, _ = forge.expert_combine_backward(dy, None, pos, w, want_dweights=False)
        dG, dU, H = forge.expert_gated_dgrad(dYp, wd, G, V, offsets)
        for s, a, b in ((blk.down, H, dYp), (blk.gate, Xp, dG), (blk.up, Xp, dU)):
            forge.expert_wgrad_step(a, b, s.weight.detach(), s.m, s.v, offsets, "adamw", None, 3, s.seed)

    keep = [[t.clone() for t in (s.weight.detach(), s.m, s.v)] for s in (graphed.gate, graphed.up, graphed.down)]
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(graphed)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        steps(graphed)
    with torch.no_grad():
        for s, k in zip((graphed.gate, graphed.up, graphed.down), keep):
            for t, v in zip((s.weight, s.m, s.v), k):
                t.copy_(v)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        steps(eager)
        for s, r in ((graphed.gate, eager.gate), (graphed.up, eager.up), (graphed.down, eager.down)):
            assert torch.equal(s.weight, r.weight) and torch.equal(s.m, r.m) and torch.equal(s.v, r.v)


def test_memory_of_a_call_on_another_stream():
    """what a call on another stream allocated is not handed out while it is written there"""
    x, idx, w, W = data(1, t=2000)
    s = torch.cuda.Stream()
    want = chain(x, idx, w, W)
    torch.cuda.synchronize()
    for _ in range(5):
        got = chain(x, idx, w, W, stream=s)
        junk = [torch.full((500, 192), float("nan"), device="cuda", dtype=BF) for _ in range(20)]
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        del junk


def test_one_block_trains():
    """a run of the operators together: some steps lower the loss of a fixed batch's fit (finite, changing weights)"""
    blk = make(hyper={"lr": 1e-2})
    x, target = rnd(2, 256, 128), rnd(3, 256, 128)
    router = rnd(4, 5, 128, std=0.1, dtype=F).requires_grad_()
    W = stacks(blk)
    for n in range(4):
        z = x.float() @ router.t()
        p, idx = torch.topk(z, 2, dim=1)
        y = blk(x, idx, torch.softmax(p, 1), residual=x)
        loss = (y.float() - target.float()).pow(2).mean()
        loss.backward()
        assert torch.isfinite(loss) and torch.isfinite(router.grad).all() and router.grad.abs().max() > 0
    assert blk.gate.step_count == 4
    for a, b in zip(stacks(blk), W):
        assert torch.isfinite(a).all() and not torch.equal(a, b)


# ---- what a call allocates -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("short", [True, False])
def test_new_tensors_are_those_of_torch(short, monkeypatch):
    """a call's new tensors honour what torch.empty does: the fill of deterministic mode and dispatch modes, by the shorter
    way and, where forge_calls is not there, by torch.empty itself"""
    from torch.utils._python_dispatch import TorchDispatchMode

    impl = forge.forge
    assert impl._new is not None
    if not short:
        monkeypatch.setattr(impl, "_new", None)
    x, W, off = rnd(1, 40, 128), rnd(2, 3, 264, 128), torch.tensor([0, 10, 10, 25], device="cuda")
    want = forge.expert_linear(x, W, off)[:25].clone()

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(str(func))
            return func(*args, **(kwargs or {}))

    with Seen() as seen:
        y, z = forge.linear(x, W[0], save=True)
        forge.expert_plan(torch.zeros(40, 2, device="cuda", dtype=torch.int64), 3)
    assert sum("empty" in n for n in seen.names) == 4
    assert y.shape == z.shape == (40, 264) and y.dtype == BF and y.is_contiguous() and y.device == x.device
    torch.use_deterministic_algorithms(True)
    try:
        for _ in range(3):
            junk = [torch.full((40, 264), 7.0, device="cuda", dtype=BF) for _ in range(8)]
            del junk  # (what torch.empty would hand out as it is)
            y = forge.expert_linear(x, W, off)
            assert torch.equal(y[:25], want) and torch.isnan(y[25:]).all()
    finally:
        torch.use_deterministic_algorithms(False)
    d = impl._here[0]
    assert d.empty((3,), torch.int64).shape == (3,) and d.empty((2, 0), F).shape == (2, 0)
    assert d.empty((2, 3, 5), F).stride() == (15, 5, 1)


# ---- other ways to run a block -----------------------------------------------------------------------------------------
def test_forward_passes_captured():
    """a block's forward pass and its 8-bit form in graphs, replayed with other tokens and routes"""
    blk = make()
    served = ExpertsQ8(blk)
    x, (idx, w) = rnd(1, 300, 128), routed(2, 300, 2, 5)

    def both():
        with torch.no_grad():
            return blk(x, idx, w, residual=x), served(x, idx, w, residual=x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for n in range(3):
        x.copy_(rnd(20 + n, 300, 128))
        i2, w2 = routed(30 + n, 300, 2, 5, dropped=(0.0, 1.0, 0.3)[n])
        idx.copy_(i2), w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, both())), n


def test_checkpointed_block_equals_the_block():
    """under activation checkpointing the forward pass runs again before the steps: the same bits"""
    from torch.utils.checkpoint import checkpoint

    out = []
    for again in (False, True):
        blk = make(act="gelu")
        x, r = rnd(1, 130, 128).requires_grad_(), rnd(2, 130, 128).requires_grad_()
        idx, w = routed(3, 130, 2, 5)
        w.requires_grad_()
        y = checkpoint(blk, x, idx, w, r, use_reentrant=False) if again else blk(x, idx, w, r)
        y.backward(rnd(4, 130, 128, std=1e-2))
        assert blk.gate.step_count == blk.down.step_count == 1
        out.append([y.detach(), x.grad, r.grad, w.grad, *stacks(blk), blk.up.m, blk.up.v])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_copied_and_restored_blocks():
    """a deep copy, and a block that takes another's weights and moments, go on as the block itself"""
    import copy

    idx, w = routed(3, 70, 2, 5)
    x, dy = rnd(1, 70, 128), rnd(4, 70, 128, std=1e-2)
    blk = make(states="q8")
    other = make(states="q8")
    blk(x, idx, w).backward(dy)
    two = copy.deepcopy(blk)
    assert two.gate.step_count == 1
    other.load_state_dict(blk.state_dict())
    for s, o in ((blk.gate, other.gate), (blk.up, other.up), (blk.down, other.down)):
        o._step_count = s.step_count
    for b in (blk, two, other):
        b(x, idx, w).backward(dy)
    for s, *rest in zip(*[(b.gate, b.up, b.down) for b in (blk, two, other)]):
        for o in rest:
            assert torch.equal(s.weight, o.weight) and torch.equal(s.m, o.m) and torch.equal(s.v_scale, o.v_scale)


def test_one_router_and_block_used_for_several_leading_dimensions():
    """tokens in two dimensions with routing weights in bfloat16 or float64, gradients in their shapes and types"""
    for dt in (BF, torch.float64):
        blk = make()
        x = rnd(1, 4, 9, 128).requires_grad_()
        idx, w = routed(3, 36, 2, 5)
        w = w.to(dt).reshape(4, 9, 2).requires_grad_()
        y = blk(x, idx.reshape(4, 9, 2), w, residual=x)
        y.backward(rnd(4, 4, 9, 128, std=1e-2))
        assert y.shape == x.shape and x.grad.shape == x.shape and w.grad.shape == w.shape and w.grad.dtype == dt
        flat = make()
        x2, w2 = x.detach().reshape(36, 128).requires_grad_(), w.detach().float().reshape(36, 2).requires_grad_()
        flat(x2, idx, w2, residual=x2).backward(rnd(4, 4, 9, 128, std=1e-2).reshape(36, 128))
        assert torch.equal(x.grad.reshape(36, 128), x2.grad) and torch.equal(w.grad.reshape(36, 2), w2.grad.to(dt))
