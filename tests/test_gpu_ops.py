"""GPU parity of the operators around the fused step against their float64 forms: the linear
layer's epilogue, the gated block, the grouped input gradient and the cross entropy of a
linear head, at ragged sizes, one token, no token, pitched rows, in bfloat16 and float32.
Tolerances are derived in tests/_ops64.py."""
import pytest
import torch

import optimizer_gemm_amd as forge
from _ops64 import (act64, close, gated64, gated_back64, linear64, mm64, xent64, xent_grad64)

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F) * std).to(dtype)


def pitched(t, extra=16):
    """The same values as a view with wider rows, whose padding holds NaN."""
    big = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device, dtype=t.dtype)
    view = big[:, : t.shape[1]]
    view.copy_(t)
    return view


# tokens, in, out: one token; odd tokens; sizes that are no multiple of any tile; tiles in
# every direction; more tiles than compute units
SIZES = [(1, 8, 8), (1, 512, 264), (3, 72, 40), (7, 4096, 128), (33, 136, 1032), (130, 264, 520), (257, 96, 328),
         (511, 1000, 776), (1000, 256, 2056), (2049, 520, 1288), (2049, 264, 4104), (16, 64, 70008)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,i,o", SIZES)
def test_linear(t, i, o, dt):
    g = gen(t * 7 + i + o)
    X, W = rnd(g, t, i, dtype=DT[dt]), rnd(g, o, i, dtype=DT[dt], std=i ** -0.5)
    b, R = rnd(g, o, dtype=DT[dt]), rnd(g, t, o, dtype=DT[dt])
    act = forge.ACTS[(t + o) % 5]
    Y, Z = forge.linear(X, W, bias=b, act=act, residual=R, save=True)
    y, dy, z, dz = linear64(X, W, b, act, R)
    close(f"Y {act}", Y, y, dy)
    close("Z", Z, z, dz)
    close("plain", forge.linear(X, W), *linear64(X, W)[:2])


@pytest.mark.parametrize("act", forge.ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_activations_and_parts(act, dt):
    g = gen(5)
    X, W = rnd(g, 150, 200, dtype=DT[dt], std=2.0), rnd(g, 344, 200, dtype=DT[dt], std=0.2)
    b, R = rnd(g, 344, dtype=F), rnd(g, 150, 344, dtype=DT[dt])
    for bias in (None, b):
        for res in (None, R):
            Y = forge.linear(X, W, bias=bias, act=act, residual=res)
            close(f"{act} {bias is not None} {res is not None}", Y, *linear64(X, W, bias, act, res)[:2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 5, 300])
def test_linear_pitched_rows(t, dt):
    g = gen(11)
    X, W, R = rnd(g, t, 264, dtype=DT[dt]), rnd(g, 392, 264, dtype=DT[dt], std=0.06), rnd(g, t, 392, dtype=DT[dt])
    out = torch.full((t, 400), 7.0, device="cuda", dtype=DT[dt])
    forge.linear(pitched(X), pitched(W, 8), residual=pitched(R), act="silu", out=out[:, :392])
    close("Y", out[:, :392], *linear64(X, W, None, "silu", R)[:2])
    assert torch.all(out[:, 392:] == 7.0)


def test_linear_extreme_values():
    """Saturated activations keep their limits; a NaN or an infinity stays in its own row."""
    X = torch.zeros(5, 8, device="cuda", dtype=BF)
    X[:, 0] = torch.tensor([60.0, -60.0, 3e38, -3e38, float("nan")], device="cuda")
    W = torch.zeros(8, 8, device="cuda", dtype=BF)
    W[:, 0] = 1.0
    for act in forge.ACTS:
        Y = forge.linear(X, W, act=act)
        assert torch.all(Y[0] == 60.0), act
        # silu's left tail is -60 e^-60 = -5.25e-25, no zero: half a bfloat16 step and the
        # exponential's argument (60 1.45 2^-24); the others' tails are below every float
        want = act64(torch.tensor(-60.0, dtype=torch.float64), act)[0].item()
        if abs(want) < 1e-45:
            assert torch.all(Y[1].float().abs() < 1e-37), act
        else:
            assert torch.all((Y[1].double() / want - 1).abs() <= 2.0 ** -8 + 100 * 2.0 ** -24), act
        assert torch.all(Y[2].float() > 1e38), act
        if act != "none":
            assert torch.all(Y[3].float() == 0.0), act
        assert torch.all(torch.isnan(Y[4])), act


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,o", [(1, 8), (2, 264), (17, 1000), (1025, 2056), (4099, 40)])
def test_linear_act_backward(t, o, dt):
    g = gen(t + o)
    dY, Z = rnd(g, t, o, dtype=DT[dt]), rnd(g, t, o, dtype=DT[dt], std=2.0)
    for act in forge.ACTS:
        dZ, db = forge.linear_act_backward(dY, Z, act=act)
        a, d = act64(Z.double(), act)
        want = dY.double() * d
        err = dY.double().abs() * (48 * 2.0 ** -24) * (1 + Z.double().abs()) + 2.0 ** -24 * want.abs()
        if act == "none":
            assert dZ is dY
        else:
            close(f"dZ {act}", dZ, want, err)
        close(f"db {act}", db, want.sum(0), err.sum(0) + t * 2.0 ** -24 * want.abs().sum(0))
    dZ, db = forge.linear_act_backward(pitched(dY), pitched(Z), act="silu", want_bias=False)
    assert db is None
    assert torch.equal(dZ, forge.linear_act_backward(dY, Z, act="silu")[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,i,o", SIZES)
def test_gated(t, i, o, dt):
    g = gen(t + i * 3 + o)
    X = rnd(g, t, i, dtype=DT[dt])
    Wg, Wu = rnd(g, o, i, dtype=DT[dt], std=i ** -0.5), rnd(g, o, i, dtype=DT[dt], std=i ** -0.5)
    act = forge.ACTS[(t + o) % 4 + 1]
    H, G, U = forge.gated(X, Wg, Wu, act=act, save=True)
    h, dh, gg, dg, uu, du = gated64(X, Wg, Wu, act)
    close(f"H {act}", H, h, dh)
    close("G", G, gg, dg)
    close("U", U, uu, du)
    assert torch.equal(forge.gated(X, Wg, Wu, act=act), H)
    assert torch.equal(forge.gated(pitched(X), pitched(Wg), pitched(Wu, 8), act=act), H)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,i,o", SIZES)
def test_gated_backward(t, i, o, dt):
    """dH = dY Wd formed in registers, the same from a given dH, then dX of both projections."""
    g = gen(t + i + o * 3)
    dY, Wd = rnd(g, t, i, dtype=DT[dt]), rnd(g, i, o, dtype=DT[dt], std=o ** -0.5)
    G, U = rnd(g, t, o, dtype=DT[dt], std=2.0), rnd(g, t, o, dtype=DT[dt])
    act = forge.ACTS[(t + o) % 4 + 1]
    dG, dU, H = forge.gated_dgrad(dY, Wd, G, U, act=act)
    dh, ddh = mm64(dY, Wd)
    dg, eg, du, eu, h, eh = gated_back64(dh, ddh, G, U, act)
    close(f"dG {act}", dG, dg, eg)
    close("dU", dU, du, eu)
    close("H", H, h, eh)
    dH = rnd(g, t, o, dtype=DT[dt])
    dG2, dU2, H2 = forge.gated_backward(dH, pitched(G), U, act=act)
    dg, eg, du, eu, h, eh = gated_back64(dH.double(), torch.zeros_like(dh), G, U, act)
    close("dG of dH", dG2, dg, eg)
    close("dU of dH", dU2, du, eu)
    close("H of dH", H2, h, eh)
    a, b, none = forge.gated_dgrad(pitched(dY), pitched(Wd), pitched(G), pitched(U), act=act, want_h=False)
    assert none is None and torch.equal(a, dG) and torch.equal(b, dU)
    Wg, Wu = rnd(g, o, i, dtype=DT[dt]), rnd(g, o, i, dtype=DT[dt])
    dX = forge.dgrad_group([dG, dU], [Wg, Wu])
    x1, e1 = mm64(dG, Wg)
    x2, e2 = mm64(dU, Wu)
    close("dX", dX, x1 + x2, 2 * (e1 + e2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,i", [(205, 456), (2049, 4104)])
@pytest.mark.parametrize("outs", [(8,), (264, 40), (1032, 264, 264), (72, 8, 200, 520)])
def test_dgrad_group(outs, t, i, dt):
    g = gen(sum(outs))
    dYs = [rnd(g, t, o, dtype=DT[dt]) for o in outs]
    Ws = [rnd(g, o, i, dtype=DT[dt]) for o in outs]
    want, bound = 0, 0
    for d, w in zip(dYs, Ws):
        x, e = mm64(d, w)
        want, bound = want + x, bound + len(outs) * e
    close("dX", forge.dgrad_group([pitched(d) for d in dYs], [pitched(w) for w in Ws]), want, bound)


def head(seed, t, i, v, dtype, ignored=0.2, ignore=-100):
    g = gen(seed)
    W = rnd(g, v, i, dtype=dtype, std=2.0 * i ** -0.5)
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    X = (torch.randn(t, i, generator=g, device="cuda") + 2.0 * W[y].float()).to(dtype)
    drop = torch.rand(t, generator=g, device="cuda") < ignored
    return X, W, torch.where(drop, torch.full_like(y, ignore), y)


# tokens, in, vocabulary (odd and tiny ones; a single entry: its loss is 0)
HEADS = [(1, 8, 1), (1, 64, 7), (2, 136, 1000), (65, 264, 513), (130, 72, 2051), (300, 520, 4099), (1025, 256, 5003), (260, 200, 20011),
         (4100, 2056, 4103)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,i,v", HEADS)
def test_cross_entropy(t, i, v, dt):
    X, W, y = head(t + v, t, i, v, DT[dt])
    loss, dl, lse, de, _, _, keep = xent64(X, W, y, -100)
    for red in ("none", "sum", "mean"):
        got, got_lse, total = forge.linear_cross_entropy(pitched(X), pitched(W), y, reduction=red)
        close("lse", got_lse, lse, de, F)
        n = int(keep.sum())
        assert float(total[1]) == n
        if red == "none":
            close("loss", got, loss, dl, F)
        elif red == "sum":
            close("sum", got, loss.sum(), dl.sum(), F)
        elif n:
            close("mean", got, loss.sum() / n, dl.sum() / n + 2.0 ** -23 * loss.sum() / n, F)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("red", ["mean", "sum", "none"])
@pytest.mark.parametrize("t,i,v", HEADS)
def test_cross_entropy_gradients(t, i, v, red, dt):
    X, W, y = head(t * 3 + v, t, i, v, DT[dt])
    y[0] = v - 1
    keep = y != -100
    n = int(keep.sum())
    g = gen(17)
    dloss = torch.rand(t if red == "none" else 1, generator=g, device="cuda") + 0.5
    f = dloss.double() / (n if red == "mean" else 1)
    f = (f if red == "none" else f.expand(t)) * keep
    dx, ex, dw, ew = xent_grad64(X, W, y, -100, f, DT[dt])
    _, lse, total = forge.linear_cross_entropy(X, W, y, reduction=red)
    for piece in (0, 8, 264):
        dX, dW = forge.linear_cross_entropy_backward(pitched(X), pitched(W), y, lse, dloss, reduction=red, total=total,
                                                     piece=piece)
        if piece == 8 and v > 600:
            continue
        close(f"dX {piece}", dX, dx, ex)
        close(f"dW {piece}", dW, dw, ew)
    only_x, none = forge.linear_cross_entropy_backward(X, W, y, lse, dloss, reduction=red, total=total, want_dw=False)
    none2, only_w = forge.linear_cross_entropy_backward(X, W, y, lse, dloss, reduction=red, total=total, want_dx=False)
    both = forge.linear_cross_entropy_backward(X, W, y, lse, dloss, reduction=red, total=total)
    assert none is None and none2 is None
    assert torch.equal(only_x, both[0]) and torch.equal(only_w, both[1])
    assert torch.all(both[0][~keep] == 0)


def test_cross_entropy_against_differences():
    """The float32 gradient against central differences of the float32 loss."""
    X, W, y = head(3, 6, 16, 37, F, ignored=0.0)
    y[2] = -100
    _, lse, total = forge.linear_cross_entropy(X, W, y)
    one = torch.ones((), device="cuda")
    dX, dW = forge.linear_cross_entropy_backward(X, W, y, lse, one, total=total)
    h = 2.0 ** -7
    for t, grad in ((X, dX), (W, dW)):
        for k in (0, 5, 33, t.numel() - 1):
            flat = t.view(-1)
            keep = float(flat[k])
            flat[k] = keep + h
            up = float(forge.linear_cross_entropy(X, W, y)[0])
            flat[k] = keep - h
            down = float(forge.linear_cross_entropy(X, W, y)[0])
            flat[k] = keep
            # third differences of a softmax loss are below max|W|^3 (or |X|^3) h^2 / 6; the
            # loss (about 5) is held to 2^-21 or so, twice, over 2 h
            other = W if t is X else X
            tol = float(other.abs().max()) ** 3 * h * h / 6 + 2 * 5 * 2.0 ** -21 / (2 * h)
            assert abs((up - down) / (2 * h) - float(grad.view(-1)[k])) <= tol


def test_cross_entropy_masks():
    X, W, y = head(9, 40, 64, 300, BF, ignored=0.0)
    # nothing counts: the mean of nothing is NaN, the sum 0, the gradients 0
    none = torch.full_like(y, -100)
    one = torch.ones((), device="cuda")
    loss, lse, total = forge.linear_cross_entropy(X, W, none)
    assert torch.isnan(loss) and float(total[0]) == 0 and float(total[1]) == 0
    dX, dW = forge.linear_cross_entropy_backward(X, W, none, lse, one, total=total)
    assert torch.all(dX == 0) and torch.all(dW == 0)
    # an ignored index inside the vocabulary
    l5, _, t5 = forge.linear_cross_entropy(X, W, y, ignore_index=int(y[3]), reduction="none")
    assert float(t5[1]) == int((y != y[3]).sum()) and torch.all(l5[y == y[3]] == 0)
    # targets outside the vocabulary: that token's loss and gradient are NaN, the others' are not
    for bad in (300, -1, 2 ** 62, -2 ** 63):
        z = y.clone()
        z[7] = bad
        lb, lse_b, tb = forge.linear_cross_entropy(X, W, z, reduction="none")
        ok = torch.arange(40, device="cuda") != 7
        assert torch.isnan(lb[7]) and torch.isfinite(lb[ok]).all()
        dXb, _ = forge.linear_cross_entropy_backward(X, W, z, lse_b, one, reduction="sum")
        assert torch.isnan(dXb[7]).all() and torch.isfinite(dXb[ok]).all()
    # a NaN or an infinity in an ignored token's hidden state reaches no other token
    Xn = X.clone()
    Xn[5], Xn[6] = float("nan"), float("inf")
    z = y.clone()
    z[5] = z[6] = -100
    ln, lse_n, tn = forge.linear_cross_entropy(Xn, W, z, reduction="none")
    assert torch.isfinite(ln).all() and torch.all(ln[5:7] == 0)
    dXn, _ = forge.linear_cross_entropy_backward(Xn, W, z, lse_n, one, reduction="sum", want_dw=False)
    assert torch.isfinite(dXn).all() and torch.all(dXn[5:7] == 0)


def test_cross_entropy_large_logits():
    """Logits of +-600: no exponential overflows, a certain token's loss is 0."""
    X = torch.zeros(3, 8, device="cuda", dtype=BF)
    W = torch.zeros(200, 8, device="cuda", dtype=BF)
    X[:, 0] = torch.tensor([600.0, -600.0, 0.0], device="cuda")
    W[17, 0] = 1.0
    y = torch.tensor([17, 17, 3], device="cuda")
    loss, lse, _ = forge.linear_cross_entropy(X, W, y, reduction="none")
    want = torch.logsumexp(X.double() @ W.double().t(), 1)
    assert torch.allclose(lse.double(), want, rtol=1e-6)
    assert torch.allclose(loss.double(), torch.tensor([0.0, 600.0 + float(want[1]), float(want[2])], device="cuda",
                                                      dtype=torch.float64), rtol=1e-6, atol=1e-4)


def test_empty_sizes():
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=BF)  # noqa: E731
    assert forge.linear(z(0, 64), z(32, 64)).shape == (0, 32)
    assert forge.gated(z(0, 64), z(32, 64), z(32, 64)).shape == (0, 32)
    b = torch.randn(32, device="cuda").to(BF)
    # no inner dimension: what is left is act(bias) + residual
    R = torch.randn(4, 32, device="cuda").to(BF)
    got = forge.linear(z(4, 0), z(32, 0), bias=b, act="silu", residual=R)
    close("no inner dimension", got, *linear64(z(4, 0), z(32, 0), b, "silu", R)[:2])
    dZ, db = forge.linear_act_backward(z(0, 32), z(0, 32), act="silu")
    assert dZ.shape == (0, 32) and torch.all(db == 0)
    assert torch.all(forge.dgrad_group([z(5, 0)], [z(0, 16)]) == 0)
    y = torch.zeros(0, device="cuda", dtype=torch.int64)
    loss, lse, total = forge.linear_cross_entropy(z(0, 64), z(100, 64), y)
    assert torch.isnan(loss) and lse.numel() == 0 and float(total[0]) == 0 and float(total[1]) == 0
    dX, dW = forge.linear_cross_entropy_backward(z(0, 64), z(100, 64), y, lse, torch.ones((), device="cuda"),
                                                 total=total)
    assert dX.shape == (0, 64) and torch.all(dW == 0)


STEP_OPTS = [("adamw", "f32"), ("sgd", "f32"), ("lion", "bf16"), ("adamw", "q8"), ("adamw", "q8dyn"),
             ("rmsprop", "f32")]


@pytest.mark.parametrize("opt,states", STEP_OPTS)
@pytest.mark.parametrize("v", [1000, 1003])
def test_cross_entropy_step(opt, states, v):
    """The head's fused step in pieces of the vocabulary equals the fused step of the whole W on
    the same dz (bit for bit: same element indices and random streams), and dX is of the old W."""
    t, i = 190, 128
    X, W, y = head(v, t, i, v, BF)
    dloss = torch.full((), 0.75, device="cuda")
    code = "dynamic" if states == "q8dyn" else "linear"
    _, lse, total = forge.linear_cross_entropy(X, W, y)
    old = W.clone()

    def run(piece):
        w = old.clone()
        m, vv, ms, vs = forge.new_states(w, opt, states)
        outs = []
        for step in (1, 2):
            outs.append(forge.linear_cross_entropy_step(X, w, m, vv, y, lse, dloss, opt, None, step, 99, ms, vs,
                                                        code=code, total=total, piece=piece))
        return outs + [t_ for t_ in (w, m, vv, ms, vs) if t_ is not None]

    whole = run(0)
    dx, ex, _, _ = xent_grad64(X, old, y, -100, dloss.double() / total[1].double() * (y != -100), BF)
    close("dX", whole[0], dx, ex)
    assert not torch.equal(whole[2], old)
    for piece in (256, 520):
        part = run(piece)
        for a, b in zip(whole[2:], part[2:]):
            # the tile shape, and with it the order of the token sum, follows the piece's size:
            # 190 tokens give one order of tokens in every configuration but the k-split ones
            assert a.shape == b.shape
        # dX of a piecewise sum differs by its float32 order only
        close(f"dX of pieces {piece}", part[0], dx, ex)
        # weights: within the step that a gradient error of the FP32 sum can make
        d = (whole[2].float() - part[2].float()).abs()
        assert float(d.max()) <= 2.0 ** -7 * float(old.abs().max()) * 2


def test_step_on_a_multiple_of_eight_equals_wgrad_step():
    """One piece: the head's step is wgrad_step on the dz that the plain gradient call forms."""
    t, i, v = 100, 64, 264
    X, W, y = head(5, t, i, v, F, ignored=0.0)
    _, lse, total = forge.linear_cross_entropy(X, W, y, reduction="sum")
    one = torch.ones((), device="cuda")
    w = W.clone()
    forge.linear_cross_entropy_step(X, w, None, None, y, lse, one, "sgd", {"lr": 1.0, "stochastic_round": 0}, 1, 0,
                                    reduction="sum")
    _, dW = forge.linear_cross_entropy_backward(X, W, y, lse, one, reduction="sum")
    # the fp32 GEMMs differ in their order of summation only
    _, _, _, ew = xent_grad64(X, W, y, -100, torch.ones(t, device="cuda", dtype=torch.float64), F)
    err = ((W - w).double() - dW.double()).abs()
    assert torch.all(err <= 2 * ew + 2.0 ** -23 * W.double().abs() + 2.0 ** -22 * dW.double().abs())


@pytest.mark.parametrize("t,i,outs", [(5, 64, (6568, 6568)), (15, 5120, (11672, 11672)), (140, 672, (4824, 40, 4824)),
                                      (700, 264, (13000,)), (1, 8, (16384, 8, 16384, 8))])
def test_dgrad_group_of_few_tiles(t, i, outs):
    """Few output tiles over a long sum: several workgroups share a tile's sum. The same bits
    every time, also when a graph replays it."""
    n = sum(outs)
    assert forge.lib().forge_linear_dgrad_group_workspace(t, i, n, forge.forge.BF16) > 0
    g = gen(t + n)
    dYs = [rnd(g, t, o) for o in outs]
    Ws = [rnd(g, o, i, std=n ** -0.5) for o in outs]
    want, bound = 0, 0
    for d, w in zip(dYs, Ws):
        x, e = mm64(d, w)
        want, bound = want + x, bound + 2 * len(outs) * e
    dX = forge.dgrad_group([pitched(d) for d in dYs], [pitched(w) for w in Ws])
    close("dX", dX, want, bound)
    out = torch.full((t, i + 8), 7.0, device="cuda", dtype=BF)
    forge.dgrad_group(dYs, Ws, dX=out[:, :i])
    assert torch.equal(out[:, :i], dX) and torch.all(out[:, i:] == 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = forge.dgrad_group(dYs, Ws)
    for _ in range(3):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, dX)


@pytest.mark.parametrize("t,o", [(7839, 144), (70001, 8), (513, 520), (16, 1536), (4099, 12)])
def test_linear_act_backward_shapes(t, o):
    """Narrow outputs over many rows, columns that end inside a vector's group of lanes; float32
    and bfloat16 (whose rows are multiples of 8)."""
    for dtype in (F, BF):
        if dtype == BF and o % 8:
            continue
        g = gen(t + o)
        dY, Z = rnd(g, t, o, dtype=dtype), rnd(g, t, o, dtype=dtype, std=2.0)
        dZ, db = forge.linear_act_backward(dY, Z, act="gelu")
        _, d = act64(Z.double(), "gelu")
        want = dY.double() * d
        err = dY.double().abs() * (48 * 2.0 ** -24) * (1 + Z.double().abs()) + 2.0 ** -24 * want.abs()
        close("dZ", dZ, want, err)
        close("db", db, want.sum(0), err.sum(0) + t * 2.0 ** -24 * want.abs().sum(0))


@pytest.mark.parametrize("stages", range(0, 11))
def test_products_of_every_ring_position(stages):
    """The 256x256 tiles keep two and a half stages of 64 k in a ring of five slots: every place in
    it where a tile's sum can end, several tiles per workgroup, epilogues with inputs."""
    t, o, i = 4360, 4360, 64 * stages
    g = gen(stages)
    X, W, R = rnd(g, t, i), rnd(g, o, i, std=max(1, i) ** -0.5), rnd(g, t, o)
    for _ in range(2):
        close("Y", forge.linear(X, W, act="silu", residual=R), *linear64(X, W, None, "silu", R)[:2])
    close("dX", forge.dgrad_group([X], [W.t().contiguous()]), *mm64(X, W.t().contiguous()))


@pytest.mark.parametrize("o", [40, 2056, 4104, 9000, 33000])
@pytest.mark.parametrize("t", [1, 4, 5, 16, 17, 32, 33])
def test_few_tokens(t, o):
    """Both sides of the choice between the kernel for a few tokens and the tiles."""
    g = gen(t * 7 + o)
    i = 136
    X, W, W2 = rnd(g, t, i), rnd(g, o, i, std=i ** -0.5), rnd(g, o, i, std=i ** -0.5)
    b, R = rnd(g, o), rnd(g, t, o)
    Y, Z = forge.linear(pitched(X), W, bias=b, act="gelu", residual=pitched(R), save=True)
    y, dy, z, dz = linear64(X, W, b, "gelu", R)
    close("Y", Y, y, dy)
    close("Z", Z, z, dz)
    H, G, U = forge.gated(X, W, pitched(W2), act="silu", save=True)
    h, dh, gg, dg, uu, du = gated64(X, W, W2, "silu")
    close("H", H, h, dh)
    close("G", G, gg, dg)
    close("U", U, uu, du)


@pytest.mark.parametrize("t,i,v", [(24, 8192, 140003), (70000, 8192, 264)])
def test_cross_entropy_past_32_bit_offsets(t, i, v):
    """Weights and their gradient of more than 2^31 bytes; float32 sums of dX of more."""
    X, W, y = head(t + v, t, i, v, BF)
    y[-1] = v - 1
    keep = y != -100
    n = int(keep.sum())
    loss, lse, total = forge.linear_cross_entropy(X, W, y)
    dX, dW = forge.linear_cross_entropy_backward(X, W, y, lse, torch.ones((), device="cuda"), total=total)
    want, dl, want_lse, de, _, _, _ = xent64(X, W, y, -100)
    close("lse", lse, want_lse, de, F)
    close("mean", loss, want.sum() / n, dl.sum() / n + 2.0 ** -23 * want.sum() / n, F)
    del want, dl, want_lse, de
    dx, ex, dw, ew = xent_grad64(X, W, y, -100, keep.double() / n, BF)
    close("dX", dX, dx, ex)
    close("dW", dW, dw, ew)
    del dx, ex, dw, ew
    torch.cuda.empty_cache()


def test_float32_gelu_in_its_left_tail():
    """Relative to the value itself, down to z = -12: z Phi(z) and its derivative Phi + z phi. u = 2^-24.
    Phi = erfc(x) / 2 with x = |z| / sqrt 2 held to 2 u (its constant, its product), which moves erfc by
    2 u (2 x^2 + 1) of itself at most; erfc and the exponential are the device library's, 16 and 3 ulps
    at most (32 u, 6 u); the exponential's argument z^2 / 2 is held to 1 u, which moves it by
    u z^2 / 2; up to 4 u of products and half a step of the result."""
    U = 2.0 ** -24
    n = 4096
    z = torch.linspace(-12.0, -0.25, n * 8, device="cuda", dtype=F).reshape(n, 8)
    one = torch.ones_like(z)
    zd = z.double()
    a, d = act64(zd, "gelu")
    phi = 0.5 * torch.special.erfc(-zd / 2 ** 0.5)
    pdf = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    rel = (2 * (zd * zd + 1) + 32 + 4 + 1) * U
    tol_d = rel * phi + (zd * zd / 2 + 6 + 4) * U * (zd * pdf).abs() + U * d.abs()
    ident = torch.eye(8, device="cuda", dtype=F)
    value = forge.linear(z, ident, act="gelu").double()
    wide = forge.linear(z, ident.repeat(16, 1), act="gelu")  # many columns: other tiles
    dG, dU, H = forge.gated_backward(one, z, one, act="gelu")
    dZ, _ = forge.linear_act_backward(one, z, act="gelu")
    for name, got in (("linear", value), ("gated", dU.double()), ("H", H.double())):
        worst = float(((got - a).abs() / (rel * a.abs())).max())
        print(f"[ops] {name}: worst error / bound {worst:.3f}")
        assert worst <= 1.0, name
    assert torch.equal(wide, forge.linear(z, ident, act="gelu").repeat(1, 16))
    for name, got in (("dZ", dZ.double()), ("dG", dG.double())):
        worst = float(((got - d).abs() / tol_d).max())
        print(f"[ops] {name}: worst error / bound {worst:.3f}")
        assert worst <= 1.0, name


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_derivatives_of_extreme_values(dt):
    """Far out every activation's derivative is its limit, 0 or 1, also where z^2 overflows; NaN
    stays NaN in its own element."""
    mags = [100.0, 1e4, 1e10, 1e19, 6e19, 1e25, 3e38]
    z = torch.tensor(mags + [-m for m in mags] + [float("nan"), 0.0], device="cuda").to(DT[dt]).reshape(2, 8)
    one, two = torch.ones_like(z), torch.full_like(z, 2.0)
    lim = torch.tensor([1.0] * 7 + [0.0] * 7, device="cuda")
    for act in forge.ACTS[1:]:
        dZ, _ = forge.linear_act_backward(one, z, act=act)
        dG, _, _ = forge.gated_backward(one, z, two, act=act)
        for got, scale in ((dZ, 1.0), (dG, 2.0)):
            got = got.float().reshape(-1)
            assert torch.equal(got[:14], lim * scale), act
            assert torch.isnan(got[14]) and torch.isfinite(got[15]), act


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t", [0, 1, 33, 1025])
def test_linear_act_backward_into_a_given_tensor(t, dt):
    """A tensor given for dZ is written and returned, also without an activation."""
    g = gen(t)
    dY, Z = rnd(g, t, 264, dtype=DT[dt]), rnd(g, t, 264, dtype=DT[dt], std=2.0)
    for act in forge.ACTS:
        want, want_db = forge.linear_act_backward(dY, Z, act=act)
        for bias in (True, False):
            buf = torch.full((t, 272), 7.0, device="cuda", dtype=DT[dt])
            dZ, db = forge.linear_act_backward(dY, Z, act=act, want_bias=bias, dZ=buf[:, :264])
            assert dZ.data_ptr() == buf.data_ptr()
            assert torch.equal(dZ, want) and torch.all(buf[:, 264:] == 7.0)
            assert torch.equal(db, want_db) if bias else db is None
    same, _ = forge.linear_act_backward(dY, dZ=dY)
    assert same is dY


def up8(n):
    return (n + 7) // 8 * 8


def exact_head(seed, t, i, v, dtype, kind):
    """A head whose dz and gradients are exact in every order of summation. kind "targets": lse so large
    that every probability is 0, so dz = -[target] w, any W. kind "ones": X and W live in different
    halves of the columns, so every logit is 0, and lse = 0: dz = (1 - [target]) w for all entries.
    X holds whole numbers up to 2, W eighths up to 2, w powers of two."""
    g = gen(seed)
    X = torch.randint(-2, 3, (t, i), generator=g, device="cuda").to(F)
    W = torch.randint(-16, 17, (up8(v), i), generator=g, device="cuda").to(F) / 8
    if kind == "ones":
        X[:, : i // 2] = 0
        W[:, i // 2:] = 0
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    if t > 2:
        y[0], y[1] = v - 1, 0
        y[2::5] = -100
    lse = torch.full((t,), 1e30 if kind == "targets" else 0.0, device="cuda")
    w = 2.0 ** -torch.randint(0, 4, (t,), generator=g, device="cuda").to(F)
    dz = torch.zeros(t, up8(v), device="cuda", dtype=F)
    if kind == "ones":
        dz[:, :v] = 1.0
    keep = y != -100
    r = torch.nonzero(keep)[:, 0]
    dz[r, y[r]] -= 1.0
    dz[~keep] = 0
    return X.to(dtype), W.to(dtype), y, lse, w, dz, keep


HEAD_STEPS = [("bf16", o, s_) for o, s_ in
              [("adamw", "f32"), ("adamw", "bf16"), ("adamw", "q8"), ("adamw", "q8dyn"), ("sgd", "f32"), ("lion", "bf16"),
               ("rmsprop", "q8"), ("nadam", "f32")]] + [("f32", "adamw", "f32"), ("f32", "sgd_momentum", "f32")]


@pytest.mark.parametrize("kind", ["targets", "ones"])
@pytest.mark.parametrize("dt,opt,states", HEAD_STEPS)
@pytest.mark.parametrize("t,v", [(190, 1003), (1501, 2051), (1, 13), (0, 264)])
def test_head_step_of_exact_gradients(t, v, dt, opt, states, kind):
    """Every piece of the head's step against wgrad_step of the whole W on a dz formed here, bit for
    bit: weights with stochastic rounding, moments, scales, from moments that are all different, at a
    step that is not the first; and dX, exact too, of the old W."""
    i = 128
    X, W, y, lse, w, dz, keep = exact_head(t + v, t, i, v, DT[dt], kind)
    g = gen(7)
    m, vv, ms, vs = forge.new_states(W, opt, states)
    for mom in (m, vv):
        if mom is None:
            continue
        if mom.dtype in (torch.int8, torch.uint8):
            lo = -120 if mom.dtype == torch.int8 else 0
            mom.copy_(torch.randint(lo, 120, mom.shape, generator=g, device="cuda"))
        else:
            mom.copy_(torch.rand(mom.shape, generator=g, device="cuda") * 0.25)
    for sc in (ms, vs):
        if sc is not None:
            sc.copy_(torch.rand(sc.shape, generator=g, device="cuda") * 0.01 + 1e-3)
    code = "dynamic" if states == "q8dyn" else "linear"
    hyper = {"lr": 0.05}
    n = int(keep.sum())
    # "none": a factor per token; "sum": one for all
    for red, dloss in (("none", w), ("sum", torch.full((), 0.25, device="cuda"))):
        full = (dz * (w[:, None] if red == "none" else 0.25)).to(DT[dt])
        ref = [None if a is None else a.clone() for a in (W, m, vv, ms, vs)]
        forge.wgrad_step(X, full, ref[0], ref[1], ref[2], opt, hyper, 5, 99, ref[3], ref[4], code=code)
        want_dx = (full.double() @ W.double()).to(F).to(DT[dt])
        for piece in (0, 8, 256, 520):
            if piece == 8 and v > 1500:
                continue
            got = [None if a is None else a[:v].clone() for a in (W, m, vv, ms, vs)]
            dX = forge.linear_cross_entropy_step(X, got[0], got[1], got[2], y, lse, dloss, opt, hyper, 5, 99, got[3],
                                                 got[4], code=code, reduction=red, piece=piece)
            assert torch.equal(dX, want_dx), (red, piece)
            for name, a, b in zip(("W", "m", "v", "m scale", "v scale"), got, ref):
                if a is not None:
                    assert torch.equal(a, b[:v]), (name, red, piece)
            assert n == 0 or not torch.equal(got[0], W[:v])


@pytest.mark.parametrize("kind", ["targets", "ones"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,v", [(190, 1003), (1501, 2051), (1, 13)])
def test_head_gradients_that_are_exact(t, v, dt, kind):
    """dX and dW in pieces of every size: the exact sums, rounded once."""
    i = 128
    X, W, y, lse, w, dz, keep = exact_head(t + v, t, i, v, DT[dt], kind)
    total = torch.tensor([0.0, 128.0, 0.0], device="cuda")  # a mean over 128: a power of two
    one = torch.ones((), device="cuda")
    for red, dloss, f in (("none", w, w[:, None].double()), ("sum", one, 1.0), ("mean", one, 2.0 ** -7)):
        d = dz.double() * f
        want_x = (d @ W.double()).to(F).to(DT[dt])
        want_w = (d.t() @ X.double()).to(F).to(DT[dt])[:v]
        for piece in (0, 8, 256, 520):
            if piece == 8 and v > 1500:
                continue
            dX, dW = forge.linear_cross_entropy_backward(X, W[:v], y, lse, dloss, reduction=red, total=total, piece=piece)
            assert torch.equal(dX, want_x) and torch.equal(dW, want_w), (red, piece)


@pytest.mark.parametrize("t,i,o", [(2100, 512, 29 * 128), (8445, 520, 1024)])
def test_gated_of_a_little_more_than_a_round(t, i, o):
    """261 and 264 tiles of 256 x 128 outputs: the tiles past the first 256 run as smaller ones, as a
    band of columns and as a band of rows."""
    g = gen(t)
    X = rnd(g, t, i)
    Wg, Wu = rnd(g, o, i, std=i ** -0.5), rnd(g, o, i, std=i ** -0.5)
    H, G, U = forge.gated(X, Wg, Wu, act="silu", save=True)
    h, dh, gg, dg, uu, du = gated64(X, Wg, Wu, "silu")
    close("H", H, h, dh)
    close("G", G, gg, dg)
    close("U", U, uu, du)


@pytest.mark.parametrize("t,i,o", [(2100, 512, 29 * 256), (8445, 520, 2048)])
def test_gated_dgrad_of_a_little_more_than_a_round(t, i, o):
    """The same for the gradient through the layer behind."""
    g = gen(t)
    dY, Wd = rnd(g, t, i), rnd(g, i, o, std=o ** -0.5)
    G, U = rnd(g, t, o, std=2.0), rnd(g, t, o)
    dG, dU, H = forge.gated_dgrad(dY, Wd, G, U, act="gelu")
    dh, ddh = mm64(dY, Wd)
    dg, eg, du, eu, h, eh = gated_back64(dh, ddh, G, U, "gelu")
    close("dG", dG, dg, eg)
    close("dU", dU, du, eu)
    close("H", H, h, eh)


def test_cross_entropy_sums_of_dx_past_32_bit_offsets():
    """The float32 sums of dX over two pieces of the vocabulary take 2.3 GB: written with the first
    piece, read with the second."""
    t, i, v = 70000, 8192, 520
    assert t * i * 4 > 2 ** 31
    X, W, y, lse, w, dz, keep = exact_head(3, t, i, v, BF, "targets")
    dX, dW = forge.linear_cross_entropy_backward(X, W, y, lse, w, reduction="none", piece=264)
    # one term per token: -w W[target], exact
    want = torch.zeros(t, i, device="cuda", dtype=BF)
    want[keep] = (-w[keep, None] * W[y[keep]].float()).to(BF)
    assert torch.equal(dX, want)
    del want, dX
    want_w = torch.zeros(v, i, device="cuda", dtype=torch.float64)
    want_w.index_add_(0, y[keep], -w[keep, None].double() * X[keep].double())
    assert torch.equal(dW, want_w.to(F).to(BF))
    del want_w, X, dW
    torch.cuda.empty_cache()


def c_tensor(t):
    import ctypes
    return ctypes.byref(forge.forge._ten(t))


def test_dgrad_group_without_a_workspace():
    """The C call that takes no workspace: the same product with a tile's whole sum in one workgroup."""
    g = gen(4)
    t, i, outs = 15, 512, (6568, 40, 6568)
    dYs, Ws = [rnd(g, t, o) for o in outs], [rnd(g, o, i, std=0.01) for o in outs]
    dX = torch.full((t, i), float("nan"), device="cuda", dtype=BF)
    A = forge.forge.ForgeTensor * len(outs)
    stream = torch.cuda.current_stream().cuda_stream
    st = forge.lib().forge_linear_dgrad_group(len(outs), A(*[forge.forge._ten(d) for d in dYs]),
                                              A(*[forge.forge._ten(w) for w in Ws]), c_tensor(dX), stream)
    assert st == 0
    want, bound = 0, 0
    for d, w in zip(dYs, Ws):
        x, e = mm64(d, w)
        want, bound = want + x, bound + len(outs) * e
    close("dX", dX, want, bound)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("piece", [0, 256])
def test_factors_per_token_of_a_mean(dt, piece):
    """The C calls with a factor per token and a total: every factor is divided by the count. Outputs with
    rows of their own pitch."""
    import ctypes
    t, i, v = 190, 128, 1003
    X, W, y, lse, w, dz, keep = exact_head(t, t, i, v, DT[dt], "targets")
    W = W[:v].contiguous()
    total = torch.tensor([0.0, 128.0, 0.0], device="cuda")
    lib, stream = forge.lib(), torch.cuda.current_stream().cuda_stream
    f = (dz.double() * w[:, None].double() / 128)[:, :v]
    want_x, want_w = (f @ W.double()).to(F).to(DT[dt]), (f.t() @ X.double()).to(F).to(DT[dt])
    big_x = torch.full((t, i + 16), 7.0, device="cuda", dtype=DT[dt])
    big_w = torch.full((v, i + 16), 7.0, device="cuda", dtype=DT[dt])
    need = lib.forge_linear_xent_workspace(t, i, v, forge.forge._DT[DT[dt]], 1, piece)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = lib.forge_linear_xent_backward(c_tensor(X), c_tensor(W), y.data_ptr(), -100, lse.data_ptr(), w.data_ptr(), 1,
                                        total.data_ptr(), c_tensor(big_x[:, :i]), c_tensor(big_w[:, :i]), piece,
                                        ws.data_ptr(), need, stream)
    assert st == 0
    assert torch.equal(big_x[:, :i], want_x) and torch.equal(big_w[:, :i], want_w)
    assert torch.all(big_x[:, i:] == 7.0) and torch.all(big_w[:, i:] == 7.0)
    h = forge.make_hyper("sgd", lr=0.5, stochastic_round=0)
    w1 = W.clone()
    st = lib.forge_linear_xent_step(c_tensor(X), c_tensor(w1), None, None, forge.forge.OPT_ID["sgd"], ctypes.byref(h), 1, 0,
                                    y.data_ptr(), -100, lse.data_ptr(), w.data_ptr(), 1, total.data_ptr(),
                                    c_tensor(big_x[:, :i]), piece, ws.data_ptr(), need, stream)
    assert st == 0
    # sums and products by powers of two are exact: W - lr dW in float32, rounded once
    assert torch.equal(w1, (W.double() - 0.5 * (f.t() @ X.double())).to(F).to(DT[dt]))
    assert torch.equal(big_x[:, :i], want_x)


@pytest.mark.parametrize("piece", [0, 256])
def test_head_step_of_pitched_tensors(piece):
    """W and the moments as views with wider rows, X too: the same bits, the padding untouched."""
    t, i, v = 190, 128, 1003
    X, W, y, lse, w, dz, keep = exact_head(5, t, i, v, BF, "targets")
    W = W[:v].contiguous()
    g = gen(3)
    m, vv = torch.rand(v, i, generator=g, device="cuda"), torch.rand(v, i, generator=g, device="cuda")
    want = [a.clone() for a in (W, m, vv)]
    dX = forge.linear_cross_entropy_step(X, *want, y, lse, w, "adamw", {"lr": 0.05}, 3, 11, reduction="none", piece=piece)
    bigs = []
    for a, extra in ((W, 40), (m, 8), (vv, 24)):
        big = torch.full((v, i + extra), 7.0, device="cuda", dtype=a.dtype)
        big[:, :i] = a
        bigs.append(big)
    got = forge.linear_cross_entropy_step(pitched(X), *[b[:, :i] for b in bigs], y, lse, w, "adamw", {"lr": 0.05}, 3, 11,
                                          reduction="none", piece=piece)
    assert torch.equal(got, dX)
    for a, b in zip(want, bigs):
        assert torch.equal(b[:, :i], a) and torch.all(b[:, i:] == 7.0)


def test_head_of_distant_rows():
    """Rows of W 4 MB apart: a piece of the vocabulary holds fewer of them, in the documented workspace."""
    t, i, v = 190, 128, 1500
    X, W, y, lse, w, dz, keep = exact_head(6, t, i, v, BF, "targets")
    big = torch.empty(v, 1 << 21, device="cuda", dtype=BF)
    far = big[:, :i]
    far.copy_(W[:v])
    want = forge.linear_cross_entropy_backward(X, W[:v], y, lse, w, reduction="none")
    got = forge.linear_cross_entropy_backward(X, far, y, lse, w, reduction="none")
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a, b = forge.linear_cross_entropy(X, W[:v], y), forge.linear_cross_entropy(X, far, y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del big, far
    torch.cuda.empty_cache()


def test_pieces_in_a_graph():
    """Gradients and steps over several pieces of the vocabulary, captured and replayed with eager work
    between the replays."""
    t, i, v = 190, 128, 1003
    X, W, y, lse, w, dz, keep = exact_head(8, t, i, v, BF, "targets")
    W = W[:v].contiguous()
    live, eager = W.clone(), W.clone()
    sl, se = forge.new_states(W, "adamw")[:2], forge.new_states(W, "adamw")[:2]

    def both(wt, st):
        out = forge.linear_cross_entropy_backward(X, wt, y, lse, w, reduction="none", piece=256)
        return [*out, forge.linear_cross_entropy_step(X, wt, *st, y, lse, w, "adamw", {"lr": 0.05}, 2, 11,
                                                      reduction="none", piece=256)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(live, sl)
    torch.cuda.synchronize()
    live.copy_(W)
    for s in sl:
        s.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(live, sl)
    torch.cuda.synchronize()
    for _ in range(4):
        for o in out:
            o.zero_()
        graph.replay()
        want = both(eager, se)
        torch.cuda.synchronize()
        for a, b in zip(out + [live, *sl], want + [eager, *se]):
            assert torch.equal(a, b)


def test_calls_of_two_threads():
    """Two host threads, a stream each: the same bits as one after the other."""
    import threading
    t, i, v = 190, 128, 1003
    cases = [exact_head(k, t, i, v, BF, "targets") for k in (1, 2)]
    G, U = rnd(gen(1), t, 264), rnd(gen(2), t, 264)

    def work(c):
        X, W, y, lse, w, dz, keep = c
        out = [forge.linear(X, W, act="gelu"), *forge.gated(X, W, W, save=True), *forge.gated_backward(G, U, G)]
        return out + list(forge.linear_cross_entropy_backward(X, W[:v], y, lse, w, reduction="none", piece=256))

    want = [work(c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = work(cases[k])
                s.synchronize()
                bad.extend(k for a, b in zip(got, want[k]) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad
