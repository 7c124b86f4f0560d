"""GPU parity of the layers of experts against their float64 forms: the plan of the routes, the rows' way there and back,
the products grouped by expert and their gradients, the fused step of the stack; ragged sizes, experts without rows, dropped
routes, one token, no token, pitched rows, bfloat16 and float32. Tolerances are derived in tests/_ops64.py and
tests/_experts64.py."""
import pytest
import torch

import optimizer_gemm_amd as forge
from _experts64 import (combine64, expert_dgrad64, expert_gated64, expert_gated_dgrad64, expert_linear64, expert_wgrad64,
                        plan64, routes, spans)
from _ops64 import U, close

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F}
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F) * std).to(dtype)


def pitched(t, extra=16):
    """The same values as a view with wider rows, whose padding holds NaN."""
    big = torch.full((*t.shape[:-1], t.shape[-1] + extra), NAN, device=t.device, dtype=t.dtype)
    big[..., : t.shape[-1]] = t
    return big[..., : t.shape[-1]]


def filled(*shape, dtype=BF):
    return torch.full(shape, 7.0, device="cuda", dtype=dtype)


def sizes_to_offsets(sizes, first=0):
    o = [first]
    for n in sizes:
        o.append(o[-1] + n)
    return torch.tensor(o, device="cuda")


# ---- plan ----------------------------------------------------------------------------------------------------
PLANS = [(1, 1, 1), (1, 8, 64), (3, 2, 2), (37, 4, 64), (255, 1, 7), (257, 3, 300), (512, 2, 1024), (1025, 1, 8),
         (1777, 2, 16), (8192, 8, 64), (4099, 5, 1000), (300, 9, 4)]


@pytest.mark.parametrize("t,k,e", PLANS)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_plan(t, k, e, dropped):
    idx = routes(t + k, t, k, e, dropped)
    want_o, want_p = plan64(idx, e)
    offsets, pos = forge.expert_plan(idx.cuda(), e)
    assert offsets.dtype == torch.int64 and pos.dtype == torch.int32
    assert torch.equal(offsets.cpu(), want_o)
    assert torch.equal(pos.cpu(), want_p)


def test_plan_extremes():
    for e in (1, 5, 1024):
        # every route dropped, by every kind of value outside; no token at all; one expert takes all
        bad = torch.tensor([[-1, e], [2 ** 40, -2 ** 62]], device="cuda")
        offsets, pos = forge.expert_plan(bad, e)
        assert torch.all(offsets == 0) and torch.all(pos == -1)
        offsets, pos = forge.expert_plan(torch.empty(0, 3, dtype=torch.int64, device="cuda"), e)
        assert torch.all(offsets == 0) and offsets.numel() == e + 1 and pos.shape == (0, 3)
        idx = torch.full((700, 3), e - 1, device="cuda", dtype=torch.int64)
        offsets, pos = forge.expert_plan(idx, e)
        assert torch.equal(pos.reshape(-1).cpu(), torch.arange(2100, dtype=torch.int32))
        assert offsets[-1] == 2100 and torch.all(offsets[:-1] == 0)


@pytest.mark.parametrize("t,k,e", [(256, 2, 1024), (171, 3, 5), (2047, 1, 1024), (1024, 2, 64), (683, 3, 1), (1, 2048, 9)])
def test_plan_of_one_block_and_its_borders(t, k, e):
    for n in (0.0, 0.3):
        idx = routes(t + e, t, k, e, dropped=n)
        off, pos = forge.expert_plan(idx.cuda(), e)
        o, p = plan64(idx, e)
        assert torch.equal(off.cpu(), o) and torch.equal(pos.cpu(), p)


def test_plan_beyond_512_blocks():
    """blocks of more than one turn: 512 x 1024 routes and some"""
    idx = torch.randint(-1, 33, (600001, 1), device="cuda", generator=gen(1))
    offsets, pos = forge.expert_plan(idx, 32)
    key = idx[:, 0].clone()
    key[(key < 0) | (key >= 32)] = 32
    order = torch.sort(key, stable=True).indices
    want = torch.empty_like(key)
    want[order] = torch.arange(key.numel(), device="cuda")
    want[key == 32] = -1
    assert torch.equal(pos[:, 0].long(), want)
    assert torch.equal(offsets[1:], torch.bincount(key, minlength=33)[:32].cumsum(0))


# ---- there and back -------------------------------------------------------------------------------------------
ROWS = [(1, 2, 4, 64), (3, 1, 2, 8), (37, 4, 64, 2048), (255, 8, 5, 520), (1777, 2, 16, 136), (4100, 3, 8, 1032), (130, 11, 16, 4104),
        (5, 2, 4, 16392)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,k,e,d", ROWS)
def test_dispatch_and_combine(t, k, e, d, dt):
    g = gen(t + d)
    idx = routes(t + d, t, k, e, dropped=0.2 if t > 1 else 0.0).cuda()
    offsets, pos = forge.expert_plan(idx, e)
    n = int(offsets[-1])
    X, R = rnd(g, t, d, dtype=DT[dt]), rnd(g, t, d, dtype=DT[dt])
    w = torch.rand(t, k, device="cuda", generator=g)
    Xp = forge.expert_dispatch(X, pos, out=filled(t * k, d, dtype=DT[dt]))
    want = filled(t * k, d, dtype=DT[dt])
    at = torch.nonzero(pos.reshape(-1) >= 0)[:, 0]
    want[pos.reshape(-1)[at].long()] = X[at // k]
    assert torch.equal(Xp, want)
    assert n == t * k or torch.all(Xp[n:] == 7.0)
    # rows that no route has hold NaN, and reach nothing
    Yp = rnd(g, t * k, d, dtype=DT[dt])
    Yp[n:] = NAN
    close("combine", forge.expert_combine(Yp, pos, w), *combine64(Yp, pos, w))
    close("ones", forge.expert_combine(Yp, pos), *combine64(Yp, pos, None))
    close("residual", forge.expert_combine(Yp, pos, w, residual=R), *combine64(Yp, pos, w, R))
    dY = rnd(g, t, d, dtype=DT[dt])
    dYp, dw = forge.expert_combine_backward(dY, Yp, pos, w)
    wp = torch.zeros(t * k, device="cuda", dtype=torch.float64)
    tok = torch.zeros(t * k, device="cuda", dtype=torch.int64)
    rows = pos.reshape(-1)[at].long()
    wp[rows], tok[rows] = w.reshape(-1)[at].double(), at // k
    want = dY.double()[tok[:n]] * wp[:n, None]
    close("dYp", dYp[:n], want, U * want.abs())
    prod = torch.where((pos >= 0)[:, :, None], Yp.double()[pos.long().clamp(min=0)] * dY.double()[:, None, :], 0.0)
    close("dw", dw, prod.sum(2), (d + 1) * U * prod.abs().sum(2))
    assert torch.all(dw[pos < 0] == 0)
    only, none = forge.expert_combine_backward(dY, None, pos, w, want_dweights=False)
    assert none is None and torch.equal(only[:n], dYp[:n])


@pytest.mark.parametrize("t,k,e,d", ROWS)
def test_float32_results_of_bfloat16_tokens(t, k, e, d):
    """Yp in float32, the tokens' side in bfloat16: combined and back"""
    g = gen(t + d)
    offsets, pos = forge.expert_plan(routes(t + d, t, k, e, dropped=0.2 if t > 1 else 0.0).cuda(), e)
    n = int(offsets[-1])
    Yp, R, dY = rnd(g, t * k, d, dtype=F), rnd(g, t, d), rnd(g, t, d)
    Yp[n:] = NAN
    w = torch.rand(t, k, device="cuda", generator=g)
    close("combine", forge.expert_combine(Yp, pos, w, out_dtype=BF), *combine64(Yp, pos, w))
    Y = forge.expert_combine(Yp, pos, w, residual=R)
    assert Y.dtype == BF
    close("residual", Y, *combine64(Yp, pos, w, R))
    dYp, dw = forge.expert_combine_backward(dY, Yp, pos, w)
    same, _ = forge.expert_combine_backward(dY, Yp.to(BF), pos, w)
    assert dYp.dtype == BF and torch.equal(dYp[:n], same[:n])
    prod = torch.where((pos >= 0)[:, :, None], Yp.double()[pos.long().clamp(min=0)] * dY.double()[:, None, :], 0.0)
    close("dw", dw, prod.sum(2), (d + 1) * U * prod.abs().sum(2))


def test_combine_pitched_rows_and_repeats():
    g = gen(3)
    idx = routes(3, 50, 3, 6, 0.2).cuda()
    offsets, pos = forge.expert_plan(idx, 6)
    w = torch.rand(50, 3, device="cuda", generator=g)
    X, Yp, dY = rnd(g, 50, 264), rnd(g, 150, 264), rnd(g, 50, 264)
    out = filled(50, 280)
    got = forge.expert_combine(pitched(Yp), pos, w, residual=pitched(X, 8), out=out[:, :264])
    assert torch.equal(got, forge.expert_combine(Yp, pos, w, residual=X)) and torch.all(out[:, 264:] == 7.0)
    big = filled(150, 272)
    forge.expert_dispatch(pitched(X), pos, out=big[:, :264])
    n = int(offsets[-1])
    assert torch.equal(big[:n, :264], forge.expert_dispatch(X, pos)[:n])
    assert torch.all(big[:, 264:] == 7.0) and torch.all(big[n:] == 7.0)
    a = forge.expert_combine_backward(dY, Yp, pos, w)
    b = forge.expert_combine_backward(pitched(dY), pitched(Yp, 8), pos, w)
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1], b[1])


def test_places_outside_are_skipped():
    X = torch.ones(4, 16, device="cuda", dtype=BF)
    pos = torch.tensor([[0, 5], [-7, 2], [2 ** 30, -1], [1, 3]], device="cuda", dtype=torch.int32)
    out = filled(4, 16)
    forge.expert_dispatch(X, pos, out=out)
    assert torch.all(out == 1.0)
    Y = forge.expert_combine(X, pos)
    assert Y[:, 0].tolist() == [1.0, 1.0, 0.0, 2.0]
    _, dw = forge.expert_combine_backward(X, X, pos)
    assert dw.tolist() == [[16.0, 0.0], [0.0, 16.0], [0.0, 0.0], [16.0, 16.0]]


def test_dispatch_takes_int8_rows_and_their_factors():
    g = gen(4)
    for t, d in ((1, 16), (9, 4112), (300, 64)):
        Q = torch.randint(-127, 128, (t, d), device="cuda", generator=g).to(torch.int8)
        s = torch.rand(t, device="cuda", generator=g)
        offsets, pos = forge.expert_plan(routes(t, t, 2, 4, 0.1).cuda(), 4)
        Qp, sp = forge.expert_dispatch(Q, pos, scale=s)
        for j in range(2):
            at = torch.nonzero(pos[:, j] >= 0)[:, 0]
            assert torch.equal(Qp[pos[at, j].long()], Q[at]) and torch.equal(sp[pos[at, j].long()], s[at])


# ---- products -----------------------------------------------------------------------------------------------
# rows of each expert, in, out: one row; rows of one expert only; tiles in every direction; more experts than a wave
# has lanes; hundreds of rows
SIZES = [([1], 8, 8), ([0, 1, 0], 512, 264), ([2, 0, 3], 72, 40), ([7, 0, 0, 9], 4096, 128), ([33, 1], 136, 1032),
         ([0, 130, 0, 64, 65, 1], 264, 520), ([257, 40, 0, 300], 96, 328), ([511, 513, 1], 1000, 776), ([1000], 256, 2056),
         ([20] * 70, 128, 136), ([2500, 1, 0, 900, 1800], 192, 2600), ([1100, 1500, 700, 1290], 128, 4360), ([0] * 65 + [3, 150] + [0] * 100 + [1], 200, 72), ([900, 10, 1300, 700], 520, 1288)]


def stacked(g, e, o, i, dtype, std=None):
    return rnd(g, e, o, i, dtype=dtype, std=i ** -0.5 if std is None else std)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_products(case, dt):
    sizes, i, o = SIZES[case]
    dtype, e = DT[dt], len(sizes)
    g = gen(case * 31 + i + o)
    # rows in front of the first expert's and behind the last one's belong to none
    first, behind = (3, 5) if case % 2 else (0, 0)
    off = sizes_to_offsets(sizes, first)
    n = int(off[-1])
    R = n + behind
    act = forge.ACTS[case % 5]
    used = slice(first, n)

    def rows(*shape, std=1.0):
        t = rnd(g, *shape, dtype=dtype, std=std)
        t[:first], t[n:] = NAN, NAN
        return t

    def rest(t):
        assert torch.all(t[:first] == 7.0) and torch.all(t[n:] == 7.0)
        return t[used]

    loc = off - first
    X, W, Wu = rows(R, i), stacked(g, e, o, i, dtype), stacked(g, e, o, i, dtype)
    y, dy, z, dz = expert_linear64(X[used], W, loc, act)
    close(f"linear {act}", rest(forge.expert_linear(X, W, off, act=act, out=filled(R, o, dtype=dtype))), y, dy)
    if i % 8 == 0 and o % 8 == 0:
        y, dy = expert_linear64(X[used], W, loc, "none")[:2]
        close("float32 sums", rest(forge.expert_linear(X, W, off, out=filled(R, o, dtype=F))), y, dy)
    Y, Z = forge.expert_linear(X, W, off, act=act, save=True)
    close("Z", Z[used], z, dz)
    h, dh, gt, dg, u, du = expert_gated64(X[used], W, Wu, loc, act)
    close(f"gated {act}", rest(forge.expert_gated(X, W, Wu, off, act=act, out=filled(R, o, dtype=dtype))), h, dh)
    H, G, V = forge.expert_gated(X, W, Wu, off, act=act, save=True)
    assert torch.equal(H[used], forge.expert_gated(X, W, Wu, off, act=act)[used])
    close("G", G[used], gt, dg)
    close("U", V[used], u, du)
    # backward: the layer behind has weights [e, i, o] and gradient rows of i
    Wd, dYd, G, V = stacked(g, e, i, o, dtype), rows(R, i), rows(R, o), rows(R, o)
    got = forge.expert_gated_dgrad(dYd, Wd, G, V, off, act=act)
    want = expert_gated_dgrad64(dYd[used], Wd, G[used], V[used], loc, act)
    for name, a, b in zip(("dG", "dU", "H"), got, (want[:2], want[2:4], want[4:])):
        close(f"{name} {act}", a[used], *b)
    d1, d2 = rows(R, o), rows(R, o)
    dX = forge.expert_dgrad_group([d1, d2], [W, Wu], off, dX=filled(R, i, dtype=dtype))
    close("dX", rest(dX), *expert_dgrad64([d1[used], d2[used]], [W, Wu], loc))
    close("dX of one", forge.expert_dgrad_group([d1], [W], off)[used], *expert_dgrad64([d1[used]], [W], loc))
    dW = forge.expert_wgrad(X, d1, off)
    close("dW", dW, *expert_wgrad64(X[used], d1[used], loc))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_products_pitched(dt):
    dtype = DT[dt]
    g = gen(8)
    off = sizes_to_offsets([40, 0, 3, 100])
    X, W, Wu, D = rnd(g, 143, 264, dtype=dtype), stacked(g, 4, 200, 264, dtype), stacked(g, 4, 200, 264, dtype), rnd(g, 143, 200, dtype=dtype)
    pX, pW, pWu, pD = pitched(X), pitched(W, 8), pitched(Wu), pitched(D, 24)
    out = filled(143, 208, dtype=dtype)
    assert torch.equal(forge.expert_linear(pX, pW, off, act="silu", out=out[:, :200]), forge.expert_linear(X, W, off, act="silu"))
    assert torch.all(out[:, 200:] == 7.0)
    assert torch.equal(forge.expert_gated(pX, pW, pWu, off), forge.expert_gated(X, W, Wu, off))
    assert torch.equal(forge.expert_dgrad_group([pD, D], [pW, Wu], off), forge.expert_dgrad_group([D, D], [W, Wu], off))
    dW = filled(4, 200, 272, dtype=F)
    assert torch.equal(forge.expert_wgrad(pX, pD, off, dW=dW[:, :, :264]), forge.expert_wgrad(X, D, off))
    assert torch.all(dW[:, :, 264:] == 7.0)


# input gradients of few tiles over a long k, which workgroups share: rows of each expert, the layers' out, in
SPLITS = [([481], [11160, 11160], 64), ([3, 0, 700, 50], [4096, 3000, 1104], 264), ([600, 101, 0, 500], [26304], 440),
          ([7] * 70, [1200, 1200], 72), ([9, 0, 12], [8200], 136), ([1], [6400], 8)]


@pytest.mark.parametrize("case", range(len(SPLITS)))
def test_input_gradient_shared_along_k(case):
    sizes, outs, i = SPLITS[case]
    e, g = len(sizes), gen(100 + case)
    first, behind = (3, 5) if case % 2 else (0, 0)
    off = sizes_to_offsets(sizes, first)
    n = int(off[-1])
    R = n + behind
    assert forge.lib().forge_expert_dgrad_group_workspace(R, i, sum(outs), e, forge.forge.BF16) > 0
    W, D = [stacked(g, e, o, i, BF, std=o ** -0.5) for o in outs], [rnd(g, R, o) for o in outs]
    for d in D:
        d[:first], d[n:] = NAN, NAN
    dX = forge.expert_dgrad_group(D, W, off, dX=filled(R, i))
    assert torch.all(dX[:first] == 7.0) and torch.all(dX[n:] == 7.0)
    close("dX", dX[first:n], *expert_dgrad64([d[first:n] for d in D], W, off - first))
    out = filled(R, i + 16)
    forge.expert_dgrad_group([pitched(d) for d in D], [pitched(w) for w in W], off, dX=out[:, :i])
    assert torch.equal(out[first:n, :i], dX[first:n]) and torch.all(out[:, i:] == 7.0)
    # offsets that are none reach nothing outside
    around = filled(R + 20, i)
    for o in ([-5] + [2 ** 40] * e, [R] * e + [0], [0, R] * ((e + 1) // 2) + [R] * ((e + 1) % 2)):
        forge.expert_dgrad_group(D, W, torch.tensor(o, device="cuda"), dX=around[10:R + 10])
        assert torch.all(around[:10] == 7.0) and torch.all(around[R + 10:] == 7.0)


def test_no_rows():
    W, off = rnd(gen(1), 3, 16, 24), torch.zeros(4, dtype=torch.int64, device="cuda")
    X, D = torch.empty(0, 24, device="cuda", dtype=BF), torch.empty(0, 16, device="cuda", dtype=BF)
    assert forge.expert_linear(X, W, off).shape == (0, 16)
    assert forge.expert_gated(X, W, W, off).shape == (0, 16)
    assert forge.expert_dgrad_group([D], [W], off).shape == (0, 24)
    assert torch.all(forge.expert_wgrad(X, D, off) == 0)
    # rows there, but all of them behind the last expert's
    X = torch.full((5, 24), NAN, device="cuda", dtype=BF)
    out = forge.expert_linear(X, W, off, out=filled(5, 16))
    assert torch.all(out == 7.0)
    assert torch.all(forge.expert_wgrad(X, torch.full((5, 16), NAN, device="cuda", dtype=BF), off) == 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t", [3, 700])
def test_no_inner_dimension(t, dt):
    """sums of nothing are zeros, for the rows that belong to an expert"""
    dtype = DT[dt]
    off = torch.tensor([0, 1, 1, t - 1], device="cuda")

    def none(*shape):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def zeros(a):
        assert torch.all(a[:t - 1] == 0)

    out = filled(t, 264, dtype=dtype)
    zeros(forge.expert_linear(none(t, 0), none(3, 264, 0), off, act="silu", out=out))
    assert torch.all(out[t - 1:] == 7.0)
    zeros(forge.expert_gated(none(t, 0), none(3, 264, 0), none(3, 264, 0), off))
    zeros(forge.expert_dgrad_group([none(t, 0)], [none(3, 0, 264)], off))
    G = filled(t, 264, dtype=dtype)
    dG, dU, H = forge.expert_gated_dgrad(none(t, 0), none(3, 0, 264), G, G, off)
    zeros(dG)
    zeros(dU)
    assert torch.all(H[:t - 1] == H[0, 0]) and float(H[0, 0]) > 48
    if dt == "bf16":
        zeros(forge.expert_linear(none(t, 0), none(3, 264, 0), off, out=filled(t, 264, dtype=F)))


def test_operands_that_are_refused():
    X, W, off = rnd(gen(1), 8, 32), rnd(gen(2), 2, 16, 32), torch.tensor([0, 4, 8], device="cuda")
    pos = torch.arange(8, device="cuda", dtype=torch.int32).reshape(8, 1)
    Q, s = forge.quantize_rows(X)
    q, sw = forge.quantize_rows(W.reshape(-1, 32))
    q = q.view(2, 16, 32)
    for what, call in (
            ("contiguous", lambda: forge.expert_linear(rnd(gen(1), 32, 8).t(), W, off)),
            ("contiguous", lambda: forge.expert_linear(X, rnd(gen(2), 2, 32, 16).transpose(1, 2), off)),
            ("one pitch", lambda: forge.expert_linear(X, rnd(gen(2), 2, 20, 32)[:, :16], off)),
            ("two dimensions", lambda: forge.expert_linear(X[None], W, off)),
            ("two dimensions", lambda: forge.quantize_rows(X[0])),
            ("unsupported dtype", lambda: forge.expert_linear(X.double(), W, off)),
            ("unsupported dtype", lambda: forge.expert_dispatch(X.half(), pos)),
            ("one device", lambda: forge.expert_linear(X, W.cpu(), off)),
            ("one device", lambda: forge.expert_combine(X, pos.cpu())),
            ("one device", lambda: forge.expert_linear(X, W, off.cpu())),
            ("offsets", lambda: forge.expert_linear(X, W, off.int())),
            ("int8 codes", lambda: forge.linear_q8(X, s, q[0], sw[:16])),
            ("factors", lambda: forge.linear_q8(Q, s[:7], q[0], sw[:16])),
            ("factors", lambda: forge.linear_q8(Q, s.double(), q[0], sw[:16])),
            ("factors", lambda: forge.expert_linear_q8(Q, s, q, sw[:31], off)),
            ("factors", lambda: forge.expert_dispatch(Q, pos, scale=s[::2])),
            ("contiguous vector", lambda: forge.linear_q8(Q, s, q[0], sw[:16], bias=torch.zeros(1, 16, device="cuda"))),
            ("group holds", lambda: forge.expert_dgrad_group([X], [W, W], off))):
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: forge.expert_linear(X.float(), W, off), lambda: forge.expert_linear(X[:, :24], W, off),
                 lambda: forge.expert_linear(X, W, off, out=X[:, :16]), lambda: forge.expert_dispatch(X, pos, out=X)):
        with pytest.raises(forge.ForgeError):
            call()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_that_are_no_offsets_stay_inside(dt):
    """values outside 0 .. rows or out of order reach no memory outside the operands: the rows around the views keep
    their values, and the call returns"""
    dtype = DT[dt]
    g = gen(9)
    around = filled(300, 64, dtype=dtype)
    X, W = rnd(g, 100, 32, dtype=dtype), stacked(g, 4, 64, 32, dtype)
    for o in ([-5, 10, 400, 50, 2 ** 40], [90, 20, 10, 0, -1], [2 ** 62, -2 ** 62, 2 ** 62, 7, 100], [100, 100, 100, 100, 2 ** 33],
              [0, 100, 0, 100, 0], [100, 0, 100, 0, 100]):
        off = torch.tensor(o, device="cuda")
        forge.expert_linear(X, W, off, out=around[100:200])
        forge.expert_gated(X, W, W, off, out=around[100:200])
        D = rnd(g, 100, 64, dtype=dtype)
        forge.expert_dgrad_group([D], [W], off)
        forge.expert_wgrad(X, D, off)
        if dtype == BF:
            forge.expert_linear(X, W, off, out=filled(100, 64, dtype=F))
            Q, s = forge.quantize_rows(X)
            q, sw = forge.quantize_rows(W.reshape(-1, 32))
            forge.expert_linear_q8(Q, s, q.view(4, 64, 32), sw, off, out=around[100:200])
            forge.expert_gated_q8(Q, s, q.view(4, 64, 32), sw, q.view(4, 64, 32), sw, off, out=around[100:200])
        assert torch.all(around[:100] == 7.0) and torch.all(around[200:] == 7.0)


def test_a_stack_past_two_gigabytes():
    """the last expert's matrix begins past 2^31 bytes"""
    g = gen(2)
    e, o, i = 9, 8192, 16384
    W = torch.zeros(e, o, i, device="cuda", dtype=BF)
    W[8] = rnd(g, o, i, std=i ** -0.5)
    off = torch.tensor([0] * 7 + [2, 2, 43], device="cuda")
    X = rnd(g, 43, i)
    Y = forge.expert_linear(X, W, off)
    assert torch.all(Y[:2] == 0)
    from _ops64 import linear64
    close("last expert", Y[2:], *linear64(X[2:], W[8])[:2])
    D = rnd(g, 43, o)
    dX = forge.expert_dgrad_group([D], [W], off)
    from _ops64 import mm64
    close("its dX", dX[2:], *mm64(D[2:], W[8]))


# ---- the fused step --------------------------------------------------------------------------------------------
def exact_operands(g, sizes, i, o, dtype):
    """small whole numbers times powers of two: every sum of the gradient is exact in float32, in any order"""
    off = sizes_to_offsets(sizes)
    n = int(off[-1])
    X = torch.randint(-4, 5, (n, i), device="cuda", generator=g).to(dtype)
    dY = (torch.randint(-4, 5, (n, o), device="cuda", generator=g).to(F) * 2.0 ** -12).to(dtype)
    return off, X, dY


STEPS = [([40, 0, 3, 100], 64, 72), ([0, 700, 33, 0, 1, 300], 192, 264), ([5] * 67, 128, 64), ([900, 1200], 512, 520)]


def states(W, opt, fmt, g):
    m, v, ms, vs = forge.new_states(W, opt, fmt)
    code = "dynamic" if fmt == "q8dyn" else "linear"
    for t, s in ((m, ms), (v, vs)):
        if t is None:
            continue
        if t.dtype == torch.int8:
            t.copy_(torch.randint(-127, 128, t.shape, device="cuda", generator=g))
        elif t.dtype == torch.uint8:
            t.copy_(torch.randint(0, 256, t.shape, device="cuda", generator=g))
        else:
            t.copy_(torch.rand(t.shape, device="cuda", generator=g) * 1e-3)
        if s is not None:
            s.copy_(torch.rand(s.shape, device="cuda", generator=g) * 1e-4)
    return m, v, ms, vs, code


def clones(ts):
    return [t.clone() if isinstance(t, torch.Tensor) else t for t in ts]


@pytest.mark.parametrize("case", range(len(STEPS)))
@pytest.mark.parametrize("fmt", ["f32", "bf16", "q8", "q8dyn"])
def test_step_is_that_of_the_stack_as_one_layer(case, fmt):
    """On exact gradients the step has the same bits as the stand-alone optimizer pass over the stack as one layer
    [experts * out, in] with the stored gradient."""
    sizes, i, o = STEPS[case]
    e = len(sizes)
    opts = forge.OPTIMIZERS if case == 1 else (forge.OPTIMIZERS[case], "adamw")
    for n, opt in enumerate(opts):
        g = gen(case * 10 + n)
        off, X, dY = exact_operands(g, sizes, i, o, BF)
        W = rnd(g, e, o, i, std=0.02)
        st = states(W, opt, fmt, g)
        W2, st2 = W.clone(), clones(st)
        sr = {"stochastic_round": n % 2}
        forge.expert_wgrad_step(X, dY, W, st[0], st[1], off, opt, sr, 5, 99, st[2], st[3], code=st[4])
        dW = forge.expert_wgrad(X, dY, off)
        assert torch.equal(dW.double(), expert_wgrad64(X, dY, off)[0])
        flat = lambda t: None if t is None else t.view(e * o, -1)  # noqa: E731
        forge.optimizer_step(flat(dW), flat(W2), flat(st2[0]), flat(st2[1]), opt, sr, 5, 99, flat(st2[2]), flat(st2[3]),
                             code=st[4])
        assert torch.equal(W, W2), opt
        for a, b in zip(st[:4], st2[:4]):
            assert a is None or torch.equal(a, b), (opt, fmt)


@pytest.mark.parametrize("case", range(len(STEPS)))
def test_step_float32(case):
    sizes, i, o = STEPS[case]
    e = len(sizes)
    for n, opt in enumerate(forge.OPTIMIZERS):
        g = gen(case * 10 + n)
        off, X, dY = exact_operands(g, sizes, i, o, F)
        W = rnd(g, e, o, i, dtype=F, std=0.02)
        st = states(W, opt, "f32", g)
        W2, st2 = W.clone(), clones(st)
        forge.expert_wgrad_step(X, dY, W, st[0], st[1], off, opt, None, 3, 1)
        dW = forge.expert_wgrad(X, dY, off)
        flat = lambda t: None if t is None else t.view(e * o, -1)  # noqa: E731
        forge.optimizer_step(flat(dW), flat(W2), flat(st2[0]), flat(st2[1]), opt, None, 3, 1)
        # both passes round each operation of the update on its own path: a step of float32 or two
        close("W", W, W2.double(), 8 * U * W2.double().abs() + 8 * U * 1e-3)
        for a, b in zip(st[:2], st2[:2]):
            if a is not None:
                close("moment", a, b.double(), 4 * U * b.double().abs() + 4 * U * 1e-6)


def test_step_pitched_stack():
    g = gen(12)
    off, X, dY = exact_operands(g, [30, 0, 170], 128, 72, BF)
    W, m, v = rnd(g, 3, 72, 128), rnd(g, 3, 72, 128, dtype=F, std=1e-3), rnd(g, 3, 72, 128, dtype=F, std=1e-3).abs()
    pW, pm, pv = pitched(W, 8), pitched(m, 4), pitched(v, 12)
    forge.expert_wgrad_step(pitched(X), pitched(dY, 8), pW, pm, pv, off, "adamw", None, 2, 7)
    forge.expert_wgrad_step(X, dY, W, m, v, off, "adamw", None, 2, 7)
    assert torch.equal(pW, W) and torch.equal(pm, m) and torch.equal(pv, v)


def test_an_expert_without_rows_still_steps():
    g = gen(13)
    W = rnd(g, 2, 64, 64)
    W2 = W.clone()
    off = torch.tensor([0, 0, 10], device="cuda")
    X, dY = rnd(g, 10, 64), rnd(g, 10, 64)
    forge.expert_wgrad_step(X, dY, W, None, None, off, "sgd", {"lr": 0.5, "weight_decay": 0.5, "stochastic_round": 0}, 1, 1)
    # theta - lr wd theta, rounded to bfloat16 once from float32
    assert torch.equal(W[0], (W2[0].float() - 0.5 * (0.5 * W2[0].float())).to(BF))
    assert not torch.equal(W[1], W2[1])


# ---- the roundings of a token's gradient -------------------------------------------------------------------------------
@pytest.mark.parametrize("k", [1, 2, 8])
def test_gradient_of_a_token_with_several_routes(k):
    """The input gradient of each route is a bfloat16 row (the half step of each is in the bound), their sum is float32 and
    rounded once more"""
    g = gen(40 + k)
    t, e, d, h = 300, 8, 264, 520
    offsets, pos = forge.expert_plan(routes(k, t, k, e, dropped=0.1).cuda(), e)
    n = int(offsets[-1])
    W = [stacked(g, e, h, d, BF), stacked(g, e, h, d, BF)]
    D = [rnd(g, t * k, h), rnd(g, t * k, h)]
    dX = forge.expert_combine(forge.expert_dgrad_group(D, W, offsets), pos)
    x, dx = expert_dgrad64([a[:n] for a in D], W, offsets)
    dx = dx + 2.0 ** -8 * (x.abs() + dx)
    p, got = pos.long().clamp(min=0), (pos >= 0)[:, :, None]
    rows, bound = torch.where(got, x[p.clamp(max=n - 1)], 0.0), torch.where(got, dx[p.clamp(max=n - 1)], 0.0)
    want, bound = rows.sum(1), bound.sum(1) + (k + 1) * U * (rows.abs() + bound).sum(1)
    close(f"dx of {k} routes", dX, want, bound)
    print(f"[ops] relative error {float((dX.double() - want).norm() / want.norm()):.5f}, of one rounding "
          f"{float((want.to(BF).double() - want).norm() / want.norm()):.5f}")


# ---- a gradient against differences ------------------------------------------------------------------------------
def test_gradients_against_differences():
    """The block's input gradient in float32 against central differences of the float64 form at the same point"""
    g = gen(21)
    t, k, e, d, h = 6, 2, 3, 16, 24
    idx = routes(21, t, k, e).cuda()
    offsets, pos = forge.expert_plan(idx, e)
    X, w = rnd(g, t, d, dtype=F), torch.rand(t, k, device="cuda", generator=g)
    Wg, Wu, Wd = (stacked(g, e, h, d, F), stacked(g, e, h, d, F), stacked(g, e, d, h, F))
    dY = rnd(g, t, d, dtype=F)

    def loss(x, wts):
        out = 0.0
        for tt in range(t):
            for j in range(k):
                a = int(idx[tt, j])
                hid = torch.nn.functional.silu(Wg[a].double() @ x[tt]) * (Wu[a].double() @ x[tt])
                out = out + wts[tt, j] * ((Wd[a].double() @ hid) @ dY[tt].double())
        return float(out)

    Xp = forge.expert_dispatch(X, pos)
    H, G, V = forge.expert_gated(Xp, Wg, Wu, offsets, save=True)
    Yp = forge.expert_linear(H, Wd, offsets)
    dYp, dw = forge.expert_combine_backward(dY, Yp, pos, w)
    dG, dU, _ = forge.expert_gated_dgrad(dYp, Wd, G, V, offsets)
    dX = forge.expert_combine(forge.expert_dgrad_group([dG, dU], [Wg, Wu], offsets), pos)
    x64, w64, eps = X.double(), w.double(), 1e-5
    for tt, c in ((0, 0), (2, 5), (5, 15), (3, 8)):
        up, dn = x64.clone(), x64.clone()
        up[tt, c] += eps
        dn[tt, c] -= eps
        diff = (loss(up, w64) - loss(dn, w64)) / (2 * eps)
        # differences: the third derivative times eps^2; the kernels: some hundred float32 roundings of sums of order 1
        assert abs(diff - float(dX[tt, c])) <= 1e-7 + 300 * U * max(1.0, float(dX.abs().max()))
    for tt, j in ((0, 0), (4, 1)):
        up, dn = w64.clone(), w64.clone()
        up[tt, j] += eps
        dn[tt, j] -= eps
        diff = (loss(x64, up) - loss(x64, dn)) / (2 * eps)
        assert abs(diff - float(dw[tt, j])) <= 1e-7 + 300 * U * max(1.0, float(dw.abs().max()))


# ---- rows past 2^31 bytes ------------------------------------------------------------------------------------------
def test_float32_results_past_two_gigabytes():
    """float32 results of bfloat16 and 8-bit operands, combined and back: 150003 rows of 4096, 2.46e9 bytes. A row of a
    product does not depend on the others, nor, with one stage of k, on the tiles: the same bits as in calls of fewer rows."""
    g = gen(31)
    t, k, e, i, d = 50001, 3, 4, 64, 4096
    off = sizes_to_offsets([40000, 0, 70000, 40003])
    R = t * k
    assert R * d * 4 > 2 ** 31 and int(off[-1]) == R
    X, W = rnd(g, R, i), stacked(g, e, d, i, BF)
    Q, s = forge.quantize_rows(X)
    q, sw = forge.quantize_rows(W.reshape(-1, i))
    q = q.view(W.shape)

    def by_parts(whole, call):
        for a, b, c in spans(off):
            lo = max(b, c - 7000)
            part = torch.zeros(e + 1, device="cuda", dtype=torch.int64)
            part[a + 1:] = c - lo
            assert torch.equal(whole[lo:c], call(lo, c, part))

    Yp = forge.expert_linear_q8(Q, s, q, sw, off, out_dtype=F)
    by_parts(Yp, lambda lo, hi, o: forge.expert_linear_q8(Q[lo:hi], s[lo:hi], q, sw, o, out_dtype=F))
    del Yp
    Yp = forge.expert_linear(X, W, off, out_dtype=F)
    by_parts(Yp, lambda lo, hi, o: forge.expert_linear(X[lo:hi], W, o, out_dtype=F))
    pos = torch.randperm(R, device="cuda", generator=g).to(torch.int32).reshape(t, k)
    w, dY = torch.rand(t, k, device="cuda", generator=g), rnd(g, t, d)
    Y = forge.expert_combine(Yp, pos, w, out_dtype=BF)
    dYp, dw = forge.expert_combine_backward(dY, Yp, pos, w)
    assert torch.any(pos > 2 ** 31 // (4 * d))
    for lo in range(0, t, 10000):
        at = slice(lo, min(t, lo + 10000))
        close("combine", Y[at], *combine64(Yp, pos[at], w[at]))
        rows = pos[at].long()
        p = Yp[rows].double() * dY[at].double()[:, None, :]
        close("dw", dw[at], p.sum(2), (d + 1) * U * p.abs().sum(2))
        want = dY[at].double()[:, None, :] * w[at].double()[:, :, None]
        close("dYp", dYp[rows].reshape(-1, d), want.reshape(-1, d), U * want.abs().reshape(-1, d))
        del p, want
