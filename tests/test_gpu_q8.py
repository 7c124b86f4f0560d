"""GPU parity of the products of 8-bit integers and of the rows' quantisation against their float64 forms: one token to
hundreds, sizes that are no multiple of any tile, the largest codes, extreme rows, grouped by expert. Tolerances are
derived in tests/_ops64.py and tests/_experts64.py."""
import numpy as np
import pytest
import torch

import optimizer_gemm_amd as forge
from _experts64 import gated_q8_64, grouped, linear_q8_64, spans
from _ops64 import U, close

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    return torch.randint(-127, 128, shape, device="cuda", generator=g).to(torch.int8)


def scales(g, *shape):
    return (torch.rand(*shape, device="cuda", generator=g) + 0.5) * 1e-3


def rnd(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F) * std).to(dtype)


# ---- quantisation ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("t,d", [(1, 16), (1, 4096), (3, 48), (37, 1040), (513, 2048), (5, 16384), (2, 40000), (4100, 1056)])
def test_quantize_rows(t, d, dt):
    g = gen(t + d)
    X = rnd(g, t, d, dtype=dt)
    X[0, d // 2] *= 50.0
    Q, s = forge.quantize_rows(X)
    x = X.float().cpu().numpy()
    want = np.abs(x).max(axis=1) / np.float32(127)          # float32 quotient
    assert np.array_equal(s.cpu().numpy(), want)
    q = Q.cpu().numpy().astype(np.float64)
    exact = x.astype(np.float64) / want.astype(np.float64)[:, None]
    # the nearest whole number of the quotient rounded to float32
    assert np.abs(q - exact).max() <= 0.5 + 127.5 * U
    assert np.array_equal(q, np.rint(x / want[:, None]))
    assert np.abs(q).max(axis=1).min() == 127


def test_quantize_extreme_rows():
    X = torch.zeros(8, 32, device="cuda", dtype=F)
    X[1, 3], X[2, 5], X[3, 7] = float("inf"), float("nan"), -float("inf")
    X[4, 0], X[5, 0], X[6, 1] = 3e38, 1e-45, -1e-39
    X[7] = torch.linspace(-254, 254, 32)
    Q, s = forge.quantize_rows(X)
    assert s[0] == 0 and torch.all(Q[0] == 0)
    assert torch.all(torch.isnan(s[1:4])) and torch.all(Q[1:4] == 0)
    assert Q[4, 0] == 127 and Q[4, 1:].abs().max() == 0
    assert s[5] == 0 and Q[5].abs().max() == 0          # 1e-45 / 127 is below every float
    assert Q[6, 1] == -127
    assert Q[7, 0] == -127 and Q[7, -1] == 127
    Y = forge.linear_q8(Q, s, codes(gen(1), 16, 32), scales(gen(2), 16))
    assert torch.all(Y[0] == 0) and torch.all(torch.isnan(Y[1:4])) and torch.isfinite(Y[4:]).all()


def test_quantize_ties_and_pitch():
    # scale 1 exactly: halves go to the even code
    row = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5] + [0.0] * 8, device="cuda")
    big = torch.full((3, 32), float("nan"), device="cuda")
    big[:, :16] = row
    Q, s = forge.quantize_rows(big[:, :16])
    assert torch.all(s == 1.0)
    assert Q[1].tolist()[:8] == [127, 0, 2, 2, 0, -2, 126, -126]


# ---- products ------------------------------------------------------------------------------------------------
SIZES = [(1, 16, 8), (1, 4096, 264), (3, 80, 40), (7, 4096, 128), (33, 144, 1032), (130, 272, 520), (257, 96, 328),
         (511, 1008, 776), (1000, 256, 2056), (2049, 528, 1288), (2049, 272, 4104), (16, 64, 70008), (700, 2064, 2304)]


@pytest.mark.parametrize("t,i,o", SIZES)
def test_linear_q8(t, i, o):
    g = gen(t * 7 + i + o)
    X, W, sx, sw = codes(g, t, i), codes(g, o, i), scales(g, t), scales(g, o)
    b, R = rnd(g, o), rnd(g, t, o)
    act = forge.ACTS[(t + o) % 5]
    close(f"Y {act}", forge.linear_q8(X, sx, W, sw, bias=b, act=act, residual=R), *linear_q8_64(X, sx, W, sw, b, act, R))
    close("plain", forge.linear_q8(X, sx, W, sw), *linear_q8_64(X, sx, W, sw))
    close("float32 bias", forge.linear_q8(X, sx, W, sw, bias=b.float()), *linear_q8_64(X, sx, W, sw, b))


@pytest.mark.parametrize("t,i,o", SIZES)
def test_gated_q8(t, i, o):
    g = gen(t * 5 + i + o)
    X, sx = codes(g, t, i), scales(g, t)
    Wg, Wu, sg, su = codes(g, o, i), codes(g, o, i), scales(g, o), scales(g, o)
    act = forge.ACTS[(t + o) % 5]
    close(f"H {act}", forge.gated_q8(X, sx, Wg, sg, Wu, su, act=act), *gated_q8_64(X, sx, Wg, sg, Wu, su, act))


def test_largest_sums_are_exact():
    """every code -128 (which quantisation does not make, but the type holds), the longest k: 2^14 (2^17 - 16) < 2^31"""
    i = 2 ** 17 - 16
    for t, o in ((1, 16), (300, 264), (40, 520)):
        X = torch.full((t, i), -128, device="cuda", dtype=torch.int8)
        W = torch.full((o, i), -128, device="cuda", dtype=torch.int8)
        W[1::2] = 127
        one = torch.ones(max(t, o), device="cuda")
        Y = forge.linear_q8(X, one[:t], W, one[:o] * 2.0 ** -20)
        assert torch.all(Y[:, 0::2] == float(torch.tensor(i * 2.0 ** 14 * 2.0 ** -20).to(BF)))
        assert torch.all(Y[:, 1::2] == float(torch.tensor(-i * 128.0 * 127.0 * 2.0 ** -20).to(BF)))


def test_no_inner_dimension():
    for t in (2, 300):
        X, W = codes(gen(1), t, 0), codes(gen(1), 264, 0)
        sx, sw, b, R = scales(gen(2), t), scales(gen(2), 264), rnd(gen(3), 264), rnd(gen(4), t, 264)
        close("act(bias) + residual", forge.linear_q8(X, sx, W, sw, bias=b, act="silu", residual=R),
              *linear_q8_64(X, sx, W, sw, b, "silu", R))
        assert torch.all(forge.gated_q8(X, sx, W, sw, W, sw) == 0)
        off = torch.tensor([0, t - 1], device="cuda")
        assert torch.all(forge.expert_linear_q8(X, sx, W[None], sw, off)[:t - 1] == 0)


def test_pitched_rows():
    g = gen(3)
    for t in (1, 5, 300):
        X, W = codes(g, t, 272), codes(g, 392, 272)
        sx, sw, R = scales(g, t), scales(g, 392), rnd(g, t, 392)
        bx, bw = codes(g, t, 304), codes(g, 392, 288)
        bx[:, :272], bw[:, :272] = X, W
        out = torch.full((t, 400), 7.0, device="cuda", dtype=BF)
        forge.linear_q8(bx[:, :272], sx, bw[:, :272], sw, act="silu", residual=R, out=out[:, :392])
        assert torch.equal(out[:, :392], forge.linear_q8(X, sx, W, sw, act="silu", residual=R))
        assert torch.all(out[:, 392:] == 7.0)


GROUPS = [([1], 16, 8), ([0, 1, 0], 512, 264), ([2, 0, 3], 80, 40), ([7, 0, 0, 9], 4096, 128), ([33, 1], 144, 1032),
          ([0, 130, 0, 64, 65, 1], 272, 520), ([257, 40, 0, 300], 96, 328), ([511, 513, 1], 1008, 776),
          ([20] * 70, 128, 136), ([2500, 1, 0, 900, 1800], 192, 2600), ([1100, 1500, 700, 1290], 128, 4360), ([900, 10, 1300, 700], 528, 1288)]


@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_by_expert(case):
    sizes, i, o = GROUPS[case]
    e, g = len(sizes), gen(case)
    first = 2 if case % 2 else 0
    off = torch.tensor([first] + sizes, device="cuda").cumsum(0)
    n, R = int(off[-1]), int(off[-1]) + 3
    X, sx = codes(g, R, i), scales(g, R)
    sx[:first], sx[n:] = float("nan"), float("nan")
    Wg, Wu, sg, su = codes(g, e, o, i), codes(g, e, o, i), scales(g, e, o), scales(g, e, o)
    act = forge.ACTS[case % 5]
    out = torch.full((R, o), 7.0, device="cuda", dtype=BF)
    forge.expert_linear_q8(X, sx, Wg, sg, off, act=act, out=out)
    loc = off - first
    close(f"linear {act}", out[first:n],
          *grouped(loc, lambda a, x, s: linear_q8_64(x, s, Wg[a], sg[a], None, act), X[first:n], sx[first:n]))
    assert torch.all(out[:first] == 7.0) and torch.all(out[n:] == 7.0)
    wide = torch.full((R, o), 7.0, device="cuda")
    forge.expert_linear_q8(X, sx, Wg, sg, off, out=wide)
    close("float32 sums", wide[first:n],
          *grouped(loc, lambda a, x, s: linear_q8_64(x, s, Wg[a], sg[a]), X[first:n], sx[first:n]))
    assert torch.all(wide[:first] == 7.0) and torch.all(wide[n:] == 7.0)
    out.fill_(7.0)
    forge.expert_gated_q8(X, sx, Wg, sg, Wu, su, off, act=act, out=out)
    close(f"gated {act}", out[first:n],
          *grouped(loc, lambda a, x, s: gated_q8_64(x, s, Wg[a], sg[a], Wu[a], su[a], act), X[first:n], sx[first:n]))
    assert torch.all(out[:first] == 7.0) and torch.all(out[n:] == 7.0)


def test_a_served_block_of_experts():
    """the operators as a program runs them: quantised once per token, to the experts, through both layers, back"""
    g = gen(30)
    t, k, e, d, h = 33, 2, 4, 128, 192
    X = rnd(g, t, d)
    idx = torch.randint(0, e, (t, k), device="cuda", generator=g)
    w = torch.rand(t, k, device="cuda", generator=g)
    stack = [rnd(g, e, a, b, std=b ** -0.5) for a, b in ((h, d), (h, d), (d, h))]
    q = [forge.quantize_rows(W.reshape(-1, W.shape[2])) for W in stack]
    (qg, sg), (qu, su), (qd, sd) = [(c.view(W.shape), s) for (c, s), W in zip(q, stack)]
    offsets, pos = forge.expert_plan(idx, e)
    Q, s = forge.quantize_rows(X)
    Qp, sp = forge.expert_dispatch(Q, pos, scale=s)
    H = forge.expert_gated_q8(Qp, sp, qg, sg, qu, su, offsets)
    Hq, hs = forge.quantize_rows(H)
    Y = forge.expert_combine(forge.expert_linear_q8(Hq, hs, qd, sd, offsets), pos, w, residual=X)
    # against the same layers unquantised: a code is off by half at most, |x| / 254 of the row's largest, independent
    # from element to element; the block's relative error is the three roundings' together, some hundredths
    want = X.double().clone()
    for a, lo, hi in spans(offsets):
        rows = torch.nonzero((pos >= lo) & (pos < hi))
        x = X[rows[:, 0]].double()
        hid = torch.nn.functional.silu(x @ stack[0][a].double().t()) * (x @ stack[1][a].double().t())
        want.index_add_(0, rows[:, 0], (hid @ stack[2][a].double().t()) * w[rows[:, 0], rows[:, 1]].double()[:, None])
    assert float((Y.double() - want).norm() / want.norm()) < 0.02
