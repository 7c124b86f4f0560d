"""GPU parity of the products by expert on their large tiles, which small sizes never take: 256x256 tiles in several rounds
of the chip, a last round in quarters, of more than 64 experts too, with rows that belong to none around them, in bfloat16
and 8 bits; and the stack's gradient and step on large tiles in several rounds, sorted by rows or not. Which tiles a case has
is asserted, so that another choice of tiles cannot leave these kernels untested. Tolerances are derived in tests/_ops64.py
and tests/_experts64.py."""
import pytest
import torch

import optimizer_gemm_amd as forge
from _experts64 import (expert_dgrad64, expert_gated64, expert_gated_dgrad64, expert_linear64, expert_wgrad64, gated_q8_64,
                        grouped, linear_q8_64)
from _ops64 import U, close, gated64, gated_back64, mm64

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NAN = float("nan")
LINEAR, SUMS, GATED, GATED_DGRAD, DGRAD, WGRAD = range(6)
FIRST, BEHIND = 3, 5  # rows in front of the first expert's, behind the last one's


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F) * std).to(dtype)


def offsets_of(sizes):
    return torch.tensor([FIRST] + list(sizes), device="cuda").cumsum(0)


def units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def rounds(product, sizes, cols, k, dtype):
    """(whole rounds of 256x256 tiles, tiles of the last one, whether it runs as quarters) of a product that takes them"""
    rows = FIRST + sum(sizes) + BEHIND
    assert forge.lib().forge_expert_tile(product, rows, cols, k, len(sizes), dtype) == 256
    if product == DGRAD:
        assert forge.lib().forge_expert_dgrad_group_workspace(rows, cols, k, len(sizes), dtype) == 0
    tiles = -(-(2 * cols if product == GATED else cols) // 256) * sum(-(-n // 256) for n in sizes)
    full, rem = divmod(tiles, units())
    return full, rem, full > 0 and 0 < 2 * rem <= units()


def edged(g, sizes, cols, make=rnd, **kw):
    """rows of the experts, NaN around them"""
    t = make(g, FIRST + sum(sizes) + BEHIND, cols, **kw)
    t[:FIRST], t[FIRST + sum(sizes):] = NAN, NAN
    return t


def filled(sizes, cols, dtype=BF):
    return torch.full((FIRST + sum(sizes) + BEHIND, cols + 8), 7.0, device="cuda", dtype=dtype)


def inner(out, sizes, cols):
    """the experts' rows of a pitched result around which nothing was written"""
    n = FIRST + sum(sizes)
    assert torch.all(out[:FIRST] == 7.0) and torch.all(out[n:] == 7.0) and torch.all(out[:, cols:] == 7.0)
    return out[FIRST:n, :cols]


UNEVEN, MANY = [700, 1500, 0, 700, 1290], [300] * 69 + [10]
# product, rows of each expert, columns, k, whether the last round runs as quarters
CASES = [(LINEAR, UNEVEN, 4360, 4096, True), (LINEAR, MANY, 2048, 2048, True), (LINEAR, [2000, 1500, 1, 700, 1290], 5000, 4096, False),
         (LINEAR, [3000, 1500, 700, 1290], 8200, 2048, True),
         (SUMS, UNEVEN, 4360, 4096, True), (SUMS, MANY, 2048, 2048, True), (SUMS, [2000, 1500, 1, 700, 1290], 5000, 4096, False),
         (GATED, UNEVEN, 4360, 4096, True), (GATED, [1100, 1500, 0, 700, 1290], 2184, 4096, True),
         (GATED, [2000, 1500, 1, 700, 1290], 5000, 4096, False),
         (GATED_DGRAD, UNEVEN, 4360, 4096, True), (GATED_DGRAD, MANY, 2048, 2048, True),
         (GATED_DGRAD, [2000, 1500, 1, 700, 1290], 5000, 2048, False),
         (DGRAD, UNEVEN, 4360, 4096, True), (DGRAD, MANY, 2048, 2048, True), (DGRAD, [2000, 1500, 1, 700, 1290], 5000, 4096, False)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_products_on_large_tiles(case):
    product, sizes, cols, k, quarters = CASES[case]
    full, rem, tail = rounds(product, sizes, cols, k, forge.forge.BF16)
    print(f"{full} rounds and {rem} tiles, quarters: {tail}")
    assert full >= 1 and rem > 0 and tail == quarters
    e, g, off = len(sizes), gen(case), offsets_of(sizes)
    loc, act = off - FIRST, forge.ACTS[case % 5]
    used = slice(FIRST, FIRST + sum(sizes))
    if product in (LINEAR, SUMS):
        X, W = edged(g, sizes, k), rnd(g, e, cols, k, std=k ** -0.5)
        act = "none" if product == SUMS else act
        out = filled(sizes, cols, F if product == SUMS else BF)
        forge.expert_linear(X, W, off, act=act, out=out[:, :cols])
        close(act, inner(out, sizes, cols), *expert_linear64(X[used], W, loc, act)[:2])
        if product == LINEAR:
            Y, Z = forge.expert_linear(X, W, off, act=act, save=True)
            assert torch.equal(Y[used], out[used, :cols])
            close("Z", Z[used], *expert_linear64(X[used], W, loc, "none")[:2])
    elif product == GATED:
        X, Wg, Wu = edged(g, sizes, k), rnd(g, e, cols, k, std=k ** -0.5), rnd(g, e, cols, k, std=k ** -0.5)
        out = filled(sizes, cols)
        forge.expert_gated(X, Wg, Wu, off, act=act, out=out[:, :cols])
        h, dh, gt, dg, u, du = expert_gated64(X[used], Wg, Wu, loc, act)
        close(f"H {act}", inner(out, sizes, cols), h, dh)
        H, G, U = forge.expert_gated(X, Wg, Wu, off, act=act, save=True)
        assert torch.equal(H[used], out[used, :cols])
        close("G", G[used], gt, dg)
        close("U", U[used], u, du)
    elif product == GATED_DGRAD:
        dY, Wd = edged(g, sizes, k), rnd(g, e, k, cols, std=k ** -0.5)
        G, U = edged(g, sizes, cols), edged(g, sizes, cols)
        got = forge.expert_gated_dgrad(dY, Wd, G, U, off, act=act)
        want = expert_gated_dgrad64(dY[used], Wd, G[used], U[used], loc, act)
        for name, a, b in zip(("dG", "dU", "H"), got, (want[:2], want[2:4], want[4:])):
            close(f"{name} {act}", a[used], *b)
    else:
        outs = [1536, k - 1536]  # two layers, whose sums run into one
        D, W = [edged(g, sizes, o) for o in outs], [rnd(g, e, o, cols, std=k ** -0.5) for o in outs]
        out = filled(sizes, cols)
        forge.expert_dgrad_group(D, W, off, dX=out[:, :cols])
        close("dX", inner(out, sizes, cols), *expert_dgrad64([d[used] for d in D], W, loc))


CASES8 = [(LINEAR, [2100, 2600, 2100], 4360, 4112, True), (LINEAR, [900, 1, 2600, 300, 0, 2600], 2184, 4112, True),
          (LINEAR, [0, 129, 2600, 2100, 700, 2100], 5128, 4112, False),
          (SUMS, [2100, 2600, 2100], 4360, 4112, True), (SUMS, [0, 129, 2600, 2100, 700, 2100], 5128, 4112, False),
          (GATED, [3000, 300, 2000], 3336, 8192, True), (GATED, [1500, 2100, 2100, 1], 2568, 4112, True),
          (GATED, [300, 0, 300, 256, 2100, 700], 5128, 4112, False)]


@pytest.mark.parametrize("case", range(len(CASES8)))
def test_8_bit_products_on_large_tiles(case):
    """the factors differ from expert to expert by powers of two; those of rows of no expert are NaN"""
    product, sizes, cols, k, quarters = CASES8[case]
    full, rem, tail = rounds(product, sizes, cols, k, forge.forge.I8)
    print(f"{full} rounds and {rem} tiles, quarters: {tail}")
    assert full >= 1 and rem > 0 and tail == quarters
    e, g, off = len(sizes), gen(case), offsets_of(sizes)
    loc, act = off - FIRST, forge.ACTS[case % 5]
    used = slice(FIRST, FIRST + sum(sizes))
    R = FIRST + sum(sizes) + BEHIND

    def codes(*shape):
        return torch.randint(-127, 128, shape, device="cuda", generator=g).to(torch.int8)

    def factors():
        s = (torch.rand(e, cols, device="cuda", generator=g) + 0.5) * 1e-3
        return s * 2.0 ** -torch.arange(e, device="cuda", dtype=F)[:, None]

    X, sx = codes(R, k), (torch.rand(R, device="cuda", generator=g) + 0.5) * 1e-2
    sx[:FIRST], sx[used.stop:] = NAN, NAN
    W, sw = codes(e, cols, k), factors()
    out = filled(sizes, cols, F if product == SUMS else BF)
    if product == GATED:
        W2, s2 = codes(e, cols, k), factors()
        forge.expert_gated_q8(X, sx, W, sw, W2, s2, off, act=act, out=out[:, :cols])
        want = grouped(loc, lambda a, x, s: gated_q8_64(x, s, W[a], sw[a], W2[a], s2[a], act), X[used], sx[used])
    else:
        act = "none" if product == SUMS else act
        forge.expert_linear_q8(X, sx, W, sw, off, act=act, out=out[:, :cols])
        want = grouped(loc, lambda a, x, s: linear_q8_64(x, s, W[a], sw[a], None, act), X[used], sx[used])
    close(act, inner(out, sizes, cols), *want)


# ---- the stack's gradient and step -----------------------------------------------------------------------------
# rows of each expert, in, out, edge of the tiles, rounds of the chip (one large tile a unit, two small ones)
STACKS = [([700, 0, 33, 0, 1, 300, 129, 2000, 64], 1088, 1800, 256, 2), ([5, 0, 200] * 23 + [64], 320, 520, 256, 2),
          ([40, 64, 0, 300] * 4 + [1], 1088, 1800, 256, 3), ([30, 0, 200, 7] * 10, 128, 1920, 128, 2),
          ([3, 0, 70] * 200, 128, 128, 128, 2)]


def stack_case(case):
    sizes, i, o, edge, want = STACKS[case]
    e = len(sizes)
    assert forge.lib().forge_expert_tile(WGRAD, FIRST + sum(sizes) + BEHIND, i, o, e, forge.forge.BF16) == edge
    tiles, place = -(-i // edge) * -(-o // edge) * e, units() * (1 if edge == 256 else 2)
    assert -(-tiles // place) == want and tiles % place  # several rounds, the last one not full
    g, off = gen(case), offsets_of(sizes)

    # small whole numbers times powers of two: every sum of the gradient is exact in float32, in any order
    def whole(g, *shape):
        return torch.randint(-4, 5, shape, device="cuda", generator=g).to(BF)

    return g, off, edged(g, sizes, i, whole), edged(g, sizes, o, whole) * 2.0 ** -12, (e, o, i)


@pytest.mark.parametrize("case", range(len(STACKS)))
def test_gradient_in_several_rounds(case):
    g, off, X, dY, shape = stack_case(case)
    e, o, i = shape
    used = slice(FIRST, int(off[-1]))
    dW = torch.full((e, o, i + 4), 7.0, device="cuda")
    forge.expert_wgrad(X, dY, off, dW=dW[:, :, :i])
    want = expert_wgrad64(X[used], dY[used], off - FIRST)[0]
    assert torch.equal(dW[:, :, :i].double(), want) and torch.all(dW[:, :, i:] == 7.0)
    assert torch.equal(forge.expert_wgrad(X, dY, off), dW[:, :, :i])


def random_states(W, opt, fmt, g):
    m, v, ms, vs = forge.new_states(W, opt, fmt)
    for t, s in ((m, ms), (v, vs)):
        if t is None:
            continue
        if t.dtype in (torch.int8, torch.uint8):
            lo, hi = (-127, 128) if t.dtype == torch.int8 else (0, 256)
            t.copy_(torch.randint(lo, hi, t.shape, device="cuda", generator=g))
            s.copy_(torch.rand(s.shape, device="cuda", generator=g) * 1e-4)
        else:
            t.copy_(torch.rand(t.shape, device="cuda", generator=g) * 1e-3)
    return m, v, ms, vs


@pytest.mark.parametrize("fmt", ["f32", "bf16", "q8", "q8dyn"])
@pytest.mark.parametrize("case", range(len(STACKS)))
def test_step_in_several_rounds(case, fmt):
    """the same bits as the stand-alone optimizer pass over the stack as one layer on the exact gradient: every optimizer and
    rounding on the first case"""
    g, off, X, dY, shape = stack_case(case)
    e, o, i = shape
    code = "dynamic" if fmt == "q8dyn" else "linear"
    dW = expert_wgrad64(X[FIRST:int(off[-1])], dY[FIRST:int(off[-1])], off - FIRST)[0].float().view(e * o, i)
    for opt in forge.OPTIMIZERS if case == 0 else ("adamw", forge.OPTIMIZERS[case]):
        for sr in (0, 1):
            W = rnd(g, *shape, std=0.02)
            st = random_states(W, opt, fmt, g)
            W2, st2 = W.clone(), [None if t is None else t.clone() for t in st]
            forge.expert_wgrad_step(X, dY, W, st[0], st[1], off, opt, {"stochastic_round": sr}, 5, 99, st[2], st[3], code=code)
            flat = [None if t is None else t.view(e * o, -1) for t in (W2, *st2)]
            forge.optimizer_step(dW, flat[0], flat[1], flat[2], opt, {"stochastic_round": sr}, 5, 99, flat[3], flat[4], code=code)
            assert torch.equal(W, W2), (opt, sr)
            for a, b in zip(st, st2):
                assert a is None or torch.equal(a, b), (opt, sr)


# ---- stacks past 2^31 bytes --------------------------------------------------------------------------------------
@pytest.fixture
def emptied():
    yield
    torch.cuda.empty_cache()


def far_stack(g, e, o, i):
    """zeros but for the last expert's matrix, which begins past 2^31 bytes"""
    W = torch.zeros(e, o, i, device="cuda", dtype=BF)
    W[e - 1] = rnd(g, o, i, std=i ** -0.5)
    assert (e - 1) * o * i * 2 >= 2 ** 31
    return W


@pytest.mark.parametrize("rows", [[1, 2, 9], [0, 3, 70], [100, 300, 1100]])
def test_gated_block_past_two_gigabytes(rows, emptied):
    """the gated product and its backward pass: an expert of zeros, and the last one, for a few rows and for tiles"""
    e, h, d = 17, 8192, 8192
    g, n = gen(sum(rows)), sum(rows)
    off = torch.tensor([0] * 15 + [rows[0], rows[0] + rows[1], n], device="cuda")
    last = slice(rows[0] + rows[1], n)
    Wg, Wu = far_stack(g, e, h, d), far_stack(g, e, h, d)
    X = rnd(g, n, d)
    H, G, V = forge.expert_gated(X, Wg, Wu, off, act="silu", save=True)
    assert torch.all(H[:last.start] == 0) and torch.all(G[:last.start] == 0) and torch.all(V[:last.start] == 0)
    h64, dh, gt, dg, u, du = gated64(X[last], Wg[-1], Wu[-1], "silu")
    close("H", H[last], h64, dh)
    close("G", G[last], gt, dg)
    close("U", V[last], u, du)
    del Wu
    dY, G, V = rnd(g, n, h), rnd(g, n, d), rnd(g, n, d)  # (the first stack as the layer behind: [e, h, d])
    dG, dU, H = forge.expert_gated_dgrad(dY, Wg, G, V, off, act="gelu")
    assert torch.all(dG[:last.start] == 0) and torch.all(dU[:last.start] == 0)
    want = gated_back64(*mm64(dY[last], Wg[-1]), G[last], V[last], "gelu")
    for name, a, b in zip(("dG", "dU", "H"), (dG, dU, H), (want[:2], want[2:4], want[4:])):
        close(name, a[last], *b)


@pytest.mark.parametrize("rows", [[1, 2, 9], [100, 300, 1100]])
def test_8_bit_products_past_two_gigabytes(rows, emptied):
    e, o, i = 9, 16384, 16384
    g, n = gen(sum(rows)), sum(rows)
    off = torch.tensor([0] * 7 + [rows[0], rows[0] + rows[1], n], device="cuda")
    last = slice(rows[0] + rows[1], n)
    assert (e - 1) * o * i >= 2 ** 31

    def stack():
        W = torch.zeros(e, o, i, device="cuda", dtype=torch.int8)
        W[-1] = torch.randint(-127, 128, (o, i), device="cuda", generator=g).to(torch.int8)
        return W, (torch.rand(e, o, device="cuda", generator=g) + 0.5) * 1e-3

    X, sx = torch.randint(-127, 128, (n, i), device="cuda", generator=g).to(torch.int8), torch.rand(n, device="cuda", generator=g) * 1e-2
    (W, sw), (W2, s2) = stack(), stack()
    for dtype in (BF, F):
        Y = forge.expert_linear_q8(X, sx, W, sw, off, out_dtype=dtype)
        assert torch.all(Y[:last.start] == 0)
        close("linear", Y[last], *linear_q8_64(X[last], sx[last], W[-1], sw[-1]))
    H = forge.expert_gated_q8(X, sx, W, sw, W2, s2, off, act="silu")
    assert torch.all(H[:last.start] == 0)
    close("gated", H[last], *gated_q8_64(X[last], sx[last], W[-1], sw[-1], W2[-1], s2[-1], "silu"))


def far_gradient(g, e, o, i, dtype):
    """rows of the first and of the last expert, and the stack's gradient, which is exact in float32"""
    off = torch.tensor([0, 40] + [40] * (e - 2) + [107], device="cuda")
    X = torch.randint(-4, 5, (107, i), device="cuda", generator=g).to(dtype)
    dY = (torch.randint(-4, 5, (107, o), device="cuda", generator=g).to(F) * 2.0 ** -12).to(dtype)
    dW = torch.zeros(e, o, i, device="cuda")
    for x, r in ((0, slice(0, 40)), (e - 1, slice(40, 107))):
        dW[x] = (dY[r].double().t() @ X[r].double()).float()
    return off, X, dY, dW


@pytest.mark.parametrize("dtype", [BF, F])
def test_gradient_past_two_gigabytes(dtype, emptied):
    e, o, i = 9, 8192, 8192
    off, X, dY, want = far_gradient(gen(1), e, o, i, dtype)
    assert (e - 1) * o * i * 4 >= 2 ** 31
    dW = torch.full((e, o, i), NAN, device="cuda")
    forge.expert_wgrad(X, dY, off, dW=dW)
    assert torch.equal(dW, want)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "q8", "q8dyn"])
def test_step_past_two_gigabytes(fmt, emptied):
    """weights and moments of every format: the bits of the stand-alone optimizer pass over the stack as one layer"""
    e, o, i = 17, 8192, 16384
    g = gen(2)
    off, X, dY, dW = far_gradient(g, e, o, i, BF)
    assert (e - 1) * o * i >= 2 ** 31  # bytes of 8-bit moments, the smallest
    W = torch.empty(e, o, i, device="cuda", dtype=BF).normal_(0.0, 0.02, generator=g)
    code = "dynamic" if fmt == "q8dyn" else "linear"
    st = random_states(W, "adamw", fmt, g)
    W2, st2 = W.clone(), [None if t is None else t.clone() for t in st]
    forge.expert_wgrad_step(X, dY, W, st[0], st[1], off, "adamw", None, 5, 99, st[2], st[3], code=code)
    flat = [None if t is None else t.view(e * o, -1) for t in (W2, *st2)]
    forge.optimizer_step(dW.view(e * o, i), flat[0], flat[1], flat[2], "adamw", None, 5, 99, flat[3], flat[4], code=code)
    assert torch.equal(W, W2)
    for a, b in zip(st, st2):
        assert a is None or torch.equal(a, b)


def test_float32_step_past_two_gigabytes(emptied):
    e, o, i = 9, 4096, 16384
    g = gen(3)
    off, X, dY, dW = far_gradient(g, e, o, i, F)
    assert (e - 1) * o * i * 4 >= 2 ** 31
    W = rnd(g, e, o, i, dtype=F, std=0.02)
    st = random_states(W, "adamw", "f32", g)
    W2, st2 = W.clone(), [t if t is None else t.clone() for t in st]
    forge.expert_wgrad_step(X, dY, W, st[0], st[1], off, "adamw", None, 3, 1)
    flat = [None if t is None else t.view(e * o, -1) for t in (W2, *st2)]
    forge.optimizer_step(dW.view(e * o, i), flat[0], flat[1], flat[2], "adamw", None, 3, 1)
    for x in range(e):
        # both passes round each operation of the update on its own path: a step of float32 or two
        close("W", W[x], W2[x].double(), 8 * U * W2[x].double().abs() + 8 * U * 1e-3)
        for a, b in zip(st[:2], st2[:2]):
            close("moment", a[x], b[x].double(), 4 * U * b[x].double().abs() + 4 * U * 1e-6)
