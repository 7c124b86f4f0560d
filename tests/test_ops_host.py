"""Host checks of the operators around the fused step, on the CPU: every refusal the C ABI
documents is returned before anything is enqueued (the descriptors hold made-up addresses),
workspace sizes, and the Python layer's own argument checks."""
import ctypes

import pytest
import torch

import optimizer_gemm_amd as forge
from optimizer_gemm_amd.forge import BF16, E4M3, F32, ForgeTensor

NULL, SHAPE, DTYPE, ALIGN, UNSUP, HYPER, ALIAS, SCRATCH = -1, -2, -3, -4, -5, -6, -8, -9
L = forge.lib()
BASE = 1 << 32


def ten(k, rows, cols, dt=BF16, ld=None, off=0):
    """descriptor number k, far from the others'"""
    return ForgeTensor(BASE + (k << 33) + off, dt, 0, rows, cols, cols if ld is None else ld, None)


def ref(t):
    return ctypes.byref(t) if t is not None else None


def linear(X=None, W=None, bias=None, act=0, R=None, Y=None, Z=None):
    X = X or ten(0, 16, 64)
    W = W or ten(1, 32, 64)
    Y = Y or ten(2, 16, 32)
    return L.forge_linear_forward(ref(X), ref(W), ref(bias), act, ref(R), ref(Y), ref(Z), None)


def test_linear_refusals():
    assert L.forge_linear_forward(None, ref(ten(1, 32, 64)), None, 0, None, ref(ten(2, 16, 32)), None, None) == NULL
    assert linear(act=5) == UNSUP and linear(act=-1) == UNSUP
    assert linear(X=ten(0, 16, 72)) == SHAPE
    assert linear(Y=ten(2, 16, 40)) == SHAPE and linear(Y=ten(2, 8, 32)) == SHAPE
    assert linear(X=ten(0, 16, 64, F32)) == DTYPE
    assert linear(X=ten(0, 16, 64, E4M3), W=ten(1, 32, 64, E4M3)) == UNSUP
    assert linear(W=ten(1, 32, 64, 2)) == DTYPE
    assert linear(X=ten(0, 16, 64, ld=68)) == ALIGN and linear(X=ten(0, 16, 64, off=8)) == ALIGN
    assert linear(W=ten(1, 36, 64), Y=ten(2, 16, 36)) == ALIGN
    assert linear(X=ten(0, 16, 64, ld=56)) == SHAPE
    assert linear(bias=ten(3, 1, 40)) == SHAPE and linear(bias=ten(3, 2, 32)) == SHAPE
    assert linear(bias=ten(3, 1, 32, 2)) == DTYPE
    assert linear(R=ten(3, 16, 24)) == SHAPE and linear(R=ten(3, 16, 32, F32)) == DTYPE
    assert linear(Y=ten(0, 16, 32)) == ALIAS
    assert linear(R=ten(2, 16, 32)) == ALIAS
    assert linear(Z=ten(2, 16, 32, off=32)) == ALIAS
    assert linear(X=ten(0, 1 << 25, 64), Y=ten(2, 1 << 25, 32)) == UNSUP


def test_act_backward_refusals():
    dY, Z, dZ = ten(0, 4096, 64), ten(1, 4096, 64), ten(2, 4096, 64)
    need = L.forge_linear_act_backward_workspace(4096, 64)
    assert need > 0 and need % 16 == 0 and L.forge_linear_act_backward_workspace(1, 64) == 0

    def call(dY=dY, Z=Z, act=2, dZ=dZ, db=BASE + (5 << 33), ws=BASE + (6 << 33), n=need):
        return L.forge_linear_act_backward(ref(dY), ref(Z), act, ref(dZ), db, ws, n, None)

    assert call(act=9) == UNSUP
    assert call(Z=None) == NULL and call(dZ=None) == NULL and call(ws=None) == NULL
    assert call(n=need - 1) == SCRATCH
    assert call(ws=BASE + (6 << 33) + 4) == ALIGN and call(db=BASE + 4) == ALIGN
    assert call(Z=ten(1, 4096, 72)) == SHAPE
    assert call(dZ=ten(0, 4096, 64)) == ALIAS
    assert call(db=BASE + (6 << 33)) == ALIAS
    assert call(dY=ten(0, 4096, 64, E4M3)) == UNSUP


def test_gated_refusals():
    X, Wg, Wu, H = ten(0, 16, 64), ten(1, 32, 64), ten(2, 32, 64), ten(3, 16, 32)

    def call(X=X, Wg=Wg, Wu=Wu, act=2, H=H, G=None, U=None):
        return L.forge_gated_forward(ref(X), ref(Wg), ref(Wu), act, ref(H), ref(G), ref(U), None)

    assert call(G=ten(4, 16, 32)) == NULL and call(U=ten(4, 16, 32)) == NULL
    assert call(act=7) == UNSUP
    assert call(Wu=ten(2, 40, 64)) == SHAPE and call(Wu=ten(2, 32, 56)) == SHAPE
    assert call(G=ten(4, 16, 32), U=ten(5, 16, 40)) == SHAPE
    assert call(G=ten(4, 16, 32), U=ten(4, 16, 32)) == ALIAS
    assert call(H=ten(1, 16, 32)) == ALIAS
    assert call(Wu=ten(2, 32, 64, F32)) == DTYPE


def test_gated_backward_refusals():
    a = [ten(k, 16, 32) for k in range(6)]

    def call(**kw):
        t = dict(zip(("dH", "G", "U", "dG", "dU", "H"), a), **kw)
        return L.forge_gated_backward(ref(t["dH"]), ref(t["G"]), ref(t["U"]), 2, ref(t["dG"]), ref(t["dU"]), ref(t["H"]),
                                      None)

    assert call(G=None) == NULL and call(dU=None) == NULL and call(dH=None) == NULL
    assert call(U=ten(2, 16, 40)) == SHAPE
    assert call(dG=a[0]) == ALIAS and call(dU=a[1]) == ALIAS and call(H=a[3]) == ALIAS

    def fused(**kw):
        t = dict(zip(("G", "U", "dG", "dU", "H"), a[1:]), dY=ten(7, 16, 48), Wd=ten(8, 48, 32), **kw)
        t.update(kw)
        return L.forge_gated_dgrad(ref(t["dY"]), ref(t["Wd"]), ref(t["G"]), ref(t["U"]), 2, ref(t["dG"]), ref(t["dU"]),
                                   ref(t["H"]), None)

    assert L.forge_gated_dgrad(ref(ten(7, 16, 48)), None, ref(a[1]), ref(a[2]), 2, ref(a[3]), ref(a[4]), None,
                               None) == NULL
    assert fused(G=ten(1, 16, 40)) == SHAPE
    assert fused(dG=ten(8, 16, 32)) == ALIAS and fused(H=ten(7, 16, 32)) == ALIAS


def test_dgrad_group_refusals():
    def call(n, dys, ws, dx):
        A = ForgeTensor * max(1, len(dys))
        return L.forge_linear_dgrad_group(n, A(*dys), A(*ws), ref(dx), None)

    dY, W, dX = ten(0, 16, 32), ten(1, 32, 64), ten(2, 16, 64)
    assert call(0, [dY], [W], dX) == SHAPE and call(5, [dY], [W], dX) == SHAPE
    assert call(1, [ten(0, 8, 32)], [W], dX) == SHAPE
    assert call(2, [dY, ten(3, 16, 40)], [W, ten(4, 48, 64)], dX) == SHAPE
    assert call(2, [dY, ten(3, 16, 40)], [W, ten(4, 40, 72)], dX) == SHAPE
    assert call(2, [dY, ten(3, 16, 40, F32)], [W, ten(4, 40, 64)], dX) == DTYPE
    assert call(1, [dY], [W], ten(1, 16, 64)) == ALIAS


def test_xent_refusals():
    T, D, V = 32, 64, 1001
    X, W = ten(0, T, D), ten(1, V, D)
    tgt, lse, tot, ws = (BASE + (k << 33) for k in (4, 5, 6, 7))
    need = L.forge_linear_xent_workspace(T, D, V, BF16, 0, 0)

    def fwd(X=X, W=W, tgt=tgt, loss=None, lse=lse, tot=tot, ws=ws, n=need):
        return L.forge_linear_xent_forward(ref(X), ref(W), tgt, -100, loss, lse, tot, ws, n, None)

    assert fwd(X=None) == NULL and fwd(W=None) == NULL and fwd(tgt=None) == NULL and fwd(lse=None) == NULL
    assert fwd(tot=None) == NULL and fwd(ws=None) == NULL
    assert fwd(n=need - 1) == SCRATCH and fwd(ws=ws + 8) == ALIGN and fwd(tgt=tgt + 4) == ALIGN
    assert fwd(X=ten(0, T, 72)) == SHAPE and fwd(W=ten(1, 0, D)) == SHAPE
    assert fwd(X=ten(0, T, D, F32)) == DTYPE and fwd(X=ten(0, T, D, E4M3)) == UNSUP
    assert fwd(lse=ws) == ALIAS and fwd(loss=lse) == ALIAS and fwd(tot=tgt) == ALIAS

    dX, dW = ten(2, T, D), ten(3, V, D)
    need_b = L.forge_linear_xent_workspace(T, D, V, BF16, 1, 0)
    dl = BASE + (8 << 33)

    def bwd(X=X, W=W, lse=lse, dl=dl, per=0, tot=tot, dX=dX, dW=dW, piece=0, ws=ws, n=need_b):
        return L.forge_linear_xent_backward(ref(X), ref(W), tgt, -100, lse, dl, per, tot, ref(dX), ref(dW), piece, ws, n,
                                            None)

    assert bwd(lse=None) == NULL and bwd(dl=None) == NULL and bwd(ws=None) == NULL
    assert bwd(n=need_b - 1) == SCRATCH
    assert bwd(piece=12) == SHAPE and bwd(piece=-8) == SHAPE
    assert bwd(dX=ten(2, T, 72)) == SHAPE and bwd(dW=ten(3, V - 1, D)) == SHAPE
    assert bwd(dX=ten(1, T, D)) == ALIAS and bwd(dW=ten(2, V, D)) == ALIAS and bwd(dl=ws) == ALIAS
    assert bwd(dW=ten(3, V, D, F32)) == DTYPE

    h = forge.make_hyper("adamw")
    m, v = ten(9, V, D, F32), ten(10, V, D, F32)

    def step(W=W, m=m, v=v, opt=0, n=need_b, t=1, dX=dX):
        return L.forge_linear_xent_step(ref(X), ref(W), ref(m), ref(v), opt, ctypes.byref(h), t, 0, tgt, -100, lse, dl, 0,
                                        tot, ref(dX), 0, ws, n, None)

    assert step(opt=8) == HYPER and step(t=0) == HYPER
    assert step(m=None) == NULL and step(m=ten(9, V, 72, F32)) == SHAPE and step(v=ten(10, V, D)) == DTYPE
    assert step(n=need_b - 1) == SCRATCH
    assert step(m=ten(1, V, D, F32)) == ALIAS and step(dX=ten(0, T, D)) == ALIAS
    assert step(W=ten(1, 1 << 24, D), m=ten(9, 1 << 24, D, F32), v=ten(10, 1 << 24, D, F32)) == UNSUP


def test_xent_workspace_sizes():
    """Grows with what it holds; a piece bounds the gradient's; nonsense is 0."""
    f = L.forge_linear_xent_workspace
    assert f(-1, 64, 10, BF16, 0, 0) == 0 and f(4, 64, 0, BF16, 1, 0) == 0 and f(4, 64, 8, BF16, 1, -1) == 0
    t, d, v = 8192, 4096, 131072
    whole, small = f(t, d, v, BF16, 1, 0), f(t, d, v, BF16, 1, 1024)
    assert small == t * 1024 * 2 + t * d * 4
    assert whole <= (1 << 30) * 1.05 + t * d * 4 and whole > small
    # the forward pass holds pairs per block of the vocabulary, far below the logits
    assert f(t, d, v, BF16, 0, 0) < t * v * 2 / 10
    # dz of a piece stays below 2^31 bytes, whatever is asked for
    assert f(1 << 20, 64, 1 << 20, BF16, 1, 1 << 20) < (1 << 31) + (1 << 20) * 64 * 4 + 16


def test_python_checks():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="device tensors"):
        forge.linear(z(4, 64), z(32, 64))
    with pytest.raises(ValueError, match="unknown activation"):
        forge.linear(z(4, 64), z(32, 64), act="tanh")
    with pytest.raises(ValueError, match="unknown activation"):
        forge.gated(z(4, 64), z(32, 64), z(32, 64), act="swish")
    with pytest.raises(ValueError, match="needs Z"):
        forge.linear_act_backward(z(4, 64), act="relu")
    with pytest.raises(ValueError, match="1..4 layers"):
        forge.dgrad_group([], [])
    with pytest.raises(ValueError, match="1..4 layers"):
        forge.dgrad_group([z(4, 8)], [z(8, 8), z(8, 8)])
    with pytest.raises(ValueError, match="unknown reduction"):
        forge.linear_cross_entropy(z(4, 64), z(32, 64), torch.zeros(4, dtype=torch.int64), reduction="avg")
    with pytest.raises(ValueError, match="one device"):
        forge.linear(z(4, 64), torch.zeros(32, 64, dtype=torch.bfloat16, device="meta"))


def test_dgrad_group_split_refusals():
    A1 = ForgeTensor * 1
    T, rows, cols = 5, 8192, 64
    dY, W, dX, ws = ten(0, T, rows), ten(1, rows, cols), ten(2, T, cols), BASE + (3 << 33)
    need = L.forge_linear_dgrad_group_workspace(T, cols, rows, BF16)
    assert need > 0 and need % (T * cols * 4) == 0
    assert L.forge_linear_dgrad_group_workspace(8192, 4096, rows, BF16) == 0  # enough tiles
    assert L.forge_linear_dgrad_group_workspace(T, cols, 512, BF16) == 0      # a short sum
    assert L.forge_linear_dgrad_group_workspace(T, cols, rows, F32) == 0
    assert L.forge_linear_dgrad_group_workspace(-1, cols, rows, BF16) == 0

    def call(ws=ws, n=need, dX=dX):
        return L.forge_linear_dgrad_group_split(1, A1(dY), A1(W), ref(dX), ws, n, None)

    assert call(n=need - 1) == SCRATCH and call(ws=None) == NULL and call(ws=ws + 4) == ALIGN
    assert call(ws=BASE) == ALIAS and call(ws=BASE + (2 << 33)) == ALIAS and call(dX=ten(1, T, cols)) == ALIAS


def test_xent_backward_refuses_distant_rows():
    """Rows of W or dW 2^23 bytes apart or more."""
    T, D, V = 4, 64, 100
    tgt, lse, tot, ws, dl = (BASE + (k << 33) for k in (4, 5, 6, 7, 8))
    n = 1 << 40

    def bwd(W, dW):
        return L.forge_linear_xent_backward(ref(ten(0, T, D)), ref(W), tgt, -100, lse, dl, 0, tot, None, ref(dW), 0, ws, n,
                                            None)

    far = 1 << 22
    assert bwd(ten(1, V, D, ld=far), ten(3, V, D)) == UNSUP
    assert bwd(ten(1, V, D), ten(3, V, D, ld=far)) == UNSUP


def test_new_tensors_come_from_the_stream_that_writes_them(monkeypatch):
    """On a stream other than the current one a call allocates from that stream's pool (memory of
    the current stream's may be in use there), and notes the current one for the new tensor and
    the other one for the call's tensors."""
    import contextlib

    from optimizer_gemm_amd import forge as impl

    log, active = [], [11]

    class FakeStream:
        def __init__(self, raw):
            self.cuda_stream = raw

    class FakeTensor:
        device = torch.device("cuda", 0)

        def __init__(self, name):
            self.name = name

        def get_device(self):
            return 0

        def record_stream(self, s):
            log.append((self.name, s.cuda_stream))

    @contextlib.contextmanager
    def stream(s):
        active.append(s.cuda_stream)
        yield
        active.pop()

    def empty(shape, dtype, device):
        log.append(("new", "from", active[-1]))
        return FakeTensor("new")

    monkeypatch.setattr(impl.torch, "empty", empty)
    monkeypatch.setattr(impl.torch.cuda, "current_stream", lambda d=None: FakeStream(11))
    monkeypatch.setattr(impl.torch.cuda, "stream", stream)
    monkeypatch.setattr(impl.torch.cuda, "ExternalStream", lambda raw, device=None: FakeStream(raw))
    monkeypatch.setattr(impl.torch.cuda, "default_stream", lambda d=None: FakeStream(0))
    monkeypatch.setattr(impl, "_raw_stream", lambda d: 11)
    monkeypatch.setattr(impl, "_current_device", lambda: 0)
    for given, want in ((22, [("x", 22), ("new", "from", 22), ("new", 11)]),
                        (0, [("x", 0), ("new", "from", 0), ("new", 11)]),
                        (11, [("new", "from", 11)]), (None, [("new", "from", 11)])):
        log.clear()
        with impl._On(given, FakeTensor("x"), None) as on:
            on.empty((4,), torch.float32)
            assert on.stream == (11 if given is None else given)
        assert log == want, given
    # the calls that came before these operators
    log.clear()
    impl._empty((4,), torch.float32, torch.device("cuda", 0), 22)
    assert log == [("new", "from", 22), ("new", 11)]


def test_a_refused_step_leaves_the_step_counts(monkeypatch):
    """Layers whose step is refused count no step."""
    from types import SimpleNamespace

    from optimizer_gemm_amd import nn as fnn

    def refuse(*a, **kw):
        raise forge.ForgeError(-5, "refused")

    monkeypatch.setattr(fnn.forge, "wgrad_step", refuse)
    monkeypatch.setattr(fnn.forge, "wgrad_step_group", refuse)
    layers = [SimpleNamespace(fused=True, _step_count=4, timing=None, weight=torch.zeros(8, 8), m=None, v=None,
                              m_scale=None, v_scale=None, opt="sgd", hyper=None, seed=0, code="linear") for _ in range(2)]
    for some in (layers, layers[:1]):
        with pytest.raises(forge.ForgeError):
            fnn._update(some, None, [None] * len(some), group=len(some) > 1)
        assert [L._step_count for L in layers] == [4, 4]


def test_without_torch_s_short_ways_to_the_stream():
    """A torch without the two private functions: the public ones serve."""
    import os
    import subprocess
    import sys

    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from optimizer_gemm_amd import forge
class S: cuda_stream = 77
torch.cuda.current_stream = lambda index=None: S
torch.cuda.current_device = lambda: 3
assert forge._raw_stream(0) == 77 and forge._current_device() == 3
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_xent_refuses_more_logits_than_the_memory_holds_partial_results_of():
    T, V, D = 1 << 21, 1 << 21, 64
    tgt, lse, tot, ws, dl = (BASE + (k << 33) for k in (4, 5, 6, 7, 8))
    n = 1 << 60
    for dt in (BF16, F32):
        X, W, few = ten(0, T, D, dt), ten(1, V, D, dt), ten(0, T - 1, D, dt)
        for back in (0, 1):
            assert L.forge_linear_xent_workspace(T, D, V, dt, back, 0) == 0
            assert L.forge_linear_xent_workspace(T - 1, D, V, dt, back, 0) > 0
        assert L.forge_linear_xent_forward(ref(X), ref(W), tgt, -100, None, lse, tot, ws, n, None) == UNSUP
        assert L.forge_linear_xent_backward(ref(X), ref(W), tgt, -100, lse, dl, 0, tot, ref(ten(2, T, D, dt)), None, 0, ws,
                                            n, None) == UNSUP
        # one row less: the next check answers
        assert L.forge_linear_xent_forward(ref(few), ref(W), tgt, -100, None, lse, tot, ws, 0, None) == SCRATCH


def test_modules_refuse_rows_in_another_order():
    """A residual or targets whose leading dimensions hold as many rows in another order, and rows of
    another length, are refused; a flat list of rows and dimensions of 1 are the same rows."""
    from optimizer_gemm_amd.nn import ForgeHead, ForgeLinear, linear_cross_entropy

    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    y = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731
    layer, head, w = ForgeLinear(16, 24, act="silu"), ForgeHead(16, 40), z(40, 16)
    for x, r in ((z(2, 3, 16), z(3, 2, 24)), (z(2, 3, 16), z(6, 4, 24)), (z(6, 16), z(5, 24)), (z(2, 3, 16), z(24))):
        with pytest.raises(ValueError, match="leading shape"):
            layer(x, r)
    for x, r in ((z(6, 16), z(3, 48)), (z(3, 32), z(6, 24)), (z(2, 3, 16), z(2, 3, 1, 12))):
        with pytest.raises(ValueError, match="elements wanted"):
            layer(x, r)
    for x, t in ((z(2, 3, 16), y(3, 2)), (z(2, 3, 16), y(5)), (z(6, 16), y(2, 2))):
        for f in (head, lambda a, b: linear_cross_entropy(a, w, b)):
            with pytest.raises(ValueError, match="leading shape"):
                f(x, t)
    with pytest.raises(ValueError, match="elements wanted"):
        linear_cross_entropy(z(3, 32), w, y(6))
    # these get as far as the kernels, which take no CPU tensors
    for x, r in ((z(2, 3, 16), z(2, 3, 24)), (z(2, 3, 16), z(6, 24)), (z(6, 16), z(2, 3, 24)), (z(2, 1, 3, 16), z(2, 3, 24))):
        with pytest.raises(ValueError, match="device tensors"):
            layer(x, r)
    for x, t in ((z(2, 3, 16), y(2, 3)), (z(2, 3, 16), y(6)), (z(6, 16), y(2, 3)), (z(1, 6, 16), y(6, 1))):
        with pytest.raises(ValueError, match="device tensors"):
            head(x, t)
