"""Host checks of the layers of experts and of the 8-bit products, on the CPU: every refusal the C ABI documents is
returned before anything is enqueued (the descriptors hold made-up addresses), workspace sizes, and the Python layer's own
argument checks."""
import ctypes

import pytest
import torch

import optimizer_gemm_amd as forge
from optimizer_gemm_amd.forge import BF16, E4M3, F32, I8, ForgeTensor, make_hyper

NULL, SHAPE, DTYPE, ALIGN, UNSUP, HYPER, ALIAS, SCRATCH = -1, -2, -3, -4, -5, -6, -8, -9
L = forge.lib()
BASE = 1 << 40
OFF = BASE + (40 << 34)


def ten(k, rows, cols, dt=BF16, ld=None, off=0, scale=None):
    """descriptor number k, far from the others'"""
    return ForgeTensor(BASE + (k << 34) + off, dt, 0, rows, cols, cols if ld is None else ld, scale)


def q8(k, rows, cols, ld=None, scale=True, off=0):
    return ten(k, rows, cols, I8, ld, off, BASE + (k << 34) + (1 << 33) if scale is True else scale)


def ref(t):
    return ctypes.byref(t) if t is not None else None


def test_plan_refusals():
    idx, offs, pos, ws = BASE, BASE + (1 << 34), BASE + (2 << 34), BASE + (3 << 34)
    need = L.forge_expert_plan_workspace(5000, 2, 16)
    assert need == 10 * 16 * 4 and L.forge_expert_plan_workspace(512, 2, 16) == 0
    assert L.forge_expert_plan_workspace(0, 2, 16) == 0 and L.forge_expert_plan_workspace(5000, 2, 0) == 0
    assert L.forge_expert_plan_workspace(1 << 20, 8, 1024) <= 512 * 1024 * 4  # the blocks grow, not their number

    def call(idx=idx, T=5000, k=2, e=16, offs=offs, pos=pos, ws=ws, n=need):
        return L.forge_expert_plan(idx, T, k, e, offs, pos, ws, n, None)

    assert call(e=0) == SHAPE and call(e=1025) == SHAPE and call(T=-1) == SHAPE and call(k=0) == SHAPE
    assert call(idx=None) == NULL and call(offs=None) == NULL and call(pos=None) == NULL and call(ws=None) == NULL
    assert call(idx=idx + 4) == ALIGN and call(offs=offs + 4) == ALIGN and call(pos=pos + 2) == ALIGN and call(ws=ws + 8) == ALIGN
    assert call(n=need - 1) == SCRATCH
    assert call(T=1 << 30) == UNSUP and call(T=1 << 25, k=32) == UNSUP and call(T=1 << 29, k=1 << 29) == UNSUP
    assert call(pos=idx + 8) == ALIAS and call(offs=idx) == ALIAS and call(ws=pos) == ALIAS


def test_dispatch_refusals():
    def call(X=None, pos=BASE + (9 << 34), k=2, Y=None):
        return L.forge_expert_dispatch(ref(X or ten(0, 16, 64)), pos, k, ref(Y or ten(1, 32, 64)), None)

    assert L.forge_expert_dispatch(None, BASE, 2, ref(ten(1, 32, 64)), None) == NULL
    assert call(pos=None) == NULL and call(pos=BASE + 2) == ALIGN and call(k=0) == SHAPE
    assert call(Y=ten(1, 32, 72)) == SHAPE and call(Y=ten(1, 32, 64, F32)) == DTYPE and call(X=ten(0, 16, 64, E4M3)) == UNSUP
    assert call(X=ten(0, 16, 60)) == ALIGN and call(X=ten(0, 16, 64, 3)) == DTYPE
    assert call(Y=ten(0, 32, 64, off=64)) == ALIAS and call(pos=BASE + (1 << 34)) == ALIAS
    assert call(X=ten(0, 1 << 26, 8), Y=ten(1, 16, 8)) == UNSUP
    assert call(X=q8(0, 16, 64)) == DTYPE
    assert call(X=q8(0, 16, 64), Y=q8(1, 32, 64, scale=None)) == NULL
    assert call(X=q8(0, 16, 72), Y=q8(1, 32, 72)) == ALIGN
    assert call(X=q8(0, 16, 64), Y=q8(1, 32, 64, scale=BASE + (1 << 33))) == ALIAS


def test_combine_refusals():
    P, W = BASE + (9 << 34), BASE + (10 << 34)

    def call(Yp=None, pos=P, k=2, w=W, R=None, Y=None):
        return L.forge_expert_combine(ref(Yp or ten(0, 32, 64)), pos, k, w, ref(R), ref(Y or ten(1, 16, 64)), None)

    assert call(pos=None) == NULL and call(pos=P + 1) == ALIGN and call(w=W + 2) == ALIGN and call(k=0) == SHAPE
    assert call(Yp=ten(0, 32, 72)) == SHAPE and call(R=ten(2, 16, 72)) == SHAPE and call(R=ten(2, 15, 64)) == SHAPE
    assert call(Yp=ten(0, 32, 64), Y=ten(1, 16, 64, F32)) == DTYPE and call(R=ten(2, 16, 64, F32)) == DTYPE
    assert call(Y=ten(0, 16, 64)) == ALIAS and call(R=ten(1, 16, 64)) == ALIAS and call(w=BASE + (1 << 34)) == ALIAS

    def back(dY=None, Yp=0, pos=P, k=2, w=W, dYp=0, dw=BASE + (11 << 34)):
        Yp = ten(0, 32, 64) if Yp == 0 else Yp
        dYp = ten(3, 32, 64) if dYp == 0 else dYp
        return L.forge_expert_combine_backward(ref(dY or ten(1, 16, 64)), ref(Yp), pos, k, w, ref(dYp), dw, None)

    assert back(Yp=None) == NULL and back(pos=None) == NULL
    assert back(dYp=ten(3, 31, 64)) == SHAPE and back(dYp=ten(3, 32, 72)) == SHAPE
    assert back(dw=BASE + (11 << 34) + 2) == ALIGN and back(dYp=ten(3, 32, 64, F32)) == DTYPE
    assert back(dYp=ten(1, 32, 64)) == ALIAS and back(dw=W) == ALIAS and back(dw=BASE + (3 << 34)) == ALIAS


def test_product_refusals():
    def lin(X=None, W=None, e=4, off=OFF, act=0, Y=None, Z=None):
        return L.forge_expert_linear(ref(X or ten(0, 16, 64)), ref(W or ten(1, 128, 64)), e, off, act,
                                     ref(Y or ten(2, 16, 32)), ref(Z), None)

    assert lin(e=0) == SHAPE and lin(e=1025) == SHAPE and lin(e=3) == SHAPE and lin(off=None) == NULL
    assert lin(off=OFF + 4) == ALIGN and lin(act=5) == UNSUP and lin(X=ten(0, 16, 72)) == SHAPE
    assert lin(X=ten(0, 16, 64, F32)) == DTYPE and lin(X=ten(0, 16, 64, E4M3), W=ten(1, 128, 64, E4M3)) == UNSUP
    assert lin(Y=ten(2, 16, 40)) == SHAPE and lin(Y=ten(2, 15, 32)) == SHAPE and lin(Z=ten(3, 16, 40)) == SHAPE
    assert lin(Y=ten(0, 16, 32)) == ALIAS and lin(Z=ten(2, 16, 32)) == ALIAS
    assert lin(off=BASE + (2 << 34)) == ALIAS
    assert lin(Y=ten(2, 16, 32, F32), act=1) == UNSUP and lin(Y=ten(2, 16, 32, F32), Z=ten(3, 16, 32)) == UNSUP
    # one expert's part past 2^31 bytes is refused, the whole stack's is not (here: refused for its alignment only)
    assert lin(X=ten(0, 16, 65536), W=ten(1, 4 * 16384, 65536)) == UNSUP
    assert lin(X=ten(0, 1 << 24, 64), Y=ten(2, 1 << 24, 32)) == UNSUP
    assert lin(W=ten(1, 144, 64), Y=ten(2, 16, 36)) == ALIGN

    def gat(Wu=None, G=None, U=None, H=None, e=4, off=OFF):
        return L.forge_expert_gated(ref(ten(0, 16, 64)), ref(ten(1, 128, 64)), ref(Wu or ten(2, 128, 64)), e, off, 2,
                                    ref(H or ten(3, 16, 32)), ref(G), ref(U), None)

    assert gat(G=ten(4, 16, 32)) == NULL and gat(Wu=ten(2, 132, 64)) == SHAPE and gat(Wu=ten(2, 128, 56)) == SHAPE
    assert gat(e=5) == SHAPE and gat(off=None) == NULL and gat(H=ten(1, 16, 32)) == ALIAS
    assert gat(G=ten(4, 16, 32), U=ten(4, 16, 32)) == ALIAS

    def gd(dY=None, Wd=None, G=None, dG=None, H=None, e=4, off=OFF):
        return L.forge_expert_gated_dgrad(ref(dY or ten(0, 16, 64)), ref(Wd or ten(1, 256, 32)), ref(G or ten(2, 16, 32)),
                                          ref(ten(3, 16, 32)), e, off, 2, ref(dG or ten(4, 16, 32)), ref(ten(5, 16, 32)), ref(H),
                                          None)

    assert gd(dY=ten(0, 16, 72)) == SHAPE and gd(G=ten(2, 16, 40)) == SHAPE and gd(e=0) == SHAPE and gd(off=None) == NULL
    assert gd(dG=ten(2, 16, 32)) == ALIAS and gd(H=ten(5, 16, 32)) == ALIAS and gd(Wd=ten(1, 256, 32, F32)) == DTYPE

    def dg(n=2, e=4, off=OFF, dX=None, W1=None):
        dy = (ForgeTensor * 2)(ten(0, 16, 32), ten(1, 16, 40))
        w = (ForgeTensor * 2)(ten(2, 128, 64), W1 or ten(3, 160, 64))
        return L.forge_expert_dgrad_group(n, dy, w, e, off, ref(dX or ten(4, 16, 64)), None)

    assert dg(n=0) == SHAPE and dg(n=5) == SHAPE and dg(e=3) == SHAPE and dg(off=None) == NULL
    assert dg(W1=ten(3, 160, 72)) == SHAPE and dg(dX=ten(4, 16, 72)) == SHAPE and dg(dX=ten(1, 16, 64)) == ALIAS


def test_dgrad_group_split_refusals():
    T, rows, cols, ws = 20, 8192, 64, BASE + (5 << 34)
    need = L.forge_expert_dgrad_group_workspace(T, cols, rows, 4, BF16)
    assert need > 0 and need % (T * cols * 4) == 0
    for a in ((16384, 4096, 28672, 8, BF16), (T, cols, 512, 4, BF16), (T, cols, rows, 4, F32), (0, cols, rows, 4, BF16),
              (T, 0, rows, 4, BF16), (T, cols, 0, 4, BF16), (T, cols, rows, 0, BF16), (T, cols, rows, 1025, BF16),
              (1 << 40, cols, rows, 4, BF16)):
        assert L.forge_expert_dgrad_group_workspace(*a) == 0
    dy, w = (ForgeTensor * 1)(ten(0, T, rows)), (ForgeTensor * 1)(ten(1, 4 * rows, cols))

    def call(ws=ws, n=need, dX=ten(2, T, cols), off=OFF):
        return L.forge_expert_dgrad_group_split(1, dy, w, 4, off, ref(dX), ws, n, None)

    assert call(n=need - 1) == SCRATCH and call(ws=None) == NULL and call(ws=ws + 4) == ALIGN
    assert call(ws=BASE) == ALIAS and call(ws=BASE + (2 << 34)) == ALIAS and call(dX=ten(1, T, cols)) == ALIAS
    assert call(ws=OFF & ~15) == ALIAS and call(off=None) == NULL


def test_step_refusals():
    h = make_hyper("adamw")

    def step(X=None, dY=None, W=None, m=None, v=None, e=4, off=OFF, opt=0, h=h, t=1):
        return L.forge_expert_wgrad_step(ref(X or ten(0, 16, 64)), ref(dY or ten(1, 16, 32)), ref(W or ten(2, 128, 64)),
                                         ref(m or ten(3, 128, 64, F32)), ref(v or ten(4, 128, 64, F32)), e, off, opt, ref(h), t,
                                         1, None)

    assert step(t=0) == HYPER and step(opt=8) == HYPER and step(e=0) == SHAPE and step(e=3) == SHAPE and step(off=None) == NULL
    assert step(X=ten(0, 15, 64)) == SHAPE and step(dY=ten(1, 16, 40)) == SHAPE and step(W=ten(2, 128, 72)) == SHAPE
    assert step(X=ten(0, 16, 64, E4M3)) == UNSUP and step(X=ten(0, 16, 64, F32)) == DTYPE and step(m=ten(3, 120, 64, F32)) == SHAPE
    assert step(m=ten(3, 128, 64, BF16)) == DTYPE                   # m and v in two formats
    assert step(m=ten(3, 128, 64, I8), v=ten(4, 128, 64, 3)) == NULL  # codes without scales
    assert step(v=ten(3, 128, 64, F32)) == ALIAS and step(m=ten(0, 128, 64, F32)) == ALIAS
    assert step(X=ten(0, 16, 8192), dY=ten(1, 16, 131072), W=ten(2, 4 * 131072, 8192), m=ten(3, 4 * 131072, 8192, F32),
                v=ten(4, 4 * 131072, 8192, F32)) == UNSUP           # 2^32 weights
    assert step(X=ten(0, 16, 8192), dY=ten(1, 16, 65536), W=ten(2, 4 * 65536, 8192), m=ten(3, 4 * 65536, 8192, F32),
                v=ten(4, 4 * 65536, 8192, F32)) == UNSUP            # an expert's moments past 2^31 bytes

    def wg(X=None, dY=None, e=4, off=OFF, dW=BASE + (5 << 34), ld=64):
        return L.forge_expert_wgrad(ref(X or ten(0, 16, 64)), ref(dY or ten(1, 16, 32)), e, off, dW, ld, None)

    assert wg(dW=None) == NULL and wg(off=None) == NULL and wg(e=0) == SHAPE and wg(ld=60) == SHAPE and wg(ld=66) == ALIGN
    assert wg(dW=BASE + 8) == ALIGN and wg(X=ten(0, 16, 64, E4M3)) == UNSUP and wg(dY=ten(1, 17, 32)) == SHAPE
    assert wg(dW=BASE) == ALIAS


def test_q8_refusals():
    def quant(X=None, Q=None):
        return L.forge_quantize_rows(ref(X or ten(0, 16, 64)), ref(Q or q8(1, 16, 64)), None)

    assert quant(X=ten(0, 16, 64, I8)) == DTYPE and quant(X=ten(0, 16, 64, E4M3)) == UNSUP and quant(Q=ten(1, 16, 64)) == DTYPE
    assert quant(Q=q8(1, 16, 64, scale=None)) == NULL and quant(Q=q8(1, 15, 64)) == SHAPE
    assert quant(X=ten(0, 16, 72), Q=q8(1, 16, 72)) == ALIGN and quant(Q=q8(1, 16, 64, ld=72)) == ALIGN
    assert quant(Q=q8(1, 16, 64, scale=BASE)) == ALIAS and quant(Q=q8(0, 16, 64)) == ALIAS
    assert quant(X=ten(0, 1 << 26, 16), Q=q8(1, 1 << 26, 16)) == UNSUP

    def lin(X=None, W=None, b=None, act=0, R=None, Y=None):
        return L.forge_linear_q8(ref(X or q8(0, 16, 64)), ref(W or q8(1, 32, 64)), ref(b), act, ref(R), ref(Y or ten(2, 16, 32)),
                                 None)

    assert lin(act=5) == UNSUP and lin(X=ten(0, 16, 64)) == DTYPE and lin(W=ten(1, 32, 64)) == DTYPE
    assert lin(X=q8(0, 16, 64, scale=None)) == NULL and lin(W=q8(1, 32, 64, scale=BASE + 4)) == ALIGN
    assert lin(X=q8(0, 16, 80)) == SHAPE and lin(Y=ten(2, 16, 40)) == SHAPE and lin(Y=ten(2, 16, 32, F32)) == DTYPE
    assert lin(X=q8(0, 16, 72), W=q8(1, 32, 72)) == ALIGN and lin(W=q8(1, 36, 64), Y=ten(2, 16, 36)) == ALIGN
    assert lin(b=ten(3, 1, 40)) == SHAPE and lin(R=ten(3, 16, 32, F32)) == DTYPE and lin(R=ten(2, 16, 32)) == ALIAS
    assert lin(X=q8(0, 16, 1 << 17), W=q8(1, 32, 1 << 17)) == UNSUP  # 32-bit sums
    assert lin(Y=ten(2, 16, 32, off=0), X=q8(0, 16, 64, scale=BASE + (2 << 34))) == ALIAS

    def gat(Wu=None, H=None):
        return L.forge_gated_q8(ref(q8(0, 16, 64)), ref(q8(1, 32, 64)), ref(Wu), 2, ref(H or ten(3, 16, 32)), None)

    assert gat() == NULL and gat(Wu=q8(2, 40, 64)) == SHAPE and gat(Wu=ten(2, 32, 64)) == DTYPE
    assert gat(Wu=q8(2, 32, 64), H=ten(2, 16, 32)) == ALIAS

    def ex(W=None, e=4, off=OFF, Y=None):
        return L.forge_expert_linear_q8(ref(q8(0, 16, 64)), ref(W or q8(1, 128, 64)), e, off, 0, ref(Y or ten(3, 16, 32)), None)

    assert ex(off=None) == NULL and ex(e=0) == SHAPE and ex(e=3) == SHAPE and ex(off=OFF + 4) == ALIGN
    assert ex(Y=ten(3, 16, 128)) == SHAPE and ex(Y=ten(3, 16, 32, 3)) == DTYPE
    assert L.forge_expert_gated_q8(ref(q8(0, 16, 64)), ref(q8(1, 128, 64)), None, 4, OFF, 0, ref(ten(3, 16, 32)), None) == NULL


def test_python_checks():
    i64 = torch.zeros(4, 2, dtype=torch.int64)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    X = torch.zeros(4, 16, dtype=torch.bfloat16)
    W = torch.zeros(3, 8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="int64"):
        forge.expert_plan(i64.int(), 4)
    with pytest.raises(ValueError, match="experts"):
        forge.expert_plan(i64, 1025)
    with pytest.raises(ValueError, match="one route"):
        forge.expert_plan(i64[:, :0].contiguous(), 4)
    with pytest.raises(ValueError, match="device tensors"):
        forge.expert_plan(i64, 4)
    with pytest.raises(ValueError, match="int32"):
        forge.expert_dispatch(X, i64)
    with pytest.raises(ValueError, match="factors"):
        forge.expert_dispatch(X, pos, scale=torch.zeros(4))
    with pytest.raises(ValueError, match="factors"):
        forge.expert_dispatch(X.to(torch.int8), pos)
    with pytest.raises(ValueError, match="float32 tensor of pos's shape"):
        forge.expert_combine(X, pos, torch.zeros(4, 3))
    with pytest.raises(ValueError, match="needs Yp"):
        forge.expert_combine_backward(X, None, pos)
    with pytest.raises(ValueError, match="unknown activation"):
        forge.expert_linear(X, W, torch.zeros(4, dtype=torch.int64), act="tanh")
    with pytest.raises(ValueError, match="a group holds"):
        forge.expert_dgrad_group([X], [W, W], torch.zeros(4, dtype=torch.int64))
    from optimizer_gemm_amd import forge as f
    with pytest.raises(ValueError, match="offsets"):
        f._experts(W, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="stacked"):
        f._experts(X, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="one pitch"):
        f._stack(torch.zeros(3, 10, 16)[:, :8])
    with pytest.raises(ValueError, match="contiguous"):
        f._stack(W.transpose(1, 2))
    # a stack of one row each: the pitch is the distance of the experts
    d = f._stack(torch.zeros(3, 4, 16)[:, :1])
    assert (d.rows, d.cols, d.ld) == (3, 16, 64)
    d = f._stack(torch.zeros(3, 8, 32)[:, :, :16])
    assert (d.rows, d.cols, d.ld) == (24, 16, 32)


def test_states_of_a_stack():
    W = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    m, v, ms, vs = forge.new_states(W, "adamw", "q8")
    assert m.shape == v.shape == W.shape and ms.shape == vs.shape == (3, 8, 2)
    m, v, ms, vs = forge.new_states(W[0], "lion", "bf16")
    assert m.shape == (8, 128) and m.dtype == torch.bfloat16 and v is None and ms is None
    with pytest.raises(ValueError):
        forge.new_states(W, "adamw", "fp4")


def test_calls_check_their_arguments():
    """the calls that take tensors as they are: counts, types, ranges and devices, and a status as an exception"""
    from optimizer_gemm_amd import forge as f
    c, t = f._calls, torch.zeros(4, 16)
    with pytest.raises(TypeError, match="takes 3 arguments"):
        c.forge_quantize_rows(t, t)
    with pytest.raises(TypeError):
        c.forge_expert_plan_workspace(1, 2, "x")
    with pytest.raises(ValueError, match="out of range"):
        c.forge_expert_plan_workspace(1, 2, 2 ** 31)
    with pytest.raises(OverflowError):
        c.forge_expert_plan_workspace(2 ** 64, 2, 1)
    with pytest.raises(ValueError, match="a tensor wanted"):
        c.forge_quantize_rows("x", None, 0)
    with pytest.raises(ValueError, match="one device"):
        c.forge_quantize_rows(t, (t.char(), t[:, 0]), 0)
    with pytest.raises(forge.ForgeError, match="forge_quantize_rows") as e:
        c.forge_quantize_rows(None, None, 0)
    assert e.value.status == -1
    with pytest.raises(forge.ForgeError) as e:
        c.forge_expert_plan(None, 4, 2, 0, None, None, None, 0, 0)
    assert e.value.status == -2
    assert c.forge_expert_plan_workspace(65536, 8, 64) == f.lib().forge_expert_plan_workspace(65536, 8, 64) > 0


def test_the_package_loads_without_the_python_calls(tmp_path):
    """forge_calls.so is built against one torch's C++ interface. Where it is missing, is no module or belongs to another
    torch, the package and every call that goes another way work; those that go through it say why they do not."""
    import os
    import subprocess
    import sys

    from optimizer_gemm_amd import forge as f

    pkg = os.path.dirname(f.__file__)
    assert f._calls.torch_version and torch.__version__.startswith(f._calls.torch_version)
    check = """
import sys, torch
if len(sys.argv) > 2:
    torch.__version__ = sys.argv[2]
import optimizer_gemm_amd as forge
from optimizer_gemm_amd import nn
from optimizer_gemm_amd import forge as f
assert f.__file__.startswith(sys.argv[1]), f.__file__
assert forge.lib().forge_version() > 0 and forge.step_scalars("adamw", None, 1) is not None
assert forge.lib().forge_expert_plan_workspace(512, 2, 16) == 0
assert nn.ForgeLinear(16, 16).step_count == 0
try:
    f._calls.forge_expert_plan_workspace(512, 2, 16)
except ImportError as e:
    assert "forge_expert_plan_workspace" in str(e) and "build.py" in str(e), e
    print("refused:", e)
"""
    for n, (calls, argv, why) in enumerate((("missing", (), "not built"), ("garbage", (), "does not load"),
                                            ("real", ("1.2.3+cpu",), "built against torch"), ("real", (), None))):
        root = tmp_path / str(n)
        (root / "optimizer_gemm_amd" / "_lib").mkdir(parents=True)
        for name in os.listdir(pkg):
            if name.endswith(".py"):
                os.symlink(os.path.join(pkg, name), root / "optimizer_gemm_amd" / name)
        os.symlink(f.LIB_PATH, root / "optimizer_gemm_amd" / "_lib" / "libforge.so")
        so = root / "optimizer_gemm_amd" / "_lib" / "forge_calls.so"
        if calls == "garbage":
            so.write_bytes(b"no module")
        elif calls == "real":
            os.symlink(os.path.join(pkg, "_lib", "forge_calls.so"), so)
        r = subprocess.run([sys.executable, "-B", "-c", check, str(root), *argv], cwd=root, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        assert (why in r.stdout) if why else (r.stdout == ""), r.stdout


def test_states_are_those_of_a_layer_or_a_stack():
    """no step takes moments of other dimensions, so none are made"""
    for shape in ((), (128,), (2, 3, 8, 128)):
        for fmt in ("f32", "bf16", "q8"):
            with pytest.raises(ValueError, match="stack"):
                forge.new_states(torch.zeros(shape, dtype=torch.bfloat16), "adamw", fmt)
    assert forge.new_states(torch.zeros(1, 128), "adamw")[0].shape == (1, 128)


def test_float32_rows_beside_bfloat16_hold_as_many_elements():
    """float32 results of bfloat16 or 8-bit operands, and the combination that reads them: refused from 2^30 elements on, as
    bfloat16 rows are, not from 2^31 bytes (the calls below that size overlap an input, so that nothing is launched)"""
    n, P, W = 1 << 20, BASE + (9 << 34), BASE + (10 << 34)

    def lin(rows, cols, q=False, ld=None):
        Y = ten(0, rows, cols, F32, ld)  # (where X is)
        if q:
            return L.forge_expert_linear_q8(ref(q8(0, rows, 16)), ref(q8(1, 4 * cols, 16)), 4, OFF, 0, ref(Y), None)
        return L.forge_expert_linear(ref(ten(0, rows, 16)), ref(ten(1, 4 * cols, 16)), 4, OFF, 0, ref(Y), None, None)

    def com(rows, cols, dt=BF16):
        return L.forge_expert_combine(ref(ten(0, rows, cols, F32)), P, 2, W, None, ref(ten(0, 16, cols, dt)), None)

    def back(rows, cols):
        return L.forge_expert_combine_backward(ref(ten(1, 16, cols)), ref(ten(0, rows, cols, F32)), P, 2, W,
                                               ref(ten(1, rows, cols)), BASE + (11 << 34), None)

    for q in (False, True):
        assert lin(n, 512, q) == lin(n, 1016, q) == ALIAS and lin(n, 1024, q) == UNSUP and lin(n, 512, q, 1024) == UNSUP
        assert lin(511, 512, q, 1 << 21) == UNSUP  # 256 rows of them past 2^31 bytes
    assert com(n, 512) == com(n, 1016) == ALIAS and com(n, 1024) == UNSUP and com(n, 512, F32) == UNSUP
    assert back(n, 512) == back(n, 1016) == ALIAS and back(n, 1024) == UNSUP


def test_new_tensors_check_their_arguments():
    from optimizer_gemm_amd import forge as f
    for bad in ((), (0,), (0, "float32", 3), (0, torch.float32, "x"), ("x", torch.float32, 3), (0, torch.float32, 1, 1, 1, 1, 1),
                (0, torch.float32, -1)):
        with pytest.raises((RuntimeError, TypeError, ValueError)):
            f._calls.empty(*bad)


def test_a_stack_that_no_step_takes_is_refused_by_the_forward_pass():
    """the limits of the step (2^32 weights, 2^31 bytes of an expert) are checked before a training step's forward pass; a
    forward pass without a gradient goes on (here to the check of the device)"""
    from optimizer_gemm_amd.nn import ForgeExperts

    idx, w = torch.zeros(2, 1, dtype=torch.int64, device="meta"), torch.zeros(2, 1, device="meta")

    def block(d, h, e, **kw):
        return ForgeExperts(d, h, e, device="meta", **kw), torch.zeros(2, d, dtype=torch.bfloat16, device="meta")

    for args, kw, match in (((8192, 65536, 8), {"opt": "sgd"}, "fewer than 2.32 weights"),
                            ((8192, 65536, 4), {}, "moments span less than 2.31"),
                            ((8192, 65536, 4), {"states": "bf16", "fused": False}, "gradient spans less than 2.31"),
                            ((8192, 131072, 2), {"opt": "sgd"}, "moments span less than 2.31")):
        blk, x = block(*args, **kw)
        with pytest.raises(ValueError, match=match):
            blk(x, idx, w)
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            blk(x, idx, w)
    for args, kw in (((8192, 65536, 7), {"states": "bf16"}), ((8192, 65536, 7), {"opt": "sgd"}), ((8192, 65528, 7), {})):
        blk, x = block(*args, **kw)
        with pytest.raises(ValueError, match="device tensors"):
            blk(x, idx, w)


def test_tiles_of_a_product():
    """which tiles a product takes is told for every kind, and refused for what is none"""
    t = L.forge_expert_tile
    for p in range(6):
        for bad in ((0, 64, 64, 4), (16, 0, 64, 4), (16, 64, -1, 4), (16, 64, 64, 0), (16, 64, 64, 1025), (1 << 30, 64, 64, 4)):
            assert t(p, *bad, BF16) == SHAPE
        assert t(p, 16, 64, 64, 4, F32) == DTYPE
        assert t(p, 20000, 4096, 4096, 8, BF16) in (256, 128, 64)
        assert t(p, 20000, 4096, 4096, 8, I8) in ((256, 128, 64) if p < 3 else (DTYPE,))
        # a few rows: forward products have a kernel of their own
        assert t(p, 16, 4096, 4096, 8, BF16) == 0 if p < 3 else t(p, 16, 4096, 4096, 8, BF16) > 0
    assert t(6, 16, 64, 64, 4, BF16) == UNSUP and t(-1, 16, 64, 64, 4, BF16) == UNSUP
    assert t(1, 16, 4096, 4096, 8, I8) == 0 and t(2, 16, 4096, 14336, 8, I8) > 0  # (gated over much memory: tiles)
    assert t(5, 16, 1 << 29, 1 << 29, 4, BF16) == UNSUP and t(5, 16, 8192, 65536, 4, BF16) == UNSUP
    # one row of tiles, half as wide but two a unit: as many rounds, so the small ones
    assert t(5, 16, 0x1FFFFFFF, 1, 1024, BF16) == 128 and t(4, 16, 0x3FFFFFFF, 0x3FFFFFFF, 1024, BF16) > 0
    # the stack's gradient: two small rounds are taken for two large ones, five not for three
    assert t(5, 100, 128, 1920, 40, BF16) == 128 and t(5, 100, 1088, 1800, 17, BF16) == 256


def test_a_captured_backward_pass_of_a_block_is_refused(monkeypatch):
    """its steps are counted on the host, where a replay does not come by"""
    from types import SimpleNamespace

    from optimizer_gemm_amd import nn as fnn

    stack = SimpleNamespace(_step_count=0)
    ctx = SimpleNamespace(block=SimpleNamespace(gate=stack, up=stack, down=stack), counts=[0, 0, 0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="a graph takes the operators' calls"):
        fnn._ExpertsFn.backward(ctx, torch.zeros(2, 8))
    assert stack._step_count == 0
