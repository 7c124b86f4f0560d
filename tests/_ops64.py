"""Plain float64 forms of the operators around the fused step, with the error each float32
kernel result may have, for the GPU tests.

Error terms, first order (u = 2^-24, half a float32 step):
* a sum of K products in FP32, in any order: K u sum |a b| (matrix instructions included);
* an activation of z: its argument's error times the largest slope, 1.13, plus the
  evaluation: the hardware exponential and reciprocal are within one ulp of their results, the
  exponential's argument c z is rounded (relative error of the result |c z| u, |c z| at most
  1.6 |z| (1 + 0.045 z^2), but the result it multiplies falls at least as fast as e^-|c z|, so
  |c z| counts up to 8 only), and the Gaussian's polynomial form is within 1.5e-7 = 2.6 u:
  ACT_U u |z| for the value, ACT_U u (1 + |z|) for the derivative, ACT_U = 48;
* rounding to the output type: half a step, finfo(type).eps / 2 relative.
"""
import math

import torch

U = 2.0 ** -24
ACT_U = 48 * U
SLOPE = 1.13


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act64(z, act):
    """value and derivative"""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return torch.clamp(z, min=0), (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z) / 2


def mm64(a, b):
    """a [n, k] b [k, m] in float64 and its FP32 summation bound."""
    a, b = a.double(), b.double()
    return a @ b, a.shape[1] * U * (a.abs() @ b.abs())


def act_err(z, dz, act):
    if act in ("none", "relu"):
        return dz
    return SLOPE * dz + ACT_U * z.abs()


def slope_err(z, act):
    return torch.zeros_like(z) if act in ("none", "relu") else ACT_U * (1 + z.abs())


def linear64(X, W, bias=None, act="none", residual=None):
    """(Y, its bound, Z, its bound)"""
    z, dz = mm64(X, W.t())
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * z.abs()
    y = act64(z, act)[0]
    dy = act_err(z, dz, act)
    if residual is not None:
        y = y + residual.double()
        dy = dy + U * y.abs()
    return y, dy, z, dz


def gated64(X, Wg, Wu, act):
    g, dg = mm64(X, Wg.t())
    u, du = mm64(X, Wu.t())
    a = act64(g, act)[0]
    return a * u, act_err(g, dg, act) * u.abs() + a.abs() * du + U * (a * u).abs(), g, dg, u, du


def gated_back64(dh, ddh, G, U_, act):
    """dG, dU, H and their bounds, from dH with bound ddh and the stored G, U"""
    g, u = G.double(), U_.double()
    a, d = act64(g, act)
    ea = act_err(g, torch.zeros_like(g), act)
    ed = slope_err(g, act)
    dg, du, h = dh * u * d, dh * a, a * u
    return (dg, ddh * (u * d).abs() + (dh * u).abs() * ed + 2 * U * dg.abs(),
            du, ddh * a.abs() + dh.abs() * ea + U * du.abs(),
            h, ea * u.abs() + U * h.abs())


def close(name, got, want, bound, dtype=None):
    """got within bound of want plus half a step of its type; the worst ratio is printed."""
    dtype = dtype or got.dtype
    tol = bound + half_step(dtype) * (want.abs() + bound)
    # below the type's normal range half a step is absolute
    tol = tol + torch.finfo(dtype).tiny * half_step(dtype)
    err = (got.double() - want).abs()
    assert got.shape == want.shape, name
    if got.numel() == 0:
        return
    worst = float((err / tol).max())
    print(f"[ops] {name}: worst error / bound {worst:.3f}")
    assert torch.isfinite(got).all(), name
    assert worst <= 1.0, f"{name}: {worst} of the bound at {int((err / tol).argmax())}"


def xent64(X, W, y, ignore):
    """per-token loss, lse (float64), the bound of either, logits, the logits' bound, counted rows"""
    z, dz = mm64(X, W.t())
    lse = torch.logsumexp(z, dim=1)
    keep = y != ignore
    loss = torch.zeros_like(lse)
    r = torch.nonzero(keep)[:, 0]
    loss[r] = lse[r] - z[r, y[r]]
    zmax = z.max(dim=1).values
    # the sum of exponentials: each term's argument error |z - max| 2u (weighted by the terms,
    # so at most the largest that still matters, 40), each term and each addition half a step
    terms = 64 + W.shape[0] / 64 + 80 + 8
    de = dz.max(dim=1).values + terms * U + 2 * U * (lse.abs() + zmax.abs())
    dl = de + dz.max(dim=1).values + U * loss.abs()
    return loss, dl, lse, de, z, dz, keep


def xent_grad64(X, W, y, ignore, g, dtype):
    """dX, dW for per-token factors g (float64, 0 where ignored), with bounds that count the
    rounding of dz to `dtype`"""
    loss, dl, lse, de, z, dz, keep = xent64(X, W, y, ignore)
    p = torch.exp(z - lse[:, None])
    d = p.clone()
    r = torch.nonzero(keep)[:, 0]
    d[r, y[r]] -= 1
    d = d * g[:, None]
    # p's error: its argument's (z, lse and the subtraction), the exponential's ulp
    rel = dz + de[:, None] + 2 * U * (z - lse[:, None]).abs() + 4 * U
    e = (p * rel + 2 * U) * g.abs()[:, None] + half_step(dtype) * d.abs()
    Xd, Wd = X.double(), W.double()
    dx, dw = d @ Wd, d.t() @ Xd
    ex = e @ Wd.abs() + (W.shape[0] + 8) * U * (d.abs() @ Wd.abs())
    ew = e.t() @ Xd.abs() + (X.shape[0] + 8) * U * (d.abs().t() @ Xd.abs())
    # the common factor: its quotient, its product
    return dx, ex + 4 * U * dx.abs(), dw, ew + 4 * U * dw.abs()
