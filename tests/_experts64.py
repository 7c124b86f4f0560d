"""Plain float64 forms of the layers of experts and of the 8-bit products, with the error each float32 kernel result may
have (tests/_ops64.py has the terms), for the GPU tests."""
import torch

from _ops64 import U, act64, act_err, gated64, gated_back64, linear64, mm64


def plan64(idx, experts):
    """offsets, pos by the definition: routes in order of (expert, token, slot)"""
    flat = idx.reshape(-1).tolist()
    rows = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            rows[e].append(i)
    pos, offsets, n = [-1] * len(flat), [0], 0
    for r in rows:
        for i in r:
            pos[i] = n
            n += 1
        offsets.append(n)
    return torch.tensor(offsets), torch.tensor(pos, dtype=torch.int32).reshape(idx.shape)


def routes(seed, t, k, experts, dropped=0.0, skew=1.0, empty=()):
    """idx [t, k]: distinct experts per token where there are enough, uneven popularity, some dropped"""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(t, experts, generator=g) + skew * torch.randn(1, experts, generator=g)
    for e in empty:
        z[:, e] = -1e9
    idx = torch.topk(z, min(k, experts), dim=1).indices
    if k > experts:
        idx = torch.cat([idx] * (k // experts + 1), dim=1)[:, :k]
    drop = torch.rand(t, k, generator=g) < dropped
    return torch.where(drop, torch.full_like(idx, -1), idx).contiguous()


def spans(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def grouped(offsets, f, *rows):
    """Applies f(e, rows of expert e) -> a tuple of results and bounds, and joins them by rows"""
    outs = [f(e, *[r[a:b] for r in rows]) for e, a, b in spans(offsets)]
    return [torch.cat([o[i] for o in outs]) for i in range(len(outs[0]))]


def expert_linear64(X, W, offsets, act):
    return grouped(offsets, lambda e, x: linear64(x, W[e], None, act), X)


def expert_gated64(X, Wg, Wu, offsets, act):
    return grouped(offsets, lambda e, x: gated64(x, Wg[e], Wu[e], act), X)


def expert_gated_dgrad64(dY, Wd, G, U_, offsets, act):
    def f(e, dy, g, u):
        dh, ddh = mm64(dy, Wd[e])
        return gated_back64(dh, ddh, g, u, act)
    return grouped(offsets, f, dY, G, U_)


def expert_dgrad64(dYs, Ws, offsets):
    def f(e, *dys):
        ps = [mm64(dy, W[e]) for dy, W in zip(dys, Ws)]
        k = sum(W.shape[1] for W in Ws)
        x = sum(p[0] for p in ps)
        a = sum(dy.double().abs() @ W[e].double().abs() for dy, W in zip(dys, Ws))
        return x, k * U * a  # one accumulation over all the layers
    return grouped(offsets, f, *dYs)


def expert_wgrad64(X, dY, offsets):
    o = offsets.tolist()
    out, err = [], []
    for e in range(len(o) - 1):
        x, d = X[o[e]:o[e + 1]].double(), dY[o[e]:o[e + 1]].double()
        out.append(d.t() @ x)
        err.append(max(1, x.shape[0]) * U * (d.abs().t() @ x.abs()))
    return torch.stack(out), torch.stack(err)


def combine64(Yp, pos, w, residual=None):
    """sum over the slots; each product and each addition rounds once"""
    p = pos.long()
    rows = Yp.double()[p.clamp(min=0)] if Yp.shape[0] else torch.zeros(*p.shape, Yp.shape[1], device=Yp.device).double()
    f = (p >= 0).double() * (1.0 if w is None else w.double())
    terms = torch.where((p >= 0)[:, :, None], rows * f[:, :, None], torch.zeros_like(rows))
    y, a = terms.sum(1), terms.abs().sum(1)
    err = (p.shape[1] + 1) * U * a
    if residual is not None:
        y = y + residual.double()
        err = err + U * (a + residual.double().abs())
    return y, err


# ---- 8 bits: integer sums are exact; the conversion to float32, the product of the two factors and the product with it
# round once each
def q8_product64(Q, s, W, ws):
    z = (Q.double() @ W.double().t()) * (s.double()[:, None] * ws.double()[None, :])
    return z, 3 * U * z.abs()


def linear_q8_64(Q, s, W, ws, bias=None, act="none", residual=None):
    z, dz = q8_product64(Q, s, W, ws)
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * z.abs()
    y, dy = act64(z, act)[0], act_err(z, dz, act)
    if residual is not None:
        y = y + residual.double()
        dy = dy + U * y.abs()
    return y, dy


def gated_q8_64(Q, s, Wg, gs, Wu, us, act):
    g, dg = q8_product64(Q, s, Wg, gs)
    u, du = q8_product64(Q, s, Wu, us)
    a = act64(g, act)[0]
    return a * u, act_err(g, dg, act) * u.abs() + a.abs() * du + U * (a * u).abs()
