"""Training-step integration: a linear layer whose backward pass performs its own update.

FORGE (explainer pages, §2 Method) folds the optimizer step into the weight-
gradient computation of the backward pass; the input gradient must be read
before the weights change (§5, limitations). ForgeLinear wires that into
PyTorch autograd: forward is Y = X W^T; backward computes dX = dY W with the
library's dgrad kernel on the current (old) W, then enqueues the fused
wgrad + optimizer kernel on the same stream, which updates W and its moments in
place. The weight gradient is never materialised: backward returns None for it,
so `weight.grad` stays None and no optimizer.step() follows.

Each backward call is one optimizer step of that layer (a module used several
times per step, such as a tied embedding, is outside what the method supports;
layers with an epilogue, joined blocks and heads, which keep more of the forward
pass than its input, refuse the second of two backward passes).

For comparison the same module runs the usual two-phase schedule with
fused=False: backward stores the float32 dW (the "gradient floor" every layer
holds until the optimizer runs) and `step_all(model)` then applies the update
with the library's stand-alone optimizer pass. Both schedules use the same
kernels and the same per-element update, so they differ only in when the
gradient exists and where it lives.

Around the linear layers: ForgeLinear takes a bias and an activation and adds a residual in
its forward product's epilogue, SwiGLUBlock(joined=True) runs gate, up, activation and
product as one kernel, and ForgeHead is a linear head whose softmax cross entropy never
stores its logits and whose backward pass steps its weights piece by piece of the vocabulary.
"""
from __future__ import annotations

import functools
import math
from typing import Optional

import torch
import torch.utils.checkpoint

from . import forge

_SEED_MIX = 0x9E3779B97F4A7C15


class _ForgeLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, layer: "ForgeLinear") -> torch.Tensor:
        ctx.layer = layer
        ctx.save_for_backward(x)
        # forward product (not part of the fused path): a plain library GEMM
        return torch.matmul(x, weight.t())

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        (x,) = ctx.saved_tensors
        layer: ForgeLinear = ctx.layer
        w = layer.weight
        x2 = x.reshape(-1, w.shape[1])
        dy2 = dy.reshape(-1, w.shape[0])
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        if not dy2.is_contiguous() or dy2.dtype != w.dtype:
            dy2 = dy2.to(w.dtype).contiguous()
        dx = None
        if ctx.needs_input_grad[0]:
            dx = forge.dgrad(dy2, w.detach()).reshape(x.shape)  # old W, before the update below
        _update([layer], x2, [dy2])
        return dx, None, None


def _differentiated(*tensors) -> bool:
    """Whether autograd will record a node of these: without, a forward pass keeps nothing for
    backward (inside a node's own forward the mode is off already)."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _rows(t: torch.Tensor, cols: int, dtype: torch.dtype) -> torch.Tensor:
    """t as contiguous rows of `cols` elements of `dtype`."""
    if t.dim() == 0 or t.shape[-1] != cols:
        raise ValueError(f"rows of {cols} elements wanted, not a tensor of shape {tuple(t.shape)}")
    t = t.reshape(-1, cols)
    return t if t.is_contiguous() and t.dtype == dtype else t.to(dtype).contiguous()


def _update(layers, x2: torch.Tensor, dy2s, group: bool = False) -> None:
    """The weight-gradient half of a backward pass: a layer's fused step on x2, or, with `group`,
    the grouped one of layers that read x2 and are _alike; or, two-phase, the float32 gradients for
    step_all(). A call that is refused leaves the step counts as they were."""
    L0 = layers[0]
    if not L0.fused:
        for L, dy2 in zip(layers, dy2s):
            # the float32 gradient waits for step_all(); a second backward before it adds to it, as
            # the usual gradient accumulation does
            g = forge.wgrad(x2, dy2)
            if L.grad32 is None:
                L.grad32 = g
            else:
                L.grad32.add_(g)
        return
    step = L0._step_count + 1
    ev = L0.timing
    if ev is not None:
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
    if not group:
        forge.wgrad_step(x2, dy2s[0], L0.weight.detach(), L0.m, L0.v, L0.opt, L0.hyper, step, L0.seed,
                         L0.m_scale, L0.v_scale, code=L0.code)
    else:
        forge.wgrad_step_group(x2, dy2s, [L.weight.detach() for L in layers], [L.m for L in layers],
                               [L.v for L in layers], L0.opt, L0.hyper, step, [L.seed for L in layers],
                               [L.m_scale for L in layers], [L.v_scale for L in layers], code=L0.code)
    for L in layers:
        L._step_count = step
    if ev is not None:
        e1.record()
        ev.append((e0, e1))


def _same_rows(what: str, lead, x_lead) -> None:
    """Leading dimensions of two tensors that are taken row by row: the same rows in the same order
    (dimensions of 1 and a flat list of rows count as the same)."""
    if len(lead) == 1 or len(x_lead) == 1:
        same = math.prod(lead) == math.prod(x_lead)
    else:
        same = [n for n in lead if n != 1] == [n for n in x_lead if n != 1]
    if not same:
        raise ValueError(f"{what} of leading shape {tuple(lead)} beside an input of {tuple(x_lead)}")


class _NoDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, gg):
        raise RuntimeError("the operators are differentiated once: their gradients have no derivatives")


def _once(backward):
    """A backward pass whose gradients are no functions for autograd. Under create_graph they come
    out with a node that refuses to be differentiated, where without one a loss that holds them would
    lose that part silently."""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(None if g is None else _NoDerivative.apply(g.detach().requires_grad_()) for g in out)
    return run


def _check_unstepped(layers, counts) -> None:
    """What a forward pass kept (pre-activations, projections) belongs to its weights, and so does
    the input gradient: refuses a backward pass once they have been stepped. (Steps write through raw
    pointers, which autograd's own check of saved tensors does not see.)"""
    if [L._step_count for L in layers] != counts:
        raise RuntimeError("the layer's weights were stepped after this output was computed")


class _ForgeLinearEpiFn(torch.autograd.Function):
    """ForgeLinear with a bias, an activation or a residual: forward is one product with an
    epilogue; backward takes the gradient through the activation, then dX, then the steps."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, layer, recorded):
        x2 = _rows(x, weight.shape[1], weight.dtype)
        r2 = None if residual is None else _rows(residual, weight.shape[0], weight.dtype)
        if residual is not None:
            _same_rows("a residual", residual.shape[:-1], x.shape[:-1])
        keep = recorded and layer.act != "none"
        y = forge.linear(x2, weight.detach(), bias=None if bias is None else bias.detach(), act=layer.act, residual=r2,
                         save=keep)
        y, z = y if keep else (y, None)
        ctx.layer, ctx.x_shape, ctx.r_shape = layer, x.shape, None if residual is None else residual.shape
        ctx.counts = [layer._step_count]
        ctx.save_for_backward(x2, z, weight)
        return y.reshape(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @_once
    def backward(ctx, dy):
        layer = ctx.layer
        _check_unstepped([layer], ctx.counts)
        x2, z, weight = ctx.saved_tensors
        w = weight.detach()
        dy2 = _rows(dy, w.shape[0], w.dtype)
        dz, db = forge.linear_act_backward(dy2, z, act=layer.act, want_bias=layer.bias is not None)
        # old W, before the update below
        dx = forge.dgrad(dz, w).reshape(ctx.x_shape) if ctx.needs_input_grad[0] else None
        _update([layer], x2, [dz])
        if db is not None:
            layer._bias_update(db)
        return dx, None, None, (dy.reshape(ctx.r_shape) if ctx.needs_input_grad[3] else None), None, None


class ForgeLinear(torch.nn.Module):
    """Y = X W^T with the optimizer step fused into the backward pass.

    weight: [out, in] bf16 or float32 parameter. opt / hyper: the optimizer and its
    hyper-parameters (forge_hyper fields). states: "f32", "bf16", "q8" (INT8
    block-64, linear codes) or "q8dyn" (INT8 block-64, dynamic 8-bit code).
    fused: True for the fused step in backward; False for the two-phase schedule
    (float32 gradient kept in `grad32`, update applied by `step()`).
    timing: if a list, each fused call appends its (start, end) CUDA events.
    bias, act: Y = act(X W^T + bias) (act one of forge.ACTS), and forward(x, residual) adds
    `residual`, all in the product's epilogue; the bias takes the same optimizer with float32
    moments, as a stand-alone step after the weights' (its gradient is a float32 sum over the
    tokens; two-phase: kept in `bias_grad32`). Without any of the three the layers are bias-free,
    as those the pages evaluate, and forward is a plain library product.
    """

    def __init__(self, in_features: int, out_features: int, opt: str = "adamw", hyper: Optional[dict] = None,
                 states: str = "f32", dtype: torch.dtype = torch.bfloat16, device=None, seed: int = 0,
                 weight: Optional[torch.Tensor] = None, fused: bool = True, bias: bool = False, act: str = "none"):
        super().__init__()
        if act not in forge.ACTS:
            raise ValueError(f"unknown activation {act!r}; one of {', '.join(forge.ACTS)}")
        self.fused = bool(fused)
        self.act = act
        self.grad32: Optional[torch.Tensor] = None
        self.timing: Optional[list] = None
        if weight is None:
            weight = torch.empty(out_features, in_features, dtype=dtype, device=device)
            torch.nn.init.normal_(weight, std=0.02)
        self.weight = torch.nn.Parameter(weight, requires_grad=True)
        self.opt = opt
        self.hyper = forge.make_hyper(opt, **(hyper or {}))
        m, v, ms, vs = forge.new_states(self.weight.detach(), opt, states)
        self.code = "dynamic" if states == "q8dyn" else "linear"
        for name, t in (("m", m), ("v", v), ("m_scale", ms), ("v_scale", vs)):
            if t is None:
                setattr(self, name, None)
            else:
                self.register_buffer(name, t)
        self.seed = (int(seed) * _SEED_MIX) & (2 ** 64 - 1)
        self._step_count = 0
        self.bias: Optional[torch.nn.Parameter] = None
        self.bias_grad32: Optional[torch.Tensor] = None
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(self.weight.shape[0], dtype=self.weight.dtype,
                                                       device=self.weight.device))
            bm, bv, _, _ = forge.new_states(self.bias.detach().unsqueeze(0), opt, "f32")
            for name, t in (("bias_m", bm), ("bias_v", bv)):
                if t is None:
                    setattr(self, name, None)
                else:
                    self.register_buffer(name, t)

    @property
    def step_count(self) -> int:
        return self._step_count

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if self.bias is not None or self.act != "none" or residual is not None:
            return _ForgeLinearEpiFn.apply(x, self.weight, self.bias, residual, self,
                                           _differentiated(x, self.weight, self.bias, residual))
        return _ForgeLinearFn.apply(x, self.weight, self)

    def _bias_update(self, db: torch.Tensor) -> None:
        if self.fused:
            self._bias_step(db)
        elif self.bias_grad32 is None:
            self.bias_grad32 = db
        else:
            self.bias_grad32.add_(db)

    def _bias_step(self, db: torch.Tensor) -> None:
        # the bias draws its stochastic rounding from a stream of its own
        forge.optimizer_step(db.unsqueeze(0), self.bias.detach().unsqueeze(0), self.bias_m, self.bias_v, self.opt,
                             self.hyper, self._step_count, self.seed ^ _SEED_MIX)

    def step(self) -> None:
        """Two-phase schedule: apply the optimizer to the stored gradient and free it
        (nothing to do for a fused layer, whose backward already stepped)."""
        if self.fused or self.grad32 is None:
            return
        self._step_count += 1
        forge.optimizer_step(self.grad32, self.weight.detach(), self.m, self.v, self.opt, self.hyper,
                             self._step_count, self.seed, self.m_scale, self.v_scale, code=self.code)
        self.grad32 = None
        if self.bias_grad32 is not None:
            self._bias_step(self.bias_grad32)
            self.bias_grad32 = None


class _ForgeGroupFn(torch.autograd.Function):
    """Several ForgeLinear layers applied to the same input: forward Y_l = X W_l^T for each;
    backward dX = sum_l dY_l W_l (each on the old W_l) and then one grouped fused step of
    all the layers (forge_linear_wgrad_step_group), where the layers' tiles share the
    launch."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, layers, *weights: torch.Tensor):
        ctx.layers = layers
        ctx.save_for_backward(x)
        return tuple(torch.matmul(x, w.t()) for w in weights)

    @staticmethod
    def backward(ctx, *dys):
        (x,) = ctx.saved_tensors
        layers = ctx.layers
        ws = [L.weight.detach() for L in layers]
        x2 = x.reshape(-1, ws[0].shape[1])
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        dy2s = []
        for w, dy in zip(ws, dys):
            if dy is None:  # an output that reached no loss: a zero gradient, the layer still steps
                dy2s.append(torch.zeros((x2.shape[0], w.shape[0]), dtype=w.dtype, device=w.device))
                continue
            dy2 = dy.reshape(-1, w.shape[0])
            dy2s.append(dy2 if dy2.is_contiguous() and dy2.dtype == w.dtype else dy2.to(w.dtype).contiguous())
        dx = None
        if ctx.needs_input_grad[0]:
            dx = forge.dgrad(dy2s[0], ws[0])  # old W, before the update below
            for w, dy2 in zip(ws[1:], dy2s[1:]):
                dx.add_(forge.dgrad(dy2, w))
            dx = dx.reshape(x.shape)
        _update(layers, x2, dy2s, group=True)
        return (dx, None) + (None,) * len(layers)


def _alike(layers) -> bool:
    """Whether one grouped step may take the layers: the same optimizer, hyper-parameters, moment
    format, schedule, type and step count."""
    L0 = layers[0]
    return not any(
        (L.opt, L.code, L.fused, L._step_count, L.weight.dtype) != (L0.opt, L0.code, L0.fused, L0._step_count,
                                                                     L0.weight.dtype) or
        (L.m is None) != (L0.m is None) or (L.v is None) != (L0.v is None) or
        (L.m is not None and L.m.dtype != L0.m.dtype) or (L.v is not None and L.v.dtype != L0.v.dtype) or
        any(getattr(L.hyper, n) != getattr(L0.hyper, n) for n, _ in L0.hyper._fields_) for L in layers[1:])


def grouped_linear(layers, x: torch.Tensor):
    """Y_l = X W_l^T for ForgeLinear layers that read the same input x, as one autograd node
    whose backward steps all of them in one grouped launch (the layers' outputs as a tuple).
    The layers must agree in optimizer, hyper-parameters, moment format, schedule and step
    count; the group's time is recorded on the first layer's `timing` list."""
    layers = list(layers)
    if not 1 <= len(layers) <= forge.MAX_GROUP:
        raise ValueError(f"a group holds 1..{forge.MAX_GROUP} layers")
    for L in layers:
        if L.bias is not None or L.act != "none":
            raise ValueError("grouped layers have no bias and no activation")
    if not _alike(layers):
        raise ValueError("grouped layers must share optimizer, hyper-parameters, states, schedule and step")
    return _ForgeGroupFn.apply(x, layers, *[L.weight for L in layers])


def step_all(model: torch.nn.Module) -> None:
    """The optimizer phase of the two-phase schedule for every ForgeLinear in `model`."""
    for mod in model.modules():
        if isinstance(mod, ForgeLinear):
            mod.step()


def _rms_norm(x: torch.Tensor, eps: float = 1e-5) -> torch.Tensor:
    xf = x.float()
    return (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + eps)).to(x.dtype)


class _GatedBlockFn(torch.autograd.Function):
    """y = r + down(silu(gate(h)) * up(h)) as two kernels: the gated product (its projections G, U
    kept, its result not: the backward pass forms it again), and the down projection with the
    residual r in its epilogue. Backward: dG, dU and H from dy's product with the down weights,
    dh of both projections in one accumulation - all on the old weights - and then the steps."""

    @staticmethod
    def forward(ctx, h, r, wg, wu, wd, block, recorded):
        h2, r2 = _rows(h, wg.shape[1], wg.dtype), _rows(r, wd.shape[0], wd.dtype)
        out = forge.gated(h2, wg.detach(), wu.detach(), act="silu", save=recorded)
        H, G, U = out if recorded else (out, None, None)
        y = forge.linear(H, wd.detach(), residual=r2)
        ctx.block, ctx.h_shape, ctx.r_shape = block, h.shape, r.shape
        ctx.counts = [L._step_count for L in (block.gate, block.up, block.down)]
        ctx.save_for_backward(h2, G, U, wg, wu, wd)
        return y.reshape(r.shape)

    @staticmethod
    @_once
    def backward(ctx, dy):
        gate, up, down = ctx.block.gate, ctx.block.up, ctx.block.down
        _check_unstepped((gate, up, down), ctx.counts)
        h2, G, U, wg, wu, wd = ctx.saved_tensors
        wg, wu, wd = wg.detach(), wu.detach(), wd.detach()
        dy2 = _rows(dy, wd.shape[0], wd.dtype)
        dG, dU, H = forge.gated_dgrad(dy2, wd, G, U, act="silu")
        dh = forge.dgrad_group([dG, dU], [wg, wu]).reshape(ctx.h_shape) if ctx.needs_input_grad[0] else None
        _update([down], H, [dy2])
        if wg.dtype == torch.bfloat16 and _alike((gate, up)):
            _update([gate, up], h2, [dG, dU], group=True)
        else:  # the grouped step takes bf16 layers that agree
            _update([gate], h2, [dG])
            _update([up], h2, [dU])
        return dh, (dy.reshape(ctx.r_shape) if ctx.needs_input_grad[1] else None), None, None, None, None, None


class SwiGLUBlock(torch.nn.Module):
    """Residual SwiGLU MLP block of a Llama-style decoder layer built from ForgeLinear:
    y = x + down(silu(gate(n(x))) * up(n(x))), with n a parameter-free RMS norm.
    gate / up: [hidden, d] weights, down: [d, hidden]. With checkpoint=True the block
    keeps only its input for backward and recomputes the rest (activation
    checkpointing); the recomputation runs before any of the block's layers steps,
    so it sees the same weights as the forward pass. With grouped=True gate and up, which
    read the same n(x), take their fused steps in one grouped launch. With joined=True gate,
    up, activation and product are one kernel, the residual is added by the down projection,
    and the backward pass is joined likewise (gate and up stepped in one launch where they are bf16
    and agree in optimizer, states and step count, else one after the other); results as the
    separate layers' up to rounding."""

    def __init__(self, d: int, hidden: int, checkpoint: bool = False, seed: int = 0, grouped: bool = False,
                 joined: bool = False, **kw):
        super().__init__()
        for name in ("bias", "act", "weight"):
            if name in kw:
                raise ValueError(f"SwiGLUBlock's layers take no {name}")
        self.gate = ForgeLinear(d, hidden, seed=3 * seed, **kw)
        self.up = ForgeLinear(d, hidden, seed=3 * seed + 1, **kw)
        self.down = ForgeLinear(hidden, d, seed=3 * seed + 2, **kw)
        self.checkpoint = checkpoint
        self.grouped = grouped
        self.joined = joined

    def _body(self, x: torch.Tensor) -> torch.Tensor:
        h = _rms_norm(x)
        if self.joined:
            weights = (self.gate.weight, self.up.weight, self.down.weight)
            return _GatedBlockFn.apply(h, x, *weights, self, _differentiated(h, x, *weights))
        if self.grouped:
            g, u = grouped_linear((self.gate, self.up), h)
        else:
            g, u = self.gate(h), self.up(h)
        return x + self.down(torch.nn.functional.silu(g) * u)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.checkpoint and torch.is_grad_enabled():
            return torch.utils.checkpoint.checkpoint(self._body, x, use_reentrant=False)
        return self._body(x)


class _LinearCrossEntropyFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, reduction, head):
        x2 = _rows(x, weight.shape[1], weight.dtype)
        _same_rows("targets", targets.shape, x.shape[:-1])
        t1 = targets.reshape(-1).contiguous()
        loss, lse, total = forge.linear_cross_entropy(x2, weight.detach(), t1, ignore_index=ignore_index,
                                                      reduction=reduction)
        ctx.args, ctx.head, ctx.x_shape = (ignore_index, reduction), head, x.shape
        ctx.step = None if head is None else head._step_count
        # the scalar is a part of `total`, which backward needs: a copy goes out
        ctx.save_for_backward(x2, t1, lse, total, weight)
        return loss.reshape(targets.shape) if reduction == "none" else loss.clone()

    @staticmethod
    @_once
    def backward(ctx, dloss):
        x2, t1, lse, total, weight = ctx.saved_tensors
        ignore_index, reduction = ctx.args
        g = dloss.float().reshape(-1).contiguous()
        head, w = ctx.head, weight.detach()
        if head is None:
            dx, dw = forge.linear_cross_entropy_backward(x2, w, t1, lse, g, ignore_index=ignore_index,
                                                         reduction=reduction, total=total,
                                                         want_dx=ctx.needs_input_grad[0],
                                                         want_dw=ctx.needs_input_grad[1])
        else:
            if head._step_count != ctx.step:
                # lse belongs to the weights of the forward pass
                raise RuntimeError("the head's weights were stepped after this loss was computed")
            dx, dw = forge.linear_cross_entropy_step(x2, w, head.m, head.v, t1, lse, g, head.opt, head.hyper,
                                                     head._step_count + 1, head.seed, head.m_scale, head.v_scale,
                                                     code=head.code, ignore_index=ignore_index, reduction=reduction,
                                                     total=total, want_dx=ctx.needs_input_grad[0], piece=head.piece), None
            head._step_count += 1
        return (None if dx is None else dx.reshape(ctx.x_shape)), dw, None, None, None, None


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean") -> torch.Tensor:
    """Softmax cross entropy of the logits x weight^T without storing them, differentiable by x and
    weight (gradients in their types). x [..., d], targets [...] int64; reduction "mean" over the
    tokens that are not ignore_index, "sum" or "none". Once: a second derivative is refused."""
    return _LinearCrossEntropyFn.apply(x, weight, targets, ignore_index, reduction, None)


class ForgeHead(torch.nn.Module):
    """Linear head with softmax cross entropy: forward(x, targets) is the loss, its logits never
    stored; backward computes dX and steps the weights [vocab, d] piece by piece of the
    vocabulary, the gradient never stored either. Arguments as ForgeLinear's; `piece` the
    vocabulary entries per piece (0: the library's choice). The step takes weights and moments
    of less than 2^31 bytes each (131072 x 4096 in bf16, with bf16 or 8-bit moments). Each backward
    call is one step, of a loss computed with the weights as they are: a loss from before another
    one's step is refused."""

    def __init__(self, d: int, vocab: int, opt: str = "adamw", hyper: Optional[dict] = None, states: str = "f32",
                 dtype: torch.dtype = torch.bfloat16, device=None, seed: int = 0,
                 weight: Optional[torch.Tensor] = None, ignore_index: int = -100, piece: int = 0):
        super().__init__()
        if weight is None:
            weight = torch.empty(vocab, d, dtype=dtype, device=device)
            torch.nn.init.normal_(weight, std=0.02)
        self.weight = torch.nn.Parameter(weight, requires_grad=True)
        self.opt, self.hyper = opt, forge.make_hyper(opt, **(hyper or {}))
        m, v, ms, vs = forge.new_states(self.weight.detach(), opt, states)
        self.code = "dynamic" if states == "q8dyn" else "linear"
        for name, t in (("m", m), ("v", v), ("m_scale", ms), ("v_scale", vs)):
            if t is None:
                setattr(self, name, None)
            else:
                self.register_buffer(name, t)
        self.seed = (int(seed) * _SEED_MIX) & (2 ** 64 - 1)
        self.ignore_index, self.piece = int(ignore_index), int(piece)
        self._step_count = 0

    @property
    def step_count(self) -> int:
        return self._step_count

    def forward(self, x: torch.Tensor, targets: torch.Tensor, reduction: str = "mean") -> torch.Tensor:
        return _LinearCrossEntropyFn.apply(x, self.weight, targets, self.ignore_index, reduction, self)
