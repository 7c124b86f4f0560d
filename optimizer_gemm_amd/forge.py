"""Python binding of libforge.so (ctypes): argument marshalling only.

Every computation runs in the library's HIP kernels. PyTorch provides device
memory and the current HIP stream; tensors are described to the C ABI by data
pointer, dtype, shape and row pitch. There is no fallback: if the library is
not built, importing this module raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import re
from typing import Dict, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("FORGE_LIB", os.path.join(_PKG, "_lib", "libforge.so"))

F32, BF16, I8, U8, E4M3, E5M2, I8_DYN, U8_DYN = 0, 1, 2, 3, 4, 5, 6, 7
OPTIMIZERS = ("adamw", "sgd", "sgd_momentum", "lion", "rmsprop", "adagrad", "nadam", "radam")
OPT_ID = {name: k for k, name in enumerate(OPTIMIZERS)}
# slot usage per optimizer: (uses m, uses v)
SLOTS = {"adamw": (1, 1), "sgd": (0, 0), "sgd_momentum": (1, 0), "lion": (1, 0), "rmsprop": (0, 1),
         "adagrad": (0, 1), "nadam": (1, 1), "radam": (1, 1)}

STATUS = {0: "FORGE_OK", -1: "FORGE_ERR_NULL", -2: "FORGE_ERR_SHAPE", -3: "FORGE_ERR_DTYPE",
          -4: "FORGE_ERR_ALIGN", -5: "FORGE_ERR_UNSUPPORTED", -6: "FORGE_ERR_HYPER", -7: "FORGE_ERR_HIP",
          -8: "FORGE_ERR_ALIAS", -9: "FORGE_ERR_SCRATCH"}


class ForgeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("scale", ctypes.c_void_p)]


class ForgeHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("momentum", ctypes.c_double),
                ("dampening", ctypes.c_double), ("alpha", ctypes.c_double), ("lr_decay", ctypes.c_double),
                ("momentum_decay", ctypes.c_double), ("nesterov", ctypes.c_int32),
                ("stochastic_round", ctypes.c_int32)]


class ForgeScalars(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in ("lr", "decay", "wd", "b1", "omb1", "b2", "omb2", "step_size",
                                              "inv_sqrt_bc2", "eps", "c_g", "c_m")] + \
               [("flag", ctypes.c_int32), ("opt", ctypes.c_int32)]


class ForgeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_str(status)})")
        self.status = status


class _NoCalls:
    """In the place of forge_calls where it does not load: the calls that go through it say why, all others work."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name: str):
        raise ImportError(f"{name}: {self._why}; run `python optimizer_gemm_amd/build.py`")


def _load_calls():
    """The module of csrc/forge_calls.cpp: entry points that take tensors as they are, at a fraction of ctypes' time. It is
    built against one torch's C++ interface, so with another one, or without it, the package loads all the same."""
    path = os.path.join(_PKG, "_lib", "forge_calls.so")
    if not os.path.exists(path):
        return _NoCalls(f"forge_calls.so not built at {path}")
    spec = importlib.util.spec_from_file_location("forge_calls", path)
    try:
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        if not re.match(re.escape(mod.torch_version) + r"(?!\d)", torch.__version__):
            return _NoCalls(f"forge_calls.so was built against torch {mod.torch_version}, this is {torch.__version__}")
        mod.load(LIB_PATH, ForgeError)
    except (ImportError, AttributeError) as e:
        return _NoCalls(f"forge_calls.so does not load ({e})")
    return mod


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libforge.so not built at {LIB_PATH}; run `python optimizer_gemm_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sigs = {
        "forge_linear_wgrad_step": ([P(ForgeTensor)] * 5 + [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64,
                                                             ctypes.c_uint64, ctypes.c_void_p], ctypes.c_int),
        "forge_linear_wgrad_step_group": ([P(ForgeTensor), ctypes.c_int32] + [P(ForgeTensor)] * 4 +
                                          [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64, P(ctypes.c_uint64),
                                           ctypes.c_void_p], ctypes.c_int),
        "forge_linear_dgrad": ([P(ForgeTensor)] * 3 + [ctypes.c_void_p], ctypes.c_int),
        "forge_linear_wgrad": ([P(ForgeTensor), P(ForgeTensor), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p],
                               ctypes.c_int),
        "forge_optimizer_step": ([ctypes.c_void_p, ctypes.c_int64] + [P(ForgeTensor)] * 3 +
                                 [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p],
                                 ctypes.c_int),
        "forge_linear_wgrad_unfused": ([P(ForgeTensor)] * 5 + [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64,
                                                                ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int64,
                                                                ctypes.c_void_p], ctypes.c_int),
        "forge_linear_wgrad_unfused_noalloc": ([P(ForgeTensor)] * 5 + [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64,
                                                                        ctypes.c_uint64, ctypes.c_void_p], ctypes.c_int),
        "forge_step_scalars": ([ctypes.c_int32, P(ForgeHyper), ctypes.c_int64, P(ForgeScalars)], ctypes.c_int),
        "forge_default_hyper": ([ctypes.c_int32, P(ForgeHyper)], ctypes.c_int),
        "forge_rand16": ([ctypes.c_uint64, ctypes.c_int64, ctypes.c_uint32], ctypes.c_uint32),
        "forge_sr_bf16": ([ctypes.c_float, ctypes.c_uint32], ctypes.c_uint16),
        "forge_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "forge_dyn_value": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_float),
        "forge_mfma_peak": ([ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, ctypes.c_float,
                             ctypes.c_void_p], ctypes.c_int),
        "forge_mfma_peak_flops": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_double),
        "forge_dyn_encode": ([ctypes.c_int32, ctypes.c_float], ctypes.c_int32),
        "forge_version": ([], ctypes.c_int),
        "forge_linear_forward": ([P(ForgeTensor)] * 3 + [ctypes.c_int32] + [P(ForgeTensor)] * 3 + [ctypes.c_void_p],
                                 ctypes.c_int),
        "forge_linear_act_backward_workspace": ([ctypes.c_int64] * 2, ctypes.c_int64),
        "forge_linear_act_backward": ([P(ForgeTensor)] * 2 + [ctypes.c_int32, P(ForgeTensor), ctypes.c_void_p,
                                                              ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p],
                                      ctypes.c_int),
        "forge_gated_forward": ([P(ForgeTensor)] * 3 + [ctypes.c_int32] + [P(ForgeTensor)] * 3 + [ctypes.c_void_p],
                                ctypes.c_int),
        "forge_gated_backward": ([P(ForgeTensor)] * 3 + [ctypes.c_int32] + [P(ForgeTensor)] * 3 + [ctypes.c_void_p],
                                 ctypes.c_int),
        "forge_gated_dgrad": ([P(ForgeTensor)] * 4 + [ctypes.c_int32] + [P(ForgeTensor)] * 3 + [ctypes.c_void_p],
                              ctypes.c_int),
        "forge_linear_dgrad_group_workspace": ([ctypes.c_int64] * 3 + [ctypes.c_int32], ctypes.c_int64),
        "forge_linear_dgrad_group_split": ([ctypes.c_int32] + [P(ForgeTensor)] * 3 +
                                           [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p], ctypes.c_int),
        "forge_linear_dgrad_group": ([ctypes.c_int32] + [P(ForgeTensor)] * 3 + [ctypes.c_void_p], ctypes.c_int),
        "forge_linear_xent_workspace": ([ctypes.c_int64] * 3 + [ctypes.c_int32] * 2 + [ctypes.c_int64], ctypes.c_int64),
        "forge_linear_xent_forward": ([P(ForgeTensor)] * 2 + [ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 4 +
                                      [ctypes.c_int64, ctypes.c_void_p], ctypes.c_int),
        "forge_linear_xent_backward": ([P(ForgeTensor)] * 2 + [ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 2 +
                                       [ctypes.c_int32, ctypes.c_void_p] + [P(ForgeTensor)] * 2 +
                                       [ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p],
                                       ctypes.c_int),
        "forge_linear_xent_step": ([P(ForgeTensor)] * 4 + [ctypes.c_int32, P(ForgeHyper), ctypes.c_int64,
                                                           ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int64] +
                                   [ctypes.c_void_p] * 2 + [ctypes.c_int32, ctypes.c_void_p, P(ForgeTensor),
                                                            ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                                            ctypes.c_void_p], ctypes.c_int),
        "forge_expert_plan_workspace": ([ctypes.c_int64] * 2 + [ctypes.c_int32], ctypes.c_int64),
        "forge_expert_plan": ([ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32] + [ctypes.c_void_p] * 3 +
                              [ctypes.c_int64, ctypes.c_void_p], ctypes.c_int),
        "forge_expert_dispatch": ([P(ForgeTensor), ctypes.c_void_p, ctypes.c_int64, P(ForgeTensor), ctypes.c_void_p],
                                  ctypes.c_int),
        "forge_expert_combine": ([P(ForgeTensor), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p] +
                                 [P(ForgeTensor)] * 2 + [ctypes.c_void_p], ctypes.c_int),
        "forge_expert_combine_backward": ([P(ForgeTensor)] * 2 + [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                                  P(ForgeTensor), ctypes.c_void_p, ctypes.c_void_p],
                                          ctypes.c_int),
        "forge_expert_linear": ([P(ForgeTensor)] * 2 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32] +
                                [P(ForgeTensor)] * 2 + [ctypes.c_void_p], ctypes.c_int),
        "forge_expert_gated": ([P(ForgeTensor)] * 3 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32] +
                               [P(ForgeTensor)] * 3 + [ctypes.c_void_p], ctypes.c_int),
        "forge_expert_gated_dgrad": ([P(ForgeTensor)] * 4 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32] +
                                     [P(ForgeTensor)] * 3 + [ctypes.c_void_p], ctypes.c_int),
        "forge_expert_dgrad_group": ([ctypes.c_int32] + [P(ForgeTensor)] * 2 +
                                     [ctypes.c_int32, ctypes.c_void_p, P(ForgeTensor), ctypes.c_void_p], ctypes.c_int),
        "forge_expert_dgrad_group_workspace": ([ctypes.c_int64] * 3 + [ctypes.c_int32] * 2, ctypes.c_int64),
        "forge_expert_dgrad_group_split": ([ctypes.c_int32] + [P(ForgeTensor)] * 2 +
                                           [ctypes.c_int32, ctypes.c_void_p, P(ForgeTensor), ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p], ctypes.c_int),
        "forge_expert_wgrad": ([P(ForgeTensor)] * 2 + [ctypes.c_int32] + [ctypes.c_void_p] * 2 +
                               [ctypes.c_int64, ctypes.c_void_p], ctypes.c_int),
        "forge_expert_wgrad_step": ([P(ForgeTensor)] * 5 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                                            P(ForgeHyper), ctypes.c_int64, ctypes.c_uint64,
                                                            ctypes.c_void_p], ctypes.c_int),
        "forge_expert_tile": ([ctypes.c_int32] + [ctypes.c_int64] * 3 + [ctypes.c_int32] * 2, ctypes.c_int32),
        "forge_quantize_rows": ([P(ForgeTensor)] * 2 + [ctypes.c_void_p], ctypes.c_int),
        "forge_linear_q8": ([P(ForgeTensor)] * 3 + [ctypes.c_int32] + [P(ForgeTensor)] * 2 + [ctypes.c_void_p],
                            ctypes.c_int),
        "forge_gated_q8": ([P(ForgeTensor)] * 3 + [ctypes.c_int32, P(ForgeTensor), ctypes.c_void_p], ctypes.c_int),
        "forge_expert_linear_q8": ([P(ForgeTensor)] * 2 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                                           P(ForgeTensor), ctypes.c_void_p], ctypes.c_int),
        "forge_expert_gated_q8": ([P(ForgeTensor)] * 3 + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                                          P(ForgeTensor), ctypes.c_void_p], ctypes.c_int),
    }
    for name, (argt, rest) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argt
        fn.restype = rest
    return lib


_lib = _load()
_calls = _load_calls()


def lib() -> ctypes.CDLL:
    return _lib


def status_str(status: int) -> str:
    return _lib.forge_status_str(int(status)).decode()


def version() -> int:
    return _lib.forge_version()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8, torch.uint8: U8,
       torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
_FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def describe(t: Optional[torch.Tensor], scale: Optional[torch.Tensor] = None, *, device: bool = True,
             code: str = "linear"):
    """forge_tensor for a 2-D row-major tensor (None -> None). int8 / uint8 moments
    hold linear codes (code="linear") or the dynamic 8-bit code (code="dynamic")."""
    if t is None:
        return None
    if code not in ("linear", "dynamic"):
        raise ValueError(f"unknown moment code {code!r}")
    if t.dim() != 2:
        raise ValueError("forge tensors are 2-D")
    if device and not t.is_cuda:
        raise ValueError("forge kernels take device tensors")
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if t.numel() == 0:
        return ForgeTensor(None, _DT[t.dtype], 0, t.shape[0], t.shape[1], t.shape[1],
                           scale.data_ptr() if scale is not None and scale.numel() else None)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))
    if scale is not None:
        if device and not scale.is_cuda:
            raise ValueError("scales must be device tensors")
        if scale.dtype != torch.float32 or not scale.is_contiguous():
            raise ValueError("scales are contiguous float32")
        if t.dtype in _FP8:
            if scale.numel() != 1:
                raise ValueError("an FP8 tensor has one float32 scale")
        elif tuple(scale.shape) != (t.shape[0], t.shape[1] // 64):
            raise ValueError("block scale shape must be [rows, cols/64]")
    elif t.dtype in _FP8:
        raise ValueError("an FP8 tensor needs its float32 scale")
    dt = _DT[t.dtype]
    if code == "dynamic" and dt in (I8, U8):
        dt = I8_DYN if dt == I8 else U8_DYN
    return ForgeTensor(t.data_ptr(), dt, 0, t.shape[0], t.shape[1], ld,
                       scale.data_ptr() if scale is not None else None)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def default_hyper(opt: str) -> Dict[str, float]:
    h = ForgeHyper()
    st = _lib.forge_default_hyper(OPT_ID[opt], ctypes.byref(h))
    if st:
        raise ForgeError(st, "forge_default_hyper")
    return {n: getattr(h, n) for n, _ in ForgeHyper._fields_}


def make_hyper(opt: str, **over) -> ForgeHyper:
    d = default_hyper(opt)
    for k, v in over.items():
        if k not in d:
            raise KeyError(k)
        d[k] = v
    h = ForgeHyper()
    for n, _ in ForgeHyper._fields_:
        setattr(h, n, int(d[n]) if n in ("nesterov", "stochastic_round") else float(d[n]))
    return h


def _hyper(opt: str, hyper) -> ForgeHyper:
    if isinstance(hyper, ForgeHyper):
        return hyper
    return make_hyper(opt, **(hyper or {}))


def step_scalars(opt: str, hyper=None, step: int = 1) -> Dict[str, float]:
    s = ForgeScalars()
    st = _lib.forge_step_scalars(OPT_ID[opt], ctypes.byref(_hyper(opt, hyper)), int(step), ctypes.byref(s))
    if st:
        raise ForgeError(st, "forge_step_scalars")
    return {n: getattr(s, n) for n, _ in ForgeScalars._fields_}


def rand16(seed: int, step: int, idx: int) -> int:
    return int(_lib.forge_rand16(seed & (2 ** 64 - 1), int(step), int(idx)))


def sr_bf16(x: float, r16: int) -> int:
    return int(_lib.forge_sr_bf16(float(x), int(r16)))


def mfma_peak(n_workgroups: Optional[int] = None, iters: int = 4000, reps: int = 5, stream=None) -> Dict[str, float]:
    """Achieved bf16 MFMA rate of the device (the library's microbenchmark): median
    TFLOP/s over `reps` timed launches on the current stream, after one warm-up. The
    outputs are checked exactly (A = 1, B = 2^-10: every thread writes 2 * iters)."""
    if n_workgroups is None:
        n_workgroups = 3 * torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = torch.empty(n_workgroups * 256, dtype=torch.float32, device="cuda")
    st = _stream(stream)
    times = []
    for r in range(reps + 1):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        rc = _lib.forge_mfma_peak(out.data_ptr(), n_workgroups, iters, 1.0, 2.0 ** -10, st)
        e1.record()
        if rc:
            raise ForgeError(rc, "forge_mfma_peak")
        torch.cuda.synchronize()
        if r:
            times.append(e0.elapsed_time(e1))
    if not bool(torch.all(out == 2.0 * iters)):
        raise RuntimeError("forge_mfma_peak: accumulator check failed")
    ms = sorted(times)[len(times) // 2]
    flops = _lib.forge_mfma_peak_flops(n_workgroups, iters)
    return {"tflops": flops / (ms * 1e-3) / 1e12, "ms": ms, "workgroups": n_workgroups, "iters": iters}


def dyn_value(is_signed: bool, code: int) -> float:
    """Value of a dynamic 8-bit moment code (host helper of the library)."""
    return float(_lib.forge_dyn_value(int(bool(is_signed)), int(code)))


def dyn_encode(is_signed: bool, y: float) -> int:
    """The dynamic code the kernels store for a normalised value y (host helper)."""
    return int(_lib.forge_dyn_encode(int(bool(is_signed)), float(y)))


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _side(stream, device) -> torch.cuda.Stream:
    """A given stream as torch's object (whose wrapper of a raw handle takes 0 for "a new one", not
    for the default stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A new tensor that a call writes on `stream` (None: the current one). Memory of the current
    stream's pool may still be in use by work queued there when another stream writes it, so on
    another stream it comes from that stream's own; the current stream, which may read it later,
    is noted for the allocator."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if _stream(stream) == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_side(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def wgrad_step(X: torch.Tensor, dY: torch.Tensor, W: torch.Tensor, m: Optional[torch.Tensor],
               v: Optional[torch.Tensor], opt: str = "adamw", hyper=None, step: int = 1, seed: int = 0,
               m_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, stream=None,
               x_scale: Optional[torch.Tensor] = None, dy_scale: Optional[torch.Tensor] = None,
               code: str = "linear") -> None:
    """Fused dW = dY^T X + optimizer step; W, m, v (and scales) updated in place.

    FP8 inputs (X float8_e4m3fn, dY float8_e4m3fn or float8_e5m2) carry their
    dequantisation scales as one-element float32 device tensors x_scale, dy_scale.
    int8 / uint8 moments hold linear codes, or the dynamic 8-bit code with code="dynamic".
    """
    h = _hyper(opt, hyper)
    st = _lib.forge_linear_wgrad_step(_ref(describe(X, x_scale)), _ref(describe(dY, dy_scale)), _ref(describe(W)),
                                      _ref(describe(m, m_scale, code=code)), _ref(describe(v, v_scale, code=code)),
                                      OPT_ID[opt],
                                      ctypes.byref(h), int(step), seed & (2 ** 64 - 1), _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_wgrad_step")


MAX_GROUP = 4


def wgrad_step_group(X: torch.Tensor, dYs, Ws, ms, vs, opt: str = "adamw", hyper=None, step: int = 1, seeds=(0,),
                     m_scales=None, v_scales=None, stream=None, code: str = "linear",
                     x_scale: Optional[torch.Tensor] = None, dy_scales=None) -> None:
    """Fused steps of the layers that share the input X, in one launch (forge_linear_wgrad_step_group):
    layer l has gradient dYs[l], weights Ws[l], moments ms[l] / vs[l] (lists; None entries, or
    None for the whole list, where the optimizer keeps no such slot) and seed seeds[l]. FP8
    inputs as in wgrad_step: x_scale for X, dy_scales[l] for dYs[l]."""
    n = len(Ws)
    if not (len(dYs) == n and len(seeds) == n) or n < 1 or n > MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} layers, each with its dY, W and seed")

    def arr(ts, scales=None):
        if ts is None or all(t is None for t in ts):
            return None
        if any(t is None for t in ts):
            raise ValueError("a moment slot is given for some layers of the group and not others")
        sc = scales if scales is not None else [None] * n
        return (ForgeTensor * n)(*[describe(t, s, code=code) for t, s in zip(ts, sc)])

    h = _hyper(opt, hyper)
    dy_a, w_a = arr(dYs, dy_scales), arr(Ws)
    m_a, v_a = arr(ms, m_scales), arr(vs, v_scales)
    seeds_a = (ctypes.c_uint64 * n)(*[s & (2 ** 64 - 1) for s in seeds])
    st = _lib.forge_linear_wgrad_step_group(_ref(describe(X, x_scale)), n, dy_a, w_a, m_a, v_a, OPT_ID[opt],
                                            ctypes.byref(h),
                                            int(step), seeds_a, _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_wgrad_step_group")


def dgrad(dY: torch.Tensor, W: torch.Tensor, dX: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX = dY W (from the weights as they are now, i.e. before the step)."""
    if dX is None:
        dX = _empty((dY.shape[0], W.shape[1]), W.dtype, W.device, stream)
    st = _lib.forge_linear_dgrad(_ref(describe(dY)), _ref(describe(W)), _ref(describe(dX)), _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_dgrad")
    return dX


def wgrad(X: torch.Tensor, dY: torch.Tensor, dW: Optional[torch.Tensor] = None, stream=None,
          x_scale: Optional[torch.Tensor] = None, dy_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Unfused baseline part 1: float32 dW = dY^T X written to device memory (FP8 inputs as in wgrad_step)."""
    if dW is None:
        dW = _empty((dY.shape[1], X.shape[1]), torch.float32, X.device, stream)
    if dW.dtype != torch.float32 or dW.dim() != 2 or (dW.shape[1] > 1 and dW.stride(1) != 1) or not dW.is_cuda:
        raise ValueError("dW must be a row-major float32 device tensor")
    st = _lib.forge_linear_wgrad(_ref(describe(X, x_scale)), _ref(describe(dY, dy_scale)), dW.data_ptr(),
                                 dW.stride(0), _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_wgrad")
    return dW


def optimizer_step(dW: torch.Tensor, W: torch.Tensor, m: Optional[torch.Tensor], v: Optional[torch.Tensor],
                   opt: str = "adamw", hyper=None, step: int = 1, seed: int = 0,
                   m_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   stream=None, code: str = "linear") -> None:
    """Unfused baseline part 2: element-wise optimizer pass reading the stored dW."""
    if dW.dtype != torch.float32 or not dW.is_cuda or (dW.shape[1] > 1 and dW.stride(1) != 1):
        raise ValueError("dW must be a row-major float32 device tensor")
    h = _hyper(opt, hyper)
    st = _lib.forge_optimizer_step(dW.data_ptr(), dW.stride(0), _ref(describe(W)),
                                   _ref(describe(m, m_scale, code=code)), _ref(describe(v, v_scale, code=code)),
                                   OPT_ID[opt], ctypes.byref(h), int(step),
                                   seed & (2 ** 64 - 1), _stream(stream))
    if st:
        raise ForgeError(st, "forge_optimizer_step")


def _workspace(ws: Optional[torch.Tensor], W: torch.Tensor, stream=None) -> torch.Tensor:
    if ws is None:
        ws = _empty(tuple(W.shape), torch.float32, W.device, stream)
    if ws.dtype != torch.float32 or ws.dim() != 2 or (ws.shape[1] > 1 and ws.stride(1) != 1) or not ws.is_cuda:
        raise ValueError("dW_workspace must be a row-major float32 device tensor")
    return ws


def wgrad_unfused(X, dY, W, m, v, opt="adamw", hyper=None, step=1, seed=0, m_scale=None, v_scale=None,
                  dW_workspace: Optional[torch.Tensor] = None, stream=None, x_scale=None,
                  dy_scale=None, code: str = "linear") -> torch.Tensor:
    """The two-phase baseline in one call (forge_linear_wgrad_unfused): float32 dW into the
    workspace (allocated here if not given), then a separate optimizer pass. Returns dW."""
    ws = _workspace(dW_workspace, W, stream)
    h = _hyper(opt, hyper)
    st = _lib.forge_linear_wgrad_unfused(_ref(describe(X, x_scale)), _ref(describe(dY, dy_scale)), _ref(describe(W)),
                                         _ref(describe(m, m_scale, code=code)), _ref(describe(v, v_scale, code=code)),
                                         OPT_ID[opt], ctypes.byref(h), int(step), seed & (2 ** 64 - 1),
                                         ws.data_ptr() if ws.numel() else None, ws.stride(0), _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_wgrad_unfused")
    return ws


def wgrad_unfused_noalloc(X, dY, W, m, v, opt="adamw", hyper=None, step=1, seed=0, m_scale=None, v_scale=None,
                          stream=None, x_scale=None, dy_scale=None, code: str = "linear") -> None:
    """The two-phase baseline with dW in the library's static per-GPU scratch
    (forge_linear_wgrad_unfused_noalloc): allocates nothing; out*in <= 2^24."""
    h = _hyper(opt, hyper)
    st = _lib.forge_linear_wgrad_unfused_noalloc(_ref(describe(X, x_scale)), _ref(describe(dY, dy_scale)),
                                                 _ref(describe(W)), _ref(describe(m, m_scale, code=code)),
                                                 _ref(describe(v, v_scale, code=code)), OPT_ID[opt], ctypes.byref(h),
                                                 int(step), seed & (2 ** 64 - 1), _stream(stream))
    if st:
        raise ForgeError(st, "forge_linear_wgrad_unfused_noalloc")


def new_states(W: torch.Tensor, opt: str = "adamw", fmt: str = "f32"):
    """Zero moment slots for `opt` in format f32, bf16, q8 (linear codes) or q8dyn (dynamic
    codes; pass code="dynamic" to the step): returns (m, v, m_scale, v_scale), the moments of W's shape (a layer's
    [out, in], a stack's [experts, out, in])."""
    if W.dim() not in (2, 3):
        raise ValueError(f"weights [out, in] or a stack [experts, out, in] wanted, not a tensor of shape {tuple(W.shape)}")
    use_m, use_v = SLOTS[opt]
    m = v = ms = vs = None
    if fmt not in ("f32", "bf16", "q8", "q8dyn"):
        raise ValueError(fmt)
    q8 = fmt in ("q8", "q8dyn")

    def zeros(dtype, shape):
        return torch.zeros(shape, dtype=dtype, device=W.device)

    blocks = (*W.shape[:-1], W.shape[-1] // 64)
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float32
    if use_m:
        m, ms = zeros(torch.int8 if q8 else dtype, W.shape), zeros(torch.float32, blocks) if q8 else None
    if use_v:
        v, vs = zeros(torch.uint8 if q8 else dtype, W.shape), zeros(torch.float32, blocks) if q8 else None
    return m, v, ms, vs


# ---------------------------------------------------------------------------
# operators around the fused step
# ---------------------------------------------------------------------------
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
ACT_ID = {name: k for k, name in enumerate(ACTS)}


def _act(act: str) -> int:
    if act not in ACT_ID:
        raise ValueError(f"unknown activation {act!r}; one of {', '.join(ACTS)}")
    return ACT_ID[act]


class _On:
    """The device and stream of a call: every tensor on one device, which is made current for
    the call; the work goes to `stream`, or to that device's current stream. Work queued on another
    stream before the call is the caller's to wait for, as with any kernel on a given stream;
    the tensors' memory is safe without: what the call allocates comes from the pool of the stream
    that writes it, and the allocator hands out no tensor of the call again before that stream (for
    a new tensor: the current one too) is done with it."""

    __slots__ = ("device", "stream", "_given", "_guard", "_index", "_others", "_current")

    def __init__(self, stream, first, *others):
        self._index = index = first.get_device()
        for t in others:
            if t is not None and (t.get_device() != index or (index < 0 and t.device != first.device)):
                raise ValueError("the tensors of a call live on one device")
        self.device = first.device
        if self.device.type != "cuda":
            raise ValueError("forge kernels take device tensors")
        if stream is not None and isinstance(stream, torch.cuda.Stream) and stream.device != self.device:
            raise ValueError("the stream belongs to another device than the tensors")
        self._given = stream
        self._guard = self._current = None
        self._others = (first, *others) if stream is not None else None

    def __enter__(self):
        given = None if self._given is None else _stream(self._given)
        if given is not None and given != _raw_stream(self._index):
            # one switch of device and stream for all that the call allocates
            side, self._current = _side(self._given, self.device), torch.cuda.current_stream(self.device)
            for t in self._others:
                if t is not None:
                    t.record_stream(side)
            self._guard = torch.cuda.stream(side)
        elif _current_device() != self._index:
            self._guard = torch.cuda.device(self._index)
        if self._guard is not None:
            self._guard.__enter__()
        self.stream = _raw_stream(self._index) if given is None else given
        return self

    def __exit__(self, *exc):
        return self._guard.__exit__(*exc) if self._guard is not None else None

    def empty(self, shape, dtype) -> torch.Tensor:
        """A new tensor that this call writes."""
        t = torch.empty(*shape, dtype=dtype, device=self.device)  # (0.4 us less than with the shape as a tuple)
        if self._current is not None:
            t.record_stream(self._current)
        return t


_F32 = torch.float32


class _Here:
    """_On's common case, a call without a stream on tensors of the current device: nothing to switch, nothing to
    note; one object per device, which calls of all threads share."""

    __slots__ = ("device", "_index")

    def __init__(self, device):
        self.device, self._index = device, device.index

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return None

    @property
    def stream(self) -> int:
        return _raw_stream(self._index)

    def empty(self, shape, dtype) -> torch.Tensor:
        if _new is not None:
            return _new(self._index, dtype, *shape)
        return torch.empty(*shape, dtype=dtype, device=self.device)


_here: Dict[int, _Here] = {}


def _on(stream, first, *others):
    """The device and stream of a call: _On, or its common case at half the host's time"""
    index = first.get_device()
    if stream is not None or index < 0 or index != _current_device():
        return _On(stream, first, *others)
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("the tensors of a call live on one device")
    return _here.get(index) or _here_new(first)


def _at(stream, first, *others):
    """_on for the calls of forge_calls.cpp, which check the others' device themselves"""
    index = first.get_device()
    if stream is not None or index < 0 or index != _current_device():
        return _On(stream, first, *others)
    return _here.get(index) or _here_new(first)


def _here_new(first) -> _Here:
    return _here.setdefault(first.get_device(), _Here(first.device))


# torch.empty by a shorter way (0.9 us of the host's time against 1.25), where forge_calls is there
_new = None if isinstance(_calls, _NoCalls) else _calls.empty
# torch's own short ways to the device's current stream and to the current device: a few microseconds less per call than
# the public ones with the checks around them, which a tensor on the device makes needless (the public ones where a build
# of torch lacks them)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


def _ten(t: Optional[torch.Tensor]):
    """describe() for the operands of the calls below: 2-D, no scales, device checked by _On
    (an argument of pointer type takes the structure itself)."""
    if t is None:
        return None
    rows, cols = t.shape
    s0, s1 = t.stride()
    dt = _DT.get(t.dtype)
    if s1 == 1 and rows and cols and dt is not None:
        return ForgeTensor(t.data_ptr(), dt, 0, rows, cols, s0 if rows > 1 else cols)
    if dt is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if rows == 0 or cols == 0:
        return ForgeTensor(None, dt, 0, rows, cols, cols)
    if s1 != 1 and cols > 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    return ForgeTensor(t.data_ptr(), dt, 0, rows, cols, s0 if rows > 1 else cols)


def _same(on: "_On", out: Optional[torch.Tensor], shape, dtype) -> torch.Tensor:
    return on.empty(shape, dtype) if out is None else out


def _check(st: int, what: str) -> None:
    if st:
        raise ForgeError(st, what)


def _row(b: Optional[torch.Tensor]):
    """_ten() of a vector as one row"""
    if b is None:
        return None
    if b.dim() != 1 or not b.is_contiguous():
        raise ValueError("bias is a contiguous vector")
    dt, n = _DT.get(b.dtype), b.numel()
    if dt is None:
        raise ValueError(f"unsupported dtype {b.dtype}")
    return ForgeTensor(b.data_ptr() if n else None, dt, 0, 1, n, n)


def _vec(t: torch.Tensor, n: int, dtype: torch.dtype, what: str) -> torch.Tensor:
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous {dtype} values wanted")
    return t


def linear(X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, save: bool = False, out: Optional[torch.Tensor] = None,
           stream=None):
    """Y = act(X W^T + bias) + residual, one kernel (forge_linear_forward). X [T, in], W [out, in],
    both bfloat16 or both float32; bias [out] in that type or float32; residual [T, out];
    act one of ACTS. With save=True returns (Y, Z), Z = X W^T + bias, which
    linear_act_backward needs for an activation."""
    a = _act(act)
    with _on(stream, X, W, bias, residual, out) as on:
        Y = _same(on, out, (X.shape[0], W.shape[0]), W.dtype)
        Z = on.empty((X.shape[0], W.shape[0]), W.dtype) if save else None
        _check(_lib.forge_linear_forward(_ten(X), _ten(W), _row(bias), a,
                                         _ten(residual), _ten(Y), _ten(Z), on.stream),
               "forge_linear_forward")
    return (Y, Z) if save else Y


def linear_act_backward(dY: torch.Tensor, Z: Optional[torch.Tensor] = None, act: str = "none",
                        want_bias: bool = True, dZ: Optional[torch.Tensor] = None, stream=None):
    """Backward of linear's epilogue (forge_linear_act_backward): (dZ, dbias) with
    dZ = dY * act'(Z) and dbias its float32 sum over the tokens (None with want_bias=False).
    act="none": dZ is dY itself, or, with a tensor dZ given, a copy of it there."""
    a = _act(act)
    if act != "none" and Z is None:
        raise ValueError("the gradient through an activation needs Z")
    with _on(stream, dY, Z, dZ) as on:
        T, out = dY.shape
        if act == "none" and dZ is dY:
            dZ = None  # nothing to copy
        if dZ is not None or act != "none":
            dZ = _same(on, dZ, (T, out), dY.dtype)
        db = ws = None
        need = 0
        if want_bias:
            db = on.empty((out,), torch.float32)
            need = _lib.forge_linear_act_backward_workspace(T, out)
            if need:
                ws = on.empty((need,), torch.uint8)
        _check(_lib.forge_linear_act_backward(_ten(dY), _ten(Z), a, _ten(dZ),
                                              db.data_ptr() if db is not None and out else None,
                                              ws.data_ptr() if ws is not None else None, need, on.stream),
               "forge_linear_act_backward")
    return (dY if dZ is None else dZ), db


def gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu", save: bool = False,
          out: Optional[torch.Tensor] = None, stream=None):
    """H = act(X Wg^T) * (X Wu^T), one kernel (forge_gated_forward): X [T, in], Wg and Wu
    [hidden, in]. With save=True returns (H, G, U), the projections the backward pass reads."""
    a = _act(act)
    with _on(stream, X, Wg, Wu, out) as on:
        shape = (X.shape[0], Wg.shape[0])
        H = _same(on, out, shape, Wg.dtype)
        G, U = (on.empty(shape, Wg.dtype), on.empty(shape, Wg.dtype)) if save else (None, None)
        _check(_lib.forge_gated_forward(_ten(X), _ten(Wg), _ten(Wu), a,
                                        _ten(H), _ten(G), _ten(U), on.stream),
               "forge_gated_forward")
    return (H, G, U) if save else H


def gated_backward(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor, act: str = "silu", want_h: bool = True,
                   stream=None):
    """Backward of the gated product from dH: (dG, dU, H), dG = dH * U * act'(G),
    dU = dH * act(G), H = act(G) * U (None with want_h=False)."""
    a = _act(act)
    with _on(stream, dH, G, U) as on:
        dG, dU = on.empty(dH.shape, dH.dtype), on.empty(dH.shape, dH.dtype)
        H = on.empty(dH.shape, dH.dtype) if want_h else None
        _check(_lib.forge_gated_backward(_ten(dH), _ten(G), _ten(U), a,
                                         _ten(dG), _ten(dU), _ten(H), on.stream),
               "forge_gated_backward")
    return dG, dU, H


def gated_dgrad(dY: torch.Tensor, Wd: torch.Tensor, G: torch.Tensor, U: torch.Tensor, act: str = "silu",
                want_h: bool = True, stream=None):
    """gated_backward with dH = dY Wd (the linear layer behind the block, its weights as they
    are now) formed in registers and never stored (forge_gated_dgrad): (dG, dU, H)."""
    a = _act(act)
    with _on(stream, dY, Wd, G, U) as on:
        shape = (dY.shape[0], Wd.shape[1])
        dG, dU = on.empty(shape, Wd.dtype), on.empty(shape, Wd.dtype)
        H = on.empty(shape, Wd.dtype) if want_h else None
        _check(_lib.forge_gated_dgrad(_ten(dY), _ten(Wd), _ten(G), _ten(U), a,
                                      _ten(dG), _ten(dU), _ten(H), on.stream),
               "forge_gated_dgrad")
    return dG, dU, H


def dgrad_group(dYs, Ws, dX: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX = sum_l dYs[l] Ws[l] for layers that read the same input, in one accumulation
    (forge_linear_dgrad_group_split; from the weights as they are now)."""
    n = len(Ws)
    if len(dYs) != n or not 1 <= n <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} layers, each with its dY and W")
    with _on(stream, *dYs, *Ws, dX) as on:
        dX = _same(on, dX, (dYs[0].shape[0], Ws[0].shape[1]), Ws[0].dtype)
        dy_a = (ForgeTensor * n)(*[_ten(t) for t in dYs])
        w_a = (ForgeTensor * n)(*[_ten(t) for t in Ws])
        need = _lib.forge_linear_dgrad_group_workspace(*dX.shape, sum(w.shape[0] for w in Ws), _DT.get(dX.dtype, -1))
        ws = on.empty((need,), torch.uint8) if need else None
        _check(_lib.forge_linear_dgrad_group_split(n, dy_a, w_a, _ten(dX), _ptr(ws), need, on.stream),
               "forge_linear_dgrad_group_split")
    return dX


_REDUCTIONS = ("mean", "sum", "none")


def _reduction(reduction: str) -> str:
    if reduction not in _REDUCTIONS:
        raise ValueError(f"unknown reduction {reduction!r}; one of {', '.join(_REDUCTIONS)}")
    return reduction


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return t.data_ptr() if t is not None and t.numel() else None


def linear_cross_entropy(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean", stream=None):
    """Softmax cross entropy of the logits X W^T against `targets`, the logits never stored
    (forge_linear_xent_forward). X [T, in], W [vocab, in]; targets: T int64 in [0, vocab) or
    ignore_index (another value makes the loss NaN; rows of X whose target is ignored
    reach no other token, but dW takes 0 times them: they are finite). Returns (loss, lse, total): the loss by
    `reduction` ("mean" over the tokens that count, "sum", or "none": one per token, 0 where
    ignored), each token's log sum of exponentials, and total = (sum of the losses, tokens
    counted, mean); linear_cross_entropy_backward takes the last two."""
    _reduction(reduction)
    with _on(stream, X, W, targets) as on:
        T = X.shape[0]
        _vec(targets, T, torch.int64, "targets")
        loss = on.empty((T,), torch.float32) if reduction == "none" else None
        lse, total = on.empty((T,), torch.float32), on.empty((3,), torch.float32)
        need = _lib.forge_linear_xent_workspace(T, X.shape[1], W.shape[0], _DT.get(W.dtype, -1), 0, 0)
        ws = on.empty((need,), torch.uint8)
        _check(_lib.forge_linear_xent_forward(_ten(X), _ten(W), _ptr(targets), int(ignore_index),
                                              _ptr(loss), _ptr(lse), total.data_ptr(), _ptr(ws), need, on.stream),
               "forge_linear_xent_forward")
    return (loss if reduction == "none" else total[2 if reduction == "mean" else 0]), lse, total


def _xent_grad_args(on, X, W, targets, lse, dloss, reduction, total, piece):
    T = X.shape[0]
    _vec(targets, T, torch.int64, "targets")
    _vec(lse, T, torch.float32, "lse")
    _vec(dloss, T if reduction == "none" else 1, torch.float32, "dloss")
    if reduction == "mean":
        if total is None:
            raise ValueError("the gradient of a mean needs `total` of the forward pass")
        _vec(total, 3, torch.float32, "total")
    need = _lib.forge_linear_xent_workspace(T, X.shape[1], W.shape[0], _DT.get(W.dtype, -1), 1, int(piece))
    return need, on.empty((need,), torch.uint8), (total if reduction == "mean" else None)


def linear_cross_entropy_backward(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                                  dloss: torch.Tensor, ignore_index: int = -100, reduction: str = "mean",
                                  total: Optional[torch.Tensor] = None, want_dx: bool = True, want_dw: bool = True,
                                  piece: int = 0, stream=None):
    """Gradients of linear_cross_entropy (forge_linear_xent_backward): (dX, dW) in the operands'
    type, None where not wanted. dloss: float32 device scalar, or T values with
    reduction="none"; lse and total as linear_cross_entropy returned them. Works through the
    vocabulary `piece` entries at a time (0: the library's choice)."""
    _reduction(reduction)
    with _on(stream, X, W, targets, lse, dloss, total) as on:
        need, ws, tot = _xent_grad_args(on, X, W, targets, lse, dloss, reduction, total, piece)
        dX = on.empty(X.shape, X.dtype) if want_dx else None
        dW = on.empty(W.shape, W.dtype) if want_dw else None
        _check(_lib.forge_linear_xent_backward(_ten(X), _ten(W), _ptr(targets), int(ignore_index),
                                               _ptr(lse), _ptr(dloss), int(reduction == "none"), _ptr(tot),
                                               _ten(dX), _ten(dW), int(piece), _ptr(ws), need,
                                               on.stream), "forge_linear_xent_backward")
    return dX, dW


def linear_cross_entropy_step(X: torch.Tensor, W: torch.Tensor, m: Optional[torch.Tensor], v: Optional[torch.Tensor],
                              targets: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, opt: str = "adamw",
                              hyper=None, step: int = 1, seed: int = 0, m_scale: Optional[torch.Tensor] = None,
                              v_scale: Optional[torch.Tensor] = None, code: str = "linear", ignore_index: int = -100,
                              reduction: str = "mean", total: Optional[torch.Tensor] = None, want_dx: bool = True,
                              piece: int = 0, stream=None) -> Optional[torch.Tensor]:
    """linear_cross_entropy_backward with the head's fused optimizer step in the place of dW
    (forge_linear_xent_step): W, m, v (and scales) updated in place piece by piece; returns
    dX (from the old W) or None. Optimizer arguments as in wgrad_step; W, m and v of less than
    2^31 bytes each."""
    _reduction(reduction)
    h = _hyper(opt, hyper)
    with _on(stream, X, W, m, v, targets, lse, dloss, m_scale, v_scale, total) as on:
        need, ws, tot = _xent_grad_args(on, X, W, targets, lse, dloss, reduction, total, piece)
        dX = on.empty(X.shape, X.dtype) if want_dx else None
        _check(_lib.forge_linear_xent_step(_ten(X), _ten(W), _ref(describe(m, m_scale, code=code)),
                                           _ref(describe(v, v_scale, code=code)), OPT_ID[opt], ctypes.byref(h),
                                           int(step), seed & (2 ** 64 - 1), _ptr(targets), int(ignore_index),
                                           _ptr(lse), _ptr(dloss), int(reduction == "none"), _ptr(tot),
                                           _ten(dX), int(piece), _ptr(ws), need, on.stream),
               "forge_linear_xent_step")
    return dX


# ---------------------------------------------------------------------------
# layers of experts
# ---------------------------------------------------------------------------
MAX_EXPERTS = 1024


def _stack(W: Optional[torch.Tensor]):
    """_ten() of stacked matrices [experts, out, in] as one tensor of experts * out rows"""
    if W is None:
        return None
    if W.dim() != 3:
        raise ValueError("stacked matrices [experts, out, in] wanted")
    e, rows, cols = W.shape
    dt = _DT.get(W.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {W.dtype}")
    if W.numel() == 0:
        return ForgeTensor(None, dt, 0, e * rows, cols, cols)
    s0, s1, s2 = W.stride()
    if s2 != 1 and cols > 1:
        raise ValueError("rows must be contiguous (stride(2) == 1)")
    ld = s1 if rows > 1 else (s0 if e > 1 else cols)
    if e > 1 and s0 != rows * ld:
        raise ValueError("the rows of a stack follow one another in one pitch (stride(0) == out * stride(1))")
    return ForgeTensor(W.data_ptr(), dt, 0, e * rows, cols, ld)


def _experts(W: torch.Tensor, offsets: torch.Tensor, *others) -> int:
    e = W.shape[0]
    if W.dim() != 3:
        raise ValueError("stacked matrices [experts, out, in] wanted")
    for w in others:
        if w.dim() != 3 or w.shape[0] != e:
            raise ValueError("stacked matrices [experts, out, in] of the same experts wanted")
    _vec(offsets, e + 1, torch.int64, "offsets")
    return e


def _places(pos: torch.Tensor) -> int:
    if pos.dim() != 2 or pos.dtype != torch.int32 or not pos.is_contiguous():
        raise ValueError("pos: a contiguous [T, k] int32 tensor, as expert_plan returned it, wanted")
    if pos.shape[1] < 1:
        raise ValueError("a token has one route at least")
    return pos.shape[1]


def _factors(weights: Optional[torch.Tensor], pos: torch.Tensor) -> None:
    if weights is not None and (weights.shape != pos.shape or weights.dtype != torch.float32 or not weights.is_contiguous()):
        raise ValueError("weights: a contiguous float32 tensor of pos's shape wanted")


def expert_plan(idx: torch.Tensor, experts: int, stream=None):
    """The routes of a router ordered by expert (forge_expert_plan): idx [T, k] int64, the experts of each
    token; a value outside [0, experts) drops the route. Returns (offsets, pos): expert x owns rows
    offsets[x] .. offsets[x + 1] - 1 (int64, experts + 1 of them), pos [T, k] int32 is each route's row, -1
    for a dropped one. Routes of an expert keep the tokens' order. Both stay on the device: no call waits for them."""
    if idx.dim() != 2 or idx.dtype != torch.int64 or not idx.is_contiguous():
        raise ValueError("idx: a contiguous [T, k] int64 tensor wanted")
    if idx.shape[1] < 1:
        raise ValueError("a token has one route at least")
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"1..{MAX_EXPERTS} experts")
    with _at(stream, idx) as on:
        T, k = idx.shape
        offsets, pos = on.empty((experts + 1,), torch.int64), on.empty((T, k), torch.int32)
        need = _calls.forge_expert_plan_workspace(T, k, experts)
        ws = on.empty((need,), torch.uint8) if need else None
        _calls.forge_expert_plan(idx, T, k, experts, offsets, pos, ws, need, on.stream)
    return offsets, pos


def expert_dispatch(X: torch.Tensor, pos: torch.Tensor, scale: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream=None):
    """Rows to their experts, Xp[pos[t, j]] = X[t] (forge_expert_dispatch): X [T, cols] float32, bfloat16, or
    int8 with its rows' factors `scale` (T float32), which go along: returns Xp [T * k, cols], with them
    (Xp, factors). Rows that no route has (those of dropped ones, at the end) are not written. Its gradient is
    expert_combine(dXp, pos)."""
    k = _places(pos)
    if (X.dtype == torch.int8) != (scale is not None):
        raise ValueError("int8 rows come with their factors, others without")
    with _at(stream, X, pos, scale, out) as on:
        if X.shape[0] != pos.shape[0]:
            raise ValueError("pos has the routes of another number of tokens")
        Xp = _same(on, out, (pos.numel(), X.shape[1]), X.dtype)
        if scale is None:
            _calls.forge_expert_dispatch(X, pos, k, Xp, on.stream)
            return Xp
        sp = on.empty((Xp.shape[0],), _F32)
        _calls.forge_expert_dispatch((X, scale), pos, k, (Xp, sp), on.stream)
        return Xp, sp


def expert_combine(Yp: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """The experts' results back to their tokens, Y[t] = sum_j weights[t, j] Yp[pos[t, j]] + residual[t], dropped
    routes left out (forge_expert_combine); weights float32 or None for ones. Y is of Yp's type, or bfloat16 of
    float32 Yp with out_dtype=torch.bfloat16 (or a residual or out of that type)."""
    k = _places(pos)
    _factors(weights, pos)
    with _at(stream, Yp, pos, weights, residual, out) as on:
        Y = _same(on, out, (pos.shape[0], Yp.shape[1]), out_dtype or (Yp if residual is None else residual).dtype)
        if Y.shape[0] != pos.shape[0]:
            raise ValueError("pos has the routes of another number of tokens")
        _calls.forge_expert_combine(Yp, pos, k, weights, residual, Y, on.stream)
    return Y


def expert_combine_backward(dY: torch.Tensor, Yp: Optional[torch.Tensor], pos: torch.Tensor,
                            weights: Optional[torch.Tensor] = None, want_dweights: bool = True, stream=None):
    """Backward of expert_combine (forge_expert_combine_backward): (dYp, dweights), dYp[pos[t, j]] = weights[t, j]
    dY[t] (rows that no route has are not written), dweights[t, j] = <dY[t], Yp[pos[t, j]]> in float32 (0 for a
    dropped route; None with want_dweights=False, where Yp may be None)."""
    k = _places(pos)
    _factors(weights, pos)
    if want_dweights and Yp is None:
        raise ValueError("the weights' gradient needs Yp")
    with _at(stream, dY, Yp, pos, weights) as on:
        if dY.shape[0] != pos.shape[0]:
            raise ValueError("pos has the routes of another number of tokens")
        rows = pos.numel() if Yp is None else Yp.shape[0]
        dYp = on.empty((rows, dY.shape[1]), dY.dtype)
        dw = on.empty(pos.shape, torch.float32) if want_dweights else None
        _calls.forge_expert_combine_backward(dY, Yp if want_dweights else None, pos, k, weights, dYp, dw, on.stream)
    return dYp, dw


def expert_linear(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, act: str = "none", save: bool = False,
                  out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None):
    """Y[r] = act(X[r] W[x]^T) for the rows r of each expert x (forge_expert_linear): X [R, in] in expert_plan's
    order, W [experts, out, in], offsets as expert_plan returned them. Rows behind offsets[-1] are
    neither read nor written. With save=True returns (Y, Z), Z the pre-activation. out_dtype=torch.float32 of bfloat16
    operands, without an activation: the sums unrounded, for expert_combine."""
    a = _act(act)
    with _at(stream, X, W, offsets, out) as on:
        e = _experts(W, offsets)
        shape = (X.shape[0], W.shape[1])
        Y = _same(on, out, shape, out_dtype or W.dtype)
        Z = on.empty(shape, W.dtype) if save else None
        _calls.forge_expert_linear(X, W, e, offsets, a, Y, Z, on.stream)
    return (Y, Z) if save else Y


def expert_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, offsets: torch.Tensor, act: str = "silu",
                 save: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """gated() with each row's expert's matrices (forge_expert_gated): Wg, Wu [experts, hidden, in], rows and
    offsets as in expert_linear. With save=True returns (H, G, U)."""
    a = _act(act)
    with _at(stream, X, Wg, Wu, offsets, out) as on:
        e = _experts(Wg, offsets, Wu)
        shape = (X.shape[0], Wg.shape[1])
        H = _same(on, out, shape, Wg.dtype)
        G, U = (on.empty(shape, Wg.dtype), on.empty(shape, Wg.dtype)) if save else (None, None)
        _calls.forge_expert_gated(X, Wg, Wu, e, offsets, a, H, G, U, on.stream)
    return (H, G, U) if save else H


def expert_gated_dgrad(dY: torch.Tensor, Wd: torch.Tensor, G: torch.Tensor, U: torch.Tensor, offsets: torch.Tensor,
                       act: str = "silu", want_h: bool = True, stream=None):
    """gated_dgrad() with each row's expert's matrix (forge_expert_gated_dgrad): Wd [experts, out, hidden];
    (dG, dU, H)."""
    a = _act(act)
    with _at(stream, dY, Wd, G, U, offsets) as on:
        e = _experts(Wd, offsets)
        shape = (dY.shape[0], Wd.shape[2])
        dG, dU = on.empty(shape, Wd.dtype), on.empty(shape, Wd.dtype)
        H = on.empty(shape, Wd.dtype) if want_h else None
        _calls.forge_expert_gated_dgrad(dY, Wd, G, U, e, offsets, a, dG, dU, H, on.stream)
    return dG, dU, H


def expert_dgrad_group(dYs, Ws, offsets: torch.Tensor, dX: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX[r] = sum_l dYs[l][r] Ws[l][x] for the rows r of each expert x (forge_expert_dgrad_group_split): Ws[l]
    [experts, out_l, in]; from the weights as they are now, before their step."""
    n = len(Ws)
    if len(dYs) != n or not 1 <= n <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} layers, each with its dY and W")
    with _at(stream, *dYs, *Ws, offsets, dX) as on:
        e = _experts(Ws[0], offsets, *Ws[1:])
        dX = _same(on, dX, (dYs[0].shape[0], Ws[0].shape[2]), Ws[0].dtype)
        need = _calls.forge_expert_dgrad_group_workspace(*dX.shape, sum([w.shape[1] for w in Ws]), e, _DT.get(dX.dtype, -1))
        ws = on.empty((need,), torch.uint8) if need else None
        _calls.forge_expert_dgrad_group_split(n, list(dYs), list(Ws), e, offsets, dX, ws, need, on.stream)
    return dX


def expert_wgrad(X: torch.Tensor, dY: torch.Tensor, offsets: torch.Tensor, dW: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """The stack's gradient dW[x] = dY^T X over each expert's rows, float32 [experts, out, in]
    (forge_expert_wgrad): the two-phase schedule's first half (optimizer_step on the stack as one
    [experts * out, in] layer is its second)."""
    with _at(stream, X, dY, offsets, dW) as on:
        e = offsets.numel() - 1
        _vec(offsets, e + 1, torch.int64, "offsets")
        shape, ld = (e, dY.shape[1], X.shape[1]), X.shape[1]
        if dW is None:
            dW = on.empty(shape, _F32)
        elif dW.dtype is not _F32 or tuple(dW.shape) != shape:
            raise ValueError("dW: float32 [experts, out, in] wanted")
        else:
            ld = _stack(dW).ld
        _calls.forge_expert_wgrad(X, dY, e, offsets, dW, ld, on.stream)
    return dW


def expert_wgrad_step(X: torch.Tensor, dY: torch.Tensor, W: torch.Tensor, m: Optional[torch.Tensor],
                      v: Optional[torch.Tensor], offsets: torch.Tensor, opt: str = "adamw", hyper=None, step: int = 1,
                      seed: int = 0, m_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                      code: str = "linear", stream=None) -> None:
    """wgrad_step() of every expert of a stack in one launch (forge_expert_wgrad_step): X [R, in], dY [R, out] in
    expert_plan's order, W [experts, out, in]; m and v of W's shape, block scales
    [experts, out, in / 64], as new_states(W) makes them. The step is that of the stack as one [experts * out, in] layer:
    same element indices and random streams. Experts without rows step on a gradient of zero."""
    h = _hyper(opt, hyper)
    with _on(stream, X, dY, W, m, v, offsets, m_scale, v_scale) as on:
        e = _experts(W, offsets)

        def state(t, scale):
            if t is None:
                return None
            if tuple(t.shape) != tuple(W.shape):
                raise ValueError("moments have the weights' shape")
            d = _stack(t)
            if scale is not None:
                if scale.dtype != torch.float32 or not scale.is_contiguous() or \
                        tuple(scale.shape) != (e, W.shape[1], W.shape[2] // 64):
                    raise ValueError("block scale shape must be [experts, out, in / 64]")
                d.scale = _ptr(scale)
            if code not in ("linear", "dynamic"):
                raise ValueError(f"unknown moment code {code!r}")
            if code == "dynamic" and d.dtype in (I8, U8):
                d.dtype = I8_DYN if d.dtype == I8 else U8_DYN
            return _ref(d)

        _check(_lib.forge_expert_wgrad_step(_ten(X), _ten(dY), _stack(W), state(m, m_scale), state(v, v_scale), e,
                                            offsets.data_ptr(), OPT_ID[opt], ctypes.byref(h), int(step),
                                            seed & (2 ** 64 - 1), on.stream), "forge_expert_wgrad_step")


# ---------------------------------------------------------------------------
# products of 8-bit integers
# ---------------------------------------------------------------------------
def quantize_rows(X: torch.Tensor, stream=None):
    """Rows to 8 bits (forge_quantize_rows): X [rows, cols] float32 or bfloat16, cols a multiple of 16; returns (Q, scale),
    int8 codes and one float32 factor per row, scale = max |x| / 127 and Q = x / scale to the nearest. A
    row of zeros has scale 0; one with an infinity or NaN has scale NaN, and so NaN for its products. Weights
    are quantised the same way, one factor per output channel: a stack [experts, out, in] as its rows
    W.reshape(-1, in)."""
    with _at(stream, X) as on:
        shape = X.shape
        Q, scale = on.empty(shape, torch.int8), on.empty((shape[0],), _F32)
        _calls.forge_quantize_rows(X, (Q, scale), on.stream)
    return Q, scale


def linear_q8(X: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, act: str = "none", residual: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear() of 8-bit integers (forge_linear_q8): X [T, in] and W [out, in] int8 with a factor for each row (token,
    output channel), as quantize_rows makes them; the sums are exact, the epilogue float32, Y bfloat16."""
    a = _act(act)
    with _at(stream, X, x_scale, W, w_scale, bias, residual, out) as on:
        Y = _same(on, out, (X.shape[0], W.shape[0]), torch.bfloat16)
        _calls.forge_linear_q8((X, x_scale), (W, w_scale), bias, a, residual, Y, on.stream)
    return Y


def gated_q8(X: torch.Tensor, x_scale: torch.Tensor, Wg: torch.Tensor, wg_scale: torch.Tensor, Wu: torch.Tensor,
             wu_scale: torch.Tensor, act: str = "silu", out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """gated() of 8-bit integers (forge_gated_q8), operands as in linear_q8; H bfloat16."""
    a = _act(act)
    with _at(stream, X, x_scale, Wg, wg_scale, Wu, wu_scale, out) as on:
        H = _same(on, out, (X.shape[0], Wg.shape[0]), torch.bfloat16)
        _calls.forge_gated_q8((X, x_scale), (Wg, wg_scale), (Wu, wu_scale), a, H, on.stream)
    return H


def expert_linear_q8(X: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
                     offsets: torch.Tensor, act: str = "none", out: Optional[torch.Tensor] = None,
                     out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """expert_linear() of 8-bit integers (forge_expert_linear_q8): W [experts, out, in] int8 with experts * out
    factors, X and its factors as expert_dispatch(Q, pos, scale) returned them; Y bfloat16, or float32 without an
    activation, for expert_combine."""
    a = _act(act)
    with _at(stream, X, x_scale, W, w_scale, offsets, out) as on:
        e = _experts(W, offsets)
        Y = _same(on, out, (X.shape[0], W.shape[1]), out_dtype)
        _calls.forge_expert_linear_q8((X, x_scale), (W, w_scale), e, offsets, a, Y, on.stream)
    return Y


def expert_gated_q8(X: torch.Tensor, x_scale: torch.Tensor, Wg: torch.Tensor, wg_scale: torch.Tensor, Wu: torch.Tensor,
                    wu_scale: torch.Tensor, offsets: torch.Tensor, act: str = "silu", out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """expert_gated() of 8-bit integers (forge_expert_gated_q8), operands as in expert_linear_q8; H bfloat16."""
    a = _act(act)
    with _at(stream, X, x_scale, Wg, wg_scale, Wu, wu_scale, offsets, out) as on:
        e = _experts(Wg, offsets, Wu)
        H = _same(on, out, (X.shape[0], Wg.shape[1]), torch.bfloat16)
        _calls.forge_expert_gated_q8((X, x_scale), (Wg, wg_scale), (Wu, wu_scale), e, offsets, a, H, on.stream)
    return H
